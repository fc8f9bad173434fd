"""Global gradient norm and clipping against the fp64 oracle.

Tolerances.  The norm: a lane sums at most 2 x 33 squares one after the other in fp32
before the sum is carried with its error, so the sum of squares is within 66 units of
2^-24, the root within half of that and one rounding: 2.1e-6 at the very worst;
NORM_TOL is 2.5e-6.  The factor divides by the norm and is rounded once: 2.6e-6.
The elements: one rounding of the product with the returned factor, checked bit for bit.
"""
import math

import numpy as np
import pytest

from gpu_util import nsm
from oracle import losses

pytestmark = pytest.mark.gpu
NORM_TOL = 2.5e-6


@pytest.fixture(scope="module")
def m():
    return nsm()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _flat_views(torch, sizes, dtype, gen, lead=0, scale=1e-2):
    """Consecutive views of one buffer, the first `lead` elements after its start."""
    flat = torch.randn(lead + sum(sizes) + 3, generator=gen, device="cuda").mul_(scale).to(dtype)
    at, got = lead, []
    for n in sizes:
        got.append(flat[at:at + n])
        at += n
    return flat, got


def _expected(torch, g, c, dtype):
    return (g.float() * c).to(dtype)


def _check(torch, m, grads, max_norm, out=None, eps=1e-6):
    before = [g.clone() for g in grads]
    norm = losses.grad_norm([_f64(g) for g in grads])
    result = m.muon_clip_grad_norm(grads, max_norm, out=out, eps=eps)
    got = result.cpu().numpy()
    assert got[0] == pytest.approx(norm, rel=NORM_TOL, abs=0)
    assert got[1] == pytest.approx(losses.clip_factor(norm, max_norm, eps), rel=2.6e-6, abs=0)
    for b, o in zip(before, out if out is not None else grads):
        assert torch.equal(o, _expected(torch, b, result[1], o.dtype))
    return got


SIZES = [[], [0], [1], [7], [8], [9], [255], [2047], [2048], [2049], [4096, 0, 3], [1, 1, 1, 5, 2056, 17],
         [131072], [100003, 64, 1]]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lead", [0, 1, 5])
def test_in_place(m, sizes, dtype, lead):
    import torch
    gen = torch.Generator("cuda").manual_seed(len(sizes) + lead)
    flat, grads = _flat_views(torch, sizes, getattr(torch, dtype), gen, lead)
    ends = flat[:lead].clone(), flat[lead + sum(sizes):].clone()
    _check(torch, m, grads, 0.05)
    # nothing outside the tensors is touched
    assert torch.equal(flat[:lead], ends[0]) and torch.equal(flat[lead + sum(sizes):], ends[1])


@pytest.mark.parametrize("sizes", [[9], [2049, 7], [4096, 0, 3], [100003, 64, 1]], ids=str)
@pytest.mark.parametrize("src", ["float32", "bfloat16"])
@pytest.mark.parametrize("dst", ["float32", "bfloat16"])
@pytest.mark.parametrize("leads", [(0, 0), (3, 3), (0, 1), (2, 5)])
@pytest.mark.parametrize("max_norm", [0.05, 1e9])
def test_into_other_buffers(m, sizes, src, dst, leads, max_norm):
    import torch
    gen = torch.Generator("cuda").manual_seed(3)
    _, grads = _flat_views(torch, sizes, getattr(torch, src), gen, leads[0])
    flat, out = _flat_views(torch, sizes, getattr(torch, dst), gen, leads[1])
    ends = flat[:leads[1]].clone(), flat[leads[1] + sum(sizes):].clone()
    keep = [g.clone() for g in grads]
    _check(torch, m, grads, max_norm, out)
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))
    assert torch.equal(flat[:leads[1]], ends[0]) and torch.equal(flat[leads[1] + sum(sizes):], ends[1])


@pytest.mark.parametrize("n", [64, 65, 640, 641, 1500])
def test_many_tensors(m, n):
    import torch
    gen = torch.Generator("cuda").manual_seed(n)
    sizes = np.random.default_rng(n).integers(0, 3000, n).tolist()
    _, a = _flat_views(torch, sizes[::2], torch.float32, gen)
    _, b = _flat_views(torch, sizes[1::2], torch.bfloat16, gen, 1)
    mixed = [t for pair in zip(a, b) for t in pair] + a[len(b):]
    _check(torch, m, mixed, 0.3)


def test_layer_and_norm_call(m):
    import torch
    gen = torch.Generator("cuda").manual_seed(9)
    shapes = [(4096, 2560), (1024, 2560), (1024, 2560), (2560, 4096), (9728, 2560)]
    grads = [torch.randn(s, generator=gen, device="cuda").mul_(1e-3).bfloat16() for s in shapes]
    got = _check(torch, m, grads, 1.0, [torch.empty(s, device="cuda") for s in shapes])
    norm = m.muon_grad_norm(grads)
    assert norm.item() == got[0]            # one sum, one order


def test_strided_and_permuted_layouts(m):
    import torch
    gen = torch.Generator("cuda").manual_seed(5)
    base = torch.randn(6, 48, 130, generator=gen, device="cuda").bfloat16()
    keep = base.clone()
    views = [base[:, 8:20], base[:, 20:].permute(1, 0, 2)[5:9]]
    norm = losses.grad_norm([_f64(v) for v in views])
    result = m.muon_clip_grad_norm(views, 1.0)
    assert result[0].item() == pytest.approx(norm, rel=NORM_TOL)
    want = keep.clone()
    for v in (want[:, 8:20], want[:, 20:].permute(1, 0, 2)[5:9]):
        v.copy_(_expected(torch, v, result[1], torch.bfloat16))
    assert torch.equal(base, want)
    one = torch.randn(12, 7, generator=gen, device="cuda").t()
    _check(torch, m, [one], 0.1, [torch.empty(12, 7, device="cuda").t()])


def test_output_layouts_beside_a_strided_gradient(m):
    import torch
    # what counts as an output's layout does not depend on the set's other tensors
    flat = torch.randn(6, device="cuda")
    wide = torch.randn(4, 5, device="cuda")
    whole = torch.empty(2, 3, device="cuda")
    out = torch.empty(4, 5, device="cuda")[:, :3]
    result = m.muon_clip_grad_norm([flat, wide[:, :3]], 0.5, out=[whole, out])
    factor = result[1].item()
    assert torch.equal(whole.flatten(), flat * factor) and torch.equal(out, wide[:, :3] * factor)
    one = torch.empty(1, 7, 5, device="cuda").as_strided((1, 7, 3), (99, 5, 1))   # a stride that nothing uses
    src = torch.randn(1, 7, 5, device="cuda")[:, :, :3]
    factor = m.muon_clip_grad_norm([src], 0.5, out=[one])[1].item()
    assert torch.equal(one, src * factor)
    for wrong in (torch.empty(4, 6, device="cuda")[:, :3], torch.empty(4, 3, device="cuda"), torch.empty(6, 5, device="cuda")[:, :2]):
        with pytest.raises(ValueError, match="layout"):
            m.muon_clip_grad_norm([wide[:, :3]], 0.5, out=[wrong])


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e-17, 1e15, 1e19, 1e25, 1e33])
@pytest.mark.parametrize("n", [5, 70001])
def test_full_range(m, scale, n):
    import torch
    gen = torch.Generator("cuda").manual_seed(1)
    g = torch.randn(n, generator=gen, device="cuda") * scale
    assert m.muon_grad_norm([g]).item() == pytest.approx(losses.grad_norm([_f64(g)]), rel=NORM_TOL, abs=0)
    # a small set beside a large one, and zeros beside both
    h = torch.zeros(5000, device="cuda")
    h[17] = 1.0
    assert m.muon_grad_norm([g, h]).item() == pytest.approx(losses.grad_norm([_f64(g), _f64(h)]), rel=NORM_TOL)


def test_largest_and_smallest_numbers(m):
    import torch
    for x in (3.0e38, 1.4e-45, -1.4e-45, 1.2e-38):
        g = torch.zeros(4099, device="cuda")
        g[4098] = x
        assert m.muon_grad_norm([g]).item() == float(np.float32(abs(x)))
    g = torch.full((4096,), 2.0e38, device="cuda")
    assert m.muon_grad_norm([g]).item() == math.inf       # above fp32: reported as such
    r = m.muon_clip_grad_norm([g], 1.0)                    # and still clipped: 2e38 * 64 is finite in 64 bits
    assert r[1].item() == pytest.approx(1 / (2.0e38 * 64), rel=1e-5)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [0, 2047, 5000])
def test_nonfinite(m, bad, at):
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        g = torch.ones(5001, device="cuda", dtype=dtype)
        h = torch.full((300,), 2.0, device="cuda", dtype=dtype)
        g[at] = bad
        keep = g.clone()
        r = m.muon_clip_grad_norm([g, h], 1.0, nonfinite=m.MUON_NONFINITE_KEEP)
        assert not math.isfinite(r[0].item()) and r[1].item() == 1.0
        assert torch.equal(g.nan_to_num(7.0), keep.nan_to_num(7.0)) and (h == 2).all()
        r = m.muon_clip_grad_norm([g, h], 1.0, nonfinite=m.MUON_NONFINITE_ZERO)
        assert r[1].item() == 0.0 and (g == 0).all() and (h == 0).all()


def test_limits(m):
    import torch
    for max_norm, c in ((0.0, 0.0), (math.inf, 1.0), (5.0, 1.0), (4.0, 0.8)):
        g = torch.tensor([3.0, 0.0, 4.0], device="cuda")
        r = m.muon_clip_grad_norm([g], max_norm, eps=0.0)
        assert r.tolist() == pytest.approx([5.0, c], rel=1e-7)
        assert g.tolist() == pytest.approx([3 * c, 0, 4 * c], rel=1e-6)
    z = torch.zeros(10, device="cuda")
    assert m.muon_clip_grad_norm([z], 0.0, eps=0.0).tolist() == [0.0, 1.0]
    assert m.muon_clip_grad_norm([], 1.0).tolist() == [0.0, 1.0]


def test_same_bits_each_time_and_on_another_stream(m):
    import torch
    gen = torch.Generator("cuda").manual_seed(8)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in (300001, 17, 65536)]
    keys = m.GradSet(grads)
    first = m.muon_grad_norm(keys)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    seen = [m.muon_grad_norm(keys, stream=side) for _ in range(20)]
    seen += [m.muon_grad_norm(keys, stream=side.cuda_stream) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, s) for s in seen)


def test_graph_capture(m):
    import torch
    gen = torch.Generator("cuda").manual_seed(4)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in (70000, 31)]
    out = [torch.empty_like(g) for g in grads]
    keys = m.GradSet(grads, out)
    ws = torch.empty(m.muon_clip_workspace_bytes(keys), dtype=torch.uint8, device="cuda")
    result = torch.empty(2, device="cuda")
    m.muon_clip_grad_norm(keys, 1.0, result=result, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        m.muon_clip_grad_norm(keys, 1.0, result=result, workspace=ws, stream=side)
    for scale in (2.0, 0.5):
        [g.mul_(scale) for g in grads]
        graph.replay()
        torch.cuda.synchronize()
        norm = losses.grad_norm([_f64(g) for g in grads])
        assert result[0].item() == pytest.approx(norm, rel=NORM_TOL)
        assert all(torch.equal(o, g * result[1]) for g, o in zip(grads, out))


def test_refusals(m):
    import torch
    g = torch.zeros(8, device="cuda")
    for bad in ([g.half()], [g.cpu()], [g.expand(3, 8)], [g.long()]):
        with pytest.raises((TypeError, ValueError)):
            m.muon_grad_norm(bad)
    with pytest.raises(ValueError):
        m.muon_clip_grad_norm([g], 1.0, out=[g[:4]])
    with pytest.raises(ValueError):
        m.muon_clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(ValueError):
        m.muon_clip_grad_norm(m.GradSet([g]), 1.0, out=[g])
    with pytest.raises(ValueError):
        m.muon_clip_grad_norm([g], 1.0, result=torch.zeros(3, device="cuda"))
    for kw in (dict(max_norm=-1.0), dict(max_norm=1.0, eps=-1.0), dict(max_norm=1.0, nonfinite=5)):
        with pytest.raises(m.MuonError) as e:
            m.muon_clip_grad_norm([g], **kw)
        assert e.value.status == m.MUON_ERR_INVALID
    with pytest.raises(m.MuonError) as e:
        m.muon_grad_norm([g], workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == m.MUON_ERR_NO_WORKSPACE
    assert m.muon_grad_norm([g]).item() == 0.0             # and the library still works


def test_clipped_gradients_step(m):
    """Gradients clipped by the library, then stepped on: the step's input norms are scaled."""
    import torch
    gen = torch.Generator("cuda").manual_seed(6)
    w = [torch.randn(256, 512, generator=gen, device="cuda"), torch.randn(384, 192, generator=gen, device="cuda")]
    grads = [torch.randn_like(x) for x in w]
    plan = m.muon_plan([tuple(x.shape) for x in w], config=m.muon_config_default(grad_dtype=m.MUON_DTYPE_F32))
    m.allocate_workspace(plan)
    r = m.muon_clip_grad_norm(grads, 1.0)
    m.muon_step(plan, w, grads, [torch.zeros_like(x) for x in w], 0.02, 0.0, False, 0.0)
    assert m.muon_sync(plan)[0] == m.MUON_OK
    norms = m.muon_get_input_norms(plan)
    assert math.hypot(*norms) == pytest.approx(1.0, rel=1e-5)
    assert r[1].item() == pytest.approx(1.0 / (r[0].item() + 1e-6), rel=1e-6)
