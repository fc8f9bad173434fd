"""8-bit activation checkpoints against float64.

Saving and loading are exact: bytes and values are compared for equality.  Tolerances of the
rest, derived before the first run:
  gated activation   expf is within 2 units of 2^-23, then 1 + e, its reciprocal and two or three products
                     at 2^-24 each: GATED = 7e-7 of the formula's terms (for dgate, whose terms
                     may cancel, of the sum of their magnitudes); half a step, 2^-8, more in
                     bf16.  Below gate = -128 ln 2 = -88.7228 e^-gate is infinite and the
                     sigmoid, 2^-128 and less, 0; as |gate| e^gate falls there, FLOOR is 88.7228
                     2^-128 = 2.6073e-37 of the other factors, and TINY a subnormal's step
  weight gradient    products are exact in fp32; an accumulation of 16 of them rounds by 2^-23 of the
                     sum of magnitudes at most: (T / 16 + 4) 2^-23 sum |dy| |x|, three times
                     as many for fp32 gradients, which go through as three bf16 parts, and
                     2^-24 sum |dy| |x| for what the parts leave; half a step, 2^-8, in bf16
"""
import numpy as np
import pytest

from gpu_util import nsm
from oracle import checkpoint

pytestmark = pytest.mark.gpu
GATED, FLOOR, TINY = 7e-7, 2.61e-37, 2.0 ** -149
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}


@pytest.fixture(scope="module")
def m():
    return nsm()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _matrix(rng, rows, cols, dtype="float32", pad=0, lead=0, scale=1.0, wide=True):
    """(matrix on the device inside memory that holds 300, its float64 values)"""
    import torch
    x = rng.normal(0, scale, (rows, cols))
    if wide:
        x *= np.exp(rng.normal(0, 1.5, (1, cols)))
    buffer = torch.full((lead + rows * (cols + pad) + 8,), 300.0, device="cuda").to(getattr(torch, dtype))
    t = buffer[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.from_numpy(x.astype(np.float32)).cuda())
    return t, _f64(t)


def _encoded(ck):
    """(q, b) as the device holds them."""
    data = ck.data.cpu().numpy()
    blocks = -(-ck.cols // 32)
    q = data[:ck.rows * blocks * 32].view(np.int8).reshape(ck.rows, -1)
    return q, data[ck.rows * blocks * 32:].reshape(ck.rows, blocks)


SHAPES = [(1, 1, 0, 0), (3, 31, 0, 1), (5, 32, 0, 0), (7, 33, 3, 0), (131, 1000, 0, 0), (64, 1003, 5, 3), (2, 40000, 0, 0),
          (1025, 96, 8, 0), (4099, 17, 0, 0), (333, 9728, 64, 8)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES)
def test_save_and_load(m, rows, cols, pad, lead, dtype):
    import torch
    rng = np.random.default_rng([rows, cols])
    x, v = _matrix(rng, rows, cols, dtype, pad, lead)
    ck = m.muon_checkpoint_save(x)
    q, b = checkpoint.encode(v)
    got_q, got_b = _encoded(ck)
    assert (got_b == b).all() and (got_q == q).all()
    want = checkpoint.decode(q, b, cols)
    for out in ("bfloat16", "float32"):
        y, _ = _matrix(rng, rows, cols, out, pad, lead)
        assert m.muon_checkpoint_load(ck, out=y) is y
        assert (_f64(y) == want).all()
        base = y._base if y._base is not None else y
        if pad or lead:  # the memory around the rows is as it was
            flat = base.reshape(-1)
            keep = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
            idx = lead + torch.arange(rows, device="cuda")[:, None] * (cols + pad) + torch.arange(cols, device="cuda")
            keep[idx.reshape(-1)] = False
            assert (flat[keep] == 300).all()
    assert torch.equal(m.muon_checkpoint_load(ck), m.muon_checkpoint_load(ck, dtype=torch.float32).bfloat16())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_special_values(m, dtype):
    import torch
    rng = np.random.default_rng(1)
    x, _ = _matrix(rng, 12, 64, dtype)
    t = x.dtype
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 63] = float("inf")
    x[3, 0] = -float("inf")
    x[4, 7] = torch.finfo(t).max
    x[5, 7] = -torch.finfo(t).max
    x[6] = torch.finfo(t).tiny
    x[7] = 0
    x[7, 3] = torch.finfo(t).tiny / 2   # a subnormal
    x[8, :32] = 0
    x[8, 0] = 127.5
    x[9, :32] = torch.arange(32, device="cuda", dtype=t) * 0.5
    x[9, 0] = 127.0
    x[10] = -0.0
    x[11, :32] = 2.0 ** 127
    v = _f64(x)
    got = _f64(m.muon_checkpoint_load(m.muon_checkpoint_save(x)))
    want = checkpoint.values(v)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isnan(got[1, :32]).all() and not np.isnan(got[1, 32:]).any() and np.isnan(got[2, 32:]).all()


def test_past_2_31_elements(m):
    import torch
    rows, cols = 70001, 32768
    x = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    at = torch.arange(rows, device="cuda") * 7919 % cols
    x.scatter_(1, at[:, None], 3.0)
    ck = m.muon_checkpoint_save(x)
    x.fill_(5.0)
    m.muon_checkpoint_load(ck, out=x)
    assert (x.gather(1, at[:, None]) == 3).all() and x[-100:].float().sum() == 300 and x[:100].float().sum() == 300
    assert (x.float().sum(1) == 3).all()


def test_nothing(m):
    import torch
    x = torch.zeros(0, 40, device="cuda")
    ck = m.muon_checkpoint_save(x)
    assert m.muon_checkpoint_load(ck).shape == (0, 40)
    h, g, u = m.muon_swiglu_forward(x, x)
    dg, du, again = m.muon_swiglu_backward(x, g, u, with_h=True)
    assert h.shape == dg.shape == du.shape == again.shape == (0, 40)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES)
def test_gated(m, rows, cols, pad, lead, dtype):
    rng = np.random.default_rng([rows, cols, 1])
    gate, vg = _matrix(rng, rows, cols, dtype, pad, lead, 2.0)
    up, vu = _matrix(rng, rows, cols, dtype, 0, lead)
    h, cg, cu = m.muon_swiglu_forward(gate, up)
    for ck, v in ((cg, vg), (cu, vu)):
        q, b = _encoded(ck)
        wq, wb = checkpoint.encode(v)
        assert (q == wq).all() and (b == wb).all()
    tol = GATED + (HALF[dtype] if dtype == "bfloat16" else 0)
    want = checkpoint.swiglu(vg, vu)
    assert (np.abs(_f64(h) - want) <= tol * np.abs(want) + FLOOR * np.abs(vu) + TINY).all()
    dh, vd = _matrix(rng, rows, cols, dtype, pad, 0, 0.1, False)
    g, u = checkpoint.values(vg), checkpoint.values(vu)
    dgate, dup, again = m.muon_swiglu_backward(dh, cg, cu, with_h=True)
    wg, wu = checkpoint.swiglu_backward(vd, g, u)
    s = checkpoint.sigmoid(g)
    terms = np.abs(vd * u) * s * (1 + np.abs(g) * (1 - s))
    half = HALF[dtype] if dtype == "bfloat16" else 0
    assert (np.abs(_f64(dgate) - wg) <= 2 * GATED * terms + half * np.abs(wg) + 2 * FLOOR * np.abs(vd * u) + TINY).all()
    assert (np.abs(_f64(dup) - wu) <= tol * np.abs(wu) + FLOOR * np.abs(vd) + TINY).all()
    want = checkpoint.swiglu(g, u)
    assert (np.abs(_f64(again) - want) <= tol * np.abs(want) + FLOOR * np.abs(u) + TINY).all()
    dgate2, dup2, none = m.muon_swiglu_backward(dh, cg, cu)
    assert none is None and (dgate2 == dgate).all() and (dup2 == dup).all()


def test_gated_extremes(m):
    """Gates at which the exponential leaves fp32's range, and what is not finite."""
    import torch
    gate = torch.tensor([[-200.0, 200.0, -90.0, 90.0, 0.0, -1.2784645] + [1.0] * 26, [float("nan")] + [1.0] * 31],
                        device="cuda")
    up = torch.full_like(gate, 2.0)
    h, cg, cu = m.muon_swiglu_forward(gate, up)
    assert h[0, :5].tolist()[1] == 400 and abs(h[0, 0]) < 1e-30 and h[0, 4] == 0 and h[1, 0].isnan()
    assert not h[1, 1:].isnan().any()
    dg, du, _ = m.muon_swiglu_backward(torch.ones_like(gate), cg, cu)
    assert not dg[0].isnan().any() and not du[0].isnan().any() and dg[0, 1] == 2 and abs(dg[0, 0]) < 1e-30
    assert dg[1].isnan().all() and du[1].isnan().all()   # the block is not a number


def test_gated_halves_in_place_and_graph(m):
    import torch
    rng = np.random.default_rng(4)
    both, v = _matrix(rng, 50, 208, "bfloat16")
    gate, up = both[:, :104], both[:, 104:]
    h, cg, cu = m.muon_swiglu_forward(gate, up)
    alone = m.muon_swiglu_forward(gate.contiguous(), up.contiguous())
    assert torch.equal(h, alone[0]) and torch.equal(cg.data, alone[1].data) and torch.equal(cu.data, alone[2].data)
    over = both.clone()
    m.muon_swiglu_forward(over[:, :104], over[:, 104:], h=over[:, :104])
    assert torch.equal(over[:, :104], h) and torch.equal(over[:, 104:], up)
    dh = torch.randn(50, 104, device="cuda").bfloat16()
    grads = torch.empty_like(both)
    dg, du, again = m.muon_swiglu_backward(dh, cg, cu, dgate=grads[:, :104], dup=grads[:, 104:], with_h=True)
    for k in range(3):   # each output in the place of dh
        mine = dh.clone()
        out = [None, None, torch.empty_like(dh)]
        out[k] = mine
        got = m.muon_swiglu_backward(mine, cg, cu, dgate=out[0], dup=out[1], h=out[2])
        assert torch.equal(got[0], dg) and torch.equal(got[1], du) and torch.equal(got[2], again)
    graph = torch.cuda.CUDAGraph()
    held = dh.clone()
    with torch.cuda.graph(graph):
        hh, g2, u2 = m.muon_swiglu_forward(gate, up)
        got = m.muon_swiglu_backward(held, g2, u2, with_h=True)
    graph.replay()
    assert torch.equal(hh, h) and all(torch.equal(a, b) for a, b in zip(got, (dg, du, again)))
    both.mul_(0.5)
    graph.replay()
    fresh = m.muon_swiglu_forward(gate, up)
    assert torch.equal(hh, fresh[0])


def test_streams(m):
    import torch
    x = torch.randn(1000, 1000, device="cuda")
    want = m.muon_checkpoint_load(m.muon_checkpoint_save(x))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    ck = m.muon_checkpoint_save(x, stream=stream)
    got = m.muon_checkpoint_load(ck, stream=stream.cuda_stream)
    stream.synchronize()
    assert torch.equal(got, want)


def _check_weight(got, dy, x, steps, parts, dtype, base=None):
    """|error| <= (steps + 4) 2^-23 sum |dy| |x| (parts times), the type's rounding, and the sum with dw's values."""
    want = dy.T @ x
    terms = np.abs(dy).T @ np.abs(x)
    if base is not None:
        want = want + base
        terms = terms + np.abs(base)
    tol = (parts * steps + 4) * 2.0 ** -23 * terms + HALF[dtype] * np.abs(want) + TINY
    err = np.abs(_f64(got) - want)
    assert (err <= tol).all(), (err - tol).max()


GRADS = [(1, 1, 1, 0, 0), (1, 300, 40, 0, 0), (5, 40, 300, 0, 0), (63, 129, 65, 0, 0), (64, 256, 256, 0, 0), (65, 257, 255, 3, 1),
         (200, 8, 1000, 8, 8), (1000, 512, 128, 0, 0), (1024, 8, 8, 0, 0), (777, 300, 700, 5, 0), (300, 2000, 1537, 0, 2),
         (4099, 264, 33, 0, 0), (130, 5000, 4999, 0, 0)]


@pytest.mark.parametrize("dtype,out", [("bfloat16", "float32"), ("bfloat16", "bfloat16"), ("float32", "float32")])
@pytest.mark.parametrize("rows,outs,cols,pad,lead", GRADS)
def test_weight_grad(m, rows, outs, cols, pad, lead, dtype, out):
    import torch
    rng = np.random.default_rng([rows, outs, cols])
    x, v = _matrix(rng, rows, cols)
    dy, vd = _matrix(rng, rows, outs, dtype, pad, lead, 0.1)
    ck = m.muon_checkpoint_save(x)
    saved = checkpoint.values(v)
    steps, parts = -(-rows // 16), 3 if dtype == "float32" else 1
    dw, base = _matrix(rng, outs, cols, out, pad, lead)
    got = m.muon_checkpoint_weight_grad(ck, dy, out=dw)
    assert got is dw
    _check_weight(dw, vd, saved, steps, parts, out)
    flat = (dw._base if dw._base is not None else dw).reshape(-1)   # the memory around the rows is as it was
    assert (flat[:lead] == 300).all() and (flat[lead + outs * (cols + pad):] == 300).all()
    if pad:
        assert (flat[lead:lead + outs * (cols + pad)].view(outs, cols + pad)[:, cols:] == 300).all()
    dw2, base = _matrix(rng, outs, cols, out, pad, lead)
    m.muon_checkpoint_weight_grad(ck, dy, out=dw2, accumulate=True)
    _check_weight(dw2, vd, saved, steps, parts, out, base)
    again = m.muon_checkpoint_weight_grad(ck, dy, dtype=getattr(torch, out))
    assert torch.equal(again, dw)


def test_weight_grad_every_tile(m):
    """More tiles than pairs of SMs, and sums divided among pairs."""
    for rows, outs, cols in ((40, 2600, 5200), (5000, 600, 600)):
        rng = np.random.default_rng(rows)
        x, v = _matrix(rng, rows, cols, "bfloat16")
        dy, vd = _matrix(rng, rows, outs, "bfloat16")
        ck = m.muon_checkpoint_save(x)
        import torch
        got = m.muon_checkpoint_weight_grad(ck, dy, dtype=torch.float32)
        _check_weight(got, vd, checkpoint.values(v), -(-rows // 16), 1, "float32")


def test_weight_grad_fp32_keeps_all_bits(m):
    """One token: each element is a product of an fp32 and a bf16 number, whose sum of three parts rounds twice."""
    import torch
    rng = np.random.default_rng(6)
    x, v = _matrix(rng, 1, 64)
    dy, vd = _matrix(rng, 1, 100, scale=1e3)
    dy[0, 0] = torch.finfo(torch.float32).max
    dy[0, 1] = -torch.finfo(torch.float32).max
    x[0, :32] = 0.5
    vd, v = _f64(dy), _f64(x)
    got = _f64(m.muon_checkpoint_weight_grad(m.muon_checkpoint_save(x), dy))
    want = vd.T @ checkpoint.values(v)
    fits = np.abs(want) < 3e38
    assert (np.abs(got - want)[fits] <= 3 * 2.0 ** -24 * np.abs(want)[fits]).all()


def test_weight_grad_sums_do_not_drift(m):
    """The tensor cores cut off what a sum cannot hold, less than a unit, 2^-23 of the sum so far, for each
    accumulation of 16 tokens.  An accumulator takes 64 of them, so that terms of one sign lose less
    than sum_{k <= 64} k / 64 2^-23 = 3.9e-6 of the whole, and what adds the accumulators up rounds to
    nearest; one accumulator over all 512 could lose eight times as much.  (80 tiles: the tokens of
    none of them are divided.)"""
    import torch
    gen = torch.Generator("cuda").manual_seed(10)
    x = torch.rand(8192, 2048, generator=gen, device="cuda") + 0.5
    x *= (0.5 * torch.randn(8192, 1, generator=gen, device="cuda")).exp()
    dy = torch.randn(8192, 2560, generator=gen, device="cuda").exp().bfloat16()
    ck = m.muon_checkpoint_save(x)
    got = m.muon_checkpoint_weight_grad(ck, dy, dtype=torch.float32).double()
    want = dy.double().t() @ m.muon_checkpoint_load(ck).double()
    assert ((got - want) / want).mean().abs() <= 3.9e-6


def test_weight_grad_small_fp32_gradients(m):
    """Below 2^-110 an fp32 number has bits under 2^-133, the smallest bf16 number: the third part is cut there."""
    import torch
    rng = np.random.default_rng(11)
    x, v = _matrix(rng, 300, 64)
    x.mul_(2.0 ** 60)
    dy, vd = _matrix(rng, 300, 50)
    dy.mul_(2.0 ** -112)
    dy[:, 25:] *= 2.0 ** -12
    vd, v = _f64(dy), checkpoint.values(_f64(x))
    got = _f64(m.muon_checkpoint_weight_grad(m.muon_checkpoint_save(x), dy))
    terms = np.abs(vd).T @ np.abs(v)
    tol = (3 * -(-300 // 16) + 4) * 2.0 ** -23 * terms + 2.0 ** -133 * np.abs(v).sum(0)
    assert (np.abs(got - vd.T @ v) <= tol).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_weight_grad_not_finite(m, dtype):
    import torch
    rng = np.random.default_rng(7)
    x, v = _matrix(rng, 100, 96, dtype)
    dy, vd = _matrix(rng, 100, 40, dtype)
    x[70, 40] = float("inf")
    dy[99, 3] = float("nan")
    dy[98, 5] = float("inf")
    got = m.muon_checkpoint_weight_grad(m.muon_checkpoint_save(x), dy, dtype=torch.float32)
    assert got[:, 32:64].isnan().all() and got[3].isnan().all()
    assert not got[5, :32].isfinite().any()
    keep = [i for i in range(40) if i not in (3, 5)]
    assert got[keep][:, :32].isfinite().all() and got[keep][:, 64:].isfinite().all()


def test_weight_grad_of_no_tokens(m):
    import torch
    ck = m.muon_checkpoint_save(torch.zeros(0, 37, device="cuda"))
    dy = torch.zeros(0, 11, device="cuda", dtype=torch.bfloat16)
    assert (m.muon_checkpoint_weight_grad(ck, dy, dtype=torch.float32) == 0).all()
    dw = torch.full((11, 37), 5.0, device="cuda")
    m.muon_checkpoint_weight_grad(ck, dy, out=dw, accumulate=True)
    assert (dw == 5).all()


def test_weight_grad_graph_and_streams(m):
    """Two captured graphs, an eager call and another stream, none of which share a workspace."""
    import torch
    rng = np.random.default_rng(8)
    sets = []
    for k in range(2):
        x, _ = _matrix(rng, 900, 300)
        dy, _ = _matrix(rng, 900, 200)
        sets.append((m.muon_checkpoint_save(x), dy))
    want = [m.muon_checkpoint_weight_grad(*s) for s in sets]
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.muon_checkpoint_weight_grad(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = m.muon_checkpoint_weight_grad(*sets[0])
        side = m.muon_checkpoint_weight_grad(*sets[1], stream=streams[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs + [eager, side], want + want))


def test_layer_backward_matches_autograd(m):
    """A gated layer's weight gradients through the checkpoints, clipped and stepped on, against
    float64 gradients of the same layer on the saved values."""
    import torch
    gen = torch.Generator("cuda").manual_seed(9)
    T, inputs, hidden = 500, 96, 160
    x = torch.randn(T, inputs, generator=gen, device="cuda").bfloat16()
    weights = [torch.randn(hidden, inputs, generator=gen, device="cuda") * 0.1 for _ in range(2)]
    weights.append(torch.randn(inputs, hidden, generator=gen, device="cuda") * 0.1)
    gate, up = (x @ w.bfloat16().t() for w in weights[:2])
    saved_x = m.muon_checkpoint_save(x)
    h, cg, cu = m.muon_swiglu_forward(gate, up)
    dy = torch.randn(T, inputs, generator=gen, device="cuda").bfloat16()
    dh = dy @ weights[2].bfloat16()
    dgate, dup, again = m.muon_swiglu_backward(dh, cg, cu, with_h=True)
    saved_h = m.muon_checkpoint_save(again)
    grads = [m.muon_checkpoint_weight_grad(saved_x, dgate, dtype=torch.float32),
             m.muon_checkpoint_weight_grad(saved_x, dup, dtype=torch.float32),
             m.muon_checkpoint_weight_grad(saved_h, dy, dtype=torch.float32)]
    # in 64 bits: autograd through the activation on the loaded values, products by torch
    lx, lh = m.muon_checkpoint_load(saved_x).double(), m.muon_checkpoint_load(saved_h).double()
    g, u = (m.muon_checkpoint_load(c).double().requires_grad_() for c in (cg, cu))
    (torch.nn.functional.silu(g) * u).backward(dh.double())
    for got, d, v, exact in zip(grads, (dgate, dup, dy), (lx, lx, lh), (g.grad, u.grad, dy.double())):
        assert (d.double() - exact).abs().max() <= 2.0 ** -7 * exact.abs().max()
        _check_weight(got, _f64(d), v.detach().cpu().numpy(), -(-T // 16), 1, "float32")
    norm = m.muon_clip_grad_norm(grads, 1.0)
    total = sum((t.double() ** 2).sum() for t in grads).sqrt()
    assert abs(total.item() - 1) < 1e-4 and norm[0] > 1
    plan = m.muon_plan([tuple(w.shape) for w in weights], config=m.muon_config_default(grad_dtype=m.MUON_DTYPE_F32))
    m.allocate_workspace(plan)
    before = [w.clone() for w in weights]
    m.muon_step(plan, weights, grads, [torch.zeros_like(w) for w in weights], 0.02, 0.9, True, 0.0)
    status, nonfinite = m.muon_sync(plan)
    assert status == m.MUON_OK and nonfinite == 0
    assert all((a - b).abs().max() > 0 for a, b in zip(before, weights))


def test_two_threads_on_one_stream(m):
    """Each thread has a workspace of its own."""
    import threading

    import torch
    rng = np.random.default_rng(21)
    sets = []
    for k in range(2):
        x, _ = _matrix(rng, 700, 130)
        dy, _ = _matrix(rng, 700, 90)
        sets.append((m.muon_checkpoint_save(x), dy))
    want = [m.muon_checkpoint_weight_grad(*s) for s in sets]
    torch.cuda.synchronize()
    got, stream = [[], []], torch.cuda.current_stream()

    def work(k):
        for _ in range(20):
            got[k].append(m.muon_checkpoint_weight_grad(*sets[k], stream=stream))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(len(g) == 20 and torch.equal(t, want[k]) for k, g in enumerate(got) for t in g)


def test_large_workspaces_are_not_held(m):
    """What a call over many tokens needs beside its operands is free again after it, on every stream."""
    import threading

    import torch
    x = torch.randn(16384, 2048, device="cuda").bfloat16()
    dy = torch.randn(16384, 64, device="cuda").bfloat16()
    ck, out = m.muon_checkpoint_save(x), torch.empty(2, 64, 2048, device="cuda")
    assert m.muon_weight_grad_workspace_bytes(ck, dy) >= x.numel() * 2
    torch.cuda.synchronize()
    grown, side = [], torch.cuda.Stream()

    def work():   # a thread has its workspaces to itself
        for k, stream in enumerate((None, side)):
            before = torch.cuda.memory_allocated()
            for _ in range(3):
                m.muon_checkpoint_weight_grad(ck, dy, out=out[k], stream=stream)
            grown.append(torch.cuda.memory_allocated() - before)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert len(grown) == 2 and max(grown) < x.numel() * 2
    assert torch.equal(out[0], out[1])
    steps = 16384 // 16
    _check_weight(out[0], _f64(dy), _f64(m.muon_checkpoint_load(ck)), steps, 1, "float32")


def test_refusals(m):
    import torch
    x = torch.randn(10, 70, device="cuda")
    ck = m.muon_checkpoint_save(x)
    other = m.muon_checkpoint_save(x[:9])
    dy = torch.randn(10, 30, device="cuda")
    with pytest.raises(TypeError):
        m.muon_checkpoint_save(x.half())
    with pytest.raises(ValueError):
        m.muon_checkpoint_save(x, checkpoint=other)
    with pytest.raises(ValueError):
        m.muon_checkpoint_save(x.t())
    with pytest.raises(ValueError):
        m.muon_checkpoint_load(ck, out=torch.empty(10, 71, device="cuda"))
    with pytest.raises(TypeError):
        m.muon_checkpoint_load(ck, dtype=torch.float16)
    with pytest.raises(ValueError):
        m.muon_checkpoint_load(ck, out=x, dtype=torch.bfloat16)
    with pytest.raises(m.MuonError):
        m.muon_checkpoint_load(m.Checkpoint(1, 5, torch.zeros(41, dtype=torch.uint8, device="cuda")[8:]))   # off its boundary
    for bad in (dict(dy=dy[:9]), dict(dy=dy.cpu()), dict(out=torch.empty(30, 71, device="cuda")),
                dict(out=torch.empty(70, 30, device="cuda").t()), dict(accumulate=True),
                dict(out=torch.empty(30, 70, device="cuda"), dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            m.muon_checkpoint_weight_grad(**{"checkpoint": ck, "dy": dy, **bad})
    with pytest.raises(TypeError):
        m.muon_checkpoint_weight_grad(ck, dy.half())
    with pytest.raises(m.MuonError) as e:
        m.muon_checkpoint_weight_grad(ck, dy, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == m.MUON_ERR_NO_WORKSPACE
    with pytest.raises(ValueError):
        m.muon_swiglu_forward(x, x.bfloat16())
    with pytest.raises(ValueError):
        m.muon_swiglu_forward(x, x[:9])
    with pytest.raises(m.MuonError):
        m.muon_swiglu_forward(x, x, gate_checkpoint=ck, up_checkpoint=ck)
    with pytest.raises(ValueError):
        m.muon_swiglu_backward(x, ck, other)
    out = torch.empty_like(x)
    with pytest.raises(m.MuonError):
        m.muon_swiglu_backward(x, ck, m.muon_checkpoint_save(x), dgate=out, dup=out)


def test_rows_written_again(m):
    """A checkpoint, a gradient and a workspace used again hold nothing of what was there."""
    import torch
    x = torch.full((64, 64), float("inf"), device="cuda")
    ck = m.muon_checkpoint_save(x)
    dy = torch.ones(64, 64, device="cuda")
    space = torch.full((m.muon_weight_grad_workspace_bytes(ck, dy),), 255, dtype=torch.uint8, device="cuda")
    dw = m.muon_checkpoint_weight_grad(ck, dy, workspace=space)
    assert dw.isnan().all()
    m.muon_checkpoint_save(torch.ones_like(x), checkpoint=ck)
    m.muon_checkpoint_weight_grad(ck, dy, out=dw, workspace=space)
    assert (dw == 64).all()
