"""The losses' row kernels over many rows: every launch shape, rows enough that each
cluster's ring of row scalars is refilled several times, masks in blocks.

The reference is torch in float64 on the GPU, row by row chunks, from the formulas; the
tolerances are those of test_gpu_losses.py (its derivation holds for any row here: at most
1100 terms are added one after the other).
"""
import math

import pytest

from gpu_util import nsm

pytestmark = pytest.mark.gpu
LP_ABS, LP_REL = 1e-5, 4e-7


@pytest.fixture(scope="module")
def m():
    return nsm()


def _inputs(n, v, dtype, mask, pad=0, seed=0):
    import torch
    gen = torch.Generator("cuda").manual_seed(seed)
    full = torch.randn(n, v + pad, generator=gen, device="cuda").mul_(2.5).to(getattr(torch, dtype))
    z = full[:, :v]
    y = torch.randint(0, v, (n,), generator=gen, device="cuda")
    z.scatter_(1, y[:, None], (6 + 3 * torch.randn(n, 1, generator=gen, device="cuda")).to(z.dtype))
    t = torch.arange(n, device="cuda")
    live = {"none": None, "all": t >= 0, "blocks": (t // 37) % 3 != 0, "front": t < n // 2, "back": t >= n - 5,
            "random": torch.rand(n, generator=gen, device="cuda") < 0.7}[mask]
    return z, y, live, gen


def _reference(z, y, live, temperature):
    """(logp, softmax chunk function) in float64."""
    import torch
    n, v = z.shape
    logp = torch.zeros(n, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 25) // v)
    for a in range(0, n, step):
        x = z[a:a + step].double() / temperature
        logp[a:a + step] = x.gather(1, y[a:a + step, None])[:, 0] - torch.logsumexp(x, 1)
    return logp if live is None else torch.where(live, logp, torch.zeros_like(logp))


def _check_grad(z, y, live, temperature, grad, slope, scale):
    import torch
    n, v = z.shape
    step = max(1, (1 << 24) // v)
    eps = 2.0 ** -8 if z.dtype == torch.bfloat16 else 0.0
    for a in range(0, n, step):
        p = torch.softmax(z[a:a + step].double() / temperature, 1)
        k = torch.arange(p.shape[0], device="cuda")
        want = -p
        want[k, y[a:a + step]] += 1
        want *= (slope[a:a + step] / temperature)[:, None]
        p[k, y[a:a + step]] += 1
        bound = 4e-5 * scale[a:a + step, None] / temperature * p + eps * want.abs() + 1e-37
        if live is not None:
            dead = ~live[a:a + step]
            want[dead] = 0
            bound[dead] = 0
        off = (grad[a:a + step].double() - want).abs() - bound
        assert (off <= 0).all(), (a, off.max().item())


# (rows, logits, type): a warp a row (4, 8 and 16 units a lane); one CTA with three rows,
# two and four CTAs, four with two rows, eight; and rows too long for them
SHAPES = [(20000, 1000, "bfloat16"), (9000, 1030, "float32"), (6000, 2047, "bfloat16"), (5000, 4096, "bfloat16"),
          (30000, 4105, "bfloat16"), (12000, 8200, "bfloat16"), (6001, 17001, "float32"), (5003, 40001, "bfloat16"),
          (2900, 76001, "bfloat16"), (2800, 100000, "bfloat16"), (2500, 131072, "bfloat16"), (700, 152064, "bfloat16"),
          (600, 230001, "bfloat16"), (400, 131072, "float32"), (40, 500003, "bfloat16"), (33, 250001, "float32")]


@pytest.mark.parametrize("n,v,dtype", SHAPES)
@pytest.mark.parametrize("mask", ["none", "blocks", "random"])
def test_policy_rows(m, n, v, dtype, mask):
    _policy(m, n, v, dtype, mask)


# one row's CTAs and the rows of their ring: 2/2, 8/2 with several CTAs an SM, 4/3, 8/3
MORE_SHAPES = [(3001, 20001, "bfloat16"), (2000, 54005, "bfloat16"), (3000, 45001, "bfloat16"), (2001, 90007, "bfloat16"),
               (1000, 200064, "bfloat16"), (900, 240001, "bfloat16"), (500, 320003, "bfloat16"),
               (3000, 11001, "float32"), (2500, 25003, "float32"), (1500, 50001, "float32"), (1000, 100001, "float32"),
               (700, 120003, "float32"), (500, 151936, "float32")]


@pytest.mark.parametrize("n,v,dtype", MORE_SHAPES)
@pytest.mark.parametrize("mask", ["all", "random"])
def test_policy_rows_of_more_launch_shapes(m, n, v, dtype, mask):
    _policy(m, n, v, dtype, mask, pad=1)


@pytest.mark.parametrize("n", [1, 2, 31, 152, 153, 600, 1217, 2431, 2433, 5000])
@pytest.mark.parametrize("mask", ["all", "front", "back", "blocks"])
@pytest.mark.parametrize("v,dtype", [(9001, "bfloat16"), (600, "float32"), (33003, "float32")])
def test_policy_row_counts(m, n, v, dtype, mask):
    _policy(m, n, v, dtype, mask, pad=3)


def _policy(m, n, v, dtype, mask, pad=0):
    import torch
    z, y, live, gen = _inputs(n, v, dtype, mask, pad, seed=n + v)
    temperature = 0.9
    logp = _reference(z, y, live, temperature)
    delta = 0.3 * torch.randn(n, generator=gen, device="cuda", dtype=torch.float64)
    for lim in (math.log(0.8), math.log(1.2)):
        delta = torch.where((delta - lim).abs() < 2e-3, delta + 5e-3, delta)
    old, adv = (logp - delta).float(), torch.randn(n, generator=gen, device="cuda")
    ref = (logp + 0.3).float()
    cfg = m.muon_policy_config_default(kl_beta=0.1)
    stats, got, grad = m.muon_policy_loss(z, y, old, adv, mask=live, ref_logp=ref, temperature=temperature, config=cfg)
    w = torch.ones(n, dtype=torch.float64, device="cuda") if live is None else live.double()
    w /= w.sum().clamp(min=1)
    r = (logp - old.double()).exp()
    plain, held = r * adv, r.clamp(float(torch.tensor(1 - 0.2)), float(torch.tensor(1.2))) * adv
    cut = held < plain
    d = ref.double() - logp
    slope = w * (torch.where(cut, 0.0, -plain) - 0.1 * torch.expm1(d))
    scale = w * (plain.abs() + 0.1 * (1 + d.exp()))
    s, k = torch.minimum(plain, held), torch.expm1(d) - d
    want = torch.stack([(w * (0.1 * k - s)).sum(), -(w * s).sum(), (w * k).sum(), (w * cut).sum()])
    assert ((got.double() - logp).abs() <= LP_ABS + LP_REL * logp.abs()).all()
    assert ((stats.double() - want).abs() <= 2e-5 * (scale.sum() + 2)).all()
    _check_grad(z, y, live, temperature, grad, slope, scale)


@pytest.mark.parametrize("n,v,dtype", [(3000, 4105, "bfloat16"), (2600, 131072, "bfloat16"), (5000, 700, "float32")])
def test_policy_in_place_over_many_rows(m, n, v, dtype):
    import torch
    z, y, live, gen = _inputs(n, v, dtype, "blocks", 5)
    old, adv = torch.zeros(n, device="cuda") - 1.0, torch.randn(n, generator=gen, device="cuda")
    first = m.muon_policy_loss(z, y, old, adv, mask=live)
    stats, logp, grad = m.muon_policy_loss(z, y, old, adv, mask=live, grad=z)
    assert grad.data_ptr() == z.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(first, (stats, logp, grad)))


@pytest.mark.parametrize("n,v,dtype", [(20000, 1000, "bfloat16"), (5000, 9001, "bfloat16"), (1500, 131072, "bfloat16"),
                                       (300, 33003, "float32"), (90, 131072, "bfloat16"), (60, 200001, "float32")])
@pytest.mark.parametrize("mask", ["none", "blocks"])
def test_preference_rows(m, n, v, dtype, mask):
    import torch
    z, y, live, gen = _inputs(n, v, dtype, mask, seed=n)
    logp = _reference(z, y, live, 1.0)
    pairs = 3
    off = torch.tensor([0, n // 7, n // 3, n // 2, n // 2 + 2, n - n // 9, n], device="cuda")
    sums = torch.stack([logp[a:b].sum() for a, b in zip(off[:-1].tolist(), off[1:].tolist())])
    ref = (sums + 4 * torch.randn(6, generator=gen, device="cuda", dtype=torch.float64)).float()
    loss, margins, seq, grad = m.muon_preference_loss(z, y, off, ref, mask=live)
    gain = sums - ref.double()
    h = 0.1 * (gain[:3] - gain[3:])
    # every position may be off by LP_ABS + LP_REL |logp|
    each = LP_ABS + LP_REL * logp.abs()
    tol = torch.stack([each[a:b].sum() for a, b in zip(off[:-1].tolist(), off[1:].tolist())])
    assert ((seq.double() - sums).abs() <= tol + 2.0 ** -23 * sums.abs() + 1e-6).all()
    moff = 0.1 * (tol[:3] + tol[3:]) + 2.0 ** -22 * (1 + h.abs())
    assert ((margins.double() - h).abs() <= moff).all()
    assert abs(loss.item() - torch.nn.functional.softplus(-h).mean().item()) <= moff.max().item() + 2e-6
    slope = torch.zeros(n, dtype=torch.float64, device="cuda")
    for i in range(pairs):
        d = -0.1 / pairs * torch.sigmoid(-h[i])
        slope[off[i]:off[i + 1]] = d
        slope[off[pairs + i]:off[pairs + i + 1]] = -d
    # the slope moves by at most a quarter of the margin's error, relative to beta / P
    scale = slope.abs() + 0.25 * 0.1 / pairs * moff.max() / 4e-5
    _check_grad(z, y, live, 1.0, grad, slope, scale)


def test_two_threads_on_one_stream(m):
    """Calls of two threads interleave on a stream; neither uses the other's workspace."""
    import threading

    import torch
    z, y, live, gen = _inputs(800, 3001, "bfloat16", "blocks")
    old, adv = torch.zeros(800, device="cuda") - 1.0, torch.randn(800, generator=gen, device="cuda")
    off = torch.tensor([0, 300, 800], device="cuda")
    refs = torch.zeros(2, device="cuda")

    def policy():
        return m.muon_policy_loss(z, y, old, adv, mask=live)

    def preference():
        return m.muon_preference_loss(z, y, off, refs, mask=live)

    want, seen = {f: f() for f in (policy, preference)}, {policy: [], preference: []}
    threads = [threading.Thread(target=lambda f=f: seen[f].extend(f() for _ in range(200))) for f in seen]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for f in seen:
        assert len(seen[f]) == 200
        assert all(torch.equal(a, b) for got in seen[f] for a, b in zip(want[f], got))


# rows, logits, type: without a gradient rows come from memory with 64, 128, 256 and 512
# threads (both sides of each step), through a cluster where they are few, or a warp a row
LOSS_ONLY = [(5000, 9001, "bfloat16"), (1217, 20001, "float32"), (1216, 20001, "float32"), (609, 20001, "bfloat16"),
             (608, 20001, "bfloat16"), (304, 33003, "float32"), (2500, 131072, "bfloat16"), (400, 131072, "bfloat16"),
             (304, 131072, "float32"), (31, 33003, "float32"), (5, 131072, "bfloat16"), (20000, 1000, "bfloat16"),
             (1, 50001, "float32")]


@pytest.mark.parametrize("n,v,dtype", LOSS_ONLY)
@pytest.mark.parametrize("mask", ["none", "blocks"])
def test_policy_without_a_gradient_writes_every_output(m, n, v, dtype, mask):
    """The statistics and log-probabilities of a loss-only call, into tensors that hold NaN before it."""
    import torch
    z, y, live, gen = _inputs(n, v, dtype, mask, 2, seed=n + v)
    logp = _reference(z, y, live, 0.9)
    delta = 0.3 * torch.randn(n, generator=gen, device="cuda", dtype=torch.float64)
    for lim in (math.log(0.8), math.log(1.2)):
        delta = torch.where((delta - lim).abs() < 2e-3, delta + 5e-3, delta)
    old, adv = (logp - delta).float(), torch.randn(n, generator=gen, device="cuda")
    ref = (logp + 0.3).float()
    cfg = m.muon_policy_config_default(kl_beta=0.1)
    stats, got = (torch.full((k,), math.nan, device="cuda") for k in (4, n))
    out = m.muon_policy_loss(z, y, old, adv, mask=live, ref_logp=ref, temperature=0.9, config=cfg, with_grad=False,
                             stats=stats, logp=got)
    assert out[0] is stats and out[1] is got and out[2] is None
    w = torch.ones(n, dtype=torch.float64, device="cuda") if live is None else live.double()
    w /= w.sum().clamp(min=1)
    r = (logp - old.double()).exp()
    plain, held = r * adv, r.clamp(float(torch.tensor(1 - 0.2)), float(torch.tensor(1.2))) * adv
    d = ref.double() - logp
    s, k = torch.minimum(plain, held), torch.expm1(d) - d
    want = torch.stack([(w * (0.1 * k - s)).sum(), -(w * s).sum(), (w * k).sum(), (w * (held < plain)).sum()])
    size = (w * (plain.abs() + 0.1 * (1 + d.exp()))).sum() + 2
    assert ((got.double() - logp).abs() <= LP_ABS + LP_REL * logp.abs()).all()
    assert ((stats.double() - want).abs() <= 2e-5 * size).all(), (stats.tolist(), want.tolist())


@pytest.mark.parametrize("n,v,dtype", LOSS_ONLY)
def test_preference_without_a_gradient_writes_every_output(m, n, v, dtype):
    import torch
    z, y, live, _ = _inputs(n, v, dtype, "blocks", 2, seed=n)
    off = torch.tensor([0, n // 3, n // 2, n // 2, n], device="cuda")
    refs = torch.zeros(4, device="cuda")
    want = m.muon_preference_loss(z, y, off, refs, mask=live)
    outs = [torch.full((k,), math.nan, device="cuda") for k in (1, 2, 4)]
    got = m.muon_preference_loss(z, y, off, refs, mask=live, with_grad=False, loss=outs[0], margins=outs[1],
                                 seq_logp=outs[2])
    assert got[3] is None and all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))
    assert all(torch.isfinite(t).all() for t in got[:3])
