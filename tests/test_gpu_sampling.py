"""Sampling and draft verification against float64.

Tolerances, derived before the first run.  A term 2^x, x = c (z - m), has the relative
error of its argument, at most 3 roundings of |x| 2^-24 and so ln 2 * 3 * 2^-24 |x|, and 2^-22
of the exponential.  Weighted by the terms, |x| is at most log2 V + 4 = 22 for the rows used
here, so that a cumulated share is off by at most 22 * 1.25e-7 + 2.4e-7 = 3e-6 where all errors
have one sign.
  token      drawn with u, lies where |u - its share| <= SHARE = 3e-6; for differences p - q,
             whose terms carry the errors of p and q, 2 SHARE / sum max(p - q, 0)
  accepted   u at least 1e-3 away from p / q, relative errors of which are 1e-5 at most
  logp       as for muon_token_logprobs: LP_ABS + LP_REL |logp|
"""
import numpy as np
import pytest

from gpu_util import nsm
from oracle import sampling

pytestmark = pytest.mark.gpu
LP_ABS, LP_REL, SHARE = 1e-5, 4e-7, 3e-6


@pytest.fixture(scope="module")
def m():
    return nsm()


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _rows(rng, n, v, dtype="float32", pad=0, lead=0, temperature=1.0, like=None, noise=0.5):
    """(logits on the device, their float64 values); other memory holds 300."""
    import torch
    if like is None:
        z = rng.normal(0, 2.5 * temperature, (n, v))
        z[np.arange(n), rng.integers(0, v, n)] += rng.uniform(0, 8, n) * temperature
    else:
        z = like + rng.normal(0, noise * temperature, (n, v))
    buffer = torch.full((lead + n * (v + pad),), 300.0, device="cuda").to(getattr(torch, dtype))
    logits = buffer[lead:].view(n, v + pad)[:, :v]
    logits.copy_(_dev(z.astype(np.float32)))
    return logits, logits.double().cpu().numpy()


def _logp(p, tokens):
    """log p of each row's token; where it is nearly 1, from the sum of the others."""
    n = np.arange(len(tokens))
    at = p[n, tokens]
    others = p.copy()
    others[n, tokens] = 0
    return np.where(at > 0.5, np.log1p(-others.sum(1)), np.log(np.where(at > 0, at, 1)))


def _check_logp(got, want):
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= LP_ABS + LP_REL * np.abs(want)).all(), err.max()


def _check_sample(m, logits, z, u, mask=None, temperature=1.0, **kw):
    tokens, logp = m.muon_sample_tokens(logits, _dev(u.astype(np.float32)), mask=None if mask is None else _dev(mask),
                                        temperature=temperature, **kw)
    p = sampling.probabilities(z, temperature)
    got = tokens.cpu().numpy()
    live = np.ones(len(z), bool) if mask is None else mask
    assert (got[~live] == -1).all() and (logp.cpu().numpy()[~live] == 0).all()
    for t in np.nonzero(live)[0]:
        assert 0 <= got[t] < z.shape[1] and p[t, got[t]] > 0
        assert sampling.distance(p[t], float(np.float32(u[t])), got[t]) <= SHARE, t
    _check_logp(logp[_dev(live)], _logp(p[live], got[live]))
    return tokens, logp


@pytest.mark.parametrize("n,v,dtype,pad,lead", [
    (1, 1, "float32", 0, 0), (3, 2, "bfloat16", 0, 1), (5, 7, "float32", 1, 3), (9, 8, "bfloat16", 0, 0),
    (4, 9, "bfloat16", 2, 5), (40, 1000, "bfloat16", 3, 1), (40, 1023, "float32", 0, 1), (700, 1024, "bfloat16", 0, 0),
    (700, 1025, "float32", 0, 0), (33, 4099, "bfloat16", 0, 7), (2, 32773, "float32", 5, 2), (1, 131072, "bfloat16", 0, 0),
    (300, 16384, "float32", 0, 0), (64, 50001, "float32", 3, 0), (7, 160001, "bfloat16", 0, 1)])
def test_sample(m, n, v, dtype, pad, lead):
    rng = np.random.default_rng([n, v])
    logits, z = _rows(rng, n, v, dtype, pad, lead, 0.8)
    _check_sample(m, logits, z, rng.random(n), rng.random(n) < 0.8, 0.8)


def test_sample_long_row(m):
    """More strips than a CTA's table has room for, so that strips are longer."""
    rng = np.random.default_rng(5)
    logits, z = _rows(rng, 2, 3000017, "bfloat16", 0, 3)
    _check_sample(m, logits, z, rng.random(2))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("v", [5, 2048, 70001])
def test_sample_ends(m, dtype, v):
    """Uniforms at and outside the ends, and tokens that cannot be taken there."""
    import torch
    rng = np.random.default_rng(v)
    logits, z = _rows(rng, 6, v, dtype)
    logits[:, 0] = logits[:, v - 1] = -np.inf
    z[:, 0] = z[:, v - 1] = -np.inf
    u = torch.tensor([0.0, -3.0, 1 - 2.0 ** -24, 1.0, 7.0, float("inf")], device="cuda")
    tokens, logp = m.muon_sample_tokens(logits, u)
    p = sampling.probabilities(z)
    got = tokens.cpu().numpy()
    assert (got[:2] == 1).all() and (got[3:] == v - 2).all()
    assert sampling.distance(p[2], 1 - 2.0 ** -24, got[2]) <= SHARE and p[2, got[2]] > 0
    _check_logp(logp, _logp(p, got))


def test_sample_rows_without_probabilities(m):
    import torch
    z = torch.randn(7, 5003, device="cuda")
    z[0, 17] = float("nan")
    z[1, 4999] = float("inf")
    z[2] = -float("inf")
    z[3] = float("nan")
    z[4] = -float("inf")
    z[4, 3333] = -200.0
    z[5, :] = 3e38
    z[6, :] = -3e38
    tokens, logp = m.muon_sample_tokens(z, torch.full((7,), 0.4999, device="cuda"))
    assert tokens.tolist()[:5] == [-1, -1, -1, -1, 3333]
    assert logp[:4].isnan().all() and logp[4] == 0
    for t in (5, 6):  # equal logits
        assert abs((tokens[t].item() + 0.5) / 5003 - 0.4999) < 2e-4
        assert abs(logp[t].item() + np.log(5003)) < 1e-5


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sample_nearly_certain_token_keeps_its_digits(m, dtype):
    import torch
    for gap in (4.0, 12.0, 30.0):
        z = torch.zeros(3, 4001, device="cuda", dtype=getattr(torch, dtype))
        z[:, 2000] = gap + float(np.log(4000.0))
        tokens, logp = m.muon_sample_tokens(z, torch.full((3,), 0.5, device="cuda"))
        # log p = log1p(-others) would lose digits of the sum of the others, S e^-z
        want = -np.log1p(4000 * np.exp(-float(z[0, 2000])))
        assert tokens.tolist() == [2000] * 3
        # terms at |x| <= 56 bits, 56 * 1.25e-7, the exponential's 2.4e-7 and two roundings
        assert (logp.double() / want - 1).abs().max() <= 8e-6


def test_sample_temperatures(m):
    rng = np.random.default_rng(3)
    logits, z = _rows(rng, 8, 3001)
    u = rng.random(8)
    for temperature in (0.05, 3.0, 1e3):
        _check_sample(m, logits, z, u, None, temperature)
    # the largest logit
    tokens, logp = m.muon_sample_tokens(logits, _dev(np.full(8, 0.5, np.float32)), temperature=1e-20)
    assert (tokens.cpu().numpy() == z.argmax(1)).all() and (logp == 0).all()


def _drafts(rng, lengths, v, dtype="float32", pad=0, lead=0, temperature=1.0, noise=0.5, form="logp", off=0):
    """A seeded verification: what the call takes, and the same in float64."""
    lengths = np.asarray(lengths)
    n, s = int(lengths.sum()), len(lengths)
    seq = np.repeat(np.arange(s), lengths)
    target, z = _rows(rng, n + s, v, dtype, pad, lead, temperature)
    p = sampling.probabilities(z, temperature)
    rows = np.arange(n) + seq
    draft, zq = _rows(rng, n, v, dtype, 0, off, temperature, z[rows], noise)
    q = sampling.probabilities(zq, temperature) if n else np.zeros((0, v))
    drafts = np.array([sampling.pick(w, u) for w, u in zip(q, rng.random(n))], np.int64)
    if form == "certain":
        q = np.zeros((n, v))
        q[np.arange(n), drafts] = 1
    qx = q[np.arange(n), drafts]
    u = rng.random(n)
    ratio = p[rows, drafts] / qx
    u = np.where(np.abs(u - ratio) < 1e-3, np.where(ratio > 0.5, ratio - 4e-3, ratio + 4e-3), u).astype(np.float32)
    su = rng.random(s).astype(np.float32)
    args = dict(logits=target, drafts=_dev(drafts), draft_offsets=_dev(np.concatenate([[0], lengths.cumsum()])),
                accept_uniforms=_dev(u), sample_uniforms=_dev(su), temperature=temperature)
    if form != "certain":
        args["draft_logits"] = draft
    if form == "logp":
        args["draft_logp"] = _dev(np.log(qx).astype(np.float32))
    return args, dict(p=p, q=q, drafts=drafts, lengths=lengths, u=u, su=su, qx=qx)


def _check_verify(args, e, got):
    tokens, counts, logp = (t.cpu().numpy() for t in got)
    want, weights = sampling.verify(e["p"], e["q"], e["drafts"], e["lengths"], e["u"], e["qx"])
    assert (counts == want).all()
    row = d = 0
    for s, n in enumerate(e["lengths"]):
        a = counts[s]
        assert (tokens[row:row + a] == e["drafts"][d:d + a]).all()
        x, w = tokens[row + a], weights[s]
        assert 0 <= x < w.shape[0] and w[x] > 0
        # weights of p sum to 1; those of max(p - q, 0) carry the errors of both
        assert sampling.distance(w, float(e["su"][s]), x) <= (SHARE if a == n else 2 * SHARE / w.sum()), s
        assert (tokens[row + a + 1:row + n + 1] == -1).all() and (logp[row + a + 1:row + n + 1] == 0).all()
        row, d = row + n + 1, d + n
    live = tokens >= 0
    err = np.abs(logp[live] - _logp(e["p"][live], tokens[live]))
    assert (err <= LP_ABS + LP_REL * np.abs(logp[live])).all(), err.max()


LENGTHS = {"one": [4], "none": [0], "empty": [0, 0, 3, 0], "mixed": [2, 0, 5, 1, 7, 3], "long": [19, 1, 40],
           "many": [4] * 170, "more": [3, 0, 1] * 250}


@pytest.mark.parametrize("form", ["logp", "logits", "certain"])
@pytest.mark.parametrize("lengths,v,dtype,pad,lead,off", [
    ("one", 131072, "bfloat16", 0, 0, 0), ("one", 1000, "float32", 1, 1, 0), ("none", 517, "bfloat16", 0, 0, 0),
    ("empty", 4099, "bfloat16", 0, 3, 1), ("mixed", 4099, "bfloat16", 0, 0, 0), ("mixed", 50001, "float32", 3, 0, 1),
    ("long", 2053, "float32", 0, 0, 0), ("long", 8192, "bfloat16", 8, 0, 5), ("many", 5000, "bfloat16", 0, 0, 0),
    ("many", 1, "float32", 0, 0, 0), ("more", 3, "bfloat16", 0, 1, 1), ("more", 1029, "float32", 0, 0, 2)])
def test_verify(m, lengths, v, dtype, pad, lead, off, form):
    rng = np.random.default_rng([v, len(lengths)])
    args, e = _drafts(rng, LENGTHS[lengths], v, dtype, pad, lead, 0.9, 0.6, form, off)
    _check_verify(args, e, m.muon_verify_drafts(**args))


@pytest.mark.parametrize("form", ["logp", "logits", "certain"])
@pytest.mark.parametrize("taken", [False, True])
def test_verify_one_long_sequence_among_many(m, form, taken):
    """Its rows take several rounds of CTAs, and more sequences than one CTA draws for."""
    rng = np.random.default_rng(21)
    args, e = _drafts(rng, [0, 1, 2] * 220 + [30, 1], 700, "float32", 1, 0, 1.0, 0.3, form)
    if taken:
        e["u"] = np.zeros(len(e["u"]), np.float32)
        args["accept_uniforms"] = _dev(e["u"])
    got = m.muon_verify_drafts(**args)
    _check_verify(args, e, got)
    again = m.muon_verify_drafts(**args)
    assert all((x == y).all() for x, y in zip(got, again))


def test_sample_masked_halves(m):
    """All of some CTAs' rows are masked."""
    rng = np.random.default_rng(22)
    logits, z = _rows(rng, 1300, 9000, "bfloat16", 0, 0, 1.0)
    mask = np.arange(1300) % 7 < 2
    mask[200:900] = False
    u = rng.random(1300).astype(np.float32)
    tokens, logp = m.muon_sample_tokens(logits, _dev(u), mask=_dev(mask))
    tokens, logp = tokens.cpu().numpy(), logp.cpu().numpy()
    assert (tokens[~mask] == -1).all() and (logp[~mask] == 0).all()
    p = sampling.probabilities(z, 1.0)
    for t in np.flatnonzero(mask):
        assert sampling.distance(p[t], float(u[t]), tokens[t]) <= SHARE
    err = np.abs(logp[mask] - _logp(p[mask], tokens[mask]))
    assert (err <= LP_ABS + LP_REL * np.abs(logp[mask])).all(), err.max()


@pytest.mark.parametrize("form", ["logp", "logits", "certain"])
def test_verify_all_taken_or_none(m, form):
    rng = np.random.default_rng(11)
    for share in (1, 0):
        args, e = _drafts(rng, [9, 2, 16, 0, 1], 3001, noise=1.5, form=form)
        e["u"] = np.zeros(28, np.float32)
        if not share:  # above any ratio
            e["u"] = (e["p"].max() / e["qx"] + 1).astype(np.float32)
        args["accept_uniforms"] = _dev(e["u"])
        got = m.muon_verify_drafts(**args)
        _check_verify(args, e, got)
        assert got[1].tolist() == ([9, 2, 16, 0, 1] if share else [0, 0, 0, 0, 0])


def test_verify_equal_models(m):
    """Refused although p = q (u = 1.5): nothing is left over and the token comes from p."""
    rng = np.random.default_rng(12)
    args, e = _drafts(rng, [2, 1], 2000, noise=0.0)
    args["accept_uniforms"] = _dev(np.full(3, 1.5, np.float32))
    args["draft_logits"].copy_(args["logits"][[0, 1, 3]])
    tokens, counts, logp = m.muon_verify_drafts(**args)
    assert counts.tolist() == [0, 0]
    for s, row in ((0, 0), (1, 3)):
        assert sampling.distance(e["p"][row], float(e["su"][s]), tokens[row].item()) <= SHARE


def test_verify_one_certain_token(m):
    """A draft that holds all of p, refused: nothing is left without it."""
    import torch
    z = torch.full((2, 999), -float("inf"), device="cuda")
    z[:, 500] = 1.0
    got = m.muon_verify_drafts(z, _dev(np.array([500])), _dev(np.array([0, 1])), _dev(np.array([1.0], np.float32)),
                               _dev(np.array([0.3], np.float32)))
    assert got[0].tolist() == [500, -1] and got[1].tolist() == [0] and got[2].tolist() == [0, 0]


@pytest.mark.parametrize("form", ["logp", "logits", "certain"])
def test_verify_drafts_out_of_range_are_refused(m, form):
    rng = np.random.default_rng(13)
    args, e = _drafts(rng, [3, 3], 1500, form=form)
    e["u"][:] = 0
    args["accept_uniforms"].zero_()
    args["drafts"][1] = 1500
    args["drafts"][3] = -1
    tokens, counts, logp = m.muon_verify_drafts(**args)
    assert counts.tolist() == [1, 0]
    for s, row, d in ((0, 1, 1), (1, 4, 3)):
        w = e["p"][row] if form == "certain" else np.maximum(e["p"][row] - e["q"][d], 0)
        assert sampling.distance(w, float(e["su"][s]), tokens[row].item()) <= 2 * SHARE / w.sum()


@pytest.mark.parametrize("count", [5, 700])
@pytest.mark.parametrize("v,dtype", [(1500, "float32"), (40001, "bfloat16")])
def test_verify_certain_drafts_past_32_bits(m, v, dtype, count):
    """A draft outside [0, vocab) is none of the tokens, whatever its low 32 bits say: the token that
    they name is drawn with the share that p gives it."""
    import torch
    rng = np.random.default_rng([v, count])
    logits, z = _rows(rng, 2 * count, v, dtype)
    ends = np.array([0, 2 ** 32, -2 ** 32, 2 ** 40, -2 ** 63, 3 * 2 ** 32])
    likely = rng.integers(0, v, count)
    first = 2 * np.arange(count)
    logits[_dev(first), _dev(likely)] = 12.0 + float(np.log(v))
    logits[0] = -np.inf   # one token only
    logits[0, int(likely[0])] = 3.0
    z = logits.double().cpu().numpy()
    p = sampling.probabilities(z[first])
    at = np.arange(count)
    su = (np.cumsum(p, 1) - 0.5 * p)[at, likely].astype(np.float32)   # in the middle of the token's share
    drafts = likely + ends[1 + at % 5]
    assert (drafts.astype(np.int32) == likely).all() and ((drafts < 0) | (drafts >= v)).all()
    tokens, counts, logp = m.muon_verify_drafts(logits, _dev(drafts), torch.arange(count + 1, device="cuda"),
                                                torch.zeros(count, device="cuda"), _dev(su))
    assert (counts == 0).all() and (tokens[1::2] == -1).all() and (logp[1::2] == 0).all()
    assert (tokens[::2].cpu().numpy() == likely).all()
    _check_logp(logp[::2], _logp(p, likely))


def test_verify_rows_without_probabilities(m):
    rng = np.random.default_rng(14)
    args, e = _drafts(rng, [2, 2, 2], 700)
    args["accept_uniforms"].zero_()
    args["logits"][1, 5] = float("nan")   # sequence 0: its second draft
    args["logits"][5] = -float("inf")     # sequence 1: the row after its drafts
    args["accept_uniforms"][4] = 1e6      # sequence 2 refuses at its first, whose model has no probabilities
    args["draft_logits"][4, 3] = float("inf")
    tokens, counts, logp = m.muon_verify_drafts(**args)
    assert counts.tolist() == [1, 2, 0]
    assert tokens[[1, 5, 6]].tolist() == [-1, -1, -1] and logp[[1, 5, 6]].isnan().all()
    assert tokens[2].item() == -1 and logp[2].item() == 0


def test_verify_touches_nothing_else(m):
    """Memory around the outputs stays as it was; offsets out of range read and write nothing
    outside the arrays."""
    import torch
    rng = np.random.default_rng(15)
    args, e = _drafts(rng, [2, 3], 600)
    out = [torch.full((20,), 77, device="cuda") for _ in range(2)] + [torch.full((20,), 77.0, device="cuda")]
    m.muon_verify_drafts(**args, tokens=out[0][4:11], counts=out[1][4:6], logp=out[2][4:11])
    assert all((t[:4] == 77).all() for t in out) and (out[0][11:] == 77).all() and (out[2][11:] == 77).all()
    assert (out[1][6:] == 77).all()
    for offsets in ([0, 9, 5], [0, -4, 5], [3, 1, 2 ** 40]):
        args["draft_offsets"] = _dev(np.array(offsets))
        m.muon_verify_drafts(**args, tokens=out[0][4:11], counts=out[1][4:6], logp=out[2][4:11])
    torch.cuda.synchronize()
    assert all((t[:4] == 77).all() for t in out) and (out[0][11:] == 77).all() and (out[2][11:] == 77).all()


def test_sampled_rows_past_2_31_elements(m):
    import torch
    n, v = 16411, 131072
    logits = torch.zeros(n, v, device="cuda", dtype=torch.bfloat16)
    at = torch.arange(n, device="cuda") * 7919 % v
    logits.scatter_(1, at[:, None], 40.0)
    tokens, logp = m.muon_sample_tokens(logits, torch.full((n,), 0.5, device="cuda"))
    assert (tokens == at).all() and (logp.abs() < 1e-10).all()
    offsets = torch.arange(0, n // 2 + 1, device="cuda")   # one draft a sequence
    rows = torch.arange(n // 2, device="cuda") * 2
    half = torch.full((n // 2,), 0.5, device="cuda")
    got, counts, _ = m.muon_verify_drafts(logits[:2 * (n // 2)], at[rows], offsets, half, half)
    assert (counts == 1).all() and (got == at[:2 * (n // 2)]).all()


def test_graph_streams_and_repeats(m):
    """The same bits on every call, from a captured graph with new inputs too, and on another stream."""
    import torch
    rng = np.random.default_rng(16)
    args, e = _drafts(rng, [4, 0, 6, 2], 30011, "bfloat16")
    first = m.muon_verify_drafts(**args)
    out = [torch.zeros_like(t) for t in first]
    graph = torch.cuda.CUDAGraph()
    held = {k: v.clone() if torch.is_tensor(v) else v for k, v in args.items()}
    with torch.cuda.graph(graph):
        m.muon_verify_drafts(**held, tokens=out[0], counts=out[1], logp=out[2])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    held["sample_uniforms"].copy_(_dev(rng.random(4).astype(np.float32)))
    graph.replay()
    again = m.muon_verify_drafts(**{**args, "sample_uniforms": held["sample_uniforms"]})
    assert all(torch.equal(a, b) for a, b in zip(again, out))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    other = m.muon_verify_drafts(**args, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))


def test_drafted_rollout_feeds_the_policy_loss(m):
    """Drafts sampled from one model, verified by another: the log-probabilities are those that
    the policy loss computes, so that its ratios are 1 and nothing is clipped."""
    import torch
    rng = np.random.default_rng(17)
    s, k, v = 6, 3, 2000
    target, z = _rows(rng, s * (k + 1), v, "bfloat16")
    draft, _ = _rows(rng, s * k, v, "bfloat16", like=z.reshape(s, k + 1, v)[:, :k].reshape(s * k, v), noise=1.0)
    u = torch.rand(3, s * k, device="cuda")
    drafts, draft_logp = m.muon_sample_tokens(draft, u[0], temperature=0.7)
    offsets = torch.arange(0, s * k + 1, k, device="cuda")
    tokens, counts, logp = m.muon_verify_drafts(target, drafts, offsets, u[1], u[2, :s], draft_logits=draft,
                                                draft_logp=draft_logp, temperature=0.7)
    live = tokens >= 0
    assert live.sum() == counts.sum() + s
    direct = m.muon_token_logprobs(target, tokens, mask=live, temperature=0.7)
    assert (direct - logp).abs().max() <= 2 * LP_ABS
    advantages = torch.randn(s * (k + 1), device="cuda")
    stats, _, grad = m.muon_policy_loss(target, tokens, logp, advantages, mask=live, temperature=0.7)
    assert abs(stats[0].item() + (advantages * live).sum().item() / live.sum().item()) <= 1e-4 and stats[3] == 0
    assert (grad[~live] == 0).all() and (grad[live].abs().sum(1) > 0).all()


@pytest.mark.parametrize("form", ["logp", "logits"])
def test_verify_with_the_drafts_own_temperature(m, form):
    rng = np.random.default_rng(18)
    args, e = _drafts(rng, [3, 5, 0, 2], 2501, form=form)
    q = sampling.probabilities(args["draft_logits"].double().cpu().numpy(), 1.7)
    e["q"], e["qx"] = q, q[np.arange(10), e["drafts"]]
    rows = np.arange(10) + np.repeat(np.arange(4), [3, 5, 0, 2])
    ratio = e["p"][rows, e["drafts"]] / e["qx"]
    u = rng.random(10)
    e["u"] = np.where(np.abs(u - ratio) < 1e-3, u / 2, u).astype(np.float32)
    args["accept_uniforms"] = _dev(e["u"])
    if form == "logp":
        args["draft_logp"] = _dev(np.log(e["qx"]).astype(np.float32))
    _check_verify(args, e, m.muon_verify_drafts(**args, draft_temperature=1.7))


def test_two_threads_on_one_stream(m):
    """Each thread has a workspace of its own."""
    import threading

    import torch
    rng = np.random.default_rng(19)
    sets = [_drafts(rng, [4, 2, 7] * 9, 9001, "bfloat16")[0] for _ in range(2)]
    logits = [s["logits"] for s in sets]
    u = torch.rand(len(logits[0]), device="cuda")
    want = [(m.muon_verify_drafts(**s), m.muon_sample_tokens(z, u)) for s, z in zip(sets, logits)]
    torch.cuda.synchronize()
    got, stream = [[], []], torch.cuda.current_stream()

    def work(k):
        for _ in range(20):
            got[k].append((m.muon_verify_drafts(**sets[k], stream=stream), m.muon_sample_tokens(logits[k], u, stream=stream)))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in range(2):
        assert len(got[k]) == 20
        for a, b in got[k]:
            assert all(torch.equal(x, y) for x, y in zip(a + b, want[k][0] + want[k][1]))


def test_refusals(m):
    import torch
    z = torch.randn(6, 50, device="cuda")
    u = torch.rand(6, device="cuda")
    for bad in (dict(uniforms=u[:5]), dict(uniforms=u.cpu()), dict(uniforms=u.double()), dict(mask=torch.ones(6, device="cuda")),
                dict(tokens=torch.zeros(6, device="cuda", dtype=torch.int32)), dict(logp=torch.zeros(5, device="cuda")),
                dict(workspace=torch.zeros(1 << 12))):
        with pytest.raises((ValueError, TypeError)):
            m.muon_sample_tokens(z, **{"uniforms": u, **bad})
    with pytest.raises(m.MuonError) as e:
        m.muon_sample_tokens(z, u, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == m.MUON_ERR_NO_WORKSPACE
    with pytest.raises(ValueError):
        m.muon_sample_tokens(z.t(), torch.rand(50, device="cuda"))
    with pytest.raises(TypeError):
        m.muon_sample_tokens(z.half(), u)
    args, _ = _drafts(np.random.default_rng(20), [2, 1], 50)
    for bad in (dict(drafts=args["drafts"][:2]), dict(drafts=args["drafts"].int()), dict(draft_offsets=args["draft_offsets"][:2]),
                dict(draft_offsets=args["draft_offsets"][:0]), dict(accept_uniforms=args["sample_uniforms"]),
                dict(sample_uniforms=args["accept_uniforms"]), dict(draft_logits=args["draft_logits"][:2]),
                dict(draft_logits=args["draft_logits"][:, :40]), dict(draft_logits=args["draft_logits"].bfloat16()),
                dict(draft_logp=args["draft_logp"].double())):
        with pytest.raises(ValueError):
            m.muon_verify_drafts(**{**args, **bad})
    with pytest.raises(m.MuonError) as e:
        m.muon_verify_drafts(**{**args, "draft_logits": None})   # log-probabilities of certain drafts
    assert e.value.status == m.MUON_ERR_INVALID
