"""The operators around the optimizer step: global gradient norm and clipping, token
log-probabilities, the clipped policy loss and the preference loss with their gradients.

Each case is one call as a training or scoring program makes it.  `run` computes it with
elementary torch operations in fp32, or, with `own` set, through the library.
"""
import math

import torch

own = False

# the matrices of one Qwen3-4B-shaped layer: q, k, v, o, gate, up, down
LAYER = [(4096, 2560), (1024, 2560), (1024, 2560), (2560, 4096), (9728, 2560), (9728, 2560), (2560, 9728)]
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CLIP_LOW, CLIP_HIGH = 0.2, 0.28   # the policy loss's ratio range 1 - CLIP_LOW .. 1 + CLIP_HIGH
EPS = 1e-6                        # added to the gradient norm before dividing


def listed():
    return [
        # the gradient of one small fp32 weight: nothing but latency
        dict(name="clip_one_matrix", op="clip", sets="matrices", rows=256, cols=512, n=1, dtype="f32", out="f32",
             max_norm=1.0),
        # the bf16 gradients of one layer, clipped into the fp32 gradients that the step reads
        dict(name="clip_layer", op="clip", sets="layers", n=1, dtype="bf16", out="f32", max_norm=1.0),
        # gains, biases and adapter factors: many small tensors, views of two flat buffers at odd offsets
        dict(name="clip_ragged", op="clip", sets="ragged", n=1003, most=40000, out="f32", max_norm=0.5),
        # the whole model's gradients in place, and the norm below its limit, as in most steps
        dict(name="clip_model_below", op="clip", sets="layers", n=36, dtype="bf16", out="", max_norm=1e6),
        # scoring one token
        dict(name="logprob_one_token", op="logprob", tokens=1, vocab=131072, dtype="bf16", pad=0, drop=0.0, temp=1.0),
        # log-probabilities under the reference policy of a long packed batch: over 2^31 logits
        dict(name="logprob_batch", op="logprob", tokens=16411, vocab=131072, dtype="bf16", pad=0, drop=0.1, temp=0.7),
        # a few short answers, fp32 logits of an odd vocabulary in padded rows
        dict(name="policy_short", op="policy", tokens=131, vocab=50001, dtype="f32", pad=3, drop=0.3, temp=1.0, seqs=9,
             beta=0.04, reduce="sequence"),
        # one step's token batch, a fifth of it prompt
        dict(name="policy_batch", op="policy", tokens=4096, vocab=131072, dtype="bf16", pad=0, drop=0.2, temp=1.0,
             seqs=16, beta=0.04, reduce="token"),
        # a small vocabulary and many tokens, an odd row length, no reference policy
        dict(name="policy_small_vocab", op="policy", tokens=20011, vocab=4099, dtype="bf16", pad=0, drop=0.1, temp=0.8,
             seqs=33, beta=0.0, reduce="token"),
        # three pairs of short answers
        dict(name="preference_short", op="preference", tokens=301, vocab=32003, dtype="bf16", pad=0, drop=0.2, temp=1.0,
             pairs=3, beta=0.1, smooth=0.0, mean=False),
        # fp32 logits, length-normalised, smoothed labels
        dict(name="preference_f32", op="preference", tokens=1024, vocab=65536, dtype="f32", pad=0, drop=0.3, temp=1.0,
             pairs=4, beta=2.0, smooth=0.1, mean=True),
        # long answers
        dict(name="preference_batch", op="preference", tokens=8192, vocab=131072, dtype="bf16", pad=0, drop=0.25,
             temp=1.0, pairs=8, beta=0.1, smooth=0.0, mean=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["clip", "logprob", "policy", "preference"])
    if op == "clip":
        sets = rng.choice(["matrices", "layers", "ragged"])
        # in place only below the limit: gradients already clipped would make another case
        out = rng.choice(["bf16", "f32", ""])
        case = dict(op=op, sets=sets, out=out, max_norm=rng.choice([0.1, 1.0, 1e6]) if out else 1e6)
        if sets == "matrices":
            case.update(rows=spread(1, 3000), cols=spread(1, 3000), n=spread(1, 60), dtype=rng.choice(["bf16", "f32"]))
        elif sets == "layers":
            case.update(n=spread(1, 8), dtype=rng.choice(["bf16", "f32"]))
        else:
            case.update(n=spread(2, 3000), most=spread(2, 50000))
        return case
    vocab = spread(500, 160000)
    longest = 8192 if op == "preference" else 20000
    tokens = spread(2 if op == "preference" else 1, max(2, min(longest, 400000000 // vocab)))
    case = dict(op=op, tokens=tokens, vocab=vocab, dtype=rng.choice(["bf16", "bf16", "f32"]),
                pad=rng.choice([0, 0, 5, 64]), drop=rng.choice([0.0, 0.1, 0.4]), temp=rng.choice([1.0, 1.0, 0.6]))
    if op == "policy":
        case.update(seqs=spread(1, min(64, tokens)), beta=rng.choice([0.0, 0.04]),
                    reduce=rng.choice(["token", "sequence", "sum"]))
    elif op == "preference":
        mean = rng.choice([False, True])
        case.update(pairs=spread(1 + tokens // 1024, max(1 + tokens // 1024, min(16, tokens // 2))), beta=2.0 if mean else 0.1, smooth=rng.choice([0.0, 0.1]),
                    mean=mean)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _views(flat, sizes):
    """Consecutive tensors of the given sizes in a flat buffer."""
    at, got = 0, []
    for n in sizes:
        got.append(flat[at:at + n])
        at += n
    return got


def _sizes(case):
    """[(dtype, element count of each tensor)], one entry for each flat buffer."""
    if case["sets"] == "matrices":
        return [(case["dtype"], [case["rows"] * case["cols"]] * case["n"])]
    if case["sets"] == "layers":
        return [(case["dtype"], [r * c for r, c in LAYER] * case["n"])]
    rs = torch.Generator().manual_seed(case["n"])
    sizes = torch.randint(1, case["most"] + 1, (case["n"],), generator=rs).tolist()
    half = len(sizes) // 2
    return [("f32", sizes[:half]), ("bf16", sizes[half:])]


def _prepare_clip(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    state = dict(case=case, grads=[], outs=[], flats=[])
    for dtype, sizes in _sizes(case):
        total = sum(sizes)
        flat = torch.randn(total, generator=gen, device="cuda", dtype=DTYPES[dtype]).mul_(1e-3)
        grads = _views(flat, sizes)
        state["grads"] += grads
        if case["out"]:
            out = torch.zeros(total, device="cuda", dtype=DTYPES[case["out"]])
            state["outs"] += _views(out, sizes)
            flat = out
        state["flats"].append(flat)
    return state


def _offsets(n, parts, gen):
    """parts + 1 offsets of 0..n, device int64; a part may be empty."""
    inner = torch.randint(0, n + 1, (parts - 1,), generator=gen, device="cuda").sort().values
    ends = torch.tensor([0, n], device="cuda")
    return torch.cat([ends[:1], inner, ends[1:]])


def _prepare_rows(case, seed):
    """Logits of a language model: a normal background and a likely next token."""
    gen = torch.Generator("cuda").manual_seed(seed)
    T, V, tau = case["tokens"], case["vocab"], case["temp"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    full = torch.randn(T, V + case["pad"], generator=gen, device="cuda", dtype=DTYPES[case["dtype"]]).mul_(2.5 * tau)
    logits = full[:, :V]
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    level = math.log(V) + 0.5 * 2.5 ** 2
    logits.scatter_(1, targets[:, None], ((level + 1.5 * normal(T, 1)) * tau).to(logits.dtype))
    mask = torch.rand(T, generator=gen, device="cuda") >= case["drop"]
    state = dict(case=case, logits=logits, targets=targets, mask=mask)
    if case["op"] == "logprob":
        return state
    rows = torch.cat([(c.float() / tau).log_softmax(1).gather(1, t[:, None])[:, 0]
                      for c, t in zip(logits.split(1024), targets.split(1024))])
    if case["op"] == "policy":
        state["seq_offsets"] = _offsets(T, case["seqs"], gen)
        part = torch.bucketize(torch.arange(T, device="cuda"), state["seq_offsets"][1:], right=True)
        state["advantages"] = normal(case["seqs"])[part]
        # the rollout's policy is a few updates older; a ratio that rounding could put on
        # either side of a clip limit is moved off it
        delta = 0.15 * normal(T)
        low, high = math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)
        near = ((delta - low).abs() < 1e-3) | ((delta - high).abs() < 1e-3)
        state["old_logp"] = rows - torch.where(near, delta - 4e-3, delta)
        state["ref_logp"] = rows + 0.3 * normal(T) if case["beta"] else None
    else:
        # chosen sequences first, then rejected ones; the reference's sums are near the policy's
        state["seq_offsets"] = _offsets(T, 2 * case["pairs"], gen)
        sums, _ = _sequence_sums(torch.where(mask, rows, 0.0), mask, state["seq_offsets"], case["mean"])
        state["ref_logp"] = sums + 2 * normal(2 * case["pairs"]) / case["beta"]
    return state


def prepare(case, seed):
    return _prepare_clip(case, seed) if case["op"] == "clip" else _prepare_rows(case, seed)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _plain_clip(state):
    case = state["case"]
    total = torch.stack([g.float().square().sum() for g in state["grads"]]).sum().sqrt()
    coef = (case["max_norm"] / (total + EPS)).clamp(max=1.0)
    [o.copy_(g.float() * coef) for g, o in zip(state["grads"], state["outs"] or state["grads"])]
    return dict(norm=torch.stack([total, coef]), grads=state["flats"])


def _plain_logp(state):
    """log-probability of each target (0 where masked), and the softmax."""
    x = state["logits"].float() / state["case"]["temp"]
    x = x - x.amax(1, keepdim=True)
    e = x.exp()
    s = e.sum(1, keepdim=True)
    logp = (x.gather(1, state["targets"][:, None]) - s.log())[:, 0]
    return torch.where(state["mask"], logp, 0.0), e / s


def _plain_grad(state, dlogp, p):
    """dlogp (onehot - p) / temperature, in the logits' type."""
    dlogp = dlogp / state["case"]["temp"]
    grad = p * -dlogp[:, None]
    grad.scatter_add_(1, state["targets"][:, None], dlogp[:, None])
    return torch.where(state["mask"][:, None], grad, 0.0).to(state["logits"].dtype)


def _sequence_sums(values, mask, offsets, mean):
    """Sum (or mean over unmasked tokens) of each sequence, and its unmasked token count."""
    n = values.shape[0]
    part = torch.bucketize(torch.arange(n, device=values.device), offsets[1:], right=True)
    member = part == torch.arange(offsets.shape[0] - 1, device=values.device)[:, None]
    count = (member & mask).sum(1).to(values.dtype)
    sums = torch.where(member, values, 0.0).sum(1)
    return (sums / count.clamp(min=1) if mean else sums), count


def _plain_policy(state):
    case, mask = state["case"], state["mask"]
    logp, p = _plain_logp(state)
    live = mask.float()
    if case["reduce"] == "token":
        w = live / live.sum().clamp(min=1)
    elif case["reduce"] == "sequence":
        _, count = _sequence_sums(live, mask, state["seq_offsets"], False)
        part = torch.bucketize(torch.arange(len(live), device="cuda"), state["seq_offsets"][1:], right=True)
        w = live / (count.clamp(min=1) * case["seqs"])[part]
    else:
        w = live
    adv = state["advantages"]
    ratio = (logp - state["old_logp"]).exp()
    plain, clipped = ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
    cut = clipped < plain
    policy = -torch.where(cut, clipped, plain)
    dlogp = -torch.where(cut, 0.0, plain)
    kl = torch.zeros_like(policy)
    if case["beta"]:
        d = state["ref_logp"] - logp
        kl = d.exp() - d - 1
        dlogp = dlogp + case["beta"] * (1 - d.exp())
    terms = torch.stack([policy + case["beta"] * kl, policy, kl, cut.float()])
    stats = torch.where(mask, terms * w, 0.0).sum(1)
    return dict(stats=stats, logp=logp, grad=_plain_grad(state, w * dlogp, p))


def _plain_preference(state):
    case, mask, P = state["case"], state["mask"], state["case"]["pairs"]
    logp, p = _plain_logp(state)
    sums, count = _sequence_sums(logp, mask, state["seq_offsets"], case["mean"])
    gain = sums - state["ref_logp"]
    margin = case["beta"] * (gain[:P] - gain[P:])
    e = case["smooth"]
    softplus = margin.abs().neg().exp().log1p()  # of -|margin|
    loss = ((1 - e) * (softplus - margin.clamp(max=0)) + e * (softplus + margin.clamp(min=0))).mean()
    pos, neg = 1 / (1 + (-margin).exp()), 1 / (1 + margin.exp())
    dsum = case["beta"] / P * (e * pos - (1 - e) * neg)
    dsum = torch.cat([dsum, -dsum])
    if case["mean"]:
        dsum = dsum / count.clamp(min=1)
    part = torch.bucketize(torch.arange(len(logp), device="cuda"), state["seq_offsets"][1:], right=True)
    return dict(loss=loss[None], margins=margin, seq_logp=sums, grad=_plain_grad(state, dsum[part], p))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(state):
    import newton_schulz_muon_gb300 as nsm

    case = state["case"]
    if case["op"] == "clip":
        norm = nsm.muon_clip_grad_norm(state["grads"], case["max_norm"], out=state["outs"] or None, eps=EPS)
        return dict(norm=norm, grads=state["flats"])
    if case["op"] == "logprob":
        return dict(logp=nsm.muon_token_logprobs(state["logits"], state["targets"], mask=state["mask"],
                                                 temperature=case["temp"]))
    if case["op"] == "policy":
        config = nsm.muon_policy_config_default(
            clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_beta=case["beta"],
            reduction={"token": nsm.MUON_REDUCE_TOKEN_MEAN, "sequence": nsm.MUON_REDUCE_SEQUENCE_MEAN,
                       "sum": nsm.MUON_REDUCE_SUM}[case["reduce"]])
        stats, logp, grad = nsm.muon_policy_loss(
            state["logits"], state["targets"], state["old_logp"], state["advantages"], mask=state["mask"],
            ref_logp=state["ref_logp"], seq_offsets=state["seq_offsets"], temperature=case["temp"], config=config)
        return dict(stats=stats, logp=logp, grad=grad)
    config = nsm.muon_preference_config_default(beta=case["beta"], label_smoothing=case["smooth"],
                                                length_normalize=int(case["mean"]))
    loss, margins, seq_logp, grad = nsm.muon_preference_loss(
        state["logits"], state["targets"], state["seq_offsets"], state["ref_logp"], mask=state["mask"],
        temperature=case["temp"], config=config)
    return dict(loss=loss, margins=margins, seq_logp=seq_logp, grad=grad)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "clip":
        return _plain_clip(state)
    if op == "logprob":
        return dict(logp=_plain_logp(state)[0])
    return _plain_policy(state) if op == "policy" else _plain_preference(state)


def work(case):
    if case["op"] == "clip":
        size = {"bf16": 2, "f32": 4, "": 0}
        bytes_, elems = 0, 0
        for dtype, sizes in _sizes(case):
            elems += sum(sizes)
            bytes_ += sum(sizes) * (size[dtype] + size[case["out"]])
        # a square and an addition; a product where something is written
        return {"bytes": bytes_, "flops": elems * (3 if case["out"] else 2)}
    T, V, es = case["tokens"], case["vocab"], 2 if case["dtype"] == "bf16" else 4
    live = T * (1 - case["drop"])
    rows = T * (8 + 1)                   # targets and mask
    if case["op"] == "logprob":
        return {"bytes": live * V * es + rows + 4 * T, "flops": 4 * live * V}
    # the logits of unmasked rows are read and every row of the gradient is written
    rows += T * (4 + 4 + 4 + (4 if case["beta"] else 0)) if case["op"] == "policy" else 16 * case["pairs"]
    return {"bytes": live * V * es + T * V * es + rows, "flops": 8 * live * V}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_clip(case, seed):
    state = _prepare_clip(case, seed)
    squares = 0.0
    for g in state["grads"]:
        squares += float(torch.dot(g.double(), g.double()))
    norm = math.sqrt(squares)
    coef = min(1.0, case["max_norm"] / (norm + EPS))
    flats, at = [], 0
    for _, sizes in _sizes(case):
        flats.append(torch.cat([g.double() * coef for g in state["grads"][at:at + len(sizes)]]))
        at += len(sizes)
    return dict(norm=torch.tensor([norm, coef], dtype=torch.float64), grads=flats)


def _exact_rows(case, seed):
    state = _prepare_rows(case, seed)
    T, tau = case["tokens"], case["temp"]
    dev = state["logits"].device
    live = state["mask"]
    logits, y = state["logits"], state["targets"]
    logp = torch.zeros(T, dtype=torch.float64, device=dev)
    chunk = max(1, (1 << 27) // case["vocab"])
    for a in range(0, T, chunk):
        z = logits[a:a + chunk].double() / tau
        logp[a:a + chunk] = z.gather(1, y[a:a + chunk, None])[:, 0] - torch.logsumexp(z, 1)
    logp = torch.where(live, logp, torch.zeros_like(logp))
    if case["op"] == "logprob":
        return dict(logp=logp)
    bounds = state["seq_offsets"].tolist()
    part = [slice(a, b) for a, b in zip(bounds[:-1], bounds[1:])]
    counts = [int(live[s].sum()) for s in part]
    slope = torch.zeros(T, dtype=torch.float64, device=dev)
    if case["op"] == "policy":
        w = torch.zeros(T, dtype=torch.float64, device=dev)
        for s, n in zip(part, counts):
            w[s] = {"token": 1.0 / max(1, sum(counts)), "sequence": 1.0 / (len(part) * max(1, n)),
                    "sum": 1.0}[case["reduce"]]
        w = w * live
        adv, old = state["advantages"].double(), state["old_logp"].double()
        ratio = torch.exp(logp - old)
        surrogate = torch.minimum(ratio * adv, torch.clamp(ratio, 1 - CLIP_LOW, 1 + CLIP_HIGH) * adv)
        held = ((adv > 0) & (ratio > 1 + CLIP_HIGH)) | ((adv < 0) & (ratio < 1 - CLIP_LOW))
        slope = -(adv * ratio) * ~held
        kl = torch.zeros_like(slope)
        if case["beta"]:
            gap = state["ref_logp"].double() - logp
            kl = torch.expm1(gap) - gap
            slope = slope - case["beta"] * torch.expm1(gap)
        slope = slope * w
        stats = torch.stack([(w * (case["beta"] * kl - surrogate)).sum(), -(w * surrogate).sum(), (w * kl).sum(),
                             (w * held).sum()])
        answer = dict(stats=stats, logp=logp)
    else:
        P = case["pairs"]
        per = [max(1, n) if case["mean"] else 1 for n in counts]
        sums = torch.stack([logp[s].sum() / n for s, n in zip(part, per)])
        gain = sums - state["ref_logp"].double()
        margins = case["beta"] * (gain[:P] - gain[P:])
        up = torch.nn.functional.logsigmoid
        e = case["smooth"]
        loss = -((1 - e) * up(margins) + e * up(-margins)).sum() / P
        d = case["beta"] / P * (e * torch.sigmoid(margins) - (1 - e) * torch.sigmoid(-margins))
        for i, s in enumerate(part):
            slope[s] = (d[i] if i < P else -d[i - P]) / per[i]
        answer = dict(loss=loss.reshape(1), margins=margins, seq_logp=sums)
    grad = torch.zeros(T, case["vocab"], dtype=torch.float64, device=dev)
    for a in range(0, T, chunk):
        rows = slice(a, min(T, a + chunk))
        g = -torch.softmax(logits[rows].double() / tau, 1)
        g[torch.arange(g.shape[0], device=dev), y[rows]] += 1
        g *= (slope[rows] / tau)[:, None]
        grad[rows] = torch.where(live[rows, None], g, torch.zeros_like(g))
    answer["grad"] = grad
    return answer


def exact(case, seed):
    return _exact_clip(case, seed) if case["op"] == "clip" else _exact_rows(case, seed)
