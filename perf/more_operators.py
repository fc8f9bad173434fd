"""The operators on both sides of a fine-tuning step: sampling tokens and verifying drafted
ones against the target's probabilities (what a policy is trained on), activation
checkpoints in 8 bits and the backward pass that reads them (where its gradients come from).

Each case is one call, or the calls that belong to one pass, as a training or sampling
program makes it.  `run` computes it with elementary torch operations in fp32, or, with
`own` set, through the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32     # consecutive columns of a checkpoint's row that share one power of two
SPREAD = 2.5   # standard deviation of a row's logits


def listed():
    return [
        # the next token of one sequence: nothing but latency
        dict(name="sample_one_token", op="sample", tokens=1, vocab=131072, dtype="bf16", pad=0, drop=0.0, temp=1.0),
        # one decoding step of a large rollout batch, some of its sequences finished
        dict(name="sample_batch", op="sample", tokens=2048, vocab=131072, dtype="bf16", pad=0, drop=0.1, temp=0.8),
        # four drafted tokens of one sequence
        dict(name="verify_one_sequence", op="verify", seqs=1, most=4, even=True, vocab=131072, dtype="bf16", pad=0,
             temp=1.0, noise=0.5, draft="logp"),
        # a few sequences with drafts of their own lengths, fp32 logits of an odd vocabulary in
        # padded rows; the drafts' probabilities come from the draft model's logits
        dict(name="verify_ragged", op="verify", seqs=37, most=7, even=False, vocab=50001, dtype="f32", pad=3, temp=0.7,
             noise=0.8, draft="logits"),
        # one verification step of a rollout batch
        dict(name="verify_batch", op="verify", seqs=512, most=4, even=True, vocab=131072, dtype="bf16", pad=0,
             temp=1.0, noise=0.5, draft="logp"),
        # the activations of a few tokens, saved and read back
        dict(name="checkpoint_short", op="checkpoint", tokens=131, cols=1000, dtype="f32", pad=0),
        # the widest activations of one layer
        dict(name="checkpoint_layer", op="checkpoint", tokens=16384, cols=9728, dtype="bf16", pad=0),
        # a small layer's weight gradient
        dict(name="weight_small", op="weight", tokens=1024, more=0, outs=512, cols=128, dtype="bf16", out="bf16", pad=0),
        # fp32 gradients of odd sizes in padded rows, over two micro-batches
        dict(name="weight_ragged", op="weight", tokens=1003, more=517, outs=2005, cols=1537, dtype="f32", out="f32",
             pad=3),
        # the weight gradient of one up projection, as the step reads it
        dict(name="weight_layer", op="weight", tokens=8192, more=0, outs=9728, cols=2560, dtype="bf16", out="f32", pad=0),
        # a gated activation of few tokens, forward and backward
        dict(name="gated_short", op="gated", tokens=67, cols=1003, dtype="f32", fused=False),
        # one layer's gated activation, gate and up halves of one matrix
        dict(name="gated_layer", op="gated", tokens=8192, cols=9728, dtype="bf16", fused=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["sample", "verify", "verify", "checkpoint", "weight", "weight", "gated"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 5, 64]))
    if op == "sample":
        vocab = spread(500, 160000)
        case.update(vocab=vocab, tokens=spread(1, max(2, min(4096, 268000000 // vocab // 2))),
                    drop=rng.choice([0.0, 0.1, 0.4]), temp=rng.choice([1.0, 1.0, 0.6]))
    elif op == "verify":
        vocab = spread(500, 160000)
        most = rng.randint(1, 8)
        rows = 268000000 // vocab // 2
        case.update(vocab=vocab, most=most, seqs=spread(1, max(2, min(1024, rows // (2 * most + 1)))),
                    even=rng.choice([True, False]), temp=rng.choice([1.0, 1.0, 0.6]), noise=rng.choice([0.2, 0.5, 1.0]),
                    draft=rng.choice(["logp", "logp", "logits", "certain"]))
    elif op == "weight":
        outs, cols = spread(1, 9728), spread(1, 9728)
        # fp32 gradients count as three of bf16
        rows = (8192 * 9728 * 2560 if case["dtype"] == "bf16" else 8192 * 9728 * 853) // (outs * cols)
        first = spread(1, max(2, min(16384, rows // 2)))
        more = 0 if rng.random() < 0.6 else spread(1, first + 1)   # a second micro-batch
        case.update(tokens=first, more=more, outs=outs, cols=cols, out=rng.choice(["bf16", "f32"]))
    else:
        cols = spread(16, 9728)
        case.update(tokens=spread(1, min(16384, (16384 if op == "checkpoint" else 8192) * 9728 // 2 // cols)), cols=cols)
        if op == "gated":
            case.update(fused=rng.choice([True, False]))
            del case["pad"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _logits(rows, case, gen):
    """Logits of a language model: a normal background and a likely next token."""
    V, tau = case["vocab"], case["temp"]
    full = torch.randn(rows, V + case["pad"], generator=gen, device="cuda", dtype=DTYPES[case["dtype"]])
    logits = full.mul_(SPREAD * tau)[:, :V]
    likely = torch.randint(0, V, (rows,), generator=gen, device="cuda")
    level = math.log(V) + 0.5 * SPREAD ** 2
    value = (level + 1.5 * torch.randn(rows, 1, generator=gen, device="cuda")) * tau
    return logits.scatter_(1, likely[:, None], value.to(logits.dtype))


def _inside(weights, gen):
    """A uniform for each row of weights, in the middle of some token's share of [0, 1): a
    number that rounding could put on either side of a border is moved off it."""
    ends = weights.cumsum(1)
    total = ends[:, -1:]
    u = torch.rand(weights.shape[0], 1, generator=gen, device="cuda", dtype=torch.float64)
    # the first token from u on whose share is wide enough, else the widest
    wide = weights >= torch.minimum(8e-6 * total, weights.amax(1, keepdim=True))
    index = torch.arange(weights.shape[1], device="cuda")
    after = wide & (index >= (ends <= u * total).sum(1, keepdim=True))
    token = torch.where(after.any(1), after.int().argmax(1), wide.int().argmax(1))[:, None]
    return ((ends - 0.5 * weights).gather(1, token) / total).float()[:, 0]


def _probs(logits, temp):
    z = logits.double() / temp
    e = (z - z.amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True)


def _prepare_sample(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T = case["tokens"]
    logits = _logits(T, case, gen)
    mask = torch.rand(T, generator=gen, device="cuda") >= case["drop"]
    u = torch.cat([_inside(_probs(part, case["temp"]), gen) for part in logits.split(256)])
    return dict(case=case, logits=logits, uniforms=u, mask=mask)


def _lengths(case):
    """How many tokens were drafted for each sequence."""
    if case["even"]:
        return [case["most"]] * case["seqs"]
    rs = torch.Generator().manual_seed(case["seqs"])
    return torch.randint(0, case["most"] + 1, (case["seqs"],), generator=rs).tolist()


def _prepare_verify(case, seed):
    """The target's logits, and those of a draft model near it, which the drafts are sampled
    from.  A certain draft is one that the draft model gives with probability 1."""
    gen = torch.Generator("cuda").manual_seed(seed)
    S, tau = case["seqs"], case["temp"]
    lengths = torch.tensor(_lengths(case), device="cuda")
    offsets = torch.cat([torch.zeros_like(lengths[:1]), lengths.cumsum(0)])
    N = int(offsets[-1])
    target = _logits(N + S, case, gen)
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), lengths)
    rows = torch.arange(N, device="cuda") + seq
    state = dict(case=case, target=target, draft_offsets=offsets, draft_logits=None, draft_logp=None)
    drafts = torch.zeros(N, dtype=torch.int64, device="cuda")
    px, qx = torch.zeros(2, N, dtype=torch.float64, device="cuda")
    noisy = torch.empty(N, case["vocab"] + case["pad"], device="cuda", dtype=target.dtype)[:, :case["vocab"]]
    for part in torch.arange(N, device="cuda").split(256):
        p = _probs(target[rows[part]], tau)
        noise = torch.randn(p.shape, generator=gen, device="cuda") * (case["noise"] * tau)
        noisy[part] = (target[rows[part]] + noise).to(target.dtype)
        q = _probs(noisy[part], tau)
        x = torch.multinomial(q.float(), 1, generator=gen) if len(part) else drafts[:, None]
        drafts[part], px[part], qx[part] = x[:, 0], p.gather(1, x)[:, 0], q.gather(1, x)[:, 0]
    if case["draft"] == "certain":
        qx = torch.ones_like(qx)
    else:
        state["draft_logits"] = noisy
        if case["draft"] == "logp":
            state["draft_logp"] = qx.log().float()
    # a number that rounding could put on either side of p / q is moved off it
    u = torch.rand(N, generator=gen, device="cuda", dtype=torch.float64)
    ratio = px / qx
    u = torch.where((u - ratio).abs() < 1e-3, torch.where(ratio > 0.5, ratio - 4e-3, ratio + 4e-3), u).float()
    at = torch.arange(N, device="cuda") - offsets[seq]
    counts = lengths.scatter_reduce(0, seq, torch.where(u.double() < ratio, lengths[seq], at), "amin")
    sample = torch.empty(S, device="cuda")
    for part in torch.arange(S, device="cuda").split(256):
        r = _probs(target[offsets[part] + part + counts[part]], tau)
        if N:
            held = counts[part] < lengths[part]
            at = (offsets[part] + counts[part]).clamp(max=N - 1)
            if case["draft"] == "certain":
                q = torch.zeros_like(r).scatter_(1, drafts[at][:, None], 1.0)
            else:
                q = _probs(noisy[at], tau)
            r = torch.where(held[:, None], (r - q).clamp(min=0), r)
        sample[part] = _inside(r, gen)
    state.update(drafts=drafts, accept_uniforms=u, sample_uniforms=sample)
    return state


def _activations(rows, case, gen, cols=None):
    """[rows, cols]: features of their own sizes, a few of them far larger."""
    cols = cols or case["cols"]
    scale = (0.5 * torch.randn(cols, generator=gen, device="cuda")).exp()
    scale = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.003, 30 * scale, scale)
    full = torch.randn(rows, cols + case.get("pad", 0), generator=gen, device="cuda")
    full[:, :cols] *= scale
    return full.to(DTYPES[case["dtype"]])[:, :cols]


def _gradient(rows, cols, case, gen):
    full = torch.randn(rows, cols + case.get("pad", 0), generator=gen, device="cuda") * 1e-2
    return full.to(DTYPES[case["dtype"]])[:, :cols]


def _batches(case):
    return [case["tokens"], case["more"]] if case["more"] else [case["tokens"]]


def _prepare_weight(case, seed):
    """What the forward pass left: the checkpoint of each micro-batch's activations."""
    gen = torch.Generator("cuda").manual_seed(seed)
    parts = []
    for T in _batches(case):
        x = _activations(T, case, gen)
        parts.append((_plain_save(x), _gradient(T, case["outs"], case, gen)))
    return dict(case=case, parts=parts)


def _prepare_gated(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, C = case["tokens"], case["cols"]
    both = _activations(T, case, gen, 2 * C)
    gate, up = both[:, :C], both[:, C:]
    if not case["fused"]:
        gate, up = gate.contiguous(), up.contiguous()
    return dict(case=case, gate=gate, up=up, dh=_gradient(T, C, case, gen))


def prepare(case, seed):
    if case["op"] == "sample":
        return _prepare_sample(case, seed)
    if case["op"] == "verify":
        return _prepare_verify(case, seed)
    if case["op"] == "checkpoint":
        gen = torch.Generator("cuda").manual_seed(seed)
        return dict(case=case, x=_activations(case["tokens"], case, gen))
    return _prepare_weight(case, seed) if case["op"] == "weight" else _prepare_gated(case, seed)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _plain_save(x):
    """The checkpoint of x [rows, cols]: int8 values, rows padded to whole blocks, then one
    byte a block; a value stands for q 2^(byte - 133)."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = torch.zeros(rows, blocks * BLOCK, device=x.device)
    v[:, :cols] = x.float()
    v = v.view(rows, blocks, BLOCK)
    bits = v.abs().amax(2).view(torch.int32)
    # the smallest power of two for which the block's largest value rounds to 127 or less
    byte = ((bits + 0x10000) >> 23).clamp(7, 254)
    byte = torch.where((bits >= 0x7F800000) | v.isnan().any(2), 255, byte)
    inverse = ((260 - byte).clamp(min=1) << 23).view(torch.float32)
    q = (v * inverse[:, :, None]).round().clamp(-127, 127)
    q = torch.where(byte[:, :, None] == 255, 0.0, q).to(torch.int8)
    return torch.cat([q.view(torch.uint8).reshape(-1), byte.to(torch.uint8).reshape(-1)])


def _plain_load(data, rows, cols):
    """The values of a checkpoint, fp32."""
    blocks = -(-cols // BLOCK)
    q = data[:rows * blocks * BLOCK].view(torch.int8).view(rows, blocks, BLOCK)
    byte = data[rows * blocks * BLOCK:].view(rows, blocks).int()
    step = torch.where(byte == 255, math.nan, ((byte - 6).clamp(min=1) << 23).view(torch.float32))
    return (q.float() * step[:, :, None]).view(rows, blocks * BLOCK)[:, :cols]


def _plain_logp(logits, temp):
    x = logits.float() / temp
    x = x - x.amax(1, keepdim=True)
    return x - x.exp().sum(1, keepdim=True).log()


def _pick(weights, uniforms):
    """The first token whose cumulated weight exceeds the uniform's share of the whole."""
    ends = weights.cumsum(1)
    return (ends <= uniforms.double()[:, None] * ends[:, -1:]).sum(1).clamp(max=weights.shape[1] - 1)


def _plain_sample(state):
    case = state["case"]
    token = _pick(_probs(state["logits"], case["temp"]), state["uniforms"])
    logp = _plain_logp(state["logits"], case["temp"]).gather(1, token[:, None])[:, 0]
    return dict(tokens=torch.where(state["mask"], token, -1), logp=torch.where(state["mask"], logp, 0.0))


def _plain_verify(state):
    case, offsets, drafts = state["case"], state["draft_offsets"], state["drafts"]
    S, N, tau = case["seqs"], len(drafts), case["temp"]
    index = torch.arange(N, device="cuda")
    seq = torch.bucketize(index, offsets[1:], right=True)
    logp = _plain_logp(state["target"], tau)
    px = logp[index + seq].gather(1, drafts[:, None])[:, 0].exp()
    if case["draft"] == "logp":
        qx = state["draft_logp"].exp()
    elif case["draft"] == "logits":
        qx = _plain_logp(state["draft_logits"], tau).gather(1, drafts[:, None])[:, 0].exp()
    else:
        qx = torch.ones_like(px)
    lengths = offsets[1:] - offsets[:-1]
    accepted = state["accept_uniforms"] * qx < px
    counts = lengths.scatter_reduce(0, seq, torch.where(accepted, lengths[seq], index - offsets[seq]), "amin")
    # the token after the accepted ones: from what the target gives more than the draft model
    # where a draft was rejected, else from the target's row after the drafts
    first = offsets[:-1] + torch.arange(S, device="cuda")
    weights = _probs(state["target"][first + counts], tau)
    if N:
        at = (offsets[:-1] + counts).clamp(max=N - 1)
        if case["draft"] == "certain":
            q = torch.zeros_like(weights).scatter_(1, drafts[at][:, None], 1.0)
        else:
            q = _probs(state["draft_logits"][at], tau)
        left = (weights - q).clamp(min=0)
        left = torch.where((counts < lengths)[:, None], left, weights)
        weights = torch.where(left.sum(1, keepdim=True) > 0, left, weights)
    token = _pick(weights, state["sample_uniforms"])
    row_seq = torch.bucketize(torch.arange(N + S, device="cuda"), first + lengths + 1, right=True)
    at = torch.arange(N + S, device="cuda") - first[row_seq]
    tokens = torch.full((N + S,), -1, device="cuda")
    tokens[index + seq] = drafts
    tokens = torch.where(at < counts[row_seq], tokens, torch.where(at == counts[row_seq], token[row_seq], -1))
    taken = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    return dict(tokens=tokens, counts=counts, logp=torch.where(tokens >= 0, taken, 0.0))


def _plain_weight(state):
    case = state["case"]
    total = torch.zeros(case["outs"], case["cols"], device="cuda")
    for data, dy in state["parts"]:
        total += dy.float().t() @ _plain_load(data, dy.shape[0], case["cols"])
    return total.to(DTYPES[case["out"]])


def _plain_gated(state):
    gate, up, dtype = state["gate"].float(), state["up"].float(), state["gate"].dtype
    h = gate / (1 + (-gate).exp()) * up
    saved = [_plain_save(state["gate"]), _plain_save(state["up"])]
    # the backward pass, from the checkpoints
    gate, up = (_plain_load(data, *gate.shape) for data in saved)
    dh = state["dh"].float()
    sig = 1 / (1 + (-gate).exp())
    dgate = dh * up * sig * (1 + gate * (1 - sig))
    dup = dh * gate * sig
    return dict(h=h.to(dtype), dgate=dgate.to(dtype), dup=dup.to(dtype), again=(gate * sig * up).to(dtype))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(state):
    import newton_schulz_muon_gb300 as nsm

    case = state["case"]
    if case["op"] == "sample":
        tokens, logp = nsm.muon_sample_tokens(state["logits"], state["uniforms"], mask=state["mask"],
                                              temperature=case["temp"])
        return dict(tokens=tokens, logp=logp)
    if case["op"] == "verify":
        tokens, counts, logp = nsm.muon_verify_drafts(
            state["target"], state["drafts"], state["draft_offsets"], state["accept_uniforms"],
            state["sample_uniforms"], draft_logits=state["draft_logits"], draft_logp=state["draft_logp"],
            temperature=case["temp"])
        return dict(tokens=tokens, counts=counts, logp=logp)
    if case["op"] == "checkpoint":
        saved = nsm.muon_checkpoint_save(state["x"])
        return dict(x=nsm.muon_checkpoint_load(saved, dtype=state["x"].dtype))
    if case["op"] == "weight":
        out = None
        for data, dy in state["parts"]:
            saved = nsm.Checkpoint(dy.shape[0], case["cols"], data)
            out = nsm.muon_checkpoint_weight_grad(saved, dy, out=out, accumulate=out is not None,
                                                  dtype=torch.float32 if len(state["parts"]) > 1 else DTYPES[case["out"]])
        return out.to(DTYPES[case["out"]])
    h, *saved = nsm.muon_swiglu_forward(state["gate"], state["up"])
    dgate, dup, again = nsm.muon_swiglu_backward(state["dh"], *saved, with_h=True)
    return dict(h=h, dgate=dgate, dup=dup, again=again)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "sample":
        return _plain_sample(state)
    if op == "verify":
        return _plain_verify(state)
    if op == "checkpoint":
        x = state["x"]
        return dict(x=_plain_load(_plain_save(x), *x.shape).to(x.dtype))
    return _plain_weight(state) if op == "weight" else _plain_gated(state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    saved = 1 + 1 / BLOCK                # bytes of a checkpoint's element
    if case["op"] == "sample":
        live = case["tokens"] * (1 - case["drop"])
        return {"bytes": live * case["vocab"] * es + case["tokens"] * (4 + 1 + 8 + 4), "flops": 4 * live * case["vocab"]}
    if case["op"] == "verify":
        # a row is needed where the drafts before it were accepted, each with probability
        # sum min(p, q); the draft model's row only where its draft was rejected, or for its
        # probability where that is not given
        S, V, lengths = case["seqs"], case["vocab"], _lengths(case)
        if case["draft"] == "certain":
            a = 0.3                      # sum p q: mostly the likely token's p q
        else:
            a = math.erfc(case["noise"] / (2 * math.sqrt(2)))
        target = sum(a ** i for n in lengths for i in range(n + 1))
        passed = sum(a ** n for n in lengths)
        rows = target + {"logp": S - passed, "certain": 0, "logits": target - passed}[case["draft"]]
        return {"bytes": rows * V * es + sum(lengths) * (8 + 4 + 4 + 8 + 4) + S * (8 + 4 + 8 + 8 + 4),
                "flops": 4 * rows * V}
    if case["op"] == "weight":
        rows = sum(_batches(case))
        return {"bytes": rows * (case["outs"] * es + case["cols"] * saved)
                + case["outs"] * case["cols"] * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * rows * case["outs"] * case["cols"]}
    elems = case["tokens"] * case["cols"]
    if case["op"] == "checkpoint":
        # saved: x read, the checkpoint written; loaded: the checkpoint read, x written
        return {"bytes": elems * 2 * (es + saved), "flops": 4 * elems}
    # forward: gate and up read, h and two checkpoints written; backward: dh and two
    # checkpoints read, three matrices written
    return {"bytes": elems * (7 * es + 4 * saved), "flops": 30 * elems}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_row(logits, temp):
    return torch.log_softmax(logits.to(torch.float64) / temp, -1)


def _exact_pick(weights, u):
    ends = torch.cumsum(weights, -1)
    # the first index whose cumulated weight is above the threshold
    return int(torch.searchsorted(ends, ends[-1:] * u, right=True).clamp(max=len(ends) - 1))


def _exact_sample(case, seed):
    state = _prepare_sample(case, seed)
    tokens, logps = [], []
    for row, u, live in zip(state["logits"], state["uniforms"].double(), state["mask"].tolist()):
        if not live:
            tokens.append(-1)
            logps.append(row.new_zeros((), dtype=torch.float64))
            continue
        logp = _exact_row(row, case["temp"])
        tokens.append(_exact_pick(logp.exp(), u))
        logps.append(logp[tokens[-1]])
    return dict(tokens=torch.tensor(tokens, device="cuda"), logp=torch.stack(logps))


def _exact_verify(case, seed):
    state = _prepare_verify(case, seed)
    offsets, tau = state["draft_offsets"].tolist(), case["temp"]
    drafts, accept = state["drafts"].tolist(), state["accept_uniforms"].tolist()
    tokens, counts, logps = [], [], []
    for s in range(case["seqs"]):
        lo, hi = offsets[s], offsets[s + 1]
        taken, weights = 0, None
        for d in range(lo, hi):
            logp = _exact_row(state["target"][d + s], tau)
            if case["draft"] == "certain":
                q = torch.zeros_like(logp)
                q[drafts[d]] = 1
                qx = 1.0
            else:
                q = _exact_row(state["draft_logits"][d], tau).exp()
                qx = float(q[drafts[d]] if case["draft"] == "logits" else state["draft_logp"][d].double().exp())
            if not accept[d] * qx < float(logp[drafts[d]].exp()):
                weights = torch.relu(logp.exp() - q)
                if float(weights.sum()) == 0:
                    weights = logp.exp()
                break
            tokens.append(drafts[d])
            logps.append(logp[drafts[d]])
            taken += 1
        if weights is None:
            logp = _exact_row(state["target"][hi + s], tau)
            weights = logp.exp()
        tokens.append(_exact_pick(weights, state["sample_uniforms"][s].double()))
        logps.append(logp[tokens[-1]])
        counts.append(taken)
        tokens += [-1] * (hi - lo - taken)
        logps += [logp.new_zeros(())] * (hi - lo - taken)
    return dict(tokens=torch.tensor(tokens, device="cuda"), counts=torch.tensor(counts, device="cuda"),
                logp=torch.stack(logps))


def _exact_values(x):
    """What an 8-bit checkpoint of x stands for: in each block of a row, multiples of the
    smallest power of two (no smaller than 2^-126) of which 127 or fewer reach the largest."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for a in range(0, x.shape[1], BLOCK):
        v = x[:, a:a + BLOCK].double()
        most = v.abs().max(1, keepdim=True).values
        mantissa, exponent = torch.frexp(most)       # most = mantissa 2^exponent, mantissa in [1/2, 1)
        power = exponent - 7 + (mantissa * 128 >= 127.5)
        power = torch.where(most == 0, -126, power.clamp(-126, 121)).long()
        step = (power + 1023 << 52).view(torch.float64)   # 2^power
        out[:, a:a + BLOCK] = torch.clamp(torch.round(v / step), -127, 127) * step
    return out


def _exact_weight(case, seed):
    # the same inputs: the activations whose checkpoints `prepare` makes
    gen = torch.Generator("cuda").manual_seed(seed)
    total = torch.zeros(case["outs"], case["cols"], dtype=torch.float64, device="cuda")
    for T in _batches(case):
        x = _activations(T, case, gen)
        dy = _gradient(T, case["outs"], case, gen)
        total.addmm_(dy.double().t(), _exact_values(x))
    return total


def _exact_gated(case, seed):
    state = _prepare_gated(case, seed)
    silu = torch.nn.functional.silu
    h = silu(state["gate"].double()) * state["up"].double()
    gate, up, dh = _exact_values(state["gate"]), _exact_values(state["up"]), state["dh"].double()
    slope = torch.sigmoid(gate) + silu(gate) * torch.sigmoid(-gate)
    return dict(h=h, dgate=dh * up * slope, dup=dh * silu(gate), again=silu(gate) * up)


def exact(case, seed):
    if case["op"] == "sample":
        return _exact_sample(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, seed)
    if case["op"] == "checkpoint":
        return dict(x=_exact_values(prepare(case, seed)["x"]))
    return _exact_weight(case, seed) if case["op"] == "weight" else _exact_gated(case, seed)
