"""The loss and clipping entry points: defaults, workspace sizes and refusals (no kernel runs)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_muon_gb300.build as b
    b.build()
    import newton_schulz_muon_gb300 as m
    return m


def test_defaults(nsm):
    p = nsm.muon_policy_config_default()
    assert (p.clip_low, p.clip_high, p.kl_beta, p.grad_scale) == pytest.approx((0.2, 0.2, 0.0, 1.0))
    assert p.reduction == nsm.MUON_REDUCE_TOKEN_MEAN
    q = nsm.muon_preference_config_default(label_smoothing=0.1)
    assert (q.beta, q.label_smoothing, q.grad_scale, q.length_normalize) == pytest.approx((0.1, 0.1, 1.0, 0))
    with pytest.raises(AttributeError):
        nsm.muon_policy_config_default(nothing=1)


def test_workspace_bytes(nsm):
    assert nsm.muon_loss_workspace_bytes(0, 0) >= 16
    assert nsm.muon_loss_workspace_bytes(1000, 8) > nsm.muon_loss_workspace_bytes(10, 8)
    for bad in ((-1, 0), (0, -1), (1 << 31, 0)):
        with pytest.raises(nsm.MuonError) as e:
            nsm.muon_loss_workspace_bytes(*bad)
        assert e.value.status == nsm.MUON_ERR_INVALID


def _grads(nsm, **over):
    base = dict(g=1 << 20, out=1 << 20, elems=100, count=1, stride_elems=0, dtype=0, out_dtype=0)
    base.update(over)
    arr = (nsm.muon_grad * 1)()
    arr[0] = tuple(base[k] for k in ("g", "out", "elems", "count", "stride_elems", "dtype", "out_dtype"))
    return arr


@pytest.mark.parametrize("over", [
    dict(elems=-1), dict(count=-1), dict(stride_elems=99, count=2), dict(dtype=2), dict(out_dtype=1), dict(g=0),
    dict(g=(1 << 20) + 2), dict(out=(1 << 21) + 1), dict(elems=1 << 41), dict(out=1 << 21, out_dtype=7)])
def test_clip_refuses_bad_tensors(nsm, over):
    st = nsm.lib.muon_clip_grad_norm(_grads(nsm, **over), 1, 1.0, 1e-6, 0, 1 << 22, 1 << 23, 1 << 20, None)
    assert st == nsm.MUON_ERR_INVALID


def test_clip_refuses_bad_arguments(nsm):
    call = nsm.lib.muon_clip_grad_norm
    g = _grads(nsm)
    inv, ws = nsm.MUON_ERR_INVALID, 1 << 23
    assert call(None, 1, 1.0, 1e-6, 0, 1 << 22, ws, 1 << 20, None) == inv
    assert call(g, -1, 1.0, 1e-6, 0, 1 << 22, ws, 1 << 20, None) == inv
    assert call(g, 1, -1.0, 1e-6, 0, 1 << 22, ws, 1 << 20, None) == inv
    assert call(g, 1, float("nan"), 1e-6, 0, 1 << 22, ws, 1 << 20, None) == inv
    assert call(g, 1, 1.0, -1e-6, 0, 1 << 22, ws, 1 << 20, None) == inv
    assert call(g, 1, 1.0, float("inf"), 0, 1 << 22, ws, 1 << 20, None) == inv
    assert call(g, 1, 1.0, 1e-6, 2, 1 << 22, ws, 1 << 20, None) == inv
    assert call(g, 1, 1.0, 1e-6, 0, None, ws, 1 << 20, None) == inv
    assert call(g, 1, 1.0, 1e-6, 0, 1 << 22, ws + 8, 1 << 20, None) == inv
    assert call(g, 1, 1.0, 1e-6, 0, 1 << 22, None, 1 << 20, None) == nsm.MUON_ERR_NO_WORKSPACE
    assert call(g, 1, 1.0, 1e-6, 0, 1 << 22, ws, 8, None) == nsm.MUON_ERR_NO_WORKSPACE
    size = ctypes.c_size_t()
    assert nsm.lib.muon_clip_workspace_bytes(g, 1, None) == inv
    assert nsm.lib.muon_clip_workspace_bytes(None, 0, ctypes.byref(size)) == nsm.MUON_OK and size.value > 0


def _batch(nsm, **over):
    base = dict(logits=1 << 20, targets=1 << 21, mask=0, tokens=4, vocab=10, row_stride=0, dtype=0, temperature=1.0)
    base.update(over)
    return nsm.muon_token_batch(*[base[k] for k in ("logits", "targets", "mask", "tokens", "vocab", "row_stride",
                                                    "temperature", "dtype")])


def _policy(nsm, batch=None, cfg=None, old=1 << 22, ref=0, adv=1 << 22, offsets=0, n_seqs=0, stats=1 << 22, logp=0,
            grad=1 << 23, grad_stride=0, ws=1 << 24, nbytes=1 << 20):
    b = batch or _batch(nsm)
    return nsm.lib.muon_policy_loss(ctypes.byref(b), None if cfg is None else ctypes.byref(cfg), old, ref, adv,
                                    offsets, n_seqs, stats, logp, grad, grad_stride, ws, nbytes, None)


BAD_BATCHES = [dict(tokens=-1), dict(tokens=1 << 31), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(row_stride=9),
               dict(dtype=2), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
               dict(temperature=float("inf")), dict(logits=0), dict(targets=0), dict(logits=(1 << 20) + 2),
               dict(targets=(1 << 21) + 4)]


@pytest.mark.parametrize("over", BAD_BATCHES)
def test_bad_batches_are_refused(nsm, over):
    b = _batch(nsm, **over)
    assert nsm.lib.muon_token_logprobs(ctypes.byref(b), 1 << 22, None) == nsm.MUON_ERR_INVALID
    assert _policy(nsm, b) == nsm.MUON_ERR_INVALID
    assert nsm.lib.muon_preference_loss(ctypes.byref(b), None, 1 << 22, 1 << 22, 1, 1 << 22, 0, 0, 0, 0, 1 << 24,
                                        1 << 20, None) == nsm.MUON_ERR_INVALID


def test_null_batch_and_outputs_are_refused(nsm):
    assert nsm.lib.muon_token_logprobs(None, 1 << 22, None) == nsm.MUON_ERR_INVALID
    b = _batch(nsm)
    assert nsm.lib.muon_token_logprobs(ctypes.byref(b), None, None) == nsm.MUON_ERR_INVALID
    assert nsm.lib.muon_token_logprobs(ctypes.byref(b), (1 << 22) + 2, None) == nsm.MUON_ERR_INVALID
    assert nsm.lib.muon_token_logprobs(ctypes.byref(_batch(nsm, tokens=0)), None, None) == nsm.MUON_OK


@pytest.mark.parametrize("cfg", [dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_high=-0.1),
                                 dict(kl_beta=float("nan")), dict(grad_scale=float("inf")), dict(reduction=3),
                                 dict(reduction=-1), dict(kl_beta=0.1), dict(reduction=1)])
def test_bad_policy_configurations_are_refused(nsm, cfg):
    # the last two: a KL term without ref_logp, a sequence mean without sequences
    assert _policy(nsm, cfg=nsm.muon_policy_config_default(**cfg)) == nsm.MUON_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(old=0), dict(adv=0), dict(stats=0), dict(old=(1 << 22) + 2), dict(grad_stride=9),
                                dict(grad=(1 << 23) + 2), dict(n_seqs=-1), dict(logp=(1 << 22) + 1),
                                dict(grad=1 << 20, grad_stride=16), dict(ws=(1 << 24) + 4)])
def test_bad_policy_arguments_are_refused(nsm, kw):
    assert _policy(nsm, **kw) == nsm.MUON_ERR_INVALID


def test_small_workspaces_are_refused(nsm):
    assert _policy(nsm, ws=0) == nsm.MUON_ERR_NO_WORKSPACE
    assert _policy(nsm, nbytes=nsm.muon_loss_workspace_bytes(4, 0) - 1) == nsm.MUON_ERR_NO_WORKSPACE


@pytest.mark.parametrize("cfg", [dict(beta=0.0), dict(beta=float("inf")), dict(label_smoothing=-0.1),
                                 dict(label_smoothing=1.1), dict(grad_scale=float("nan")), dict(length_normalize=2)])
def test_bad_preference_configurations_are_refused(nsm, cfg):
    b = _batch(nsm)
    c = nsm.muon_preference_config_default(**cfg)
    assert nsm.lib.muon_preference_loss(ctypes.byref(b), ctypes.byref(c), 1 << 22, 1 << 22, 1, 1 << 22, 0, 0, 0, 0,
                                        1 << 24, 1 << 20, None) == nsm.MUON_ERR_INVALID


@pytest.mark.parametrize("ref,offsets,pairs,loss", [(0, 1 << 22, 1, 1 << 22), (1 << 22, 0, 1, 1 << 22),
                                                    (1 << 22, 1 << 22, -1, 1 << 22), (1 << 22, 1 << 22, 1, 0),
                                                    (1 << 22, (1 << 22) + 4, 1, 1 << 22)])
def test_bad_preference_arguments_are_refused(nsm, ref, offsets, pairs, loss):
    b = _batch(nsm)
    assert nsm.lib.muon_preference_loss(ctypes.byref(b), None, ref, offsets, pairs, loss, 0, 0, 0, 0, 1 << 24,
                                        1 << 20, None) == nsm.MUON_ERR_INVALID


def test_python_checks_need_no_gpu(nsm):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 10)
    with pytest.raises(ValueError):
        nsm.muon_token_logprobs(x, torch.zeros(4, dtype=torch.int64))     # not on a GPU
    with pytest.raises(ValueError):
        nsm.GradSet([x])
    with pytest.raises(ValueError):
        nsm.GradSet([], [x])


@pytest.mark.parametrize("make,want", [
    (lambda t: t.empty(6, 8, 4), (192, 1, 0)),
    (lambda t: t.empty(6, 8, 4).permute(1, 2, 0), (192, 1, 0)),
    (lambda t: t.empty(6, 8, 4)[:, 2:5], (12, 6, 32)),
    (lambda t: t.empty(3, 4, 10)[:, :, :8], (8, 12, 10)),
    (lambda t: t.empty(5, 0, 2), (0, 1, 0)),
    (lambda t: t.empty(()), (1, 1, 0)),
    (lambda t: t.empty(20)[::2], (1, 10, 2)),
])
def test_gradient_layouts(nsm, make, want):
    torch = pytest.importorskip("torch")
    assert nsm._blocks(make(torch)) == want


@pytest.mark.parametrize("make", [lambda t: t.empty(5, 1).expand(5, 4), lambda t: t.empty(4, 4)[::2, ::2],
                                  lambda t: t.empty(10).as_strided((3, 4), (2, 1))])
def test_overlapping_or_scattered_gradients_are_refused(nsm, make):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        nsm._blocks(make(torch))


class _TwoDevices:
    """Two devices of a GPU machine, on the CPU: tensors carry the index that they would have,
    and library calls note the device that was current."""

    def __init__(self, nsm, torch, patch):
        self.torch, self.current, self.calls, self.made, self.index = torch, 0, [], [], {}
        owner, empty, strided = self, torch.empty, torch.empty_strided

        def home(make):
            def made(*size, device=None, **kw):
                owner.made.append(owner.current if device is None else int(getattr(device, "index", device)))
                return owner.put(make(*size, **kw), owner.made[-1])
            return made

        class device:
            def __init__(self, index):
                self.index = index

            def __enter__(self):
                self.before, owner.current = owner.current, self.index

            def __exit__(self, *_):
                owner.current = self.before

        class Stream:
            def __init__(self, index):
                self.cuda_stream, self.device_index, self.device = 0x77, index, type("D", (), {"index": index})

        class library:
            def __getattr__(self, name):
                if name.endswith("_bytes"):
                    return lambda *a: 0
                return lambda *a: owner.calls.append((name, owner.current)) or 0

        patch.setattr(nsm, "_lib", lambda: library())
        patch.setattr(nsm, "_SPACES", type("S", (), {})())
        patch.setattr(torch.Tensor, "get_device", lambda t: owner.of(t), raising=False)
        patch.setattr(torch.Tensor, "is_cuda", property(lambda t: owner.of(t) >= 0), raising=False)
        patch.setattr(torch.Tensor, "device", property(lambda t: type("D", (), {"index": owner.of(t)})), raising=False)
        patch.setattr(torch, "empty", home(empty))
        patch.setattr(torch, "empty_strided", home(strided))
        patch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
        patch.setattr(torch.cuda, "current_device", lambda: owner.current)
        patch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        patch.setattr(torch.cuda, "device", device)
        patch.setattr(torch.cuda, "Stream", Stream)
        patch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: Stream(owner.current if device is None else device))
        patch.setattr(torch.cuda, "stream", lambda s: device(s.device_index))
        self.stream, self.keep = Stream, []

    def put(self, t, device):
        self.index[t.untyped_storage().data_ptr()] = device
        self.keep.append(t)
        return t

    def of(self, t):
        return self.index.get(t.untyped_storage().data_ptr(), -1)   # a view's is its base's

    def batch(self, device, tokens=4, vocab=10):
        t = self.torch
        return (self.put(t.zeros(tokens, vocab), device), self.put(t.zeros(tokens, dtype=t.int64), device),
                self.put(t.zeros(tokens), device), self.put(t.tensor([0, 2, 4]), device), self.put(t.zeros(2), device))


def _calls(nsm, fake, device):
    """name -> (call, the tensors it takes by name), all on `device`"""
    t, put = fake.torch, fake.put
    z, y, f, off, two = fake.batch(device)
    mask, grad = put(t.ones(4, dtype=t.bool), device), put(t.zeros(4, 10), device)
    ws = put(t.zeros(1 << 16, dtype=t.uint8), device)
    one, four = put(t.zeros(1), device), put(t.zeros(4), device)
    return {
        "logprobs": (lambda **kw: nsm.muon_token_logprobs(**{**dict(logits=z, targets=y, mask=mask, logp=f), **kw}),
                     dict(targets=y, mask=mask, logp=f)),
        "policy": (lambda **kw: nsm.muon_policy_loss(**{**dict(
            logits=z, targets=y, old_logp=f, advantages=f, mask=mask, ref_logp=f, seq_offsets=off, grad=grad, logp=f,
            stats=four, workspace=ws), **kw}),
            dict(targets=y, old_logp=f, advantages=f, mask=mask, ref_logp=f, seq_offsets=off, grad=grad, logp=f,
                 stats=four, workspace=ws)),
        "preference": (lambda **kw: nsm.muon_preference_loss(**{**dict(
            logits=z, targets=y, seq_offsets=off, ref_logp=two, mask=mask, grad=grad, loss=one, margins=one,
            seq_logp=two, workspace=ws), **kw}),
            dict(targets=y, seq_offsets=off, ref_logp=two, mask=mask, grad=grad, loss=one, margins=one, seq_logp=two,
                 workspace=ws)),
        "norm": (lambda **kw: nsm.muon_grad_norm(**{**dict(grads=[z], norm=one, workspace=ws), **kw}),
                 dict(norm=one, workspace=ws)),
        "clip": (lambda **kw: nsm.muon_clip_grad_norm(**{**dict(grads=[z], max_norm=1.0, result=two, workspace=ws), **kw}),
                 dict(result=two, workspace=ws)),
    }


CALLS = ["logprobs", "policy", "preference", "norm", "clip"]


@pytest.mark.parametrize("which", CALLS)
@pytest.mark.parametrize("stream", [None, "object", "handle"])
@pytest.mark.parametrize("device", [0, 1])
def test_calls_launch_on_their_tensors_device(nsm, monkeypatch, which, stream, device):
    """What a call allocates and launches belongs to the tensors' device, whichever is current."""
    fake = _TwoDevices(nsm, pytest.importorskip("torch"), monkeypatch)
    call, named = _calls(nsm, fake, device)[which]
    with_stream = {} if stream is None else dict(stream=fake.stream(device) if stream == "object" else 0x77)
    call(**with_stream)
    call(**with_stream, **{k: None for k in named if k in ("logp", "stats", "grad", "loss", "margins", "seq_logp",
                                                           "norm", "result", "workspace")})
    assert [d for _, d in fake.calls] == [device] * len(fake.calls) and fake.calls
    assert fake.made and set(fake.made) == {device} and fake.current == 0


@pytest.mark.parametrize("which", CALLS)
def test_tensors_of_another_device_are_refused(nsm, monkeypatch, which):
    fake = _TwoDevices(nsm, pytest.importorskip("torch"), monkeypatch)
    call, named = _calls(nsm, fake, 0)[which]
    for name, t in named.items():
        elsewhere = fake.put(t.clone(), 1)
        with pytest.raises(ValueError, match=name):
            call(**{name: elsewhere})
    with pytest.raises(ValueError, match="stream"):
        call(stream=fake.stream(1))
    assert fake.calls == []
