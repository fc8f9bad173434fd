"""The sampling and checkpoint calls on tensors of another device than the current one, and on
streams, with fake devices (no kernel runs)."""
import gc

import pytest

from test_abi_losses_cpu import _TwoDevices


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_muon_gb300.build as b
    b.build()
    import newton_schulz_muon_gb300 as m
    return m


@pytest.fixture
def fake(nsm, monkeypatch):
    gc.collect()   # other tests' plans go through the library that they were made by
    two = _TwoDevices(nsm, pytest.importorskip("torch"), monkeypatch)
    monkeypatch.setattr(nsm, "muon_checkpoint_bytes", lambda rows, cols: 64)
    monkeypatch.setattr(nsm, "muon_sample_workspace_bytes", lambda *a: 512)
    monkeypatch.setattr(nsm, "muon_weight_grad_workspace_bytes", lambda *a: 1024)
    return two


def _calls(nsm, fake, device):
    """name -> (call, the tensors it takes by name, those that it makes where they are left out)"""
    t = fake.torch
    put = lambda x: fake.put(x, device)   # noqa: E731
    z, zd, u, su = (put(t.zeros(6, 10)), put(t.zeros(4, 10)), put(t.zeros(4)), put(t.zeros(2)))
    i6, i4, i3, i2 = (put(t.zeros(n, dtype=t.int64)) for n in (6, 4, 3, 2))
    u6, f6, mask = put(t.zeros(6)), put(t.zeros(6)), put(t.ones(6, dtype=t.bool))
    ws = put(t.zeros(1 << 12, dtype=t.uint8))
    ck, other = (nsm.Checkpoint(6, 10, put(t.zeros(64, dtype=t.uint8))) for _ in range(2))
    x, y, h, g1, g2, dw = (put(t.zeros(6, 10)) for _ in range(6))

    def call(f, made, **base):
        return lambda **kw: f(**{**base, **kw}), {k: v for k, v in base.items() if k != "accumulate"}, made

    return {
        "sample": call(nsm.muon_sample_tokens, ("tokens", "logp", "workspace"), logits=z, uniforms=u6, mask=mask, tokens=i6,
                       logp=f6, workspace=ws),
        "verify": call(nsm.muon_verify_drafts, ("tokens", "counts", "logp", "workspace"), logits=z, drafts=i4,
                       draft_offsets=i3, accept_uniforms=u, sample_uniforms=su, draft_logits=zd, draft_logp=put(t.zeros(4)),
                       tokens=i6, counts=i2, logp=f6, workspace=ws),
        "save": call(nsm.muon_checkpoint_save, ("checkpoint",), x=x, checkpoint=ck),
        "load": call(nsm.muon_checkpoint_load, ("out",), checkpoint=ck, out=x),
        "weight": call(nsm.muon_checkpoint_weight_grad, ("out", "workspace"), checkpoint=ck, dy=y,
                       out=put(t.zeros(10, 10)), workspace=ws),
        "gated": call(nsm.muon_swiglu_forward, ("h", "gate_checkpoint", "up_checkpoint"), gate=x, up=y, h=h,
                      gate_checkpoint=ck, up_checkpoint=other),
        "gated_back": call(nsm.muon_swiglu_backward, ("dgate", "dup", "h"), dh=x, gate_checkpoint=ck, up_checkpoint=other,
                           dgate=g1, dup=g2, h=dw),
    }


CALLS = ["sample", "verify", "save", "load", "weight", "gated", "gated_back"]


@pytest.mark.parametrize("which", CALLS)
@pytest.mark.parametrize("stream", [None, "object", "handle"])
@pytest.mark.parametrize("device", [0, 1])
def test_calls_launch_on_their_tensors_device(nsm, fake, which, stream, device):
    """What a call allocates and launches belongs to the tensors' device, whichever is current."""
    call, named, made = _calls(nsm, fake, device)[which]
    with_stream = {} if stream is None else dict(stream=fake.stream(device) if stream == "object" else 0x77)
    call(**with_stream)
    call(**with_stream, **{k: None for k in made})
    assert [d for _, d in fake.calls] == [device] * 2
    assert fake.made and set(fake.made) == {device} and fake.current == 0


@pytest.mark.parametrize("which", CALLS)
def test_tensors_of_another_device_are_refused(nsm, fake, which):
    call, named, _ = _calls(nsm, fake, 0)[which]
    first = next(iter(named))   # the one whose device counts
    for name, t in named.items():
        if name == first:
            continue
        if isinstance(t, nsm.Checkpoint):
            elsewhere = nsm.Checkpoint(t.rows, t.cols, fake.put(t.data.clone(), 1))
        else:
            elsewhere = fake.put(t.clone(), 1)
        with pytest.raises(ValueError, match=name):
            call(**{name: elsewhere})
    with pytest.raises(ValueError, match="stream"):
        call(stream=fake.stream(1))
    assert fake.calls == []
