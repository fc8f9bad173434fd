"""The sampling and verification entry points: refusals (no kernel runs)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_muon_gb300.build as b
    b.build()
    import newton_schulz_muon_gb300 as m
    return m


A = 1 << 20


def _batch(nsm, **over):
    base = dict(logits=A, targets=A, mask=None, tokens=6, vocab=100, row_stride=0, temperature=1.0, dtype=0)
    base.update(over)
    return nsm.muon_token_batch(*[base[k] for k in ("logits", "targets", "mask", "tokens", "vocab", "row_stride",
                                                    "temperature", "dtype")])


@pytest.mark.parametrize("over", [
    dict(tokens=-1), dict(tokens=1 << 31), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(row_stride=99), dict(dtype=2),
    dict(temperature=0.0), dict(temperature=float("nan")), dict(temperature=1e21), dict(logits=None),
    dict(logits=A + 2), dict(logits=A + 1, dtype=1)])
def test_sample_refuses_bad_batches(nsm, over):
    b = _batch(nsm, **over)
    assert nsm.lib.muon_sample_tokens(ctypes.byref(b), A, A, A, A, 1 << 40, None) == nsm.MUON_ERR_INVALID


def test_sample_refuses_bad_arguments(nsm):
    call, b = nsm.lib.muon_sample_tokens, _batch(nsm)
    ref = ctypes.byref(b)
    assert call(None, A, A, A, A, 1 << 40, None) == nsm.MUON_ERR_INVALID
    for args in ((None, A, A), (A, None, A), (A, A, None), (A + 2, A, A), (A, A + 4, A), (A, A, A + 1)):
        assert call(ref, *args, A, 1 << 40, None) == nsm.MUON_ERR_INVALID
    assert call(ref, A, A, A, None, 1 << 40, None) == nsm.MUON_ERR_NO_WORKSPACE
    assert call(ref, A, A, A, A, 5, None) == nsm.MUON_ERR_NO_WORKSPACE
    assert call(ref, A, A, A, A + 8, 1 << 40, None) == nsm.MUON_ERR_INVALID
    empty = _batch(nsm, tokens=0, logits=None)
    assert call(ctypes.byref(empty), None, None, None, None, 0, None) == nsm.MUON_OK


def _verify(nsm, target=None, draft=None, n_seqs=2, draft_logp=None, offsets=A, accept=A, sample=A, tokens=A, counts=A,
            logp=A, ws=A, nbytes=1 << 40):
    t = _batch(nsm, **{"targets": None, **(target or {})})
    d = _batch(nsm, **{"tokens": 4, **(draft or {})})
    return nsm.lib.muon_verify_drafts(ctypes.byref(t), ctypes.byref(d), draft_logp, offsets, n_seqs, accept, sample,
                                      tokens, counts, logp, ws, nbytes, None)


@pytest.mark.parametrize("over", [
    dict(target=dict(tokens=7)), dict(draft=dict(tokens=5)), dict(n_seqs=-1), dict(n_seqs=3), dict(target=dict(vocab=0)),
    dict(draft=dict(vocab=101)), dict(draft=dict(dtype=1)), dict(draft=dict(temperature=-1.0)), dict(target=dict(mask=A)),
    dict(draft=dict(mask=A)), dict(draft=dict(logits=None), draft_logp=A), dict(target=dict(logits=None)),
    dict(draft=dict(targets=None)), dict(draft=dict(targets=A + 4)), dict(draft_logp=A + 2), dict(offsets=None),
    dict(offsets=A + 4), dict(accept=None), dict(accept=A + 1), dict(sample=None), dict(sample=A + 2), dict(tokens=None),
    dict(tokens=A + 4), dict(counts=None), dict(counts=A + 4), dict(logp=None), dict(logp=A + 2),
    dict(draft=dict(row_stride=99)), dict(draft=dict(logits=A + 2))])
def test_verify_refuses(nsm, over):
    assert _verify(nsm, **over) == nsm.MUON_ERR_INVALID


def test_verify_of_nothing(nsm):
    assert nsm.lib.muon_verify_drafts(None, None, None, None, 0, None, None, None, None, None, None, 0, None) == nsm.MUON_ERR_INVALID
    assert _verify(nsm, dict(tokens=0, logits=None), dict(tokens=0, logits=None), 0, None, None, None, None, None, None,
                   None) == nsm.MUON_OK


def test_workspace(nsm):
    import torch
    need = nsm.muon_sample_workspace_bytes
    assert need(0, 5, torch.float32) == 0
    assert need(10, 1000, torch.float32) == 10 * 2 * 8                  # two strips of 512 a row
    assert need(1 << 20, 1 << 30, torch.bfloat16) == (1 << 20) * 512 * 8   # 512 strips at most
    for bad in ((-1, 5), (1 << 32, 5), (5, 0), (5, (1 << 30) + 1)):
        with pytest.raises(nsm.MuonError) as e:
            need(*bad, torch.float32)
        assert e.value.status == nsm.MUON_ERR_INVALID
    with pytest.raises(TypeError):
        need(5, 5, torch.float16)
    assert _verify(nsm, ws=None) == nsm.MUON_ERR_NO_WORKSPACE
    assert _verify(nsm, nbytes=6 * 8) == nsm.MUON_ERR_NO_WORKSPACE     # the draft model's rows too
    assert _verify(nsm, draft_logp=A, nbytes=5 * 8) == nsm.MUON_ERR_NO_WORKSPACE
    assert _verify(nsm, ws=A + 8) == nsm.MUON_ERR_INVALID


def test_binding_refuses_host_tensors(nsm):
    import torch
    z = torch.zeros(3, 5)
    with pytest.raises(ValueError, match="CUDA"):
        nsm.muon_sample_tokens(z, torch.zeros(3))
    with pytest.raises(ValueError, match="CUDA"):
        nsm.muon_verify_drafts(z, torch.zeros(2, dtype=torch.int64), torch.tensor([0, 2]), torch.zeros(2), torch.zeros(1))
