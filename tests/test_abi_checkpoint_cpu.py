"""The checkpoint entry points: sizes and refusals (no kernel runs)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_muon_gb300.build as b
    b.build()
    import newton_schulz_muon_gb300 as m
    return m


A = 1 << 20


def _ck(nsm, data=A, rows=6, cols=100):
    return nsm.muon_checkpoint(data, rows, cols)


def test_bytes(nsm):
    assert nsm.muon_checkpoint_bytes(0, 5) == 0
    assert nsm.muon_checkpoint_bytes(1, 1) == 33 and nsm.muon_checkpoint_bytes(7, 33) == 7 * 66
    assert nsm.muon_checkpoint_bytes(1 << 20, 1 << 20) == (1 << 40) // 32 * 33
    for bad in ((-1, 5), (1 << 31, 5), (5, 0), (5, (1 << 30) + 1)):
        with pytest.raises(nsm.MuonError) as e:
            nsm.muon_checkpoint_bytes(*bad)
        assert e.value.status == nsm.MUON_ERR_INVALID


BAD = [dict(data=None), dict(data=A + 8), dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=(1 << 30) + 1)]


@pytest.mark.parametrize("over", BAD)
def test_bad_checkpoints(nsm, over):
    lib, bad, good = nsm.lib, ctypes.byref(_ck(nsm, **over)), ctypes.byref(_ck(nsm, 2 * A))
    assert lib.muon_checkpoint_save(A, 0, 0, bad, None) == nsm.MUON_ERR_INVALID
    assert lib.muon_checkpoint_load(bad, A, 0, 0, None) == nsm.MUON_ERR_INVALID
    assert lib.muon_swiglu_forward(A, 0, A, 0, 0, A, 0, bad, good, None) == nsm.MUON_ERR_INVALID
    assert lib.muon_swiglu_forward(A, 0, A, 0, 0, A, 0, good, bad, None) == nsm.MUON_ERR_INVALID
    assert lib.muon_swiglu_backward(A, 0, 0, bad, good, A, 0, 2 * A, 0, None, 0, None) == nsm.MUON_ERR_INVALID
    assert lib.muon_swiglu_backward(A, 0, 0, good, bad, A, 0, 2 * A, 0, None, 0, None) == nsm.MUON_ERR_INVALID


def test_bad_matrices(nsm):
    lib, ck, other = nsm.lib, ctypes.byref(_ck(nsm)), ctypes.byref(_ck(nsm, 2 * A))
    odd, bad = ctypes.byref(_ck(nsm, 3 * A, 7)), nsm.MUON_ERR_INVALID
    for p, stride, dtype in ((None, 0, 0), (A + 2, 0, 0), (A + 1, 0, 1), (A, 99, 0), (A, -1, 0), (A, 1 << 41, 0), (A, 0, 2)):
        assert lib.muon_checkpoint_save(p, stride, dtype, ck, None) == bad
        assert lib.muon_checkpoint_load(ck, p, stride, dtype, None) == bad
        assert lib.muon_swiglu_forward(p, stride, A, 0, dtype, A, 0, ck, other, None) == bad
        assert lib.muon_swiglu_forward(A, 0, p, stride, dtype, A, 0, ck, other, None) == bad
        assert lib.muon_swiglu_forward(A, 0, A, 0, dtype, p, stride, ck, other, None) == bad
        assert lib.muon_swiglu_backward(p, stride, dtype, ck, other, A, 0, 2 * A, 0, None, 0, None) == bad
        assert lib.muon_swiglu_backward(A, 0, dtype, ck, other, p, stride, 2 * A, 0, None, 0, None) == bad
        assert lib.muon_swiglu_backward(A, 0, dtype, ck, other, A, 0, p, stride, None, 0, None) == bad
        if p:
            assert lib.muon_swiglu_backward(A, 0, dtype, ck, other, A, 0, 2 * A, 0, p, stride, None) == bad
    assert lib.muon_checkpoint_save(A, 0, 0, None, None) == bad
    assert lib.muon_checkpoint_load(None, A, 0, 0, None) == bad
    assert lib.muon_swiglu_forward(A, 0, A, 0, 0, A, 0, ck, ck, None) == bad       # one checkpoint for both
    assert lib.muon_swiglu_forward(A, 0, A, 0, 0, A, 0, ck, odd, None) == bad      # two shapes
    assert lib.muon_swiglu_backward(A, 0, 0, ck, odd, A, 0, 2 * A, 0, None, 0, None) == bad
    for outs in ((A, A, None), (A, 2 * A, A), (A, 2 * A, 2 * A)):                  # two outputs in one place
        assert lib.muon_swiglu_backward(3 * A, 0, 0, ck, other, outs[0], 0, outs[1], 0, outs[2], 0, None) == bad
    empty, also = ctypes.byref(_ck(nsm, None, 0)), ctypes.byref(_ck(nsm, None, 0))
    assert lib.muon_checkpoint_save(None, 0, 0, empty, None) == nsm.MUON_OK
    assert lib.muon_swiglu_forward(None, 0, None, 0, 1, None, 0, empty, also, None) == nsm.MUON_OK


def test_binding_refuses(nsm):
    import torch
    with pytest.raises(ValueError, match="CUDA"):
        nsm.muon_checkpoint_save(torch.zeros(3, 5))
    with pytest.raises(ValueError, match="CUDA"):
        nsm.Checkpoint(3, 5, torch.zeros(3 * 33, dtype=torch.uint8))
    with pytest.raises(ValueError, match="uint8"):
        nsm.Checkpoint(3, 5, torch.zeros(3 * 33))
