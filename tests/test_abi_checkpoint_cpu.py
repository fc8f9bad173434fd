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


def _wg(nsm, ck=None, dy=A, dy_stride=0, dy_dtype=1, outs=64, dw=2 * A, dw_stride=0, dw_dtype=0, accumulate=0, ws=3 * A,
        nbytes=1 << 40):
    return nsm.lib.muon_checkpoint_weight_grad(ctypes.byref(ck or _ck(nsm)), dy, dy_stride, dy_dtype, outs, dw, dw_stride,
                                               dw_dtype, accumulate, ws, nbytes, None)


@pytest.mark.parametrize("over", [
    dict(dy=None), dict(dy=A + 1), dict(dy=A + 2, dy_dtype=0), dict(dy_stride=63), dict(dy_stride=-1), dict(dy_dtype=2),
    dict(outs=0), dict(outs=(1 << 30) + 1), dict(dw=None), dict(dw=A + 2), dict(dw=A + 1, dw_dtype=1), dict(dw_stride=99),
    dict(dw_dtype=3), dict(accumulate=2)])
def test_weight_grad_refuses(nsm, over):
    assert _wg(nsm, **over) == nsm.MUON_ERR_INVALID


@pytest.mark.parametrize("over", BAD)
def test_weight_grad_refuses_bad_checkpoints(nsm, over):
    assert _wg(nsm, _ck(nsm, **over)) == nsm.MUON_ERR_INVALID


def test_weight_grad_workspace(nsm):
    def need(rows, cols, outs, dtype, dy=A, stride=0):
        v = ctypes.c_size_t()
        st = nsm.lib.muon_weight_grad_workspace_bytes(ctypes.byref(_ck(nsm, A, rows, cols)), dy, stride, dtype, outs,
                                                      ctypes.byref(v))
        assert st == nsm.MUON_OK
        return v.value

    assert need(8192, 2560, 9728, 1) == 8192 * 2560 * 2        # x in bf16; dy as it lies, a tile a pair
    assert need(8192, 2560, 9728, 1, dy=A + 2) >= 8192 * 9728 * 2
    assert need(8192, 2560, 9728, 1, stride=9729) >= 8192 * 9728 * 2
    assert need(8192, 2560, 9728, 0) >= 3 * 8192 * 9728 * 2
    assert need(100000, 40, 40, 1) > 100000 * 40 * 2           # the sums of the tokens' parts
    assert need(0, 40, 40, 1) == 0
    short = _wg(nsm, dy_dtype=0, nbytes=10)
    assert short == nsm.MUON_ERR_NO_WORKSPACE
    assert _wg(nsm, dy_dtype=0, ws=None) == nsm.MUON_ERR_NO_WORKSPACE
    assert _wg(nsm, dy_dtype=0, ws=A + 8) == nsm.MUON_ERR_INVALID
    v = ctypes.c_size_t()
    assert nsm.lib.muon_weight_grad_workspace_bytes(None, A, 0, 1, 64, ctypes.byref(v)) == nsm.MUON_ERR_INVALID
    assert nsm.lib.muon_weight_grad_workspace_bytes(ctypes.byref(_ck(nsm)), A, 0, 1, 64, None) == nsm.MUON_ERR_INVALID


def test_workspaces_that_are_held(nsm, monkeypatch):
    """A thread holds a stream's small workspaces, and gives the large ones back."""
    torch = pytest.importorskip("torch")
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *size, device=None, **kw: empty(*size, **kw))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(nsm, "_SPACES", type("S", (), {})())
    small = nsm._space(None, 1000, 0, 7)
    assert nsm._space(None, 2000, 0, 7)[1] == small[1] and nsm._space(None, 2000, 0, 8)[1] != small[1]
    large, at, size = nsm._space(None, 1 << 26, 0, 7)
    assert large.numel() == size == 1 << 26 and at == large.data_ptr()
    assert nsm._space(None, 1000, 0, 7)[1] == small[1]
    assert sum(w.numel() for w, _, _ in nsm._SPACES.held.values()) <= 1 << 20


def test_gated_outputs_in_place_of_an_input_have_its_stride(nsm):
    """Rows of an output that lie elsewhere than the input's would be written over before they are read."""
    lib, ck, other = nsm.lib, ctypes.byref(_ck(nsm)), ctypes.byref(_ck(nsm, 2 * A))
    bad = nsm.MUON_ERR_INVALID
    assert lib.muon_swiglu_forward(A, 200, 3 * A, 0, 0, A, 0, ck, other, None) == bad
    assert lib.muon_swiglu_forward(A, 0, 3 * A, 200, 0, 3 * A, 100, ck, other, None) == bad
    assert lib.muon_swiglu_forward(A, 0, 3 * A, 0, 0, A, 101, ck, other, None) == bad
    for k in range(3):
        outs = [4 * A, 0, 5 * A, 0, 6 * A, 0]
        outs[2 * k:2 * k + 2] = A, 300
        assert lib.muon_swiglu_backward(A, 0, 0, ck, other, *outs, None) == bad
        assert b"stride" in lib.muon_last_error()
