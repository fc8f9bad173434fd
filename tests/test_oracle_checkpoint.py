"""The float64 checkpoint oracle against its definition and against differences."""
import numpy as np

from oracle import checkpoint


def test_a_step_holds_127_and_no_smaller_one_does():
    rng = np.random.default_rng(0)
    x = (rng.normal(0, 1, (50, 96)) * np.exp(rng.normal(0, 20, (50, 1)))).astype(np.float32).astype(np.float64)
    x[0] = 0
    x[1, :32] = [127.5] + [1.0] * 31          # rounds to 128: a step twice as large
    x[2, :32] = [127.4375] + [0.5] * 31
    q, b = checkpoint.encode(x)
    step = np.ldexp(1.0, b.astype(np.int64) - 133)
    v = x.reshape(50, 3, 32)
    most = np.abs(v).max(2)
    assert (np.rint(most / step) <= 127).all()
    smaller = (np.rint(most / (step / 2)) > 127) | (b == 7)
    assert smaller.all()
    assert b[1, 0] == 134 and b[2, 0] == 133 and b[0].tolist() == [7, 7, 7]
    assert (np.abs(checkpoint.values(x).reshape(v.shape) - v) <= step[:, :, None] / 2).all()
    assert (step / 2 <= np.maximum(most / 127.5, 2.0 ** -127)).all()


def test_special_values():
    big = float(np.finfo(np.float32).max)
    x = np.array([[np.inf, 1.0], [np.nan, 2.0], [big, 1.0], [1e-45, -1e-45], [2.0 ** -126, 2.0 ** -127]])
    v = checkpoint.values(x)
    assert np.isnan(v[:2]).all()
    assert v[2].tolist() == [127 * 2.0 ** 121, 0.0] and v[3].tolist() == [0.0, 0.0] and v[4].tolist() == [2.0 ** -126, 0.0]


def test_values_are_bf16_numbers():
    import torch
    rng = np.random.default_rng(1)
    v = torch.from_numpy(checkpoint.values(rng.normal(0, 3, (40, 100))))
    assert torch.equal(v.bfloat16().double(), v)


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(2)
    gate, up, dh = rng.normal(0, 3, (3, 400))
    dgate, dup = checkpoint.swiglu_backward(dh, gate, up)
    d = 1e-6
    for got, a, b in ((dgate, (gate + d, up), (gate - d, up)), (dup, (gate, up + d), (gate, up - d))):
        want = dh * (checkpoint.swiglu(*a) - checkpoint.swiglu(*b)) / (2 * d)
        # second differences: rounding 1e-16 / d times the values, and d^2
        np.testing.assert_allclose(got, want, atol=1e-8)
