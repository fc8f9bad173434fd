"""8-bit activation checkpoints and a gated activation, in float64 numpy (test infrastructure
only)."""
import numpy as np

BLOCK = 32


def encode(x):
    """(q [rows, P] int8, b [rows, P / 32] uint8) of x [rows, cols]."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = np.zeros((rows, blocks * BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, blocks, BLOCK)
    bad = ~np.isfinite(v).all(2)
    v = np.where(bad[:, :, None], 0.0, v)
    most = np.abs(v).max(2)
    # most = mantissa 2^exponent with mantissa in [1/2, 1): 64 to 128 steps of 2^(exponent - 7)
    mantissa, exponent = np.frexp(most)
    power = exponent - 7 + (mantissa * 128 >= 127.5)
    power = np.clip(np.where(most == 0, -126, power), -126, 121)
    q = np.clip(np.rint(np.ldexp(v, -power[:, :, None])), -127, 127)
    b = np.where(bad, 255, power + 133)
    return q.astype(np.int8).reshape(rows, -1), b.astype(np.uint8)


def decode(q, b, cols):
    with np.errstate(over="ignore"):
        step = np.where(b == 255, np.nan, np.ldexp(1.0, b.astype(np.int64) - 133))
    return (q.reshape(*b.shape, BLOCK) * step[:, :, None]).reshape(len(q), -1)[:, :cols]


def values(x):
    return decode(*encode(x), x.shape[1])


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def swiglu(gate, up):
    return gate * sigmoid(gate) * up


def swiglu_backward(dh, gate, up):
    s = sigmoid(gate)
    return dh * up * s * (1 + gate * (1 - s)), dh * gate * s
