"""Inputs whose softmax has a long tail: one key (a sink) far ahead of all others, whose value is zero or small, so that
the tail is what the result is made of."""

import numpy as np

import oracle as o


def sink(rng, n, gap, heads=1, kv=1, d=16, lift=0, mean=0.0, group=o.ROW, flat_rows=False, value=0):
    """(X, scale): n tokens; the first one's key is `gap` nats ahead of the others for every query (for every second one with
    flat_rows), its row's exponent `lift` above theirs; the other keys differ by a few hundredths of a nat, the other values are
    40 wide around `mean`, the sink's are `value`."""
    c = np.zeros((n, heads + 2 * kv, d), np.int64)
    c[:, :heads] = np.clip(np.rint(rng.normal(0, 3, (n, heads, d))), -127, 127)
    c[:, :heads, 0] = 100
    if flat_rows:
        c[1::2, :heads, 0] = 0
    c[:, heads:heads + kv] = np.clip(np.rint(rng.normal(0, 4, (n, kv, d))), -127, 127)
    c[:, heads:heads + kv, 0] = 0
    c[:, heads + kv:] = np.clip(np.rint(rng.normal(mean, 40, (n, kv, d))), -127, 127)
    c[0, heads:] = 0
    c[0, heads + kv:] = value
    # 100 C 2^(2 e + lift) scale = gap, C at most 120
    scale, e = 0.25, -8
    while gap / (scale * 100 * 2.0 ** (2 * e + lift)) > 120:
        e += 1
    c[0, heads:heads + kv, 0] = round(gap / (scale * 100 * 2.0 ** (2 * e + lift)))
    if group == o.TENSOR:
        return o.QT(c.reshape(n, -1).astype(np.int8), np.array([e], np.int8), o.TENSOR), scale
    x = np.full(n, e, np.int8)
    x[0] += lift
    return o.QT(c.reshape(n, -1).astype(np.int8), x, o.ROW), scale


def marks(tops):
    """Rows of fine weights, by the last bit of their largest score."""
    return (np.ascontiguousarray(tops, dtype=np.float32).view(np.int32) & 1).astype(bool)
