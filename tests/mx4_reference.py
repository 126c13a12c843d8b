"""The MX4 operators in plain fp64 numpy, from the format's definition (32 elements share a scale
2^(s - 127); elements are E2M1 numbers), independent of the library: expected values of the tests."""
import numpy as np

BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f32_of_bf16_bits(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def bf16_bits(v):
    """The bf16 bits nearest to v (finite or infinite), ties to even."""
    u = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def quantize(bits):
    """bf16 bits [..., cols] -> (codes uint8 [..., cols / 2], scales uint8 [..., cols / 32])."""
    bits = np.asarray(bits, np.uint16)
    v = f32_of_bf16_bits(bits).astype(np.float64).reshape(*bits.shape[:-1], -1, BLOCK)
    bad = ~np.isfinite(v).all(-1)
    m = np.where(np.isfinite(v), np.abs(v), 0).max(-1)
    e = np.frexp(np.where(m > 0, m, 4.0))[1] - 1 - 2  # floor(log2 m) - 2
    e = np.maximum(e, -127)
    q = np.where(np.isfinite(v), np.abs(v), 0) / np.exp2(e.astype(np.float64))[..., None]
    # nearest of the eight magnitudes; a tie goes to the even code
    dist = np.abs(q[..., None] - E2M1)
    best = dist.min(-1, keepdims=True)
    tied = dist == best
    first = tied.argmax(-1)
    last = 7 - tied[..., ::-1].argmax(-1)
    code = np.where(first % 2 == 0, first, last)
    code = np.where(bad[..., None], 0, code | (np.signbit(v).astype(np.int64) << 3))
    code = code.reshape(bits.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def values(q, s):
    """fp64 values of codes and scales."""
    q, s = np.asarray(q, np.uint8), np.asarray(s, np.uint8)
    code = np.stack((q & 15, q >> 4), -1).reshape(*s.shape, BLOCK)
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return (v * scale[..., None]).reshape(*q.shape[:-1], -1)


def grouped(xv, offsets, wv):
    """y and the rms-style size sqrt(sum (x w)^2) of every output's terms; rows of no expert: NaN."""
    y = np.full((xv.shape[0], wv.shape[1]), np.nan)
    size = np.zeros_like(y)
    for e in range(wv.shape[0]):
        r = slice(offsets[e], offsets[e + 1])
        y[r] = xv[r] @ wv[e].T
        size[r] = np.sqrt((xv[r] ** 2) @ (wv[e] ** 2).T)
    return y, size


def layer(x_bits, router, bias, w1, w3, w2):
    """The layer on the values w1, w3 [E][F][d], w2 [E][d][F] of the experts' MX4 weights."""
    x = f32_of_bf16_bits(x_bits).astype(np.float64)
    z = x @ router.astype(np.float64).T + (0 if bias is None else bias.astype(np.float64))
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :2]
    xv = values(*quantize(x_bits))
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for k in range(2):
            e = ids[t, k]
            g, u = w1[e] @ xv[t], w3[e] @ xv[t]
            h = bf16_bits((g / (1 + np.exp(-g)) * u).astype(np.float32))
            y[t] += p[t, e] * (w2[e] @ values(*quantize(h)))
    return y, ids, np.take_along_axis(p, ids, 1), z
