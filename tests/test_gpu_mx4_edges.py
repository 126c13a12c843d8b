"""MX4 products and layer where their smaller tests do not reach: bands of token tiles, wide layers, gates far below
zero, rows of no expert in bf16.

Products are compared for equality: `exact_operands` gives scales of 1 or 2, so every partial sum, in any order, is a
multiple of 1/4 and, by the bound that it checks for the case's own K, a number that fp32 holds."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import int8_expert_weight_b200 as jm  # noqa: E402
import mx4_reference as ref  # noqa: E402
from gpu_layer import bf16_to_dev, dev_to_bf16_bits  # noqa: E402
from helpers import assert_y_close  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int8_expert_weight_b200 import build
    build.build()
    jm.load_library()


def exact_operands(seed, n, rows, cols, experts, scales=(127,)):
    """Codes and scales on the device.  An element is at most 6 * 2^(s - 127) and a multiple of half its scale."""
    assert 4 * 36 * 4 ** (max(scales) - 127) * cols <= 2 ** 24, "partial sums beyond fp32"
    g = torch.Generator("cuda").manual_seed(seed)

    def one(*shape):
        q = torch.randint(0, 256, shape + (cols // 2,), generator=g, dtype=torch.uint8, device="cuda")
        s = torch.randint(min(scales), max(scales) + 1, shape + (cols // 32,), generator=g, device="cuda")
        return q, s.to(torch.uint8)

    return one(n), one(experts, rows)


def values(q, s):
    return ref.values(q.cpu().numpy(), s.cpu().numpy())


def product(x, w, offsets, dtype=torch.float32, y=None):
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return jm.jamba_moe_grouped_mx4(*x, off, *w, out_dtype=dtype, y=y)


# The tiles of a group are walked in bands of as many token tiles as have 32 MB of codes: 64-row tiles (few rows on
# average) 128 of them at K = 8192, 208-row tiles 19 at K = 16384.
@pytest.mark.parametrize("counts,rows,cols", [([3] + [0] * 200 + [9001, 17] + [0] * 53, 130, 8192),
                                              ([4700, 50], 300, 16384), ([0, 8000], 257, 8192)])
def test_bands_of_token_tiles(counts, rows, cols):
    x, w = exact_operands(rows, sum(counts), rows, cols, len(counts))
    at = np.concatenate([[0], np.cumsum(counts)])
    y = product(x, w, at)
    for e in np.nonzero(counts)[0]:
        wv = values(w[0][e], w[1][e])
        # every 13th row, so some of each tile, and both ends
        r = np.unique(np.concatenate([np.arange(at[e], at[e + 1], 13), [at[e], at[e + 1] - 1]]))
        r_dev = torch.from_numpy(r).cuda()
        want = values(x[0][r_dev], x[1][r_dev]) @ wv.T
        assert np.array_equal(y[r_dev].cpu().numpy(), want), e


@pytest.mark.parametrize("counts,rows,cols", [([33], 64, 16384), ([300], 70, 16384), ([257, 0, 90], 129, 32768)])
def test_long_sums_are_exact(counts, rows, cols):
    x, w = exact_operands(cols, sum(counts), rows, cols, len(counts), (127, 128) if cols == 16384 else (127,))
    at = np.concatenate([[0], np.cumsum(counts)])
    want = ref.grouped(values(*x), at, values(*w))[0]
    assert np.array_equal(product(x, w, at).cpu().numpy(), want)
    assert np.array_equal(dev_to_bf16_bits(product(x, w, at, torch.bfloat16)), ref.bf16_bits(want))


@pytest.mark.parametrize("rows", [33, 136])
@pytest.mark.parametrize("scale", [1, 10])  # single CTAs, pairs
def test_rows_of_no_expert_in_bf16(rows, scale):
    at = [11 * scale, 40 * scale, 40 * scale, 81 * scale]
    n = 90 * scale
    x, w = exact_operands(n, n, rows, 128, 3)
    y = torch.full((n, rows), 7.0, dtype=torch.bfloat16, device="cuda")
    product(x, w, at, torch.bfloat16, y)
    want = ref.grouped(values(*x), at, values(*w))[0]
    got = dev_to_bf16_bits(y)
    assert np.array_equal(got[at[0]:at[3]], ref.bf16_bits(want[at[0]:at[3]]))
    seven = ref.bf16_bits(np.float32(7))
    assert (got[:at[0]] == seven).all() and (got[at[3]:] == seven).all()


@pytest.mark.parametrize("cols", [2880, 160, 32])
def test_width_padded_with_zeros(cols):
    """Rows of a width that the product refuses, padded with zeros before they are quantised."""
    g = torch.Generator("cuda").manual_seed(cols)
    x = torch.randint(-6, 7, (50, cols), generator=g, device="cuda").bfloat16()
    w = torch.randint(-6, 7, (2, 40, cols), generator=g, device="cuda").bfloat16()
    pad = -cols % 128
    with pytest.raises(jm.JmoeError):
        product(jm.jamba_moe_quantize_mx4(x), jm.jamba_moe_quantize_mx4(w), [0, 20, 50])
    xp, wp = (jm.jamba_moe_quantize_mx4(torch.nn.functional.pad(t, (0, pad))) for t in (x, w))
    y = product(xp, wp, [0, 20, 50])
    # blocks' largest magnitudes are 1 to 6: scales 1/4 to 1, sums multiples of 2^-6 and below 36 * 2880
    assert 36 * cols * 2 ** 6 <= 2 ** 24
    want = ref.grouped(values(*jm.jamba_moe_quantize_mx4(x)), [0, 20, 50], values(*jm.jamba_moe_quantize_mx4(w)))[0]
    assert np.array_equal(y.cpu().numpy(), want)


# ------------------------------------------------------------------ the layer at the widths that models have
def value_table(q, s):
    """fp64 values of one matrix on the device."""
    lut = torch.tensor([*ref.E2M1, *-ref.E2M1], dtype=torch.float64, device="cuda")
    code = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)
    powers = torch.tensor(np.exp2(np.arange(-127.0, 128)), device="cuda")
    return lut[code.long()] * powers[s.long()].repeat_interleave(32, 1)


def rows_mx4(rows):
    """fp64 values of bf16 rows in MX4, by the reference."""
    q, s = ref.quantize(dev_to_bf16_bits(rows))
    return torch.from_numpy(ref.values(q, s)).cuda()


@pytest.mark.parametrize("T,d,F", [(40, 4096, 1536), (500, 4096, 1536), (900, 1152, 4224), (450, 2048, 14336)])
def test_wide_layer(T, d, F):
    """T = 40: single CTAs, else pairs; against the definition in fp64."""
    g = torch.Generator("cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rand(2 * T, d).bfloat16()
    router = rand(16, d) * d ** -0.5
    z = x.double() @ router.double().T
    top = z.sort(1, descending=True).values
    clear = (top[:, 1] - top[:, 2] > 1e-3).nonzero().squeeze(1)[:T]  # routing that rounding does not decide
    x, z = x[clear].contiguous(), z[clear]
    assert x.shape[0] == T
    w = [jm.jamba_moe_quantize_mx4((rand(16, r, c) * c ** -0.5).bfloat16()) for r, c in ((F, d), (F, d), (d, F))]
    y, ids, p = jm.jamba_moe_forward_mx4(x, router, None, *w[0], *w[1], *w[2])
    prob = torch.softmax(z, 1)
    best = z.topk(2, 1).indices
    assert torch.equal(ids.sort(1).values.long(), best.sort(1).values)
    xv = rows_mx4(x)
    want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in range(16):
        t = (best == e).any(1).nonzero().squeeze(1)
        if t.numel():
            gate, up = (xv[t] @ value_table(w[i][0][e], w[i][1][e]).T for i in (0, 1))
            h = rows_mx4((gate * torch.sigmoid(gate) * up).bfloat16())
            want[t] += prob[t, e, None] * (h @ value_table(w[2][0][e], w[2][1][e]).T)
    assert_y_close(dev_to_bf16_bits(y), want.cpu().numpy())


@pytest.mark.parametrize("T", [1, 900])  # single CTAs, pairs
def test_gates_far_below_zero(T):
    """h_j = SiLU(n_j) * 2^m_j for whole n_j from 20 down to -119, with 2^m_j the power of two (up to 2^120) that brings
    |h_j| into [1, 2); W2 passes h through.  Down to a gate of -87 h is right up to the rounding to bf16 and to the
    code; below, where |SiLU| < 2^-119, it may come out as 0."""
    F = d = 256
    n = np.tile(np.concatenate([np.arange(20, -44, -1), np.arange(-56, -120, -1)]), 2)  # -88 starts a block of 32
    far = n <= -88
    silu = n / (1 + np.exp(-n.astype(np.float64)))
    m = np.where(n == 0, 0, np.minimum(-np.floor(np.log2(np.abs(np.where(n == 0, 1, silu)))), 120))
    # gate and up as sums over x's ones, each in a block of 32 of its own: n's binary digits and sign, and 2^m
    w1, w3 = np.zeros((F, d)), np.zeros((F, d))
    for b in range(7):
        w1[:, 32 * b] = np.sign(n) * ((np.abs(n) >> b) & 1) * 2.0 ** b
    w3[:, 32 * 7] = np.exp2(m)
    x = np.zeros((T, d))
    x[:, ::32] = 1
    bias = np.zeros(16, np.float32)
    bias[[3, 11]] = 60, 50  # two experts of the same weights: their probabilities add to 1
    dev = lambda a: bf16_to_dev(ref.bf16_bits(a.astype(np.float32)))  # noqa: E731
    w = [t for a in (w1, w3, np.eye(d))
         for t in jm.jamba_moe_quantize_mx4(dev(a)[None].expand(16, -1, -1).contiguous())]
    y, _, _ = jm.jamba_moe_forward_mx4(dev(x), torch.zeros(16, d, device="cuda"), torch.from_numpy(bias).cuda(), *w)
    y = ref.f32_of_bf16_bits(dev_to_bf16_bits(y)).astype(np.float64)
    assert (y == y[0]).all()
    # SiLU's error at a gate of -87 is the exponential's 2 + 1.173 * 87 units in the last place, the division's 2 and two
    # roundings, each unit at most 2^-23 of the value: together below 2^-16.  Where both ends of that interval round to
    # one code, y is its value
    ends = [ref.values(*ref.quantize(ref.bf16_bits((silu * np.exp2(m) * (1 + off)).astype(np.float32))[None]))[0]
            for off in (-2.0 ** -16, 2.0 ** -16)]
    sure = (ends[0] == ends[1]) & ~far
    assert sure.sum() >= 0.95 * (~far).sum()
    assert np.array_equal(y[0][sure], ends[0][sure])
    assert ((y[0][far] == 0) | (y[0][far] == ends[0][far]) | (y[0][far] == ends[1][far])).all()
