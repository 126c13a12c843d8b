"""GPU parity of the MX4 operators with the fp64 reference of tests/mx4_reference.py.

Codes, scales and dequantized values are compared bit for bit.  The grouped product is compared for
equality where every partial sum, in any order, is an fp32 number (small codes and scales: the sums are
multiples of a fixed quantum and below 2^24 of it), and otherwise within the error of K fp32 additions:
each is off by at most 2^-23 of its partial sum (truncation; rounding would be half of that), and the
partial sums of K zero-mean terms stay within 6 times their root-sum-square `size`, so the total error is at
most K * 2^-23 * 6 * size.  A bf16 result adds half a step, 2^-8 of the value."""
import dataclasses

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import int8_expert_weight_b200 as jm  # noqa: E402
import mx4_reference as ref  # noqa: E402
import synth  # noqa: E402
from gpu_layer import bf16_to_dev, dev_to_bf16_bits  # noqa: E402
from helpers import assert_routing, assert_y_close, gap_inputs, workload  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int8_expert_weight_b200 import build
    build.build()
    jm.load_library()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ quantization
def assert_quantize_equal(bits):
    Q, S = jm.jamba_moe_quantize_mx4(bf16_to_dev(bits))
    q, s = ref.quantize(bits)
    assert np.array_equal(S.cpu().numpy(), s), "scales differ"
    assert np.array_equal(Q.cpu().numpy(), q), "codes differ"
    return Q, S


@pytest.mark.parametrize("shape", [(1, 32), (3, 5, 96), (7, 160), (64, 4096), (2, 33, 14336), (1, 1 << 20), (4099, 64)])
def test_quantize_random(shape):
    rng = np.random.default_rng(sum(shape))
    w = rng.standard_normal(shape) * np.exp(4 * rng.standard_normal(shape[:-1] + (1,)))
    bits = synth.f32_to_bf16_bits(w.astype(np.float32))
    Q, S = assert_quantize_equal(bits)
    back = jm.jamba_moe_dequantize_mx4(Q, S)
    assert np.array_equal(dev_to_bf16_bits(back), ref.bf16_bits(ref.values(*ref.quantize(bits))))


def test_quantize_every_bf16_value():
    # each of the 65536 bit patterns as a block's largest magnitude's neighbour: a 1 beside it
    bits = np.zeros((65536, 32), np.uint16)
    bits[:, 5] = np.arange(65536)
    bits[:, 6] = 0x3F80
    bits[:, 7] = np.arange(65536)[::-1]
    assert_quantize_equal(bits)
    bits[:, 6:8] = 0  # alone: its own scale, subnormals and zeros of both signs among them
    assert_quantize_equal(bits)


@pytest.mark.parametrize("skip", [8, 24, 16])
def test_quantize_views_off_32_bytes(skip):
    """Rows that start on a 16-byte boundary only (or on the next 32-byte one), codes 16 and scales 4 bytes in."""
    rng = np.random.default_rng(skip)
    bits = synth.f32_to_bf16_bits(rng.standard_normal((5, 224)).astype(np.float32))
    W = torch.zeros(5 * 224 + skip, dtype=torch.bfloat16, device="cuda")[skip:].view(5, 224)
    W.copy_(bf16_to_dev(bits))
    Q = torch.zeros(5 * 112 + 16, dtype=torch.uint8, device="cuda")
    S = torch.zeros(5 * 7 + 8, dtype=torch.uint8, device="cuda")
    out = Q[16:].view(5, 112), S[4:39].view(5, 7)
    jm.jamba_moe_quantize_mx4(W, out=out)
    q, s = ref.quantize(bits)
    assert np.array_equal(out[0].cpu().numpy(), q) and np.array_equal(out[1].cpu().numpy(), s)
    assert not Q[:16].any() and not S[:4].any() and not S[39:].any()
    W.zero_()
    jm.jamba_moe_dequantize_mx4(*out, out=W)
    assert np.array_equal(dev_to_bf16_bits(W), ref.bf16_bits(ref.values(q, s)))


def test_quantize_ties_at_every_scale():
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 7.0, 4.0])
    row = np.concatenate([grid, -grid])
    e = np.arange(-124, 125)
    assert_quantize_equal(ref.bf16_bits((row[None] * np.exp2(e)[:, None]).astype(np.float32)))


def test_dequantize_every_code_and_scale():
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    got = synth.bf16_bits_to_f32(dev_to_bf16_bits(jm.jamba_moe_dequantize_mx4(cuda(q), cuda(s))))
    with np.errstate(over="ignore"):
        want = ref.f32_of_bf16_bits(ref.bf16_bits(np.nan_to_num(ref.values(q, s)).astype(np.float32)))
    assert np.array_equal(got[:255], want[:255]) and np.isnan(got[255]).all()


# ------------------------------------------------------------------ grouped products
def operands(rng, n, rows, cols, experts, scales):
    def one(*shape):
        return (rng.integers(0, 256, shape + (cols // 2,), np.uint8),
                rng.choice(np.array(scales, np.uint8), shape + (cols // 32,)))

    return one(n), one(experts, rows)


def run_grouped(x, w, offsets, dtype=torch.float32, y=None):
    return jm.jamba_moe_grouped_mx4(cuda(x[0]), cuda(x[1]), cuda(np.asarray(offsets, np.int32)), cuda(w[0]), cuda(w[1]),
                                    out_dtype=dtype, y=y)


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)])


# sizes on both sides of every tile edge: rows 128 / 256, tokens 16 / 32 / 64 / 208, k 128 / 256 / 1024; the
# stages of few tiles divided among many CTAs
SHAPES = [
    ([1], 1, 128), ([1], 128, 256), ([0, 1, 0], 129, 384), ([16, 17], 127, 128), ([31, 33, 32], 130, 512),
    ([64, 65, 0, 63], 256, 640), ([223, 224, 225], 100, 256), ([255, 0, 257, 1], 384, 384), ([449], 131, 128),
    ([1000], 64, 256), ([0, 0, 0, 700], 257, 512), ([3] * 100, 65, 256), ([2, 0] * 128, 40, 128),
    ([5] * 17, 1411, 2176),
    ([1500, 40], 640, 1024), ([207, 208, 209], 255, 256), ([416, 417], 257, 1024), ([96, 97, 161, 160, 113], 129, 1152),
    ([1], 1, 2048), ([40], 128, 14336), ([1, 1], 300, 4224), ([48, 0, 48, 47, 5], 777, 3968), ([33], 64, 16384),
]


@pytest.mark.parametrize("counts,rows,cols", SHAPES)
def test_grouped_exact(counts, rows, cols):
    # products are multiples of 1/4 of the scales' product and below 36 of it: with scales of 1 and 2 the sums are
    # multiples of 1/4, below 4 * 36 * 2176 < 2^19: fp32 holds them all
    rng = np.random.default_rng(rows + cols)
    n = sum(counts)
    x, w = operands(rng, n, rows, cols, len(counts), [127, 128])
    y = run_grouped(x, w, offsets_of(counts)).cpu().numpy()
    want, _ = ref.grouped(ref.values(*x), offsets_of(counts), ref.values(*w))
    assert np.array_equal(y, want)
    bf = run_grouped(x, w, offsets_of(counts), torch.bfloat16)
    assert np.array_equal(dev_to_bf16_bits(bf), ref.bf16_bits(want))


@pytest.mark.parametrize("counts,rows,cols", [([3, 40], 200, 1024), ([300, 5], 140, 2048), ([1], 513, 8192)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_mixed_scales(counts, rows, cols, dtype):
    rng = np.random.default_rng(cols)
    n = sum(counts)
    x, w = operands(rng, n, rows, cols, len(counts), range(118, 132))
    y = run_grouped(x, w, offsets_of(counts), dtype).double().cpu().numpy()
    want, size = ref.grouped(ref.values(*x), offsets_of(counts), ref.values(*w))
    tol = cols * 2.0 ** -23 * 6 * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    assert (np.abs(y - want) <= tol).all(), np.max(np.abs(y - want) / tol)


@pytest.mark.parametrize("counts,rows,cols", [([2], 40, 32768), ([70], 40, 32768), ([3, 1], 65536, 128),
                                              ([0, 200], 65535, 256)])
def test_grouped_largest_sizes(counts, rows, cols):
    # sums of at most 32768 terms that are multiples of 1/4 and below 36: 4 * 36 * 2^15 < 2^23
    rng = np.random.default_rng(cols)
    x, w = operands(rng, sum(counts), rows, cols, len(counts), [127])
    y = run_grouped(x, w, offsets_of(counts)).cpu().numpy()
    assert np.array_equal(y, ref.grouped(ref.values(*x), offsets_of(counts), ref.values(*w))[0])


@pytest.mark.parametrize("n", [30, 400])  # single CTAs, pairs
def test_grouped_operands_off_32_bytes(n):
    """Scales on 4-byte, codes and results on 16-byte boundaries only, at a K whose scales could be read 32 bytes
    at a time."""
    rng = np.random.default_rng(n)
    x, w = operands(rng, n, 72, 2048, 1, [127, 128])

    def shifted(a, by):
        t = torch.zeros(a.size + by, dtype=torch.uint8, device="cuda")[by:].view(a.shape)
        return t.copy_(cuda(a))

    off = cuda(np.array([0, n], np.int32))
    want = ref.grouped(ref.values(*x), [0, n], ref.values(*w))[0]
    y = torch.zeros(n * 72 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(n, 72)
    jm.jamba_moe_grouped_mx4(shifted(x[0], 16), shifted(x[1], 4), off, shifted(w[0], 48), shifted(w[1], 20), y=y)
    assert np.array_equal(dev_to_bf16_bits(y), ref.bf16_bits(want))


def test_grouped_far_scales():
    # x near the top of the scales' range, w near its bottom: the products are ordinary numbers
    rng = np.random.default_rng(8)
    x, w = operands(rng, 20, 70, 256, 1, [127])
    want, _ = ref.grouped(ref.values(*x), [0, 20], ref.values(*w))
    for up in (120, 127):
        x[1][:], w[1][:] = 127 + up, 127 - up
        assert np.array_equal(run_grouped(x, w, [0, 20]).cpu().numpy(), want), up


def test_grouped_nan_scale_stays_in_its_row():
    rng = np.random.default_rng(9)
    x, w = operands(rng, 50, 140, 384, 2, [127])
    clean, _ = ref.grouped(ref.values(*x), [0, 20, 50], ref.values(*w))
    x[1][19, 3] = 255
    w[1][1, 139, 11] = 255
    y = run_grouped(x, w, [0, 20, 50]).cpu().numpy()
    bad = np.zeros_like(clean, bool)
    bad[19] = True
    bad[20:, 139] = True
    assert np.isnan(y[bad]).all() and np.array_equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_leaves_other_rows(dtype):
    rng = np.random.default_rng(10)
    x, w = operands(rng, 90, 33, 128, 3, [127])
    y = torch.full((90, 33), 7.0, dtype=dtype, device="cuda")
    run_grouped(x, w, [11, 40, 40, 81], dtype, y)
    y = y.float().cpu().numpy()
    want, _ = ref.grouped(ref.values(*x), [11, 40, 40, 81], ref.values(*w))
    assert (y[:11] == 7).all() and (y[81:] == 7).all()
    if dtype == torch.float32:
        assert np.array_equal(y[11:81], want[11:81])


def test_grouped_no_rows():
    rng = np.random.default_rng(11)
    _, w = operands(rng, 1, 33, 128, 3, [127])
    x = (np.zeros((0, 64), np.uint8), np.zeros((0, 4), np.uint8))
    assert run_grouped(x, w, [0, 0, 0, 0]).shape == (0, 33)
    x, w = operands(rng, 5, 33, 128, 3, [127])  # rows, but of no expert
    y = torch.full((5, 33), 7.0, device="cuda")
    run_grouped(x, w, [2, 2, 2, 2], torch.float32, y)
    assert (y == 7).all()


@pytest.mark.parametrize("offsets", [[0, 9, 5, 20], [-3, 5, 10, 20], [0, 5, 10, 21], [30, 5, 10, 20],
                                     [0, 2 ** 31 - 1, -2 ** 31, 20]])
def test_grouped_bad_offsets_are_reported(offsets):
    rng = np.random.default_rng(12)
    x, w = operands(rng, 20, 40, 128, 3, [127])
    ws = torch.zeros(jm.jamba_moe_grouped_mx4_workspace_size(20, 40, 128, 3), dtype=torch.uint8, device="cuda")
    args = [cuda(x[0]), cuda(x[1]), cuda(np.asarray(offsets, np.int32)), cuda(w[0]), cuda(w[1])]
    whole = torch.full((60, 40), 7.0, device="cuda")
    jm.jamba_moe_grouped_mx4(*args, out_dtype=torch.float32, y=whole[20:40], workspace=ws)
    assert jm.jamba_moe_read_device_status(ws) == 6
    assert (whole == 7).all()
    args[2] = cuda(np.asarray([0, 5, 10, 20], np.int32))  # the status is this call's, not the last one's
    jm.jamba_moe_grouped_mx4(*args, out_dtype=torch.float32, workspace=ws)
    assert jm.jamba_moe_read_device_status(ws) == 0


def test_grouped_graph_and_streams():
    """A captured call follows its inputs; calls on two streams, each with its own workspace, do not meet."""
    rng = np.random.default_rng(13)
    counts = [40, 0, 260]
    off = cuda(offsets_of(counts).astype(np.int32))
    sets = [operands(rng, 300, 200, 512, 3, [127, 128]) for _ in range(2)]
    want = [ref.grouped(ref.values(*x), offsets_of(counts), ref.values(*w))[0] for x, w in sets]
    dev = [[cuda(a) for a in (*x, *w)] for x, w in sets]
    ws = [torch.empty(jm.jamba_moe_grouped_mx4_workspace_size(300, 200, 512, 3), dtype=torch.uint8, device="cuda")
          for _ in range(3)]
    live = [t.clone() for t in dev[0]]
    out = torch.empty(300, 200, device="cuda")

    def call(d, y, k):
        return jm.jamba_moe_grouped_mx4(d[0], d[1], off, d[2], d[3], out_dtype=torch.float32, y=y, workspace=ws[k])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(live, out, 0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(live, out, 0)
    torch.cuda.current_stream().wait_stream(side)
    for k in (1, 0, 1):
        for a, b in zip(live, dev[k]):
            a.copy_(b)
        graph.replay()
        assert np.array_equal(out.cpu().numpy(), want[k])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.zeros(300, 200, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                call(dev[k], got[k], 1 + k)
    torch.cuda.synchronize()
    for k in range(2):
        assert np.array_equal(got[k].cpu().numpy(), want[k])


@pytest.mark.parametrize("counts", [[3, 40, 8], [300, 5, 209]])  # single CTAs, pairs
def test_grouped_wait_runs_out(counts):
    """A copy left out: the wait for it runs out, the call reports it and returns; the next call is right."""
    rng = np.random.default_rng(15)
    n = sum(counts)
    x, w = operands(rng, n, 300, 4096, 3, [127])
    ws = torch.empty(jm.jamba_moe_grouped_mx4_workspace_size(n, 300, 4096, 3), dtype=torch.uint8, device="cuda")
    args = [cuda(x[0]), cuda(x[1]), cuda(offsets_of(counts).astype(np.int32)), cuda(w[0]), cuda(w[1])]
    jm.jamba_moe_debug_skip_copy(True)
    try:
        jm.jamba_moe_grouped_mx4(*args, out_dtype=torch.float32, workspace=ws)
        assert jm.jamba_moe_read_device_status(ws) == 5
    finally:
        jm.jamba_moe_debug_skip_copy(False)
    y = jm.jamba_moe_grouped_mx4(*args, out_dtype=torch.float32, workspace=ws)
    assert jm.jamba_moe_read_device_status(ws) == 0
    assert np.array_equal(y.cpu().numpy(), ref.grouped(ref.values(*x), offsets_of(counts), ref.values(*w))[0])


def test_memory_of_calls_on_a_given_stream():
    """What a call on another stream allocated for itself is not handed out again while that stream is still before it."""
    rng = np.random.default_rng(16)
    x, w = operands(rng, 40, 300, 512, 2, [127])
    args = [cuda(x[0]), cuda(x[1]), cuda(np.array([0, 30, 40], np.int32)), cuda(w[0]), cuda(w[1])]
    L = Layer(20, 256, 256)
    fixed = [bf16_to_dev(L.x), torch.from_numpy(L.wr).cuda(), None if L.bias is None else cuda(L.bias), *L.dev]
    want = jm.jamba_moe_forward_mx4(*fixed)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # some 50 ms
    y = jm.jamba_moe_grouped_mx4(*args, out_dtype=torch.float32, stream=side)
    z = jm.jamba_moe_forward_mx4(*fixed, stream=side)[0]
    sizes = [4096, 512, jm.jamba_moe_workspace_size_mx4(20, 256, 256)]
    others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in others)
    assert np.array_equal(y.cpu().numpy(), ref.grouped(ref.values(*x), [0, 30, 40], ref.values(*w))[0])
    assert torch.equal(z, want)


def test_grouped_deterministic():
    rng = np.random.default_rng(14)
    x, w = operands(rng, 700, 300, 4096, 4, range(110, 140))
    off = offsets_of([5, 600, 0, 95])
    a = run_grouped(x, w, off)
    for _ in range(3):
        assert torch.equal(a, run_grouped(x, w, off))


def test_far_rows_of_a_long_batch():
    """Outputs and operands whose byte offsets pass 2^31: the last rows of the largest batch."""
    n, rows, cols = 1 << 20, 1100, 4224  # y: 4.6 GB in fp32, x codes 2.2 GB
    g = torch.Generator("cuda").manual_seed(5)
    xq = torch.randint(0, 256, (n, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
    xs = torch.full((n, cols // 32), 127, dtype=torch.uint8, device="cuda")
    q = torch.randint(0, 256, (2, rows, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
    s = torch.full((2, rows, cols // 32), 127, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, n - 300, n], dtype=torch.int32, device="cuda")
    y = jm.jamba_moe_grouped_mx4(xq, xs, off, q, s, out_dtype=torch.float32)
    for r, e in ((slice(0, 40), 0), (slice(n - 340, n - 300), 0), (slice(n - 300, n), 1)):
        xv, wv = ref.values(xq[r].cpu().numpy(), xs[r].cpu().numpy()), ref.values(q[e].cpu().numpy(), s[e].cpu().numpy())
        want = xv @ wv.T
        assert np.array_equal(y[r].cpu().numpy(), want)


# ------------------------------------------------------------------ the layer
class Layer:
    def __init__(self, T, d, F, name="tiny"):
        wl = dataclasses.replace(workload(name), T=T, d=d, F=F)
        inp = gap_inputs(wl)
        self.x, self.wr, self.bias = inp["x"], inp["wr"], inp["bias"]
        self.w = [synth.gen_experts(wl, which) for which in ("w1", "w3", "w2")]
        self.dev = [t for w in self.w for t in jm.jamba_moe_quantize_mx4(bf16_to_dev(w))]

    def forward(self, **kw):
        bias = None if self.bias is None else torch.from_numpy(self.bias).cuda()
        return jm.jamba_moe_forward_mx4(bf16_to_dev(self.x), torch.from_numpy(self.wr).cuda(), bias, *self.dev, **kw)

    def ref(self):
        return ref.layer(self.x, self.wr, self.bias, *[ref.values(*ref.quantize(w)) for w in self.w])


@pytest.mark.parametrize("T,d,F", [(1, 256, 512), (3, 128, 128), (17, 384, 640), (64, 256, 512), (129, 256, 1152),
                                   (700, 128, 256)])
def test_layer(T, d, F):
    """Within the layer tolerance of the other paths: only codes of h whose fp32 value sits within rounding
    distance of a code's border can differ, ~1e-5 of them, each moving y by well under the tolerance."""
    L = Layer(T, d, F)
    y, ids, w = L.forward()
    want, rid, rw, z = L.ref()
    assert_routing(ids.cpu().numpy(), w.cpu().numpy(), rid, rw, z)
    assert_y_close(dev_to_bf16_bits(y), want)


def test_layer_one_expert_and_checks():
    """A bias that sends every token to the same two experts; the debug checks find nothing amiss."""
    L = Layer(200, 256, 384)
    L.bias = np.zeros(16, np.float32)
    L.bias[[3, 11]] = [60, 50]
    ws = torch.empty(jm.jamba_moe_workspace_size_mx4(200, 256, 384), dtype=torch.uint8, device="cuda")
    jm.jamba_moe_debug_checks(True)
    try:
        y, ids, _ = L.forward(workspace=ws)
        assert jm.jamba_moe_read_device_status(ws) == 0
    finally:
        jm.jamba_moe_debug_checks(False)
    assert (ids.cpu().numpy() == [3, 11]).all()
    assert_y_close(dev_to_bf16_bits(y), L.ref()[0])
    assert torch.equal(y, L.forward()[0])  # the same bits again, with a new workspace


def test_layer_bad_routing_id_is_reported():
    """The corruption hook puts one routing id out of range: reported, the other tokens' results are right."""
    L = Layer(70, 256, 256)
    ws = torch.empty(jm.jamba_moe_workspace_size_mx4(70, 256, 256), dtype=torch.uint8, device="cuda")
    want = L.forward()[0]
    ws.fill_(0x11)
    jm.jamba_moe_debug_corrupt(jm.CORRUPT_ROUTE_ID)  # of assignment 0: token 0
    y = L.forward(workspace=ws)[0]
    assert jm.jamba_moe_read_device_status(ws) == 6
    assert torch.equal(y[1:], want[1:])
    # x on a 16-byte boundary only
    x = torch.zeros(70 * 256 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(70, 256)
    x.copy_(bf16_to_dev(L.x))
    y = jm.jamba_moe_forward_mx4(x, torch.from_numpy(L.wr).cuda(), None if L.bias is None else cuda(L.bias), *L.dev)[0]
    assert torch.equal(y, want)


@pytest.mark.parametrize("T", [20, 900])  # single CTAs, pairs
def test_layer_wait_runs_out(T):
    L = Layer(T, 1024, 256)
    ws = torch.empty(jm.jamba_moe_workspace_size_mx4(T, 1024, 256), dtype=torch.uint8, device="cuda")
    want = L.forward()[0]
    jm.jamba_moe_debug_skip_copy(True)
    try:
        L.forward(workspace=ws)
        assert jm.jamba_moe_read_device_status(ws) == 5
    finally:
        jm.jamba_moe_debug_skip_copy(False)
    assert torch.equal(L.forward(workspace=ws)[0], want)
    assert jm.jamba_moe_read_device_status(ws) == 0


@pytest.mark.parametrize("T", [20, 600])
def test_layer_captured(T):
    """Two graphs of the layer that share one workspace, replayed in turn, follow their inputs."""
    a, b = Layer(T, 256, 384), Layer(T, 256, 384)
    b.x = synth.f32_to_bf16_bits(-synth.bf16_bits_to_f32(a.x))
    want = [L.forward()[0] for L in (a, b)]
    ws = torch.empty(jm.jamba_moe_workspace_size_mx4(T, 256, 384), dtype=torch.uint8, device="cuda")
    wr = torch.from_numpy(a.wr).cuda()
    bias = None if a.bias is None else cuda(a.bias)
    side = torch.cuda.Stream()
    graphs, outs, xs = [], [], [bf16_to_dev(L.x) for L in (a, b)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for L, x in zip((a, b), xs):
            y = torch.zeros(T, 256, dtype=torch.bfloat16, device="cuda")
            ids, w = torch.zeros(T, 2, dtype=torch.int32, device="cuda"), torch.zeros(T, 2, device="cuda")
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                jm.jamba_moe_forward_mx4(x, wr, bias, *L.dev, y=y, topk_ids=ids, topk_w=w, workspace=ws)
            graphs.append(g)
            outs.append((y, ids, w))
        for k in (0, 1, 1, 0):
            graphs[k].replay()
            side.synchronize()
            assert torch.equal(outs[k][0], want[k]) and jm.jamba_moe_read_device_status(ws, stream=side) == 0
            outs[k][0].zero_()


def test_layer_no_tokens():
    L = Layer(1, 128, 128)
    L.x = L.x[:0]
    y, ids, w = L.forward()
    assert y.shape == (0, 128) and ids.shape == (0, 2) and w.shape == (0, 2)


def test_operators_together():
    """The operators as a program composes them: tokens packed by expert, quantized rows, the up products, SwiGLU,
    the down product, weighted sum; and the whole-layer call on the same inputs."""
    L = Layer(90, 256, 512)
    x = bf16_to_dev(L.x)
    d = jm.jamba_moe_ep_dispatch(x, torch.from_numpy(L.wr).cuda(), None if L.bias is None else cuda(L.bias), 1)
    counts = torch.bincount(d["send_expert"].long(), minlength=16)
    off = torch.cat((counts.new_zeros(1), counts.cumsum(0))).int()
    q1, s1, q3, s3, q2, s2 = L.dev
    xq, xs = jm.jamba_moe_quantize_mx4(d["send_x"])
    g = jm.jamba_moe_grouped_mx4(xq, xs, off, q1, s1, out_dtype=torch.float32)
    u = jm.jamba_moe_grouped_mx4(xq, xs, off, q3, s3, out_dtype=torch.float32)
    h = (torch.nn.functional.silu(g) * u).bfloat16()
    o = jm.jamba_moe_grouped_mx4(*jm.jamba_moe_quantize_mx4(h), off, q2, s2, out_dtype=torch.float32)
    y = jm.jamba_moe_ep_combine((o * d["send_w"][:, None]).contiguous(), d["pos"])
    want = L.ref()[0]
    assert_y_close(dev_to_bf16_bits(y), want)
    assert_y_close(dev_to_bf16_bits(L.forward()[0]), want)
