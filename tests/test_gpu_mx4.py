"""GPU parity of the microscaled 4-bit calls with the oracle: quantization,
values and the reduce bit for bit, products against 64 bits, and the calls
together as an exchange and a layer's training step use them."""

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from oracle import mx4 as OM
from oracle import step as OS
from tests import helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    H.need_gpu()
    yield
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _data(rows, cols, seed, kind="normal"):
    """float32 values that bf16 holds exactly."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))
    if kind == "wide":  # exponents over binary32's whole range, subnormals among them
        x = x * 2.0 ** rng.integers(-140, 120, (rows, -(-cols // 32))).repeat(32, 1)[:, :cols]
    if kind == "special":
        x[rng.random(x.shape) < 0.02] = 0.0
        x[rng.random(x.shape) < 0.02] = -0.0
        for bad in (np.nan, np.inf, -np.inf):
            x[rng.random(x.shape) < 0.005] = bad
        x[rng.random(rows) < 0.2] = 0.0
    with np.errstate(all="ignore"):
        return OS.bf16_to_f32(OS.f32_to_bf16(x.astype(np.float32)))


def _device(x, dtype, pad=0, shift=0):
    """x on the device, rows `pad` elements further apart than they are long,
    from element `shift` of a buffer on."""
    import torch
    t = torch.from_numpy(x).to(H.dev())
    t = t if dtype == "f32" else t.bfloat16()
    rows, cols = x.shape
    wide = torch.full((shift + rows * (cols + pad),), 7.0, dtype=t.dtype, device=t.device)
    view = wide[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def _guarded_mx4(rows, cols):
    """An Mx4 inside guard bytes, and a check of them."""
    import torch
    kb = -(-cols // 32)
    big = [torch.full((rows * w + 512,), 0xA5, dtype=torch.uint8, device=H.dev())
           for w in (16 * kb, kb)]
    q = sbp.Mx4(*(b[256:256 + rows * w].view(rows, w) for b, w in zip(big, (16 * kb, kb))),
                (rows, cols))
    return q, lambda: all(bool((b[:256] == 0xA5).all() and (b[-256:] == 0xA5).all()) for b in big)


def _same_codes(q, want, what):
    code, scale = want
    got = q.codes.cpu().numpy()
    H.assert_bits_equal(q.scales.cpu().numpy(), scale, f"{what} scales")
    H.assert_bits_equal(got, OM.pack(code), f"{what} codes")


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (1, 8191), (1, 100003), (3, 64), (33, 1), (128, 128),
          (129, 127), (31, 257), (300, 96), (257, 400)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("along", ["rows", "cols", "both"])
@pytest.mark.parametrize("seed", [None, 0xFEDCBA9876543210])
def test_quantize(shape, dtype, along, seed):
    x = _data(*shape, 1)
    if dtype == "f32":  # all 24 bits
        x = x * np.float32(1 + 2.0 ** -9)
    d = _device(x, dtype)
    shapes = {"rows": [shape], "cols": [shape[::-1]], "both": [shape, shape[::-1]]}[along]
    outs = [_guarded_mx4(*s) for s in shapes]
    out = [q for q, _ in outs]
    sbp.mx_quantize(d, along, out if along == "both" else out[0], seed, offset=(5 << 32) + 9)
    import torch
    torch.cuda.synchronize()
    if along != "cols":
        _same_codes(out[0], OM.quantize(x, seed, (5 << 32) + 9), "rows")
    if along != "rows":
        _same_codes(out[-1], OM.quantize(x.T, seed, (5 << 32) + 9, True), "cols")
    assert all(intact() for _, intact in outs)


@pytest.mark.parametrize("kind", ["wide", "special"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seed", [None, 77])
def test_quantize_extremes(kind, dtype, seed):
    x = _data(70, 200, 2, kind)
    a, t = sbp.mx_quantize(_device(x, dtype), "both", seed=seed)
    _same_codes(a, OM.quantize(x, seed), "rows")
    _same_codes(t, OM.quantize(x.T, seed, 0, True), "cols")
    flat = x.reshape(1, -1)
    _same_codes(sbp.mx_quantize(_device(flat, dtype)[0], seed=seed), OM.quantize(flat, seed), "flat")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (8, 8), (64, 3)])
def test_quantize_strided_and_unaligned(dtype, pad, shift):
    """The same codes wherever the rows lie."""
    x = _data(75, 224, 3)
    d = _device(x, dtype, pad, shift)
    for seed in (None, 4):
        a, t = sbp.mx_quantize(d, "both", seed=seed)
        _same_codes(a, OM.quantize(x, seed), "rows")
        _same_codes(t, OM.quantize(x.T, seed, 0, True), "cols")
        _same_codes(sbp.mx_quantize(d, seed=seed), OM.quantize(x, seed), "rows alone")


@pytest.mark.parametrize("n", [4 * 256 * 256 * 8 - 5, 4 * 256 * 256 * 8 + 32 * 7 + 3])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("seed", [None, 8])
def test_quantize_long(n, shift, seed):
    """Around the length from which a lane takes several octets."""
    x = _data(1, n, 4)
    q = sbp.mx_quantize(_device(x, "bf16", 0, shift)[0], seed=seed)
    _same_codes(q, OM.quantize(x, seed), f"n={n}")


@pytest.mark.parametrize("shape", SHAPES + [(1, 4 * 256 * 256 * 8 + 9), (700, 12001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_dequantize(shape, dtype, pad, shift):
    import torch
    rng = np.random.default_rng(5)
    kb = -(-shape[1] // 32)
    codes = rng.integers(0, 256, (shape[0], kb * 16), np.uint8)
    scales = rng.integers(0, 256, (shape[0], kb), np.uint8)
    q = sbp.Mx4(torch.from_numpy(codes).to(H.dev()), torch.from_numpy(scales).to(H.dev()), shape)
    out = _device(np.zeros(shape, np.float32), dtype, pad, shift)
    whole = out._base
    sbp.mx_dequantize(q, out)
    with np.errstate(over="ignore"):
        want = OM.values(codes, scales, shape[1]).astype(np.float32)
    got = out.float().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got[want == 0]), np.signbit(want[want == 0]))
    # what lies between and before the rows is left as it was
    rest = whole.clone()
    rest[shift:].view(shape[0], -1)[:, :shape[1]] = 7.0
    assert bool((rest == 7.0).all())


def test_dequantize_makes_its_output():
    import torch
    x = _data(40, 100, 6)
    q = sbp.mx_quantize(_device(x, "f32"))
    a, b = sbp.mx_dequantize(q), sbp.mx_dequantize(q, dtype=torch.float32)
    assert a.dtype == torch.bfloat16 and b.dtype == torch.float32 and a.shape == b.shape == x.shape
    code, scale = OM.quantize(x)
    want = OM.values(OM.pack(code), scale, 100)
    assert np.array_equal(b.cpu().numpy(), want) and bool((a.float() == b).all())


# ---- reduce ----------------------------------------------------------------------------

def _peers(R, n, seed, special=False):
    """R peers as the device has them, and their float32 values."""
    import torch
    rng = np.random.default_rng(seed)
    kb = -(-n // 32)
    peers, values = [], []
    for _ in range(R):
        codes = rng.integers(0, 256, (1, kb * 16), np.uint8)
        scales = rng.integers(0 if special else 110, 256 if special else 124, (1, kb), np.uint8)
        peers.append(sbp.Mx4(torch.from_numpy(codes).to(H.dev()),
                             torch.from_numpy(scales).to(H.dev()), (1, n)))
        with np.errstate(over="ignore"):
            values.append(OM.values(codes, scales, n)[0].astype(np.float32))
    return peers, values


@pytest.mark.parametrize("n", [1, 7, 8, 33, 2047, 100003, 300 * 2048 + 5])
@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 8, 16])
@pytest.mark.parametrize("acc", ["none", "other", "in place"])
def test_reduce(n, R, acc):
    import torch
    peers, values = _peers(R, n, 7)
    before = np.random.default_rng(8).standard_normal(n).astype(np.float32)
    whole, out, guard = H.guarded_from(before)
    a = {"none": None, "other": torch.from_numpy(before).to(H.dev()), "in place": out}[acc]
    scale = np.float32(1 / 3)
    sbp.mx_reduce_shard(peers, a, scale, out)
    torch.cuda.synchronize()
    want = OM.reduce(values, None if acc == "none" else before, scale)
    H.assert_bits_equal(H.to_np_f32(out), want, f"R={R} n={n} {acc}")
    assert H.canaries_intact(whole, guard)


@pytest.mark.parametrize("R", [1, 3, 8])
def test_reduce_extremes(R):
    """Every scale, NaN among them, and sums that overflow."""
    import torch
    peers, values = _peers(R, 9999, 9, special=True)
    out = torch.empty(9999, device=H.dev())
    sbp.mx_reduce_shard(peers, None, 1.0, out)
    got, want = H.to_np_f32(out), OM.reduce(values, None, 1.0)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    H.assert_bits_equal(got[ok], want[ok], "extremes")


# ---- products ----------------------------------------------------------------------------
# Tolerance.  A product of two values is exact in the matrix unit; the k products
# of an entry are summed in binary32, k roundings of at most 2^-24 of the sum of
# their magnitudes each, whatever the order (joining partial sums adds no more
# than one rounding a part, and there are fewer parts than products).  A bf16
# output adds half a step, 2^-8 of the entry's own magnitude; accumulating adds a
# rounding of 2^-24 of the sum with the accumulator.

def _operand(rows, k, seed):
    """An Mx4 on the device and its float64 values: normal rows of sizes around
    one, and some blocks of zeros."""
    x = _data(rows, k, seed)
    x[np.random.default_rng(seed + 1).random(x.shape) < 0.1] = 0
    code, scale = OM.quantize(x)
    import torch
    q = sbp.Mx4(torch.from_numpy(OM.pack(code)).to(H.dev()), torch.from_numpy(scale).to(H.dev()),
                (rows, k))
    return q, OM.values(OM.pack(code), scale, k)


def _check_product(got, a, b, bf16, before=None, what=""):
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = a.shape[1] * 2.0 ** -24 * size
    if before is not None:
        want = want + before
        tol = tol + 2.0 ** -24 * (np.abs(want) + tol)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    off = np.abs(got.astype(np.float64) - want)
    worst = np.argmax(off - tol)
    assert (off <= tol).all(), (f"{what}: {(off > tol).sum()} entries off, worst at {worst}: "
                                f"{got.ravel()[worst]} for {want.ravel()[worst]}")


PRODUCTS = [(1, 1, 1), (1, 16, 32), (2, 3, 5), (1, 4096, 4096), (7, 100, 777), (16, 1000, 256),
            (17, 33, 129), (40, 2000, 600), (64, 64, 64), (65, 130, 1000), (128, 128, 128),
            (130, 260, 100), (200, 300, 2080), (256, 256, 512), (257, 255, 545), (509, 1021, 777),
            (640, 768, 768), (31, 5, 20000), (300, 140, 33), (1030, 520, 96),
            # on both sides of where the form changes: few rows, tiles, parts of the sum
            (1, 9000, 100), (2, 9000, 544), (16, 8192, 64), (17, 8192, 64), (32, 4096, 100),
            (33, 4096, 100), (100, 300, 8192), (70, 61, 6144), (70, 61, 6113), (64, 1024, 7200),
            (5, 8200, 6200), (1300, 1100, 544), (1300, 1101, 1056)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("form", ["bf16", "f32", "accumulate"])
def test_matmul(m, n, k, form):
    import torch
    a, av = _operand(m, k, 10)
    b, bv = _operand(n, k, 20)
    dtype = torch.bfloat16 if form == "bf16" else torch.float32
    before = np.random.default_rng(3).standard_normal((m, n)).astype(np.float32)
    whole = torch.full((m + 2, n + 24), 9.0, dtype=dtype, device=H.dev())
    out = whole[1:m + 1, 8:8 + n]
    out.copy_(torch.from_numpy(before))
    got = sbp.mx_matmul(a, b, out, accumulate=form == "accumulate")
    assert got is out
    _check_product(got.float().cpu().numpy(), av, bv, form == "bf16",
                   before if form == "accumulate" else None, f"{m}x{n}x{k}")
    rest = whole.clone()
    rest[1:m + 1, 8:8 + n] = 9.0
    assert bool((rest == 9.0).all())


@pytest.mark.parametrize("m,n,k", [(m, n, k) for m, n in ((1700, 1750), (2900, 2952), (2817, 2817))
                                   for k in (1, 33, 97, 128, 129, 500, 512, 520, 1100)]
                         # more tiles than compute units: several to a block
                         + [(4400, 4304, k) for k in (100, 512, 1600)]
                         + [(4353, 4351, 700), (1100, 20008, 200), (20001, 1000, 40)])
@pytest.mark.parametrize("form", ["bf16", "accumulate"])
def test_matmul_large(m, n, k, form):
    """Larger tiles, at contracted lengths that end anywhere in a slice and in a
    chunk of four."""
    import torch
    a, av = _operand(m, k, 15)
    b, bv = _operand(n, k, 25)
    if form == "bf16":
        out, before = sbp.mx_matmul(a, b), None
    else:
        out = torch.randn(m, n, device=H.dev())
        before = out.cpu().numpy()
        sbp.mx_matmul(a, b, out, accumulate=True)
    _check_product(out.float().cpu().numpy(), av, bv, form == "bf16", before, f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(1, 512, 1024), (50, 70, 300), (300, 512, 512), (513, 300, 640)])
@pytest.mark.parametrize("ld,shift", [(0, 0), (1, 0), (8, 1), (3, 5)])
def test_matmul_output_strides(m, n, k, ld, shift):
    import torch
    a, av = _operand(m, k, 11)
    b, bv = _operand(n, k, 21)
    for dtype in (torch.bfloat16, torch.float32):
        whole = torch.full((shift + m * (n + ld),), 9.0, dtype=dtype, device=H.dev())
        out = whole[shift:].view(m, n + ld)[:, :n]
        sbp.mx_matmul(a, b, out)
        _check_product(out.float().cpu().numpy(), av, bv, dtype == torch.bfloat16, what=f"{ld}")
        rest = whole.clone()
        rest[shift:].view(m, n + ld)[:, :n] = 9.0
        assert bool((rest == 9.0).all())


@pytest.mark.parametrize("m,n,k", [(3, 40, 200), (70, 90, 1000), (300, 280, 700), (520, 530, 300),
                                   (1700, 1730, 300), (2900, 2950, 300)])
def test_matmul_nan_stays_in_its_row(m, n, k):
    """A NaN block of A takes its row of C, one of B its column; the rest has the
    same bits as without them."""
    import torch
    a, _ = _operand(m, k, 12)
    b, _ = _operand(n, k, 22)
    clean = sbp.mx_matmul(a, b, dtype=torch.float32)
    a.scales[m // 2, -1] = 255
    b.scales[n - 1, 0] = 255
    got = sbp.mx_matmul(a, b, dtype=torch.float32)
    nan = torch.zeros((m, n), dtype=torch.bool, device=H.dev())
    nan[m // 2] = True
    nan[:, n - 1] = True
    assert bool((got.isnan() == nan).all()) and bool((got[~nan] == clean[~nan]).all())


def test_matmul_extreme_scales():
    """Scales at both ends: products near 2^126 and at the least subnormals."""
    import torch
    for sa, sb in ((252, 120), (10, 100), (0, 0), (254, 254), (0, 254)):
        codes = torch.full((20, 16 * 5), 0x22, dtype=torch.uint8, device=H.dev())  # all ones
        q = [sbp.Mx4(codes, torch.full((20, 5), s, dtype=torch.uint8, device=H.dev()), (20, 160))
             for s in (sa, sb)]
        got = sbp.mx_matmul(*q, dtype=torch.float32)
        want = np.float64(160.0) * 2.0 ** (sa - 127.0) * 2.0 ** (sb - 127.0)
        with np.errstate(over="ignore"):
            assert bool((got == float(np.float32(want))).all()), (sa, sb, got[0, 0], want)


def test_matmul_rows_of_a_buffer():
    """Operands that are rows of larger ones, scales at odd addresses."""
    a, av = _operand(70, 160, 13)
    b, bv = _operand(90, 160, 23)
    got = sbp.mx_matmul(a.rows_of(3, 60), b.rows_of(1, 88))
    _check_product(got.float().cpu().numpy(), av[3:60], bv[1:88], True, what="views")


def test_matmul_empty():
    import torch
    e = lambda r, c: sbp.Mx4.empty(r, c, H.dev())  # noqa: E731
    assert sbp.mx_matmul(e(0, 64), e(5, 64)).shape == (0, 5)
    assert sbp.mx_matmul(e(5, 64), e(0, 64)).shape == (5, 0)
    assert bool((sbp.mx_matmul(e(300, 0), e(1111, 0)) == 0).all())
    out = torch.full((7, 9), 2.5, device=H.dev())
    sbp.mx_matmul(e(7, 0), e(9, 0), out, accumulate=True)
    assert bool((out == 2.5).all())


@pytest.mark.parametrize("m,n,k", [(1, 300, 2000), (300, 520, 1100)])
def test_matmul_is_the_same_every_time(m, n, k):
    import torch
    a, _ = _operand(m, k, 14)
    b, _ = _operand(n, k, 24)
    first = sbp.mx_matmul(a, b, dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(sbp.mx_matmul(a, b, dtype=torch.float32), first)
    # rows do not know of each other, as long as the sizes choose the same form
    same = sbp.mx_matmul(a, b.rows_of(0, n), dtype=torch.float32)
    assert torch.equal(same, first)


def test_calls_refuse_bad_tensors():
    import torch
    q = sbp.Mx4.empty(4, 64, H.dev())
    f = lambda *s: torch.zeros(s, device=H.dev())  # noqa: E731
    for call in (
            lambda: sbp.mx_quantize(f(4, 64), out=sbp.Mx4.empty(4, 65, H.dev())),
            lambda: sbp.mx_quantize(f(64, 4).T), lambda: sbp.mx_quantize(f(4, 64), seed=-1),
            lambda: sbp.mx_quantize(f(4, 64), seed=1 << 64),
            lambda: sbp.mx_quantize(f(4, 64), out=sbp.Mx4.empty(4, 64, "cpu")),
            lambda: sbp.mx_dequantize(q, f(4, 63)), lambda: sbp.mx_dequantize(q, f(64, 4).T),
            lambda: sbp.mx_dequantize(q, f(4, 64), dtype=torch.bfloat16),
            lambda: sbp.mx_dequantize(q, f(4, 64).half()),
            lambda: sbp.mx_reduce_shard([q], None, 1.0, f(255)),
            lambda: sbp.mx_reduce_shard([sbp.Mx4.empty(4, 60, H.dev())], None, 1.0, f(240)),
            lambda: sbp.mx_reduce_shard([q], f(200), 1.0, f(256)),
            lambda: sbp.mx_matmul(q, q, f(4, 5)), lambda: sbp.mx_matmul(q, q, f(4, 4).cpu()),
            lambda: sbp.mx_matmul(q, q, f(4, 4), dtype=torch.bfloat16),
            lambda: sbp.mx_matmul(q, q, f(4, 8)[:, ::2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sbp.SbpError):
        sbp.mx_reduce_shard([], None, 1.0, f(256))


# ---- the calls together ----------------------------------------------------------------

def test_exchange_into_the_step():
    """Two ranks' gradients over two microbatches: quantized at random, exchanged,
    accumulated in fp32, the AdamW step from the accumulator, and its master shard
    to 4 bits and back to bf16 for the all-gather: every array bit for bit."""
    import torch
    R, n, seed = 2, 40003, 99
    rng = np.random.default_rng(30)
    acc_d = torch.zeros(n, device=H.dev())
    acc = np.zeros(n, np.float32)
    for micro in range(2):
        peers, values = [], []
        for r in range(R):
            g = OS.bf16_to_f32(OS.f32_to_bf16((rng.standard_normal(n) * 1e-3).astype(np.float32)))
            off = micro * R + r
            peers.append(sbp.mx_quantize(_device(g[None], "bf16")[0], seed=seed, offset=off))
            c, s = OM.quantize(g[None], seed, off)
            values.append(OM.values(OM.pack(c), s, n)[0].astype(np.float32))
        sbp.mx_reduce_shard(peers, acc_d, 1.0, acc_d)
        acc = OM.reduce(values, acc, 1.0)
    H.assert_bits_equal(H.to_np_f32(acc_d), acc, "accumulator")
    hp = sbp.AdamW(lr=1e-2)
    th = (rng.standard_normal(n) * 0.02).astype(np.float32)
    master = torch.from_numpy(th).to(H.dev())
    m, v = torch.zeros(n, device=H.dev()), torch.zeros(n, device=H.dev())
    p = H.empty_u16(n)
    scale = sbp.mean_scale(R, 2)
    sbp.adamw_shard([], acc_d, scale, master, m, v, p, hp, 1)
    z = np.zeros(n, np.float32)
    want = OS.shard_step([], acc, scale, th, z, z, hp, 1)
    H.assert_bits_equal(H.to_np_f32(master), want[0], "master")
    back = sbp.mx_dequantize(sbp.mx_quantize(master))
    c, s = OM.quantize(want[0][None])
    assert np.array_equal(back.float().cpu().numpy(), OM.values(OM.pack(c), s, n))


def test_layer_step_from_gathered_shards():
    """A weight of whole rows per rank, quantized by each rank, gathered as the
    product's operand; the layer's output and both gradients against 64 bits on
    the quantized values, and the input's gradient against differences of the
    output in its own direction."""
    import torch
    t, d_in, d_out, N = 96, 160, 224, 2
    x, w = _data(t, d_in, 40), _data(d_out, d_in, 41) * np.float32(0.1)
    w = OS.bf16_to_f32(OS.f32_to_bf16(w))
    dy = _data(t, d_out, 42)
    dev = {k: _device(a, "bf16") for k, a in (("x", x), ("w", w), ("dy", dy))}
    shards = [sbp.mx_quantize(dev["w"][r * d_out // N:(r + 1) * d_out // N]) for r in range(N)]
    gathered = sbp.Mx4(torch.cat([q.codes for q in shards]), torch.cat([q.scales for q in shards]),
                       (d_out, d_in))
    whole, wt = sbp.mx_quantize(dev["w"], "both")
    assert torch.equal(gathered.codes, whole.codes) and torch.equal(gathered.scales, whole.scales)
    xq, xt = sbp.mx_quantize(dev["x"], "both")
    gq, gt = sbp.mx_quantize(dev["dy"], "both", seed=6)
    y = sbp.mx_matmul(xq, gathered, dtype=torch.float32)
    dx = sbp.mx_matmul(gq, wt, dtype=torch.float32)
    dw = torch.ones(d_out, d_in, device=H.dev())
    sbp.mx_matmul(gt, xt, dw, accumulate=True)

    def val(a, seed=None, upper=False):
        c, s = OM.quantize(a, seed, 0, upper)
        return OM.values(OM.pack(c), s, a.shape[1])

    X, W, G = val(x), val(w), val(dy, 6)
    WT, GT, XT = val(w.T, upper=True), val(dy.T, 6, True), val(x.T, upper=True)
    _check_product(y.cpu().numpy(), X, W, False, what="y")
    _check_product(dx.cpu().numpy(), G, WT, False, what="dx")
    _check_product(dw.cpu().numpy(), GT, XT, False, np.ones((d_out, d_in)), "dw")
    # <G, y(X + d) - y(X)> = <dx, d> for a linear map: with the operands of the
    # gradient in both places, d one of x's own quantized rows
    d = xq.rows_of(0, 1)
    yd = sbp.mx_matmul(d, sbp.mx_quantize(_device(np.ascontiguousarray(WT.T.astype(np.float32)),
                                                    "f32")), dtype=torch.float32)
    D = val(x[:1])
    W2 = val(WT.T.astype(np.float32))
    _check_product(yd.cpu().numpy(), D, W2, False, what="difference")
    lhs = G[0] @ (D @ W2.T)[0]
    rhs = (G[:1] @ W2)[0] @ D[0]
    assert abs(lhs - rhs) <= 1e-12 * np.abs(G[0]) @ np.abs(D @ W2.T)[0]


def test_captured_and_replayed():
    """The whole run in a graph, replayed with eager calls of other sizes in
    between: every replay has the eager bits."""
    import torch
    t, d_in, d_out = 130, 300, 520
    x, w = _device(_data(t, d_in, 50), "bf16"), _device(_data(d_out, d_in, 51), "bf16")
    R, n = 3, t * d_out
    y = torch.empty(t, d_out, device=H.dev())
    out = torch.empty(n, device=H.dev())
    xq, wq = sbp.Mx4.empty(t, d_in, H.dev()), sbp.Mx4.empty(d_out, d_in, H.dev())
    peers = [sbp.Mx4.empty(1, n, H.dev()) for _ in range(R)]
    back = torch.empty(n, dtype=torch.bfloat16, device=H.dev())
    ws = torch.empty(max(sbp.mx_matmul_workspace(t, d_out, d_in), 1), dtype=torch.uint8,
                     device=H.dev())

    def run():
        sbp.mx_quantize(x, out=xq)
        sbp.mx_quantize(w, out=wq)
        sbp.mx_matmul(xq, wq, y, workspace=ws)
        for r in range(R):
            sbp.mx_quantize(y.view(-1), out=peers[r], seed=r)
        sbp.mx_reduce_shard(peers, None, 0.5, out)
        sbp.mx_dequantize(peers[0], back)

    run()
    torch.cuda.synchronize()
    want = [v.clone() for v in (y, out, back)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(4):
        sbp.mx_matmul(*(sbp.mx_quantize(_device(_data(400, 700, 52), "bf16")),) * 2)
        for v in (y, out):
            v.fill_(float("nan"))
        back.fill_(3.0)
        for q in (xq, wq):
            q.codes.fill_(0x77)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, out, back), want)), rep


def test_two_streams_at_once():
    """Two products on streams of their own, each with its own workspace."""
    import torch
    a, av = _operand(300, 2000, 60)
    b, bv = _operand(280, 2000, 61)
    want = sbp.mx_matmul(a, b, dtype=torch.float32)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [sbp.mx_matmul(a, b, dtype=torch.float32, stream=s) for s in streams * 4]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    x = _device(_data(50, 3000, 62), "bf16")
    torch.cuda.synchronize()
    q = sbp.mx_quantize(x, stream=streams[0])
    v = sbp.mx_dequantize(q, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(v, sbp.mx_dequantize(sbp.mx_quantize(x)))
