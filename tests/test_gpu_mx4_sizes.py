"""The microscaled 4-bit calls at their ends: operands of a few blocks, the longest
sums, buffers past 2^32 bytes and values, scales at any address, and each form of the
product with both kinds of results."""

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from oracle import mx4 as OM
from tests import helpers as H
from tests.test_gpu_mx4 import _check_product, _operand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    H.need_gpu()
    yield
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# an operand of fewer than 16 scales (a lane reads 16, or 8, at a time), next to any other
@pytest.mark.parametrize("m,n,k", [(20001, 1, 32), (20001, 1, 7), (1, 20001, 30), (3, 5000, 100),
                                   (5000, 3, 100), (15, 70000, 32), (70000, 15, 32),
                                   (16, 9000, 32), (300, 5, 96), (8, 9001, 33), (9001, 8, 33),
                                   (40, 40, 1), (4097, 2, 224), (2, 8193, 225)])
@pytest.mark.parametrize("form", ["bf16", "accumulate"])
def test_few_blocks(m, n, k, form):
    import torch
    a, av = _operand(m, k, 31)
    b, bv = _operand(n, k, 32)
    if form == "bf16":
        out, before = sbp.mx_matmul(a, b), None
    else:
        out = torch.randn(m, n, device=H.dev())
        before = out.cpu().numpy()
        sbp.mx_matmul(a, b, out, accumulate=True)
    _check_product(out.float().cpu().numpy(), av, bv, form == "bf16", before, f"{m}x{n}x{k}")


SPARSE = 48  # non-zero values of a row


def _sparse(rows, k, at, seed):
    """An Mx4 of zeros but for +-1 and +-2 at the places `at`, with scales from 1/2 to 2,
    and its values there (float64, on the device): every sum of their products is exact."""
    import torch
    g = torch.Generator(device=H.dev()).manual_seed(seed)
    kb = -(-k // 32)
    codes = torch.zeros((rows, 16 * kb), dtype=torch.uint8, device=H.dev())
    scales = torch.randint(126, 129, (rows, kb), dtype=torch.uint8, device=H.dev(), generator=g)
    kind = torch.randint(0, 4, (rows, len(at)), device=H.dev(), generator=g)
    code = torch.tensor([2, 4, 10, 12], dtype=torch.uint8, device=H.dev())[kind]
    value = torch.tensor([1.0, 2.0, -1.0, -2.0], dtype=torch.float64, device=H.dev())[kind]
    where = torch.tensor(at, device=H.dev())
    for i, place in enumerate(at):
        codes[:, place // 2] |= code[:, i] << (4 * (place % 2))
    value = value * torch.exp2(scales[:, where // 32].double() - 127)
    return sbp.Mx4(codes, scales, (rows, k)), value


def _places(k, seed):
    """The first and the last value and others."""
    at = np.random.default_rng(seed).choice(k, SPARSE, replace=False)
    return sorted({0, k - 1, *at.tolist()})


@pytest.mark.parametrize("m,n,k", [
    (1, 3, sbp.MX_MAX_K), (20, 30, sbp.MX_MAX_K - 31), (40, 70, sbp.MX_MAX_K),
    (300, 310, sbp.MX_MAX_K - 512 + 1), (70, 4200, 500001), (1300, 1400, 131072 + 96),
    (2900, 2950, 131072 + 64 + 5),
    # codes past 2^32 bytes: few rows, tiles, large tiles
    (2, 9000, 1 << 20), (9000, 40, (1 << 20) - 32), (8300, 8290, 1 << 20)])
def test_long_sums_and_operands(m, n, k):
    import torch
    at = _places(k, m)
    a, av = _sparse(m, k, at, 1)
    b, bv = _sparse(n, k, at, 2)
    got = sbp.mx_matmul(a, b, dtype=torch.float32)
    assert bool((got == (av @ bv.T).float()).all())


@pytest.mark.parametrize("m,n", [(1, sbp.MX_MAX_DIM), (17, sbp.MX_MAX_DIM), (sbp.MX_MAX_DIM, 1),
                                 (sbp.MX_MAX_DIM, 33), (65601, 65700)])
def test_results_past_32_bits(m, n):
    import torch
    k = 32
    a, av = _sparse(m, k, list(range(0, 32, 5)), 3)
    b, bv = _sparse(n, k, list(range(0, 32, 5)), 4)
    got = sbp.mx_matmul(a, b)
    for rows in (slice(0, 50), slice(m // 2, m // 2 + 50), slice(max(m - 50, 0), m)):
        for cols in (slice(0, 50), slice(n // 2, n // 2 + 50), slice(max(n - 50, 0), n)):
            assert bool((got[rows, cols] == (av[rows] @ bv[cols].T).bfloat16()).all()), (rows, cols)


@pytest.mark.parametrize("m,n,k,ld", [(3, 50, 64, (1 << 31) + 16), (70, 90, 100, (1 << 26) + 8),
                                      (2900, 2900, 64, 1 << 20)])
def test_result_rows_far_apart(m, n, k, ld):
    import torch
    at = list(range(0, k, 5))
    a, av = _sparse(m, k, at, 5)
    b, bv = _sparse(n, k, at, 6)
    whole = torch.zeros((m - 1) * ld + n + 64, dtype=torch.bfloat16, device=H.dev())
    out = torch.as_strided(whole, (m, n), (ld, 1), 16)
    sbp.mx_matmul(a, b, out)
    assert bool((out == (av @ bv.T).bfloat16()).all())
    assert int(torch.count_nonzero(whole)) == int(torch.count_nonzero(out))


LONG = (1 << 32) + 32 * 1000 + 9


def _noise(n):
    """n bf16 values, their period of 2^20 + 7 no power of two."""
    import torch
    period = (1 << 20) + 7
    g = torch.Generator(device=H.dev()).manual_seed(7)
    one = torch.randn(period, device=H.dev(), generator=g).bfloat16()
    x = torch.empty(n, dtype=torch.bfloat16, device=H.dev())
    for i in range(0, n, period * 256):
        part = x[i:i + period * 256]
        part.copy_(one.repeat(-(-part.numel() // period))[:part.numel()])
    return x


def test_flat_buffers_past_32_bits():
    """A flat buffer of more than 2^32 values and its stretches by themselves: codes,
    values and sums with the same bits."""
    import torch
    x = _noise(LONG)
    q = sbp.mx_quantize(x)
    seeded = sbp.mx_quantize(x, seed=11)
    back = sbp.mx_dequantize(q, dtype=torch.bfloat16).view(-1)
    total = torch.empty(LONG, device=H.dev())
    sbp.mx_reduce_shard([q, seeded], None, 0.5, total)
    for start in (0, 1 << 31, (1 << 32) - 64, (1 << 32), LONG // 32 * 32 - 96):
        stop = min(start + 4096, LONG)
        part = sbp.mx_quantize(x[start:stop].clone())
        blocks = slice(start // 32, -(-stop // 32))
        kb = blocks.stop - blocks.start
        assert torch.equal(q.scales[0, blocks], part.scales[0])
        assert torch.equal(q.codes[0, 16 * blocks.start:16 * blocks.stop], part.codes[0])
        values = sbp.mx_dequantize(part, dtype=torch.float32).view(-1)
        assert torch.equal(back[start:stop].float(), values)
        other = sbp.Mx4(seeded.codes[0, 16 * blocks.start:16 * blocks.stop].clone().view(1, 16 * kb),
                        seeded.scales[0, blocks].clone().view(1, kb), (1, stop - start))
        drawn = sbp.mx_dequantize(other, dtype=torch.float32).view(-1)
        # a code's neighbours are at most 2 apart, in units of the scale, and nothing is cut off
        step = 2.0 * torch.exp2(other.scales[0].float() - 127).repeat_interleave(32)[:stop - start]
        assert bool(((drawn - x[start:stop].float()).abs() < step).all())
        assert torch.equal(total[start:stop], 0.5 * (values + drawn))


def test_matrix_past_32_bits():
    import torch
    rows, cols = 66001, 65600
    x = _noise(rows * cols).view(rows, cols)
    q, t = sbp.mx_quantize(x, "both")
    for r in (0, rows // 2 // 32 * 32, (rows - 40) // 32 * 32):
        part = sbp.mx_quantize(x[r:r + 32].clone())
        assert torch.equal(q.codes[r:r + 32], part.codes)
        assert torch.equal(q.scales[r:r + 32], part.scales)
    for c in (0, cols // 2, cols - 32):
        part = sbp.mx_quantize(x[:, c:c + 32].clone(), "cols")
        assert torch.equal(t.codes[c:c + 32], part.codes)
        assert torch.equal(t.scales[c:c + 32], part.scales)
    del t
    back = sbp.mx_dequantize(q, dtype=torch.bfloat16)
    part = q.rows_of(rows - 33, rows)
    assert torch.equal(back[rows - 33:], sbp.mx_dequantize(part, dtype=torch.bfloat16))


FORMS = [(1, 4096, 2048), (1, 900, 300), (20, 500, 1500), (64, 1024, 7200), (70, 61, 6113),
         (300, 700, 100), (512, 512, 512), (1500, 1500, 1024), (2900, 2952, 300), (4400, 4304, 520)]


@pytest.mark.parametrize("m,n,k", FORMS)
def test_bf16_results_are_the_rounded_fp32_ones(m, n, k):
    import torch
    a, _ = _operand(m, k, 41)
    b, _ = _operand(n, k, 42)
    exact = sbp.mx_matmul(a, b, dtype=torch.float32)
    assert torch.equal(sbp.mx_matmul(a, b), exact.bfloat16())


@pytest.mark.parametrize("m,n,k", FORMS)
@pytest.mark.parametrize("shift", [1, 6])
def test_scales_at_odd_addresses(m, n, k, shift):
    """Scales that end where their buffer ends, at any address: the same bits."""
    import torch
    a, _ = _operand(m, k, 43)
    b, _ = _operand(n, k, 44)
    want = sbp.mx_matmul(a, b)

    def moved(q):
        wide = torch.full((shift + q.scales.numel(),), 255, dtype=torch.uint8, device=H.dev())
        scales = wide[shift:].view(q.scales.shape)
        scales.copy_(q.scales)
        return sbp.Mx4(q.codes, scales, q.shape)

    assert torch.equal(sbp.mx_matmul(moved(a), moved(b)), want)
    assert torch.equal(sbp.mx_matmul(moved(a), b), want)
    back = sbp.mx_dequantize(a, dtype=torch.float32)
    assert torch.equal(sbp.mx_dequantize(moved(a), dtype=torch.float32), back)


def test_the_longest_row_is_the_oracles():
    """One row of 2^23 values, against the oracle."""
    import torch
    n = sbp.MX_MAX_K
    x = np.random.default_rng(51).standard_normal((1, n)).astype(np.float32)
    q = sbp.mx_quantize(torch.from_numpy(x).to(H.dev()))
    code, scale = OM.quantize(x)
    H.assert_bits_equal(q.codes.cpu().numpy(), OM.pack(code), "codes")
    H.assert_bits_equal(q.scales.cpu().numpy(), scale, "scales")
