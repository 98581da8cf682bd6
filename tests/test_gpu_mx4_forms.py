"""Every form of the product at its own sizes: few rows, tiles of 64, parts of a long sum,
tiles of 128 over several chunks, tiles of 256.  Operands are chosen so that every sum is
exact in binary32 whatever its order, and results are compared bit for bit."""

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from tests import helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    H.need_gpu()
    yield
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


VALUES = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def exact_operand(rows, k, seed):
    """An Mx4 of random codes with scales of 1/2, 1 and 2, and its values (float64, on the
    device).  Products are multiples of 1/16 of at most 144, so k of them have an exact sum
    in 24 bits for k up to 2^24 / (16 * 144) = 7281."""
    import torch
    assert k <= 7281
    g = torch.Generator(device=H.dev()).manual_seed(seed)
    kb = -(-k // 32)
    code = torch.randint(0, 16, (rows, kb * 32), dtype=torch.uint8, device=H.dev(), generator=g)
    code[:, k:] = 0
    scales = torch.randint(126, 129, (rows, kb), dtype=torch.uint8, device=H.dev(), generator=g)
    values = torch.tensor(VALUES, dtype=torch.float64, device=H.dev())[code.long()]
    values = (values.view(rows, kb, 32) * torch.exp2(scales.double() - 127)[..., None]).flatten(1)
    codes = (code[:, 0::2] | code[:, 1::2] << 4).contiguous()
    return sbp.Mx4(codes, scales, (rows, k)), values[:, :k]


# tiles of 128: whole chunks of 512 values (kb a multiple of 16), k that end in a block too
MIDDLE = [(2048, 2048, 4096), (2047, 2050, 1505), (1700, 1750, 1000), (1600, 2100, 2560),
          (1801, 1900, 2048)]


@pytest.mark.parametrize("m,n,k", MIDDLE)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (1, 0), (3, 5)])
@pytest.mark.parametrize("form", ["bf16", "f32", "accumulate"])
def test_tiles_of_128_over_several_chunks(m, n, k, pad, shift, form):
    import torch
    a, av = exact_operand(m, k, 1)
    b, bv = exact_operand(n, k, 2)
    dtype = torch.bfloat16 if form == "bf16" else torch.float32
    whole = torch.full((shift + m * (n + pad),), 9.0, dtype=dtype, device=H.dev())
    out = whole[shift:].view(m, n + pad)[:, :n]
    sbp.mx_matmul(a, b, out, accumulate=form == "accumulate")
    # with 9: a multiple of 1/16 below 2^20 + 9, one rounding at the most
    want = (av @ bv.T).float()
    want = want + 9.0 if form == "accumulate" else want.to(dtype)
    assert torch.equal(out, want)
    rest = whole.clone()
    rest[shift:].view(m, n + pad)[:, :n] = 9.0
    assert bool((rest == 9.0).all())


@pytest.mark.parametrize("m,n,k", MIDDLE[:3])
def test_tiles_of_128_nan_and_scales_anywhere(m, n, k):
    """A NaN block in the first, a middle and the last chunk takes its row or column, with
    scales at an odd address."""
    import torch
    a, av = exact_operand(m, k, 3)
    b, bv = exact_operand(n, k, 4)
    want = (av @ bv.T).float()
    kb = a.scales.shape[1]
    wide = torch.zeros(3 + m * kb, dtype=torch.uint8, device=H.dev())
    scales = wide[3:].view(m, kb)
    scales.copy_(a.scales)
    a = sbp.Mx4(a.codes, scales, (m, k))
    assert torch.equal(sbp.mx_matmul(a, b, dtype=torch.float32), want)
    for row, block in ((m - 1, kb - 1), (m // 2, kb // 2), (0, 0)):
        scales[row, block] = 255
        want[row] = float("nan")
    b.scales[n - 2, kb // 2 + 1] = 255
    want[:, n - 2] = float("nan")
    got = sbp.mx_matmul(a, b, dtype=torch.float32)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))


# a size of each form: few rows, tiles of 64, parts, tiles of 128 and of 256
SIZES = [(20, 20, 160), (1, 300, 2048), (65, 130, 1024), (70, 61, 6144), (300, 700, 128),
         (1700, 1750, 1024), (2900, 2952, 160)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("sa,sb", [(252, 120), (10, 100), (0, 0), (254, 254), (0, 254), (254, 0),
                                   (0, 105), (0, 127), (1, 127), (240, 128), (250, 126), (130, 0)])
def test_scales_at_both_ends(m, n, k, sa, sb):
    """All ones: sums of k equal powers of two, exact down to the least subnormal, and
    infinity from 2^128 on; in bf16 the same rounded once, subnormals too."""
    import torch
    q = [sbp.Mx4(torch.full((rows, k // 2), 0x22, dtype=torch.uint8, device=H.dev()),
                 torch.full((rows, k // 32), s, dtype=torch.uint8, device=H.dev()), (rows, k))
         for rows, s in ((m, sa), (n, sb))]
    with np.errstate(over="ignore"):
        want = float(np.float32(np.float64(k) * 2.0 ** (sa - 127.0) * 2.0 ** (sb - 127.0)))
    got = sbp.mx_matmul(*q, dtype=torch.float32)
    assert bool((got == want).all()), (got.min(), got.max(), want)
    half = float(torch.tensor(want).bfloat16())
    got = sbp.mx_matmul(*q)
    assert bool((got == half).all()), (got.min(), got.max(), half)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_order_of_a_sum_depends_on_the_sizes_alone(m, n, k):
    """The same bits every time, and with the rows of both operands in another order: on
    values whose sums round."""
    import torch
    from tests.test_gpu_mx4 import _operand
    a, b = _operand(m, k, 5)[0], _operand(n, k, 6)[0]
    first = sbp.mx_matmul(a, b, dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(sbp.mx_matmul(a, b, dtype=torch.float32), first)
    pa, pb = (torch.randperm(r, generator=torch.Generator().manual_seed(r)).to(H.dev())
              for r in (m, n))
    moved = [sbp.Mx4(q.codes[p], q.scales[p], q.shape) for q, p in ((a, pa), (b, pb))]
    assert torch.equal(sbp.mx_matmul(*moved, dtype=torch.float32), first[pa][:, pb])
