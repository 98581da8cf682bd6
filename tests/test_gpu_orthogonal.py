"""GPU parity of the momentum-orthogonalising step's calls with the oracle:
momentum and update bit for bit, Newton-Schulz against the iteration in 64
bits, and the three as one step."""

import itertools

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
import synth
from oracle import step as OS
from tests import helpers as H
from tests import ns_models as NS

pytestmark = pytest.mark.gpu

SIZES = [1, 7, 8, 9, 2047, 256 * 8 * 3 + 5]
# tile grids that end in a partial round of the order dealt to the XCDs
ROUNDS = [300 * 2048 + 5]


@pytest.fixture(autouse=True)
def _gpu():
    H.need_gpu()
    yield
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", SIZES + ROUNDS)
@pytest.mark.parametrize("R,with_acc", [(0, True), (1, False), (2, True), (3, False), (8, False),
                                        (8, True), (16, True)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_momentum_shard(n, R, with_acc, nesterov):
    import torch
    m = synth.normal_f32(21, synth.master_stream(0), n, 1e-3)
    mw, md, mg = H.guarded_from(m)
    uw, ud, ug = H.guarded(n, 2)
    acc_d = acc_h = None
    scale = np.float32(sbp.mean_scale(max(R, 1), 2 if with_acc else 1))
    for t in (1, 2):  # the second call continues from the first one's momentum
        if with_acc:
            acc_d = torch.empty(n, dtype=torch.float32, device=H.dev())
            sbp.accumulate_grads(acc_d, H.dev_peers(21, t, 0, 2, n, 1e-3), first=True)
            acc_h = OS.reduce_peers(H.host_peers(21, t, 0, 2, n, 1e-3))
        peers = H.dev_peers(21, t, 1, R, n, 1e-3) if R else []
        sbp.momentum_shard(peers, acc_d, scale, md, ud, 0.95, nesterov)
        S = OS.reduce_peers(H.host_peers(21, t, 1, R, n, 1e-3)) if R else None
        G = S if acc_h is None else acc_h if S is None else acc_h + S
        m, u = OS.momentum_step(G, scale, m, 0.95, nesterov)
    torch.cuda.synchronize()
    H.assert_bits_equal(H.to_np_f32(md), m, f"m R={R} n={n}")
    H.assert_bits_equal(H.to_np_u16(ud), u, f"u R={R} n={n}")
    assert H.canaries_intact(mw, mg) and H.canaries_intact(uw, ug)


SPECIAL = np.array([0x0000, 0x8000, 0x7F80, 0xFF80, 0x7FC1, 0x0001, 0x8001, 0x7F7F, 0xFF7F],
                   np.uint16)


def test_momentum_special_values():
    """Signed zeros, infinities, NaN, subnormals and the largest bf16 in every
    pairing of two peers."""
    import torch
    a, b = (x.ravel() for x in np.meshgrid(SPECIAL, SPECIAL))
    n = a.size
    md = torch.zeros(n, dtype=torch.float32, device=H.dev())
    ud = H.empty_u16(n)
    with np.errstate(all="ignore"):
        sbp.momentum_shard([H.from_np_u16(a), H.from_np_u16(b)], None, 1.0, md, ud, 0.5)
        m, u = OS.momentum_step(OS.reduce_peers([a, b]), 1.0, np.zeros(n, np.float32), 0.5, True)
    torch.cuda.synchronize()
    got = H.to_np_f32(md)
    nan = np.isnan(m)
    assert np.array_equal(nan, np.isnan(got))
    H.assert_bits_equal(got[~nan], m[~nan], "m")
    gu, gn = H.to_np_u16(ud), np.isnan(OS.bf16_to_f32(u))
    assert np.array_equal(gn, np.isnan(OS.bf16_to_f32(gu)))
    H.assert_bits_equal(gu[~gn], u[~gn], "u")


@pytest.mark.parametrize("n", SIZES + ROUNDS)
@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_update_shard(n, wd):
    import torch
    th = synth.normal_f32(22, synth.master_stream(1), n, 0.02)
    u = synth.normal_bf16(22, synth.peer_stream(1, 0, 0), n, 0.02)
    tw, td, tg = H.guarded_from(th)
    pw, pd, pg = H.guarded(n, 2)
    sbp.update_shard(H.from_np_u16(u), td, pd, 0.02, wd)
    torch.cuda.synchronize()
    want, p = OS.update_step(u, th, 0.02, wd)
    H.assert_bits_equal(H.to_np_f32(td), want, f"master n={n}")
    H.assert_bits_equal(H.to_np_u16(pd), p, f"param n={n}")
    assert H.canaries_intact(tw, tg) and H.canaries_intact(pw, pg)


def test_streaming_calls_refuse_bad_tensors():
    import torch
    n = 64
    f = lambda: torch.zeros(n, dtype=torch.float32, device=H.dev())  # noqa: E731
    with pytest.raises(ValueError):
        sbp.momentum_shard([H.empty_u16(n)], None, 1.0, f(), H.empty_u16(n + 1), 0.9)
    with pytest.raises(ValueError):
        sbp.momentum_shard([H.empty_u16(n - 1)], None, 1.0, f(), H.empty_u16(n), 0.9)
    with pytest.raises(ValueError):
        sbp.momentum_shard([H.empty_u16(n)], None, 1.0, f().double(), H.empty_u16(n), 0.9)
    with pytest.raises(ValueError):
        sbp.update_shard(H.empty_u16(n), f(), H.empty_u16(n + 2), 0.1)
    with pytest.raises(ValueError):
        sbp.update_shard(H.empty_u16(2 * n)[::2], f(), H.empty_u16(n), 0.1)


# ---- Newton-Schulz -------------------------------------------------------------------
# Tolerance.  The device rounds X, A and b A + c A A to binary16 and the result
# to bf16; everything else is binary32.  The result's rounding moves each entry
# by at most 2^-8 of it (bf16's half step), so the 2-norm by at most 2^-8.  The
# binary16 roundings are the ones oracle.newton_schulz_rounded makes, in
# float64: its distance from the exact iteration is their effect, and the
# device's roundings, each within the same half steps, are taken to have at
# most twice that.  A binary32 sum of k products adds at most k 2^-24 to an
# entry of A, under a hundredth of binary16's 2^-11 for k <= 64 and, rounding
# at random, for k up to 2^14; the factor of two covers it.

def _tolerance(U, exact, steps, coefs, eps=1e-7):
    r = OS.newton_schulz_rounded(U, steps, coefs, eps)
    return 2.0 ** -8 * np.linalg.norm(exact) + 2 * np.linalg.norm(r - exact)


def _u(shape, seed, kind="strong", size=1e-3):
    """bf16 bits of an update: noise, with a few strong directions over it, or
    four directions and noise 30 times weaker."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape)
    k = min(4, *shape[-2:])
    if kind != "flat":
        s = rng.standard_normal(shape[:-1] + (k,)) @ rng.standard_normal(
            shape[:-2] + (k, shape[-1]))
        x = s + (1.0 if kind == "strong" else 0.03) * x
    return OS.f32_to_bf16((size * x).astype(np.float32))


def _bf(bits):
    """bf16 device tensor of 16-bit patterns."""
    import torch
    return H.from_np_u16(bits).view(torch.bfloat16)


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check_ns(out, bits, steps=5, coefs=sbp.NS_COEFS, eps=1e-7, scale=1.0, what=""):
    """Every matrix of `out` against the 64-bit iteration on `bits`."""
    got = _f64(out).reshape((-1,) + out.shape[-2:])
    U = OS.bf16_to_f32(bits).astype(np.float64).reshape(got.shape)
    for i in range(len(U)):
        want = OS.newton_schulz(U[i], steps, coefs, eps)
        off = np.linalg.norm(got[i] / scale - want)
        tol = _tolerance(U[i], want, steps, coefs, eps)
        assert off <= tol, f"{what} matrix {i}: off by {off:.3e}, tolerance {tol:.3e}"


SHAPES = [(1, 1), (1, 7), (5, 1), (2, 3), (16, 16), (63, 65), (64, 64), (65, 64), (64, 130),
          (130, 64), (127, 300), (300, 128), (256, 1024), (1024, 256), (509, 1021), (777, 640),
          (40, 700), (700, 40), (120, 700), (700, 120), (100, 2500), (2500, 100)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["flat", "strong", "steep"])
def test_newton_schulz_shapes(shape, kind):
    import torch
    bits = _u(shape, 31, kind)
    out, = sbp.newton_schulz([_bf(bits)])
    torch.cuda.synchronize()
    _check_ns(out, bits, what=f"{shape} {kind}")


@pytest.mark.parametrize("shape", [(1, 1048576), (1048576, 3), (100, 200000), (200000, 100),
                                   (130, 100000), (100000, 130)])
def test_newton_schulz_long(shape):
    """Up to SBP_NS_MAX_DIM.  Sums of 2^17.6 products off by 2^-24 of them at
    random are off by 2^-15, which the tolerance's factor of two covers."""
    import torch
    bits = _u(shape, 37)
    out, = sbp.newton_schulz([_bf(bits)])
    torch.cuda.synchronize()
    _check_ns(out, bits, what=str(shape))


@pytest.mark.parametrize("steps", [1, 2])
@pytest.mark.parametrize("shape", [(40, 70), (40, 900), (900, 40), (100, 2500), (2500, 100),
                                   (150, 200), (200, 150)])
def test_newton_schulz_few_steps_in_place(steps, shape):
    """Where the first step is also the last one or next to it, the input is
    read close to the output's stores."""
    import torch
    x = _bf(_u((3,) + shape, 38))
    want, = sbp.newton_schulz([x], steps=steps)
    got, = sbp.newton_schulz([x], out=[x], steps=steps)
    torch.cuda.synchronize()
    assert got.data_ptr() == x.data_ptr()
    assert torch.equal(x.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 16])
@pytest.mark.parametrize("shape", [(30, 90), (500, 20), (70, 200), (200, 70), (90, 700),
                                   (150, 200), (200, 150)])
def test_newton_schulz_steps(steps, shape):
    bits = _u(shape, 32)
    out, = sbp.newton_schulz([_bf(bits)], steps=steps)
    _check_ns(out, bits, steps=steps, what=f"steps {steps}")


def test_newton_schulz_coefficients_per_step():
    bits = _u((96, 160), 33)
    coefs = [(4.0, -6.0, 2.5), (3.5, -5.0, 2.0), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)]
    out, = sbp.newton_schulz([_bf(bits)], steps=4, coefs=coefs)
    _check_ns(out, bits, steps=4, coefs=coefs)


def test_newton_schulz_of_a_scaled_permutation():
    """All singular values equal: the result is the polynomial of one number on
    the permutation, and zero elsewhere, exactly zero."""
    n = 96
    perm = np.random.default_rng(3).permutation(n)
    U = np.zeros((n, n), np.float32)
    U[np.arange(n), perm] = np.where(np.arange(n) % 2, -0.375, 0.375)
    out, = sbp.newton_schulz([_bf(OS.f32_to_bf16(U))])
    got = _f64(out)
    x = 1 / np.sqrt(n)
    for _ in range(5):
        a, b, c = (float(np.float32(v)) for v in sbp.NS_COEFS)
        x = a * x + b * x ** 3 + c * x ** 5
    assert np.all(got[U == 0] == 0)
    # bf16's half step, and per step three binary16 roundings of half a step
    # 2^-11; the polynomial's logarithmic slope is at most 1 along the way up
    # and B's and A's roundings enter X' with weights below 4
    assert np.max(np.abs(got[U != 0] / np.sign(U[U != 0]) - x)) <= x * (2.0 ** -8 + 5 * 9 * 2.0 ** -11)


def test_newton_schulz_batches_groups_and_scales():
    """Groups of different shapes in one call, 2-D and 3-D, with their own
    factors; each result as if called alone, bit for bit."""
    import torch
    shapes = [(3, 64, 200), (200, 64), (2, 33, 47), (1, 128, 128), (90, 500)]
    bits = [_u(s, 40 + i) for i, s in enumerate(shapes)]
    xs = [_bf(b) for b in bits]
    scales = [1.0, 0.5, 2.0, 0.2 * 128 ** 0.5, -1.0]
    outs = sbp.newton_schulz(xs, out_scales=scales)
    for x, o, b, sc in zip(xs, outs, bits, scales):
        _check_ns(o, b, scale=float(np.float32(sc)), what=str(tuple(x.shape)))
        alone, = sbp.newton_schulz([x], out_scales=sc)
        assert torch.equal(alone.view(torch.int16), o.view(torch.int16))


def test_newton_schulz_more_groups_than_one_launch_takes():
    bits = [_u((20 + i, 60 - i), 60 + i) for i in range(37)]
    outs = sbp.newton_schulz([_bf(b) for b in bits])
    for i, (o, b) in enumerate(zip(outs, bits)):
        _check_ns(o, b, what=f"group {i}")


@pytest.mark.parametrize("shapes", [
    [(30, 400, 500)], [(30, 500, 400)],  # tiles of side 128
    [(48, 700, 900)], [(48, 900, 700)],  # whole rounds of side 256, the rest by quarters
    [(48, 760, 1000)], [(48, 1000, 760)],  # the same, padded sides that are multiples of 128
    [(20, 130, 1100), (36, 1000, 520), (3, 777, 2000)],  # both ways up, ragged
])
def test_newton_schulz_large_batches_equal_single_matrices(shapes):
    """What a matrix comes out as does not depend on what else the call holds,
    bit for bit, though larger calls take larger tiles; singles are held to the
    64-bit iteration elsewhere."""
    import torch
    xs = [_bf(_u(s, 70 + i, "strong")) for i, s in enumerate(shapes)]
    outs = sbp.newton_schulz(xs)
    for x, o in zip(xs, outs):
        for b in range(0, x.shape[0], 5):
            alone, = sbp.newton_schulz([x[b]])
            assert torch.equal(alone.view(torch.int16), o[b].view(torch.int16)), (x.shape, b)
    _check_ns(outs[0][:1], _bits(xs[0][:1]), what=str(shapes))


def _bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def test_newton_schulz_many_small_matrices():
    """More matrices than one part of the workspace holds (65536 of 64 x 64
    padded): first, last and the ones around the seam."""
    import torch
    B = 65536 + 700
    one = _u((64, 6, 9), 34)
    x = _bf(one).repeat(B // 64 + 1, 1, 1)[:B].contiguous()
    out, = sbp.newton_schulz([x])
    torch.cuda.synchronize()
    for lo in (0, 65472, 65536, B - 64):
        k = lo % 64
        want = np.concatenate([one[k:], one[:k]])
        _check_ns(out[lo:lo + 64], want, what=f"from {lo}")


def test_newton_schulz_strided_rows_and_untouched_gaps():
    """Rows further apart than they are long, in and out; what lies between
    the output's rows, before and behind it stays as it was."""
    import torch
    sizes = ((65, 130), (130, 65), (140, 150), (300, 7))
    for (pad, lead), (r, c) in itertools.product(((0, 1), (3, 5), (8, 8), (77, 0)), sizes):
        B = 2
        bits = _u((B, r, c), 35)
        x = torch.zeros(B * (r + 1) * (c + pad) + lead + 9, dtype=torch.bfloat16, device=H.dev())
        shape, stride = (B, r, c), ((r + 1) * (c + pad), c + pad, 1)
        view = x.as_strided(shape, stride, lead)
        view.copy_(_bf(bits))
        o = torch.full_like(x, 7.0)
        out = o.as_strided(shape, stride, lead)
        mask = torch.ones_like(o, dtype=torch.bool)
        mask.as_strided(shape, stride, lead).fill_(False)
        got, = sbp.newton_schulz([view], out=[out])
        assert got.data_ptr() == out.data_ptr()
        torch.cuda.synchronize()
        _check_ns(out, bits, what=f"pad {pad} lead {lead} {r}x{c}")
        assert bool((o[mask] == 7.0).all()), (pad, lead, r, c)


def _in_place_blocks(r, k):
    import torch
    bits = _u((r, 3 * k), 36)
    w = _bf(bits).clone()
    blocks = [w[:, k * i:k * (i + 1)] for i in range(3)]
    sbp.newton_schulz(blocks, out=blocks)
    torch.cuda.synchronize()
    for i in range(3):
        _check_ns(w[:, k * i:k * (i + 1)], np.ascontiguousarray(bits[:, k * i:k * (i + 1)]),
                  what=f"block {i} of {r}x{k}")


def test_newton_schulz_in_place_and_column_blocks():
    """In place, on three column blocks of one fused weight, and on heads that
    lie side by side in the rows."""
    import torch
    for r, k in ((48, 40), (300, 140)):
        _in_place_blocks(r, k)
    bits = _u((72, 4 * 16), 37)
    w = _bf(bits).clone()
    heads = w.view(72, 4, 16).permute(1, 0, 2)
    sbp.newton_schulz([heads], out=[heads])
    torch.cuda.synchronize()
    for h in range(4):
        _check_ns(w[:, 16 * h:16 * (h + 1)], np.ascontiguousarray(bits[:, 16 * h:16 * (h + 1)]),
                  what=f"head {h}")


def test_newton_schulz_broadcast_input():
    """One matrix read several times (a distance of zero)."""
    import torch
    bits = _u((30, 50), 38)
    x = _bf(bits).expand(3, 30, 50)
    out, = sbp.newton_schulz([x])
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    _check_ns(out[0], bits)


@pytest.mark.parametrize("size", [1e-37, 1e-20, 1e-3, 1e10, 1e36])
@pytest.mark.parametrize("shape", [(60, 100), (60, 700), (150, 140)])
def test_newton_schulz_any_size_of_norm(size, shape):
    """The direction does not depend on U's size while the norm is above eps."""
    bits = _u(shape, 39, size=size)
    out, = sbp.newton_schulz([_bf(bits)], eps=1e-38)
    _check_ns(out, bits, eps=1e-38, what=f"size {size}")


@pytest.mark.parametrize("size", [1e-30, 1e-14, 1e-9])
@pytest.mark.parametrize("shape", [(20, 30), (20, 400), (130, 140)])
def test_newton_schulz_norm_below_eps(size, shape):
    bits = _u(shape, 41, size=size / shape[1])
    out, = sbp.newton_schulz([_bf(bits)])
    U = OS.bf16_to_f32(bits).astype(np.float64)
    want = OS.newton_schulz(U, 5, sbp.NS_COEFS)
    # far below 1 the polynomial is its linear term: five roundings of X to
    # binary16 (of half a step 2^-11, the first three with their remainders)
    # and the result's; near 1 as everywhere
    tol = (2.0 ** -8 + 5 * 2.0 ** -11) * np.linalg.norm(want) if size < 1e-10 else \
        _tolerance(U, want, 5, sbp.NS_COEFS)
    assert np.linalg.norm(_f64(out) - want) <= tol


def test_newton_schulz_zero_nan_and_infinity():
    """Zeros give zeros; a NaN or an infinity fills its own matrix with NaN and
    leaves its neighbours' bits as they are without it."""
    import torch
    for shape in ((40, 70), (70, 40), (1, 3), (50, 600), (2200, 100), (140, 170), (170, 140)):
        bits = _u((5,) + shape, 42)
        bits[1] = 0
        clean, = sbp.newton_schulz([_bf(bits)])
        bits[2, -1, 0] = 0x7FC0
        bits[3, 0, -1] = 0xFF80
        out, = sbp.newton_schulz([_bf(bits)])
        torch.cuda.synchronize()
        assert bool((out[1] == 0).all())
        assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(out[3]).all())
        for i in (0, 4):
            assert torch.equal(out[i], clean[i])


def test_newton_schulz_of_zeros_without_a_floor():
    """0 / max(0, 0)."""
    import torch
    for shape in ((40, 70), (70, 40), (50, 600), (140, 170), (170, 140)):
        bits = _u((2,) + shape, 43)
        bits[1] = 0
        out, = sbp.newton_schulz([_bf(bits)], eps=0.0)
        torch.cuda.synchronize()
        assert bool(torch.isnan(out[1]).all()), shape
        _check_ns(out[:1], bits[:1], eps=0.0, what=str(shape))


def test_newton_schulz_two_streams_at_once():
    """Calls that overlap in time, each with a workspace of its own: the
    results of calls made one by one."""
    import torch
    xs = [_bf(_u((24, 300, 500), 51)), _bf(_u((24, 500, 300), 52))]
    want = [sbp.newton_schulz([x])[0] for x in xs]
    outs = [torch.empty_like(x) for x in xs]
    ws = [torch.empty(sbp.newton_schulz_workspace([x]), dtype=torch.uint8, device=H.dev())
          for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for x, o, w, s in zip(xs, outs, ws, streams):
            with torch.cuda.stream(s):
                sbp.newton_schulz([x], out=[o], workspace=w)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.view(torch.int16), w.view(torch.int16))


def test_newton_schulz_empty():
    import torch
    e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=H.dev())  # noqa: E731
    outs = sbp.newton_schulz([e(0, 5), e(5, 0), e(0, 4, 4), e(3, 0, 2)])
    assert [tuple(o.shape) for o in outs] == [(0, 5), (5, 0), (0, 4, 4), (3, 0, 2)]
    bits = _u((8, 8), 43)
    outs = sbp.newton_schulz([e(0, 5), _bf(bits)])
    _check_ns(outs[1], bits)


def test_newton_schulz_same_bits_every_time():
    import torch
    for shape in ((3, 200, 333), (3, 100, 2400), (3, 50, 90)):
        x = _bf(_u(shape, 44))
        first, = sbp.newton_schulz([x])
        for _ in range(3):
            again, = sbp.newton_schulz([x])
            assert torch.equal(first.view(torch.int16), again.view(torch.int16))


def test_newton_schulz_one_input_twice():
    import torch
    x = _bf(_u((150, 160), 48))
    a, b = sbp.newton_schulz([x, x])
    assert a.data_ptr() != b.data_ptr() and torch.equal(a, b)


def test_newton_schulz_dirty_workspace_and_streams():
    """A workspace full of NaN, and a call on a stream that is not the current
    one, with and without a workspace of its own."""
    import torch
    bits = _u((2, 150, 250), 45)
    x = _bf(bits)
    want, = sbp.newton_schulz([x])
    ws = torch.full((sbp.newton_schulz_workspace([x]) // 2,), float("nan"), dtype=torch.float16,
                    device=H.dev())
    got, = sbp.newton_schulz([x], workspace=ws)
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got, = sbp.newton_schulz([x], stream=stream)
        got2, = sbp.newton_schulz([x], stream=stream, workspace=ws)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(got2, want)


def test_newton_schulz_captured_and_replayed():
    """Two graphs with a workspace each, replayed in turn with eager calls
    between; inputs change from replay to replay."""
    import torch
    xs = [_bf(_u((2, 150, 250), 46)), _bf(_u((2300, 70), 47)), _bf(_u((3, 20, 30), 48))]
    outs = [torch.empty_like(x) for x in xs]
    ws = [torch.empty(sbp.newton_schulz_workspace([x]), dtype=torch.uint8, device=H.dev())
          for x in xs]
    graphs = []
    for x, o, w in zip(xs, outs, ws):
        sbp.newton_schulz([x], out=[o], workspace=w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sbp.newton_schulz([x], out=[o], workspace=w)
        graphs.append(g)
    for rep in range(4):
        for i, x in enumerate(xs):
            x.copy_(_bf(_u(tuple(x.shape), 50 + 7 * rep + i)))
        for g in graphs:
            g.replay()
        for x, o in zip(xs, outs):
            want, = sbp.newton_schulz([x])
            torch.cuda.synchronize()
            assert torch.equal(o, want), f"replay {rep}"


def test_newton_schulz_refuses_bad_tensors():
    import torch
    x = torch.zeros(8, 12, dtype=torch.bfloat16, device=H.dev())
    for bad in (x.float(), x.half(), x.t(), x[:, ::2], x[0]):
        with pytest.raises(ValueError):
            sbp.newton_schulz([bad])
    with pytest.raises(ValueError):
        sbp.newton_schulz([x], out=[torch.zeros_like(x).t()])
    with pytest.raises(ValueError):
        sbp.newton_schulz([x], out=[])
    with pytest.raises(ValueError):
        sbp.newton_schulz([x], out_scales=[1.0, 2.0])
    with pytest.raises(sbp.SbpError):
        sbp.newton_schulz([x], workspace=torch.empty(256, dtype=torch.uint8, device=H.dev()))
    with pytest.raises(sbp.SbpError):
        sbp.newton_schulz([x, x], out=[x, x])


# ---- the three calls as one step ---------------------------------------------------------

def test_step_of_a_rank_that_owns_whole_matrices():
    """Momentum over R peers, the matrices inside the bf16 direction
    orthogonalised in place, update: two steps against the oracle's, the second
    from the first one's state."""
    import torch
    shapes = [(48, 80), (130, 64), (1, 9)]
    plan = sbp.bucket_plan_per_tensor([r * c for r, c in shapes], 1)
    n = plan.shard_numel
    at = [plan.bucket(plan.tensor(t)[0])["shard_offset"] for t in range(len(shapes))]
    R, lr, wd, mu = 3, 0.02, 0.1, 0.95
    m, u = torch.zeros(n, dtype=torch.float32, device=H.dev()), H.empty_u16(n)
    th = synth.normal_f32(51, synth.master_stream(0), n, 0.02)
    master, param = H.from_np_f32(th), H.empty_u16(n)
    mats = [u[o:o + r * c].view(r, c) for o, (r, c) in zip(at, shapes)]
    scales = [max(1.0, r / c) ** 0.5 for r, c in shapes]
    mh = np.zeros(n, np.float32)
    for t in (1, 2):
        peers = H.dev_peers(51, t, 0, R, n, 1e-3)
        sbp.momentum_shard(peers, None, sbp.mean_scale(R), m, u, mu)
        torch.cuda.synchronize()
        mh, uh = OS.momentum_step(OS.reduce_peers(H.host_peers(51, t, 0, R, n, 1e-3)),
                                  np.float32(sbp.mean_scale(R)), mh, mu, True)
        H.assert_bits_equal(H.to_np_u16(u), uh, "direction")
        sbp.newton_schulz(mats, out=mats, out_scales=scales)
        torch.cuda.synchronize()
        for o, (r, c), sc, x in zip(at, shapes, scales, mats):
            _check_ns(x.view(torch.bfloat16), uh[o:o + r * c].reshape(r, c),
                      scale=float(np.float32(sc)), what=f"step {t} {r}x{c}")
        uh = H.to_np_u16(u)
        sbp.update_shard(u, master, param, lr, wd)
        torch.cuda.synchronize()
        th, ph = OS.update_step(uh, th, lr, wd)
        H.assert_bits_equal(H.to_np_f32(master), th, "master")
        H.assert_bits_equal(H.to_np_u16(param), ph, "param")


def test_step_of_row_shards_equals_whole_matrices():
    """Row shards over N ranks: the direction gathered, orthogonalised, cut
    again.  Every rank's parameters equal, bit for bit, those of one rank that
    owns the matrices whole."""
    import torch
    shapes, N, R = [(40, 24), (7, 96)], 2, 2
    numels, rows = [r * c for r, c in shapes], [c for _, c in shapes]
    plan = sbp.bucket_plan_per_tensor(numels, N, rows=rows)
    whole = sbp.bucket_plan_per_tensor(numels, 1, rows=rows)

    def state(p):
        z = lambda k, d: torch.zeros(k, dtype=d, device=H.dev())  # noqa: E731
        n = p.shard_numel
        return z(n, torch.float32), z(n, torch.int16), z(n, torch.float32), z(n, torch.int16)

    grads = [[H.from_np_u16(synth.normal_bf16(52, synth.tensor_stream(1, 0, r, t), k, 1e-3))
              for t, k in enumerate(numels)] for r in range(R)]
    theta = [H.from_np_u16(synth.normal_bf16(53, synth.tensor_stream(1, 0, 0, t), k, 0.02))
             for t, k in enumerate(numels)]

    def run(p):
        flats = []
        for g in grads + [theta]:
            flats.append(H.empty_u16(p.flat_numel))
            sbp.pack_grads(p, g, flats[-1])
        ranks = []
        for s in range(p.world_n):
            m, u, master, param = state(p)
            recv = [H.empty_u16(p.shard_numel) for _ in range(R + 1)]
            for f, x in zip(flats, recv):
                sbp.shard_of(p, s, f, x)
            master.copy_(recv[R].view(torch.bfloat16))
            sbp.momentum_shard(recv[:R], None, sbp.mean_scale(R), m, u, 0.9)
            ranks.append((u, master, param))
        mats = [H.empty_u16(k) for k in numels]
        sbp.unpack_shards(p, [u for u, _, _ in ranks], mats)
        views = [x.view(r, c) for x, (r, c) in zip(mats, shapes)]
        sbp.newton_schulz(views, out=views)
        flat = H.empty_u16(p.flat_numel)
        sbp.pack_grads(p, mats, flat)
        for s, (u, master, param) in enumerate(ranks):
            sbp.shard_of(p, s, flat, u)
            sbp.update_shard(u, master, param, 0.02, 0.1)
        params = [H.empty_u16(k) for k in numels]
        sbp.unpack_shards(p, [param for _, _, param in ranks], params)
        torch.cuda.synchronize()
        return [H.to_np_u16(x) for x in params]

    for a, b in zip(run(plan), run(whole)):
        H.assert_bits_equal(a, b, "parameters")


def test_newton_schulz_outputs_belong_to_the_calls_stream():
    """The block of an output that the call makes lies in memory of the stream
    that writes it, so the allocator can not hand out one that other work still
    uses."""
    import torch
    bits = _u((150, 250), 49)
    x = _bf(bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, 0):
        out, = sbp.newton_schulz([x], stream=stream)
        torch.cuda.synchronize()
        _check_ns(out, bits)
        where = [s["stream"] for s in torch.cuda.memory_snapshot()
                 if s["address"] <= out.data_ptr() < s["address"] + s["total_size"]]
        assert where == [stream if isinstance(stream, int) else stream.cuda_stream]


@pytest.mark.parametrize("shape", NS.SHAPES)
@pytest.mark.parametrize("steps", [3, 5])
def test_newton_schulz_keeps_its_remainders(shape, steps):
    """The result is nearer to the model of the device's formats than to one
    that loses a remainder or counts it with the wrong sign."""
    bits = NS.update(shape, 71, "flat")
    out, = sbp.newton_schulz([_bf(bits)], steps=steps)
    U = OS.bf16_to_f32(bits).astype(np.float64)
    assert NS.nearest(_f64(out), U, steps, sbp.NS_COEFS) is None


@pytest.mark.parametrize("shape", NS.SHAPES)
@pytest.mark.parametrize("kind", ["flat", "strong", "steep", "sixteen"])
def test_newton_schulz_is_as_far_off_as_its_formats(shape, kind):
    bits = NS.update(shape, 72, kind)
    U = OS.bf16_to_f32(bits).astype(np.float64)
    for steps in (3, 5):
        out, = sbp.newton_schulz([_bf(bits)], steps=steps)
        off = NS.off(_f64(out), U, steps, sbp.NS_COEFS)
        assert off < NS.ALLOWED, (steps, off)


SCALE_SHAPES = [(1, 1), (4, 4), (60, 250), (128, 192), (40, 700), (700, 120), (100, 2500),
                (150, 200), (200, 150)]


def _check_scaled(out, U, scale, eps=1e-7, steps=5):
    """bf16's subnormals are 2^-133 apart: half of that more for each entry."""
    want = OS.newton_schulz(U, steps, sbp.NS_COEFS, eps)
    tol = _tolerance(U, want, steps, sbp.NS_COEFS, eps) * abs(scale) + \
        2.0 ** -134 * np.sqrt(want.size)
    off = np.linalg.norm(_f64(out) - float(np.float32(scale)) * want)
    assert off <= tol, f"{U.shape} times {scale}: off by {off:.3e}, tolerance {tol:.3e}"


@pytest.mark.parametrize("shape", SCALE_SHAPES)
@pytest.mark.parametrize("steps", [1, 5])
def test_newton_schulz_any_out_scale(shape, steps):
    """From binary32's subnormals to its largest."""
    bits = _u(shape, 73)
    U = OS.bf16_to_f32(bits).astype(np.float64)
    for scale in (1e-30, -1e-36, 2.0 ** -126, 2.0 ** -130, 0.0, 1e30, 1.5e38):
        out, = sbp.newton_schulz([_bf(bits)], steps=steps, out_scales=scale)
        _check_scaled(out, U, scale, steps=steps)


def test_newton_schulz_any_out_scale_large_tiles():
    """The same on tiles of side 256 and quarters: the bits of single matrices."""
    import torch
    x = _bf(_u((48, 500, 1000), 74))
    for scale in (1e-36, 2.0 ** -130):
        out, = sbp.newton_schulz([x], out_scales=scale)
        for i in (0, 30, 47):
            alone, = sbp.newton_schulz([x[i]], out_scales=scale)
            assert torch.equal(alone.view(torch.int16), out[i].view(torch.int16))


@pytest.mark.parametrize("shape", [(1, 1), (20, 30), (20, 400), (100, 2500), (130, 140),
                                   (140, 130)])
def test_newton_schulz_norm_far_below_eps(shape):
    """The result is next to nothing and out_scale brings it back.  Far below 1
    the polynomial is its linear term: five roundings of X to binary16 (half a
    step, 2^-11 of it) and the result's."""
    for eps, size, scale in ((1e38, 1e-34, 1e38), (3e38, 1e-37, 3e38), (1.0, 1e-37, 1e30),
                             (1e-7, 1e-30, 1e-4)):
        bits = _u(shape, 75, size=size)
        out, = sbp.newton_schulz([_bf(bits)], eps=eps, out_scales=scale)
        U = OS.bf16_to_f32(bits).astype(np.float64)
        want = OS.newton_schulz(U, 5, sbp.NS_COEFS, eps, scale)
        tol = (2.0 ** -8 + 5 * 2.0 ** -11) * np.linalg.norm(want) + 2.0 ** -134 * np.sqrt(want.size)
        assert np.linalg.norm(_f64(out) - want) <= tol, (eps, size, scale)


@pytest.mark.parametrize("shape", [(1, 1), (1, 100), (39, 777), (64, 64), (100, 2000), (2000, 100),
                                   (100, 200000), (130, 300), (1000, 700), (2048, 2048)])
@pytest.mark.parametrize("steps", [1, 2, 3, 5, 8])
def test_newton_schulz_of_equal_entries(shape, steps):
    """All entries alike, up to their signs: every rounding is the same for all
    of them, so nothing averages out, and the result is the polynomial of one
    number.  With s that number's square and p = a + b s + c s^2, X' = p X: X's
    relative error e passes on times |p + 2 (b s + 2 c s^2)| / |p|, A's rounding
    u = 2^-11 comes in times |b s + 2 c s^2| / |p|, B's times |b s + c s^2| /
    |p|, X's own once, and the output's 2^-8 at the end."""
    bits = OS.f32_to_bf16(np.full(shape, 1.0078125e-3, np.float32))
    bits[::3] ^= 0x8000
    bits[:, ::2] ^= 0x8000
    out, = sbp.newton_schulz([_bf(bits)], steps=steps)
    U = OS.bf16_to_f32(bits).astype(np.float64)
    a, b, c = sbp.NS_COEFS
    x, off = 1.0, 0.0
    for _ in range(steps):
        s, u = x * x, 2.0 ** -11
        low, slope = b * s + c * s * s, b * s + 2 * c * s * s
        p = a + low
        off = (abs(p + 2 * slope) * off + (abs(slope) + abs(low)) * u) / abs(p) + u
        x *= p
    # in exact arithmetic: U over its norm, times x
    want = x * np.sign(U) / np.sqrt(U.size)
    assert np.max(np.abs(_f64(out) / want - 1)) <= off + 2.0 ** -8
