"""Every address that a tile of newton_schulz.hip's products forms, worked out
again on the CPU for ragged matrices: inside its array, or cut off by the
buffer descriptor's length.

The kernel's expressions are written out a second time here, lane by lane, as
numpy arrays over the 256 threads of a block; a change of one has to be made in
the other.  A buffer access is held to `length - scalar offset`, unsigned: a
scalar offset past the end, or a negative length, would lift the bound.  So no
scalar offsets are used, and every tile has to start inside its matrix."""

import math

import numpy as np
import pytest

THREAD = np.arange(256)
WAVE, LANE = THREAD >> 6, THREAD & 63
TILES = [(64, 64), (128, 64), (256, 32)]  # side, and elements of k a slice
SHAPES = [(1, 1), (1, 70), (70, 1), (64, 64), (65, 64), (129, 129), (100, 200), (200, 100),
          (130, 300), (320, 130), (509, 1021), (700, 333), (1024, 256), (64, 2000), (2500, 70)]


def _up(x):
    return (x + 63) // 64 * 64


def _turn_along(BK, row):
    if BK == 64:
        return row & 7
    return (((row >> 1) ^ (row >> 2)) & 2) | (((row >> 3) ^ (row >> 1)) & 1)


def _turn_across(T, row):
    if T >= 128:
        return (row & 3) | ((row >> 3) & 1) << 2
    return ((row >> 1) & 1) | ((row >> 3) & 1) << 1


def _inside(base, off, length, size):
    """Bytes from `off` on that the descriptor lets through lie in the array."""
    assert 0 < length < 2 ** 32 and off.min() >= 0 and off.max() < 2 ** 32
    ok = off < length
    assert not ok.any() or base + off[ok].max() + 16 <= size
    return ok


def _along(T, BK, rows, ld, r0, size):
    """An operand whose rows are the matrix's: loads of all its slices."""
    have = min(rows - r0, T)
    assert have >= 1
    lanes = BK // 8
    row = WAVE * (64 // lanes) + LANE // lanes
    first = row * ld * 2 + ((LANE % lanes) ^ _turn_along(BK, row)) * 16
    for s in range(ld // BK):
        for r in range(T * BK * 2 // 4096):
            at = row + r * 4 * (64 // lanes)
            ok = _inside(r0 * ld * 2 + s * BK * 2, first + r * 4 * (64 // lanes) * ld * 2,
                         have * ld * 2 - s * BK * 2, size)
            assert ok[at < have].all()  # the rows that matter come
            assert ((r * 4 + WAVE) * 1024 + LANE * 16).max() + 16 <= T * BK * 2


def _across(T, BK, k, ld, r0, size):
    """An operand whose rows are the matrix's columns."""
    lanes = T // 8
    rows = 64 // lanes
    for s in range(k // BK):
        for r in range(T * BK * 2 // 4096):
            row = (r * 4 + WAVE) * rows + LANE // lanes
            off = row * ld * 2 + (((LANE % lanes) * 16) ^ (_turn_across(T, row) * 32))
            _inside((s * BK * ld + r0) * 2, off, (BK * ld - r0) * 2, size)


def _epilogue(T, rows, cols, r0, c0, m, by_row, by_col):
    have = min(rows - r0, T)
    assert 1 <= have <= T and c0 < cols
    length, size = have * cols * 2, rows * cols * 2
    prow, pcol = THREAD // (T // 8), (THREAD % (T // 8)) * 8
    gc = c0 + pcol
    at_once = 256 // (T // 8)
    for sl in range(T // 64):
        for p in range(64 // at_once):
            row = sl * 64 + p * at_once
            off = np.where(gc < cols, (prow * cols + gc) * 2, length) + row * cols * 2
            ok = _inside(r0 * cols * 2, off, length, size)
            assert (ok == ((prow + row < have) & (gc < cols))).all()
            r = p * at_once + prow
            turned = pcol ^ ((r >> 3 & 1) << 4) ^ ((r >> 4 & 1) << 3) ^ \
                ((((r >> 5) ^ (r >> 2)) & 1) << 5)
            assert ((((r & 31) * T + turned) + 8) * 4).max() <= 32 * T * 4
            d = (prow + row) * 4
            ok = d < (have * 4 if by_row else 0)
            assert not ok.any() or r0 * 4 + d[ok].max() + 4 <= m * 4
    at = np.where(gc < cols, gc * 4, m * 4)
    for off in (at, at + 16):
        ok = off < (m * 4 if by_col else 0)
        assert not ok.any() or off[ok].max() + 16 <= m * 4


def _lower_tiles(T, m):
    side = (m + T - 1) // T
    for t in range(side * (side + 1) // 2):
        ti = int((math.sqrt(8.0 * t + 1) - 1) * 0.5)
        while ti * (ti + 1) // 2 > t:
            ti -= 1
        while (ti + 1) * (ti + 2) // 2 <= t:
            ti += 1
        yield ti, t - ti * (ti + 1) // 2


def _apply_tiles(T, rows, cols):
    tr, tc = -(-rows // T), -(-cols // T)
    for t in range(tr * tc):
        strip = t // (8 * tc)
        high, s = min(tr - strip * 8, 8), t - strip * 8 * tc
        yield strip * 8 + s % high, s // high


def _quarters(tiles, T, rows, cols, lower):
    """The quarters of tiles of twice the side that a block does not leave alone."""
    for ti, tj in tiles:
        for q in range(4):
            i, j = 2 * ti + (q >> 1), 2 * tj + (q & 1)
            if not (i * T >= rows or j * T >= cols or (lower and j > i)):
                yield i, j


@pytest.mark.parametrize("T,BK", TILES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_products_stay_inside(T, BK, rows, cols):
    rp, cp = _up(rows), _up(cols)
    m, n = min(rp, cp), max(rp, cp)
    tall = rows > cols
    want = {(i, j) for i in range(-(-m // T)) for j in range(i + 1)}
    whole = list(_lower_tiles(T, m))
    assert len(whole) == len(want) and set(whole) == want
    if T == 128:
        assert set(_quarters(_lower_tiles(256, m), T, m, m, True)) == want
    for ti, tj in whole:
        for t in (ti, tj):
            assert t * T < m
            _along(T, BK, m, m, t * T, m * m * 2)
            if tall:
                _across(T, BK, n, m, t * T, m * n * 2)
            else:
                _along(T, BK, m, n, t * T, m * n * 2)
        _epilogue(T, m, m, ti * T, tj * T, m, True, True)
    want = {(i, j) for i in range(-(-rp // T)) for j in range(-(-cp // T))}
    whole = list(_apply_tiles(T, rp, cp))
    assert len(whole) == len(want) and set(whole) == want
    if T == 128:
        assert set(_quarters(_apply_tiles(256, rp, cp), T, rp, cp, False)) == want
    for ti, tj in whole:
        assert ti * T < rp and tj * T < cp
        if tall:
            _along(T, BK, rp, m, ti * T, rp * m * 2)
            _along(T, BK, cp, m, tj * T, m * m * 2)
        else:
            _along(T, BK, rp, m, ti * T, m * m * 2)
            _across(T, BK, m, cp, tj * T, rp * cp * 2)
        _epilogue(T, rp, cp, ti * T, tj * T, m, not tall, tall)


@pytest.mark.parametrize("T,BK", TILES)
def test_fragments_come_from_where_their_slice_lies(T, BK):
    """LDS: what a lane reads lies in the slice's buffer, and across is the row
    and column that the load put there."""
    lanes, rounds = T // 8, T * BK * 2 // 4096
    lay = np.zeros((BK * T * 2 // 16, 2), int)  # row and 8-element piece of each 16 bytes
    for r in range(rounds):
        row = (r * 4 + WAVE) * (64 // lanes) + LANE // lanes
        piece = (((LANE % lanes) * 16) ^ (_turn_across(T, row) * 32)) // 16
        lay[((r * 4 + WAVE) * 1024 + LANE * 16) // 16] = np.stack([row, piece], 1)
    along = np.zeros((BK * T * 2 // 16, 2), int)
    for r in range(rounds):
        row = WAVE * (64 // (BK // 8)) + LANE // (BK // 8)
        piece = (LANE % (BK // 8)) ^ _turn_along(BK, row)
        at = row + r * 4 * (64 // (BK // 8))
        along[((r * 4 + WAVE) * 1024 + LANE * 16) // 16] = np.stack([at, piece], 1)
    low = LANE & 15
    k = (LANE >> 4) * 8 + ((LANE >> 2) & 3)
    for wrow in (0, T // 2):
        for p in range(BK // 32):
            for i in range(T // 32):
                piece = p * 4 + (LANE >> 4)
                a = (wrow + i * 16 + low) * (BK * 2) + (piece ^ _turn_along(BK, low)) * 16
                assert a.min() >= 0 and a.max() + 16 <= T * BK * 2
                assert (along[a // 16] == np.stack([wrow + i * 16 + low, piece], 1)).all()
                for half in (0, 4):
                    a = (k + p * 32 + half) * (T * 2) + (LANE & 3) * 8 + \
                        ((wrow // 16 + i) ^ _turn_across(T, k)) * 32
                    assert a.min() >= 0 and a.max() + 8 <= T * BK * 2
                    got = lay[a // 16]
                    assert (got[:, 0] == k + p * 32 + half).all()
                    assert (got[:, 1] * 8 + a % 16 // 2 == wrow + i * 16 + (LANE & 3) * 4).all()
