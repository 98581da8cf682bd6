"""GPU parity of the momentum-orthogonalising step's calls with the oracle:
momentum and update bit for bit, Newton-Schulz against the iteration in 64
bits, and the three as one step."""

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
import synth
from oracle import step as OS
from tests import helpers as H

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
