"""The momentum-orthogonalising step on the host (CPU only): the oracle's
momentum, update and Newton-Schulz iteration against closed forms, and every
refusal of the three calls (the fake addresses are never dereferenced)."""

import ctypes

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from oracle import step as OS

V = ctypes.c_void_p
F32 = np.float32


# ---- the oracle ------------------------------------------------------------------

def test_momentum_first_step_closed_form():
    """From zero momentum, m' = (1-mu) g and the look-ahead is (1-mu)(1+mu) g;
    with dyadic values every operation is exact."""
    G = np.array([1.0, -2.0, 0.5, 0.0, 4.0], F32)
    m, u = OS.momentum_step(G, 0.5, np.zeros(5, F32), 0.75, True)
    assert np.array_equal(m, G * F32(0.125))
    assert np.array_equal(OS.bf16_to_f32(u), G * F32(0.125) * F32(1.75))
    m, u = OS.momentum_step(G, 0.5, np.zeros(5, F32), 0.75, False)
    assert np.array_equal(OS.bf16_to_f32(u), m)


def test_momentum_of_a_constant_gradient_converges_to_it():
    g = np.full(3, 0.25, F32)
    m = np.zeros(3, F32)
    for t in range(1, 60):
        m, _ = OS.momentum_step(g, 1.0, m, 0.5, True)
        # exact in binary: g * (1 - 2^-t) until the bits run out
        assert np.allclose(m, 0.25 * (1 - 0.5 ** t), rtol=2.0 ** -23, atol=0)
    assert np.array_equal(m, g)


def test_momentum_zero_mu_is_the_scaled_gradient():
    g = np.array([3.0, -1.5], F32)
    m, u = OS.momentum_step(g, 2.0, np.array([7.0, np.float32(1e30)], F32), 0.0, True)
    assert np.array_equal(m, g * 2) and np.array_equal(OS.bf16_to_f32(u), g * 2)


def test_update_closed_form():
    u = OS.f32_to_bf16(np.array([1.0, -0.5, 0.0], F32))
    th, p = OS.update_step(u, np.array([2.0, 2.0, -1.0], F32), 0.5, 0.5)
    assert np.array_equal(th, np.array([1.0, 1.75, -0.75], F32))
    assert np.array_equal(OS.bf16_to_f32(p), th)
    th, _ = OS.update_step(u, np.array([2.0, 2.0, -1.0], F32), 0.0, 0.5)
    assert np.array_equal(th, np.array([2.0, 2.0, -1.0], F32))


# ---- refusals ----------------------------------------------------------------------

def _momentum(**kw):
    a = dict(peers=(V * 2)(0x100000, 0x200000), R=2, acc=None, scale=0.5, m=V(0x300000),
             u=V(0x400000), n=1024, mu=0.9, nesterov=1)
    a.update(kw)
    return sbp.lib().sbp_momentum_shard(a["peers"], a["R"], a["acc"], a["scale"], a["m"], a["u"],
                                        a["n"], a["mu"], a["nesterov"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=17), sbp.SBP_EINVAL), (dict(R=-1), sbp.SBP_EINVAL),
    (dict(R=0), sbp.SBP_EINVAL),  # R == 0 needs acc
    (dict(peers=None), sbp.SBP_EINVAL), (dict(peers=(V * 2)(0x100000, None)), sbp.SBP_EINVAL),
    (dict(n=-1), sbp.SBP_EINVAL),
    (dict(mu=1.0), sbp.SBP_EINVAL), (dict(mu=-0.1), sbp.SBP_EINVAL),
    (dict(mu=float("nan")), sbp.SBP_EINVAL),
    (dict(m=None), sbp.SBP_EINVAL), (dict(u=None), sbp.SBP_EINVAL),
    (dict(m=V(0x300004)), sbp.SBP_EALIGN), (dict(u=V(0x400002)), sbp.SBP_EALIGN),
    (dict(acc=V(0x500008)), sbp.SBP_EALIGN),
    (dict(peers=(V * 2)(0x100002, 0x200000)), sbp.SBP_EALIGN),
    (dict(n=sbp.MAX_SHARD_NUMEL + 1), sbp.SBP_ERANGE),
    (dict(u=V(0x300000 + 4080)), sbp.SBP_EINVAL),  # u_out inside m
    (dict(acc=V(0x300000)), sbp.SBP_EINVAL),  # acc is m
    (dict(peers=(V * 2)(0x100000, 0x400000)), sbp.SBP_EINVAL),  # a peer is u_out
])
def test_momentum_refusals(kw, status):
    assert _momentum(**kw) == status
    assert b"sbp_momentum_shard" in sbp.lib().sbp_last_error()


def test_momentum_empty_reads_nothing():
    assert _momentum(n=0, peers=None, m=None, u=None) == sbp.SBP_OK


def _update(**kw):
    a = dict(u=V(0x100000), master=V(0x200000), p=V(0x300000), n=1024, lr=0.1, wd=0.1)
    a.update(kw)
    return sbp.lib().sbp_update_shard(a["u"], a["master"], a["p"], a["n"], a["lr"], a["wd"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), sbp.SBP_EINVAL), (dict(lr=-1.0), sbp.SBP_EINVAL),
    (dict(lr=float("inf")), sbp.SBP_EINVAL), (dict(wd=float("nan")), sbp.SBP_EINVAL),
    (dict(u=None), sbp.SBP_EINVAL), (dict(master=None), sbp.SBP_EINVAL),
    (dict(p=None), sbp.SBP_EINVAL),
    (dict(u=V(0x100008)), sbp.SBP_EALIGN), (dict(master=V(0x200004)), sbp.SBP_EALIGN),
    (dict(p=V(0x300002)), sbp.SBP_EALIGN),
    (dict(n=sbp.MAX_SHARD_NUMEL + 1), sbp.SBP_ERANGE),
    (dict(p=V(0x100000)), sbp.SBP_EINVAL), (dict(p=V(0x200000 + 2048)), sbp.SBP_EINVAL),
    (dict(u=V(0x200000 + 4080)), sbp.SBP_EINVAL),
])
def test_update_refusals(kw, status):
    assert _update(**kw) == status
    assert b"sbp_update_shard" in sbp.lib().sbp_last_error()


def test_update_empty_reads_nothing():
    assert _update(n=0, u=None, master=None, p=None) == sbp.SBP_OK
