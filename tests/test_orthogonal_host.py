"""The momentum-orthogonalising step on the host (CPU only): the oracle's
momentum, update and Newton-Schulz iteration against closed forms, and every
refusal of the three calls (the fake addresses are never dereferenced)."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from oracle import step as OS
from tests import ns_models as NS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


# ---- Newton-Schulz -----------------------------------------------------------------

COEFS = sbp.NS_COEFS


def _poly(x, steps, coefs=COEFS):
    for _ in range(steps):
        x = coefs[0] * x + coefs[1] * x ** 3 + coefs[2] * x ** 5
    return x


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (6, 1), (5, 5), (4, 7), (9, 3)])
def test_oracle_newton_schulz_acts_on_singular_values(shape):
    """The result has U's singular vectors and the polynomial of its singular
    values: the definition by decomposition."""
    rng = np.random.default_rng(5)
    U = rng.standard_normal(shape)
    P, s, Q = np.linalg.svd(U, full_matrices=False)
    f32 = [float(F32(c)) for c in COEFS]
    want = (P * _poly(s / np.sqrt(np.sum(s * s)), 5, f32)) @ Q
    got = OS.newton_schulz(U, 5, COEFS)
    assert np.allclose(got, want, rtol=0, atol=1e-11)
    # every singular value that was not tiny ends inside the quintic's band
    assert np.all(np.linalg.svd(got, compute_uv=False)[s > 0.05 * s[0]] < 1.25)


def test_oracle_newton_schulz_edges():
    assert np.array_equal(OS.newton_schulz(np.zeros((3, 4)), 5, COEFS), np.zeros((3, 4)))
    U = np.ones((2, 3))
    U[0, 1] = np.nan
    assert np.isnan(OS.newton_schulz(U, 1, COEFS)).all()
    U[0, 1] = np.inf
    assert np.isnan(OS.newton_schulz(U, 1, COEFS)).all()
    # below eps the matrix is divided by eps: a power of the polynomial's slope
    U = np.full((1, 1), 1e-12)
    slope = float(F32(COEFS[0])) ** 3
    assert np.allclose(OS.newton_schulz(U, 3, COEFS, eps=1e-7), 1e-12 / float(F32(1e-7)) * slope,
                       rtol=1e-6)
    a = OS.newton_schulz(np.eye(3), 2, [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5)], out_scale=0.5)
    x = 1 / np.sqrt(3.0)
    x = 1.5 * x - 0.5 * x ** 3
    x = 2 * x - 1.5 * x ** 3 + 0.5 * x ** 5
    assert np.allclose(a, 0.5 * x * np.eye(3), atol=1e-14)


def test_oracle_rounded_formats_cost_little():
    """Flat and steep spectra: the kept formats move the result by less than
    half a bf16 step, 2^-8 of it (each entry is within 2^-11, fp16's half
    step, and the remainder keeps the early steps' noise from growing)."""
    rng = np.random.default_rng(6)
    for m, n in ((40, 60), (96, 96)):
        flat = rng.standard_normal((m, n))
        steep = rng.standard_normal((m, 4)) @ rng.standard_normal((4, n)) + 0.03 * flat
        for U in (flat, steep):
            U = OS.bf16_to_f32(OS.f32_to_bf16(U.astype(F32))).astype(np.float64)
            e = OS.newton_schulz(U, 5, COEFS)
            r = OS.newton_schulz_rounded(U, 5, COEFS)
            assert np.linalg.norm(r - e) < 2.0 ** -8 * np.linalg.norm(e)


def _mats(**kw):
    a = dict(in_=0x1000000, out=0x2000000, rows=64, cols=64, count=1, in_ld=64, out_ld=64,
             in_stride=0, out_stride=0, out_scale=1.0)
    a.update(kw)
    return sbp.Matrices(*[a[k] for k, _ in sbp.Matrices._fields_])


def _ns(groups, hp=None, ws=0x8000000, ws_bytes=1 << 40, n=None):
    arr = (sbp.Matrices * max(len(groups), 1))(*groups)
    hp = hp if hp is not None else sbp.NsHParams.of(5, COEFS, 1e-7, "test")
    return sbp.lib().sbp_newton_schulz(arr, len(groups) if n is None else n,
                                       ctypes.byref(hp) if hp else None, V(ws), ws_bytes, None)


def _hp(steps=5, eps=1e-7, **coefs):
    h = sbp.NsHParams.of(5, COEFS, eps, "test")
    h.steps = steps
    for k, v in coefs.items():
        h.coefs[int(k[1:])] = v
    return h


_BIG = _mats(rows=192, cols=192, in_ld=192, out_ld=192)


@pytest.mark.parametrize("groups,kw,status", [
    ([_mats()], dict(n=-1), sbp.SBP_EINVAL),
    ([_mats()], dict(hp=False), sbp.SBP_EINVAL),
    ([_mats()], dict(hp=_hp(steps=0)), sbp.SBP_EINVAL),
    ([_mats()], dict(hp=_hp(steps=17)), sbp.SBP_EINVAL),
    ([_mats()], dict(hp=_hp(eps=-1.0)), sbp.SBP_EINVAL),
    ([_mats()], dict(hp=_hp(eps=float("nan"))), sbp.SBP_EINVAL),
    ([_mats()], dict(hp=_hp(c4=65.0)), sbp.SBP_EINVAL),
    ([_mats()], dict(hp=_hp(c14=float("nan"))), sbp.SBP_EINVAL),
    ([_mats(rows=-1)], {}, sbp.SBP_EINVAL),
    ([_mats(count=-1)], {}, sbp.SBP_EINVAL),
    ([_mats(rows=(1 << 20) + 1)], {}, sbp.SBP_ERANGE),
    ([_mats(rows=1 << 17, cols=1 << 17, in_ld=1 << 17, out_ld=1 << 17)], {}, sbp.SBP_ERANGE),
    ([_mats(in_=None)], {}, sbp.SBP_EINVAL),
    ([_mats(out=None)], {}, sbp.SBP_EINVAL),
    ([_mats(in_=0x1000001)], {}, sbp.SBP_EALIGN),
    ([_mats(out=0x2000001)], {}, sbp.SBP_EALIGN),
    ([_mats(in_ld=63)], {}, sbp.SBP_EINVAL),
    ([_mats(out_ld=63)], {}, sbp.SBP_EINVAL),
    ([_mats(in_ld=(1 << 40) + 1)], {}, sbp.SBP_ERANGE),
    ([_mats(out_scale=float("inf"))], {}, sbp.SBP_EINVAL),
    ([_mats(count=2, in_stride=-4096, out_stride=4096)], {}, sbp.SBP_EINVAL),
    ([_mats(count=2, in_stride=1 << 62, out_stride=4096)], {}, sbp.SBP_ERANGE),
    ([_mats(count=2, in_stride=4096, out_stride=4095)], {}, sbp.SBP_EINVAL),
    ([_mats(count=2, in_stride=4096, out_stride=0)], {}, sbp.SBP_EINVAL),
    # side by side in rows of 150: three of 64 do not fit
    ([_mats(count=3, in_stride=4096, out_stride=64, out_ld=150)], {}, sbp.SBP_EINVAL),
    ([_mats(out=0x1000000 + 64)], {}, sbp.SBP_EINVAL),  # shifted over its input
    ([_mats(out=0x1000000, out_ld=65)], {}, sbp.SBP_EINVAL),  # same start, other distances
    ([_mats(), _mats(in_=0x3000000)], {}, sbp.SBP_EINVAL),  # two outputs in one place
    ([_mats(), _mats(in_=0x2000000, out=0x3000000)], {}, sbp.SBP_EINVAL),  # reads the first's
    ([_mats(in_ld=200, out_ld=200, in_=0x1000000, out=0x1000000),
      _mats(in_ld=200, out_ld=200, in_=0x1000000 + 2 * 32, out=0x1000000 + 2 * 32)], {},
     sbp.SBP_EINVAL),  # column blocks that share columns
    ([_mats(in_ld=200, out_ld=200, in_=0x1000000, out=0x1000000),
      _mats(in_ld=201, out_ld=201, in_=0x1000000 + 2 * 64, out=0x1000000 + 2 * 64)], {},
     sbp.SBP_EINVAL),  # column blocks of two row distances
    ([_mats()], dict(ws=None), sbp.SBP_EINVAL),
    ([_mats()], dict(ws=0x8000080), sbp.SBP_EALIGN),
    ([_mats()], dict(ws_bytes=1), sbp.SBP_EINVAL),
    ([_BIG], dict(ws_bytes=100000), sbp.SBP_EINVAL),
    ([_BIG], dict(ws=0x1000000), sbp.SBP_EINVAL),
    ([_BIG], dict(ws=0x2000000 - 4096), sbp.SBP_EINVAL),
])
def test_newton_schulz_refusals(groups, kw, status):
    assert _ns(groups, **kw) == status
    assert b"sbp_newton_schulz" in sbp.lib().sbp_last_error()


def test_newton_schulz_nothing_to_do():
    for g in ([], [_mats(rows=0)], [_mats(cols=0, in_=None)], [_mats(count=0, out=None)]):
        assert _ns(g, ws=None, ws_bytes=0) == sbp.SBP_OK
    assert sbp.lib().sbp_newton_schulz(None, 0, ctypes.byref(_hp()), None, 0, None) == sbp.SBP_OK


def test_newton_schulz_workspace_size():
    q = sbp.lib().sbp_newton_schulz_workspace
    one = q((sbp.Matrices * 1)(_mats()), 1)
    assert one > 0
    big = q((sbp.Matrices * 1)(_mats(rows=192, cols=192)), 1)
    assert q((sbp.Matrices * 1)(_mats(rows=129, cols=180)), 1) == big  # padded alike
    assert big >= 2 * 5 * 192 * 192  # the iterate twice, its remainder, A and B
    assert q((sbp.Matrices * 1)(_mats(rows=192, cols=192, count=3)), 1) > 2 * big
    assert q((sbp.Matrices * 1)(_mats(rows=0)), 1) == 0
    assert q((sbp.Matrices * 1)(_mats(rows=-1)), 1) == -1
    assert q((sbp.Matrices * 1)(_mats(cols=(1 << 20) + 1)), 1) == -1
    assert q(None, 1) == -1
    # a long list runs in parts: the workspace stays bounded
    many = (sbp.Matrices * 40)(*[_mats(rows=4096, cols=14336)] * 40)
    assert q(many, 40) < 8 * q(many, 1)


@pytest.mark.parametrize("call", ["sbp_newton_schulz_workspace", "sbp_newton_schulz"])
def test_newton_schulz_out_of_host_memory(call):
    """A list whose parts do not fit host memory is refused, in a process of
    small means: no exception leaves a C call, and nothing is launched."""
    code = f"""
import ctypes, resource, sys
sys.path.insert(0, {ROOT!r})
import sharded_bucket_plan_amd as sbp
L = sbp.lib()
n, big = 1 << 20, 1 << 14  # a part each: 2^20 entries of a list
g = (sbp.Matrices * 1)(sbp.Matrices(1 << 20, 1 << 62, big, big, n, big, big, big * big,
                                    big * big, 1.0))
hp = sbp.NsHParams.of(5, sbp.NS_COEFS, 1e-7, "t")
L.sbp_newton_schulz_workspace((sbp.Matrices * 1)(sbp.Matrices(None, None, 64, 64, 1)), 1)
now = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (now + (16 << 20),) * 2)
if {call!r} == "sbp_newton_schulz_workspace":
    r = L.sbp_newton_schulz_workspace(g, 1)
else:
    r = L.sbp_newton_schulz(g, 1, ctypes.byref(hp), 1 << 50, 1 << 60, None)
print(r, L.sbp_last_error().decode())
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    want = -1 if call.endswith("workspace") else sbp.SBP_ENOMEM
    assert r.stdout.strip() == f"{want} {call}: out of host memory"


def test_newton_schulz_python_arguments():
    with pytest.raises(ValueError):
        sbp.NsHParams.of(0, COEFS, 1e-7, "t")
    with pytest.raises(ValueError):
        sbp.NsHParams.of(2, [COEFS] * 3, 1e-7, "t")
    with pytest.raises(ValueError):
        sbp.NsHParams.of(2, (1.0, 2.0), 1e-7, "t")
    import torch
    x = torch.zeros(4, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sbp.newton_schulz([x])  # not a device tensor
    assert sbp.newton_schulz([]) == []


class _Fake:
    """What newton_schulz reads of a device tensor, and the stream it was made on."""
    is_cuda = True

    def __init__(self, shape, dtype, device, made_on, at):
        self.shape, self.dtype, self.device = tuple(shape), dtype, device
        self.made_on, self.at, self.used_on = made_on, at, []

    def dim(self):
        return len(self.shape)

    def stride(self, d):
        return int(np.prod(self.shape[d % len(self.shape) + 1:]))

    def data_ptr(self):
        return self.at

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def record_stream(self, s):
        self.used_on.append(s)


def _fake_streams(monkeypatch):
    """torch.empty and torch's streams without a GPU; the list of what is
    allocated, each with the stream that was current."""
    import torch
    current, made = ["current"], []

    class On:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            current.append(self.s)

        def __exit__(self, *a):
            current.pop()

    def empty(*shape, dtype, device):
        shape = shape[0] if isinstance(shape[0], tuple) else shape
        made.append(_Fake(shape, dtype, device, current[-1], 0x10000000 * (len(made) + 2)))
        return made[-1]

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: current[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: f"stream {s}")
    monkeypatch.setattr(sbp, "_stream", lambda s, t: V(s))
    return made


class _NoLaunch:
    """The library, but for one call that is noted down in place of being made."""

    def __init__(self, name):
        self.library, self.name, self.streams = sbp.lib(), name, []

    def __getattr__(self, name):
        if name != self.name:
            return getattr(self.library, name)
        return lambda *a: self.streams.append(a[-1].value) or sbp.SBP_OK


ON = {None: "current", 0: "default", 77: "stream 77"}


@pytest.mark.parametrize("given", list(ON))
def test_newton_schulz_allocates_on_the_calls_stream(monkeypatch, given):
    """Outputs and workspace that the call makes belong to the stream that the
    kernels run on: a block of another stream may still be in use there."""
    import torch
    made = _fake_streams(monkeypatch)
    library = _NoLaunch("sbp_newton_schulz")
    monkeypatch.setattr(sbp, "lib", lambda: library)
    x = _Fake((64, 300), torch.bfloat16, torch.device("cuda", 0), "current", 0x1000000)
    out, = sbp.newton_schulz([x], stream=given)
    assert [m.made_on for m in made] == [ON[given]] * 2 and out is made[0]
    assert library.streams == [given or None]
    # the outputs may be used and freed on the caller's stream
    assert given is None or out.used_on == ["current"]


@pytest.mark.parametrize("given", list(ON))
def test_grad_sq_norm_allocates_on_the_calls_stream(monkeypatch, given):
    import torch
    made = _fake_streams(monkeypatch)
    library = _NoLaunch("sbp_grad_sq_norm")
    monkeypatch.setattr(sbp, "lib", lambda: library)
    x = _Fake((300,), torch.bfloat16, torch.device("cuda", 0), "current", 0x1000000)
    out = sbp.grad_sq_norm([x], None, 1.0, 300, stream=given)
    assert [m.made_on for m in made] == [ON[given]] * 2 and out is made[1]
    assert library.streams == [given or None]
    assert given is None or out.used_on == ["current"]


@pytest.mark.parametrize("shape", [(7,), (2, 3, 4, 5)])
def test_newton_schulz_workspace_of_other_dimensions(shape):
    """The sizes are asked for what the call takes, and for nothing else."""
    import torch
    with pytest.raises(ValueError, match="2-D, or 3-D"):
        sbp.newton_schulz_workspace([torch.empty(shape, dtype=torch.bfloat16, device="meta")])


def test_newton_schulz_workspace_of_refused_sizes():
    """Refused with the status that the call itself gives."""
    import torch
    x = torch.empty((1 << 20) + 1, 4, dtype=torch.bfloat16, device="meta")
    with pytest.raises(sbp.SbpError, match="SBP_NS_MAX_DIM") as e:
        sbp.newton_schulz_workspace([x])
    assert e.value.status == sbp.SBP_ERANGE


# ---- the models that the device's results are told from ----------------------------

def _values(shape, kind):
    return OS.bf16_to_f32(NS.update(shape, 61, kind)).astype(np.float64)


@pytest.mark.parametrize("shape", NS.SHAPES)
@pytest.mark.parametrize("steps", [3, 5])
def test_models_tell_a_mistake(shape, steps):
    """Results of binary32 sums, rounded to bf16, with a mistake planted in the
    oracle: each is told from the others, and none is seen where there is none."""
    U = _values(shape, "flat")
    result = lambda **kw: NS.rounded(OS.newton_schulz_rounded(  # noqa: E731
        U, steps, COEFS, sums=np.float32, **kw))
    assert NS.nearest(result(), U, steps, COEFS) is None
    for what, kw in NS.MISTAKES.items():
        if steps == 3 and "rest_x" in kw:
            continue  # none is kept in the last three steps
        found = NS.nearest(result(**kw), U, steps, COEFS)
        assert found is not None, what
        if 0.0 in kw.values():
            assert found.split("'")[0].split()[0] == what.split("'")[0].split()[0], (what, found)


@pytest.mark.parametrize("shape", NS.SHAPES)
@pytest.mark.parametrize("kind", ["flat", "strong", "steep", "sixteen"])
def test_models_size_of_the_error(shape, kind):
    """Binary32 sums are as far off as said; without B's remainder (noise), or
    without X's (steep spectra), further than is allowed."""
    U = _values(shape, kind)
    for steps in (3, 5):
        y = NS.rounded(OS.newton_schulz_rounded(U, steps, COEFS, sums=np.float32))
        assert NS.off(y, U, steps, COEFS) < NS.ALLOWED
    worse = {"flat": dict(diag_a=0.0, diag_b=0.0), "steep": dict(rest_x=0.0),
             "sixteen": dict(rest_x=0.0)}.get(kind)
    if worse:
        y = NS.rounded(OS.newton_schulz_rounded(U, 5, COEFS, sums=np.float32, **worse))
        assert NS.off(y, U, 5, COEFS) > NS.ALLOWED


def test_error_before_the_outputs_rounding():
    """What the header says of the error: 5 steps, spectra from flat to few
    directions over next to nothing."""
    rng = np.random.default_rng(8)
    for m, n in ((200, 300), (128, 512)):
        g = rng.standard_normal((m, n))
        for k in (1, 4, 16, 64):
            low = rng.standard_normal((m, k)) @ rng.standard_normal((k, n))
            for noise in (1.0, 0.1, 0.03, 0.01, 0.003, 0.0003):
                U = NS.rounded(low + noise * g)
                e = OS.newton_schulz(U, 5, COEFS)
                r = OS.newton_schulz_rounded(U, 5, COEFS)
                assert np.linalg.norm(r - e) < 2.6e-3 * np.linalg.norm(e), (m, k, noise)
