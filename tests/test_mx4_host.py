"""Microscaled 4-bit floats on the host (CPU only): the oracle's quantization,
generator and values against closed forms, and every refusal of the calls (the
fake addresses are never dereferenced)."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from oracle import mx4 as OM

V = ctypes.c_void_p
F32 = np.float32


# ---- the oracle ------------------------------------------------------------------

def _row(*xs):
    """One block: the given values, then zeros."""
    v = np.zeros((1, 32), F32)
    v[0, :len(xs)] = xs
    return v


def test_grid_values_are_kept():
    """With 4 in the block the scale is 1 and every grid value is itself."""
    g = np.concatenate([OM.GRID, -OM.GRID]).astype(F32)
    for seed in (None, 5):
        code, s = OM.quantize(_row(*g), seed)
        assert s[0, 0] == 127
        assert np.array_equal(code[0, 0, :16], np.arange(16))
        assert np.array_equal(OM.values(OM.pack(code), s, 16)[0], g)


def test_nearest_ties_go_to_the_even_code():
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    code, s = OM.quantize(_row(4.0, *mids, *[-m for m in mids]))
    assert s[0, 0] == 127
    assert code[0, 0, 1:8].tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert code[0, 0, 8:15].tolist() == [8, 10, 10, 12, 12, 14, 14]


def test_nearest_saturates_at_six():
    code, s = OM.quantize(_row(7.99, 6.5, 5.01))
    assert s[0, 0] == 127 and code[0, 0, :3].tolist() == [7, 7, 7]
    code, s = OM.quantize(_row(8.0, 7.0))
    assert s[0, 0] == 128 and code[0, 0, :2].tolist() == [6, 6]  # 3.5 -> 4


def test_random_never_saturates():
    code, s = OM.quantize(_row(6.0), 1)
    assert s[0, 0] == 127 and code[0, 0, 0] == 7
    code, s = OM.quantize(_row(np.nextafter(F32(6), F32(7))), 1)
    assert s[0, 0] == 128


def test_blocks_of_nan_zeros_and_the_least_values():
    for bad in (np.nan, np.inf, -np.inf):
        code, s = OM.quantize(_row(1.0, bad))
        assert s[0, 0] == 255 and not code.any()
        assert np.isnan(OM.values(OM.pack(code), s, 32)).all()
    code, s = OM.quantize(_row(0.0, -0.0))
    assert s[0, 0] == 0 and code[0, 0, :3].tolist() == [0, 8, 0]
    tiny = F32(2.0 ** -127)  # the scale cannot go lower: itself a grid value
    code, s = OM.quantize(_row(tiny, 3 * tiny, tiny / 4))
    assert s[0, 0] == 0 and code[0, 0, :3].tolist() == [2, 5, 0]


def test_random_rounding_is_unbiased():
    """The mean of n draws of a value t of a step above its lower code is t with
    a deviation of sqrt(t (1 - t) / n); five of them, and 2^-16 for the bits."""
    n = 1 << 16
    for x, low, step in ((0.1, 0.0, 0.5), (1.2, 1.0, 0.5), (2.3, 2.0, 1.0), (5.7, 4.0, 2.0)):
        v = np.full((n // 16, 32), 0, F32)
        v[:, 0] = 6.0
        v[:, 1:17] = F32(x)
        code, s = OM.quantize(v, 11, 3)
        got = OM.values(OM.pack(code), s, 32)[:, 1:17]
        t = (float(F32(x)) - low) / step
        assert abs((got.mean() - low) / step - t) <= 5 * np.sqrt(t * (1 - t) / n) + 2.0 ** -16
        assert set(np.unique(got)) <= {low, low + step}


def test_philox_is_the_published_one():
    """Known answers of the generator (its paper's test vectors)."""
    w = OM.philox([0], False, 0, 0)[0]
    assert [int(x) for x in w] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    full = (1 << 64) - 1
    w = OM.philox([full], False, full, full)[0]
    assert [int(x) for x in w] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert not np.array_equal(OM.philox([7], True, 1, 2), OM.philox([7], False, 1, 2))


def test_reduce_is_ascending():
    a, b, c = (np.array([x], F32) for x in (2.0 ** 24, 1.0, 1.0))
    assert OM.reduce([a, b, c], None, 1.0)[0] == 2.0 ** 24  # each 1 is lost
    assert OM.reduce([b, c, a], None, 1.0)[0] == 2.0 ** 24 + 2
    assert OM.reduce([b], np.array([3.0], F32), 0.5)[0] == 2.0


# ---- refusals ----------------------------------------------------------------------

EINVAL, EALIGN, ERANGE = sbp.SBP_EINVAL, sbp.SBP_EALIGN, sbp.SBP_ERANGE
MOST = sbp.MAX_SHARD_NUMEL


def _quantize(**kw):
    a = dict(x=V(0x1000000), type=sbp.SBP_BF16, rows=64, cols=96, ld=96, codes=V(0x2000000),
             scales=V(0x3000000), codes_t=V(0x4000000), scales_t=V(0x5000000), random=None)
    a.update(kw)
    return sbp.lib().sbp_mx_quantize(a["x"], a["type"], a["rows"], a["cols"], a["ld"], a["codes"],
                                      a["scales"], a["codes_t"], a["scales_t"], a["random"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), EINVAL), (dict(type=-1), EINVAL),
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(ld=95), EINVAL),
    (dict(ld=(1 << 40) + 1), ERANGE),
    (dict(rows=1, cols=MOST + 1), ERANGE), (dict(rows=MOST + 1, cols=1), ERANGE),
    (dict(rows=1 << 20, cols=1 << 16, ld=1 << 16), ERANGE),
    (dict(rows=MOST // 32 + 1, cols=1, ld=1), ERANGE),  # whole blocks of 32 a row
    (dict(x=None), EINVAL),
    (dict(codes=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(codes_t=None), EINVAL), (dict(scales_t=None), EINVAL),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), EINVAL),
    (dict(x=V(0x1000001)), EALIGN), (dict(x=V(0x1000002), type=sbp.SBP_F32), EALIGN),
    (dict(codes=V(0x2000008)), EALIGN), (dict(codes_t=V(0x4000008)), EALIGN),
    (dict(codes=V(0x1000000)), EINVAL), (dict(scales=V(0x1000000)), EINVAL),
    (dict(codes_t=V(0x2000000)), EINVAL), (dict(scales_t=V(0x3000000)), EINVAL),
    # the last row's end: 63 * 96 + 96 elements of 2 bytes
    (dict(codes=V(0x1000000 + 64 * 96 * 2 - 16)), EINVAL),
])
def test_quantize_refusals(kw, status):
    assert _quantize(**kw) == status
    assert "sbp_mx_quantize" in sbp.lib().sbp_last_error().decode()


def test_nothing_to_quantize():
    for kw in (dict(rows=0), dict(cols=0), dict(rows=0, x=None, codes=None, scales=None)):
        assert _quantize(**kw) == sbp.SBP_OK


def _dequantize(**kw):
    a = dict(codes=V(0x2000000), scales=V(0x3000000), rows=64, cols=96, out=V(0x1000000),
             type=sbp.SBP_BF16, ld=96)
    a.update(kw)
    return sbp.lib().sbp_mx_dequantize(a["codes"], a["scales"], a["rows"], a["cols"], a["out"],
                                        a["type"], a["ld"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=3), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=-2), EINVAL), (dict(ld=90), EINVAL),
    (dict(rows=1, cols=MOST + 1), ERANGE), (dict(ld=(1 << 40) + 1), ERANGE),
    (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(out=None), EINVAL),
    (dict(codes=V(0x2000004)), EALIGN), (dict(out=V(0x1000001)), EALIGN),
    (dict(out=V(0x1000002), type=sbp.SBP_F32), EALIGN),
    (dict(out=V(0x2000000)), EINVAL), (dict(out=V(0x3000000)), EINVAL),
])
def test_dequantize_refusals(kw, status):
    assert _dequantize(**kw) == status
    assert "sbp_mx_dequantize" in sbp.lib().sbp_last_error().decode()


def _reduce(**kw):
    a = dict(codes=(V * 2)(0x1000000, 0x2000000), scales=(V * 2)(0x3000000, 0x4000001), R=2,
             n=1000, acc=None, scale=0.5, out=V(0x5000000))
    a.update(kw)
    return sbp.lib().sbp_mx_reduce_shard(a["codes"], a["scales"], a["R"], a["n"], a["acc"],
                                          a["scale"], a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), EINVAL), (dict(R=17), EINVAL), (dict(n=-1), EINVAL), (dict(n=MOST + 1), ERANGE),
    (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(out=None), EINVAL),
    (dict(codes=(V * 2)(0x1000000, None)), EINVAL), (dict(scales=(V * 2)(None, 0x3000000)), EINVAL),
    (dict(codes=(V * 2)(0x1000000, 0x2000008)), EALIGN),
    (dict(out=V(0x5000008)), EALIGN), (dict(acc=V(0x6000004)), EALIGN),
    (dict(out=V(0x1000000)), EINVAL), (dict(out=V(0x4000000)), EINVAL),
    (dict(acc=V(0x5000010)), EINVAL),  # shifted against out
])
def test_reduce_refusals(kw, status):
    assert _reduce(**kw) == status
    assert "sbp_mx_reduce_shard" in sbp.lib().sbp_last_error().decode()


def test_nothing_to_reduce():
    assert _reduce(n=0, codes=None, scales=None, out=None) == sbp.SBP_OK


def _matmul(**kw):
    a = dict(codes_a=V(0x1000000), scales_a=V(0x2000000), codes_b=V(0x3000000),
             scales_b=V(0x4000000), m=300, n=200, k=100, out=V(0x5000000), type=sbp.SBP_BF16,
             ld=200, accumulate=0, workspace=V(0x100000000), bytes=1 << 40)
    a.update(kw)
    return sbp.lib().sbp_mx_matmul(
        a["codes_a"], a["scales_a"], a["codes_b"], a["scales_b"], a["m"], a["n"], a["k"],
        a["out"], a["type"], a["ld"], a["accumulate"], a["workspace"], a["bytes"], None)


BIG = dict(m=8192, n=8192, k=512, ld=8192, codes_b=V(0x2000000), scales_a=V(0x3000000),
           scales_b=V(0x4000000), out=V(0x50000000))
DIM, MAX_K = sbp.MX_MAX_DIM, sbp.MX_MAX_K


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), EINVAL), (dict(n=-1), EINVAL), (dict(k=-1), EINVAL),
    (dict(m=DIM + 1), ERANGE), (dict(n=DIM + 1), ERANGE), (dict(k=MAX_K + 1), ERANGE),
    (dict(m=1 << 20, k=MAX_K), ERANGE), (dict(n=1 << 20, ld=1 << 20, k=MAX_K), ERANGE),
    (dict(m=1 << 20, n=(1 << 16) + 1, ld=1 << 20), ERANGE),
    (dict(type=2), EINVAL), (dict(accumulate=1), EINVAL),
    (dict(ld=199), EINVAL), (dict(ld=(1 << 32) + 1), ERANGE),
    (dict(codes_a=None), EINVAL), (dict(scales_a=None), EINVAL),
    (dict(codes_b=None), EINVAL), (dict(scales_b=None), EINVAL), (dict(out=None), EINVAL),
    (dict(codes_a=V(0x1000008)), EALIGN), (dict(codes_b=V(0x3000001)), EALIGN),
    (dict(out=V(0x5000001)), EALIGN), (dict(out=V(0x5000002), type=sbp.SBP_F32), EALIGN),
    (dict(out=V(0x1000000)), EINVAL), (dict(out=V(0x2000000)), EINVAL),
    (dict(out=V(0x3000000)), EINVAL), (dict(out=V(0x4000000)), EINVAL),
    # 8192 x 8192: large tiles, whose workspace holds the packed scales
    (dict(BIG, workspace=None), EINVAL), (dict(BIG, workspace=V(0x100000080)), EALIGN),
    (dict(BIG, bytes=sbp.mx_matmul_workspace(8192, 8192, 512) - 1), EINVAL),
    (dict(BIG, workspace=V(0x1000000)), EINVAL), (dict(BIG, workspace=V(0x4000000)), EINVAL),
    (dict(BIG, workspace=V(0x50000000)), EINVAL),
])
def test_matmul_refusals(kw, status):
    assert _matmul(**kw) == status
    assert "sbp_mx_matmul" in sbp.lib().sbp_last_error().decode()


def test_nothing_to_multiply():
    for kw in (dict(m=0), dict(n=0), dict(k=0, type=sbp.SBP_F32, accumulate=1)):
        assert _matmul(codes_a=None, out=None, **kw) == sbp.SBP_OK


def test_workspace_of_each_form():
    """None for few rows and for tiles that are many or short; packed scales for large
    ones; parts' sums for few tiles with long sums."""
    assert sbp.mx_matmul_workspace(1, 4096, 4096) == 0
    assert sbp.mx_matmul_workspace(512, 512, 512) == 0
    assert sbp.mx_matmul_workspace(8192, 8192, 512) == 2 * 8192 * 16
    assert sbp.mx_matmul_workspace(100, 300, 8192) == 4 * 100 * 300 * 4
    assert sbp.mx_matmul_workspace(0, 10, 10) == 0


def test_workspace_refuses_bad_sizes():
    for m, n, k, status in ((-1, 4, 4, EINVAL), (4, DIM + 1, 4, ERANGE), (4, 4, MAX_K + 1, ERANGE)):
        with pytest.raises(sbp.SbpError) as e:
            sbp.mx_matmul_workspace(m, n, k)
        assert e.value.status == status


# ---- the binding's own checks (host tensors stand in: they are refused first) --------

def test_mx4_checks_its_tensors():
    import torch
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    q = sbp.Mx4(u8(5, 48), u8(5, 3), (5, 70))
    assert q.shape == (5, 70) and q.numel == 350
    assert q.rows_of(1, 3).shape == (2, 70)
    for codes, scales, shape in (
            (u8(5, 32), u8(5, 3), (5, 70)), (u8(5, 48), u8(5, 2), (5, 70)),
            (u8(5, 48).int(), u8(5, 3), (5, 70)), (u8(10, 48)[::2], u8(5, 3), (5, 70)),
            (u8(5, 48), u8(5, 6)[:, ::2], (5, 70)), (u8(5, 48), u8(5, 3), (4, 70))):
        with pytest.raises(ValueError):
            sbp.Mx4(codes, scales, shape)
    for a, b in ((-1, 2), (2, 1), (0, 6)):
        with pytest.raises(ValueError):
            q.rows_of(a, b)
    assert sbp.Mx4.empty(0, 10, "cpu").numel == 0


def test_calls_refuse_host_tensors_and_shapes():
    import torch
    x = torch.zeros(4, 64)
    q = sbp.Mx4.empty(4, 64, "cpu")
    for call in (lambda: sbp.mx_quantize(x), lambda: sbp.mx_quantize(x, along="up"),
                 lambda: sbp.mx_quantize(x.double()), lambda: sbp.mx_quantize(x[None]),
                 lambda: sbp.mx_matmul(q, sbp.Mx4.empty(4, 65, "cpu")),
                 lambda: sbp.mx_matmul(q, q, accumulate=True)):
        with pytest.raises(ValueError):
            call()


def test_one_hip_runtime_whatever_is_loaded_first():
    """The library loaded before the caller imports torch: torch's HIP runtime serves
    both (with a second one the library's calls find no device)."""
    code = ("import sharded_bucket_plan_amd as sbp; sbp.lib(); import torch; "
            "torch.cuda.is_available(); "
            "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "1", r.stdout + r.stderr


def test_planner_works_where_torch_is_not_installed():
    """Host-only use (plans, queries, sizes, factors) needs no torch."""
    code = ("import sys; sys.modules['torch'] = None; import sharded_bucket_plan_amd as sbp; "
            "plan = sbp.bucket_plan([100, 30], 1 << 20, world_n=2); "
            "print(plan.shard_numel, plan.bucket(0)['padded'], sbp.mean_scale(4), "
            "sbp.mx_matmul_workspace(8192, 8192, 512))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    # 30 values, 2 to the next multiple of 8, 100 more: padded to a multiple of 2 * 8
    assert r.stdout.split() == ["72", "144", "0.25", str(2 * 8192 * 16)]


def test_a_torch_that_does_not_load_is_not_passed_over():
    """A torch that is installed but broken raises its own error: going on without it
    would put a second HIP runtime beside it later."""
    code = ("import sys, importlib.abc\n"
            "class Broken(importlib.abc.MetaPathFinder):\n"
            "    def find_spec(self, name, path, target=None):\n"
            "        if name == 'torch': raise ImportError('torch is broken', name='torch._C')\n"
            "sys.meta_path.insert(0, Broken())\n"
            "import sharded_bucket_plan_amd as sbp\n"
            "sbp.lib()\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode != 0 and "torch is broken" in r.stderr


# rows * ld past what 64 bits hold in bytes: the overlap checks would be made with a wrapped length
FAR = [(1 << 27, 1 << 40), (1 << 29, 1 << 34), ((1 << 20) + 1, 1 << 40), ((1 << 30) - 64, 1 << 40)]


@pytest.mark.parametrize("rows,ld", FAR)
@pytest.mark.parametrize("type_", [sbp.SBP_BF16, sbp.SBP_F32])
def test_arrays_longer_than_an_address_are_refused(rows, ld, type_):
    # 0x2000000 lies behind the first row's end and inside the array
    far = dict(rows=rows, cols=32, ld=ld, type=type_)
    assert _dequantize(out=V(0x1000000), **far) == ERANGE
    assert "sbp_mx_dequantize" in sbp.lib().sbp_last_error().decode()
    assert _quantize(codes_t=None, scales_t=None, scales=V(1 << 50), **far) == ERANGE
    assert "sbp_mx_quantize" in sbp.lib().sbp_last_error().decode()


@pytest.mark.parametrize("rows,ld", [(1 << 20, 1 << 40), (1 << 27, 1 << 33)])
def test_overlaps_of_the_longest_arrays_are_seen(rows, ld):
    last = 0x1000000 + (rows - 1) * ld * 4  # where the last row begins
    far = dict(rows=rows, cols=32, ld=ld, type=sbp.SBP_F32, codes=V((1 << 62) + (1 << 40)))
    assert _dequantize(out=V(0x1000000), scales=V(last), **far) == EINVAL
    assert "overlaps" in sbp.lib().sbp_last_error().decode()
    assert _quantize(codes_t=None, scales_t=None, scales=V(last), **far) == EINVAL
    assert "overlap" in sbp.lib().sbp_last_error().decode()


# ---- from a plan to an operand --------------------------------------------------------

def _shards(plan, tensors, N):
    """Each rank's fp32 master shard: its chunk of every tensor, at the plan's places."""
    shards = [np.zeros(plan.shard_numel, F32) for _ in range(N)]
    for t, x in enumerate(tensors):
        b = plan.bucket(plan.tensor(t)[0])
        padded = np.zeros(b["padded"], F32)
        padded[:x.size] = x.reshape(-1)
        for r in range(N):
            shards[r][b["shard_offset"]:b["shard_offset"] + b["chunk"]] = \
                padded[r * b["chunk"]:(r + 1) * b["chunk"]]
    return shards


@pytest.mark.parametrize("N", [1, 2, 3, 8])
def test_gathered_chunks_of_a_plan_are_operands(N):
    """Shards quantized as flat buffers; a tensor's blocks of every rank's, one behind the
    other, are the tensor quantized as a matrix, and then rows of zeros."""
    rng = np.random.default_rng(N)
    shapes = [(50, 96), (13,), (7, 32), (1, 64), (129, 160)]
    tensors = [rng.standard_normal(s).astype(F32) for s in shapes]
    plan = sbp.bucket_plan_per_tensor([x.size for x in tensors], N,
                                      [s[-1] if len(s) == 2 else 1 for s in shapes], align=32)
    shards = [OM.quantize(s[None]) for s in _shards(plan, tensors, N)]
    for t, x in enumerate(tensors):
        if x.ndim == 1:
            continue
        b = plan.bucket(plan.tensor(t)[0])
        assert b["shard_offset"] % 32 == 0 and b["chunk"] % x.shape[1] == 0
        blocks = slice(b["shard_offset"] // 32, (b["shard_offset"] + b["chunk"]) // 32)
        code = np.concatenate([c[0, blocks] for c, _ in shards])
        scale = np.concatenate([s[0, blocks] for _, s in shards])
        kb = x.shape[1] // 32
        want_code, want_scale = OM.quantize(x)
        assert np.array_equal(code.reshape(-1, kb, 32)[:len(x)], want_code)
        assert np.array_equal(scale.reshape(-1, kb)[:len(x)], want_scale)
        assert not code.reshape(-1, kb, 32)[len(x):].any()


def test_plans_of_finer_alignment_may_begin_rows_inside_a_block():
    """Why the alignment has to be a multiple of 32."""
    plan = sbp.bucket_plan_per_tensor([13, 50 * 96], 1, [1, 96], align=8, order="forward")
    assert plan.bucket(plan.tensor(1)[0])["shard_offset"] == 16


# ---- no memory on the host ---------------------------------------------------------------

def test_no_exception_leaves_a_call(tmp_path):
    """tests/native/no_memory.cpp: operator new fails at each place where the calls use it."""
    from tests import helpers as H
    r = H.run_native("no_memory.cpp", tmp_path)
    assert r.returncode == 0 and "no exception left a call" in r.stdout, r.stdout + r.stderr
