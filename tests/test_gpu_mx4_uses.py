"""The microscaled 4-bit calls as a program uses them: operands from a plan's gathered
shards, every form of the product on streams and in graphs, with the workspaces that
they need."""

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from oracle import mx4 as OM
from tests import helpers as H
from tests.test_gpu_mx4 import _check_product, _data, _device, _operand, _same_codes
from tests.test_gpu_mx4_forms import exact_operand
from tests.test_mx4_host import _shards

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    H.need_gpu()
    yield
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N", [1, 3])
def test_from_a_plan_to_a_product(N):
    """Each rank's fp32 master shard to 4 bits as one flat buffer; the chunks of a weight,
    one behind the other, into the product."""
    import torch
    rng = np.random.default_rng(N)
    shapes = [(130, 96), (13,), (257, 160)]
    tensors = [rng.standard_normal(s).astype(np.float32) for s in shapes]
    plan = sbp.bucket_plan_per_tensor([x.size for x in tensors], N, [96, 1, 160], align=32)
    shards = [sbp.mx_quantize(torch.from_numpy(s).to(H.dev())) for s in _shards(plan, tensors, N)]
    for t in (0, 2):
        rows, cols = shapes[t]
        b = plan.bucket(plan.tensor(t)[0])
        first, last = b["shard_offset"] // 32, (b["shard_offset"] + b["chunk"]) // 32
        codes = torch.cat([q.codes[0, 16 * first:16 * last] for q in shards])
        scales = torch.cat([q.scales[0, first:last] for q in shards])
        kb = cols // 32
        w = sbp.Mx4(codes.view(-1, 16 * kb), scales.view(-1, kb), (b["padded"] // cols, cols))
        w = w.rows_of(0, rows)
        x, xv = _operand(40, cols, 70 + t)
        code, scale = OM.quantize(tensors[t])
        _check_product(sbp.mx_matmul(x, w).float().cpu().numpy(), xv,
                       OM.values(OM.pack(code), scale, cols), True, what=f"tensor {t}")


# two kernels each: parts of a long sum and their joining, packed scales and large tiles
WITH_WORKSPACE = [(300, 280, 7200), (300, 280, 6113), (2900, 2952, 300), (2900, 2950, 1600)]


@pytest.mark.parametrize("m,n,k", WITH_WORKSPACE)
@pytest.mark.parametrize("own", [False, True])
def test_workspaces_of_two_streams(m, n, k, own):
    """Products of two pairs of operands by turns on two streams, with the calls' workspaces
    (own: the caller's, one a stream, filled with NaN scales and values)."""
    import torch
    size = sbp.mx_matmul_workspace(m, n, k)
    assert size > 0
    pairs = [[exact_operand(r, k, seed + i) for i, r in enumerate((m, n))] for seed in (1, 11)]
    wants = [(a[1] @ b[1].T).float() for a, b in pairs]
    spaces = [torch.full((size,), 255, dtype=torch.uint8, device=H.dev()) if own else None
              for _ in pairs]
    streams = [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, ((a, _), (b, _)) in enumerate(pairs):
            got[i].append(sbp.mx_matmul(a, b, dtype=torch.float32, workspace=spaces[i],
                                        stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, wants[i]) for g in got[i])


@pytest.mark.parametrize("m,n,k", WITH_WORKSPACE)
@pytest.mark.parametrize("shared", [False, True])
def test_workspaces_of_two_graphs(m, n, k, shared):
    """Two captured graphs, their workspaces the calls' or one that they share, replayed by
    turns with eager calls in between."""
    import torch
    size = sbp.mx_matmul_workspace(m, n, k)
    assert size > 0
    pairs = [[exact_operand(r, k, seed + i) for i, r in enumerate((m, n))] for seed in (2, 12)]
    wants = [(a[1] @ b[1].T).float() for a, b in pairs]
    ws = torch.full((size,), 255, dtype=torch.uint8, device=H.dev()) if shared else None
    outs = [torch.empty(m, n, device=H.dev()) for _ in pairs]
    for ((a, _), (b, _)), out in zip(pairs, outs):  # before the capture: loads the kernels
        sbp.mx_matmul(a, b, out, workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for ((a, _), (b, _)), out in zip(pairs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sbp.mx_matmul(a, b, out, workspace=ws)
        graphs.append(g)
    for rep in range(4):
        eager = sbp.mx_matmul(pairs[rep % 2][0][0], pairs[rep % 2][1][0], dtype=torch.float32)
        for out in outs:
            out.fill_(float("nan"))
        if shared:
            ws.fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, wants[rep % 2]), rep
        assert all(torch.equal(o, w) for o, w in zip(outs, wants)), rep


def _grid(rows, cols, seed):
    """Values of the format's grid, a 4 or a 6 in every block of 32 along rows and columns:
    quantized either way each is itself, with scale 1."""
    g = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    rng = np.random.default_rng(seed)
    x = g[rng.integers(0, 6, (rows, cols))] * rng.choice([-1.0, 1.0], (rows, cols))
    x[(np.arange(rows)[:, None] + np.arange(cols)) % 16 == 3] = 6
    return x.astype(np.float32)


def test_layer_gradients_are_differences():
    """The device's gradients against differences of the device's outputs: with values that
    quantization keeps, every product and sum is exact, and L = <dy, x W'> is linear in each
    entry of x and of W."""
    import torch
    t, d_in, d_out = 96, 160, 224
    x, w, dy = _grid(t, d_in, 80), _grid(d_out, d_in, 81), _grid(t, d_out, 82)

    def q(v, along="rows"):
        return sbp.mx_quantize(torch.from_numpy(v).to(H.dev()), along)

    def loss(x_, w_):
        y = sbp.mx_matmul(q(x_), q(w_), dtype=torch.float32)
        return float((y.double() * torch.from_numpy(dy).to(H.dev()).double()).sum())

    assert bool((sbp.mx_dequantize(q(w)).float().cpu() == torch.from_numpy(w)).all())
    gq, gt = q(dy, "both")
    dx = sbp.mx_matmul(gq, q(w, "cols"), dtype=torch.float32).cpu().numpy()
    dw = torch.zeros(d_out, d_in, device=H.dev())
    sbp.mx_matmul(gt, q(x, "cols"), dw, accumulate=True)
    dw = dw.cpu().numpy()
    before = loss(x, w)
    for r, c in ((0, 0), (5, 31), (40, 77), (t - 1, d_in - 1), (33, 64)):
        for v, grad, of in ((x, dx, lambda u: loss(u, w)), (w, dw, lambda u: loss(x, u))):
            moved = v.copy()
            moved[r, c] = 2.0 if v[r, c] != 2.0 else -1.5
            assert of(moved) - before == float(grad[r, c]) * float(moved[r, c] - v[r, c]), (r, c)


def _packed(x, seed):
    code, scale = OM.quantize(x, seed)
    return OM.pack(code), scale


# a block of lanes ends after 2048 values, a quad of lanes after 32, an octet after 8
@pytest.mark.parametrize("n", [7, 9, 2040, 2047, 2048, 2049, 2056, 2080, 3 * 2048 - 25, 5 * 2048])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seed", [None, 3])
def test_flat_ends(n, dtype, seed):
    x = _data(1, n, n)
    q = sbp.mx_quantize(_device(x, dtype)[0], seed=seed)
    _same_codes(q, OM.quantize(x, seed), f"n={n}")
    assert np.array_equal(sbp.mx_dequantize(q).float().cpu().numpy(),
                          OM.values(*_packed(x, seed), n).astype(np.float32))


# tiles of 128 x 128 in strips of four: one to 21 of them, strips of every width, counts
# that eight do not divide
@pytest.mark.parametrize("tiles", [(1, 1), (1, 3), (9, 1), (3, 3), (2, 4), (3, 5), (2, 6), (3, 7),
                                   (1, 9)])
@pytest.mark.parametrize("seed", [None, 3])
def test_matrix_tiles(tiles, seed):
    rows, cols = (128 * n - d for n, d in zip(tiles, (37, 30)))
    x = _data(rows, cols, rows)
    a, t = sbp.mx_quantize(_device(x, "bf16"), "both", seed=seed)
    _same_codes(a, OM.quantize(x, seed), "rows")
    _same_codes(t, OM.quantize(x.T, seed, 0, True), "cols")
    _same_codes(sbp.mx_quantize(_device(x, "f32"), "cols", seed=seed),
                OM.quantize(x.T, seed, 0, True), "cols alone")
