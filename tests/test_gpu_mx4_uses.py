"""The microscaled 4-bit calls as a program uses them: operands from a plan's gathered
shards, every form of the product on streams and in graphs, with the workspaces that
they need."""

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp
from oracle import mx4 as OM
from tests import helpers as H
from tests.test_gpu_mx4 import _check_product, _data, _device, _operand
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
