"""Distances around the scaled matrix instructions that mx4_matmul.hip writes as
inline assembly (CPU only, on the disassembly of the built library): the same two
as newton_schulz.hip's, on every path, by the same reading of the code."""

import os
import shutil
import subprocess

import pytest

import sharded_bucket_plan_amd as sbp
from tests import test_matrix_unit_hazards as HZ


def test_hazards_of_scaled_products_are_found():
    """The scales are operands too: one that a vector instruction just wrote."""
    mfma = ("v_mfma_scale_f32_32x32x64_f8f6f4 a[0:15], v[0:3], v[4:7], a[0:15], v8, v9 "
            "op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4", "")
    end = ("s_endpgm", "")
    assert HZ.hazards(HZ._body([mfma, end])) == []
    assert len(HZ.hazards(HZ._body([("v_mov_b32_e32 v9, 0", ""), mfma, end]))) == 1
    assert len(HZ.hazards(HZ._body([mfma, ("v_accvgpr_read_b32 v20, a3", ""), end]))) == 1


def _of_large_tiles(lines):
    """The lines of the kernels looked at."""
    on = False
    for line in lines:
        if line.endswith(">:"):
            on = "mx4_tile_kernel" in line and "TileILi256ELi64" in line
        if on:
            yield line


@pytest.mark.skipif(shutil.which(HZ.OBJDUMP) is None, reason="needs llvm-objdump")
def test_large_tile_keeps_its_distances(tmp_path):
    sbp.lib()
    library = shutil.copy(sbp.LIB_PATH, tmp_path)
    subprocess.run([HZ.OBJDUMP, "--offloading", library], cwd=tmp_path, check=True,
                   capture_output=True)
    checked = {}
    for part in sorted(os.listdir(tmp_path)):
        if not part.endswith("gfx950"):
            continue
        r = subprocess.run([HZ.OBJDUMP, "-d", part], cwd=tmp_path, check=True,
                           capture_output=True, text=True)
        for name, body in HZ._kernels(_of_large_tiles(r.stdout.splitlines())):
            checked[name] = len([i for i in body if i.mfma])
            found = HZ.hazards(body)
            assert not found, f"{name}: {len(found)}, of them {found[:5]}"
            # accumulators are not moved about between the products
            first = min(k for k, i in enumerate(body) if i.mfma)
            last = max(k for k, i in enumerate(body) if i.mfma)
            assert not [i.text for i in body[first:last] if "accvgpr" in i.op], name
    # the three kinds of results, stored two ways; 32 products a slice, two rounds of four slices
    assert len(checked) == 6 and all(n == 32 * 8 for n in checked.values()), checked
