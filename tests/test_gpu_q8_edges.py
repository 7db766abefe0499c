"""The 8-bit operators at special values: where a NaN, an infinity or a value
at the end of fp32's range may reach, in every form of the kernels.

Oracle and tolerances are those of tests/test_gpu_q8.py.
"""
import numpy as np
import pytest
import torch

import structured_rotations_amd as H
from oracle import q8_oracle as Q
from tests.test_gpu_q8 import TOL, np64, operands, rel_rows, say, to_codes, to_scales

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- products
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_matmul_nan_stays_in_its_tile(kind):
    # 17 x 17 tiles of 256 x 256: 289, so that some of 256 workgroups compute a second one after the first.  Every
    # row of tiles has a NaN code in another row of the tile, in the last block of 128; one weight block is NaN
    say("matmul nan, two tiles per workgroup", kind)
    rng = np.random.default_rng(51)
    rows, n, k = 4352, 4352, 384
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, kind)
    bad = [256 * t + 32 + (7 * t) % 32 for t in range(17)]
    ac[bad, 300] = 0x7f
    wc[1024:1152, 256:] = 0x7f
    ws[8, 2] = np.nan
    y = H.harp_matmul_q8(to_codes(ac), to_scales(as_, kind), to_codes(wc), to_scales(ws, kind), "bf16")
    torch.cuda.synchronize()
    got = np64(y)
    mask = np.zeros((rows, n), dtype=bool)
    mask[bad] = True
    mask[:, 1024:1152] = True
    assert np.array_equal(np.isnan(got), mask)
    ok = np.setdiff1d(np.arange(rows), bad)
    cols = np.r_[0:1024, 1152:n]
    want = Q.matmul(ac[ok], as_[ok], wc, np.where(np.isnan(ws), 0, ws))
    assert rel_rows(got[np.ix_(ok, cols)], want[:, cols]) <= TOL["bf16"]
