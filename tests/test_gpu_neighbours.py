"""Packed batches whose sequences lie closer than a tile of keys: what one
sequence holds, non-finite values among it, stays out of the others, and a
buffer is read within its rows (needs a B200)."""
import numpy as np
import pytest
import torch

import gpu_helpers as H
import oracle
import workloads as W
from varlen_gqa_split_b200 import Plan

pytestmark = pytest.mark.gpu


# G * max_q up to 16: warp MMA; up to 128 and in row tiles: tcgen05
@pytest.mark.parametrize("Hq,Hkv,D,max_q", [(4, 1, 64, 1), (8, 2, 128, 1), (8, 2, 64, 4), (16, 1, 64, 2), (16, 2, 128, 7),
                                            (4, 2, 64, 100)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_foreign_rows_stay_out(Hq, Hkv, D, max_q, bad):
    """Every second sequence of short ones is poisoned (K and V, or V alone);
    the others' results are those of finite neighbours, to the bit."""
    lk = np.array([5, 3, 40, 1, 70, 20, 63, 2, 130, 64, 7, 31])
    B = len(lk)
    lq = np.minimum(max_q, 1 + np.arange(B) * 5 % max_q)        # more queries than keys among them
    sh = W.Shape("near", B=B, Hq=Hq, Hkv=Hkv, D=D, max_q=max_q, s_max=160)
    batch = W.make_batch(sh, lq, lk, seed=5)
    plan = H.plan_for(sh, deterministic=1)
    clean_o, clean_l = H.run_gpu(plan, batch)
    ref_o, ref_l = H.oracle_full(batch)
    H.compare_full(clean_o, clean_l, ref_o, ref_l, H.covered_rows(batch))
    k0, q0 = np.cumsum(lk) - lk, np.cumsum(lq) - lq
    for odd in (0, 1):
        for both in (False, True):
            dirty = W.Batch(**{**batch.__dict__, "k": batch.k.clone(), "v": batch.v.clone()})
            for b in range(odd, B, 2):
                dirty.v[k0[b]:k0[b] + lk[b]] = bad
                if both:
                    dirty.k[k0[b]:k0[b] + lk[b]] = bad
            o, l = H.run_gpu(plan, dirty)
            for b in range(1 - odd, B, 2):
                s = slice(int(q0[b]), int(q0[b] + lq[b]))
                assert torch.equal(o[s], clean_o[s]) and torch.equal(l[s], clean_l[s]), (odd, both, b)
