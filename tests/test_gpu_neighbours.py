"""Packed batches whose sequences lie closer than a tile of keys: what one
sequence holds, non-finite values among it, stays out of the others, and a
buffer is read within its rows (needs a B200)."""
import numpy as np
import pytest
import torch

import gpu_helpers as H
import varlen_gqa_split_b200 as vg
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


@pytest.mark.parametrize("Hq,max_q", [(8, 1), (16, 5), (4, 100)])
@pytest.mark.parametrize("ctas", [3, 40])
@pytest.mark.parametrize("det", [-1, 1])
def test_foreign_rows_stay_out_of_cut_units(Hq, max_q, ctas, det):
    """The same with units cut between blocks, balanced at run time too."""
    lk = np.array([300, 5, 40, 1000, 2, 63])
    lq = np.minimum(max_q, np.array([1, 9, 100, 30, 3, 70]))
    sh = W.Shape("cut", B=6, Hq=Hq, Hkv=1, D=128, max_q=max_q, s_max=1000)
    batch = W.make_batch(sh, lq, lk, seed=6)
    ref_o, ref_l = H.oracle_full(batch)
    batch.v[:300], batch.k[:300] = float("nan"), float("inf")
    batch.v[305:345] = float("inf")
    o, l = H.run_gpu(H.plan_for(sh, deterministic=det, ctas=ctas), batch)
    q0 = np.concatenate([[0], np.cumsum(lq)])
    for b in (1, 3, 4, 5):
        s = slice(int(q0[b]), int(q0[b + 1]))
        H.check_values(o[s].float().numpy(), l[s].numpy(), ref_o[s], ref_l[s])


@pytest.mark.parametrize("Hq,Hkv,D,max_q", [(4, 1, 64, 1), (8, 2, 128, 4), (16, 2, 128, 7), (8, 1, 64, 40), (4, 4, 64, 300),
                                            (130, 1, 64, 1)])
@pytest.mark.parametrize("lk,lq", [([1], [1]), ([5, 3, 1], [1, 1, 1]), ([37, 100], [1, 9]), ([0, 20, 60, 2], [1, 0, 3, 2]),
                                   ([63, 64, 65], [40, 1, 7]), ([10, 200], [300, 2])])
def test_short_buffers(Hq, Hkv, D, max_q, lk, lq):
    """Buffers of fewer rows than a box of keys or of queries, cut out of larger
    ones whose other rows are NaN, packed and strided: nothing comes from
    outside them, with the rows stated (the binding) and without (attn_run)."""
    lq = np.minimum(lq, max_q)
    sh = W.Shape("rows", B=len(lk), Hq=Hq, Hkv=Hkv, D=D, max_q=max_q, s_max=256)
    batch = W.make_batch(sh, lq, np.array(lk), seed=3)
    ref_o, ref_l = H.oracle_full(batch)
    plan = H.plan_for(sh)
    q, k, v, cu_q, cu_k = H.to_device(batch)
    if not q.shape[0]:
        return
    room = [torch.full((t.shape[0] + 600, *t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda") for t in (q, k, v)]
    wide = torch.full((k.shape[0] + 600, 2, Hkv, D), float("nan"), dtype=k.dtype, device="cuda")
    for r, t in zip(room, (q, k, v)):
        r[300:300 + t.shape[0]] = t
    wide[300:300 + k.shape[0], 0], wide[300:300 + k.shape[0], 1] = k, v
    q, k, v = (r[300:300 + t.shape[0]] for r, t in zip(room, (q, k, v)))
    w = wide[300:300 + k.shape[0]]

    def check(run):
        out, lse = H.sentinel_out(q.shape[0], Hq, D), H.sentinel_lse(q.shape[0], Hq)
        run(out, lse)
        torch.cuda.synchronize()
        assert plan.check_error() == 0
        H.compare_full(out.cpu(), lse.cpu(), ref_o, ref_l, H.covered_rows(batch))

    check(lambda o, l: plan.run(q, k, v, cu_q, cu_k, o, l))
    check(lambda o, l: plan.run(q, w[:, 0], w[:, 1], cu_q, cu_k, o, l))
    L = vg.lib()
    check(lambda o, l: H_ok(L.attn_run(plan.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(),
                                       cu_k.data_ptr(), o.data_ptr(), l.data_ptr(), None)))
    pc = W.paginate(k, v, batch.cu_k, len(lk), 16, 256, seed=1)
    check(lambda o, l: plan.run_paged(q, pc.k_cache, pc.v_cache, pc.block_table, cu_q, cu_k, o, l))


def H_ok(rc):
    assert rc == 0


@pytest.mark.parametrize("Hq,max_q", [(4, 1), (16, 8), (300, 1)])
def test_offsets_past_the_stated_rows_are_errors(Hq, max_q):
    """A sequence that reaches past the rows of q or of k is reported and left
    unwritten, the others are not touched by it."""
    sh = W.Shape("past", B=3, Hq=Hq, Hkv=1, D=64, max_q=max_q, s_max=128)
    batch = W.make_batch(sh, [1, 1, 1], [20, 100, 30], seed=4)
    plan = H.plan_for(sh)
    q, k, v, cu_q, cu_k = H.to_device(batch)
    ref_o, ref_l = H.oracle_full(batch)
    o, l = H.sentinel_out(3, Hq, 64), H.sentinel_lse(3, Hq)
    plan.run(q, k[:149], v[:150], cu_q, cu_k, o, l)              # one row short for the third
    assert plan.check_error() == vg.ATTN_DEV_ERR_OFFSETS
    H.compare_full(o.cpu(), l.cpu(), ref_o, ref_l, np.array([True, True, False]))
    o, l = H.sentinel_out(2, Hq, 64), H.sentinel_lse(2, Hq)
    plan.run(q[:2], k, v, cu_q, cu_k, o, l)
    assert plan.check_error() == vg.ATTN_DEV_ERR_OFFSETS
    H.compare_full(o.cpu(), l.cpu(), ref_o[:2], ref_l[:2], np.array([True, True]))
    pc = W.paginate(k, v, batch.cu_k, 3, 16, 128, seed=1)
    o, l = H.sentinel_out(2, Hq, 64), H.sentinel_lse(2, Hq)
    plan.run_paged(q[:2], pc.k_cache, pc.v_cache, pc.block_table, cu_q, cu_k, o, l)
    assert plan.check_error() == vg.ATTN_DEV_ERR_OFFSETS
    H.compare_full(o.cpu(), l.cpu(), ref_o[:2], ref_l[:2], np.array([True, True]))


def test_calls_without_rows():
    """No query row: nothing to do.  No key row: every query sees nothing."""
    for Hq, max_q in ((4, 1), (16, 8), (300, 1)):
        plan = Plan(2, 64, Hq, 1, 64, max_q)
        k = torch.ones(0, 1, 64, dtype=torch.bfloat16, device="cuda")
        q = torch.ones(2, Hq, 64, dtype=torch.bfloat16, device="cuda")
        cu = torch.zeros(3, dtype=torch.int32, device="cuda")
        o, l = plan.run(q[:0], k, k, cu, cu)
        assert o.shape == (0, Hq, 64) and l.shape == (0, Hq)
        o, l = plan.run(q, k, k, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), cu)
        assert (o == 0).all() and l.isneginf().all() and plan.check_error() == 0


def test_refusals_of_row_counts():
    L = vg.lib()
    plan = Plan(1, 64, 4, 1, 64, 1)
    t = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda").data_ptr()

    def run(q=t, T_q=1, k=t, v=t, T_kv=8, ks=64, vs=64):
        return L.attn_run_rows(plan.handle, q, T_q, k, v, T_kv, ks, vs, t, t, t, t, None)

    assert run(T_q=-1) == run(T_kv=-1) == run(T_q=1 << 31) == run(T_kv=1 << 31) == run(ks=60) == run(vs=68) == -1
    assert run(q=None) == run(k=None) == run(v=None) == run(q=None, T_kv=0) == -3
    assert run(q=None, T_q=0) == 0 and run(q=t + 8) == -4

    def paged(q=t, T_q=1):
        return L.attn_run_paged_rows(plan.handle, q, T_q, t, t, 1024, 64, 16, 4, t, 4, t, t, t, t, None)

    assert paged(T_q=-1) == paged(T_q=1 << 31) == -1 and paged(q=None) == -3 and paged(q=None, T_q=0) == 0
