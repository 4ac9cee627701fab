"""Edges of the operators on the cache: calls without rows, infinite sums,
strides that do not matter, overlapping outputs (needs a B200)."""
import math

import numpy as np
import pytest
import torch

import varlen_gqa_split_b200 as vg
import workloads as W
from varlen_gqa_split_b200 import Plan, Rope, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from varlen_gqa_split_b200 import build
    build.build()
    torch.cuda.init()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(shape, seed):
    return torch.randn(shape, generator=_gen(seed), device="cuda").to(torch.bfloat16)


def _cu(lens):
    return torch.from_numpy(W.cu_from_lengths(lens)).cuda()


# ---------------------------------------------------------- calls without rows

@pytest.mark.parametrize("Hq,Hkv,max_q", [(8, 2, 1), (4, 1, 300), (260, 2, 2)])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("decay", [0.0, 0.5])
def test_key_weights_without_queries(Hq, Hkv, max_q, paged, decay):
    """No query in the whole batch: every key passes on its decayed weight."""
    lk = np.array([300, 0, 17])
    k = _bf16((317, Hkv, 64), 1)
    plan = Plan(3, 300, Hq, Hkv, 64, max_q)
    q, lse = torch.empty(0, Hq, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, Hq, device="cuda")
    w = torch.rand(3, Hkv, 300, generator=_gen(2), device="cuda")
    out, born = torch.full_like(w, 7.0), torch.full((3, Hkv, 300), -5, dtype=torch.int32, device="cuda")
    seen = torch.from_numpy(lk).int().cuda()
    cu_q, cu_k = _cu([0, 0, 0]), _cu(lk)
    kw = dict(decay=decay, out=out, seen=seen, born=born)
    if paged:
        pc = W.paginate(k, k, W.cu_from_lengths(lk), 3, 16, 300, seed=3)
        plan.key_weights_paged(q, pc.k_cache, pc.block_table, cu_q, cu_k, lse, w, **kw)
    else:
        plan.key_weights(q, k, cu_q, cu_k, lse, w, **kw)
    assert plan.check_error() == 0 and (born == -5).all()
    for b, n in enumerate(lk):
        assert torch.equal(out[b, :, :n], w[b, :, :n] * decay) and (out[b, :, n:] == 7.0).all()
    # a batch that claims queries the tensor does not have
    plan.key_weights(q, k, _cu([1, 0, 0]), cu_k, lse, w, out=out)
    assert plan.check_error() == vg.ATTN_DEV_ERR_OFFSETS


@pytest.mark.parametrize("Hq", [8, 260])
def test_key_weights_without_keys(Hq):
    plan = Plan(2, 64, Hq, 2, 64, 3)
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = _cu([0, 0])
    for T, lq in ((0, [0, 0]), (3, [3, 0])):
        q, lse = _bf16((T, Hq, 64), 1), torch.full((T, Hq), -math.inf, device="cuda")
        out = torch.full((2, 2, 64), 7.0, device="cuda")
        plan.key_weights(q, k, _cu(lq), cu, lse, out=out)
        assert plan.check_error() == 0 and (out == 7.0).all()
        assert (plan.key_weights(q, k, _cu(lq), cu, lse) == 0).all()
    # keys that the tensor does not have
    plan.key_weights(_bf16((1, Hq, 64), 1), k, _cu([1, 0]), _cu([5, 0]), torch.zeros(1, Hq, device="cuda"), out=out)
    assert plan.check_error() == vg.ATTN_DEV_ERR_OFFSETS and (out == 7.0).all()


# ---------------------------------------------------------------- infinities

@pytest.mark.parametrize("Hq,Hkv,max_q", [(8, 2, 1), (8, 2, 40), (64, 64, 300), (136, 1, 40)])
@pytest.mark.parametrize("paged", [False, True])
def test_infinite_sums_stay_infinite(Hq, Hkv, max_q, paged):
    """With normalisers far below the scores every weight that a visible row
    gives is infinite, and so are the sums; what nothing adds to is finite."""
    lk, lq = np.array([700, 300]), np.minimum(max_q, np.array([40, 300]))
    plan = Plan(2, 700, Hq, Hkv, 64, max_q)
    q, k = _bf16((int(lq.sum()), Hq, 64), 1), _bf16((1000, Hkv, 64), 2)
    lse = torch.full((q.shape[0], Hq), -200.0, device="cuda")
    w = torch.rand(2, Hkv, 700, generator=_gen(3), device="cuda")
    w[0, 0, 5] = math.inf
    cu_q, cu_k = _cu(lq), _cu(lk)
    if paged:
        pc = W.paginate(k, k, W.cu_from_lengths(lk), 2, 16, 700, seed=3)
        out = plan.key_weights_paged(q, pc.k_cache, pc.block_table, cu_q, cu_k, lse, w)
    else:
        out = plan.key_weights(q, k, cu_q, cu_k, lse, w)
    for b in range(2):
        assert (out[b, :, :lk[b]] == math.inf).all(), b
    lse[:] = math.inf                                            # and the other way: no row adds anything
    if paged:
        out = plan.key_weights_paged(q, pc.k_cache, pc.block_table, cu_q, cu_k, lse, w, out=out)
    else:
        out = plan.key_weights(q, k, cu_q, cu_k, lse, w, out=out)
    for b in range(2):
        old = int(lk[b] - lq[b])
        assert torch.equal(out[b, :, :old], w[b, :, :old]) and (out[b, :, old:lk[b]] == 0).all()
    assert plan.check_error() == 0


@pytest.mark.parametrize("Hq,Hkv,max_q", [(8, 2, 1), (8, 2, 40), (4, 1, 300), (136, 1, 40)])
def test_infinite_normalisers(Hq, Hkv, max_q):
    """lse = +inf (a key scored inf): exp(s - inf) is 0 for every finite score
    and NaN for the infinite one, in tiles that the mask cuts as in whole ones."""
    lk, lq = 700, max_q
    q = _bf16((lq, Hq, 64), 1).abs() + 0.1                       # every product with the bad keys is +inf
    k = _bf16((lk, Hkv, 64), 2)
    bad = [0, 300, lk - lq]                                       # seen by every query
    k[bad] = math.inf
    plan = Plan(1, lk, Hq, Hkv, 64, max_q)
    lse = torch.full((lq, Hq), math.inf, device="cuda")
    out = plan.key_weights(q, k, _cu([lq]), _cu([lk]), lse)[0]
    rest = torch.ones(lk, dtype=torch.bool, device="cuda")
    rest[bad] = False
    assert out[:, bad].isnan().all() and (out[:, rest] == 0).all()


# ------------------------------------------------------- overlaps and strides

def test_append_in_place_refuses_shared_rows():
    """q_out may be q itself only where no key or value is read from it: they
    would be read after the rotated queries were written."""
    plan, rope = Plan(1, 64, 4, 4, 64, 8), Rope(64, *rope_table(32))
    q, k = _bf16((8, 4, 64), 1), _bf16((8, 4, 64), 2)
    kc, vc = (torch.zeros(4, 16, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt, pos = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.arange(8, dtype=torch.int32, device="cuda")[None]
    cu = _cu([8])
    was = q.clone()
    for k_, v_ in ((q, k), (k, q), (q, q)):
        with pytest.raises(vg.AttnError):
            plan.append_paged(k_, v_, kc, vc, bt, cu, cu, q=q, pos=pos, rope=rope, q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(q, was) and not kc.any()
    plan.append_paged(q, k, kc, vc, bt, cu, cu, q=q, pos=pos, rope=rope)      # apart: allowed
    assert plan.append_paged(k, k, kc, vc, bt, cu, cu, q=q, pos=pos, rope=rope, q_out=q) is q
    assert torch.equal(q, rope.apply(was, pos)) and plan.check_error() == 0


def test_a_single_token_needs_no_token_stride():
    """One token of a buffer whose token stride no call could use (odd, or
    smaller than a token): the stride is never followed."""
    D, Hq, Hkv = 64, 4, 2
    plan, rope = Plan(1, 64, Hq, Hkv, D, 1), Rope(D, *rope_table(32))
    pos, cu = torch.tensor([[7]], dtype=torch.int32, device="cuda"), _cu([1])
    bt = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    for stride in (Hq * D + 4, 3, 0):
        q, k, v = (torch.as_strided(_bf16((1000,), i), (1, h, D), (stride, D, 1)) for i, h in ((1, Hq), (2, Hkv), (3, Hkv)))
        assert torch.equal(rope.apply(q, pos), rope.apply(q.contiguous(), pos))
        kc, vc = (torch.zeros(4, 16, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        qo = plan.append_paged(k, v, kc, vc, bt, cu, cu, q=q, pos=pos, rope=rope)
        assert torch.equal(qo, rope.apply(q, pos)) and torch.equal(kc[0, 0], rope.apply(k, pos)[0])
        assert torch.equal(vc[0, 0], v[0])
        lse = torch.zeros(1, Hq, device="cuda")
        w = plan.key_weights(qo, k, cu, cu, lse)
        assert torch.equal(w, plan.key_weights(qo, k.contiguous(), cu, cu, lse))
