"""Kernels launched as programmatic dependents: each waits for the kernel
before it (read from the sources, CPU), and a call that follows attention
reads what attention wrote (needs a B200)."""
import glob
import os
import re

import numpy as np
import pytest
import torch

import workloads as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _kernels(text):
    """(name, body) of every __global__ function of a source."""
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\(", text):
        if m.group(1) in ("__launch_bounds__", "__grid_constant__"):
            m2 = re.compile(r"(\w+)\s*\((?=[^()]*(?:\([^()]*\)[^()]*)*\)\s*\{)").search(text, m.end() + 1)
            name, at = m2.group(1), text.index("{", m2.end())
        else:
            name, at = m.group(1), text.index("{", m.end())
        depth, i = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        yield name, text[at:i]


def test_every_programmatic_dependent_waits():
    """A grid launched as a programmatic dependent that never waits can
    complete before the grid it depends on, and the next one in the stream,
    which waits for its direct predecessor alone, would then start too early."""
    seen = []
    for path in sorted(glob.glob(os.path.join(ROOT, "varlen_gqa_split_b200", "csrc", "*.cu"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        if "ProgrammaticStreamSerialization" not in text and "launch_dependent(" not in text:
            continue
        for name, body in _kernels(text):
            assert "griddepcontrol.wait" in body or "dependent_start(" in body, f"{os.path.basename(path)}: {name}"
            seen.append(name)
    assert {"split_mma_kernel", "split_tc_kernel", "combine_slots_kernel", "rope_kernel", "append_kernel",
            "key_weights_tc_kernel", "evict_kernel"} <= set(seen)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(shape, seed):
    return torch.randn(shape, generator=_gen(seed), device="cuda").to(torch.bfloat16)


# units and blocks coincide (148 equal sequences of one KV head), whole units
# with a few cut ones, and the same on the tcgen05 path with its combine kernel
@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,lq,lens", [(148, 4, 1, 1, "equal"), (37, 16, 4, 1, "equal"), (150, 4, 1, 1, "mixed"),
                                              (148, 8, 1, 4, "equal"), (75, 16, 2, 3, "mixed")])
@pytest.mark.parametrize("paged", [False, True])
def test_calls_behind_attention_read_its_results(B, Hq, Hkv, lq, lens, paged):
    """attention -> key weights -> eviction without anything between them gives
    what the same calls give with a synchronisation after each.  The outputs'
    buffers are reused with other inputs, so an early read sees old rows."""
    from varlen_gqa_split_b200 import Plan
    D, page, n = 64, 64, 3
    lk = np.full(B, 1536) if lens == "equal" else 64 + 24 * (np.arange(B) * 37 % 61)
    s_max = int(lk.max())
    plan = Plan(B, s_max, Hq, Hkv, D, lq, deterministic=1)
    cu_q = torch.from_numpy(W.cu_from_lengths(np.full(B, lq))).cuda()
    cu_k = torch.from_numpy(W.cu_from_lengths(lk)).cuda()
    seen = torch.from_numpy(lk).int().cuda()
    keep = torch.from_numpy(np.maximum(lk - 8, 1)).int().cuda()
    T, Tk = B * lq, int(lk.sum())
    qs = [_bf16((T, Hq, D), 10 + i) for i in range(n)]
    keys = [(_bf16((Tk, Hkv, D), 20 + i), _bf16((Tk, Hkv, D), 30 + i)) for i in range(n)]
    caches = [W.paginate(k, v, W.cu_from_lengths(lk), B, page, s_max, seed=i) for i, (k, v) in enumerate(keys)]
    born = torch.arange(s_max, dtype=torch.int32, device="cuda").expand(B, Hkv, s_max).contiguous()
    out, lse = torch.empty_like(qs[0]), torch.empty(T, Hq, device="cuda")
    w, wo, bo = (torch.zeros(B, Hkv, s_max, device="cuda") for _ in range(3))
    bo = torch.zeros_like(born)
    cu_new = torch.zeros_like(cu_k)

    def step(i, wait):
        pc = caches[i]
        kc, vc = pc.k_cache.clone(), pc.v_cache.clone()
        torch.cuda.synchronize()
        if paged:
            plan.run_paged(qs[i], kc, vc, pc.block_table, cu_q, cu_k, out, lse)
        else:
            plan.run(qs[i], *keys[i], cu_q, cu_k, out, lse)
        wait()
        if paged:
            plan.key_weights_paged(qs[i], kc, pc.block_table, cu_q, cu_k, lse, out=w)
        else:
            plan.key_weights(qs[i], keys[i][0], cu_q, cu_k, lse, out=w)
        wait()
        plan.evict_paged(w, born, seen, keep, kc, vc, pc.block_table, cu_k, weight_out=wo, born_out=bo, cu_k_out=cu_new)
        torch.cuda.synchronize()
        return [t.clone() for t in (out, lse, w, wo, bo, cu_new)] + [kc, vc]

    refs = [step(i, torch.cuda.synchronize) for i in range(n)]
    assert not torch.equal(refs[0][1], refs[1][1])
    for rep in range(4):
        for i in range(n):
            for got, want in zip(step(i, lambda: None), refs[i]):
                assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), (rep, i)
    assert plan.check_error() == 0


def test_programmatic_dependents_read_by_plain_loads():
    """Read-only loads (ld.global.nc) may be moved ahead of the wait and promise
    that nothing is written while the kernel lives, and a programmatic dependent
    lives while its predecessor still writes."""
    csrc = os.path.join(ROOT, "varlen_gqa_split_b200", "csrc")
    for path in sorted(glob.glob(os.path.join(csrc, "*.cu")) + glob.glob(os.path.join(csrc, "*.cuh"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        if path.endswith(".cuh") or "ProgrammaticStreamSerialization" in text or "launch_dependent(" in text:
            assert not re.search(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc\b|__restrict__", text), os.path.basename(path)


def test_launch_rules_ask_the_device_for_its_sms():
    """No rule holds the SM count of one card as a number."""
    csrc = os.path.join(ROOT, "varlen_gqa_split_b200", "csrc")
    for path in sorted(glob.glob(os.path.join(csrc, "*.*"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        assert not re.search(r"\b148\b", text), os.path.basename(path)
