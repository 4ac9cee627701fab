"""Calls on a stream given by the caller: what the binding makes for the call
(results not passed in) is made on that stream."""
import contextlib

import numpy as np
import pytest
import torch

import varlen_gqa_split_b200 as vg
import workloads as W
from varlen_gqa_split_b200 import Plan, Rope, _binding, rope_table


class _Stream:
    cuda_stream = 7


@pytest.fixture
def host(monkeypatch):
    """The binding over a marshalling module that records and launches nothing;
    `made` lists, for every tensor it makes, whether the given stream was current."""
    from varlen_gqa_split_b200 import build
    build.build()
    vg.lib()
    current, made = [None], []

    @contextlib.contextmanager
    def on(s):
        was, current[0] = current[0], s
        try:
            yield
        finally:
            current[0] = was

    def watch(make):
        def f(*args, **kw):
            made.append(current[0] is not None and current[0].cuda_stream == 7)
            return make(*args, **kw)
        return f

    class Marshal:
        def __getattr__(self, name):
            return lambda *args: 0

    monkeypatch.setattr(_binding, "_marshal", Marshal())
    monkeypatch.setattr(_binding, "_raw_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr: _Stream())
    for name in ("zeros", "empty", "empty_like"):
        monkeypatch.setattr(torch, name, watch(getattr(torch, name)))
    plan = Plan.__new__(Plan)
    plan._h, plan._args, plan.device = object(), (), 0
    plan.info = dict(B_max=2, s_max=8, Hq=4, Hkv=2, D=64)
    yield plan, made
    plan._h = None


def test_results_are_made_on_the_given_stream(host):
    plan, made = host
    q, k = torch.ones(3, 4, 64, dtype=torch.bfloat16), torch.ones(3, 2, 64, dtype=torch.bfloat16)
    cu, led = torch.zeros(3, dtype=torch.int32), torch.ones(2, 2, 8)
    lse, cache, bt = torch.ones(3, 4), torch.ones(4, 8, 2, 64), torch.ones(2, 4, dtype=torch.int32)
    rope = Rope(64, *rope_table(32))
    for i, call in enumerate([lambda s: rope.apply(q, cu[None], stream=s),
                              lambda s: plan.append_paged(k, k, cache, cache, bt, cu, cu, q=q, stream=s),
                              lambda s: plan.key_weights(q, k, cu, cu, lse, stream=s),
                              lambda s: plan.key_weights_paged(q, cache, bt, cu, cu, lse, stream=s),
                              lambda s: plan.evict_paged(led, led.int(), cu, cu, cache, cache, bt, cu, stream=s)]):
        made.clear()
        call(_Stream())
        assert made == [True], i
    made.clear()
    plan.key_weights(q, k, cu, cu, lse, out=led, stream=_Stream())
    assert made == []                                          # nothing is made for a caller who passes it


@pytest.mark.gpu
def test_fills_and_kernels_share_the_given_stream():
    """With the current stream busy for a while, results that the binding makes
    for a call on another stream are complete once that stream is."""
    B, Hq, Hkv, D, s_max, page = 3, 8, 2, 64, 400, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    lk = np.array([400, 17, 230])
    T = 3
    q = torch.randn(T, Hq, D, generator=g, device="cuda").bfloat16()
    k = torch.randn(int(lk.sum()), Hkv, D, generator=g, device="cuda").bfloat16()
    new = torch.randn(T, Hkv, D, generator=g, device="cuda").bfloat16()
    cu_q, cu_k = (torch.from_numpy(W.cu_from_lengths(x)).cuda() for x in ([1, 1, 1], lk))
    pc = W.paginate(k, k, W.cu_from_lengths(lk), B, page, s_max, seed=1)
    plan, rope = Plan(B, s_max, Hq, Hkv, D, 1, deterministic=1), Rope(D, *rope_table(32))
    pos = torch.tensor([[399, 16, 229]], dtype=torch.int32, device="cuda")
    seen = torch.from_numpy(lk).int().cuda()
    keep = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    born = torch.arange(s_max, dtype=torch.int32, device="cuda").expand(B, Hkv, s_max).contiguous()

    def calls(s):
        kc, vc = pc.k_cache.clone(), pc.v_cache.clone()
        torch.cuda.synchronize()
        if s is not None:
            torch.cuda._sleep(20_000_000)                      # the current stream: some 10 ms
        r = rope.apply(q, pos, stream=s)
        qo = plan.append_paged(new, new, kc, vc, pc.block_table, cu_q, cu_k, q=q, pos=pos, rope=rope, stream=s)
        o, lse = plan.run_paged(qo, kc, vc, pc.block_table, cu_q, cu_k, stream=s)
        wp = plan.key_weights_paged(qo, kc, pc.block_table, cu_q, cu_k, lse, stream=s)
        w = plan.key_weights(qo, k, cu_q, cu_k, lse, stream=s)
        _, _, cu = plan.evict_paged(wp, born, seen, keep, kc, vc, pc.block_table, cu_k, weight_out=wo, born_out=bo,
                                    stream=s)
        (s or torch.cuda.current_stream()).synchronize()
        with torch.cuda.stream(s):
            return [t.cpu() for t in (r, qo, o, lse, wp, w, wo, bo, cu)]

    wo, bo = torch.zeros(B, Hkv, s_max, device="cuda"), torch.zeros_like(born)
    want = calls(None)
    side = torch.cuda.Stream()
    wo.zero_()
    bo.zero_()
    torch.cuda.synchronize()
    got = calls(side)
    torch.cuda.synchronize()
    assert plan.check_error() == 0
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i
    for b in range(B):
        assert (got[4][b, :, lk[b]:] == 0).all() and (got[5][b, :, lk[b]:] == 0).all()


@pytest.mark.gpu
def test_dropped_results_stay_with_their_stream():
    """The memory of a result that was made for a call on another stream is not
    handed to the current stream while that call is still queued."""
    rope = Rope(64, *rope_table(32))
    x = torch.ones(1000, 8, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, 1000, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    out = rope.apply(x, pos, stream=side)
    at = out.data_ptr()
    del out
    y = [torch.empty_like(x) for _ in range(4)]
    assert at not in [t.data_ptr() for t in y]
    torch.cuda.synchronize()
