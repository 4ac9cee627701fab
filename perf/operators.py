"""Cases and plain forms of the cache operators: rotary positions with several
axes, the paged append, accumulated attention weights, and eviction by them.

`run` computes each operator either in its plain form (torch operations in 32
or 64 bits) or, with `own` set, through the package's entry points.  The
lengths live on the device, as in a serving step; host code knows only the
plan's constants (largest lengths).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # 64 sequences of a decode step, query and key heads of one fused projection
        _rope("rope_decode", T=64, H=40, D=128, pairs=64, axes=3, layout="half", dtype="bf16", grad=False, extra=8),
        # the same heads over a training batch of packed image and text tokens
        _rope("rope_train", T=8192, H=72, D=128, pairs=64, axes=3, layout="half", dtype="bf16", grad=False, extra=8),
        # gradient of a vision tower's rotation: two axes, 80-wide heads, interleaved pairs, odd token count
        _rope("rope_grad", T=4097, H=16, D=80, pairs=40, axes=2, layout="interleaved", dtype="fp32", grad=True, extra=0),
        # one new token in each of 256 sequences
        _append("append_decode", B=256, Hq=64, Hkv=8, D=128, q_lo=1, q_hi=1, k_lo=1, k_hi=2048, page=64),
        # a prompt chunk of each of four sequences, behind what they hold already
        _append("append_chunk", B=4, Hq=32, Hkv=4, D=128, q_lo=512, q_hi=2048, k_lo=2048, k_hi=4096, page=16),
        # the smallest call: two short sequences
        _weights("weights_tiny", B=2, Hq=4, Hkv=1, D=64, q_lo=1, q_hi=1, k_lo=37, k_hi=100, page=0, decay=1.0),
        # a ragged decode batch, empty sequences among it
        _weights("weights_decode", B=64, Hq=32, Hkv=8, D=128, q_lo=1, q_hi=1, k_lo=0, k_hi=8192, page=0, decay=1.0),
        # several tokens a sequence (drafted ones, or short prompts) over a paged cache
        _weights("weights_short", B=32, Hq=32, Hkv=4, D=128, q_lo=1, q_hi=16, k_lo=1, k_hi=4096, page=64, decay=0.9),
        # a chunk of a long prompt over a paged cache
        _weights("weights_chunk", B=2, Hq=64, Hkv=8, D=128, q_lo=1025, q_hi=2048, k_lo=24576, k_hi=32768, page=64,
                 decay=1.0),
        # every step of a batch at its budget: a few tokens over
        _evict("evict_step", B=64, Hkv=8, D=128, k_lo=1000, k_hi=1088, keep=1024, sink=4, recent=256, page=64),
        # a long prompt cut down to a budget
        _evict("evict_prompt", B=1, Hkv=8, D=128, k_lo=32768, k_hi=32768, keep=2048, sink=4, recent=512, page=64),
        # ragged prompts, some under the budget, some empty
        _evict("evict_ragged", B=64, Hkv=8, D=128, k_lo=0, k_hi=8192, keep=1024, sink=4, recent=64, page=16),
    ]


def _rope(name, **kw):
    return {"name": name, "op": "rope", **kw}


def _append(name, **kw):
    return {"name": name, "op": "append", **kw}


def _weights(name, **kw):
    return {"name": name, "op": "weights", **kw}


def _evict(name, **kw):
    return {"name": name, "op": "evict", **kw}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "weights", "weights", "evict", "evict"])
    if op == "rope":
        D, pairs = rng.choice([(128, 64), (128, 64), (64, 32), (80, 40), (128, 32), (72, 36), (64, 16)])
        return _rope("", T=_log_int(rng, 1, 16384), H=_log_int(rng, 1, 72), D=D, pairs=pairs, axes=rng.randint(1, 4),
                     layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     grad=rng.random() < 0.4, extra=rng.choice([0, 0, 1, 8]))
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "append":
        G = rng.choice([1, 2, 4, 5, 7, 8])
        B = _log_int(rng, 1, 128)
        q_hi = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, 4096 // B))
        k_hi = max(q_hi, _log_int(rng, 16, max(16, 131072 // B)))
        return _append("", B=B, Hq=G * Hkv, Hkv=Hkv, D=D, q_lo=rng.choice([0, 1, q_hi]) if q_hi > 1 else 1, q_hi=q_hi,
                       k_lo=q_hi, k_hi=k_hi, page=page)
    if op == "weights":
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        B = _log_int(rng, 1, 64)
        kind = rng.choice(["decode", "short", "chunk"])
        if kind == "decode":
            q_lo = q_hi = 1
            k_hi = _log_int(rng, 16, min(65536, 262144 // B))
        elif kind == "short":
            q_lo, q_hi = 1, rng.randint(2, 16)
            k_hi = max(q_hi, _log_int(rng, 16, min(16384, 131072 // B)))
        else:
            B = min(B, 8)
            q_hi = _log_int(rng, 17, 2048 // B)
            q_lo = rng.randint(0, q_hi)
            k_hi = max(q_hi, _log_int(rng, 64, 8192))
        k_lo = rng.choice([0, k_hi // 2, k_hi])
        return _weights("", B=B, Hq=G * Hkv, Hkv=Hkv, D=D, q_lo=q_lo, q_hi=q_hi, k_lo=k_lo, k_hi=k_hi,
                        page=rng.choice([0, page]), decay=rng.choice([0.0, 0.9, 1.0]))
    B = _log_int(rng, 1, 64)
    k_hi = _log_int(rng, 32, min(65536, 262144 // B))
    keep = _log_int(rng, 1, k_hi)
    sink = rng.choice([0, 1, 4])
    return _evict("", B=B, Hkv=Hkv, D=D, k_lo=rng.choice([0, k_hi // 2, k_hi]), k_hi=k_hi, keep=keep, sink=sink,
                  recent=rng.randint(0, keep // 2), page=page)


# ------------------------------------------------------------------ inputs

def _frequencies(pairs, axes):
    """Frequencies 1e6^(-i / pairs) in contiguous sections, the first axis
    taking what the others leave over (two-axis tables restart at each axis)."""
    part = pairs // axes
    sections = [pairs - part * (axes - 1)] + [part] * (axes - 1)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    if axes == 2:
        freq = [1e4 ** (-i / n) for n in sections for i in range(n)]
    else:
        freq = [1e6 ** (-i / pairs) for i in range(pairs)]
    return freq, axis


def _positions(g, axes, T, dev):
    """Text runs (all axes alike) and image patches (rows and columns of their
    own), far into a long context."""
    start = torch.randint(0, 1 << 20, (1,), generator=g, device=dev)
    t = start + torch.arange(T, device=dev)
    pos = t.expand(axes, T).clone()
    image = torch.rand(T, generator=g, device=dev) < 0.5
    if axes > 1:
        grid = torch.randint(0, 64, (axes - 1, T), generator=g, device=dev)
        pos[1:] = torch.where(image, start + grid, pos[1:])
    return pos.to(torch.int32)


def _lengths(case, seed):
    rng = np.random.default_rng(seed)
    lq = rng.integers(case.get("q_lo", 0), case.get("q_hi", 0), case["B"], endpoint=True)
    lk = rng.integers(case["k_lo"], case["k_hi"], case["B"], endpoint=True)
    return lq, lk


def _cu(lens, dev):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(dev)


def _table(lk, k_hi, page, seed, dev):
    """Block table of shuffled pages for lengths `lk`, out of a cache that has
    room for the largest ones; entries past a sequence's pages hold -1."""
    n = (lk + page - 1) // page
    total = len(lk) * ((k_hi + page - 1) // page) + 2
    phys = np.random.default_rng(seed + 1).permutation(total)
    bt = np.full((len(lk), max(1, (k_hi + page - 1) // page)), -1, np.int32)
    at = 0
    for b, c in enumerate(n):
        bt[b, :c] = phys[at:at + c]
        at += c
    return torch.from_numpy(bt).to(dev), total


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        base = torch.randn(T, H + case["extra"], D, generator=g, device=dev).to(DTYPES[case["dtype"]])
        s["x"] = base[:, :H]                        # the heads to rotate of a wider projection
        s["out"] = torch.empty(T, H, D, dtype=base.dtype, device=dev)
        s["pos"] = _positions(g, case["axes"], T, dev)
        freq, axis = _frequencies(case["pairs"], case["axes"])
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor(axis, device=dev)
        if own:
            from varlen_gqa_split_b200 import Rope
            s["rope"] = Rope(D, freq, axis, layout=case["layout"], scale=1.0)
        return s
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    lq, lk = _lengths(case, seed)
    if case["op"] == "append":
        lk = np.maximum(lk, lq)
    s["cu_k"] = _cu(lk, dev)
    s_max = max(1, case["k_hi"])

    def bf16(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)

    if case["op"] in ("append", "weights"):
        Hq = case["Hq"]
        Tq = B * max(1, case["q_hi"])                # rows behind the last sequence's stay unused
        s["cu_q"] = _cu(lq, dev)
        s["max_q"] = max(1, case["q_hi"])
        if own:
            from varlen_gqa_split_b200 import Plan
            s["plan"] = Plan(B, s_max, Hq, Hkv, D, s["max_q"])
    if case["op"] == "append":
        s["bt"], pages = _table(lk, s_max, case["page"], seed, dev)
        qkv = bf16(Tq, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_out"] = torch.zeros(Tq, Hq, D, dtype=torch.bfloat16, device=dev)
        s["kc"], s["vc"] = (bf16(pages, case["page"], Hkv, D) for _ in range(2))
        s["pos"] = _positions(g, 3, Tq, dev)
        freq, axis = _frequencies(D // 2, 3)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor(axis, device=dev)
        if own:
            from varlen_gqa_split_b200 import Rope
            s["rope"] = Rope(D, freq, axis, layout="half", scale=1.0)
    elif case["op"] == "weights":
        s["q"] = bf16(Tq, Hq, D)
        if case["page"]:
            s["bt"], pages = _table(lk, s_max, case["page"], seed, dev)
            s["k"] = bf16(pages, case["page"], Hkv, D)
        else:
            s["k"] = bf16(max(1, int(lk.sum())), Hkv, D)
        # the normalisers that attention over such keys returns: scores of a
        # query are normal with variance |q|^2 / D
        b = np.repeat(np.arange(B), lq)
        qi = np.arange(len(b)) - np.repeat(np.cumsum(lq) - lq, lq)
        n = np.clip(lk[b] - lq[b] + qi + 1, 0, lk[b])
        seen_keys = torch.zeros(Tq, dtype=torch.float32, device=dev)
        seen_keys[:len(n)] = torch.from_numpy(n.astype(np.float32)).to(dev)
        s["lse"] = torch.log(seen_keys)[:, None] + s["q"].float().square().sum(-1) / (2 * D)
        s["w_in"] = torch.rand(B, Hkv, s_max, generator=g, device=dev) * 4
        s["w_out"] = torch.zeros(B, Hkv, s_max, device=dev)
        s["born"] = torch.zeros(B, Hkv, s_max, dtype=torch.int32, device=dev)
        s["seen"] = (s["cu_k"][1:] - s["cu_k"][:-1]) + torch.randint(0, 1000, (B,), generator=g, device=dev,
                                                                     dtype=torch.int32)
    else:
        s["bt"], pages = _table(lk, s_max, case["page"], seed, dev)
        s["kc"], s["vc"] = (bf16(pages, case["page"], Hkv, D) for _ in range(2))
        # weights with a heavy tail; a twentieth of the keys was never looked at
        w = torch.rand(B, Hkv, s_max, generator=g, device=dev).log().neg() ** 3
        w[torch.rand(B, Hkv, s_max, generator=g, device=dev) < 0.05] = 0.0
        s["w"] = w
        # births of keys that survived earlier evictions
        gaps = torch.randint(1, 3, (B, Hkv, s_max), generator=g, device=dev)
        s["born"] = (torch.cumsum(gaps, -1) - 1).to(torch.int32)
        last = (s["cu_k"][1:] - s["cu_k"][:-1]).long().clamp(min=1) - 1
        s["seen"] = s["born"].gather(2, last[:, None, None].expand(B, Hkv, 1)).amax((1, 2)).to(torch.int32) + 1
        s["keep"] = torch.full((B,), case["keep"], dtype=torch.int32, device=dev)
        s["w_out"] = torch.zeros(B, Hkv, s_max, device=dev)
        s["born_out"] = torch.zeros(B, Hkv, s_max, dtype=torch.int32, device=dev)
        s["cu_out"] = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        if own:
            from varlen_gqa_split_b200 import Plan
            s["plan"] = Plan(B, s_max, Hkv, Hkv, D, 1)
    return s


# ------------------------------------------------------------- plain forms

def _rotate(x, pos, freq, axis, layout, grad, out):
    n, D = freq.numel(), x.shape[-1]
    angle = pos.double()[axis].t() * freq                       # [T, n]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if grad:
        sin = -sin
    xf = x.float()
    if layout == "half":
        u, w = xf[..., :n], xf[..., n:2 * n]
        out[..., :n] = u * cos - w * sin
        out[..., n:2 * n] = u * sin + w * cos
    else:
        u, w = xf[..., 0:2 * n:2], xf[..., 1:2 * n:2]
        out[..., 0:2 * n:2] = u * cos - w * sin
        out[..., 1:2 * n:2] = u * sin + w * cos
    if 2 * n < D:
        out[..., 2 * n:] = x[..., 2 * n:]
    return out


def _plain_rope(s):
    c = s["case"]
    return _rotate(s["x"], s["pos"], s["freq"], s["axis"], c["layout"], c["grad"], s["out"])


def _tokens(cu_q, Tq):
    """Sequence and place within it of each packed query token, and whether it
    belongs to one."""
    t = torch.arange(Tq, device=cu_q.device)
    b = torch.searchsorted(cu_q[1:].contiguous(), t.to(torch.int32), right=True).clamp(max=cu_q.numel() - 2)
    return b, t - cu_q[b], t < cu_q[-1]


def _plain_append(s):
    c = s["case"]
    cu_q, cu_k, page = s["cu_q"], s["cu_k"], c["page"]
    Tq = s["q"].shape[0]
    b, qi, live = _tokens(cu_q, Tq)
    j = (cu_k[b + 1] - cu_k[b]) - (cu_q[b + 1] - cu_q[b]) + qi
    q = _rotate(s["q"], s["pos"], s["freq"], s["axis"], "half", False, torch.empty_like(s["q_out"]))
    k = _rotate(s["k"], s["pos"], s["freq"], s["axis"], "half", False, torch.empty_like(s["k"]))
    s["q_out"][live] = q[live]
    row = s["bt"][b[live], j[live] // page].long() * page + j[live] % page
    s["kc"].view(-1, c["Hkv"], c["D"])[row] = k[live]
    s["vc"].view(-1, c["Hkv"], c["D"])[row] = s["v"][live]
    return s["q_out"], s["kc"], s["vc"]


def _plain_weights(s):
    c = s["case"]
    B, Hkv, G, D = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    cu_q, cu_k, max_q, s_max = s["cu_q"].long(), s["cu_k"].long(), s["max_q"], s["w_in"].shape[-1]
    Lq, Lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    qi = torch.arange(max_q, device=cu_q.device)
    j = torch.arange(s_max, device=cu_q.device)
    q_tok = torch.where(qi < Lq[:, None], cu_q[:-1, None] + qi, 0)                    # [B, max_q]
    held = j < Lk[:, None]                                                            # [B, s_max]
    if c["page"]:
        page = torch.where(held, s["bt"][:, :].long().gather(1, (j // c["page"]).expand(B, -1)), 0)
        k_tok = page * c["page"] + (j % c["page"])
    else:
        k_tok = torch.where(held, cu_k[:-1, None] + j, 0)
    n = (Lk[:, None] - Lq[:, None] + qi + 1)                                          # keys that row qi sees
    sees = (j < n[..., None]) & (qi < Lq[:, None])[..., None] & held[:, None]         # [B, max_q, s_max]
    old = held & (j < (Lk - Lq)[:, None])
    k_all = s["k"].reshape(-1, Hkv, D)
    start = torch.where(old[:, None], c["decay"] * s["w_in"], 0.0) if c["decay"] else None
    for h in range(Hkv):
        qh = s["q"][:, h * G:(h + 1) * G][q_tok].float()                              # [B, max_q, G, D]
        kh = k_all[:, h][k_tok].float()                                               # [B, s_max, D]
        sc = torch.matmul(qh.flatten(1, 2), kh.transpose(1, 2)).view(B, max_q, G, s_max)
        sc.mul_(1 / math.sqrt(D)).sub_(s["lse"][:, h * G:(h + 1) * G][q_tok][..., None]).exp_()
        w = sc.masked_fill_(~sees[:, :, None], 0.0).sum((1, 2))
        if start is not None:
            w += start[:, h]
        s["w_out"][:, h] = torch.where(held, w, s["w_out"][:, h])
    new = held & (j >= (Lk - Lq)[:, None])
    born = (s["seen"].long() - Lk)[:, None] + j
    s["born"].copy_(torch.where(new[:, None], born[:, None], s["born"]))
    return s["w_out"], s["born"]


def _plain_evict(s):
    c = s["case"]
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    w, born = s["w"], s["born"]
    j = torch.arange(w.shape[-1], device=w.device)
    Lk = (s["cu_k"][1:] - s["cu_k"][:-1]).long()
    keep = torch.minimum(Lk, s["keep"].long().clamp(min=0))
    fixed = (born < c["sink"]) | (born >= s["seen"][:, None, None] - c["recent"])
    rank = torch.where(fixed, math.inf, torch.where(w.isnan(), -math.inf, w))
    rank = torch.where((j < Lk[:, None])[:, None], rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(rank, dtype=torch.bool)
    kept.scatter_(2, order, (j < keep[:, None])[:, None].expand(B, Hkv, -1))
    low = (j < keep[:, None])[:, None]
    holes, movers = (low & ~kept).nonzero(), (kept & ~low).nonzero()    # both in order of (b, h, j)
    src = j.expand(B, Hkv, -1).clone()
    src[tuple(holes.unbind(1))] = movers[:, 2]
    s["w_out"].copy_(torch.where(low, w.gather(2, src), s["w_out"]))
    s["born_out"].copy_(torch.where(low, born.gather(2, src), s["born_out"]))
    b, h, to, at = holes[:, 0], holes[:, 1], holes[:, 2], movers[:, 2]
    for cache in (s["kc"], s["vc"]):
        cache[s["bt"][b, to // page].long(), to % page, h] = cache[s["bt"][b, at // page].long(), at % page, h]
    s["cu_out"][1:] = torch.cumsum(keep, 0)
    return s["w_out"], s["born_out"], s["cu_out"], s["kc"], s["vc"]


def run(s):
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "weights": _plain_weights,
                "evict": _plain_evict}[c["op"]](s)
    if c["op"] == "rope":
        return s["rope"].apply(s["x"], s["pos"], s["out"], grad=c["grad"])
    if c["op"] == "append":
        s["plan"].append_paged(s["k"], s["v"], s["kc"], s["vc"], s["bt"], s["cu_q"], s["cu_k"], q=s["q"],
                               pos=s["pos"], rope=s["rope"], q_out=s["q_out"])
        return s["q_out"], s["kc"], s["vc"]
    if c["op"] == "weights":
        kw = dict(decay=c["decay"], out=s["w_out"], seen=s["seen"], born=s["born"])
        if c["page"]:
            s["plan"].key_weights_paged(s["q"], s["k"], s["bt"], s["cu_q"], s["cu_k"], s["lse"], s["w_in"], **kw)
        else:
            s["plan"].key_weights(s["q"], s["k"], s["cu_q"], s["cu_k"], s["lse"], s["w_in"], **kw)
        return s["w_out"], s["born"]
    s["plan"].evict_paged(s["w"], s["born"], s["seen"], s["keep"], s["kc"], s["vc"], s["bt"], s["cu_k"],
                          sink=c["sink"], recent=c["recent"], weight_out=s["w_out"], born_out=s["born_out"],
                          cu_k_out=s["cu_out"])
    return s["w_out"], s["born_out"], s["cu_out"], s["kc"], s["vc"]


# -------------------------------------------------------------------- work

def _mean(lo, hi):
    return (lo + hi) / 2


def work(case):
    """Bytes that have to move and operations that have to be done, at the
    mean lengths of the case's ranges."""
    D = case["D"]
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        el = case["T"] * case["H"] * D
        return {"bytes": 2 * el * size + 4 * case["axes"] * case["T"], "flops": 3 * el}
    B, Hkv = case["B"], case["Hkv"]
    if case["op"] == "append":
        tok = B * _mean(case["q_lo"], case["q_hi"])
        return {"bytes": tok * (4 * (case["Hq"] + 2 * Hkv) * D + 12) + 8 * B, "flops": tok * 3 * (case["Hq"] + Hkv) * D}
    lk = _mean(case["k_lo"], case["k_hi"])
    if case["op"] == "weights":
        lq = _mean(case["q_lo"], case["q_hi"])
        seen = lq * max(lk - lq / 2, lk / 2)               # visible (query, key) pairs
        w = 4 * Hkv * lk * (2 if case["decay"] else 1)
        return {"bytes": B * (2 * Hkv * D * lk + lq * case["Hq"] * (2 * D + 4) + w), "flops": 2 * D * case["Hq"] * B * seen}
    c = min(lk, case["keep"])
    moved = c * (1 - c / lk) if lk else 0                  # kept keys that lie at c or above, were they spread evenly
    return {"bytes": B * Hkv * (8 * lk + 8 * c + 8 * D * moved), "flops": B * Hkv * lk}


# ------------------------------------------------------------ in 64 bits

def _exact_rotate(x, pos, freq, axis, layout, grad):
    """Rotation as a product of complex numbers in 64 bits."""
    n = len(freq)
    y = x.double().clone()
    f = torch.tensor(freq, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(f).expand(pos.shape[1], n), pos[axis].double().T * f)
    if grad:
        turn = turn.conj()
    at = torch.arange(n, device=x.device)
    u, w = (at, at + n) if layout == "half" else (2 * at, 2 * at + 1)
    z = torch.complex(y[..., u], y[..., w]) * turn[:, None]
    y[..., u], y[..., w] = z.real, z.imag
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        freq, axis = _frequencies(case["pairs"], case["axes"])
        return _exact_rotate(s["x"], s["pos"], freq, axis, case["layout"], case["grad"])
    lq, lk = _lengths(case, seed)
    if case["op"] == "append":
        lk = np.maximum(lk, lq)
        freq, axis = _frequencies(case["D"] // 2, 3)
        q, k = (_exact_rotate(s[x], s["pos"], freq, axis, "half", False) for x in ("q", "k"))
        kc, vc, bt, at = s["kc"].double(), s["vc"].double(), s["bt"].cpu().numpy(), 0
        q_out = torch.zeros_like(q)
        q_out[:int(lq.sum())] = q[:int(lq.sum())]
        for b in range(case["B"]):
            j = np.arange(lk[b] - lq[b], lk[b])
            pages = torch.from_numpy(bt[b][j // case["page"]].astype(np.int64)).to(q.device)
            slots = torch.from_numpy(j % case["page"]).to(q.device)
            kc[pages, slots], vc[pages, slots] = k[at:at + lq[b]], s["v"][at:at + lq[b]].double()
            at += int(lq[b])
        return q_out, kc, vc
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "weights":
        G, out, born = case["Hq"] // Hkv, s["w_out"].double(), s["born"].clone()
        q0 = np.cumsum(lq) - lq
        k0 = np.cumsum(lk) - lk
        for b in range(case["B"]):
            Lq, Lk = int(lq[b]), int(lk[b])
            j = torch.arange(Lk, device=out.device)
            if case["page"]:
                keys = s["k"][s["bt"][b, j // case["page"]].long(), j % case["page"]]
            else:
                keys = s["k"][k0[b]:k0[b] + Lk]
            rows = torch.arange(Lq, device=out.device)
            hidden = j[None] > (Lk - Lq + rows)[:, None]
            out[b, :, :Lk] = 0.0
            old = max(0, Lk - Lq)
            if case["decay"]:
                out[b, :, :old] = case["decay"] * s["w_in"][b, :, :old].double()
            for h in range(case["Hq"]):
                score = s["q"][q0[b]:q0[b] + Lq, h].double() @ keys[:, h // G].double().T / math.sqrt(D)
                p = torch.exp(score - s["lse"][q0[b]:q0[b] + Lq, h, None].double())
                out[b, h // G, :Lk] += p.masked_fill(hidden, 0.0).sum(0)
            born[b, :, old:Lk] = int(s["seen"][b]) - Lk + j[old:].int()
        return out, born
    # eviction: one head at a time, on the host
    if case["B"] * Hkv * case["k_hi"] > 1 << 23:
        return None
    w, births, seen, page = s["w"].cpu().numpy(), s["born"].cpu().numpy(), s["seen"].cpu().numpy(), case["page"]
    w_out, b_out = np.zeros(w.shape), np.zeros(w.shape, np.int32)
    bt, cu, pairs = s["bt"].cpu().numpy(), [0], []
    for b in range(case["B"]):
        n = int(lk[b])
        c = min(n, case["keep"])
        cu.append(cu[-1] + c)
        for h in range(Hkv):
            r = np.where((births[b, h, :n] < case["sink"]) | (births[b, h, :n] >= seen[b] - case["recent"]), np.inf,
                         w[b, h, :n])
            kept = np.sort(np.lexsort((np.arange(n), -r))[:c])
            move = kept[kept >= c]
            into = np.setdiff1d(np.arange(c), kept)
            src = np.arange(c)
            src[into] = move
            w_out[b, h, :c], b_out[b, h, :c] = w[b, h, src], births[b, h, src]
            pairs.append(np.stack([bt[b, into // page], into % page, bt[b, move // page], move % page,
                                   np.full(len(into), h)], 1).astype(np.int64))
    at = torch.from_numpy(np.concatenate(pairs)).to(s["kc"].device)
    dev = s["kc"].device
    caches = []
    for cache in (s["kc"], s["vc"]):
        new = cache.double()
        new[at[:, 0], at[:, 1], at[:, 4]] = cache[at[:, 2], at[:, 3], at[:, 4]].double()
        caches.append(new)
    return (torch.from_numpy(w_out).to(dev), torch.from_numpy(b_out).to(dev),
            torch.tensor(cu, dtype=torch.int32, device=dev), *caches)
