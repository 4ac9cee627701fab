"""Operators on the cache against plain 64-bit implementations (needs a B200):
rotary positions with several axes, the paged append, accumulated attention
weights, eviction, and a serving loop of all of them.

Unused cache slots, ledger entries past a sequence and rows past the last
sequence hold NaN or a sentinel, so whatever is read or written out of place
shows.
"""
import math

import numpy as np
import pytest
import torch

import varlen_gqa_split_b200 as vg
import workloads as W
from varlen_gqa_split_b200 import Plan, Rope, rope_table

pytestmark = pytest.mark.gpu

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step
SENTINEL = 12345.0


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


def _cu(lens, entries=None):
    return torch.from_numpy(W.cu_from_lengths(lens, entries)).cuda()


# ------------------------------------------------------------------ rotation

def _rotate64(x, pos, freqs, axes, layout, scale=1.0, grad=False):
    """The rotation in 64 bits, and the magnitude |scale| (|u| + |w|) that its
    rounding errors scale with."""
    n = len(freqs)
    y, mag = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    theta = pos.double()[torch.tensor(axes, device=x.device)].t() * torch.tensor(freqs, dtype=torch.float64,
                                                                                  device=x.device)
    c, s = torch.cos(theta)[:, None] * scale, torch.sin(theta)[:, None] * scale * (-1 if grad else 1)
    at = torch.arange(n, device=x.device)
    u, w = (at, at + n) if layout == "half" else (2 * at, 2 * at + 1)
    xu, xw = x[..., u].double(), x[..., w].double()
    y[..., u], y[..., w] = xu * c - xw * s, xu * s + xw * c
    mag[..., u] = mag[..., w] = abs(scale) * (xu.abs() + xw.abs())
    return y, mag


def _check_rotation(out, ref, mag, ref_angle=0.0):
    """One rounding to the type; before it the angle is off by at most pi 2^-25
    rad, cosine and sine (float, two units in the last place) by 2^-22, and
    two products and a sum add 3 * 2^-24, all relative to |u| + |w|; so is what
    the reference's own angle is off by (ref_angle, rad)."""
    tol = ref.abs() * EPS[out.dtype] + mag * (math.pi * 2.0 ** -25 + 2.0 ** -22 + 3 * 2.0 ** -24 + ref_angle)
    tol = tol * (1 + 2.0 ** -7)             # the rounding is relative to the unrounded value
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25              # half a step of fp16's subnormals
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), (out.double() - ref).abs()[bad].max()


def _positions(axes, T, seed, lo=-(1 << 31), hi=(1 << 31) - 1):
    rng = np.random.default_rng(seed)
    p = rng.integers(lo, hi, (axes, T), endpoint=True)
    p.flat[0] = lo
    p.flat[-1] = hi
    return torch.from_numpy(p.astype(np.int32)).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,sections", [(128, (16, 24, 24)), (64, (32,)), (80, (20, 20)), (72, (36,)), (128, (8, 8)),
                                        (7, (1, 2)), (256, (128,)), (2, (1,)), (66, (1, 1, 1, 1))])
@pytest.mark.parametrize("T,H", [(1, 1), (65, 3), (700, 9)])
def test_rope_apply(dtype, layout, D, sections, T, H):
    freqs, axes = rope_table(sum(sections), sections, base=5e5)
    rope = Rope(D, freqs, axes, layout=layout, scale=1.0)
    x = torch.randn(T, H, D, generator=_gen(T + D), device="cuda").to(dtype)
    pos = _positions(len(sections), T, 3, 0, 1 << 20)
    for grad in (False, True):
        out = rope.apply(x, pos, grad=grad)
        ref, mag = _rotate64(x, pos, freqs, axes, layout, 1.0, grad)
        _check_rotation(out, ref, mag)
        assert torch.equal(out[..., 2 * len(freqs):], x[..., 2 * len(freqs):])
        again = rope.apply(x.clone(), pos, grad=grad)
        assert torch.equal(out, again)
        y = x.clone()
        assert rope.apply(y, pos, y, grad=grad) is y and torch.equal(y, out)      # in place


def test_rope_far_positions_and_scale():
    """Positions over the whole of int32, negative ones too: the angle's error
    does not grow with the distance (64-bit frequencies)."""
    freqs, axes = rope_table(32, (8, 12, 12), base=1e4)
    freqs = [f * (-1) ** i for i, f in enumerate(freqs)]
    rope = Rope(64, freqs, axes, scale=1.25)
    x = torch.randn(500, 2, 64, generator=_gen(1), device="cuda")
    pos = _positions(3, 500, 4)
    ref, mag = _rotate64(x, pos, freqs, axes, "half", 1.25)
    # the reference's own product pos * f (f <= 1) is rounded in 64 bits: 2^31 *
    # 2^-53 rad at most; the table's turns are off by 2^31 * 2^-65 turns
    _check_rotation(rope.apply(x, pos), ref, mag, 2.0 ** -22 + 2.0 ** -34 * 2 * math.pi)


@pytest.mark.parametrize("off", [0, 8, 4, 1])
def test_rope_strided_views(off):
    """Heads of one fused projection, at offsets that allow 16-byte, 8-byte
    and single-element accesses; in place, the other heads keep their bits."""
    T, D = 37, 64
    freqs, axes = rope_table(32)
    rope = Rope(D, freqs, axes)
    buf = _bf16((T * 12 * D + 64,), 5)
    keep = buf.clone()
    x = buf[off:off + T * 12 * D].view(T, 12, D)[:, 2:7]
    pos = _positions(1, T, 6, 0, 5000)
    ref, mag = _rotate64(x, pos, freqs, axes, "half")
    packed = rope.apply(x, pos)
    _check_rotation(packed, ref, mag)
    rope.apply(x, pos, x)
    assert torch.equal(x, packed)
    rest = buf.clone()
    rest[off:off + T * 12 * D].view(T, 12, D)[:, 2:7] = keep[off:off + T * 12 * D].view(T, 12, D)[:, 2:7]
    assert torch.equal(rest, keep)
    # from one set of heads to another of the same buffer
    full = keep[off:off + T * 12 * D].view(T, 12, D)
    src = full[:, 2:7].clone()
    rope.apply(full[:, 2:7], pos, full[:, 7:12])
    assert torch.equal(full[:, 7:12], packed) and torch.equal(full[:, 2:7], src)


def test_rope_gradient_is_the_transpose_and_the_difference():
    """<R x, y> = <x, R^T y>, and R^T y against differences of <R x, y> in x
    (R is linear: a difference with step 1 is exact but for rounding)."""
    freqs, axes = rope_table(6, (2, 2, 2), base=50.0)
    for layout in ("half", "interleaved"):
        rope = Rope(14, freqs, axes, layout=layout, scale=0.75)
        x = torch.randn(3, 2, 14, generator=_gen(7), device="cuda")
        y = torch.randn(3, 2, 14, generator=_gen(8), device="cuda")
        pos = _positions(3, 3, 9, -100, 100)
        gx = rope.apply(y, pos, grad=True)
        ref, mag = _rotate64(y, pos, freqs, axes, layout, 0.75, True)
        _check_rotation(gx[..., :12], ref[..., :12], mag[..., :12])
        f0 = (rope.apply(x, pos).double() * y.double()).sum()
        assert abs(f0 - (x.double() * gx.double()).sum()) < 84 * 2.0 ** -21 * 4 * 4
        for t, h, d in [(0, 0, 0), (1, 1, 5), (2, 0, 11), (2, 1, 12), (0, 1, 13)]:
            xp = x.clone()
            xp[t, h, d] += 1.0
            diff = (rope.apply(xp, pos).double() * y.double()).sum() - f0
            assert abs(diff - gx[t, h, d].double()) < 84 * 2.0 ** -21 * 4 * 4


def test_rope_refusals_of_the_binding():
    rope = Rope(64, *rope_table(32, (16, 16)))
    x, pos = _bf16((4, 2, 64), 1), _positions(2, 4, 1, 0, 9)
    with pytest.raises(TypeError):
        rope.apply(x.double(), pos)
    for bad in (x.cpu(), x[..., :32], x.transpose(0, 1).contiguous().transpose(0, 1), x[0]):
        with pytest.raises(ValueError):
            rope.apply(bad, pos)
    for bad in (pos.long(), pos[:1], pos[:, :3], pos.cpu(), pos.t().contiguous().t()):
        with pytest.raises(ValueError):
            rope.apply(x, bad)
    with pytest.raises(ValueError):
        rope.apply(x, pos, x.float())
    assert rope.apply(x[:0], pos[:, :0]).shape == (0, 2, 64)


# -------------------------------------------------------------------- append

def _cache(lens, page, Hkv, D, s_max, seed, fused=False, B=None):
    """An empty paged cache (all NaN) with room for `lens` keys."""
    lens = np.asarray(lens)
    zero = torch.zeros(int(lens.sum()), Hkv, D, dtype=torch.bfloat16, device="cuda")
    pc = W.paginate(zero, zero, W.cu_from_lengths(lens), len(lens), page, s_max, seed=seed, fused=fused, extra_cols=1)
    pc.k_cache.fill_(float("nan"))
    pc.v_cache.fill_(float("nan"))
    return pc


def _bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("page,fused", [(8, False), (16, True), (128, False)])
@pytest.mark.parametrize("Hq,Hkv,D,n", [(8, 2, 64, 32), (4, 4, 128, 64), (7, 1, 128, 20), (2, 2, 64, 3)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_paged(page, fused, Hq, Hkv, D, n, layout):
    lq = np.array([1, 0, 5, 17, 1, 64, 0, 3])
    lk = np.array([1, 9, 5, 40, 129, 64, 0, 130])
    B, s_max, T = 8, 130, int(lq.sum()) + 3                    # three rows behind the last sequence
    pc = _cache(lk, page, Hkv, D, s_max, 1, fused)
    rope = Rope(D, *rope_table(n, (n - 2, 1, 1)), layout=layout)
    qkv = _bf16((T, Hq + 2 * Hkv, D), 2)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = _positions(3, T, 3, 0, 1 << 18)
    plan = Plan(B, s_max, Hq, Hkv, D, 64)
    q_out = torch.full((T, Hq, D), SENTINEL, dtype=torch.bfloat16, device="cuda")
    cu_q, cu_k = _cu(lq), _cu(lk)
    kc, vc = pc.k_cache.clone(), pc.v_cache.clone()
    plan.append_paged(k, v, pc.k_cache, pc.v_cache, pc.block_table, cu_q, cu_k, q=q, pos=pos, rope=rope, q_out=q_out)
    assert plan.check_error() == 0
    live = int(lq.sum())
    assert torch.equal(q_out[:live], rope.apply(q, pos)[:live])
    assert (q_out[live:] == SENTINEL).all()
    kr = rope.apply(k, pos)
    at = 0
    for b in range(B):
        for qi in range(lq[b]):
            j = lk[b] - lq[b] + qi
            pg = int(pc.block_table[b, j // page])
            kc[pg, j % page], vc[pg, j % page] = kr[at], v[at]
            at += 1
    assert torch.equal(_bits(kc), _bits(pc.k_cache)) and torch.equal(_bits(vc), _bits(pc.v_cache))
    # no rotation, no queries; then a packed q in place
    pc.k_cache.fill_(float("nan"))
    plan.append_paged(k, v, pc.k_cache, pc.v_cache, pc.block_table, cu_q, cu_k)
    b, j = 3, 39
    assert torch.equal(pc.k_cache[int(pc.block_table[b, j // page]), j % page], k[int(lq[:4].sum()) - 1])
    qp = q.contiguous()
    assert plan.append_paged(k, v, pc.k_cache, pc.v_cache, pc.block_table, cu_q, cu_k, q=qp, pos=pos, rope=rope,
                             q_out=qp) is qp
    assert torch.equal(qp[:live], q_out[:live]) and torch.equal(qp[live:], q[live:])


def test_append_reads_what_the_call_before_it_wrote():
    """Rotation into a buffer and append from it, nothing between them in the
    stream: every key of every repetition is that repetition's."""
    B, L, Hkv, D, page = 4, 1024, 8, 128, 64
    T = B * L
    pc = _cache([L] * B, page, Hkv, D, L, 21)
    plan = Plan(B, L, Hkv, Hkv, D, L)
    rope, cu = Rope(D, *rope_table(64)), _cu([L] * B)
    xs = [_bf16((T, Hkv, D), 30 + i) for i in range(4)]
    pos = _positions(1, T, 22, 0, 1 << 16)
    refs = [rope.apply(x, pos) for x in xs]
    k = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    rows = pc.block_table[:, :L // page].long().flatten()
    torch.cuda.synchronize()
    for i in range(12):
        rope.apply(xs[i % 4], pos, k)
        plan.append_paged(k, k, pc.k_cache, pc.v_cache, pc.block_table, cu, cu)
        for cache in (pc.k_cache, pc.v_cache):
            assert torch.equal(_bits(cache[rows].reshape(T, Hkv, D)), _bits(refs[i % 4])), i
    assert plan.check_error() == 0


def test_append_errors_are_reported_and_contained():
    Hq, Hkv, D, page, s_max, B = 2, 1, 64, 16, 64, 4
    pc = _cache([64] * B, page, Hkv, D, s_max, 4)
    plan = Plan(B, s_max, Hq, Hkv, D, 4)
    k, v, q = _bf16((12, Hkv, D), 1), _bf16((12, Hkv, D), 2), _bf16((12, Hq, D), 3)
    rope, pos = Rope(D, *rope_table(32)), _positions(1, 12, 1, 0, 9)

    def call(lq, cu_k, bt=pc.block_table):
        pc.k_cache.fill_(float("nan"))
        pc.v_cache.fill_(float("nan"))
        out = torch.full((12, Hq, D), SENTINEL, dtype=torch.bfloat16, device="cuda")
        plan.append_paged(k, v, pc.k_cache, pc.v_cache, bt, _cu(lq), torch.tensor(cu_k, dtype=torch.int32).cuda(), q=q,
                          pos=pos, rope=rope, q_out=out)
        stored = (~pc.k_cache.isnan()).any(-1).sum().item()
        assert stored == (~pc.v_cache.isnan()).any(-1).sum().item()
        return plan.check_error(), stored, (out != SENTINEL).any(-1).all(-1).cpu().numpy()

    assert call([3, 3, 3, 3], [0, 10, 20, 30, 40])[:2] == (0, 12)
    err, stored, rows = call([5, 3, 1, 3], [0, 10, 20, 30, 40])             # more queries than the plan's
    assert err == vg.ATTN_DEV_ERR_Q_TOO_LONG and stored == 7 and not rows[:5].any() and rows[5:].all()
    err, stored, rows = call([3, 3, 3, 3], [0, 65, 75, 85, 95])
    assert err == vg.ATTN_DEV_ERR_K_TOO_LONG and stored == 9 and not rows[:3].any()
    err, stored, rows = call([3, 3, 3, 3], [0, 10, 5, 15, 25])
    assert err == vg.ATTN_DEV_ERR_OFFSETS and stored == 9 and not rows[3:6].any()
    err, stored, rows = call([3, 3, 3, 3], [0, 2, 12, 22, 32])               # a query before the first key
    assert err == 0 and stored == 11 and rows.all()
    for bad in (-1, pc.k_cache.shape[0], 1 << 30):
        bt = pc.block_table.clone()
        bt[2, 0] = bad
        err, stored, rows = call([3, 3, 3, 3], [0, 10, 20, 30, 40], bt)
        assert err == vg.ATTN_DEV_ERR_PAGE and stored == 9 and rows.all()


# --------------------------------------------------------------- key weights

def _weights64(q, keys, lq, lk, lse, G, decay, w_in, Hkv, ld):
    """Column sums in 64 bits, and a bound of the kernel's error: a score's
    fp32 products and sums are off by at most (D + 2) 2^-24 sum |q k| / sqrt D
    (any order), the exponent's argument by 2^-23 of its parts, the
    exponential by 2^-21 relative; adding up by 2^-20 relative."""
    B, D = len(lq), q.shape[-1]
    out = torch.zeros(B, Hkv, ld, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    q0 = np.cumsum(lq) - lq
    for b in range(B):
        Lq, Lk = int(lq[b]), int(lk[b])
        j = torch.arange(Lk, device="cuda")
        old = max(0, Lk - Lq)
        if w_in is not None and decay:
            out[b, :, :old] = decay * w_in[b, :, :old].double()
        sees = j[None] <= (Lk - Lq + torch.arange(Lq, device="cuda"))[:, None]
        for h in range(Hkv * G):
            qh, kh = q[q0[b]:q0[b] + Lq, h].double(), keys[b][:, h // G].double()
            s = qh @ kh.t() / math.sqrt(D)
            mag = qh.abs() @ kh.abs().t() / math.sqrt(D)
            l = lse[q0[b]:q0[b] + Lq, h, None].double()
            p = torch.exp(s - l).masked_fill(~sees | l.isneginf(), 0.0)
            out[b, h // G, :Lk] += p.sum(0)
            e = (D + 2) * 2.0 ** -24 * mag + 2.0 ** -23 * (s.abs() + l.abs()) + 2.0 ** -21
            tol[b, h // G, :Lk] += (p * e).masked_fill(~sees | l.isneginf(), 0.0).sum(0)
        tol[b, :, :Lk] += out[b, :, :Lk].abs() * 2.0 ** -20
    return out, tol


def _lse64(q, keys, lq, lk, G):
    out, q0 = torch.zeros(q.shape[0], q.shape[1], device="cuda"), np.cumsum(lq) - lq
    for b in range(len(lq)):
        Lq, Lk = int(lq[b]), int(lk[b])
        sees = torch.arange(Lk, device="cuda")[None] <= (Lk - Lq + torch.arange(Lq, device="cuda"))[:, None]
        for h in range(q.shape[1]):
            s = q[q0[b]:q0[b] + Lq, h].double() @ keys[b][:, h // G].double().t() / math.sqrt(q.shape[-1])
            out[q0[b]:q0[b] + Lq, h] = torch.logsumexp(s.masked_fill(~sees, -math.inf), -1).float()
    return out


def _check_weights(lq, lk, Hq, Hkv, D, max_q, s_max, page=0, decay=1.0, seed=0, ld=None, fused=False, alias=False,
                   births=True):
    B, G, ld = len(lq), Hq // Hkv, ld or s_max + 3
    lq, lk = np.asarray(lq), np.asarray(lk)
    q = _bf16((max(1, int(lq.sum())) + 2, Hq, D), seed)
    q[int(lq.sum()):] = float("nan")                            # rows behind the last sequence
    k = _bf16((max(1, int(lk.sum())), Hkv, D), seed + 1)
    k0 = np.cumsum(lk) - lk
    keys = [k[k0[b]:k0[b] + lk[b]] for b in range(B)]
    lse = _lse64(q, keys, lq, lk, G)
    w_in = torch.rand(B, Hkv, ld, generator=_gen(seed + 2), device="cuda") * 3
    for b in range(B):                                           # what must not be read
        w_in[b, :, max(0, lk[b] - lq[b]):] = float("nan")
    if decay == 0.0:
        w_in.fill_(float("nan"))
    out = w_in if alias else torch.full((B, Hkv, ld), SENTINEL, device="cuda")
    before = out.clone()
    born = torch.full((B, Hkv, ld), -5, dtype=torch.int32, device="cuda") if births else None
    seen = torch.from_numpy(lk + 1000 * np.arange(B)).to(torch.int32).cuda() if births else None
    ref, tol = _weights64(q, keys, lq, lk, lse, G, decay, w_in, Hkv, ld)
    plan = Plan(B, s_max, Hq, Hkv, D, max_q)
    cu_q, cu_k = _cu(lq), _cu(lk)
    kw = dict(decay=decay, out=out, seen=seen, born=born)
    if page:
        pc = W.paginate(k, k, W.cu_from_lengths(lk), B, page, s_max, seed=seed, fused=fused, extra_cols=1)
        run = lambda: plan.key_weights_paged(q, pc.k_cache, pc.block_table, cu_q, cu_k, lse, w_in, **kw)  # noqa: E731
    else:
        run = lambda: plan.key_weights(q, k, cu_q, cu_k, lse, w_in, **kw)                                 # noqa: E731
    run()
    assert plan.check_error() == 0
    first = out.clone()
    if not alias:
        for _ in range(3):
            run()
            assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(first))      # repeated calls: the same bits
    for b in range(B):
        n = int(lk[b])
        got, want = first[b, :, :n].double(), ref[b, :, :n]
        assert not got.isnan().any()
        over = (got - want).abs() - tol[b, :, :n]
        assert n == 0 or over.max() <= 0, (b, over.max().item())
        assert torch.equal(torch.nan_to_num(first[b, :, n:]), torch.nan_to_num(before[b, :, n:]))
        if births:
            old = max(0, n - int(lq[b]))
            assert torch.equal(born[b, :, old:n], (1000 * b + torch.arange(old, n, device="cuda")).int().expand(Hkv, -1))
            assert (born[b, :, :old] == -5).all() and (born[b, :, n:] == -5).all()


EDGE_K = [0, 1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 700]


@pytest.mark.parametrize("page", [0, 8, 64])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (32, 2, 64), (24, 1, 128), (48, 1, 64)])
def test_key_weights_decode(Hq, Hkv, D, page):
    _check_weights([1 if n else 0 for n in EDGE_K], EDGE_K, Hq, Hkv, D, 1, 700, page)


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("Hq,Hkv,D,max_q", [(8, 2, 128, 5), (10, 2, 64, 33), (3, 1, 128, 64), (16, 1, 64, 150),
                                            (1, 1, 128, 300)])
def test_key_weights_chunks(Hq, Hkv, D, max_q, page, decay):
    """Query lengths around the tiles' edges, from none to more queries than
    keys (rows that see nothing), with the weights of earlier tokens kept,
    decayed or dropped."""
    rng = np.random.default_rng(max_q)
    lq = np.minimum([0, 1, 2, max_q, max_q, max_q, max_q - 1, max_q // 2, 3, max_q, 1, max_q], max_q)
    lk = np.array([40, 1, 300, 0, 1, max_q, 600, 129, 2, 600, 257, max_q // 2])
    lq = np.concatenate([lq, rng.integers(0, max_q, 4, endpoint=True)])
    lk = np.concatenate([lk, rng.integers(0, 600, 4)])
    _check_weights(lq, lk, Hq, Hkv, D, max_q, 600, page, decay)


def test_key_weights_wide_groups():
    """More query heads per KV head than one row tile holds."""
    _check_weights([1, 2, 0, 2], [5, 130, 70, 2], 136, 1, 64, 2, 130)
    _check_weights([1, 3, 3], [40, 130, 2], 258, 2, 128, 3, 130, page=16)


@pytest.mark.parametrize("G,max_q", [(1, 1), (8, 1), (8, 40)])
def test_key_weights_long_units(G, max_q):
    """Few long sequences: the keys of one head over many blocks, and blocks
    that end inside a unit."""
    _check_weights([max_q, 1, max_q], [9000, 4097, 3001], 2 * G, 2, 128, max_q, 9000, births=False)
    _check_weights([max_q, 1, max_q], [9000, 4097, 3001], 2 * G, 2, 64, max_q, 9000, page=32, fused=True)


def test_key_weights_long_chunk():
    """A prompt attended to in one go, and a chunk behind a long cache: many
    row tiles, shares that cut a tile of keys between blocks."""
    _check_weights([1500, 777, 2000], [1500, 777, 2000], 8, 2, 128, 2000, 2000, page=64)
    _check_weights([1000], [3500], 16, 1, 64, 1000, 3500)


def test_key_weights_in_place_and_single_key():
    _check_weights([1, 3, 1], [500, 40, 1], 8, 2, 128, 3, 500, alias=True)
    _check_weights([1, 1], [500, 40], 8, 2, 128, 1, 500, page=16, alias=True, decay=0.5)
    _check_weights([1], [1], 1, 1, 64, 1, 1)


def test_key_weights_of_attention_sum_to_the_queries():
    """With the library's own lse, each (query, head) hands out a weight of
    one: a head's ledger adds up to the queries that saw a key."""
    sh = W.Shape("kw", B=5, Hq=32, Hkv=4, D=128, max_q=16, s_max=1200)
    lq, lk = [1, 16, 7, 16, 0], [1200, 16, 650, 10, 33]
    batch = W.make_batch(sh, lq, lk, seed=3, gen_device="cuda")
    plan = Plan(5, 1200, 32, 4, 128, 16)
    cu_q, cu_k = _cu(lq), _cu(lk)
    out, lse = plan.run(batch.q, batch.k, batch.v, cu_q, cu_k)
    w = plan.key_weights(batch.q, batch.k, cu_q, cu_k, lse)
    assert w.shape == (5, 4, 1200)
    rows = np.array([1, 16, 7, 10, 0]) * 8                      # six of the fourth's queries see nothing
    # each row's weights are off by 2^-20 at most (scores of order 1, lse of order 10)
    np.testing.assert_allclose(w.double().sum(-1).cpu().numpy(), np.repeat(rows[:, None], 4, 1), rtol=2.0 ** -16)


def test_key_weights_minus_inf_lse_and_foreign_nans():
    """Rows with lse = -inf add nothing; NaN queries and keys of one sequence
    stay out of the others, in the same tile or not."""
    B, Hq, Hkv, D = 4, 8, 2, 64
    lq, lk = np.array([3, 2, 5, 3]), np.array([40, 70, 20, 50])
    q, k = _bf16((13, Hq, D), 1), _bf16((180, Hkv, D), 2)
    k0 = np.cumsum(lk) - lk
    keys = [k[k0[b]:k0[b] + lk[b]] for b in range(B)]
    lse = _lse64(q, keys, lq, lk, 4)
    lse[1] = -math.inf
    ref, tol = _weights64(q, keys, lq, lk, lse, 4, 1.0, None, Hkv, 70)
    q[3:5] = float("nan")                                       # the second sequence
    k[40:110] = float("inf")
    plan = Plan(B, 70, Hq, Hkv, D, 5)
    out = plan.key_weights(q, k, _cu(lq), _cu(lk), lse)
    for b in (0, 2, 3):
        assert ((out[b].double() - ref[b]).abs() <= tol[b]).all(), b
    assert out[1, :, :70].isnan().all()


@pytest.mark.parametrize("Hq,Hkv,max_q,lq", [(8, 2, 40, 40), (8, 1, 1, 1), (16, 1, 8, 5), (136, 1, 3, 3)])
def test_key_weights_skips_rows_without_a_normaliser(Hq, Hkv, max_q, lq):
    """lse = -inf takes a row out whatever its query holds (NaN here), in tiles
    that every row sees as in those that the mask cuts."""
    D, lk = 64, 700
    q, k = _bf16((lq, Hq, D), 1), _bf16((lk, Hkv, D), 2)
    lse = _lse64(q, [k], np.array([lq]), np.array([lk]), Hq // Hkv)
    lse[lq // 2:, ::3] = -math.inf
    ref, tol = _weights64(q, [k], np.array([lq]), np.array([lk]), lse, Hq // Hkv, 1.0, None, Hkv, lk)
    q[lse.isneginf()] = float("nan")
    plan = Plan(1, lk, Hq, Hkv, D, max_q)
    out = plan.key_weights(q, k, _cu([lq]), _cu([lk]), lse)
    assert ((out.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("lk", [[20, 17, 18, 12], [1, 1], [127], [0, 5, 0], [60, 67, 1, 300]])
def test_key_weights_short_packed_buffers(lk):
    """Keys that end fewer than a tile's 128 rows behind the buffer's first
    row: the last few rows of a larger buffer, NaN around them."""
    B, Hq, Hkv, D, s_max = len(lk), 28, 4, 128, 320
    T = sum(lk)
    room = _bf16((T + 400, Hkv, D), 71)
    room[:200] = float("nan")
    room[200 + T:] = float("nan")
    k, q = room[200:200 + T], _bf16((B, Hq, D), 72)
    lq = np.ones(B, np.int64)
    at = np.cumsum([0] + lk)
    keys = [k[at[b]:at[b + 1]] for b in range(B)]
    lse = _lse64(q, keys, lq, lk, Hq // Hkv)
    ref, tol = _weights64(q, keys, lq, lk, lse, Hq // Hkv, 0.0, None, Hkv, s_max)
    plan = Plan(B, s_max, Hq, Hkv, D, 1)
    out = torch.full((B, Hkv, s_max), SENTINEL, device="cuda")
    plan.key_weights(q, k, _cu(lq), _cu(lk), lse, out=out)
    assert plan.check_error() == 0
    for b in range(B):
        assert ((out[b, :, :lk[b]].double() - ref[b, :, :lk[b]]).abs() <= tol[b, :, :lk[b]]).all(), b
        assert (out[b, :, lk[b]:] == SENTINEL).all()


def test_key_weights_errors_are_reported_and_contained():
    B, Hq, Hkv, D, s_max = 3, 8, 2, 64, 100
    q, k = _bf16((9, Hq, D), 1), _bf16((300, Hkv, D), 2)
    lse = torch.ones(9, Hq, device="cuda")
    plan = Plan(B, s_max, Hq, Hkv, D, 3)

    def call(cu_q, cu_k, bt=None):
        out = torch.full((B, Hkv, s_max), SENTINEL, device="cuda")
        cu_q, cu_k = (torch.tensor(x, dtype=torch.int32).cuda() for x in (cu_q, cu_k))
        if bt is None:
            plan.key_weights(q, k, cu_q, cu_k, lse, out=out)
        else:
            plan.key_weights_paged(q, bt[0], bt[1], cu_q, cu_k, lse, out=out)
        return plan.check_error(), (out != SENTINEL).sum(-1).cpu().tolist()

    assert call([0, 3, 6, 9], [0, 50, 150, 160]) == (0, [[50, 50], [100, 100], [10, 10]])
    assert call([0, 4, 6, 9], [0, 50, 150, 160]) == (vg.ATTN_DEV_ERR_Q_TOO_LONG, [[0, 0], [100, 100], [10, 10]])
    assert call([0, 3, 6, 9], [0, 101, 150, 160]) == (vg.ATTN_DEV_ERR_K_TOO_LONG, [[0, 0], [49, 49], [10, 10]])
    assert call([0, 3, 6, 9], [0, 50, 40, 60]) == (vg.ATTN_DEV_ERR_OFFSETS, [[50, 50], [0, 0], [20, 20]])
    assert call([0, 3, 2, 5], [0, 50, 60, 80]) == (vg.ATTN_DEV_ERR_OFFSETS, [[50, 50], [0, 0], [20, 20]])
    pc = W.paginate(k[:160], k[:160], np.array([0, 50, 150, 160]), B, 16, s_max, seed=3)
    for bad in (-1, pc.k_cache.shape[0], 1 << 30):
        bt = pc.block_table.clone()
        bt[1, 2] = bad
        err, n = call([0, 3, 6, 9], [0, 50, 150, 160], (pc.k_cache, bt))
        assert err == vg.ATTN_DEV_ERR_PAGE and n[0] == [50, 50] and n[2] == [10, 10]


# ------------------------------------------------------------------ eviction

def _evict_host(w, born, seen, lk, keep, sink, recent):
    """(src, c) of each unit: place i of the result holds what place src[i] held."""
    out = {}
    for b in range(w.shape[0]):
        n, c = int(lk[b]), min(int(lk[b]), max(0, int(keep[b])))
        for h in range(w.shape[1]):
            r = w[b, h, :n].astype(np.float64).copy()
            r[np.isnan(r)] = -np.inf
            fixed = (born[b, h, :n] < sink) | (born[b, h, :n] >= int(seen[b]) - recent)
            r[fixed] = np.inf
            order = sorted(range(n), key=lambda j: (-r[j], j))[:c]
            kept = np.array(sorted(order), dtype=np.int64)
            src = np.arange(c)
            src[np.setdiff1d(np.arange(c), kept)] = kept[kept >= c]
            out[b, h] = (src, c)
    return out


def _check_evict(lk, keep, Hkv=2, D=64, page=16, sink=0, recent=0, weights="tail", in_place=False, seed=0, s_max=None,
                 fused=False, births="run", ld=None, B_max=None):
    lk, keep = np.asarray(lk), np.asarray(keep)
    B = B_max or len(lk)
    lk, keep = (np.concatenate([x, np.zeros(B - len(x), np.int64)]) for x in (lk, keep))
    s_max = s_max or max(1, int(lk.max()))
    ld = ld or s_max + 5
    rng = np.random.default_rng(seed)
    k, v = _bf16((max(1, int(lk.sum())), Hkv, D), seed), _bf16((max(1, int(lk.sum())), Hkv, D), seed + 1)
    pc = W.paginate(k, v, W.cu_from_lengths(lk), B, page, s_max, seed=seed, fused=fused, extra_cols=2)
    w = {"tail": lambda: -np.log(rng.random((B, Hkv, ld))) ** 3,
         "equal": lambda: np.full((B, Hkv, ld), 0.25),
         "coarse": lambda: rng.integers(0, 4, (B, Hkv, ld)) / 2.0,
         "signed": lambda: rng.standard_normal((B, Hkv, ld)) * 10.0 ** rng.integers(-30, 30, (B, Hkv, ld)),
         "odd": lambda: rng.choice([0.0, -0.0, np.nan, np.inf, -np.inf, 1.0, -1.0, 1e-45, 3.4e38],
                                   (B, Hkv, ld))}[weights]().astype(np.float32)
    if births == "run":
        born = np.broadcast_to(np.arange(ld), (B, Hkv, ld)).copy()
    else:                                                     # scrambled by earlier evictions
        born = np.stack([np.stack([rng.permutation(2 * ld)[:ld] for _ in range(Hkv)]) for _ in range(B)])
    born = born.astype(np.int32)
    seen = (lk if births == "run" else np.full(B, 2 * ld)).astype(np.int32)
    plan = Plan(B, s_max, Hkv, Hkv, D, 1)
    wt, bt = torch.from_numpy(w).cuda(), torch.from_numpy(born).cuda()
    wo = wt.clone() if in_place else torch.full_like(wt, SENTINEL)
    bo = bt.clone() if in_place else torch.full_like(bt, -77)
    wi, bi = (wo, bo) if in_place else (wt, bt)
    wo_before, bo_before = wo.clone(), bo.clone()
    kc, vc = pc.k_cache.clone(), pc.v_cache.clone()
    cu_out = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
    args = (torch.from_numpy(seen).cuda(), torch.from_numpy(keep.astype(np.int32)).cuda(), pc.k_cache, pc.v_cache,
            pc.block_table, _cu(lk))
    plan.evict_paged(wi, bi, *args, sink=sink, recent=recent, weight_out=wo, born_out=bo, cu_k_out=cu_out)
    assert plan.check_error() == 0
    moves = _evict_host(w, born, seen, lk, keep, sink, recent)
    table = pc.block_table.cpu().numpy()
    cs = []
    wr, br = wo_before.cpu().numpy(), bo_before.cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            src, c = moves[b, h]
            wr[b, h, :c], br[b, h, :c] = w[b, h, src], born[b, h, src]
            to = np.nonzero(src != np.arange(c))[0]
            if len(to):
                at = src[to]
                pt, pa = (torch.from_numpy(table[b, x // page].astype(np.int64)).cuda() for x in (to, at))
                st, sa = (torch.from_numpy(x % page).cuda() for x in (to, at))
                kc[pt, st, h], vc[pt, st, h] = kc[pa, sa, h], vc[pa, sa, h]
        cs.append(min(lk[b], max(0, keep[b])))
    assert np.array_equal(bo.cpu().numpy(), br)
    assert np.array_equal(wo.cpu().numpy().view(np.int32), wr.view(np.int32))
    assert torch.equal(_bits(pc.k_cache), _bits(kc)) and torch.equal(_bits(pc.v_cache), _bits(vc))
    assert cu_out.cpu().tolist() == [0] + np.cumsum(cs).tolist()
    if not in_place:                                          # a repeated call does the same again
        plan.evict_paged(wi, bi, *args, sink=sink, recent=recent, weight_out=wo, born_out=bo, cu_k_out=cu_out)
        assert np.array_equal(wo.cpu().numpy().view(np.int32), wr.view(np.int32))
        assert torch.equal(_bits(pc.k_cache), _bits(kc))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("weights", ["tail", "equal", "coarse", "signed", "odd"])
@pytest.mark.parametrize("page,D,fused", [(8, 64, False), (16, 128, True), (64, 128, False)])
def test_evict_lengths(weights, page, D, fused, in_place):
    lk = [0, 1, 1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 300, 300, 300, 300, 511, 700]
    keep = [5, 0, 1, 1, 30, 31, 32, 1, 64, 60, 127, 128, 299, 300, 301, -3, 256, 100]
    _check_evict(lk, keep, D=D, page=page, weights=weights, fused=fused, in_place=in_place, B_max=len(lk) + 2)


@pytest.mark.parametrize("births", ["run", "scrambled"])
@pytest.mark.parametrize("sink,recent", [(4, 0), (0, 16), (4, 64), (100, 300), (1 << 30, 0), (0, (1 << 31) - 1)])
def test_evict_protected_keys(sink, recent, births):
    """Protected keys outrank every weight, +inf aside (a tie); where they
    alone pass the budget the lowest places win."""
    lk, keep = [400, 90, 300, 33], [128, 64, 299, 8]
    _check_evict(lk, keep, sink=sink, recent=recent, births=births)
    _check_evict(lk, keep, sink=sink, recent=recent, births=births, weights="odd", Hkv=3, in_place=True)


@pytest.mark.parametrize("Hkv,lk,keep", [(1, [20000], [1500]), (2, [5000, 20000, 0], [4990, 19999, 7]),
                                         (8, [9000], [4500]), (1, [70000], [3000]), (3, [8193], [8192])])
@pytest.mark.parametrize("weights", ["tail", "coarse"])
def test_evict_long(Hkv, lk, keep, weights):
    """Units of many keys: more than one thread block's, or shared memory's."""
    _check_evict(lk, keep, Hkv=Hkv, page=32, sink=4, recent=100, weights=weights)


def test_evict_longest_plans():
    """The largest length that eviction takes, with ties across all blocks of a
    cluster and within one, of real lengths long and short."""
    _check_evict([1 << 19], [1000], Hkv=1, page=64, weights="coarse")
    _check_evict([(1 << 19) - 33, 70], [(1 << 19) - 40, 9], Hkv=1, page=64, weights="equal", s_max=1 << 19)


def test_evict_zero_ties():
    """The threshold among keys that were never looked at: they tie at zero."""
    rng = np.random.default_rng(3)
    for n, c, hkv in ((1044, 1020, 2), (9000, 8900, 2), (20000, 17000, 1)):
        B, page, s_max = 2, 32, n
        k = _bf16((2 * n, hkv, 64), n)
        pc = W.paginate(k, k, np.array([0, n, 2 * n]), B, page, s_max, seed=n)
        w = -np.log(rng.random((B, hkv, n))) ** 3
        w[rng.random(w.shape) < 0.2] = 0.0
        w[0, 0, ::7] = -0.0
        w = w.astype(np.float32)
        born = np.broadcast_to(np.arange(n, dtype=np.int32), w.shape).copy()
        plan = Plan(B, s_max, hkv, hkv, 64, 1)
        wo = torch.zeros(w.shape, device="cuda")
        bo = torch.zeros(w.shape, dtype=torch.int32, device="cuda")
        full = torch.full((B,), n, dtype=torch.int32, device="cuda")
        plan.evict_paged(torch.from_numpy(w).cuda(), torch.from_numpy(born).cuda(), full, full * 0 + c, pc.k_cache,
                         pc.v_cache, pc.block_table, _cu([n, n]), weight_out=wo, born_out=bo)
        ref = _evict_host(w, born, [n, n], [n, n], [c, c], 0, 0)
        for (b, h), (src, _) in ref.items():
            assert np.array_equal(bo[b, h, :c].cpu().numpy(), born[b, h, src]), (n, b, h)


def test_evict_many_long_units():
    """Enough units to fill the device with one block each, of more keys than
    a block keeps in shared memory."""
    _check_evict([60000] * 19, [500] * 19, Hkv=8, D=64, page=64, weights="coarse")


def test_evict_errors_are_reported_and_contained():
    B, Hkv, D, page, s_max = 3, 2, 64, 16, 100
    k = _bf16((210, Hkv, D), 2)
    pc = W.paginate(k, k, np.array([0, 60, 140, 210]), B, page, s_max, seed=3)
    plan = Plan(B, s_max, Hkv, Hkv, D, 1)
    w = torch.rand(B, Hkv, s_max, generator=_gen(1), device="cuda")
    born = torch.arange(s_max, dtype=torch.int32, device="cuda").expand(B, Hkv, s_max).contiguous()
    seen = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    keep = torch.full((B,), 50, dtype=torch.int32, device="cuda")

    def call(cu_k, bt=pc.block_table):
        wo, bo = torch.full_like(w, SENTINEL), torch.full_like(born, -1)
        kc, vc = pc.k_cache.clone(), pc.v_cache.clone()
        _, _, cu = plan.evict_paged(w, born, seen, keep, kc, vc, bt, torch.tensor(cu_k, dtype=torch.int32).cuda(),
                                    weight_out=wo, born_out=bo)
        return plan.check_error(), cu.cpu().tolist(), (wo != SENTINEL).sum(-1).cpu().tolist(), kc

    err, cu, n, good = call([0, 60, 140, 210])
    assert (err, cu, n) == (0, [0, 50, 100, 150], [[50, 50]] * 3)
    err, cu, n, _ = call([0, 60, 161, 210])
    assert (err, cu, n) == (vg.ATTN_DEV_ERR_K_TOO_LONG, [0, 50, 50, 99], [[50, 50], [0, 0], [49, 49]])
    err, cu, n, _ = call([0, 60, 40, 110])
    assert (err, cu, n) == (vg.ATTN_DEV_ERR_OFFSETS, [0, 50, 50, 100], [[50, 50], [0, 0], [50, 50]])
    for bad in (-1, pc.k_cache.shape[0], 1 << 30):
        bt = pc.block_table.clone()
        bt[1, 4] = bad                                        # keys 64..79 of the second sequence
        err, cu, n, kc = call([0, 60, 140, 210], bt)
        assert (err, cu, n) == (vg.ATTN_DEV_ERR_PAGE, [0, 50, 100, 150], [[50, 50]] * 3)
        for b in (0, 2):
            for pg in pc.block_table[b, :3].cpu().tolist():
                assert torch.equal(_bits(kc[pg]), _bits(good[pg]))


def test_refusals_with_a_plan():
    """Bad sizes, strides, alignments and overlaps are refused before anything
    runs (C ABI), and wrong tensors by the binding."""
    L = vg.lib()
    plan = Plan(2, 64, 8, 2, 64, 4)
    h = plan.handle
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    a = buf.data_ptr()
    rope, other = Rope(64, *rope_table(32)), Rope(128, *rope_table(64))
    P = lambda i: a + i * 65536                                                     # noqa: E731
    cache = (2048, 128, 16, 4, P(15), 4)

    def append(rope=rope.handle, q=P(0), qs=512, k=P(1), ks=128, v=P(2), vs=128, T=4, pos=P(3), ps=4, qo=P(4), kc=P(5),
               vc=P(6), cache=cache, cq=P(14), ck=P(14)):
        return L.attn_append_paged(h, rope, q, qs, k, ks, v, vs, T, pos, ps, qo, kc, vc, *cache, cq, ck, None)

    for name in ("k", "v", "kc", "vc", "cq", "ck", "pos", "q", "qo"):
        assert append(**{name: None}) == -3, name
    assert append(rope=other.handle) == -1
    assert append(T=-1) == -1 and append(T=0) == 0
    assert append(qs=504) == -1 and append(ks=120) == -1 and append(vs=132) == -1
    assert append(q=P(0) + 8) == -4 and append(kc=P(5) + 8) == -4 and append(cq=P(14) + 2) == -4
    assert append(qo=P(0) + 1024) == -1 and append(qo=P(0), qs=640) == -1
    assert append(qo=P(1)) == -1 and append(qo=P(2) + 16) == -1
    bad_caches = [(2040, 128, 16, 4, P(15), 4), (2048, 120, 16, 4, P(15), 4), (2048, 128, 12, 4, P(15), 4),
                  (2048, 128, 4, 4, P(15), 16), (2048, 128, 16, 0, P(15), 4), (2048, 128, 16, 4, P(15), 3)]
    for c in bad_caches:
        assert append(cache=c) == -1, c
    assert append(cache=(2048, 128, 16, 4, None, 4)) == -3
    assert append(cache=(2048, 128, 16, 4, P(15) + 1, 4)) == -4

    def weights(q=P(0), k=P(1), ks=128, cq=P(14), ck=P(14), lse=P(2), decay=1.0, wi=P(3), wo=P(4), ld=64, seen=P(13),
                born=P(5), cache=None, T=4, Tk=20):
        tail = (cq, ck, lse, decay, wi, wo, ld, seen, born, None)
        if cache:
            return L.attn_key_weights_paged(h, q, T, k, *cache, *tail)
        return L.attn_key_weights(h, q, T, k, ks, Tk, *tail)

    for name in ("q", "k", "cq", "ck", "lse", "wo", "seen", "born"):
        assert weights(**{name: None}) == -3, name
        assert weights(cache=cache, **{name: None}) == -3, name
    assert weights(ks=120) == -1 and weights(ks=132) == -1 and weights(ld=63) == -1
    assert weights(decay=-1.0) == -1 and weights(decay=math.nan) == -1 and weights(decay=math.inf) == -1
    assert weights(wo=P(3) + 64) == -1 and weights(born=P(4)) == -1 and weights(born=P(3)) == -1
    assert weights(T=-1) == -1 and weights(T=1 << 31) == -1 and weights(Tk=-1) == -1 and weights(Tk=1 << 31) == -1
    assert weights(T=-1, cache=cache) == -1
    assert weights(q=P(0) + 8) == -4 and weights(lse=P(2) + 2) == -4
    for c in bad_caches:
        assert weights(cache=c) == -1, c

    def evict(w=P(0), born=P(1), seen=P(13), keep=P(12), sink=0, recent=0, wo=P(2), bo=P(3), ld=64, kc=P(5), vc=P(6),
              cache=cache, ck=P(14), co=P(11)):
        return L.attn_evict_paged(h, w, born, seen, keep, sink, recent, wo, bo, ld, kc, vc, *cache, ck, co, None)

    for name in ("w", "born", "seen", "keep", "wo", "bo", "kc", "vc", "ck", "co"):
        assert evict(**{name: None}) == -3, name
    assert evict(sink=-1) == -1 and evict(recent=-1) == -1 and evict(ld=63) == -1
    assert evict(wo=P(0) + 4) == -1 and evict(bo=P(1) + 512) == -1 and evict(wo=P(1)) == -1 and evict(bo=P(2)) == -1
    assert evict(co=P(14)) == -1 and evict(co=P(14) + 8) == -1 and evict(co=P(12)) == -1 and evict(co=P(13)) == -1
    assert evict(kc=P(5) + 8) == -4 and evict(keep=P(12) + 1) == -4
    for c in bad_caches:
        assert evict(cache=c) == -1, c
    big = Plan(1, (1 << 19) + 1, 1, 1, 64, 1)
    assert L.attn_evict_paged(big.handle, P(0), P(1), P(13), P(12), 0, 0, P(2), P(3), (1 << 19) + 1, P(5), P(6), 2048, 64,
                              16, 4, P(15), 1 << 20, P(14), P(11), None) == -2
    # the binding
    q, k = _bf16((4, 8, 64), 1), _bf16((20, 2, 64), 2)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    lse = torch.zeros(4, 8, device="cuda")
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    led = torch.zeros(2, 2, 64, device="cuda")
    born = led.int()
    for bad in (dict(lse=lse[:3]), dict(lse=lse.cpu()), dict(weight_in=led[:, :, :63]), dict(out=led.double()),
                dict(born=born), dict(seen=cu[:2]), dict(cu_q=cu[:2]), dict(cu_k=cu.long()),
                dict(out=torch.zeros(2, 2, 64)), dict(weight_in=led.transpose(0, 1))):
        a = dict(q=q, k=k, cu_q=cu, cu_k=cu, lse=lse)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            plan.key_weights(**a)
    for bad in (dict(k_cache=kc.cpu()), dict(k_cache=kc[..., :32]), dict(k_cache=kc.float()),
                dict(block_table=bt[:1]), dict(block_table=bt[:, :3]), dict(block_table=bt.long()),
                dict(keep=cu), dict(born=led), dict(cu_k_out=cu.long()), dict(v_cache=kc[:3])):
        a = dict(weight=led, born=born, seen=cu[:2].contiguous(), keep=cu[:2].contiguous(), k_cache=kc, v_cache=kc.clone(),
                 block_table=bt, cu_k=cu)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            plan.evict_paged(**a)
    for bad in (dict(k=k.float()), dict(v=k[:3]), dict(q=q, pos=None, rope=rope), dict(pos=born[0, :1]),
                dict(q_out=q), dict(cu_q=cu[:2]), dict(k=k.cpu()), dict(k=k[..., :32])):
        a = dict(k=k[:4], v=k[4:8], k_cache=kc, v_cache=kc.clone(), block_table=bt, cu_q=cu, cu_k=cu)
        a.update(bad)
        with pytest.raises((ValueError, TypeError, vg.AttnError)):
            plan.append_paged(**a)


# ---------------------------------------------------------- the serving loop

class _Server:
    """Append, attend, weigh and evict over one paged cache, each step in the
    plain form beside it."""

    def __init__(self, B, Hq, Hkv, D, max_q, s_max, page, seed=0):
        self.B, self.Hq, self.Hkv, self.D, self.G, self.page, self.s_max = B, Hq, Hkv, D, Hq // Hkv, page, s_max
        self.freqs, self.axes = rope_table(D // 2, (D // 4, D // 8, D // 8), base=1e4)
        self.rope = Rope(D, self.freqs, self.axes)
        self.plan = Plan(B, s_max, Hq, Hkv, D, max_q)
        pc = _cache([s_max] * B, page, Hkv, D, s_max, seed)
        self.kc, self.vc, self.bt = pc.k_cache, pc.v_cache, pc.block_table
        self.weight = torch.full((B, Hkv, s_max), float("nan"), device="cuda")
        self.born = torch.full((B, Hkv, s_max), -1, dtype=torch.int32, device="cuda")
        self.seen = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        # the plain form: per (b, hk) lists of (key, value, weight, birth)
        self.ref = [[dict(k=torch.zeros(0, D, dtype=torch.float64, device="cuda"),
                          v=torch.zeros(0, D, dtype=torch.float64, device="cuda"),
                          w=torch.zeros(0, dtype=torch.float64, device="cuda"), born=[]) for _ in range(Hkv)]
                    for _ in range(B)]
        self.total = [0] * B


def test_serving_loop():
    """Six steps of a batch at a budget: prompts, then short and single-token
    steps, evicting as it goes.  Kept keys are compared by their births, so a
    wrong selection, a wrong move or a stale ledger entry shows; selections are
    recomputed from the kernel's own weights, since two nearly alike weights
    may rank either way."""
    B, Hq, Hkv, D, s_max, page = 4, 8, 2, 64, 160, 16
    s = _Server(B, Hq, Hkv, D, 96, s_max, page)
    steps = [[96, 40, 0, 7], [1, 1, 1, 1], [30, 1, 5, 0], [1, 1, 1, 1], [2, 64, 1, 90], [1, 0, 1, 1]]
    keep = torch.tensor([64, 48, 64, 50], dtype=torch.int32, device="cuda")
    for step, lq in enumerate(steps):
        T = sum(lq)
        q, k, v = _bf16((T, Hq, D), 10 * step), _bf16((T, Hkv, D), 10 * step + 1), _bf16((T, Hkv, D), 10 * step + 2)
        pos = _positions(3, T, step, 0, 5000)
        cu_q = _cu(lq)
        s.seen += cu_q[1:] - cu_q[:-1]
        lens = s.lens + (cu_q[1:] - cu_q[:-1])
        cu_k = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cumsum(lens, 0).to(torch.int32)])
        qr = s.plan.append_paged(k, v, s.kc, s.vc, s.bt, cu_q, cu_k, q=q, pos=pos, rope=s.rope)
        out, lse = s.plan.run_paged(qr, s.kc, s.vc, s.bt, cu_q, cu_k)
        s.plan.key_weights_paged(qr, s.kc, s.bt, cu_q, cu_k, lse, s.weight, decay=0.9, out=s.weight, seen=s.seen,
                                 born=s.born)
        weighed, born_then = s.weight.cpu().numpy(), s.born.cpu().numpy()
        _, _, cu_new = s.plan.evict_paged(s.weight, s.born, s.seen, keep, s.kc, s.vc, s.bt, cu_k, sink=2, recent=8)
        assert s.plan.check_error() == 0
        s.lens = cu_new[1:] - cu_new[:-1]
        # the same in 64 bits, from the rounded rotated rows the cache holds
        q64, qm = _rotate64(q, pos, s.freqs, s.axes, "half")
        _check_rotation(qr, q64, qm)
        kr = s.rope.apply(k, pos).double()
        at = 0
        for b in range(B):
            n_new = lq[b]
            for hk in range(Hkv):
                r = s.ref[b][hk]
                r["k"] = torch.cat([r["k"], kr[at:at + n_new, hk]])
                r["v"] = torch.cat([r["v"], v[at:at + n_new, hk].double()])
                r["w"] = torch.cat([r["w"] * 0.9, torch.zeros(n_new, dtype=torch.float64, device="cuda")])
                r["born"] = r["born"] + list(range(s.total[b], s.total[b] + n_new))
                n = len(r["born"])
                assert born_then[b, hk, :n].tolist() == r["born"], (step, b, hk)
                for g in range(s.G):
                    h = hk * s.G + g
                    sc = qr[at:at + n_new, h].double() @ r["k"].t() / math.sqrt(D)
                    sees = torch.arange(n, device="cuda")[None] <= (n - n_new +
                                                                    torch.arange(n_new, device="cuda"))[:, None]
                    p = torch.softmax(sc.masked_fill(~sees, -math.inf), -1)
                    o = p @ r["v"]
                    assert n_new == 0 or (out[at:at + n_new, h].double() - o).abs().max() <= 2e-2
                    r["w"] += p.sum(0)
                assert np.allclose(weighed[b, hk, :n], r["w"].cpu().numpy(), rtol=1e-4, atol=1e-6)
                kept = _evict_host(weighed[b:b + 1, hk:hk + 1], np.array(r["born"], np.int32)[None, None],
                                   s.seen[b:b + 1].cpu().numpy(), [n], [int(keep[b])], 2, 8)[0, 0][0]
                idx = torch.from_numpy(kept).cuda()
                r["k"], r["v"], r["w"] = r["k"][idx], r["v"][idx], r["w"][idx]
                r["born"] = [r["born"][i] for i in kept]
            s.total[b] += n_new
            at += n_new
        assert s.lens.cpu().tolist() == [len(s.ref[b][0]["born"]) for b in range(B)]
        assert s.seen.cpu().tolist() == s.total


def test_two_plans_on_two_streams():
    """Two plans at work at once on streams of their own give what each gives
    alone (nothing is shared between plans)."""
    def make(seed, lq, lk, Hq, max_q):
        Hkv, D = 2, 128
        q, k = _bf16((int(np.sum(lq)), Hq, D), seed), _bf16((int(np.sum(lk)), Hkv, D), seed + 1)
        pc = W.paginate(k, k, W.cu_from_lengths(lk), len(lk), 16, 4000, seed=seed)
        x = dict(plan=Plan(len(lk), 4000, Hq, Hkv, D, max_q), q=q, pc=pc, cu_q=_cu(lq), cu_k=_cu(lk),
                 lse=torch.full((q.shape[0], Hq), 9.0, device="cuda"), w=torch.zeros(len(lk), Hkv, 4000, device="cuda"),
                 born=torch.zeros(len(lk), Hkv, 4000, dtype=torch.int32, device="cuda"),
                 seen=torch.tensor(lk, dtype=torch.int32, device="cuda"), wo=torch.zeros(len(lk), Hkv, 4000, device="cuda"),
                 bo=torch.zeros(len(lk), Hkv, 4000, dtype=torch.int32, device="cuda"),
                 keep=torch.full((len(lk),), 500, dtype=torch.int32, device="cuda"),
                 cu_new=torch.zeros(len(lk) + 1, dtype=torch.int32, device="cuda"))
        return x

    def run(x):
        x["plan"].key_weights_paged(x["q"], x["pc"].k_cache, x["pc"].block_table, x["cu_q"], x["cu_k"], x["lse"],
                                    out=x["w"], seen=x["seen"], born=x["born"])
        x["plan"].evict_paged(x["w"], x["born"], x["seen"], x["keep"], x["pc"].k_cache, x["pc"].v_cache,
                              x["pc"].block_table, x["cu_k"], recent=10, weight_out=x["wo"], born_out=x["bo"],
                              cu_k_out=x["cu_new"])

    args = [(1, [700, 30], [3900, 2000], 16, 700), (2, [1, 1, 1], [4000, 1200, 7], 8, 1)]
    alone = []
    for a in args:
        x = make(*a)
        run(x)
        torch.cuda.synchronize()
        alone.append((x["w"].clone(), x["bo"].clone(), x["pc"].k_cache.clone()))
    both = [make(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for x, s in zip(both, streams):
        with torch.cuda.stream(s):
            run(x)
    torch.cuda.synchronize()
    for x, (w, bo, kc) in zip(both, alone):
        assert x["plan"].check_error() == 0
        assert torch.equal(x["w"], w) and torch.equal(x["bo"], bo) and torch.equal(_bits(x["pc"].k_cache), _bits(kc))


def test_first_calls_inside_a_capture():
    """Nothing is set up by a first call: a fresh process may make it while
    capturing (the plan was made before)."""
    import subprocess
    import sys
    code = """
import torch
from varlen_gqa_split_b200 import Plan, Rope, rope_table
plan, rope = Plan(1, 64, 4, 2, 64, 2), Rope(64, *rope_table(32))
x, k = (torch.ones(2, h, 64, dtype=torch.bfloat16, device='cuda') for h in (4, 2))
out, q_out = torch.zeros_like(x), torch.zeros_like(x)
pos = torch.tensor([[1, 2]], dtype=torch.int32, device='cuda')
kc, vc = (torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device='cuda') for _ in range(2))
bt = torch.arange(4, dtype=torch.int32, device='cuda')[None]
cu, lse = torch.tensor([0, 2], dtype=torch.int32, device='cuda'), torch.zeros(2, 4, device='cuda')
w, born = torch.zeros(1, 2, 64, device='cuda'), torch.zeros(1, 2, 64, dtype=torch.int32, device='cuda')
seen, keep = (torch.tensor([n], dtype=torch.int32, device='cuda') for n in (2, 1))
cu_new = torch.zeros_like(cu)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    rope.apply(x, pos, out)
    plan.append_paged(k, k, kc, vc, bt, cu, cu, q=x, pos=pos, rope=rope, q_out=q_out)
    plan.key_weights_paged(q_out, kc, bt, cu, cu, lse, out=w, seen=seen, born=born)
    plan.evict_paged(w, born, seen, keep, kc, vc, bt, cu, cu_k_out=cu_new)
g.replay()
torch.cuda.synchronize()
assert torch.equal(out, q_out) and out.float().abs().sum() > 0 and cu_new.tolist() == [0, 1]
assert plan.check_error() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                       cwd=W.__file__.rsplit("/", 1)[0])
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("max_q,Hq", [(1, 8), (12, 32)])
def test_captured_step_replays_with_new_lengths(max_q, Hq):
    """One graph of append, attention, weights and eviction on a side stream,
    replayed while lengths, inputs and tables change in place; equal to the
    same calls made one by one, bit for bit but for the attention output."""
    B, Hkv, D, s_max, page = 5, 2, 128, 640, 16
    rng = np.random.default_rng(5)
    rope = Rope(D, *rope_table(64, (32, 16, 16)))
    plan, plan2 = (Plan(B, s_max, Hq, Hkv, D, max_q, deterministic=1) for _ in range(2))
    T = B * max_q
    st = [dict(q=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
               k=torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda"),
               v=torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda"),
               pos=torch.zeros(3, T, dtype=torch.int32, device="cuda"),
               kc=torch.zeros(B * 40 + 3, page, Hkv, D, dtype=torch.bfloat16, device="cuda"),
               vc=torch.zeros(B * 40 + 3, page, Hkv, D, dtype=torch.bfloat16, device="cuda"),
               bt=torch.zeros(B, 40, dtype=torch.int32, device="cuda"),
               cu_q=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
               cu_k=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
               qo=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
               out=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
               lse=torch.zeros(T, Hq, device="cuda"), w=torch.zeros(B, Hkv, s_max, device="cuda"),
               born=torch.zeros(B, Hkv, s_max, dtype=torch.int32, device="cuda"),
               seen=torch.zeros(B, dtype=torch.int32, device="cuda"),
               keep=torch.zeros(B, dtype=torch.int32, device="cuda"),
               cu_new=torch.zeros(B + 1, dtype=torch.int32, device="cuda")) for _ in range(2)]

    def step(plan, x):
        plan.append_paged(x["k"], x["v"], x["kc"], x["vc"], x["bt"], x["cu_q"], x["cu_k"], q=x["q"], pos=x["pos"],
                          rope=rope, q_out=x["qo"])
        plan.run_paged(x["qo"], x["kc"], x["vc"], x["bt"], x["cu_q"], x["cu_k"], x["out"], x["lse"])
        plan.key_weights_paged(x["qo"], x["kc"], x["bt"], x["cu_q"], x["cu_k"], x["lse"], x["w"], decay=0.5, out=x["w"],
                               seen=x["seen"], born=x["born"])
        plan.evict_paged(x["w"], x["born"], x["seen"], x["keep"], x["kc"], x["vc"], x["bt"], x["cu_k"], sink=1, recent=4,
                         cu_k_out=x["cu_new"])

    def fill(n):
        lk = rng.integers(0, s_max, B, endpoint=True)
        lk[n % B] = [0, s_max, 1, 2, 300][n % 5]
        lq = np.minimum(rng.integers(0, max_q, B, endpoint=True), lk)
        perm = rng.permutation(B * 40 + 3)[:B * 40].reshape(B, 40)
        new = dict(q=_bf16((T, Hq, D), n), k=_bf16((T, Hkv, D), n + 100), v=_bf16((T, Hkv, D), n + 200),
                   pos=_positions(3, T, n, 0, 1 << 16), kc=_bf16((B * 40 + 3, page, Hkv, D), n + 300),
                   vc=_bf16((B * 40 + 3, page, Hkv, D), n + 400), bt=torch.from_numpy(perm.astype(np.int32)).cuda(),
                   cu_q=_cu(lq), cu_k=_cu(lk), w=torch.rand(B, Hkv, s_max, generator=_gen(n), device="cuda"),
                   born=torch.arange(s_max, dtype=torch.int32, device="cuda").expand(B, Hkv, s_max),
                   seen=torch.from_numpy(lk).int().cuda(),
                   keep=torch.from_numpy(rng.integers(0, s_max, B)).int().cuda())
        for x in st:
            for key, t in new.items():
                x[key].copy_(t)
            for key in ("qo", "out", "lse"):
                x[key].zero_()

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(plan, st[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(plan, st[0])
    for n in range(1, 8):
        fill(n)
        graph.replay()
        step(plan2, st[1])
        torch.cuda.synchronize()
        assert plan.check_error() == 0 and plan2.check_error() == 0
        for key in ("qo", "w", "born", "cu_new", "lse", "out"):
            assert torch.equal(st[0][key], st[1][key]), (n, key)
        assert torch.equal(_bits(st[0]["kc"]), _bits(st[1]["kc"])) and torch.equal(_bits(st[0]["vc"]), _bits(st[1]["vc"]))
