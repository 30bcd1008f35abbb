"""GPU tests of serving from a paged cache (page tables and slot maps, rotary
positions with several axes, the append, decode attention) against plain
implementations in 64 bits, and of the four together after a prefill.

Tolerances, derived (u = 2^-11 for fp16, 2^-8 for bf16, half a step relative):
  rope: the reduced angle and its sine and cosine are within 2^-20 in all; x and
    y enter twice: |err| <= u |out| + 2^-19 (|x| + |y|), and half of fp16's
    smallest step, 2^-25.
  decode, with A = sum p |v| / l of the row: u |o| for the output, u A for P's
    rounding, and 2^-25 sum |v| / l where fp16 P is subnormal; a score is off by
    at most E = d 2^-24 max_t sm_scale sum |q k_t| (one rounding a product of
    the sum), which moves o by at most 2 E A, and exp2 and the scales' products
    by 2^-20 A.  lse: E + 2^-20 (1 + |lse|)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F64 = torch.float64


@pytest.fixture(scope="module")
def sage():
    import quantized_attention_08_b200 as s
    s.load_library()
    return s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def same_bits(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and bool(
        (a.contiguous().view(torch.uint8) == b.contiguous().view(torch.uint8)).all())


# ------------------------------------------------------------------- slots
def plain_slots(ctx, new, free, used, table, P, T):
    """The same, request by request and token by token."""
    B, width = len(ctx), table.shape[1]
    table = table.copy()
    used = min(max(used, 0), len(free))
    lens, cu, slots, pos, ids = [], [0], [], [], []
    for b in range(B):
        c = min(max(ctx[b], 0), width * P)
        n = min(max(new[b], 0), width * P - c, T - len(slots))
        held = -(-c // P)
        lost = c + n
        for i in range(held, -(-(c + n) // P)):
            if used < len(free):
                table[b, i] = free[used]
                used += 1
            else:
                table[b, i] = -1
                lost = min(lost, i * P)
        for t in range(c, c + n):
            page = int(table[b, t // P])
            slots.append(page * P + t % P if page >= 0 else -1)
            pos.append(t)
            ids.append(b)
        lens.append(lost)
        cu.append(len(slots))
    pad = [-1] * (T - len(slots))
    return lens, cu, slots + pad, pos + pad, ids + pad, used, table


@pytest.mark.parametrize("B,P,T,free_n,top_ctx,top_new", [
    (1, 16, 1, 4, 40, 1), (3, 16, 40, 40, 100, 20), (7, 48, 300, 100, 200, 80), (64, 64, 64, 70, 900, 1),
    (33, 16, 500, 20, 64, 30),      # the free list runs out
    (40, 32, 256, 500, 100, 40),    # more tokens than places
    (1500, 16, 4000, 4000, 40, 4),  # more requests than threads
    (8192, 16, 9000, 9000, 20, 2), (2, 128, 30000, 400, 1000, 16000), (5, 16, 0, 9, 30, 3)])
def test_slots(sage, B, P, T, free_n, top_ctx, top_new):
    r = np.random.default_rng(B * 1000 + P + T)
    ctx = r.integers(0, top_ctx + 1, B)
    new = r.integers(0, top_new + 1, B)
    if B > 4:
        ctx[1], new[2], new[3] = 0, 0, -5
    width = -(-(top_ctx + top_new) // P)
    if B > 6:
        ctx[4] = width * P  # a full row
    held = [-(-int(c) // P) for c in ctx]
    ids = r.permutation(sum(held) + free_n + 3).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    free, used = ids[at:at + free_n], 2
    want = plain_slots(ctx.tolist(), new.tolist(), free.tolist(), used, table, P, T)
    for again in range(2):  # written again, the same result
        tt = torch.from_numpy(table).cuda()
        got = sage.sage_kv_slots(ints(ctx.tolist()), ints(new.tolist()), torch.from_numpy(free).cuda(), ints([used]),
                                 tt, page_size=P, T=T)
        for name, g, w in zip(("seq_lens", "cu", "slots", "positions", "seq_ids", "used"), got, want):
            assert g.cpu().numpy().tolist() == np.atleast_1d(w).tolist(), name
        assert np.array_equal(tt.cpu().numpy(), want[6])


@pytest.mark.parametrize("B,T", [(3, 900), (700, 3000), (64, 64), (2000, 20000)])
def test_slots_in_place(sage, B, T):
    """seq_lens over ctx_lens and the free list's count over itself."""
    r = np.random.default_rng(B)
    ctx, new = r.integers(0, 60, B), r.integers(0, 2 * T // B, B)
    P, width = 16, 200
    held = [-(-int(c) // P) for c in ctx]
    table = np.full((B, width), -7, np.int32)
    ids = r.permutation(sum(held) + B + T).astype(np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    free = ids[at:]
    want = plain_slots(ctx.tolist(), new.tolist(), free.tolist(), 1, table, P, T)
    lens, used, tt = ints(ctx.tolist()), ints([1]), torch.from_numpy(table).cuda()
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    got = sage.sage_kv_slots(lens, ints(new.tolist()), torch.from_numpy(free).cuda(), used, tt, page_size=P, T=T,
                             out=(lens, e(B + 1), e(T), e(T), e(T), used))
    for g, w in zip(got, want):
        assert g.cpu().numpy().tolist() == np.atleast_1d(w).tolist()
    assert np.array_equal(tt.cpu().numpy(), want[6])


def test_slots_in_place_replayed(sage):
    """A captured decode step whose lengths and free list advance in place."""
    B, P, steps = 5, 16, 40
    lens, one, used = ints([0, 15, 16, 31, 3]), ints([1] * B), ints([0])
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(100, 140, dtype=torch.int32, device="cuda")
    table[:, :2] = torch.arange(10, device="cuda").reshape(B, 2).to(torch.int32)
    out = (lens, ints([0] * (B + 1)), ints([0] * 8), ints([0] * 8), ints([0] * 8), used)
    start = lens.tolist()
    run = lambda: sage.sage_kv_slots(lens, one, free, used, table, page_size=P, T=8, out=out)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for n in range(2, steps + 1):
        g.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [x + n for x in start]
        pages = table.gather(1, ((lens - 1) // P)[:, None].long())[:, 0]
        assert out[2][:B].tolist() == (pages * P + (lens - 1) % P).tolist()
        assert out[2][B:].tolist() == [-1] * 3
    held = [-(-x // P) for x in start]
    assert used.tolist() == [sum(-(-(x + steps) // P) - h for x, h in zip(start, held))]
    rows = [table[b, held[b]:-(-(start[b] + steps) // P)].tolist() for b in range(B)]
    assert len({p for r in rows for p in r}) == used.item()  # no page twice


# -------------------------------------------------------------------- rope
def plain_rope(x, pos, inv, sections, pairing):
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(x.device)
    th = pos.to(F64)[axis].permute(1, 2, 0) * inv.to(F64)
    c, s = torch.cos(th)[:, None], torch.sin(th)[:, None]
    R = inv.numel()
    y = x.to(F64)
    out, size = y.clone(), torch.zeros_like(y)
    if pairing == "half":
        i, j = slice(0, R), slice(R, 2 * R)
    else:
        i, j = slice(0, 2 * R, 2), slice(1, 2 * R, 2)
    out[..., i], out[..., j] = y[..., i] * c - y[..., j] * s, y[..., j] * c + y[..., i] * s
    size[..., i] = size[..., j] = y[..., i].abs() + y[..., j].abs()
    return out, size


def check_rope(out, x, pos, inv, sections, pairing):
    want, size = plain_rope(x, pos, inv, sections, pairing)
    err = (out.to(F64) - want).abs()
    assert bool((err <= U[x.dtype] * want.abs() + 2.0 ** -19 * size + 2.0 ** -25).all()), float(err.max())
    R = inv.numel()
    assert same_bits(out[..., 2 * R:], x[..., 2 * R:])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("B,H,Hk,N,d,sections,top", [
    (1, 4, 4, 1, 64, [32], 10), (3, 8, 2, 1, 128, [16, 24, 24], 1 << 20), (2, 5, 1, 33, 64, [8, 12, 12], 5000),
    (1, 3, 3, 257, 128, [20, 20, 24], 300), (2, 4, 2, 65, 128, [1, 3, 4, 8], 2 ** 31 - 1), (1, 40, 8, 129, 64, [0, 16], 70)])
def test_rope(sage, dtype, pairing, B, H, Hk, N, d, sections, top):
    g = gen(B + N)
    q = (3 * torch.randn(B, H, N, d, generator=g, device="cuda")).to(dtype)
    k = (3 * torch.randn(B, Hk, N, d, generator=g, device="cuda")).to(dtype)
    pos = torch.randint(-top // 2 if top < 1000 else 0, top, (len(sections), B, N), generator=g, device="cuda").to(torch.int32)
    inv = torch.cat([10000.0 ** (-torch.arange(n, device="cuda") / max(n, 1)) for n in sections]).float()
    q0, k0 = q.clone(), k.clone()
    qo, ko = sage.sage_rope_axes(q, k, pos, inv, sections, pairing=pairing)
    assert same_bits(q, q0) and same_bits(k, k0)
    check_rope(qo, q, pos, inv, sections, pairing)
    check_rope(ko, k, pos, inv, sections, pairing)
    # in place, without K, tokens first ([B, N, H, d] seen as [B, H, N, d])
    t = q.transpose(1, 2).clone(memory_format=torch.contiguous_format).transpose(1, 2)
    sage.sage_rope_axes(t, None, pos, inv, sections, pairing=pairing, q_out=t)
    assert same_bits(t, qo)
    if B == 1:  # [H, N, d] with positions shared
        a, b = sage.sage_rope_axes(q[0], k[0], pos[:, 0], inv, sections, pairing=pairing)
        assert same_bits(a, qo[0]) and same_bits(b, ko[0])


def test_rope_matches_fused_prepass(sage):
    """Rotating first and quantizing after equals the fused rotary pre-pass on
    tables of the same angles, up to codes next to a rounding border."""
    H, N, d = 4, 384, 64
    g = gen(5)
    q = torch.randn(1, H, N, d, generator=g, device="cuda").half()
    k = torch.randn(1, H, N, d, generator=g, device="cuda").half()
    pos = torch.stack([torch.arange(N, device="cuda") // 64, torch.arange(N, device="cuda") % 64]).to(torch.int32)
    inv = torch.cat([10000.0 ** (-torch.arange(16, device="cuda") / 16)] * 2).float()
    th = torch.cat([pos[0].to(F64)[:, None] * inv[:16].to(F64), pos[1].to(F64)[:, None] * inv[16:].to(F64)], 1)
    fused = sage.sage_smooth_quant_qkv_rope(q, k, th.cos().float(), th.sin().float())
    qr, kr = sage.sage_rope_axes(q, k, pos, inv, [16, 16])
    plain = sage.sage_smooth_quant_qkv(qr, kr)
    for a, b in zip(fused[:2], plain[:2]):
        diff = (a.int() - b.int()).abs()
        assert int(diff.max()) <= 1 and float((diff > 0).float().mean()) < 2e-3
    for a, b in zip(fused[2:4], plain[2:4]):
        assert bool(((a - b).abs() <= 2.0 ** -10 * b).all())


# ------------------------------------------------------------------ append
def fl32(x):
    """fp64 rounded to fp32 and back."""
    return x.float().to(F64)


def plain_codes(x, top):
    """Scales and quotients of rows x (fp64 values of fp32 numbers), each
    operation rounded to fp32 (a 64-bit product or quotient of two fp32
    numbers, rounded to fp32, is theirs)."""
    delta = fl32(x.abs().amax(-1) * float(np.float32(1) / np.float32(top)))
    delta = torch.where(delta < 2.0 ** -100, torch.zeros_like(delta), delta)
    y = torch.where(delta[..., None] > 0, fl32(x / delta[..., None]), torch.zeros_like(x))
    return delta, y


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,Hk,P,mean", [(1, 1, 16, False), (37, 3, 48, True), (300, 2, 64, True), (129, 8, 16, False)])
def test_append(sage, dtype, fmt, d, T, Hk, P, mean):
    g = gen(T + d)
    B = 3
    pages = -(-T // P) + 3
    k = (torch.randn(Hk, T, d, generator=g, device="cuda") + 3 * torch.randn(Hk, 1, d, generator=g, device="cuda")).to(dtype)
    v = torch.randn(Hk, T, d, generator=g, device="cuda").to(dtype)
    k[0, 0], v[-1, -1] = 0, 0
    v[0, T // 2, ::3] = -0.0
    if dtype == torch.bfloat16:
        k[-1, -1] *= 2.0 ** -110  # scales that count as zero, and subnormal values
        v[0, 0] *= 2.0 ** -125
    else:
        v[0, 0] *= 2.0 ** -14
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 20:
        slots[3], slots[4], slots[5] = -1, pages * P, 2 ** 31 - 1
    c = sage.SageKVCache.allocate(pages, Hk, P, d, fmt, dtype)
    parts = {n: t for n, t in (("k", c.k), ("v", c.v), ("k_scale", c.k_scale), ("v_scale", c.v_scale)) if t is not None}
    for t in parts.values():
        t.view(torch.uint8).fill_(0x5a)
    kw = {}
    x = k.to(F64)
    live = (slots >= 0) & (slots < pages * P)
    if mean:
        ids = torch.randint(0, B, (T,), generator=g, device="cuda").to(torch.int32)
        ids[6], ids[7] = -1, B
        live[6:8] = False
        m = torch.randn(B, Hk, d, generator=g, device="cuda")
        kw = dict(mean_k=m, seq_ids=ids)
        x = fl32(x - m.to(F64)[ids.clamp(0, B - 1).long()].transpose(0, 1))
    # tokens first: strides differ from the dense layout's
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)
    sage.sage_kv_append(kt, v, slots, c, **kw)
    at = slots[live].long()
    untouched = torch.ones(pages * P, dtype=torch.bool, device="cuda")
    untouched[at] = False
    for name, t in parts.items():  # the other slots are left as they were
        flat = t.transpose(1, 2).reshape(pages * P, -1)[untouched]
        assert bool((flat.contiguous().view(torch.uint8) == 0x5a).all()), name
    rows = lambda t: t.transpose(1, 2).reshape(pages * P, Hk, *t.shape[3:])[at].transpose(0, 1)  # noqa: E731
    x, w = x[:, live], v.to(F64)[:, live]
    if fmt == "16":
        assert same_bits(rows(c.k), x.to(dtype) if mean else k[:, live])
    else:
        delta, y = plain_codes(x, 127)
        assert same_bits(rows(c.k_scale), delta.float())
        assert same_bits(rows(c.k), torch.round(y).to(torch.int8))
    if fmt == "8+8":
        delta, y = plain_codes(w, 448)
        assert same_bits(rows(c.v_scale), delta.float())
        y = torch.where(w == 0, torch.zeros_like(y), y)  # a zero of either sign is code 0
        assert same_bits(rows(c.v), y.float().to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        assert same_bits(rows(c.v), v[:, live])


# ------------------------------------------------------------------ decode
def filled_cache(sage, lens, Hk, P, d, fmt, dtype, seed, spare=2, scale_v=1.0, garbage=True):
    """A cache whose requests hold `lens` tokens on shuffled pages, the 64-bit
    K and V that it stands for, and its table.  Everything that no request
    holds is garbage: NaN, -128, E4M3's NaN, and page numbers far outside."""
    g = gen(seed)
    held = [-(-n // P) for n in lens]
    pages = sum(held) + spare
    c = sage.SageKVCache.allocate(pages, Hk, P, d, fmt, dtype)
    width = max(held + [1]) + 1
    table = torch.full((len(lens), width), 2 ** 31 - 5 if garbage else -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    T = sum(lens)
    bias = torch.randn(Hk, 1, d, generator=g, device="cuda")
    k = (torch.randn(Hk, T, d, generator=g, device="cuda") + bias).to(dtype)
    v = (scale_v * torch.randn(Hk, T, d, generator=g, device="cuda")).to(dtype)
    if garbage:
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.view(torch.uint8).fill_(0xff if t.dtype != torch.int8 else 0x80)
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :held[b]] = perm[at:at + held[b]]
        pos = torch.arange(n, device="cuda")
        slots.append(table[b, pos // P].long() * P + pos % P)
        at += held[b]
    slots = torch.cat(slots).to(torch.int32)
    sage.sage_kv_append(k, v, slots, c)
    s = slots.long()
    rows = lambda t: t.transpose(1, 2).reshape(pages * P, Hk, *t.shape[3:])[s].transpose(0, 1)  # noqa: E731
    K, V = rows(c.k).to(F64), rows(c.v)
    if fmt != "16":
        K = K * rows(c.k_scale).to(F64)[..., None]
    V = V.view(torch.float8_e4m3fn).to(F64) * rows(c.v_scale).to(F64)[..., None] if fmt == "8+8" else V.to(F64)
    return c, table, K, V


def plain_decode(q, K, V, lens, causal, scale, dropped=None):
    """(o, lse, tolerance of o, tolerance of lse) in 64 bits.  dropped: {request:
    token positions that count as absent}."""
    B, H, nq, d = q.shape
    Hk, G = K.shape[0], q.shape[1] // K.shape[0]
    u = U[q.dtype]
    o = torch.zeros(q.shape, dtype=F64, device="cuda")
    tol = torch.zeros_like(o)
    lse = torch.full(q.shape[:3], -math.inf, dtype=F64, device="cuda")
    ltol = torch.zeros_like(lse)
    cu = np.concatenate([[0], np.cumsum(lens)])
    for b in range(B):
        k, v = K[:, cu[b]:cu[b + 1]], V[:, cu[b]:cu[b + 1]]
        keep = torch.ones(lens[b], dtype=torch.bool, device="cuda")
        if dropped and b in dropped:
            keep[dropped[b]] = False
        for i in range(nq):
            n = lens[b] - nq + 1 + i if causal else lens[b]
            if n <= 0 or not bool(keep[:n].any()):
                continue
            kk, vv = k[:, :n][:, keep[:n]], v[:, :n][:, keep[:n]]
            x = q[b, :, i].to(F64).reshape(Hk, G, d)
            s = scale * torch.einsum("hgd,htd->hgt", x, kk)
            E = d * 2.0 ** -24 * scale * torch.einsum("hgd,htd->hgt", x.abs(), kk.abs()).amax(-1)
            p = torch.softmax(s, -1)
            l = torch.exp(s - s.amax(-1, keepdim=True)).sum(-1)
            o[b, :, i] = torch.einsum("hgt,htd->hgd", p, vv).reshape(H, d)
            A = torch.einsum("hgt,htd->hgd", p, vv.abs())
            sub = 2.0 ** -25 * vv.abs().sum(1)[:, None] / l[..., None]
            tol[b, :, i] = (u * o[b, :, i].abs().reshape(Hk, G, d) + (u + 2 * E[..., None] + 2.0 ** -20) * A + sub +
                            2.0 ** -25).reshape(H, d)
            lse[b, :, i] = torch.logsumexp(s, -1).reshape(H)
            ltol[b, :, i] = (E + 2.0 ** -20 * (1 + lse[b, :, i].abs().reshape(Hk, G))).reshape(H)
    return o, lse, tol, ltol


def check_decode(got, want):
    (o, lse), (wo, wl, tol, ltol) = got, want
    err = (o.to(F64) - wo).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err / tol.clamp(min=1e-30)).max()))
    assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
    fin = ~torch.isneginf(wl)
    assert bool(((lse.to(F64) - wl).abs()[fin] <= ltol[fin]).all())
    assert bool((o[~fin] == 0).all())


LENS = {"tiny": [1, 0, 2, 15, 16, 17, 3], "ragged": [1, 500, 0, 64, 1023, 129, 33, 0], "one": [1], "long": [4099]}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("H,Hk,P", [(4, 4, 16), (8, 2, 64), (24, 3, 48)])
def test_decode(sage, dtype, fmt, d, lens, H, Hk, P):
    lens = LENS[lens]
    c, table, K, V = filled_cache(sage, lens, Hk, P, d, fmt, dtype, seed=H + P)
    q = (torch.randn(len(lens), H, d, generator=gen(3), device="cuda") * 1.5).to(dtype)
    got = sage.sage_attn_decode_paged(q, c, table, ints(lens), max(lens), return_lse=True)
    want = plain_decode(q[:, :, None], K, V, lens, True, 1 / math.sqrt(d))
    check_decode((got[0][:, :, None], got[1][:, :, None]), want)
    again = sage.sage_attn_decode_paged(q, c, table, ints(lens), max(lens), return_lse=True)
    assert same_bits(got[0], again[0]) and same_bits(got[1], again[1])


@pytest.mark.parametrize("dtype,fmt,d", [(torch.float16, "16", 128), (torch.bfloat16, "8+8", 128), (torch.float16, "8+8", 64),
                                         (torch.bfloat16, "B", 64)])
@pytest.mark.parametrize("nq,H,Hk", [(2, 4, 4), (3, 10, 2), (4, 8, 2), (5, 16, 1), (16, 4, 1), (8, 40, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_decode_several_tokens(sage, dtype, fmt, d, nq, H, Hk, causal):
    """Rows of one to many tiles; requests shorter than their query tokens."""
    lens = [nq, 1, 0, 200, 33, 1030, nq - 1]
    c, table, K, V = filled_cache(sage, lens, Hk, 32, d, fmt, dtype, seed=nq)
    q = torch.randn(len(lens), H, nq, d, generator=gen(4), device="cuda").to(dtype)
    got = sage.sage_attn_decode_paged(q, c, table, ints(lens), 1056, causal=causal, sm_scale=0.2, return_lse=True)
    check_decode(got, plain_decode(q, K, V, lens, causal, 0.2))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,H,Hk,P", [(1, 4, 4, 48), (1, 20, 4, 32), (5, 20, 4, 16)])
def test_decode_batch_on_one_line(sage, dtype, fmt, d, nq, H, Hk, P):
    """Requests enough that all segments share one line of steps; some empty,
    some of one token, one much longer than the rest."""
    r = np.random.default_rng(nq + P)
    lens = [int(x) for x in r.integers(0, 300, 44)] + [0, 1, 2000, 0, 15, 16, 17]
    c, table, K, V = filled_cache(sage, lens, Hk, P, d, fmt, dtype, seed=nq)
    q = torch.randn(len(lens), H, nq, d, generator=gen(5), device="cuda").to(dtype)
    assert sage.sage_attn_decode_workspace_bytes(len(lens), H, Hk, nq, d, 2000, fmt) > 0
    got = sage.sage_attn_decode_paged(q, c, table, ints(lens), 2000, return_lse=True)
    check_decode(got, plain_decode(q, K, V, lens, True, 1 / math.sqrt(d)))
    again = sage.sage_attn_decode_paged(q, c, table, ints(lens), 2000, return_lse=True)
    assert same_bits(got[0], again[0]) and same_bits(got[1], again[1])


@pytest.mark.parametrize("B,n,Hk", [(200, 90, 4), (300, 700, 2), (3, 20000, 1), (1, 66000, 2)])
def test_decode_many_and_long(sage, B, n, Hk):
    """Stretches of several segments, and segments of many stretches."""
    r = np.random.default_rng(B)
    lens = [n] + [int(x) for x in r.integers(0, n + 1, B - 1)]
    c, table, K, V = filled_cache(sage, lens, Hk, 16, 64, "8+8", torch.float16, seed=B)
    q = torch.randn(B, Hk * 2, 1, 64, generator=gen(6), device="cuda").half()
    got = sage.sage_attn_decode_paged(q, c, table, ints(lens), n, return_lse=True)
    check_decode(got, plain_decode(q, K, V, lens, True, 0.125))


def test_decode_largest_batch(sage):
    """4096 requests, the most a call takes, and the most shared memory."""
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 200, 4095)] + [700]
    c, table, K, V = filled_cache(sage, lens, 1, 16, 64, "8+8", torch.float16, seed=12)
    q = torch.randn(4096, 2, 64, generator=gen(6), device="cuda").half()
    o, lse = sage.sage_attn_decode_paged(q, c, table, ints(lens), 700, return_lse=True)
    some = list(range(0, 4096, 97)) + [4095]
    cu = np.concatenate([[0], np.cumsum(lens)])
    keep = torch.cat([torch.arange(cu[b], cu[b + 1]) for b in some]).cuda()
    want = plain_decode(q[some][:, :, None], K[:, keep], V[:, keep], [lens[b] for b in some], True, 0.125)
    check_decode((o[some][:, :, None], lse[some][:, :, None]), want)
    empty = torch.tensor([n == 0 for n in lens], device="cuda")
    assert bool((o[empty] == 0).all()) and bool(torch.isneginf(lse[empty]).all())


def test_decode_two_streams_at_once(sage):
    """Two calls that may overlap, each with its own stream and workspace."""
    cases = []
    for seed, fmt, lens in ((1, "8+8", [30000, 200, 0, 5]), (2, "16", [9, 20000])):
        c, table, K, V = filled_cache(sage, lens, 4, 32, 128, fmt, torch.bfloat16, seed=seed)
        q = torch.randn(len(lens), 8, 1, 128, generator=gen(seed), device="cuda").bfloat16()
        cases.append((q, c, table, ints(lens), max(lens), plain_decode(q, K, V, lens, True, 128 ** -0.5)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s, (q, c, table, lens, n, _w) in zip(streams, cases):
            outs.append(sage.sage_attn_decode_paged(q, c, table, lens, n, return_lse=True, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        check_decode(o, cases[i % 2][5])
        assert same_bits(o[0], outs[i % 2][0])


def test_decode_growing_request_in_one_graph(sage):
    """One captured call, replayed while the request grows across steps, pages,
    and from one warp's work to many; stale NaN stands behind the last token."""
    n, P, d = 700, 16, 64
    c, table, K, V = filled_cache(sage, [n], 2, P, d, "16", torch.float16, seed=4)
    q = torch.randn(1, 4, 1, d, generator=gen(2), device="cuda").half()
    lens = ints([1])
    run = lambda: sage.sage_attn_decode_paged(q, c, table, lens, n, return_lse=True)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for m in (0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 255, 256, 257, 512, 699, 700):
        lens.fill_(m)
        g.replay()
        torch.cuda.synchronize()
        check_decode(out, plain_decode(q, K[:, :m], V[:, :m], [m], True, 0.125))


def test_decode_small_v_beside_large(sage):
    """Rows of V whose scales differ by 2^12: the unit that P is taken in grows in
    the middle of a request."""
    d, n = 128, 400
    c, table, K, V = filled_cache(sage, [n], 1, 16, d, "8+8", torch.bfloat16, seed=6)
    at = torch.arange(0, n // 2, device="cuda")
    pg, off = table[0, at // 16].long(), at % 16
    c.v_scale[pg, 0, off] *= 2.0 ** -12
    V[:, :n // 2] *= 2.0 ** -12
    q = torch.randn(1, 3, 1, d, generator=gen(2), device="cuda").bfloat16()
    got = sage.sage_attn_decode_paged(q, c, table, ints([n]), n, return_lse=True)
    check_decode(got, plain_decode(q, K, V, [n], True, d ** -0.5))


def test_decode_extremes(sage):
    """A score far above the rest at either end, equal scores, and small and
    large V (fp16 rows near its smallest and largest numbers)."""
    d, lens = 64, [700, 700, 700]
    for fmt in ("16", "8+8"):
        for scale_v in (1e-5, 1.0, 9000.0):
            c, table, K, V = filled_cache(sage, lens, 1, 16, d, fmt, torch.float16, seed=9, scale_v=scale_v)
            q = torch.zeros(3, 2, 1, d, dtype=torch.float16, device="cuda")
            q[1, 0, 0] = (8 * K[0, 700]).half()   # request 1's first key
            q[1, 1, 0] = (8 * K[0, 1399]).half()  # and its last
            q[2] = 40 * torch.randn(2, 1, d, generator=gen(1), device="cuda").half()
            got = sage.sage_attn_decode_paged(q, c, table, ints(lens), 700, return_lse=True)
            check_decode(got, plain_decode(q, K, V, lens, True, 0.125))


@pytest.mark.parametrize("n", [40, 3000])
def test_decode_bad_pages_and_lengths(sage, n):
    """Pages outside the cache count as absent; lengths are cut to [0, max_len]."""
    P, lens = 16, [n, n, n, n]
    c, table, K, V = filled_cache(sage, lens, 2, P, 128, "16", torch.float16, seed=2)
    held = -(-n // P)
    table[0, 1], table[1, held - 1], table[2, :held] = -1, c.num_pages, -1
    span = lambda i: torch.arange(i * P, min(n, i * P + P), device="cuda")  # noqa: E731
    dropped = {0: span(1), 1: span(held - 1), 2: torch.arange(n, device="cuda")}
    q = torch.randn(4, 4, 1, 128, generator=gen(8), device="cuda").half()
    want = plain_decode(q, K, V, lens, False, 128 ** -0.5, dropped)
    check_decode(sage.sage_attn_decode_paged(q, c, table, ints([n, n, n, n + 9999]), n, causal=False, return_lse=True), want)
    o, lse = sage.sage_attn_decode_paged(q, c, table, ints([-3, 0, -2 ** 31, 0]), n, return_lse=True)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())


def test_decode_strides_and_page_strides(sage):
    """K and V pages side by side in one allocation, q as a view of a fused
    projection, on a stream of its own."""
    B, H, Hk, P, d, pages = 3, 8, 2, 32, 128, 40
    g = gen(11)
    kv = torch.randn(pages, 2, Hk, P, d, generator=g, device="cuda").half()
    c = sage.SageKVCache(kv[:, 0], kv[:, 1])
    lens = [700, 65, 31]
    table = torch.randperm(pages, generator=g, device="cuda")[:B * 12].reshape(B, 12).to(torch.int32).repeat(1, 2)
    fused = torch.randn(B, H + 2 * Hk, d, generator=g, device="cuda").half()
    q = fused[:, :H]
    pg = [table[b, :-(-n // P)].long() for b, n in enumerate(lens)]
    K, V = (torch.cat([kv[p, i].transpose(0, 1).reshape(Hk, -1, d)[:, :n] for p, n in zip(pg, lens)], 1).to(F64)
            for i in (0, 1))
    want = plain_decode(q[:, :, None], K, V, lens, True, d ** -0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, s.cuda_stream):
        o, lse = sage.sage_attn_decode_paged(q, c, table, ints(lens), 700, return_lse=True, stream=stream)
        torch.cuda.synchronize()
        check_decode((o[:, :, None], lse[:, :, None]), want)


def test_decode_offsets_past_32_bits(sage):
    """Pages whose first byte lies beyond 2^32 of the cache."""
    P, Hk, d = 64, 8, 128
    pages = (1 << 31) // (P * Hk * d) + 40  # elements past 2^31, bytes past 2^32
    k = torch.empty(pages, Hk, P, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[-20:], v[-20:] = (torch.randn(20, Hk, P, d, generator=gen(i), device="cuda").bfloat16() for i in (1, 2))
    c = sage.SageKVCache(k, v)
    lens = [20 * P - 5]
    table = (pages - 1 - torch.arange(20, device="cuda"))[None].to(torch.int32).contiguous()
    # the last token goes through the append
    new = torch.randn(2, Hk, 1, d, generator=gen(3), device="cuda").bfloat16()
    slot = table[0, 19:20] * P + P - 6
    sage.sage_kv_append(new[0], new[1], slot.contiguous(), c)
    K, V = (x[table[0].long()].transpose(0, 1).reshape(Hk, -1, d)[:, :lens[0]].to(F64) for x in (k, v))
    assert torch.equal(K[:, -1].bfloat16(), new[0][:, 0])
    q = torch.randn(1, 32, 1, d, generator=gen(4), device="cuda").bfloat16()
    got = sage.sage_attn_decode_paged(q, c, table, ints(lens), lens[0], return_lse=True)
    check_decode(got, plain_decode(q, K, V, lens, True, d ** -0.5))


def test_decode_two_graphs_share_a_workspace(sage):
    """Two captured calls of different sizes on one workspace, replayed in turn
    over a workspace full of NaN."""
    cases = []
    for seed, lens in ((1, [40000, 17]), (2, [64, 33000, 5, 0])):
        c, table, K, V = filled_cache(sage, lens, 2, 16, 64, "B", torch.float16, seed=seed)
        q = torch.randn(len(lens), 6, 1, 64, generator=gen(seed), device="cuda").half()
        cases.append((q, c, table, ints(lens), max(lens), plain_decode(q, K, V, lens, True, 0.125)))
    need = max(sage.sage_attn_decode_workspace_bytes(q.shape[0], 6, 2, 1, 64, n, "B") for q, _, _, _, n, _ in cases)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for q, c, table, lens, n, _ in cases:
        run = lambda: sage.sage_attn_decode_paged(q, c, table, lens, n, return_lse=True, workspace=ws)  # noqa: E731
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), case in zip(graphs, cases):
            ws.fill_(0xff)
            out[0].fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            check_decode(out, case[5])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("fmt", ["16", "8+8"])
def test_prefill_then_decode_steps(sage, fmt):
    """Two prompts through the packed prefill (its mean_k smooths the cache's
    K), then decode steps of slots -> rope -> append -> attention, each
    against 64-bit attention over the request's whole history."""
    d, H, Hk, P, B, steps = 64, 8, 2, 16, 2, 20
    prompt, dtype, g = [45, 130], torch.float16, gen(21)
    T0 = sum(prompt)
    sections = [8, 12, 12]
    inv = torch.cat([10000.0 ** (-torch.arange(n, device="cuda") / n) for n in sections]).float()
    bias = 5 * torch.randn(Hk, 1, d, generator=g, device="cuda")

    def new_tokens(n):
        q = torch.randn(H, n, d, generator=g, device="cuda").to(dtype)
        k = (torch.randn(Hk, n, d, generator=g, device="cuda") + bias).to(dtype)
        return q, k, torch.randn(Hk, n, d, generator=g, device="cuda").to(dtype)

    cache = sage.SageKVCache.allocate(32, Hk, P, d, fmt, dtype)
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(32, generator=g, device="cuda").to(torch.int32)
    lens, used = ints([0, 0]), ints([0])
    hist = [[], []]  # 64-bit (k, v) of each request
    mean = None
    for step in range(steps + 1):
        new = ints(prompt if step == 0 else [1, 1])
        T = T0 if step == 0 else 4  # decode steps are padded to four places
        lens, cu, slots, pos, ids, used = sage.sage_kv_slots(lens, new, free, used, table, page_size=P, T=T)
        q, k, v = new_tokens(T)
        q, k = sage.sage_rope_axes(q, k, torch.stack([pos, pos // 7, pos % 7]), inv, sections)
        if step == 0:
            mean = sage.sage_smooth_quant_qkv_varlen(q, k, cu, max(prompt))[4]
            o0 = sage.sage_attn_fwd_varlen(q, k, v, cu, max(prompt), causal=True, variant="B")
        sage.sage_kv_append(k, v, slots, cache, mean_k=mean, seq_ids=ids)
        c = cu.tolist()
        for b in range(B):
            hist[b].append((k[:, c[b]:c[b + 1]].to(F64), v[:, c[b]:c[b + 1]].to(F64)))
        if step == 0:
            continue
        qs = q[:, :B].transpose(0, 1)  # [B, H, d], a view
        o = sage.sage_attn_decode_paged(qs, cache, table, lens, 12 * P)
        for b in range(B):
            kk, vv = (torch.cat(x, 1) for x in zip(*hist[b]))
            s = torch.einsum("hgd,htd->hgt", qs[b].to(F64).reshape(Hk, -1, d), kk) / math.sqrt(d)
            want = torch.einsum("hgt,htd->hgd", torch.softmax(s, -1), vv).reshape(H, d)
            cos = torch.nn.functional.cosine_similarity(o[b].to(F64).flatten(), want.flatten(), dim=0)
            # the 16-bit cache rounds K, V and P; 8 bits the paper's bar for 8+8
            assert float(cos) >= (0.9999 if fmt == "16" else 0.998), (step, b, float(cos))
    assert lens.tolist() == [n + steps for n in prompt]
    # the decode kernel's row for the prompts' last tokens agrees with the prefill's
    last = torch.stack([o0[:, prompt[0] - 1], o0[:, T0 - 1]])
    assert bool(torch.isfinite(last).all())


def test_given_outputs_and_refusals(sage):
    """Outputs and workspaces that the caller brings, strides of one-entry axes,
    and what the binding refuses on the device."""
    c, table, K, V = filled_cache(sage, [40, 7], 2, 16, 64, "8+8", torch.bfloat16, seed=1)
    lens = ints([40, 7])
    q = torch.randn(2, 4, 64, generator=gen(2), device="cuda").bfloat16()
    o = torch.full_like(q, 9.0)
    got = sage.sage_attn_decode_paged(q, c, table, lens, 40, o=o)
    assert got.data_ptr() == o.data_ptr() and same_bits(got, sage.sage_attn_decode_paged(q, c, table, lens, 40))
    check_decode((got[:, :, None], plain_decode(q[:, :, None], K, V, [40, 7], True, 0.125)[1].float()),
                 plain_decode(q[:, :, None], K, V, [40, 7], True, 0.125))
    refused = [dict(q=q.half()), dict(q=q[..., :32]), dict(table=table[:1]), dict(lens=lens.long()), dict(lens=lens.cpu()),
               dict(o=o[:1]), dict(o=o.transpose(0, 1).contiguous().transpose(0, 1)), dict(max_len=1 << 31)]
    for kw in refused:
        a = dict(q=q, table=table, lens=lens, max_len=40, o=None)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            sage.sage_attn_decode_paged(a["q"], c, a["table"], a["lens"], a["max_len"], o=a["o"])
    with pytest.raises(sage.SageError) as e:
        sage.sage_attn_decode_paged(q, c, table, lens, table.shape[1] * 16 + 1)
    assert e.value.status == 1
    with pytest.raises(sage.SageError) as e:  # rows of q that are not 16-byte aligned
        sage.sage_attn_decode_paged(torch.zeros(2, 4, 68, device="cuda").bfloat16()[..., :64], c, table, lens, 40)
    assert e.value.status == 3
    k = torch.zeros(2, 3, 64, device="cuda").bfloat16()
    for kw in (dict(slots=ints([0, 1])), dict(v=k[:1]), dict(mean_k=torch.zeros(1, 2, 64, device="cuda"))):
        with pytest.raises(ValueError):
            sage.sage_kv_append(k, kw.pop("v", k), kw.pop("slots", ints([0, 1, 2])), c, **kw)
    # one token a sequence: the strides of its axis are whatever they are
    inv = torch.ones(32, device="cuda")
    pos = ints([[3, 5], [7, 9]]).t()[None, :, :1]  # [1, 2, 1], last stride 2
    x = torch.randn(2, 1, 4, 64, generator=gen(3), device="cuda").bfloat16().transpose(1, 2)
    out, none = sage.sage_rope_axes(x, None, pos, inv, [32])
    check_rope(out, x, pos, inv, [32], "half")
    assert none is None


@pytest.mark.parametrize("fmt,B,n0", [("8+8", 2, 40), ("16", 70, 30), ("8+8", 70, 120)])
def test_captured_step_equals_eager_steps(sage, fmt, B, n0):
    """A decode step -- slots in place, rope, append, attention, each on what the
    one before it wrote -- captured once and replayed, against the same steps
    issued one by one: the same tokens, cache and outputs, bit for bit.  The
    steps run back to back, so that their kernels' launches overlap."""
    d, H, Hk, P, steps, dtype = 128, 8, 2, 16, 25, torch.bfloat16
    g = gen(n0 + B)
    sections = [16, 24, 24]
    inv = torch.cat([10000.0 ** (-torch.arange(n, device="cuda") / n) for n in sections]).float()
    width, pages = 16, 16 * B
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    toks = [(rand(B, H, 1, d), rand(B, Hk, 1, d), rand(Hk, B, d)) for _ in range(steps)]
    first = (rand(Hk, B * n0, d), rand(Hk, B * n0, d))
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    mean = torch.randn(B, Hk, d, generator=g, device="cuda")

    def start():
        c = sage.SageKVCache.allocate(pages, Hk, P, d, fmt, dtype)
        s = dict(c=c, lens=ints([0] * B), used=ints([0]), table=torch.full((B, width), -1, dtype=torch.int32, device="cuda"),
                 one=ints([1] * B), cu=ints([0] * (B + 1)), slots=ints([0] * B), pos=ints([0] * B), ids=ints([0] * B),
                 q=toks[0][0].clone(), k=toks[0][1].clone(), v=toks[0][2].clone())
        lens, _, slots, _, ids, used = sage.sage_kv_slots(s["lens"], ints([n0] * B), free, s["used"], s["table"],
                                                          page_size=P, T=B * n0)
        s["lens"].copy_(lens)
        s["used"].copy_(used)
        sage.sage_kv_append(*first, slots, c, mean_k=mean, seq_ids=ids)
        return s

    def step(s):
        sage.sage_kv_slots(s["lens"], s["one"], free, s["used"], s["table"], page_size=P, T=B,
                           out=(s["lens"], s["cu"], s["slots"], s["pos"], s["ids"], s["used"]))
        pos = torch.stack([s["pos"]] * 3)[:, :, None]
        q, k = sage.sage_rope_axes(s["q"], s["k"], pos, inv, sections)
        sage.sage_kv_append(k[:, :, 0].transpose(0, 1), s["v"], s["slots"], s["c"], mean_k=mean, seq_ids=s["ids"])
        return sage.sage_attn_decode_paged(q, s["c"], s["table"], s["lens"], width * P)

    eager, want = start(), []
    for q, k, v in toks:
        for name, t in (("q", q), ("k", k), ("v", v)):
            eager[name].copy_(t)
        want.append(step(eager))
        torch.cuda.synchronize()  # one by one
    warm = start()
    step(warm)
    replayed = start()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(replayed)
    got = []
    for q, k, v in toks:
        for name, t in (("q", q), ("k", k), ("v", v)):
            replayed[name].copy_(t)
        graph.replay()
        got.append(out.clone())
    torch.cuda.synchronize()
    assert replayed["lens"].tolist() == [n0 + steps] * B
    for name in ("lens", "used", "table", "slots"):
        assert torch.equal(eager[name], replayed[name]), name
    for a, b in zip(want, got):
        assert same_bits(a, b) and bool(torch.isfinite(a).all())
    for a, b in ((eager["c"].k, replayed["c"].k), (eager["c"].v, replayed["c"].v)):
        assert same_bits(a, b)
