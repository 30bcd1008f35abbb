"""Cases, plain forms and exact values of the serving operators: page tables
and slot maps, rotary positions with several axes, the append to a paged
key-value cache, and the attention of new tokens over that cache."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
TINY = 2.0 ** -100  # scales below this count as zero (their reciprocal would leave fp32)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step of 256 requests: one new token each, most in a page they hold
        dict(name="slots_decode_b256", op="slots", B=256, page=16, max_ctx=4096, new="one", T=256),
        # admitting a step's prompts, some chunked, in a captured step of 65536 token places
        dict(name="slots_prompts_t65536", op="slots", B=512, page=16, max_ctx=1024, new="ragged", T=65536),
        # a decode step's queries and keys of a model that reads video: far (time, height, width) positions
        dict(name="rope_decode_b64", op="rope", B=64, H=32, Hk=8, N=1, d=128, sections="16,24,24",
             dtype="bf16", far=100000, pairing="half"),
        # the queries and keys of a whole video (8 frames of 64 x 64 patches)
        dict(name="rope_video_n32768", op="rope", B=1, H=16, Hk=16, N=32768, d=128, sections="16,24,24",
             dtype="fp16", far=0, pairing="half"),
        # the new tokens of a decode step, quantized into the cache
        dict(name="append_decode_t64", op="append", T=64, B=64, Hk=8, d=128, page=16, slack=64, fmt="8+8",
             dtype="fp16", mean=True),
        # the prompts of one step, of an odd total length, into a 16-bit cache
        dict(name="append_16_t17776", op="append", T=17776, B=3, Hk=16, d=64, page=32, slack=1, fmt="16",
             dtype="bf16", mean=False),
        # the longest step: 65536 prompt tokens, smoothed and quantized
        dict(name="append_8p8_t65536", op="append", T=65536, B=16, Hk=8, d=128, page=64, slack=1, fmt="8+8",
             dtype="fp16", mean=True),
        # one short conversation: latency
        dict(name="decode_b1_len1009", op="decode", B=1, H=32, Hk=8, d=128, nq=1, page=16, max_len=1009,
             ragged=False, fmt="16", dtype="fp16", causal=False),
        # one long document
        dict(name="decode_b1_len131072", op="decode", B=1, H=32, Hk=8, d=128, nq=1, page=64, max_len=131072,
             ragged=False, fmt="16", dtype="bf16", causal=False),
        # a full serving batch, lengths from one token to 8192, quantized cache
        dict(name="decode_b64_8p8", op="decode", B=64, H=32, Hk=8, d=128, nq=1, page=64, max_len=8192,
             ragged=True, fmt="8+8", dtype="fp16", causal=False),
        # one key head per query head, 64 channels, int8 K and 16-bit V
        dict(name="decode_mha_d64_B", op="decode", B=16, H=16, Hk=16, d=64, nq=1, page=16, max_len=4096,
             ragged=True, fmt="B", dtype="fp16", causal=False),
        # four drafted tokens a request checked at once
        dict(name="decode_draft4_8p8", op="decode", B=16, H=32, Hk=8, d=128, nq=4, page=32, max_len=8192,
             ragged=True, fmt="8+8", dtype="bf16", causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "rope", "append", "decode", "decode"])
    dtype = rng.choice(["fp16", "bf16"])
    page = rng.choice([16, 32, 64, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    d = rng.choice([64, 128])
    fmt = rng.choice(["16", "B", "8+8"])
    if op == "slots":
        B = _log(rng, 1, 1024)
        new = rng.choice(["one", "ragged"])
        return dict(op=op, B=B, page=page, max_ctx=_log(rng, 1, 4096), new=new,
                    T=B + rng.randrange(8) if new == "one" else _log(rng, 64, 65536))
    if op == "rope":
        H = Hk * rng.choice([1, 2, 4])
        N = 1 if rng.random() < 0.4 else _log(rng, 2, 32 * 32768 // max(32, H + Hk))
        B = max(1, min(_log(rng, 1, 512), 32 * 32768 // ((H + Hk) * N)))
        a = rng.choice([(d // 2,), (d // 4, d // 4), (d // 8, 3 * d // 16, 3 * d // 16), (d // 8, d // 8, d // 8)])
        return dict(op=op, B=B, H=H, Hk=Hk, N=N, d=d, sections=",".join(map(str, a)), dtype=dtype,
                    far=rng.choice([0, 4096, 1000000]), pairing=rng.choice(["half", "interleaved"]))
    if op == "append":
        T = _log(rng, 1, 65536 * 8 // max(Hk, 8))
        return dict(op=op, T=T, B=min(T, _log(rng, 1, 256)), Hk=Hk, d=d, page=page, slack=rng.choice([1, 2, 4]),
                    fmt=fmt, dtype=dtype, mean=rng.random() < 0.7)
    nq = rng.choice([1, 1, 1, 2, 3, 4, 8])
    B = _log(rng, 1, 128)
    return dict(op=op, B=B, H=Hk * rng.choice([1, 2, 4, 5, 8]), Hk=Hk, d=d, nq=nq, page=page,
                max_len=_log(rng, 1, max(64, 64 * 8192 * 8 // (2 * B * max(Hk, 8)))), ragged=rng.random() < 0.7,
                fmt=fmt, dtype=dtype, causal=rng.random() < 0.5)


# -------------------------------------------- lengths: part of the case, not of the seed
def _rng_of(case):
    return random.Random("%d %d" % (case["B"], case.get("max_len", case.get("max_ctx", case.get("T", 0)))))


def _lens(case):
    r = _rng_of(case)
    n = case["max_len"]
    if not case["ragged"]:
        return [n] * case["B"]
    return [n if b == 0 else r.randint(1, n) for b in range(case["B"])]


def _split(total, B, r):
    """B lengths >= 1 (where total allows) that add up to `total`."""
    if B >= total:
        return [1] * total + [0] * (B - total)
    cuts = sorted(r.sample(range(1, total), B - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _slot_lens(case):
    """(ctx, new) of a slots case."""
    r = _rng_of(case)
    ctx = [r.randint(0, case["max_ctx"]) for _ in range(case["B"])]
    if case["new"] == "one":
        return ctx, [1] * case["B"]
    used = max(1, case["T"] - r.randint(0, case["T"] // 64))  # a captured step is seldom full
    return [c if r.random() < 0.5 else 0 for c in ctx], _split(used, case["B"], r)


def _pages(n, P):
    return -(-n // P)


def work(case):
    op = case["op"]
    if op == "slots":
        ctx, new = _slot_lens(case)
        P = case["page"]
        got = sum(_pages(c + n, P) - _pages(c, P) for c, n in zip(ctx, new))
        part = sum(c % P != 0 for c in ctx)  # a partly filled page's entry is read
        return {"bytes": 16 * case["B"] + 8 * got + 4 * part + 12 * case["T"] + 12, "flops": 0}
    if op == "rope":
        n = case["B"] * (case["H"] + case["Hk"]) * case["N"] * case["d"]
        axes = len(case["sections"].split(","))
        return {"bytes": 4 * n + 4 * axes * case["B"] * case["N"], "flops": 3 * n}
    if op == "append":
        n = case["T"] * case["Hk"]
        out = {"16": 4 * case["d"], "B": 3 * case["d"] + 4, "8+8": 2 * case["d"] + 8}[case["fmt"]]
        mean = 4 * case["B"] * case["Hk"] * case["d"] + 4 * case["T"] if case["mean"] else 0
        return {"bytes": n * (4 * case["d"] + out) + 4 * case["T"] + mean, "flops": 6 * n * case["d"]}
    lens = _lens(case)
    row = {"16": 4 * case["d"], "B": 3 * case["d"] + 4, "8+8": 2 * case["d"] + 8}[case["fmt"]]
    rows = case["B"] * case["H"] * case["nq"]
    return {"bytes": sum(lens) * case["Hk"] * row + rows * (4 * case["d"] + 4) +
            4 * case["B"] + 4 * sum(_pages(n, case["page"]) for n in lens),
            "flops": 4 * sum(lens) * case["H"] * case["nq"] * case["d"]}


# ---------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _k_like(shape, g, bias_axes):
    """N(0, 1) plus a per-channel bias N(0, 4) with a few channels at +30."""
    x = torch.randn(shape, generator=g, device="cuda")
    bshape = [n if i in bias_axes else 1 for i, n in enumerate(shape)]
    bias = 2.0 * torch.randn(bshape, generator=g, device="cuda")
    bias[..., torch.randperm(shape[-1], generator=g, device="cuda")[:4]] += 30.0
    return x + bias, bias


def _quant_k(x):
    """int8 codes and fp32 scales of rows x (fp32), as the cache holds them."""
    delta = x.abs().amax(-1) / 127.0
    delta = torch.where(delta < TINY, torch.zeros_like(delta), delta)
    codes = torch.round(x / delta[..., None])
    return torch.where(delta[..., None] == 0, torch.zeros_like(codes), codes).to(torch.int8), delta


def _quant_v(x):
    delta = x.abs().amax(-1) / 448.0
    delta = torch.where(delta < TINY, torch.zeros_like(delta), delta)
    codes = torch.where(delta[..., None] == 0, torch.zeros_like(x), x / delta[..., None])
    return codes.to(torch.float8_e4m3fn).view(torch.uint8), delta


def _new_cache(pages, case):
    """The tensors of a paged cache, [pages, H_kv, page, d] and scales [pages, H_kv, page]."""
    shape = (pages, case["Hk"], case["page"], case["d"])
    dt = DTYPES[case["dtype"]]
    c = {"k": torch.zeros(shape, dtype=dt if case["fmt"] == "16" else torch.int8, device="cuda"),
         "v": torch.zeros(shape, dtype=torch.uint8 if case["fmt"] == "8+8" else dt, device="cuda")}
    if case["fmt"] != "16":
        c["k_scale"] = torch.zeros(shape[:3], device="cuda")
    if case["fmt"] == "8+8":
        c["v_scale"] = torch.zeros(shape[:3], device="cuda")
    return c


def _handle(c, dtype):
    import quantized_attention_08_b200 as sage
    return sage.SageKVCache(c["k"], c["v"], c.get("k_scale"), c.get("v_scale"), dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "slots":
        ctx, new = _slot_lens(case)
        P, B = case["page"], case["B"]
        width = max(_pages(c + n, P) for c, n in zip(ctx, new)) + 1
        held = sum(_pages(c, P) for c in ctx)
        need = sum(_pages(c + n, P) - _pages(c, P) for c, n in zip(ctx, new))
        order = torch.randperm(held + need + 8, generator=g, device="cuda").to(torch.int32)
        n_held = torch.tensor([_pages(c, P) for c in ctx], device="cuda")
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda")[None] < n_held[:, None]] = order[:held]
        return {"ctx": _ints(ctx), "new": _ints(new), "table": table, "free": order[held:].contiguous(),
                "used": _ints([3])}
    if op == "rope":
        B, N, dt = case["B"], case["N"], DTYPES[case["dtype"]]
        q = torch.randn(B, case["H"], N, case["d"], generator=g, device="cuda").to(dt)
        k = _k_like((B, case["Hk"], N, case["d"]), g, (1, 3))[0].to(dt)
        sec = [int(s) for s in case["sections"].split(",")]
        if case["far"]:
            pos = torch.randint(0, case["far"], (len(sec), B, N), generator=g, device="cuda").to(torch.int32)
        else:  # a grid of frames, rows and columns
            w = max(1, int(round(N ** (1 / 3))) * 2)
            n = torch.arange(N, device="cuda").expand(B, N) + torch.randint(0, 9, (B, 1), generator=g, device="cuda")
            pos = torch.stack([n // (w * w), n // w % w, n % w][:len(sec)]).to(torch.int32).contiguous()
        inv = torch.cat([10000.0 ** (-torch.arange(s, device="cuda", dtype=torch.float64) / s) for s in sec]).float()
        return {"q": q, "k": k, "pos": pos, "inv": inv, "sec": sec}
    if op == "append":
        T, B, dt = case["T"], case["B"], DTYPES[case["dtype"]]
        k, bias = _k_like((case["Hk"], T, case["d"]), g, (0, 2))
        v = torch.randn(case["Hk"], T, case["d"], generator=g, device="cuda")
        lens = _split(T, B, _rng_of(case))
        ids = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(lens, device="cuda")).to(torch.int32)
        pages = _pages(T, case["page"]) * case["slack"] + 1
        slots = torch.randperm(pages, generator=g, device="cuda")[:, None] * case["page"] + torch.arange(case["page"], device="cuda")
        if T <= 256:  # one token a request: a place of its own page each
            slots = slots.reshape(-1)[torch.randperm(slots.numel(), generator=g, device="cuda")]
        s = {"k": k.to(dt), "v": v.to(dt), "slots": slots.reshape(-1)[:T].to(torch.int32).contiguous(),
             "cache": _new_cache(pages, case)}
        if case["mean"]:
            s["mean"] = (bias.reshape(1, case["Hk"], case["d"]) +
                         0.1 * torch.randn(B, case["Hk"], case["d"], generator=g, device="cuda")).contiguous()
            s["ids"] = ids
        return s
    lens = _lens(case)
    P, B, dt = case["page"], case["B"], DTYPES[case["dtype"]]
    width = _pages(case["max_len"], P)
    total = sum(_pages(n, P) for n in lens)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n_held = torch.tensor([_pages(n, P) for n in lens], device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < n_held[:, None]] = perm
    cache = _new_cache(total, case)
    for a in range(0, total, 1024):  # by pieces: the fp32 values need not exist at once
        b = min(total, a + 1024)
        shape = (b - a, case["Hk"], P, case["d"])
        k = torch.randn(shape, generator=g, device="cuda")
        v = torch.randn(shape, generator=g, device="cuda")
        if case["fmt"] == "16":
            cache["k"][a:b] = (k + 0.5).to(dt)
        else:
            cache["k"][a:b], cache["k_scale"][a:b] = _quant_k(k)
        if case["fmt"] == "8+8":
            cache["v"][a:b], cache["v_scale"][a:b] = _quant_v(v)
        else:
            cache["v"][a:b] = v.to(dt)
    q = torch.randn(B, case["H"], case["nq"], case["d"], generator=g, device="cuda")
    q = q + torch.randn(1, case["H"], 1, case["d"], generator=g, device="cuda")
    return {"q": q.to(dt), "table": table, "lens": _ints(lens), "cache": cache}


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=case)
    if own and "cache" in state:
        state["handle"] = _handle(state["cache"], DTYPES[case["dtype"]])  # a program keeps one for its cache
    return state


# ------------------------------------------------------------------ plain forms
def _plain_slots(s):
    P, T = s["case"]["page"], s["case"]["T"]
    width, B = s["table"].shape[1], s["ctx"].numel()
    ctx, new = s["ctx"].long().clamp(0, width * P), s["new"].long().clamp(min=0)
    new = torch.minimum(new, width * P - ctx)
    start = torch.cumsum(new, 0) - new
    new = torch.minimum(new, (T - start).clamp(min=0))
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    held, need = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    need = need - held
    first = s["used"].long() + torch.cumsum(need, 0) - need
    j = torch.arange(width, device="cuda")[None] - held[:, None]
    at = first[:, None] + j
    n_free = s["free"].numel()
    page = torch.where(at < n_free, s["free"][at.clamp(0, n_free - 1)], torch.full_like(at, -1, dtype=torch.int32))
    table = s["table"]
    table.copy_(torch.where((j >= 0) & (j < need[:, None]), page, table))
    got = torch.minimum(need, (n_free - first).clamp(min=0))
    lens = torch.minimum(ctx + new, (held + got) * P)
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp(max=B - 1)
    inside = i < cu[-1]
    pos = ctx[b] + i - cu[b]
    pg = table[b, (pos // P).clamp(max=width - 1)].long()
    slot = torch.where(inside & (pg >= 0) & (pos < lens[b]), pg * P + pos % P, torch.full_like(pos, -1))
    neg = torch.full_like(pos, -1)
    return {"table": table, "seq_lens": lens.int(), "cu": cu.int(), "slots": slot.int(),
            "positions": torch.where(inside, pos, neg).int(), "seq_ids": torch.where(inside, b, neg).int(),
            "used": (s["used"].long() + got.sum()).int()}


def _plain_rope(s):
    axis = torch.repeat_interleave(torch.arange(len(s["sec"]), device="cuda"), torch.tensor(s["sec"], device="cuda"))
    angle = s["pos"].double()[axis].permute(1, 2, 0) * s["inv"].double()  # [B, N, R/2]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    half = s["inv"].numel()

    def turn(x):
        y = x.float()
        if s["case"]["pairing"] == "half":
            a, b = y[..., :half].clone(), y[..., half:2 * half].clone()
            y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., 0:2 * half:2].clone(), y[..., 1:2 * half:2].clone()
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
        return y.to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _cache_out(c):
    # the codes are returned as such, K's as whole numbers and V's as the E4M3
    # numbers they are, beside their scales: both have to be equal
    out = dict(c)
    if c["v"].dtype == torch.uint8:
        out["v"] = c["v"].view(torch.float8_e4m3fn)
    return out


def _plain_append(s):
    c, P = s["cache"], s["case"]["page"]
    page, at = s["slots"].long() // P, s["slots"].long() % P
    k, v = s["k"].transpose(0, 1), s["v"].transpose(0, 1)  # [T, H_kv, d]
    if s["case"]["mean"]:
        k = k.float() - s["mean"][s["ids"].long()]
    if s["case"]["fmt"] == "16":
        c["k"][page, :, at] = k.to(c["k"].dtype)
    else:
        c["k"][page, :, at], c["k_scale"][page, :, at] = _quant_k(k.float())
    if s["case"]["fmt"] == "8+8":
        c["v"][page, :, at], c["v_scale"][page, :, at] = _quant_v(v.float())
    else:
        c["v"][page, :, at] = v
    return _cache_out(c)


def _plain_decode(s):
    case, c, q = s["case"], s["cache"], s["q"]
    B, H, nq, d = q.shape
    Hk = case["Hk"]
    pages = s["table"].long().clamp(min=0)

    def rows(codes, scale, fp8):
        x = codes.view(torch.float8_e4m3fn) if fp8 else codes
        x = x[pages].float()  # [B, width, H_kv, P, d]
        if scale is not None:
            x = x * scale[pages][..., None]
        return x.transpose(1, 2).reshape(B, Hk, -1, d)

    k = rows(c["k"], c.get("k_scale"), False)
    x = torch.matmul(q.float().reshape(B, Hk, -1, d), k.transpose(2, 3)) / math.sqrt(d)
    del k
    t = torch.arange(x.shape[-1], device="cuda")
    seen = s["lens"].long()[:, None].expand(B, nq)
    if case["causal"]:
        seen = seen - nq + 1 + torch.arange(nq, device="cuda")
    mask = t < seen[:, None, None, :, None]  # [B, 1, 1, nq, keys]
    x = x.reshape(B, Hk, H // Hk, nq, -1).masked_fill(~mask, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    v = rows(c["v"], c.get("v_scale"), case["fmt"] == "8+8")
    v = v.masked_fill(t[:, None] >= s["lens"].long()[:, None, None, None], 0.0)
    o = torch.matmul(p.reshape(B, Hk, -1, x.shape[-1]), v).reshape(B, H, nq, d)
    l = l.reshape(B, H, nq, 1)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o.to(q.dtype), (m.reshape(B, H, nq) + torch.log(l[..., 0]))


# ------------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"slots": _plain_slots, "rope": _plain_rope, "append": _plain_append, "decode": _plain_decode}[op](s)
    import quantized_attention_08_b200 as sage
    if op == "slots":
        lens, cu, slots, pos, ids, used = sage.sage_kv_slots(s["ctx"], s["new"], s["free"], s["used"], s["table"],
                                                             page_size=case["page"], T=case["T"])
        return {"table": s["table"], "seq_lens": lens, "cu": cu, "slots": slots, "positions": pos, "seq_ids": ids,
                "used": used}
    if op == "rope":
        return sage.sage_rope_axes(s["q"], s["k"], s["pos"], s["inv"], s["sec"], pairing=case["pairing"])
    if op == "append":
        sage.sage_kv_append(s["k"], s["v"], s["slots"], s["handle"], mean_k=s.get("mean"), seq_ids=s.get("ids"))
        return _cache_out(s["cache"])
    return sage.sage_attn_decode_paged(s["q"], s["handle"], s["table"], s["lens"], case["max_len"],
                                       causal=case["causal"], return_lse=True)


# ----------------------------------------------------------------------- exact
def exact(case, seed):
    s = _inputs(case, seed)
    f = torch.float64
    if case["op"] == "slots":
        return None  # whole numbers
    if case["op"] == "rope":
        n = [int(x) for x in case["sections"].split(",")]
        R = sum(n)
        theta = torch.cat([s["pos"][a].to(f)[..., None] * p for a, p in enumerate(torch.split(s["inv"].to(f), n))], -1)
        turn = torch.polar(torch.ones_like(theta), theta)[:, None]
        out = []
        for x in (s["q"], s["k"]):
            x = x.to(f)
            if case["pairing"] == "half":
                z = torch.complex(x[..., :R], x[..., R:2 * R].contiguous()) * turn
                z = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.view_as_real(torch.view_as_complex(x[..., :2 * R].reshape(*x.shape[:-1], R, 2)) * turn).flatten(-2)
            out.append(torch.cat([z, x[..., 2 * R:]], -1))
        return tuple(out)
    if case["op"] == "append":
        # the scales in 64 bits from the definition; the 8-bit codes have no
        # value beyond themselves; 16-bit rows are the (smoothed) inputs
        page, at = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
        out = {n: None for n in s["cache"]}
        k, v = s["k"].to(f), s["v"].to(f)
        if case["mean"]:
            k = k - s["mean"].to(f)[s["ids"].long()].transpose(0, 1)
        for name, x, top in (("k", k, 127), ("v", v, 448)):
            if name + "_scale" in out:
                full = torch.zeros(s["cache"][name + "_scale"].shape, dtype=f, device="cuda")
                full[page, :, at] = (x.abs().amax(-1) / top).transpose(0, 1)
                out[name + "_scale"] = full
            else:
                full = torch.zeros(s["cache"][name].shape, dtype=f, device="cuda")
                full[page, :, at] = x.transpose(0, 1)
                out[name] = full
        return out
    # decode: request by request, kv head by kv head
    lens, P, nq, G = _lens(case), case["page"], case["nq"], case["H"] // case["Hk"]
    c = s["cache"]
    o = torch.zeros(s["q"].shape, dtype=f, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=f, device="cuda")
    for b, n in enumerate(lens):
        pg = s["table"][b, :_pages(n, P)].long()
        k, v = c["k"][pg], c["v"][pg]
        k = k.to(f) if "k_scale" not in c else k.to(f) * c["k_scale"][pg].to(f)[..., None]
        v = v.to(f) if "v_scale" not in c else v.view(torch.float8_e4m3fn).to(f) * c["v_scale"][pg].to(f)[..., None]
        k, v = (x.transpose(0, 1).reshape(case["Hk"], -1, case["d"])[:, :n] for x in (k, v))
        for i in range(nq):
            see = n - nq + 1 + i if case["causal"] else n
            if see <= 0:
                continue
            q = s["q"][b, :, i].to(f).reshape(case["Hk"], G, -1)
            z = torch.einsum("hgd,htd->hgt", q, k[:, :see]) / math.sqrt(case["d"])
            o[b, :, i] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), v[:, :see]).reshape(case["H"], -1)
            lse[b, :, i] = torch.logsumexp(z, -1).reshape(-1)
    return o, lse
