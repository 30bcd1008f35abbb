"""GPU tests of how many bits of a probability reach the decode attention's
output, on scores that are known exactly: q has one channel that is a power of
two, so that q . k is one exact product.

Tolerances, derived, with A = sum p |v| / l.  A score in log2, s', is a product
of at most four fp32 numbers less the running maximum: at most 6 roundings, 6 *
2^-24 |s'|, which move exp2 by ln 2 times that; here |s'| <= 40, so 2^-16.6 of p,
and as much of l: 2^-15.6 A.  A warp adds at most 16 products of tiles (2^-23 each,
tensor cores truncate), a join 60 pieces (2^-24 each), l as many: 2^-16.7 A;
exp2 and the scales 2^-20.  In all below 2^-15 A.  P is two 16-bit numbers whose
sum is within 2^-16 of it (bf16: half a step of a half step's remainder; fp16
keeps 2^-22 or, of the smaller ones, half its smallest step, 2^-25, of numbers
above 2^-9); of fp16 P below that, each key may lose 2^-47 of the largest
probability (2^-46 in 8+8, of the largest probability times the largest delta_V).
The output is rounded once: half its own step (relative to the value that is up
to twice as much)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F64 = torch.float64
FORMATS = [(torch.float16, "16"), (torch.bfloat16, "16"), (torch.float16, "B"), (torch.bfloat16, "B"),
           (torch.float16, "8+8"), (torch.bfloat16, "8+8")]


@pytest.fixture(scope="module")
def sage():
    import quantized_attention_08_b200 as s
    s.load_library()
    return s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def half_step(x, dtype):
    """Half the step of `dtype` at |x| (fp64)."""
    bits, low = (11, -24) if dtype == torch.float16 else (8, -133)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -140)))
    return torch.exp2((e - (bits - 1)).clamp(min=low) - 1)


def cache_of(sage, k, v, lens, P, fmt, seed):
    """k, v [H_kv, T, d] of requests of `lens` tokens on shuffled pages; the
    cache, its table, and the 64-bit K and V that it stands for."""
    Hk, T, d = k.shape
    held = [-(-n // P) for n in lens]
    c = sage.SageKVCache.allocate(sum(held) + 2, Hk, P, d, fmt, k.dtype)
    table = torch.full((len(lens), max(held)), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(sum(held) + 2, generator=gen(seed), device="cuda").to(torch.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :held[b]] = perm[at:at + held[b]]
        pos = torch.arange(n, device="cuda")
        slots.append(table[b, pos // P].long() * P + pos % P)
        at += held[b]
    s = torch.cat(slots)
    sage.sage_kv_append(k, v, s.to(torch.int32), c)
    return c, table, s


def values(c, s):
    """64-bit K and V, and V's scales, of the slots s."""
    rows = lambda t: t.transpose(1, 2).flatten(0, 1)[s].transpose(0, 1)  # noqa: E731
    K, V = rows(c.k).to(F64), rows(c.v)
    if c.format != "16":
        K = K * rows(c.k_scale).to(F64)[..., None]
    delta = torch.ones(V.shape[:2], dtype=F64, device="cuda")
    if c.format == "8+8":
        delta = rows(c.v_scale).to(F64)
        V = V.view(torch.float8_e4m3fn).to(F64) * delta[..., None]
    return K, V.to(F64), delta


def check(o, q, c, slots, lens, scale):
    """o [B, H, d] against 64 bits, by the tolerances above."""
    B, H, d = q.shape
    K, V, delta = values(c, slots)
    Hk = K.shape[0]
    bf16_p = q.dtype == torch.bfloat16 and c.format != "8+8"
    rounding = 2.0 ** -15 + 2.0 ** -16
    at = 0
    for b, n in enumerate(lens):
        k, v, dv = K[:, at:at + n], V[:, at:at + n], delta[:, at:at + n]
        at += n
        s = scale * torch.einsum("hgd,htd->hgt", q[b].to(F64).reshape(Hk, -1, d), k)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        assert float((s - s.amax(-1, keepdim=True)).abs().amax()) * math.log2(math.e) <= 40
        l = p.sum(-1, keepdim=True)
        want = torch.einsum("hgt,htd->hgd", p / l, v)
        A = torch.einsum("hgt,htd->hgd", p / l, v.abs())
        codes = v / dv.clamp(min=2.0 ** -100)[..., None]  # V itself where there are no scales
        lost = codes.abs().sum(1)[:, None] * dv.amax(-1)[:, None, None] / l
        lost = 0 if bf16_p else lost * 2.0 ** (-46 if c.format == "8+8" else -47)
        tol = half_step(want, o.dtype) + rounding * A + lost
        err = (o[b].to(F64).reshape(Hk, -1, d) - want).abs()
        assert bool((err <= tol).all()), (b, n, float((err / tol).max()))


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [2, 12])
@pytest.mark.parametrize("n", [2, 40, 1100, 9000])
def test_probabilities_keep_their_bits(sage, dtype, fmt, d, G, n):
    """Few keys with weight, so that roundings of single probabilities show: one
    key with V = 0 at the top, the others' V of every size."""
    Hk, lens = 2, [n, max(2, n // 3), 2]
    g, T = gen(n + d), sum(lens)
    k = torch.zeros(Hk, T, d, device="cuda")
    k[..., 0] = -6 - 6 * torch.rand(Hk, T, generator=g, device="cuda")
    v = torch.randn(Hk, T, d, generator=g, device="cuda")
    at = 0
    for m in lens:  # the first key has the largest score and no V; two more have weight
        k[:, at, 0], v[:, at] = 0, 0
        k[:, at + 1:at + min(m, 3), 0] *= 0.1
        at += m
    k, v = k.to(dtype), v.to(dtype)
    c, table, slots = cache_of(sage, k, v, lens, 16, fmt, n)
    q = torch.zeros(len(lens), Hk * G, d, device="cuda")
    q[..., 0] = 2.0 ** torch.randint(-1, 2, (len(lens), Hk * G), generator=g, device="cuda")
    q = q.to(dtype)
    o = sage.sage_attn_decode_paged(q, c, table, ints(lens), n, sm_scale=0.75)
    check(o, q, c, slots, lens, 0.75)


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("n", [50, 700, 20000])
@pytest.mark.parametrize("nats", [8.0, 12.0, 16.0, 17.5, 20.0])
@pytest.mark.parametrize("first", [True, False])
def test_keys_far_below_a_sink(sage, dtype, fmt, n, nats, first):
    """One key without V takes nearly all of the weight; the output is what the
    others, `nats` below it, leave, however little weight that is."""
    Hk, d, G = 1, 64, 3
    g = gen(n)
    k = torch.zeros(Hk, n, d, device="cuda")
    v = (torch.randn(Hk, n, d, generator=g, device="cuda").abs() + 1) * 30
    sink = 0 if first else n - 1
    k[:, sink, 0], v[:, sink] = 4, 0
    k, v = k.to(dtype), v.to(dtype)
    c, table, slots = cache_of(sage, k, v, [n], 16, fmt, n)
    q = torch.zeros(1, G, d, device="cuda", dtype=dtype)
    q[..., 0] = 4
    o = sage.sage_attn_decode_paged(q, c, table, ints([n]), n, sm_scale=nats / 16)
    check(o, q, c, slots, [n], nats / 16)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [50, 400, 20000])
@pytest.mark.parametrize("log2_spread", [12, 20, 24, 26])
@pytest.mark.parametrize("at", [0, 37])
def test_one_large_v_without_weight(sage, dtype, n, log2_spread, at):
    """A token whose V is 2^log2_spread times the others' and whose probability is
    nearly nothing leaves their part of the output as it is."""
    Hk, d, G = 1, 128, 3
    g = gen(n)
    k = torch.zeros(Hk, n, d, device="cuda")
    v = torch.randn(Hk, n, d, generator=g, device="cuda")
    k[:, at, 0] = -4
    c, table, slots = cache_of(sage, k.to(dtype), v.to(dtype), [n], 16, "8+8", n)
    page, row = int(slots[at]) // 16, int(slots[at]) % 16
    c.v_scale[page, 0, row] *= 2.0 ** log2_spread
    q = torch.zeros(1, G, d, device="cuda", dtype=dtype)
    q[..., 0] = 4
    o = sage.sage_attn_decode_paged(q, c, table, ints([n]), n, sm_scale=27.0 / 16)  # 2^-39 of the others
    check(o, q, c, slots, [n], 27.0 / 16)
