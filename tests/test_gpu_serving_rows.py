"""Decode attention: what one query row holds costs no other row of its group
its exactness.  (Bits may change: the running maxima of a group's rows follow
together, so where a row's is taken anew depends on the others.)"""
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


def filled(sage, n, Hk, d, fmt, dtype, scale_k=1.0):
    g = torch.Generator(device="cuda").manual_seed(n + d)
    pages = -(-n // 16)
    c = sage.SageKVCache.allocate(pages, Hk, 16, d, fmt, dtype)
    k = (scale_k * torch.randn(Hk, n, d, generator=g, device="cuda")).to(dtype)
    v = torch.randn(Hk, n, d, generator=g, device="cuda").to(dtype)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    t = torch.arange(n, device="cuda")
    s = (table[0, t // 16] * 16 + (t % 16).to(torch.int32)).contiguous()
    sage.sage_kv_append(k, v, s, c)
    rows = lambda x: x.transpose(1, 2).flatten(0, 1)[s.long()].transpose(0, 1)  # noqa: E731
    K, V = rows(c.k).to(F64), rows(c.v)
    if fmt != "16":
        K = K * rows(c.k_scale).to(F64)[..., None]
    V = V.view(torch.float8_e4m3fn).to(F64) * rows(c.v_scale).to(F64)[..., None] if fmt == "8+8" else V.to(F64)
    return c, table, K, V


def check_row(o, q, K, V, scale):
    """One row o [d] against 64 bits: scores are off by E = d 2^-24 max sum |q k|
    scale at most, P by 2^-16, sums and exp2 by 2^-16, the output by its rounding."""
    s = scale * (K @ q)
    p = torch.softmax(s, -1)
    want, A = p @ V, p @ V.abs()
    E = q.numel() * 2.0 ** -24 * scale * float((K.abs() @ q.abs()).amax())
    u = 2.0 ** (-11 if o.dtype == torch.float16 else -8)
    err = (o.to(F64) - want).abs()
    assert bool((err <= u * want.abs() + (2 * E + 2.0 ** -15) * A + 2.0 ** -25).all()), float(err.max())


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("n,nq", [(60, 3), (1000, 4), (20000, 2)])
@pytest.mark.parametrize("filler", [0.5, 3e4, float("inf"), float("nan")])
def test_rows_that_a_batch_is_padded_with(sage, dtype, fmt, n, nq, filler):
    """The last query token of a request is no token: whatever stands there, the
    rows before it are right."""
    d, Hk, G = 64, 2, 3
    c, table, K, V = filled(sage, n, Hk, d, fmt, dtype)
    g = torch.Generator(device="cuda").manual_seed(nq)
    q = torch.randn(1, Hk * G, nq, d, generator=g, device="cuda").to(dtype)
    q[:, :, -1] = filler if not (dtype == torch.bfloat16 and filler == 3e4) else 3e38
    o, lse = sage.sage_attn_decode_paged(q, c, table, ints([n]), n, causal=False, return_lse=True)
    assert bool(torch.isfinite(lse[:, :, :-1]).all())
    for h in range(Hk * G):
        for i in range(nq - 1):
            check_row(o[0, h, i], q[0, h, i].to(F64), K[h // G], V[h // G], 1 / math.sqrt(d))


@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
@pytest.mark.parametrize("G", [5, 14])
def test_rows_of_every_size(sage, fmt, G):
    """bf16 rows of one group between 2^-60 and 2^60: each row its own softmax."""
    d, n = 128, 600
    c, table, K, V = filled(sage, n, 1, d, fmt, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(G)
    q = torch.randn(1, G, d, generator=g, device="cuda")
    size = 2.0 ** torch.tensor([0, 60, -60, 25, -25, 0, 31, 2, 40, -3, 1, 17, 0, 33][:G], device="cuda")
    q = (q * size[:, None]).bfloat16()
    o = sage.sage_attn_decode_paged(q, c, table, ints([n]), n)
    for r in range(G):
        check_row(o[0, r], q[0, r].to(F64), K[0], V[0], 1 / math.sqrt(d))


@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
@pytest.mark.parametrize("log2_q", [-120, -100, 100, 118, 122, 126])
def test_large_q_and_small_k(sage, fmt, log2_q):
    """bf16 q near the type's largest and smallest numbers, K so that scores are ordinary."""
    d, n = 64, 300
    c, table, K, V = filled(sage, n, 1, d, fmt, torch.bfloat16, scale_k=2.0 ** (-log2_q if log2_q < 94 else -94))
    g = torch.Generator(device="cuda").manual_seed(3)
    q = (torch.rand(1, 2, d, generator=g, device="cuda") - 0.5).to(F64) * 2.0 ** log2_q
    q = q.float().bfloat16()
    scale = 0.125 * 2.0 ** (min(94, log2_q) - log2_q)
    o = sage.sage_attn_decode_paged(q, c, table, ints([n]), n, sm_scale=scale)
    for r in range(2):
        check_row(o[0, r], q[0, r].to(F64), K[0], V[0], scale)
