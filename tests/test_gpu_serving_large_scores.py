"""Decode attention where scores are so large that fp32's steps at them are no
longer small: the output stays the weighted mean that it is."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FORMATS = [(torch.float16, "16"), (torch.bfloat16, "16"), (torch.float16, "B"), (torch.bfloat16, "B"),
           (torch.float16, "8+8"), (torch.bfloat16, "8+8")]


@pytest.fixture(scope="module")
def sage():
    import quantized_attention_08_b200 as s
    s.load_library()
    return s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def filled(sage, k, v, fmt):
    Hk, n, d = k.shape
    pages = -(-n // 16)
    c = sage.SageKVCache.allocate(pages, Hk, 16, d, fmt, k.dtype)
    g = torch.Generator(device="cuda").manual_seed(n)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    t = torch.arange(n, device="cuda")
    slots = table[0, t // 16] * 16 + (t % 16).to(torch.int32)
    sage.sage_kv_append(k, v, slots.contiguous(), c)
    V = c.v.transpose(1, 2).flatten(0, 1)[slots.long()].transpose(0, 1)
    if fmt == "8+8":
        delta = c.v_scale.transpose(1, 2).flatten(0, 1)[slots.long()].transpose(0, 1)
        return c, table, V.view(torch.float8_e4m3fn).double() * delta.double()[..., None]
    return c, table, V.double()


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("n", [33, 900, 20000])
def test_equal_scores_of_every_size(sage, dtype, fmt, n):
    """All keys alike: the mean of V, whatever the score.  Each of n weights is the
    same number, so that only sums (2^-17 of A, as long as their terms) and the
    output's rounding are left."""
    d, G = 64, 20
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.zeros(1, n, d, device="cuda")
    k[..., 0] = 1.37 * 2.0 ** 14
    v = torch.randn(1, n, d, generator=g, device="cuda") + 0.5
    c, table, V = filled(sage, k.to(dtype), v.to(dtype), fmt)
    q = torch.zeros(1, G, d, dtype=dtype, device="cuda")
    q[0, :, 0] = 2.0 ** (torch.arange(G, device="cuda") % 14)  # scores of 2^8 and up by the rows
    for sign in (1, -1):
        for up in (1.0, 1.1 * 2 ** 4, 1.7 * 2 ** 8, 1.2 * 2 ** 13):
            o = sage.sage_attn_decode_paged(sign * q, c, table, ints([n]), n, sm_scale=up / 64)
            want, A = V.mean(1)[0], V.abs().mean(1)[0]
            u = 2.0 ** (-11 if dtype == torch.float16 else -8)
            # P's second number leaves up to 2^-16 of it, the same of every key
            tol = u * want.abs() + (2.0 ** -16 + 2.0 ** -17) * A
            err = (o[0].double() - want).abs()
            assert bool((err <= tol).all()), (sign, up, float(torch.nan_to_num(err, 9e9).max()))


@pytest.mark.parametrize("dtype,fmt", FORMATS)
@pytest.mark.parametrize("G", [3, 13])
def test_growing_scores_of_every_size(sage, dtype, fmt, G):
    """A large part that all keys share and a small one that grows along the
    request by less than the running maximum's slack at a time: every output is a
    mean of V with weights of at most 1, so between the least and the largest V."""
    d, n = 128, 2000
    g = torch.Generator(device="cuda").manual_seed(G)
    k = torch.zeros(1, n, d, device="cuda")
    k[..., 0] = 2.0 ** 13
    # int8 codes keep the small part as multiples of 2^13 / 127
    k[..., 1] = torch.linspace(0, 2.0 ** 13, n, device="cuda") + 100 * torch.rand(n, generator=g, device="cuda")
    v = torch.randn(1, n, d, generator=g, device="cuda")
    c, table, V = filled(sage, k.to(dtype), v.to(dtype), fmt)
    low, high, A = V.amin(1)[0], V.amax(1)[0], V.abs().amax(1)[0]
    u = 2.0 ** (-11 if dtype == torch.float16 else -8)
    for big in range(6, 16):       # scores of 2^19 to 2^28 and a little more
        for small in (0.02, 0.1, 0.5):
            q = torch.zeros(1, G, d, device="cuda")
            q[0, :, 0] = 2.0 ** big * (1 + torch.rand(G, generator=g, device="cuda") / 2)
            q[0, :, 1] = small * (1 + torch.rand(G, generator=g, device="cuda"))
            o = sage.sage_attn_decode_paged(q.to(dtype), c, table, ints([n]), n, sm_scale=1.0)[0].double()
            slack = (u + 2.0 ** -14) * A
            assert bool(((o >= low - slack) & (o <= high + slack)).all()), (big, small)


@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
@pytest.mark.parametrize("n", [60, 3000, 20000])
@pytest.mark.parametrize("log2_v", [-90, -60, 100, 110])
def test_v_of_every_size(sage, fmt, n, log2_v):
    """bf16 V so large that n of it are just below fp32's largest number, or small,
    under equal scores: its mean, by the bounds above."""
    d, G = 64, 3
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.zeros(1, n, d, dtype=torch.bfloat16, device="cuda")
    v = ((torch.rand(1, n, d, generator=g, device="cuda") + 1) * 2.0 ** log2_v).bfloat16()
    c, table, V = filled(sage, k, v, fmt)
    q = torch.ones(1, G, d, dtype=torch.bfloat16, device="cuda")
    o = sage.sage_attn_decode_paged(q, c, table, ints([n]), n)[0].double()
    want = V.mean(1)[0]
    assert bool(((o - want).abs() <= (2.0 ** -8 + 2.0 ** -16 + 2.0 ** -17) * want).all())
