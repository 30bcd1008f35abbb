"""The bounded waits of the decode attention: with a limit of a nanosecond a
loading warp gives up once its rings stay full for a tick of the clock, the
consuming warps follow, copies under way land, the error word says so, and the same
call is right again under the usual limit.  (A request long enough, with 16 rows a
group, keeps the rings full that long; a cluster's or a single warp's four steps
do not.)"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEFAULT_NS = 2_000_000_000


@pytest.fixture(scope="module")
def sage():
    import quantized_attention_08_b200 as s
    s.load_library()
    return s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
def test_a_loading_warp_gives_up(sage, fmt):
    lens, H, Hk = [100000], 64, 4
    d, P = 128, 32
    B, width = len(lens), max(-(-n // P) for n in lens)
    g = torch.Generator(device="cuda").manual_seed(B)
    c = sage.SageKVCache.allocate(B * width, Hk, P, d, fmt)
    table = torch.randperm(B * width, generator=g, device="cuda").reshape(B, width).to(torch.int32)
    k, v = (torch.randn(Hk, B * width * P, d, generator=g, device="cuda").half() for _ in range(2))
    sage.sage_kv_append(k, v, torch.arange(B * width * P, device="cuda").to(torch.int32), c)
    q = torch.randn(B, H, d, generator=g, device="cuda").half()
    call = lambda: sage.sage_attn_decode_paged(q, c, table, ints(lens), max(lens))  # noqa: E731
    want = call()
    assert sage.sage_get_device_error() == (sage.SAGE_OK, 0)
    try:
        sage.sage_set_wait_timeout_ns(1)
        for _ in range(20):
            call()
        st, word = sage.sage_get_device_error()
    finally:
        sage.sage_set_wait_timeout_ns(DEFAULT_NS)
    assert st == sage.SAGE_ERR_DEVICE_TIMEOUT and word & 1 and (word >> 8) & 0xFF == 0xD1
    again = call()
    assert sage.sage_get_device_error() == (sage.SAGE_OK, 0)
    assert torch.equal(want, again) and bool(torch.isfinite(want).all())
    # and right: the first request, head by head, in 64 bits
    rows = lambda t: t[table[0].long()].transpose(0, 1).reshape(Hk, -1, *t.shape[3:])[:, :lens[0]]  # noqa: E731
    K, V = rows(c.k).double(), rows(c.v)
    if fmt != "16":
        K = K * rows(c.k_scale).double()[..., None]
    if fmt == "8+8":
        V = V.view(torch.float8_e4m3fn).double() * rows(c.v_scale).double()[..., None]
    s = torch.einsum("hgd,htd->hgt", q[0].double().reshape(Hk, -1, d), K) / math.sqrt(d)
    o = torch.einsum("hgt,htd->hgd", torch.softmax(s, -1), V.double()).reshape(H, d)
    # scores to d 2^-24 of their terms, P to 2^-16, the output's rounding
    E = d * 2.0 ** -24 * float((q[0].double().abs().sum(-1).max() * K.abs().max()) / math.sqrt(d))
    A = torch.einsum("hgt,htd->hgd", torch.softmax(s, -1), V.double().abs()).reshape(H, d)
    assert bool(((again[0].double() - o).abs() <= 2.0 ** -11 * o.abs() + (2 * E + 2.0 ** -15) * A + 2.0 ** -25).all())
