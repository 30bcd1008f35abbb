"""The decode attention against the packed prefill, on the same tokens."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    import quantized_attention_08_b200 as s
    s.load_library()
    return s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
@pytest.mark.parametrize("variant", ["B", "8+8"])
@pytest.mark.parametrize("d,H,Hk", [(64, 8, 2), (128, 6, 6)])
def test_last_rows_of_prompts_agree_with_the_prefill(sage, fmt, variant, d, H, Hk):
    """slots -> rope -> prefill and append -> decode of each prompt's last token:
    the row that the prefill has for it.  Both quantize; each is within the cosine
    of 0.998 of attention in 64 bits that the prefill's tests ask for, 3.6 degrees,
    so they lie within twice that of one another: cos 7.3 degrees = 0.992."""
    prompt, P, g = [45, 130, 1, 700], 16, torch.Generator(device="cuda").manual_seed(d + H)
    T, B = sum(prompt), len(prompt)
    rand = lambda h: torch.randn(h, T, d, generator=g, device="cuda")  # noqa: E731
    q, k, v = rand(H).half(), (rand(Hk) + 5 * torch.randn(Hk, 1, d, generator=g, device="cuda")).half(), rand(Hk).half()
    cache = sage.SageKVCache.allocate(80, Hk, P, d, fmt, torch.float16)
    table = torch.full((B, 50), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(80, generator=g, device="cuda").to(torch.int32)
    lens, cu, slots, pos, ids, _ = sage.sage_kv_slots(ints([0] * B), ints(prompt), free, ints([0]), table, page_size=P, T=T)
    inv = 10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2))
    q, k = sage.sage_rope_axes(q, k, pos[None], inv, [d // 2])
    mean = sage.sage_smooth_quant_qkv_varlen(q, k, cu, max(prompt))[4]
    prefill = sage.sage_attn_fwd_varlen(q, k, v, cu, max(prompt), causal=True, variant=variant)
    sage.sage_kv_append(k, v, slots, cache, mean_k=mean, seq_ids=ids)
    last = (cu[1:] - 1).long()
    got = sage.sage_attn_decode_paged(q[:, last].transpose(0, 1), cache, table, lens, max(prompt)).double()
    want = prefill[:, last].transpose(0, 1).double()
    for b, (a, e) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
        s = torch.einsum("hgd,htd->hgt", q[:, e - 1].double().reshape(Hk, -1, d), k[:, a:e].double()) / math.sqrt(d)
        true = torch.einsum("hgt,htd->hgd", torch.softmax(s, -1), v[:, a:e].double()).reshape(-1)
        cos = lambda x, y: float(torch.nn.functional.cosine_similarity(x.flatten(), y.flatten(), dim=0))  # noqa: E731
        assert cos(got[b], true) >= 0.998 and cos(want[b], true) >= 0.998, (b, cos(got[b], true), cos(want[b], true))
        assert cos(got[b], want[b]) >= 0.992, (b, cos(got[b], want[b]))
