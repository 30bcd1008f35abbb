"""CPU checks of the serving entry points: what they refuse, before any CUDA
call (status codes of include/sage.h: 1 invalid, 2 unsupported, 3 misaligned,
7 workspace too small), and what the binding refuses before the library."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
OK = 1 << 20
ODD = P(OK + 8)
F = P(OK)


@pytest.fixture(scope="module")
def lib():
    from quantized_attention_08_b200 import build
    build.build()
    import quantized_attention_08_b200 as pkg
    return pkg.load_library()


def cache(**kw):
    import quantized_attention_08_b200 as pkg
    c = pkg._CacheStruct(OK, OK, OK, OK, 2 * 64 * 128, 2 * 64 * 128, 2 * 64, 2 * 64, 10, 64, 2, 128, 2, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
              (dict(num_pages=-1), 1), (dict(page_size=0), 1), (dict(H_kv=0), 1), (dict(k_page_stride=16384 - 16), 1),
              (dict(v_scale_page_stride=127), 1), (dict(d=96), 2), (dict(page_size=40), 2), (dict(format=3), 2),
              (dict(dtype=2), 2), (dict(num_pages=1 << 26), 2), (dict(k=OK + 4), 3), (dict(v_scale=OK + 2), 3),
              (dict(v_page_stride=16384 + 8), 3), (dict(k_scale=OK + 8), 3), (dict(k_scale_page_stride=130), 3)]


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def test_append_refusals(lib):
    f = lib.sage_kv_append
    s = strides(1280, 128)

    def call(c=None, **kw):
        a = dict(k=F, ks=s, v=F, vs=s, T=10, slots=F, mean=F, ids=F, B=2)
        a.update(kw)
        return f(*a.values(), None if c == "null" else ctypes.byref(c or cache()), None)

    for kw, want in BAD_CACHES:
        assert call(cache(**kw)) == want, kw
    assert call("null") == 1
    assert call(T=-1) == 1 and call(T=(1 << 30) + 1) == 2
    assert call(k=None) == 1 and call(v=None) == 1 and call(slots=None) == 1 and call(ks=None) == 1
    assert call(ids=None) == 1 and call(B=-1) == 1
    assert call(k=ODD) == 3 and call(v=ODD) == 3 and call(mean=ODD) == 3 and call(slots=P(OK + 2)) == 3
    assert call(ks=strides(1280, 132)) == 3 and call(vs=strides(4, 128)) == 3
    assert call(T=0, k=None, v=None, slots=None) == 0


def test_decode_refusals(lib):
    f = lib.sage_attn_decode_paged
    s = strides(1024, 128, 128)

    def call(c=None, **kw):
        a = dict(q=F, s=s, c=ctypes.byref(c or cache()), table=F, max_pages=40, lens=F, B=3, H=8, nq=1, max_len=2000,
                 causal=1, scale=0.1, o=F, lse=F, ws=F, bytes=1 << 30)
        a.update(kw)
        return f(*a.values(), None)

    for kw, want in BAD_CACHES:
        assert call(cache(**kw)) == want, kw
    assert call(c=None, B=-1) == 1 and call(nq=-1) == 1 and call(max_len=-1) == 1 and call(H=0) == 1
    assert call(max_len=40 * 64 + 1) == 1          # more than the table's rows hold
    assert call(max_pages=-1, max_len=0) == 1
    assert call(causal=2) == 1 and call(scale=0.0) == 1 and call(scale=float("inf")) == 1 and call(scale=float("nan")) == 1
    assert call(q=None) == 1 and call(s=None) == 1 and call(table=None) == 1 and call(lens=None) == 1 and call(o=None) == 1
    assert call(H=7) == 2 and call(B=4097) == 2 and call(nq=257) == 2
    assert call(q=ODD) == 3 and call(o=ODD) == 3 and call(lens=P(OK + 1)) == 3 and call(s=strides(1024, 132, 128)) == 3
    assert call(max_pages=1000, max_len=60000, ws=P(OK + 16)) == 3 and call(max_pages=1000, max_len=60000, ws=None) == 1
    need = lib.sage_attn_decode_workspace_bytes(3, 8, 2, 1, 128, 60000, 2)
    assert need > 0 and call(max_pages=1000, max_len=60000, bytes=need - 1) == 7
    import quantized_attention_08_b200 as pkg
    assert "workspace smaller" in pkg.sage_last_error_detail()
    assert call(B=0, q=None, lens=None, o=None) == 0 and call(nq=0, q=None, o=None) == 0


def test_decode_workspace_sizes(lib):
    f = lib.sage_attn_decode_workspace_bytes
    assert f(0, 8, 2, 1, 128, 2000, 2) == 0 and f(3, 8, 2, 0, 128, 2000, 2) == 0
    assert f(3, 8, 3, 1, 128, 2000, 2) == 0 and f(3, 8, 2, 1, 96, 2000, 2) == 0 and f(3, 8, 2, 1, 128, 2000, 9) == 0
    assert f(4, 8, 2, 1, 128, 16, 0) == 0          # short caches are not split
    assert f(4, 8, 2, 1, 128, 2000, 0) == 0        # nor are few longer ones, but within a cluster
    assert f(4096, 8, 2, 1, 128, 1 << 20, 0) < 1 << 27


def test_slots_refusals(lib):
    f = lib.sage_kv_slots

    def call(**kw):
        a = dict(ctx=F, new=F, B=3, free=F, num_free=5, used=F, table=F, max_pages=10, page=16, lens=F, cu=F, slots=F,
                 pos=F, ids=F, T=9, out=F)
        a.update(kw)
        return f(*a.values(), None)

    for k in ("ctx", "new", "free", "used", "table", "lens", "cu", "slots", "pos", "ids", "out"):
        assert call(**{k: None}) == 1, k
        assert call(**{k: P(OK + 2)}) == 3, k
    assert call(B=-1) == 1 and call(T=-1) == 1 and call(num_free=-1) == 1 and call(page=0) == 1 and call(max_pages=-1) == 1
    assert call(B=8193) == 2 and call(T=(1 << 30) + 1) == 2 and call(max_pages=1 << 20, page=1 << 12) == 2


def test_rope_refusals(lib):
    f = lib.sage_rope_axes
    s = strides(1024, 128, 128)

    def call(sections=(16, 24, 24), **kw):
        a = dict(q=F, qs=s, qo=F, qos=s, k=F, ks=s, ko=F, kos=s, pos=F, ps=strides(8, 0), inv=F,
                 sec=(ctypes.c_int * len(sections))(*sections), n=len(sections), B=1, H=8, Hk=2, N=1, d=128, il=0, dt=0)
        a.update(kw)
        return f(*a.values(), None)

    for k in ("q", "qs", "qo", "qos", "ks", "ko", "kos", "pos", "ps", "inv", "sec"):
        assert call(**{k: None}) == 1, k
    assert call(k=None) == 1                       # its output is left
    for k in ("q", "qo", "k", "ko"):
        assert call(**{k: ODD}) == 3, k
    assert call(pos=P(OK + 1)) == 3 and call(inv=P(OK + 2)) == 3 and call(kos=strides(1024, 132, 128)) == 3
    assert call((16, 24, 25)) == 1 and call((-8, 16)) == 1 and call((0,)) == 1 and call((8, 16, 20)) == 2
    assert call((8,) * 5) == 2 and call(d=96) == 2 and call(dt=2) == 2 and call(il=2) == 1
    assert call(B=-1) == 1 and call(N=-1) == 1 and call(H=0) == 1 and call(Hk=0) == 1 and call(n=0) == 1
    assert call(B=0, q=None) == 0 and call(N=0, q=None) == 0


def test_binding_refusals(lib):
    import quantized_attention_08_b200 as sage
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)    # noqa: E731
    with pytest.raises(TypeError):
        sage.SageKVCache(h(4, 2, 16, 64), h(4, 2, 16, 64))                       # not on a GPU
    with pytest.raises(ValueError):
        sage.SageKVCache(h(4, 2, 16, 64), h(4, 2, 16, 128))
    with pytest.raises(TypeError):
        sage.SageKVCache(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64))   # fp32
    with pytest.raises(TypeError):
        sage.SageKVCache(h(4, 2, 16, 64), h(4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sage.SageKVCache.allocate(4, 2, 16, 64, format="4")
    with pytest.raises(TypeError):
        sage.sage_kv_slots(i(3), i(3), i(9), i(1), i(3, 4), page_size=16, T=3)   # not on a GPU
    with pytest.raises(TypeError):
        sage.sage_kv_slots(i(3).long(), i(3), i(9), i(1), i(3, 4), page_size=16, T=3)
    with pytest.raises(ValueError):
        sage.sage_kv_slots(i(3), i(4), i(9), i(1), i(3, 4), page_size=16, T=3)
    with pytest.raises(ValueError):
        sage.sage_kv_slots(i(3), i(3), i(9), i(1), i(4, 3).t(), page_size=16, T=3)
    with pytest.raises(ValueError):
        sage.sage_kv_slots(i(3), i(3), i(9), i(1), i(3, 4), page_size=16, T=-1)
    with pytest.raises(ValueError):
        sage.sage_kv_slots(i(3), i(3), i(9), i(1), i(3, 4), page_size=1 << 32, T=1)
    f = torch.zeros(32)
    with pytest.raises(TypeError):
        sage.sage_rope_axes(h(1, 2, 5, 64).float(), None, i(1, 5), f, [32])
    with pytest.raises(ValueError):
        sage.sage_rope_axes(h(1, 2, 5, 64), None, i(1, 5), f, [32], pairing="other")
    with pytest.raises(ValueError):
        sage.sage_rope_axes(h(1, 2, 5, 64), None, i(1, 6), f, [32])
    with pytest.raises(ValueError):
        sage.sage_rope_axes(h(1, 2, 5, 64), h(1, 2, 6, 64), i(1, 5), f, [32])
    with pytest.raises(ValueError):
        sage.sage_rope_axes(h(1, 2, 5, 64), None, i(1, 5), f, [16])
    with pytest.raises(ValueError):
        sage.sage_rope_axes(h(1, 2, 64, 5).transpose(2, 3), None, i(1, 5), f, [32])
    with pytest.raises(TypeError):
        sage.sage_rope_axes(h(1, 2, 5, 64), None, i(1, 5), f, [32])              # not on a GPU
