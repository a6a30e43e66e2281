"""The cache calls refuse bad arguments on the host, before anything is launched
(no GPU needed), and the reference of their tests agrees with itself."""
import ctypes

import numpy as np
import pytest
import torch

import cache_ref as ref

FAKE = 1 << 20          # a 16-byte-aligned, never dereferenced address
WS = 1 << 24


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_verify_temperature_b200 import build, spec_verify
    build.build()
    return spec_verify.lib()


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def cache(**kw):
    from speculative_decoding_verify_temperature_b200 import kv_cache
    c = kv_cache._CCache(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, 64, 16, 4, 16, 2, 128, 16)
    for name, v in kw.items():
        setattr(c, name, v)
    return ctypes.byref(c)


def test_workspace_bytes():
    import speculative_decoding_verify_temperature_b200 as spec
    f = spec.spec_cache_workspace_bytes
    a = f(1, 1, 8, 128)
    assert a > 0 and a % 256 == 0 and f(32, 64, 64, 128) >= a
    assert f(-1, 1, 8, 128) == 0 and f(1, 0, 8, 128) == 0 and f(1, 257, 8, 128) == 0
    assert f(1, 1, 0, 128) == 0 and f(1, 1, 8, 96) == 0 and f(1, 1, 1025, 128) == 0


def test_plan_refusals(L):
    from speculative_decoding_verify_temperature_b200 import spec_verify as sv
    E = sv.SPEC_ERR_INVALID_ARG

    def call(B=2, N=8, depth=4, parents=FAKE, lengths=FAKE, pos=FAKE, anc=FAKE, ws=WS, wsb=1 << 30):
        return L.spec_tree_plan(B, N, depth, parents, lengths, pos, anc, ws, wsb, None)

    assert call(B=0, lengths=None) == sv.SPEC_OK
    assert call(B=-1) == E and call(N=0) == E and call(N=257) == E
    assert call(depth=-1) == E and call(depth=65) == E
    assert call(lengths=None) == E and call(pos=None) == E and call(anc=None) == E
    assert L.spec_last_error_detail()
    assert call(ws=None) == sv.SPEC_ERR_WORKSPACE and call(ws=WS + 16) == sv.SPEC_ERR_WORKSPACE
    assert call(wsb=16) == sv.SPEC_ERR_WORKSPACE


def test_norm_rope_refusals(L):
    from speculative_decoding_verify_temperature_b200 import spec_verify as sv
    E = sv.SPEC_ERR_INVALID_ARG

    def call(B=2, N=3, Hq=4, Hk=2, D=128, q=FAKE, qs=(1536, 512, 128), k=FAKE, dt=1, pos=FAKE, freq=FAKE, rot=128,
             inter=0, qw=None, kw=None, wdt=1, eps=1e-6, qo=FAKE, ko=FAKE):
        s, t = strides(*qs), strides(768, 256, 128)
        return L.spec_qk_norm_rope(B, N, Hq, Hk, D, q, s, k, t, dt, pos, freq, rot, inter, qw, kw, wdt, eps, qo, s, ko,
                                   t, None)

    assert call(B=0, q=None) == sv.SPEC_OK
    assert call(B=-1) == E and call(N=0) == E and call(Hq=0) == E and call(Hk=-1) == E and call(Hq=1025) == E
    assert call(D=0) == E and call(D=100) == E and call(D=264) == E
    assert call(dt=2) == E and call(wdt=7) == E and call(inter=2) == E
    assert call(rot=8) == E and call(rot=144) == E and call(rot=-16) == E and call(freq=None) == E
    assert call(eps=-1.0) == E and call(eps=float("nan")) == E and call(eps=float("inf")) == E
    assert call(q=None) == E and call(q=FAKE + 8) == E and call(k=None) == E and call(pos=None) == E
    assert call(qs=(1536, 512, 132)) == E and call(qw=FAKE + 4) == E and call(kw=FAKE + 2) == E
    assert call(qo=None) == E and call(ko=FAKE + 2) == E


CACHE_REFUSALS = [dict(head_dim=96), dict(page_size=48), dict(page_size=0), dict(kv_heads=0), dict(kv_heads=1025),
                  dict(max_pages=-1), dict(page_table_stride=15), dict(num_pages=-1), dict(num_pages=1 << 31),
                  dict(num_slots=1), dict(lengths=None), dict(page_table=None), dict(k_pages=None),
                  dict(v_open=None), dict(k_open=FAKE + 8), dict(v_pages=FAKE + 4), dict(k_scale=None)]


def test_attention_refusals(L):
    from speculative_decoding_verify_temperature_b200 import spec_verify as sv
    E = sv.SPEC_ERR_INVALID_ARG

    def call(B=2, N=3, Hq=4, c=None, q=FAKE, qs=(1536, 512, 128), k=FAKE, v=FAKE, scale=0.1, out=FAKE, ws=WS,
             wsb=1 << 30):
        t = strides(768, 256, 128)
        return L.spec_tree_attention(B, N, Hq, cache() if c is None else c, q, strides(*qs), k, t, v, t, FAKE, scale,
                                     out, None, ws, wsb, None)

    assert call(B=0, q=None) == sv.SPEC_OK
    assert call(B=-1) == E and call(B=16385) == E and call(N=0) == E and call(N=257) == E
    assert call(Hq=0) == E and call(Hq=5) == E and call(Hq=1026) == E
    assert call(q=None) == E and call(k=None) == E and call(v=FAKE + 2) == E and call(out=None) == E
    assert call(out=FAKE + 2) == E and call(qs=(1536, 516, 128)) == E
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == E
    assert call(ws=None) == sv.SPEC_ERR_WORKSPACE and call(wsb=256) == sv.SPEC_ERR_WORKSPACE
    for bad in CACHE_REFUSALS:
        assert call(c=cache(**bad)) == E, bad
    assert L.spec_tree_attention(2, 3, 4, None, FAKE, strides(0, 0, 0), FAKE, strides(0, 0, 0), FAKE, strides(0, 0, 0),
                                 FAKE, 0.1, FAKE, None, WS, 1 << 30, None) == E


def test_append_refusals(L):
    from speculative_decoding_verify_temperature_b200 import spec_verify as sv
    E = sv.SPEC_ERR_INVALID_ARG

    def call(B=2, T=3, width=3, c=None, k=FAKE, ks=(768, 256, 128), v=FAKE, dt=1, index=FAKE, freq=FAKE, rot=64,
             inter=0, kw=None, wdt=1, eps=1e-6, out=FAKE, ws=WS, wsb=1 << 30):
        s = strides(*ks)
        return L.spec_kv_append(B, T, width, cache() if c is None else c, k, s, v, s, dt, FAKE, index, freq, rot, inter,
                                kw, wdt, eps, out, ws, wsb, None)

    assert call(B=0, k=None) == sv.SPEC_OK
    assert call(B=-1) == E and call(T=0) == E and call(width=0) == E and call(T=(1 << 20) + 1) == E
    assert call(width=4, index=None) == E and call(width=(1 << 20) + 1) == E
    assert call(B=16385, c=cache(num_slots=20000)) == E
    assert call(k=None) == E and call(v=FAKE + 8) == E and call(dt=3) == E and call(ks=(768, 260, 128)) == E
    assert call(rot=8) == E and call(rot=144) == E and call(freq=None) == E and call(inter=-1) == E
    assert call(kw=FAKE + 8) == E and call(wdt=2) == E and call(eps=-0.5) == E and call(out=None) == E
    assert call(ws=None) == sv.SPEC_ERR_WORKSPACE and call(wsb=256) == sv.SPEC_ERR_WORKSPACE
    for bad in CACHE_REFUSALS:
        assert call(c=cache(**bad)) == E, bad


def _tensors(B=2, P=8, H=2, page=16, D=64, M=4, S=2):
    f8 = torch.float8_e4m3fn
    return dict(k_pages=torch.zeros(P, H, page, D, dtype=torch.uint8).view(f8),
                v_pages=torch.zeros(P, H, page, D, dtype=torch.uint8).view(f8), k_scale=torch.ones(P, H),
                v_scale=torch.ones(P, H), k_open=torch.zeros(S, H, 2 * page, D, dtype=torch.bfloat16),
                v_open=torch.zeros(S, H, 2 * page, D, dtype=torch.bfloat16),
                page_table=torch.zeros(B, M, dtype=torch.int32), lengths=torch.zeros(B, dtype=torch.int32))


@pytest.mark.parametrize("pages,heads,page,ok", [((1 << 26) - 1, 2, 16, True), (1 << 26, 2, 16, False),
                                                 (1 << 24, 1, 128, False), ((1 << 31) - 1, 1, 16, False)])
def test_rows_of_the_cache_have_a_limit(L, pages, heads, page, ok):
    """A row of the pages is a 32-bit coordinate: more are refused by both calls that reach them."""
    from speculative_decoding_verify_temperature_b200 import spec_verify as sv
    c = cache(num_pages=pages, kv_heads=heads, page_size=page)
    s = strides(1024, 128 * heads, 128)
    def detail(status):                                   # no output: what is refused next
        assert status == sv.SPEC_ERR_INVALID_ARG
        return L.spec_last_error_detail().decode()

    texts = [detail(L.spec_kv_append(1, 1, 1, c, FAKE, s, FAKE, s, 1, None, None, None, 0, 0, None, 1, 1e-6, None,
                                     WS, 1 << 20, None)),
             detail(L.spec_tree_attention(1, 1, heads, c, FAKE, s, FAKE, s, FAKE, s, None, 1.0, None, None, WS,
                                          1 << 30, None))]
    assert all(("rows" in t) == (not ok) for t in texts), texts


def test_binding_refusals():
    import speculative_decoding_verify_temperature_b200 as spec
    good = spec.KvCache(**_tensors())
    assert (good.B, good.kv_heads, good.page_size, good.head_dim) == (2, 2, 16, 64)
    t = _tensors()
    for name, bad in [("k_pages", t["k_pages"].view(torch.uint8)), ("v_pages", t["v_pages"][:4]),
                      ("k_scale", t["k_scale"].double()), ("v_scale", t["v_scale"].T), ("k_open", t["k_open"].float()),
                      ("v_open", t["v_open"][:, :, :16]), ("page_table", t["page_table"].long()),
                      ("lengths", t["lengths"].long()), ("lengths", t["lengths"][:1]), ("k_open", t["k_open"][:1]),
                      ("page_table", t["page_table"].T.contiguous().T)]:
        with pytest.raises((TypeError, ValueError)):
            spec.KvCache(**{**_tensors(), name: bad})
    with pytest.raises(ValueError):
        spec.KvCache(**_tensors(page=48))
    with pytest.raises(ValueError):
        spec.KvCache(**_tensors(D=96))
    bf = torch.bfloat16
    q, k = torch.zeros(2, 3, 4, 64, dtype=bf), torch.zeros(2, 3, 2, 64, dtype=bf)
    for args in [(q.float(), k, k), (q, k.float(), k), (q, k[:, :2], k), (q, k, k[..., :32]), (q[:1], k[:1], k[:1]),
                 (q, k.transpose(2, 3).contiguous().transpose(2, 3), k)]:
        with pytest.raises((TypeError, ValueError)):
            spec.spec_tree_attention(*args, good)
    with pytest.raises(ValueError, match="CUDA"):
        spec.spec_tree_attention(q, k, k, good)                 # CPU tensors: no fallback
    with pytest.raises(ValueError, match="CUDA"):
        spec.spec_kv_append(k, k, None, good)
    with pytest.raises(TypeError):
        spec.spec_kv_append(k.half(), k.half(), None, good)
    with pytest.raises(ValueError):
        spec.spec_kv_append(k, k, torch.zeros(3, dtype=torch.int32), good)
    with pytest.raises(ValueError, match="CUDA"):
        spec.spec_tree_plan(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        spec.spec_tree_plan(None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        spec.spec_qk_norm_rope(q.half(), k.half(), torch.zeros(2, 3, dtype=torch.int32), None)
    with pytest.raises(TypeError):
        spec.spec_qk_norm_rope(q, k, torch.zeros(2, 3, dtype=torch.int64), None)
    with pytest.raises(TypeError):
        spec.spec_qk_norm_rope(q, k, torch.zeros(2, 3, dtype=torch.int32), None, q_weight=torch.ones(64),
                               k_weight=torch.ones(64, dtype=bf))


def test_reference_plan_by_hand():
    """A seven-node tree worked out by hand."""
    parents = np.array([[-1, 0, 0, 1, 1, 2, 4]], dtype=np.int32)
    pos, words = ref.plan(parents, [10])
    assert pos.tolist() == [[10, 11, 11, 12, 12, 12, 13]]
    assert words[0, :, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10011, 0b100101, 0b1010011]
    m = ref.unpack(torch.from_numpy(words), 7)
    assert torch.equal(ref.pack(m), torch.from_numpy(words))


def test_reference_scale_and_rounding():
    """The block scale brings the largest value within 448, and no smaller power of two does."""
    for a in (448.0, 449.0, 447.0, 1.0, 1.75, 1.7578125, 3.5, 1e-30, 2.0 ** -133, 3e38):
        s = ref.block_scale(a)
        assert a / s <= 448 and (a / (s / 2) > 448 or s == 2.0 ** -126)
    assert ref.block_scale(0.0) == 1.0
    x = torch.tensor([448.0, 0.0, 1.0625, 1.1875, -2.0 ** -9, float("nan"), float("inf")], dtype=torch.float64)
    assert ref.e4m3(x).tolist() == [0x7E, 0, 0x38, 0x3A, 0x81, 0x7F, 0x7F]
