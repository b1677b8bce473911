"""CPU checks of the serving operators: what the C entry points and the binding refuse before any launch, workspace
sizes, valid calls reaching the library, and the plain forms' number format against torch's own 8-bit floats."""
import ctypes
import types

import numpy as np
import pytest

import kvcache_ref as ref
from test_binding_checks import FakeCuda, Recorder

torch = pytest.importorskip("torch")
import mask_aware_flash_b200 as fm  # noqa: E402
from mask_aware_flash_b200 import _build  # noqa: E402

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="hands made-up device addresses to an entry point that can launch")
STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fm.lib()


def cache_c(**kw):
    d = dict(B=2, H_kv=2, D=128, n_pages=10, max_pages=4, code_type=0, k_codes=0x10000, v_codes=0x20000, k_scale=0x30000,
             v_scale=0x40000, page_table=0x50000, weight=0x60000, pos=0x70000)
    d.update(kw)
    return fm.KVCacheC(**d)


BAD_CACHES = [(dict(B=0), 1), (dict(H_kv=0), 1), (dict(n_pages=0), 1), (dict(max_pages=-1), 1), (dict(D=96), 2),
              (dict(code_type=2), 2), (dict(B=65536), 2), (dict(k_codes=None), 1), (dict(v_codes=0x20008), 1),
              (dict(k_scale=None), 1), (dict(page_table=0x50002), 1), (dict(weight=0x60001), 1), (dict(v_scale=0x3), 1),
              (dict(n_pages=1 << 25), 2), (dict(max_pages=1 << 24), 2), (dict(max_pages=1 << 22), 2)]


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(L, bad, code):
    c, good = cache_c(**bad), cache_c()
    p = [0x100000 * (i + 1) for i in range(6)]
    a = fm.CacheAttnArgs(H=4, n_q=1, dtype=0, scale=0.1, q=p[0], len=p[1])
    r = ctypes.byref
    assert L.fm_cache_append(r(c), p[0], p[1], 0, 3, p[2], None, None, None) == code
    assert L.fm_cache_attn(r(c), r(a), p[2], p[3], p[4], 1 << 40, None) == code
    assert L.fm_cache_attn_workspace_bytes(r(c), r(a)) == 0
    assert L.fm_cache_evict(r(c), r(good), p[0], 64, 0, p[1], p[2], 1 << 40, None) == code
    assert L.fm_cache_evict_workspace_bytes(r(c), 64) == 0
    assert L.fm_cache_append(None, p[0], p[1], 0, 3, p[2], None, None, None) == fm.FM_ERR_INVALID_ARG


def test_append_refusals(L):
    c = ctypes.byref(cache_c())
    f = L.fm_cache_append
    assert f(c, None, 0x10000, 0, 1, 0x20000, None, None, None) == fm.FM_ERR_INVALID_ARG
    assert f(c, 0x10000, 0x10000, 0, 0, 0x20000, None, None, None) == fm.FM_ERR_INVALID_ARG    # no token
    assert f(c, 0x10000, 0x10000, 0, 1, None, None, None, None) == fm.FM_ERR_INVALID_ARG       # no start
    assert f(c, 0x10008, 0x10000, 0, 1, 0x20000, None, None, None) == fm.FM_ERR_INVALID_ARG    # alignment
    assert f(c, 0x10000, 0x10000, 0, 1, 0x20002, None, None, None) == fm.FM_ERR_INVALID_ARG
    assert f(c, 0x10000, 0x10000, 0, 1, 0x20000, 0x3, None, None) == fm.FM_ERR_INVALID_ARG
    assert f(c, 0x10000, 0x10000, 2, 1, 0x20000, None, None, None) == fm.FM_ERR_UNSUPPORTED    # element type


@pytest.mark.parametrize("bad,code", [
    (dict(H=3), 1), (dict(H=0), 1), (dict(n_q=0), 1), (dict(dtype=1), 2), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(causal=2), 1), (dict(accumulate=2), 1), (dict(Hm=3, n_k=8), 1), (dict(Hm=0, n_k=8), 1),
    (dict(Hm=1, n_k=0), 1), (dict(H=2 * 65), 2), (dict(H=128, n_q=17), 2), (dict(q=None), 1), (dict(q=0x100008), 1),
    (dict(len=None), 1), (dict(len=0x200002), 1), (dict(causal=1), 1),                              # causal without row
    (dict(vec=fm.VecArray(0x9000, None, None, None)), 1),                                           # vectors without Hm, n_k
    (dict(vec=fm.VecArray(0x9000, None, None, None), Hm=1, n_k=64), 1),                             # vectors without row
    (dict(vec=fm.VecArray(0x9001, None, None, None), Hm=1, n_k=64, row=0x8000), 1),
])
def test_attention_refusals(L, bad, code):
    d = dict(H=4, n_q=2, dtype=0, scale=0.1, q=0x100000, len=0x200000)
    d.update(bad)
    a = fm.CacheAttnArgs(**d)
    assert L.fm_cache_attn(ctypes.byref(cache_c()), ctypes.byref(a), 0x300000, 0x400000, 0x500000, 1 << 40, None) == code


def test_attention_workspace(L):
    a = fm.CacheAttnArgs(H=4, n_q=1, dtype=0, scale=0.1, q=0x100000, len=0x200000)
    c = cache_c()
    r = ctypes.byref
    plain = L.fm_cache_attn_workspace_bytes(r(c), r(a))
    assert plain > 0 and plain % 256 == 0
    assert L.fm_cache_attn(r(c), r(a), 0x300000, 0x400000, None, plain, None) == fm.FM_ERR_WORKSPACE
    assert L.fm_cache_attn(r(c), r(a), 0x300000, 0x400000, 0x500080, plain, None) == fm.FM_ERR_WORKSPACE
    assert L.fm_cache_attn(r(c), r(a), 0x300000, 0x400000, 0x500000, plain - 1, None) == fm.FM_ERR_WORKSPACE
    assert L.fm_cache_attn(r(c), r(a), None, 0x400000, 0x500000, plain, None) == fm.FM_ERR_INVALID_ARG
    assert L.fm_cache_attn(r(c), r(a), 0x300000, 0x400002, 0x500000, plain, None) == fm.FM_ERR_INVALID_ARG
    a.accumulate = 1
    more = L.fm_cache_attn_workspace_bytes(r(c), r(a))
    assert more >= plain + 2 * 2 * 4 * 64 * 4 * 4  # a score per slot and row (rows rounded up to 4)
    assert L.fm_cache_attn(r(c), r(a), 0x300000, 0x400000, 0x500000, plain, None) == fm.FM_ERR_WORKSPACE
    none = cache_c(weight=None)
    assert L.fm_cache_attn(r(none), r(a), 0x300000, 0x400000, 0x500000, more, None) == fm.FM_ERR_INVALID_ARG
    assert L.fm_cache_attn_workspace_bytes(r(none), r(a)) == 0


@pytest.mark.parametrize("D,group,n_q", [(64, 1, 1), (128, 4, 1), (256, 2, 3)])
@pytest.mark.parametrize("B,H_kv,max_pages", [(1, 1, 1), (1100, 8, 4), (8192, 8, 8), (65535, 8, 16), (33, 1, 31), (3, 2, 5000),
                                              (300, 8, 33), (64, 8, 2048)])
def test_attention_workspace_goes_with_the_table(L, D, group, n_q, B, H_kv, max_pages):
    """Without weights: a word per listed block (two where lists are shorter than their room), a word per (sequence, head) and list, and
    the partial sums of 148 CTAs."""
    a = fm.CacheAttnArgs(H=H_kv * group, n_q=n_q, dtype=0, scale=0.1, q=0x100000, len=0x200000)
    c = cache_c(B=B, H_kv=H_kv, D=D, max_pages=max_pages, n_pages=1 << 16)
    got = L.fm_cache_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(a))
    rows = -(-n_q * group // 8) * 8
    parts = 2 * 148 * rows * (D + 2) * 4
    assert 0 < got <= B * H_kv * (8 * max_pages + 8) + parts + 8 * 256


def test_evict_refusals(L):
    src, dst = cache_c(), cache_c(k_codes=0x110000, v_codes=0x120000, k_scale=0x130000, v_scale=0x140000, page_table=0x150000,
                                  weight=0x160000, pos=0x170000, max_pages=2)
    r = ctypes.byref
    n = L.fm_cache_evict_workspace_bytes(r(src), 100)
    assert n >= 2 * 2 * 100 * 4 and n % 256 == 0 and L.fm_cache_evict_workspace_bytes(r(src), 0) == 0

    def f(src=src, dst=dst, len_=0x200000, budget=100, recent=10, new=0x210000, ws=0x300000, nbytes=n):
        return L.fm_cache_evict(r(src), r(dst), len_, budget, recent, new, ws, nbytes, None)
    inv = fm.FM_ERR_INVALID_ARG
    assert f(budget=0) == inv and f(budget=129) == inv and f(recent=-1) == inv and f(recent=101) == inv
    assert f(len_=None) == inv and f(new=None) == inv and f(len_=0x200001) == inv
    assert f(src=cache_c(weight=None)) == inv
    assert f(dst=cache_c(D=64, weight=None, pos=None)) == inv and f(dst=cache_c(code_type=1, weight=None, pos=None)) == inv
    assert f(dst=cache_c(weight=None, pos=None)) == inv                      # the same pages
    assert f(dst=cache_c(page_table=0x150000)) == inv                        # the same weight
    assert f(dst=cache_c(page_table=0x150000, weight=None)) == inv           # the same pos
    assert f(ws=None) == fm.FM_ERR_WORKSPACE and f(ws=0x300010) == fm.FM_ERR_WORKSPACE
    assert f(nbytes=n - 1) == fm.FM_ERR_WORKSPACE


def test_evict_refuses_overlapping_weights_and_positions(L):
    """Another cache's weight or pos that shares some of its words: slots would be read after others were written."""
    r = ctypes.byref
    src = cache_c(weight=0x200000, pos=0x300000)    # 2 x 2 x 256 words: 0x1000 bytes each
    far = dict(page_table=0x150000, weight=0x400000, pos=0x500000, max_pages=2)  # 0x800 bytes each

    def f(**kw):  # (without a workspace: FM_ERR_WORKSPACE where the caches are accepted, and never a launch)
        return L.fm_cache_evict(r(src), r(cache_c(**dict(far, **kw))), 0x600000, 100, 10, 0x610000, None, 0, None)
    assert f() == fm.FM_ERR_WORKSPACE and f(weight=None, pos=None) == fm.FM_ERR_WORKSPACE
    for name, other in (("weight", 0x200000), ("pos", 0x300000), ("weight", 0x300000), ("pos", 0x200000)):
        for at in (other, other + 4, other + 0xFFC, other - 0x7FC):
            assert f(**{name: at}) == fm.FM_ERR_INVALID_ARG, (name, hex(at))
        for at in (other + 0x1000, other - 0x800):  # side by side
            assert f(**{name: at}) == fm.FM_ERR_WORKSPACE, (name, hex(at))


def key_weight_args(**kw):
    d = dict(B=1, H=4, n_q=256, n_k=256, D=128, dtype=0, scale=0.1, q=0x10000, k=0x20000, H_kv=2)
    d.update(kw)
    m = fm.MaskMetaC()
    m.d = fm.MaskDesc(1, 1, 256, 256, 128, 128)
    m.row_count = m.row_entries = m.col_count = m.col_entries = m.tile_minmax = 0x40000
    m.tile_class = m.fwd_order = m.bwd_order = 0x40000
    return fm.AttnArgs(**d), m


def test_key_weight_refusals(L):
    vec = fm.VecArray(None, None, None, None)

    def f(lse=0x50000, w=0x60000, stride=256, acc=0, **kw):
        a, m = key_weight_args(**kw)
        return L.fm_attn_key_weight(ctypes.byref(a), ctypes.byref(m), vec, lse, w, stride, acc, None)
    assert f(dtype=1, D=64) == fm.FM_ERR_UNSUPPORTED and f(D=96) == fm.FM_ERR_UNSUPPORTED
    assert f(n_k=254) == fm.FM_ERR_UNSUPPORTED
    assert f(H_kv=3) == fm.FM_ERR_INVALID_ARG and f(k=None) == fm.FM_ERR_INVALID_ARG and f(n_q=128) == fm.FM_ERR_INVALID_ARG
    assert f(lse=None) == fm.FM_ERR_INVALID_ARG and f(w=0x60002) == fm.FM_ERR_INVALID_ARG
    assert f(stride=255) == fm.FM_ERR_INVALID_ARG and f(acc=2) == fm.FM_ERR_INVALID_ARG
    assert L.fm_attn_key_weight(None, None, vec, 0x50000, 0x60000, 256, 0, None) == fm.FM_ERR_INVALID_ARG


# ------------------------------------------------------------------------------------------------- binding
def fake_cache(B=2, H_kv=2, D=128, max_pages=4, n_pages=10, dtype=torch.int8, device="cuda:0", **kw):
    f = lambda shape, t: FakeCuda(shape, t, device=device)  # noqa: E731
    d = dict(k_codes=f((n_pages, H_kv, 64, D), dtype), v_codes=f((n_pages, H_kv, 64, D), dtype),
             k_scale=f((n_pages, H_kv), torch.float32), v_scale=f((n_pages, H_kv), torch.float32),
             page_table=f((B, max_pages), torch.int32), weight=f((B, H_kv, max_pages * 64), torch.float32),
             pos=f((B, H_kv, max_pages * 64), torch.int32))
    d.update(kw)
    return fm.KVCache(**d)


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(fm, "lib", lambda: r)
    return r


def ints(*shape):
    return FakeCuda(shape, torch.int32)


@no_gpu
@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_valid_calls_reach_the_library(rec, dtype):
    c = fake_cache(dtype=dtype)
    kv = FakeCuda((2, 3, 2, 128), torch.bfloat16)
    fm.fm_cache_append(c, kv, kv, ints(2), stream=STREAM)
    kv32 = FakeCuda((2, 3, 2, 128), torch.float32)
    fm.fm_cache_append(c, kv32, kv32, ints(2), count=ints(2), row=ints(2), stream=STREAM)
    q, ws = FakeCuda((2, 1, 8, 128), torch.bfloat16), FakeCuda((4096,), torch.uint8)
    out = dict(o=q, lse=FakeCuda((2, 8, 1), torch.float32), ws=ws, stream=STREAM)
    fm.fm_cache_attn(c, q, ints(2), 0.1, **out)
    fm.fm_cache_attn(c, q, ints(2), 0.1, row=ints(2), vecs=[ints(2, 8, 50), None, None, ints(2, 8, 50)], causal=True,
                     accumulate=True, **out)
    d = fake_cache(dtype=dtype, max_pages=2)
    fm.fm_cache_evict(c, d, ints(2), 100, recent=5, new_len=ints(2), ws=ws, stream=STREAM)
    assert rec.calls == ["fm_cache_append"] * 2 + ["fm_cache_attn"] * 2 + ["fm_cache_evict"]


@pytest.mark.parametrize("bad", [
    dict(k_codes=FakeCuda((10, 2, 64, 128), torch.uint8)), dict(k_codes=FakeCuda((10, 2, 32, 128), torch.int8)),
    dict(k_codes=FakeCuda((10, 2, 64, 96), torch.int8)), dict(v_codes=FakeCuda((10, 2, 64, 128), torch.float8_e4m3fn)),
    dict(v_codes=FakeCuda((9, 2, 64, 128), torch.int8)), dict(k_scale=FakeCuda((10, 2), torch.float16)),
    dict(v_scale=FakeCuda((10, 3), torch.float32)), dict(page_table=FakeCuda((2, 4), torch.int64)),
    dict(page_table=FakeCuda((8,), torch.int32)), dict(weight=FakeCuda((2, 2, 255), torch.float32)),
    dict(pos=FakeCuda((2, 2, 256), torch.int64)), dict(pos=FakeCuda((2, 2, 256), torch.int32, contiguous=False)),
    dict(k_scale=FakeCuda((10, 2), torch.float32, device="cuda:1"))])
def test_cache_rejects_bad_tensors(rec, bad):
    with pytest.raises(fm.FmError):
        fake_cache(**bad)


@pytest.mark.parametrize("name", ["k_codes", "v_codes", "k_scale", "v_scale", "page_table", "weight", "pos", "B", "max_pages", "c"])
def test_cache_keeps_the_tensors_it_was_made_with(rec, name):
    """Calls use the addresses taken when the cache was made: another tensor in an attribute would free the one they point at."""
    c, other = fake_cache(), fake_cache()
    was = getattr(c, name)
    with pytest.raises(AttributeError, match=name):
        setattr(c, name, getattr(other, name))
    with pytest.raises(AttributeError, match=name):
        delattr(c, name)
    with pytest.raises(AttributeError):
        c.anything_else = 1
    assert getattr(c, name) is was


def test_calls_reject_bad_tensors(rec):
    c = fake_cache()
    kv = FakeCuda((2, 3, 2, 128), torch.bfloat16)
    q, ws = FakeCuda((2, 1, 8, 128), torch.bfloat16), FakeCuda((4096,), torch.uint8)
    good = dict(o=q, lse=FakeCuda((2, 8, 1), torch.float32), ws=ws, stream=STREAM)
    bad_calls = [
        lambda: fm.fm_cache_append(c, kv, FakeCuda((2, 3, 2, 128), torch.float32), ints(2), stream=STREAM),
        lambda: fm.fm_cache_append(c, FakeCuda((2, 3, 4, 128), torch.bfloat16), kv, ints(2), stream=STREAM),
        lambda: fm.fm_cache_append(c, FakeCuda((2, 3, 2, 128), torch.float16), kv, ints(2), stream=STREAM),
        lambda: fm.fm_cache_append(c, kv, kv, FakeCuda((2,), torch.int64), stream=STREAM),
        lambda: fm.fm_cache_append(c, kv, kv, ints(2), count=ints(3), stream=STREAM),
        lambda: fm.fm_cache_append(c, torch.zeros((2, 3, 2, 128), dtype=torch.bfloat16), kv, ints(2), stream=STREAM),
        lambda: fm.fm_cache_attn(c, FakeCuda((2, 1, 8, 128), torch.float32), ints(2), 0.1, **good),
        lambda: fm.fm_cache_attn(c, FakeCuda((3, 1, 8, 128), torch.bfloat16), ints(3), 0.1, **good),
        lambda: fm.fm_cache_attn(c, q, FakeCuda((2,), torch.int64), 0.1, **good),
        lambda: fm.fm_cache_attn(c, q, ints(2), 0.1, row=ints(2), vecs=[ints(2, 1, 50), ints(2, 1, 51), None, None], **good),
        lambda: fm.fm_cache_attn(c, q, ints(2), 0.1, row=ints(2), vecs=[ints(2, 50), None, None, None], **good),
        lambda: fm.fm_cache_attn(c, q, ints(2), 0.1, **dict(good, lse=FakeCuda((2, 1, 8), torch.float32))),
        lambda: fm.fm_cache_attn(c, q, ints(2), 0.1, **dict(good, o=FakeCuda((2, 1, 8, 128), torch.bfloat16, contiguous=False))),
        lambda: fm.fm_cache_evict(fake_cache(weight=None), fake_cache(max_pages=2), ints(2), 100, new_len=ints(2), ws=ws, stream=STREAM),
        lambda: fm.fm_cache_evict(c, fake_cache(D=64), ints(2), 100, new_len=ints(2), ws=ws, stream=STREAM),
        lambda: fm.fm_cache_evict(c, fake_cache(max_pages=2), ints(3), 100, new_len=ints(2), ws=ws, stream=STREAM),
        lambda: fm.fm_cache_evict(c, fake_cache(max_pages=2), ints(2), 100, new_len=ints(2), ws=FakeCuda((8,), torch.int32), stream=STREAM),
        lambda: fm.fm_cache_evict(c, fake_cache(max_pages=2, device="cuda:1"), ints(2), 100, new_len=ints(2), ws=ws, stream=STREAM),
    ]
    for call in bad_calls:
        with pytest.raises(fm.FmError):
            call()
    assert not {"fm_cache_append", "fm_cache_attn", "fm_cache_evict"} & set(rec.calls)


@no_gpu
def test_key_weight_binding(rec):
    m = fm.MaskMeta.__new__(fm.MaskMeta)
    m.desc, m.c = fm.MaskDesc(2, 1, 300, 512, 128, 128), fm.MaskMetaC()
    q, k = FakeCuda((2, 300, 4, 128), torch.bfloat16), FakeCuda((2, 512, 2, 128), torch.bfloat16)
    lse, vecs = FakeCuda((2, 4, 300), torch.float32), [FakeCuda((2, 1, 512), torch.int32)] + [None] * 3
    w = FakeCuda((2, 2, 640), torch.float32)
    fm.fm_attn_key_weight(q, k, lse, m, vecs, 0.1, weight=w, accumulate=True, stream=STREAM)
    assert rec.calls == ["fm_attn_key_weight"]
    for bad in (dict(weight=FakeCuda((2, 2, 511), torch.float32)), dict(weight=FakeCuda((2, 4, 512), torch.float32)),
                dict(weight=None, accumulate=True), dict(weight=FakeCuda((2, 1024), torch.float32))):
        with pytest.raises(fm.FmError):
            fm.fm_attn_key_weight(q, k, lse, m, vecs, 0.1, stream=STREAM, **bad)
    with pytest.raises(fm.FmError):
        fm.fm_attn_key_weight(q, FakeCuda((2, 512, 2, 64), torch.bfloat16), lse, m, vecs, 0.1, weight=w, stream=STREAM)
    with pytest.raises(fm.FmError):  # host tensors, all of them
        host = [torch.zeros(x.shape, dtype=x.dtype) for x in (q, k, lse)]
        fm.fm_attn_key_weight(*host, m, [torch.zeros((2, 1, 512), dtype=torch.int32)] + [None] * 3, 0.1, stream=STREAM)
    assert rec.calls == ["fm_attn_key_weight"]


# --------------------------------------------------------------------------------- the plain forms themselves
def test_plain_codes_match_torch():
    x = np.float32(np.random.default_rng(0).standard_normal(20000) * 60).astype(np.float64)
    ties = (ref.E4M3[1:] + ref.E4M3[:-1]) / 2
    for y in (x, ties, -ties, np.array([0.0, 1e-9, 448, 500, np.inf, -np.inf])):
        want = torch.from_numpy(np.clip(y, -448, 448).astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
        np.testing.assert_array_equal(ref.encode(y, "e4m3"), want)
    np.testing.assert_array_equal(ref.encode(np.array([0.5, 1.5, -2.5, 126.5, 300, np.nan, -np.inf]), "int8"),
                                  [0, 2, -2, 126, 127, 0, -127])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_plain_scale_rule(code):
    q = ref.QMAX[code]
    for a in (1.0, q, np.nextafter(q, 1e9), q / 2, 3e38, 2.0 ** -126, 1e-45, 0.3):
        s = ref.scale_rule(a, code)
        assert s * q >= a and (s == 2.0 ** -126 or s / 2 * q < a) and math_is_power(s)
    assert ref.scale_rule(0.0, code) == 0.0


def math_is_power(s):
    m, _ = np.frexp(s)
    return m == 0.5


def test_plain_cache_requantises_an_open_block():
    """A larger token moves the older codes of its block to the larger scale with one rounding each."""
    c = ref.Cache(1, 1, 64, 2, "int8")
    k = np.full((1, 3, 1, 64), 5.0)
    c.append(k, k, [0])
    assert c.scale["k"][0, 0, 0] == 2.0 ** -4 and (c.units["k"][0, 0, 0, :3] == 80).all()
    big = np.full((1, 1, 1, 64), 127.0 * 32)
    c.append(big, big, [3], row=[9])
    assert c.scale["k"][0, 0, 0] == 32.0
    assert (c.units["k"][0, 0, 0, :3] == np.rint(80 / 512)).all() and (c.units["k"][0, 0, 0, 3] == 127).all()
    assert list(c.pos[0, 0, :4]) == [0, 1, 2, 9]
