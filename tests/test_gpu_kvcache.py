"""The serving operators on the GPU against plain float64 forms (kvcache_ref.py).

Codes and scales of a cache are compared for equality: scales are powers of two, so every quotient is exact and a code
has a single rounding to nearest even.

Bounds of the attention (eps = 2^-24, a half step of fp32):
  score   the products of the fp16 operands are exact; their fp32 sum of D terms is off by at most D 2^-23 of the sum of
          magnitudes a_ij = scale sum_d |q_d k_d| (2^-23: the tensor core's adder may cut instead of round); scaling to
          log2 units, the row maximum's subtraction and the exponential add a few eps of |s| and 2^-22.  So
          p_ij = exp(s_ij - lse) is off by a factor within exp(+-delta), delta = (D + 8) 2^-23 max_j a_ij + 2^-20.
  LSE     within delta, and n eps from the sum of n terms, 2^-22 |lse| from the conversion to natural units.
  O       p is rounded to fp16 for the product with V (2^-11 of itself), sums are fp32, the result is rounded to bf16
          (2^-8): |dO| <= 2^-8 |O| + (2^-11 + 2 delta + n 2^-23) sum_j p_j |v_j|.
  weight  |dw| <= sum_i p_ij (2 delta + n 2^-23 + rows eps) + rows 2^-23 |w|.
"""
import math

import numpy as np
import pytest

import kvcache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
PAGE = 64


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mask_aware_flash_b200 import _build
    _build.build()
    import mask_aware_flash_b200 as m
    m.lib()
    return m


def bf16(x):
    """float64 array of bf16 numbers, and its CUDA tensor."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


class Pair:
    """A cache on the GPU, its pages shuffled among `spare` more than it uses, and its float64 counterpart."""

    def __init__(self, fm, B, H_kv, D, max_pages, code, seed=0, spare=3, fill=0, pools=None):
        r = np.random.default_rng(seed)
        n_pages = B * max_pages + spare
        pool = (n_pages, H_kv, PAGE, D)
        raw = [torch.full(pool, fill, dtype=torch.uint8, device="cuda").view(CODES[code]) for _ in range(2)]
        self.table = r.permutation(n_pages)[:B * max_pages].reshape(B, max_pages)
        self.t = fm.KVCache(*raw, *(torch.full((n_pages, H_kv), 7.0, device="cuda") for _ in range(2)), i32(self.table),
                            weight=torch.full((B, H_kv, max_pages * PAGE), 3.0, device="cuda"),
                            pos=torch.full((B, H_kv, max_pages * PAGE), -5, dtype=torch.int32, device="cuda"))
        self.ref = ref.Cache(B, H_kv, D, max_pages, code)
        self.B, self.H_kv, self.D, self.max_pages, self.code = B, H_kv, D, max_pages, code

    def append(self, fm, k, v, start, count=None, row=None):
        kd, kt = bf16(k)
        vd, vt = bf16(v)
        opt = lambda x: None if x is None else i32(x)  # noqa: E731
        fm.fm_cache_append(self.t, kt, vt, i32(start), count=opt(count), row=opt(row))
        self.ref.append(kd, vd, start, count, row)

    def check(self, lens):
        """Values, scales, weights and positions of the first lens[b] slots, equal bit for bit."""
        for name, codes, scale in (("k", self.t.k_codes, self.t.k_scale), ("v", self.t.v_codes, self.t.v_scale)):
            c = codes.float().double().cpu().numpy()
            s = scale.double().cpu().numpy()
            for b in range(self.B):
                for blk in range(-(-int(lens[b]) // PAGE)):
                    page, n = self.table[b, blk], min(PAGE, int(lens[b]) - blk * PAGE)
                    np.testing.assert_array_equal(s[page], self.ref.scale[name][b, :, blk], err_msg=f"{name} scale {b} {blk}")
                    np.testing.assert_array_equal(c[page][:, :n], self.ref.units[name][b, :, blk, :n],
                                                  err_msg=f"{name} codes {b} {blk}")
        for got, want in ((self.t.weight, self.ref.weight), (self.t.pos, self.ref.pos)):
            got = got.cpu().numpy()
            for b in range(self.B):
                np.testing.assert_array_equal(got[b, :, :int(lens[b])], want[b, :, :int(lens[b])])


def tokens(r, B, n, H_kv, D, spread=1.0):
    """K, V whose tokens differ in size, so that blocks' scales grow as tokens arrive."""
    size = np.exp2(r.uniform(-spread, spread, (B, n, H_kv, 1)))
    return r.standard_normal((B, n, H_kv, D)) * size, r.standard_normal((B, n, H_kv, D)) * size


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_token_by_token_and_in_runs(fm, D, code):
    B, H_kv = 3, 2
    r = np.random.default_rng(D)
    c = Pair(fm, B, H_kv, D, 5, code, seed=D)
    lens = np.array([0, 5, 63])
    k, v = tokens(r, B, 63, H_kv, D)
    c.append(fm, k, v, [0, 0, 0], count=lens)
    c.check(lens)
    for n_new in (1, 1, 2, 1, 70, 1, 128):  # single tokens over a page's end, runs over several pages
        k, v = tokens(r, B, n_new, H_kv, D, spread=3.0)
        c.append(fm, k, v, lens, row=lens + 11)
        lens = lens + n_new
        c.check(np.minimum(lens, 5 * PAGE))
    assert fm.fm_get_device_status() == 0


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_leaves_the_rest_alone(fm, code):
    """Slots behind the last new token, pages of nobody, tokens without a slot, counts out of range, absent pages."""
    B, H_kv, D = 4, 1, 64
    r = np.random.default_rng(1)
    c = Pair(fm, B, H_kv, D, 2, code, fill=0x33)
    c.t.page_table[3, 0] = -1           # not there
    c.t.page_table[2, 1] = 1 << 30      # not there either
    before = [x.view(torch.uint8).clone() for x in (c.t.k_codes, c.t.v_codes)]
    k, v = tokens(r, B, 90, H_kv, D)
    start, count = np.array([10, 100, 0, 0]), np.array([3, 200, 90, 90])
    c.append(fm, k, v, start, count=count)
    c.ref.scale["k"][2, :, 1] = c.ref.scale["k"][3, :, 0] = 0
    for x, was in zip((c.t.k_codes, c.t.v_codes), before):
        x = x.view(torch.uint8)
        # sequence 0: 10 old slots (fill, scale 7: re-quantised only if the scale grows), 3 new, the rest untouched
        assert torch.equal(x[c.table[0, 0], :, 13:], was[c.table[0, 0], :, 13:])
        assert torch.equal(x[c.table[0, 1]], was[c.table[0, 1]])
        assert torch.equal(x[c.table[1, 0]], was[c.table[1, 0]])
        unused = [p for p in range(x.shape[0]) if p not in c.table]
        assert torch.equal(x[unused], was[unused])
        assert torch.equal(x[c.table[2, 1]], was[c.table[2, 1]])
        assert torch.equal(x[c.table[3, 0]], was[c.table[3, 0]])
    w = c.t.weight.cpu().numpy()
    assert (w[0, 0, :10] == 3).all() and (w[0, 0, 10:13] == 0).all() and (w[0, 0, 13:] == 3).all()
    assert (w[1, 0, :100] == 3).all() and (w[1, 0, 100:128] == 0).all()
    assert (w[2, 0, 64:] == 3).all() and (w[3, 0, :64] == 3).all() and (w[3, 0, 64:90] == 0).all()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_extreme_values(fm, code):
    """Zeros, infinities, NaN, the largest and smallest bf16 numbers, exact ties, whole blocks of each."""
    D = 64
    c = Pair(fm, 1, 1, D, 6, code)
    r = np.random.default_rng(2)
    k, v = tokens(r, 1, 6 * PAGE, 1, D)
    k[0, :64] = 0
    k[0, 70, 0, 3], k[0, 71, 0, 4], k[0, 72, 0, 5] = np.inf, -np.inf, np.nan
    k[0, 128:192] = np.nan
    k[0, 192:256] *= 2.0 ** 120
    k[0, 200, 0, 0] = 3.3895313892515355e38
    k[0, 256:320] *= 2.0 ** -130
    k[0, 320:] = (np.arange(64 * 64).reshape(64, 1, 64) % 255 - 127) / 2.0  # int8: halves; e4m3: many ties
    c.append(fm, k, v, [0])
    c.check([6 * PAGE])


def test_append_float32_input(fm):
    B, H_kv, D = 2, 3, 128
    r = np.random.default_rng(3)
    c = Pair(fm, B, H_kv, D, 3, "int8")
    k, v = (x.astype(np.float32) for x in tokens(r, B, 130, H_kv, D))
    fm.fm_cache_append(c.t, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32([0, 33]))
    c.ref.append(k.astype(np.float64), v.astype(np.float64), [0, 33])
    got, want = c.t.k_codes[c.table[0, 0]].double().cpu().numpy(), c.ref.units["k"][0, :, 0]
    np.testing.assert_array_equal(got, want)
    got = c.t.v_codes[c.table[1, 1]].double().cpu().numpy()
    np.testing.assert_array_equal(got, c.ref.units["v"][1, :, 1])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_float32_values_and_runs(fm, D, code):
    """fp32 tokens of every kind: numbers that no bf16 holds, the largest and the subnormal ones, infinities and NaN, runs over
    pages' ends and single tokens into open blocks whose scale grows."""
    B, H_kv, max_pages = 2, 2, 5
    r = np.random.default_rng(D + 7)
    c = Pair(fm, B, H_kv, D, max_pages, code, seed=D)
    lens = np.array([0, 50])
    for scale in (c.t.k_scale, c.t.v_scale):  # sequence 1 begins behind 50 slots of zeros
        scale.zero_()
    c.ref.weight[1, :, :50], c.ref.pos[1, :, :50] = 3.0, -5
    first = True
    for n_new in (200, 1, 1, 30):
        k, v = (x.astype(np.float32) for x in tokens(r, B, n_new, H_kv, D, spread=4.0))
        if first:
            k[0, :64] *= np.float32(2.0 ** -140)   # a block of subnormal numbers
            k[0, 64, 0, :5] = [np.inf, -np.inf, np.nan, 3.4028235e38, -1e-45]
            v[0, 130:192] = np.nan
            v[1, 3, 1, 7] = 1e38
        first = False
        start = lens.copy()
        fm.fm_cache_append(c.t, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(start), row=i32(start + 3))
        c.ref.append(k.astype(np.float64), v.astype(np.float64), start, row=start + 3)
        lens = lens + n_new
        c.check(lens)
    assert fm.fm_get_device_status() == 0


# --------------------------------------------------------------------------------------------- attention
def mask_vectors(kind, n, B, Hm, r):
    """Four int32 arrays [B, Hm, n] (or None each)."""
    j = np.arange(n)
    out = np.zeros((4, B, Hm, n), np.int64)
    for b in range(B):
        for h in range(Hm):
            if kind == "window":
                w = 40 + 3 * h + b
                x = (np.minimum(j + w, n), np.full(n, n), np.zeros(n), j)
            elif kind == "document":
                d = 50 + 7 * h + b
                x = (np.minimum((j // d + 1) * d, n), np.full(n, n), np.zeros(n), j)
            elif kind == "all":      # every row masked for every key
                x = (np.zeros(n), np.full(n, 1 << 30), np.zeros(n), np.zeros(n))
            else:                    # random stretches, some empty, some past the rows
                x = tuple(r.integers(-20, n + 20, n) for _ in range(4))
            out[:, b, h] = x
    vecs = list(out.astype(np.int32))
    if kind == "random":
        vecs[int(r.integers(4))] = None
    return vecs


def run_attention(fm, c, lens, q, scale, row, vecs, causal, accumulate, **kw):
    vt = None if vecs is None else [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in vecs]
    return fm.fm_cache_attn(c.t, q, i32(lens), scale, row=None if row is None else i32(row), vecs=vt, causal=causal,
                            accumulate=accumulate, **kw)


def check_attention(c, lens, qd, o, lse, scale, row, vecs, causal, weight_before=None):
    B, n_q, H, D = qd.shape
    G = H // c.H_kv
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    weight = None if weight_before is None else c.t.weight.double().cpu().numpy()
    for b in range(B):
        n = int(lens[b])
        for hk in range(c.H_kv):
            K, V = c.ref.values("k", b, hk)[:n], c.ref.values("v", b, hk)[:n]
            j = c.ref.pos[b, hk, :n] if c.t.pos is not None else np.arange(n)
            add, slack = np.zeros(n), np.zeros(n)
            for hg in range(G):
                h = hk * G + hg
                i = (0 if row is None else int(row[b])) + np.arange(n_q)
                hv = None if vecs is None else [None if x is None else x[b, h if x.shape[1] > 1 else 0] for x in vecs]
                n_k = 0 if vecs is None else next(x for x in vecs if x is not None).shape[-1]
                ok = ref.seen(j, i, hv, n_k, causal)
                O, L, p, mag, absum = ref.attention(qd[b, :, h], K, V, ok, scale)
                delta = ((D + 8) * 2.0 ** -23 * np.where(ok, mag, 0).max(-1, initial=0) + 2.0 ** -20)
                tol = 2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2 * delta + n * 2.0 ** -23)[:, None] * absum + 1e-37
                live = ok.any(-1)
                err = np.abs(o[b, :, h] - O)
                assert (err <= tol).all(), f"b {b} head {h}: O off by {np.max(err - tol)} over its bound"
                assert (o[b, :, h][~live] == 0).all() and np.isneginf(lse[b, h][~live]).all()
                if live.any():
                    bound = (delta + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(L))[live]
                    e = np.abs(lse[b, h] - L)[live]
                    assert (e <= bound).all(), f"b {b} head {h}: LSE off by {e.max()}, bound {bound.min()}"
                add += p.sum(0)
                slack += (p * (2 * delta + n * 2.0 ** -23 + G * n_q * 2.0 ** -24)[:, None]).sum(0)
            if weight is not None:
                want = weight_before[b, hk, :n] + add
                e = np.abs(weight[b, hk, :n] - want)
                assert (e <= slack + G * n_q * 2.0 ** -23 * np.abs(want)).all(), f"b {b} K/V head {hk}: weight off by {e.max()}"
                np.testing.assert_array_equal(weight[b, hk, n:], weight_before[b, hk, n:])


def filled(fm, B, H_kv, D, lens, code, seed, max_pages=None, fill=0, gaps=False):
    r = np.random.default_rng(seed)
    most = max(int(max(lens)), 1)
    c = Pair(fm, B, H_kv, D, max_pages or -(-most // PAGE), code, seed=seed, fill=fill)
    k, v = tokens(r, B, most, H_kv, D)
    c.append(fm, k, v, np.zeros(B, int), count=lens)
    if gaps:  # positions with gaps, other ones in each head, as an eviction leaves them
        pos = np.cumsum(r.integers(1, 4, c.ref.pos.shape), -1) - 1
        c.ref.pos[:] = pos
        c.t.pos.copy_(torch.from_numpy(pos.astype(np.int32)))
    c.ref.weight[:] = 0
    c.t.weight.copy_(torch.from_numpy(r.uniform(0, 2, c.ref.weight.shape).astype(np.float32)))
    return c, r


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [(1,), (64, 65), (0, 1, 63, 500), (3000,)])
def test_attention_lengths(fm, D, code, lens):
    H_kv, G, B = 2, 4, len(lens)
    c, r = filled(fm, B, H_kv, D, lens, code, seed=sum(lens) + D, fill=0x7F)  # unwritten e4m3 slots hold NaN codes
    qd, q = bf16(1.5 * r.standard_normal((B, 1, H_kv * G, D)))
    scale = 1 / math.sqrt(D)
    before = c.t.weight.double().cpu().numpy()
    o, lse = run_attention(fm, c, lens, q, scale, None, None, False, True)
    assert fm.fm_get_device_status() == 0
    check_attention(c, lens, qd, o, lse, scale, None, None, False, before)
    o2, lse2 = run_attention(fm, c, lens, q, scale, None, None, False, False)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H_kv,G,n_q", [(1, 1, 1), (3, 1, 2), (2, 7, 1), (1, 8, 2), (2, 5, 5), (1, 16, 3), (1, 64, 1)])
def test_attention_heads_and_rows(fm, D, H_kv, G, n_q):
    """Row counts below, at and over a tile of 8 and over what one CTA holds."""
    lens = (130, 700)
    c, r = filled(fm, 2, H_kv, D, lens, "int8", seed=G + n_q)
    qd, q = bf16(r.standard_normal((2, n_q, H_kv * G, D)))
    row = np.array(lens) - n_q
    before = c.t.weight.double().cpu().numpy()
    o, lse = run_attention(fm, c, lens, q, 0.11, row, None, True, True)
    assert fm.fm_get_device_status() == 0
    check_attention(c, lens, qd, o, lse, 0.11, row, None, True, before)


@pytest.mark.parametrize("kind", ["window", "document", "all", "random"])
@pytest.mark.parametrize("Hm_all", [False, True])
@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_masks(fm, kind, Hm_all, gaps, causal):
    B, H_kv, G, n_q, D = 2, 2, 3, 3, 128
    lens = (40, 1500)
    c, r = filled(fm, B, H_kv, D, lens, "e4m3", seed=len(kind) + 2 * Hm_all + gaps, gaps=gaps)
    H = H_kv * G
    n = 2500
    vecs = mask_vectors(kind, n, B, H if Hm_all else 1, r)
    row = np.array([38, 2400 if gaps else 1495])
    qd, q = bf16(r.standard_normal((B, n_q, H, D)))
    before = c.t.weight.double().cpu().numpy()
    o, lse = run_attention(fm, c, lens, q, 0.09, row, vecs, causal, True)
    assert fm.fm_get_device_status() == 0
    check_attention(c, lens, qd, o, lse, 0.09, row, vecs, causal, before)


def test_attention_absent_pages_are_masked(fm):
    lens = (400,)
    c, r = filled(fm, 1, 1, 64, lens, "int8", seed=9)
    c.t.page_table[0, 2], c.t.page_table[0, 4] = -7, c.t.n_pages
    qd, q = bf16(r.standard_normal((1, 1, 2, 64)))
    before = c.t.weight.double().cpu().numpy()
    o, lse = run_attention(fm, c, lens, q, 0.125, None, None, False, True)
    # a key that is not there is a masked key: the same mask by vectors
    hide = np.zeros((1, 1, 448), np.int32)
    hide[0, 0, 128:192] = hide[0, 0, 256:320] = 1 << 20
    check_attention(c, lens, qd, o, lse, 0.125, np.array([0]), [None, None, np.zeros_like(hide), hide], False, before)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_attention_scales_far_apart(fm, code):
    """Blocks whose scales differ by large powers of two, in both directions, and blocks of zeros."""
    D, n = 128, 64 * 12
    r = np.random.default_rng(5)
    c = Pair(fm, 1, 1, D, 12, code)
    k, v = tokens(r, 1, n, 1, D)
    for blk, e in enumerate([0, 20, -20, 0, 60, -60, 0, -100, 100, 3, 0, -3]):
        v[0, blk * 64:(blk + 1) * 64] *= 2.0 ** e
        k[0, blk * 64:(blk + 1) * 64] *= 2.0 ** min(0, e)
    v[0, 640:704] = 0
    k[0, 192:256] = 0
    c.append(fm, k, v, [0])
    c.t.weight.zero_()
    qd, q = bf16(r.standard_normal((1, 1, 8, D)))
    o, lse = run_attention(fm, c, [n], q, 0.1, None, None, False, True)
    check_attention(c, [n], qd, o, lse, 0.1, None, None, False, np.zeros((1, 1, n)))
    # queries far outside fp16's range give the same scores with a scale that undoes them
    for e in (100, -100):
        qs = (q.float() * 2.0 ** e).to(torch.bfloat16)
        o2, lse2 = run_attention(fm, c, [n], qs, 0.1 * 2.0 ** -e, None, None, False, False)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attention_one_key_returns_its_value(fm):
    """A row that sees one key gets that key's value, rounded to bf16 once."""
    D = 64
    c, r = filled(fm, 1, 2, D, (200,), "int8", seed=11)
    n = 200
    vecs = [None, None, np.zeros((1, 1, n), np.int32), np.full((1, 1, n), 1 << 20, np.int32)]
    vecs[3][0, 0, 77] = 0
    _, q = bf16(r.standard_normal((1, 1, 4, D)))
    o, lse = run_attention(fm, c, [n], q, 0.3, np.array([199]), vecs, False, False)
    for h in range(4):
        want = torch.from_numpy(c.ref.values("v", 0, h // 2)[77]).to(torch.bfloat16)
        assert torch.equal(o[0, 0, h].cpu(), want)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 200, 3000])
def test_attention_of_the_largest_values(fm, D, code, n):
    """Values at the upper end of fp32: one key seen returns its value, equal keys return theirs, others their average."""
    big = {"int8": 127 * 2.0 ** 121, "e4m3": 448 * 2.0 ** 119}[code]  # the largest code under the largest scale
    r = np.random.default_rng(n + D)
    c = Pair(fm, 1, 1, D, -(-n // PAGE), code)
    k = r.standard_normal((1, n, 1, D))
    sign = np.where(r.integers(0, 2, D) > 0, 1.0, -1.0)
    c.append(fm, k, np.tile(big * sign, (1, n, 1, 1)), [0])
    qd, q = bf16(r.standard_normal((1, 2, 3, D)))
    o, _ = run_attention(fm, c, [n], q, 0.1, None, None, False, False)
    assert fm.fm_get_device_status() == 0
    assert torch.equal(o.double().cpu(), torch.from_numpy(np.broadcast_to(big * sign, (1, 2, 3, D)).copy()))
    # every row sees one key only, another one each (row t: key at[t])
    at = r.integers(0, n, 2)
    vecs = [np.full((1, 1, n), x, np.int32) for x in (0, 1, 1, 2)]  # both rows masked, each by one stretch
    vecs[1][0, 0, at[0]] = 0
    vecs[3][0, 0, at[1]] = 1
    o, lse = run_attention(fm, c, [n], q, 0.1, np.array([0]), vecs, False, False)
    assert torch.equal(o.double().cpu(), torch.from_numpy(np.broadcast_to(big * sign, (1, 2, 3, D)).copy()))
    # values of either sign and of several sizes, the largest 2^126
    v = r.uniform(-1, 1, (1, n, 1, D)) * np.exp2(126 - r.integers(0, 6, (1, n, 1, 1)))
    c.append(fm, k, v, [0])
    o, lse = run_attention(fm, c, [n], q, 0.1, None, None, False, False)
    check_attention(c, [n], qd, o, lse, 0.1, None, None, False)


def test_attention_streams_workspaces_and_graphs(fm):
    """A poisoned workspace, another stream, a captured and replayed call whose inputs change, two graphs that share a
    workspace (replayed one after the other), and equal bits every time."""
    B, H_kv, G, D = 3, 2, 4, 128
    lens = (900, 64, 2000)
    c, r = filled(fm, B, H_kv, D, lens, "e4m3", seed=21)
    qd, q = bf16(r.standard_normal((B, 1, H_kv * G, D)))
    n = i32(lens)
    want_o, want_lse = fm.fm_cache_attn(c.t, q, n, 0.1)
    ws = torch.full((fm.fm_cache_attn_workspace_bytes(c.t, q, accumulate=True),), 0xFF, dtype=torch.uint8, device="cuda")
    w0 = c.t.weight.clone()
    o, lse = fm.fm_cache_attn(c.t, q, n, 0.1, accumulate=True, ws=ws)
    first = c.t.weight.clone()
    assert torch.equal(o, want_o) and torch.equal(lse, want_lse) and torch.isfinite(first).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.t.weight.copy_(w0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        o2, lse2 = fm.fm_cache_attn(c.t, q, n, 0.1, accumulate=True, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(o2, want_o) and torch.equal(c.t.weight, first)
    outs, graphs = [], []
    for _ in range(2):
        go, gl = torch.empty_like(want_o), torch.empty_like(want_lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fm.fm_cache_attn(c.t, q, n, 0.1, o=go, lse=gl, ws=ws)
        outs.append((go, gl))
        graphs.append(graph)
    for rep in range(2):
        for graph, (go, gl) in zip(graphs, outs):
            go.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(go, want_o) and torch.equal(gl, want_lse)
    n.copy_(i32([1, 0, 1999]))  # the lengths are read on the device: a replay sees the new ones
    graphs[0].replay()
    torch.cuda.synchronize()
    short_o, short_lse = fm.fm_cache_attn(c.t, q, n, 0.1)
    assert torch.equal(outs[0][0], short_o) and torch.equal(outs[0][1], short_lse)
    check_attention(c, (1, 0, 1999), qd, short_o, short_lse, 0.1, None, None, False)
    assert fm.fm_get_device_status() == 0


def test_attention_pool_beyond_32_bits(fm):
    """Pages whose bytes lie past 2^32 in their pool, and more blocks per CTA than one list holds."""
    D, H_kv = 64, 8
    n_pages = (1 << 32) // (H_kv * PAGE * D) + 300
    n = 148 * 600 // H_kv * PAGE  # 600 blocks for each CTA
    pages = n // PAGE
    g = torch.Generator(device="cuda").manual_seed(4)
    pool = [torch.empty((n_pages, H_kv, PAGE, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.zeros((n_pages, H_kv), device="cuda") for _ in range(2)]
    table = (n_pages - 1 - torch.randperm(pages, generator=g, device="cuda")).to(torch.int32)[None].contiguous()
    for p, s in zip(pool, scale):
        p[table[0].long()] = torch.randint(-127, 128, (pages, H_kv, PAGE, D), generator=g, device="cuda", dtype=torch.int8)
        s[table[0].long()] = torch.exp2(torch.randint(-7, -4, (pages, H_kv), generator=g, device="cuda").float())
    cache = fm.KVCache(*pool, *scale, table)
    q = torch.randn((1, 1, H_kv * 2, D), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = fm.fm_cache_attn(cache, q, i32([n - 5]), 0.125)
    assert fm.fm_get_device_status() == 0
    for hk in (0, 5):
        K, V = ((p[table[0].long(), hk].double() * s[table[0].long(), hk].double()[:, None, None]).view(-1, D)[:n - 5]
                for p, s in zip(pool, scale))
        sc = 0.125 * q[0, 0, 2 * hk:2 * hk + 2].double() @ K.T
        L = torch.logsumexp(sc, -1)
        p = torch.exp(sc - L[:, None])
        mag = 0.125 * (q[0, 0, 2 * hk:2 * hk + 2].double().abs() @ K.abs().T).amax(-1)
        delta = (D + 8) * 2.0 ** -23 * mag + 2.0 ** -20
        O, absum = p @ V, p @ V.abs()
        # sums: each run's fp32 sums have at most 64 * 600 terms, 148 runs are joined
        tol = 2.0 ** -8 * O.abs() + (2.0 ** -11 + 2 * delta + 40000 * 2.0 ** -23)[:, None] * absum
        assert ((o[0, 0, 2 * hk:2 * hk + 2].double() - O).abs() <= tol).all()
        assert ((lse[0, 2 * hk:2 * hk + 2, 0].double() - L).abs() <= delta + 40000 * 2.0 ** -24 + 2.0 ** -22 * L.abs()).all()


def shared_page_cache(fm, B, H_kv, D, max_pages, n_pages, code, g, weight=False):
    """A cache whose table entries point at few pages, many sequences at the same ones (as prompts that share a prefix do)."""
    pools = [torch.randint(-100, 101, (n_pages, H_kv, PAGE, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
    if code == "e4m3":
        pools = [(p.float() / 16).to(torch.float8_e4m3fn) for p in pools]
    scales = [torch.exp2(torch.randint(-8, -4, (n_pages, H_kv), generator=g, device="cuda").float()) for _ in range(2)]
    table = torch.randint(0, n_pages, (B, max_pages), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((B, H_kv, max_pages * PAGE), generator=g, device="cuda") if weight else None
    return fm.KVCache(*pools, *scales, table, weight=w)


def check_sequence(cache, b, hk, n, q, o, lse, scale, ok=None):
    """One (sequence, K/V head) against float64 torch, with the bounds above.  q [n_q, G, D], o likewise, lse [G, n_q];
    ok [n_q, n]: which keys each query sees."""
    pages = cache.page_table[b, :-(-n // PAGE)].long()
    K, V = ((c[pages, hk].double() * s[pages, hk].double()[:, None, None]).reshape(-1, cache.D)[:n]
            for c, s in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)))
    qd = q.double()
    s = scale * torch.einsum("tgd,nd->tgn", qd, K)
    mag = scale * torch.einsum("tgd,nd->tgn", qd.abs(), K.abs())
    if ok is not None:
        s = s.masked_fill(~ok[:, None, :], float("-inf"))
        mag = mag.masked_fill(~ok[:, None, :], 0)
    L = torch.logsumexp(s, -1)
    live = torch.isfinite(L)
    p = torch.where(live[..., None], torch.exp(s - torch.where(live, L, 0)[..., None]), 0)
    delta = (cache.D + 8) * 2.0 ** -23 * mag.amax(-1) + 2.0 ** -20
    O, absum = torch.einsum("tgn,nd->tgd", p, V), torch.einsum("tgn,nd->tgd", p, V.abs())
    tol = 2.0 ** -8 * O.abs() + (2.0 ** -11 + 2 * delta + n * 2.0 ** -23)[..., None] * absum + 1e-37
    assert ((o.double() - O).abs() <= tol).all(), f"sequence {b} head {hk}: O off by {(o.double() - O).abs().max()}"
    got = lse.double().T
    assert torch.isneginf(got[~live]).all()
    assert ((got - L)[live].abs() <= (delta + n * 2.0 ** -24 + 2.0 ** -22 * L.abs())[live]).all()


@pytest.mark.parametrize("code,D,G", [("int8", 64, 2), ("int8", 64, 11), ("int8", 128, 3), ("e4m3", 128, 5), ("e4m3", 256, 2)])
@pytest.mark.parametrize("B,H_kv,max_pages", [(24, 4, 30), (1, 1, 1500), (5, 2, 3)])
def test_attention_zero_scales_over_codes_that_are_not(fm, code, D, G, B, H_kv, max_pages):
    """A pool of the caller's own may hold any codes under a scale of 0: their values are 0, as keys and as values."""
    g = torch.Generator(device="cuda").manual_seed(D + G + B)
    cache = shared_page_cache(fm, B, H_kv, D, max_pages, 90, code, g)
    cache.v_scale[::3] = 0
    cache.k_scale[::5] = 0
    lens = np.random.default_rng(B).integers(max_pages * 30, max_pages * PAGE + 1, B)
    if B == 5:
        cache.page_table[1] = 3   # a sequence of such blocks alone, and one that begins, one that ends with them
        cache.page_table[2, 0] = cache.page_table[3, -1] = 6
    q = torch.randn((B, 1, H_kv * G, D), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = fm.fm_cache_attn(cache, q, i32(lens), 0.1)
    assert fm.fm_get_device_status() == 0
    for b in range(B) if B == 5 else {0, B // 2, B - 1}:
        for hk in {0, H_kv - 1}:
            heads = slice(hk * G, hk * G + G)
            check_sequence(cache, b, hk, int(lens[b]), q[b, :, heads], o[b, :, heads], lse[b, heads], 0.1)
    if B == 5:
        assert (o[1] == 0).all()


def test_attention_many_sequences_and_long_masks(fm):
    """More (sequence, head) lists than threads, chunks of more than 64 blocks, masks over several chunks, empty sequences."""
    B, H_kv, G, D, max_pages, n_q = 520, 8, 2, 64, 200, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = shared_page_cache(fm, B, H_kv, D, max_pages, 60, "int8", g)
    r = np.random.default_rng(3)
    lens = r.integers(0, 300, B)
    lens[[5, 77, 519]] = [12000, 12800, 9001]
    n = int(max_pages * PAGE)
    j = np.arange(n)
    vecs = [np.broadcast_to(x, (B, 1, n)).astype(np.int32) for x in (np.minimum(j + 3000, n), np.full(n, n), np.zeros(n), j)]
    vecs[0][:, :, :200] = n  # the first keys stay visible: the seen blocks are two stretches of the list
    vt = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in vecs]
    q = torch.randn((B, n_q, H_kv * G, D), generator=g, device="cuda").to(torch.bfloat16)
    row = np.maximum(lens - n_q, 0)
    o, lse = fm.fm_cache_attn(cache, q, i32(lens), 0.125, row=i32(row), vecs=vt)
    assert fm.fm_get_device_status() == 0
    for b in (0, 5, 77, 300, 518, 519):
        m = int(lens[b])
        if m == 0:
            continue
        ok = torch.from_numpy(ref.seen(np.arange(m), row[b] + np.arange(n_q), [x[b, 0] for x in vecs], n, False)).cuda()
        for hk in (0, 7):
            check_sequence(cache, b, hk, m, q[b, :, hk * G:hk * G + G], o[b, :, hk * G:hk * G + G], lse[b, hk * G:hk * G + G],
                           0.125, ok)
    empty = torch.from_numpy(lens == 0).cuda()
    assert (o[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    none_o, none_lse = fm.fm_cache_attn(cache, q, torch.zeros(B, dtype=torch.int32, device="cuda"), 0.125)
    assert (none_o == 0).all() and torch.isneginf(none_lse).all()


def far_apart(fm, kind, code, D, G, B, H_kv, max_pages, seed):
    """A cache whose pages fall into three classes, in random order along each sequence: cache, class of each block, q, row, vectors."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_pages = 90
    cls = torch.arange(n_pages, device="cuda") % 3
    codes = [torch.randint(-20, 21, (n_pages, H_kv, PAGE, D), generator=g, device="cuda").float(),
             torch.randint(-100, 101, (n_pages, H_kv, PAGE, D), generator=g, device="cuda").float()]
    exps = {"seen": (100, 0, -100), "columns": (45, 0, -45), "weights": (100, 0, 0), "negative": (30, 0, -30)}[kind]
    scale = [torch.full((n_pages, H_kv), 2.0 ** -7, device="cuda"),
             torch.exp2(torch.tensor(exps, device="cuda").float())[cls][:, None].repeat(1, H_kv)]
    q = torch.randn((B, 3, H_kv * G, D), generator=g, device="cuda")
    if kind == "columns":   # an element of V that only the smaller classes have, another that only the smallest has
        codes[1][cls == 0, :, :, 5] = 0
        codes[1][cls <= 1, :, :, 17] = 0
    if kind == "weights":   # keys of the first class have softmax weights some 2^-45 of the others'
        codes[0][:, :, :, 0] = torch.where(cls == 0, -100.0, 100.0)[:, None, None]
        q[..., 0] = 200.0
    if kind == "negative":  # any scales of a pool of the caller's own: negative ones, and no powers of two
        scale = [s * (torch.rand(s.shape, generator=g, device="cuda") + 0.999) for s in scale]
        scale = [torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.5, s, -s) for s in scale]
    if code == "e4m3":
        codes, scale[0] = [x / 16 for x in codes], scale[0] * 16
    codes = [x.to(CODES[code]) for x in codes]
    table = torch.randint(0, n_pages, (B, max_pages), generator=g, device="cuda", dtype=torch.int32)
    row = torch.arange(B, device="cuda", dtype=torch.int32) + 5000
    vecs = None
    if kind == "seen":      # query 1 sees none of the first class, query 2 only the third
        of = cls[table.long()].repeat_interleave(PAGE, 1)[:, None]
        at = row[:, None, None]
        zero = torch.zeros_like(of, dtype=torch.int32)
        vecs = [torch.where(of == 0, at + 1, zero), torch.where(of == 0, at + 3, zero),
                torch.where(of == 1, at + 2, zero), torch.where(of == 1, at + 3, zero)]
        vecs = [x.to(torch.int32).contiguous() for x in vecs]
    return fm.KVCache(*codes, *scale, table), q.to(torch.bfloat16), row, vecs


@pytest.mark.parametrize("kind", ["seen", "columns", "weights", "negative"])
@pytest.mark.parametrize("code,D,G", [("int8", 64, 1), ("int8", 64, 11), ("int8", 128, 1), ("e4m3", 128, 5), ("e4m3", 256, 2)])
@pytest.mark.parametrize("B,H_kv,max_pages", [(24, 4, 30), (1, 1, 1500)])
def test_attention_value_scales_and_weights_far_apart(fm, kind, code, D, G, B, H_kv, max_pages):
    """V scales whose ratios are far beyond fp16's range, several such blocks in the hands of each warp, in every order: rows that do
    not see the larger ones, elements that these do not have, and large values under small weights keep their bits."""
    cache, q, row, vecs = far_apart(fm, kind, code, D, G, B, H_kv, max_pages, seed=D + G + B)
    lens = np.random.default_rng(D + B).integers(max_pages * 30, max_pages * PAGE + 1, B)
    o, lse = fm.fm_cache_attn(cache, q, i32(lens), 0.1, row=row, vecs=vecs)
    assert fm.fm_get_device_status() == 0
    for b in {0, B // 2, B - 1}:
        n = int(lens[b])
        ok = None
        if vecs is not None:
            i = row[b].long() + torch.arange(3, device="cuda")[:, None]
            lts, lte, uts, ute = (x[b, 0, None, :n].long() for x in vecs)
            ok = ~(((lts <= i) & (i < lte)) | ((uts <= i) & (i < ute)))
        for hk in {0, H_kv - 1}:
            heads = slice(hk * G, hk * G + G)
            check_sequence(cache, b, hk, n, q[b, :, heads], o[b, :, heads], lse[b, heads], 0.1, ok)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_as_many_rows_as_a_call_takes(fm, D):
    g = torch.Generator(device="cuda").manual_seed(D)
    cache = shared_page_cache(fm, 1, 1, D, 30, 30, "e4m3", g)
    q = torch.randn((1, 16, 64, D), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = fm.fm_cache_attn(cache, q, i32([1900]), 0.1, row=i32([1884]), causal=True)
    ok = torch.arange(1900, device="cuda") <= 1884 + torch.arange(16, device="cuda")[:, None]
    check_sequence(cache, 0, 0, 1900, q[0], o[0], lse[0], 0.1, ok)


def test_attention_calls_on_two_streams_at_once(fm):
    """Two calls over one cache that may run at the same time, a workspace each."""
    g = torch.Generator(device="cuda").manual_seed(8)
    cache = shared_page_cache(fm, 6, 4, 128, 100, 80, "int8", g)
    q = [torch.randn((6, 1, 16, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    n = i32([6400, 1, 3000, 0, 64, 5999])
    want = [fm.fm_cache_attn(cache, x, n, 0.1) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(fm.fm_cache_attn(cache, q[k], n, 0.1))
    torch.cuda.synchronize()
    for k in range(2):
        for o, lse in got[k]:
            assert torch.equal(o, want[k][0]) and torch.equal(lse, want[k][1])


def test_what_a_call_allocates_belongs_to_its_stream(fm, monkeypatch):
    """Workspace and results of a call on a stream that is not the current one come from that stream's memory."""
    g = torch.Generator(device="cuda").manual_seed(2)
    cache, dst = (shared_page_cache(fm, 2, 2, 64, 4, 8, "int8", g, weight=True) for _ in range(2))
    dst.page_table.copy_(torch.arange(8, dtype=torch.int32).view(2, 4))
    q, n = torch.randn((2, 1, 4, 64), generator=g, device="cuda").to(torch.bfloat16), i32([200, 100])
    want = fm.fm_cache_attn(cache, q, n, 0.1)
    torch.cuda.synchronize()
    side, seen = torch.cuda.Stream(), []
    for name in ("empty", "empty_like"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _real=real, **k: (seen.append(torch.cuda.current_stream()), _real(*a, **k))[1])
    got = fm.fm_cache_attn(cache, q, n, 0.1, stream=side)
    fm.fm_cache_evict(cache, dst, n, 64, stream=side)
    assert len(seen) == 5 and all(x == side for x in seen) and torch.cuda.current_stream() != side
    side.synchronize()
    monkeypatch.undo()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_step_captured_and_replayed(fm):
    """Append, attention with weights and the length's increment in one graph, replayed token by token, against the same
    calls made one by one: equal bits."""
    B, H_kv, G, D, steps = 2, 2, 4, 64, 70
    r = np.random.default_rng(1)
    k, v = (bf16(x)[1] for x in tokens(r, B, steps, H_kv, D, spread=2.0))
    q = bf16(r.standard_normal((B, steps, H_kv * G, D)))[1]

    def run(graphed):
        cache = fm.fm_cache_alloc(B, H_kv, D, 128)
        ks, vs, qs = (torch.zeros_like(x[:, :1]).contiguous() for x in (k, v, q))
        at, n = torch.tensor([0, 7], dtype=torch.int32, device="cuda"), torch.tensor([1, 8], dtype=torch.int32, device="cuda")
        o, lse = torch.empty_like(qs), torch.empty((B, H_kv * G, 1), device="cuda")
        ws = torch.empty(fm.fm_cache_attn_workspace_bytes(cache, qs, accumulate=True), dtype=torch.uint8, device="cuda")
        outs = []

        def step():
            fm.fm_cache_append(cache, ks, vs, at)
            fm.fm_cache_attn(cache, qs, n, 0.125, row=at, causal=True, accumulate=True, o=o, lse=lse, ws=ws)
            at.add_(1)
            n.add_(1)
        graph = None
        for t in range(steps):
            for dst, src in ((ks, k), (vs, v), (qs, q)):
                dst.copy_(src[:, t:t + 1])
            if graphed and t == 1:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            if graph is None:
                step()
            else:
                graph.replay()
            outs.append((o.clone(), lse.clone()))
        torch.cuda.synchronize()
        return outs, cache
    a, ca = run(False)
    b, cb = run(True)
    for (o1, l1), (o2, l2) in zip(a, b):
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert torch.equal(ca.k_codes, cb.k_codes) and torch.equal(ca.v_scale, cb.v_scale) and torch.equal(ca.weight, cb.weight)
    # every step hands out one unit of weight per query head: a weight is exp(s - lse), off by the relative error of both
    # exponents (delta each, as above) and of at most 77 additions and as many into the cache
    mag = 0.125 * q.float().abs().sum(-1).max() * k.float().abs().max() * (1 + 2.0 ** -6)
    units, delta = steps * B * H_kv * G, (D + 8) * 2.0 ** -23 * mag + 2.0 ** -20
    assert abs(float(ca.weight.double().sum()) - units) <= units * (2 * delta + 200 * 2.0 ** -24)
    assert fm.fm_get_device_status() == 0


# --------------------------------------------------------------------------------------------- key weight
def prompt(fm, B, n_q, n_k, H, H_kv, D, vecs, seed):
    r = np.random.default_rng(seed)
    qd, q = bf16(r.standard_normal((B, n_q, H, D)))
    kd, k = bf16(r.standard_normal((B, n_k, H_kv, D)))
    vt = [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in vecs]
    if all(x is None for x in vt):
        vt[2] = torch.zeros((B, 1, n_k), dtype=torch.int32, device="cuda")
    meta = fm.fm_build_mask_meta(*vt, n_q=n_q)
    _, lse = fm.fm_attn_fwd(q, k, k, meta, vt, 1 / math.sqrt(D))
    return qd, q, kd, k, vt, meta, lse


def check_key_weight(qd, kd, vecs, lse, got, scale, before=0.0):
    """p_ij = exp(s_ij - lse_i) with the forward's fp32 lse taken as it is; sums of up to G n_q terms."""
    B, n_q, H, D = qd.shape
    H_kv, n_k = kd.shape[2], kd.shape[1]
    G = H // H_kv
    lse = lse.double().cpu().numpy()
    for b in range(B):
        for hk in range(H_kv):
            want, slack = np.zeros(n_k), np.zeros(n_k)
            for h in range(hk * G, hk * G + G):
                hv = [None if x is None else x[b, h if x.shape[1] > 1 else 0] for x in vecs]
                j = np.arange(n_k)
                hv = [np.full(n_k, d) if x is None else x for x, d in zip(hv, (n_q, n_q, 0, 0))]
                ok = ref.seen(j, np.arange(n_q), hv, n_k, False) & np.isfinite(lse[b, h])[:, None]
                s = scale * (qd[b, :, h] @ kd[b, :, hk].T)
                with np.errstate(all="ignore"):
                    p = np.where(ok, np.exp(s - lse[b, h][:, None]), 0.0)
                mag = scale * (np.abs(qd[b, :, h]) @ np.abs(kd[b, :, hk]).T)
                L = np.where(np.isfinite(lse[b, h]), np.abs(lse[b, h]), 0)[:, None]
                want += p.sum(0)
                slack += (p * ((D + 8) * 2.0 ** -23 * mag + 2.0 ** -21 * L + 2.0 ** -20 + G * n_q * 2.0 ** -24)).sum(0)
            e = np.abs(got[b, hk] - (want + before))
            assert (e <= slack + 2.0 ** -23 * np.abs(want + before) + 1e-37).all(), f"{b} {hk}: {np.max(e - slack)}"
            assert (got[b, hk][want == 0] == before).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n_q,n_k", [(1, 4), (128, 128), (300, 516), (1000, 1000), (129, 2052)])
@pytest.mark.parametrize("H,H_kv,Hm_all", [(2, 2, False), (4, 1, True), (6, 2, True)])
def test_key_weight(fm, D, n_q, n_k, H, H_kv, Hm_all):
    r = np.random.default_rng(n_q + D)
    B = 2
    kind = ("window", "document", "random")[(n_q + H) % 3]
    vecs = mask_vectors(kind, n_k, B, H if Hm_all else 1, r)
    qd, q, kd, k, vt, meta, lse = prompt(fm, B, n_q, n_k, H, H_kv, D, vecs, seed=n_k)
    scale = 1 / math.sqrt(D)
    w = fm.fm_attn_key_weight(q, k, lse, meta, vt, scale)
    assert fm.fm_get_device_status() == 0
    check_key_weight(qd, kd, vecs, lse, w.double().cpu().numpy(), scale)
    again = fm.fm_attn_key_weight(q, k, lse, meta, vt, scale)
    assert torch.equal(w, again)
    # into rows of a wider weight, added to what is there
    wide = torch.full((B, H_kv, n_k + 60), 0.5, device="cuda")
    fm.fm_attn_key_weight(q, k, lse, meta, vt, scale, weight=wide, accumulate=True)
    check_key_weight(qd, kd, vecs, lse, wide[:, :, :n_k].double().cpu().numpy(), scale, before=0.5)
    assert (wide[:, :, n_k:] == 0.5).all()


def test_key_weight_rows_that_see_nothing(fm):
    n = 260
    vecs = mask_vectors("window", n, 1, 1, None)
    vecs[0][:], vecs[1][:] = 100, 200  # rows 100 .. 199 masked for every key
    qd, q, kd, k, vt, meta, lse = prompt(fm, 1, n, n, 2, 1, 64, vecs, seed=3)
    assert torch.isneginf(lse[:, :, 100:200]).all()
    w = fm.fm_attn_key_weight(q, k, lse, meta, vt, 0.125)
    check_key_weight(qd, kd, vecs, lse, w.double().cpu().numpy(), 0.125)
    # every live row's weights add up to one
    assert abs(float(w.double().sum()) - 2 * 160) < 1e-2


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,H_kv,Hm_all", [(8, 8, True), (12, 6, False)])
def test_key_weight_more_key_tiles_than_sms(fm, D, H, H_kv, Hm_all):
    """Several key tiles a CTA: long lists, short ones, empty ones and whole sequences of empty ones, one after the other."""
    B, n_q, n_k = 2, 700, 2500
    r = np.random.default_rng(D + H)
    vecs = [np.array(x) for x in mask_vectors("window", n_k, B, H if Hm_all else 1, r)]
    for x, fill in zip(vecs, (0, 1 << 30, 0, 0)):
        x[:, :, 640:1300] = fill                     # key tiles that no row sees
        x[0, 0, :] = fill                            # a head, or a whole sequence, that sees nothing
    for x, fill in zip(vecs, (n_q, n_q, 0, 0)):
        x[:, -1, 1300:1900] = fill                   # key tiles that every row sees
    qd, q, kd, k, vt, meta, lse = prompt(fm, B, n_q, n_k, H, H_kv, D, vecs, seed=n_k)
    scale = 1 / math.sqrt(D)
    w = fm.fm_attn_key_weight(q, k, lse, meta, vt, scale)
    check_key_weight(qd, kd, vecs, lse, w.double().cpu().numpy(), scale)
    # two at once, and replayed from a graph: the same bits
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(3):
        for x in streams:
            with torch.cuda.stream(x):
                got.append(fm.fm_attn_key_weight(q, k, lse, meta, vt, scale))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for x in got)
    out, graph = torch.zeros_like(w), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fm.fm_attn_key_weight(q, k, lse, meta, vt, scale, weight=out, accumulate=True)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2 * w) and fm.fm_get_device_status() == 0


def test_key_weight_nan_rows_reach_the_keys_they_see(fm):
    n, window = 300, 40
    vecs = mask_vectors("window", n, 1, 1, None)
    qd, q, kd, k, vt, meta, lse = prompt(fm, 1, n, n, 2, 1, 64, vecs, seed=3)
    lse[0, 1, 150] = float("nan")
    w = fm.fm_attn_key_weight(q, k, lse, meta, vt, 0.125)
    j = torch.arange(n, device="cuda")
    assert torch.equal(torch.isnan(w[0, 0]), (j > 150 - window) & (j <= 150))


# -------------------------------------------------------------------------------------------------- evict
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("budget,recent", [(1, 0), (64, 64), (100, 17), (200, 0), (333, 64)])
def test_evict(fm, D, code, budget, recent):
    B, H_kv = 4, 2
    lens = np.array([0, 90, 333, 1000])
    c, r = filled(fm, B, H_kv, D, lens, code, seed=budget, gaps=True)
    w = np.exp(r.standard_normal(c.ref.weight.shape)).astype(np.float32)
    w[3, 0, 100:300] = 0.75     # ties
    w[3, 1] = 0.0               # nothing but ties
    w[2, 0, 5], w[2, 0, 7], w[2, 0, 9], w[2, 1, 3] = np.nan, np.inf, -np.inf, -0.0
    c.t.weight.copy_(torch.from_numpy(w))
    c.ref.weight[:] = w
    d = Pair(fm, B, H_kv, D, -(-budget // PAGE), code, seed=1, fill=0x7F)
    ws = torch.full((fm.fm_cache_evict_workspace_bytes(c.t, budget),), 0xFF, dtype=torch.uint8, device="cuda")
    n = i32(lens)
    got = fm.fm_cache_evict(c.t, d.t, n, budget, recent=recent, ws=ws)
    want = c.ref.evict(d.ref, lens, budget, recent)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    d.check(want)
    tail = want[3] % PAGE
    if tail:  # behind the last kept slot of a block: zeros
        assert (d.t.k_codes[d.table[3, want[3] // PAGE]].float()[:, tail:] == 0).all()
    # in place of the lengths
    fm.fm_cache_evict(c.t, d.t, n, budget, recent=recent, new_len=n)
    np.testing.assert_array_equal(n.cpu().numpy(), want)
    d.check(want)
    # the evicted cache is read like any other
    qd, q = bf16(r.standard_normal((B, 1, H_kv * 2, D)))
    d.t.pos.copy_(torch.from_numpy(d.ref.pos.astype(np.int32)))
    o, lse = fm.fm_cache_attn(d.t, q, n, 0.1)
    check_attention(d, want, qd, o, lse, 0.1, None, None, False)


def test_evict_within_one_pool(fm):
    """src and dst tables over the same pools, other pages."""
    B, H_kv, D = 2, 2, 64
    lens = np.array([700, 650])
    c, r = filled(fm, B, H_kv, D, lens, "int8", seed=3)
    n_pages = c.t.n_pages
    grow = lambda x: torch.cat([x, torch.zeros_like(x[:2 * B])])  # noqa: E731
    pools = [grow(x) for x in (c.t.k_codes, c.t.v_codes, c.t.k_scale, c.t.v_scale)]
    src = fm.KVCache(*pools, c.t.page_table, weight=c.t.weight, pos=c.t.pos)
    table = torch.arange(n_pages, n_pages + 2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    dst = fm.KVCache(*pools, table, weight=torch.zeros((B, H_kv, 128), device="cuda"))
    c.ref.weight[:] = c.t.weight.cpu().numpy()
    new_len = fm.fm_cache_evict(src, dst, i32(lens), 128, recent=20)
    d = ref.Cache(B, H_kv, D, 2, "int8")
    c.ref.evict(d, lens, 128, 20)
    assert (new_len == 128).all()
    got = dst.k_codes[table.long()].double().cpu().numpy()  # [B, 2, H_kv, 64, D]
    np.testing.assert_array_equal(got.transpose(0, 2, 1, 3, 4), d.units["k"])
    np.testing.assert_array_equal(dst.weight.double().cpu().numpy(), d.weight)


@pytest.mark.parametrize("B,H_kv,max_pages", [(64, 4, 800), (1, 2, 6200), (3, 5, 300)])
def test_evict_long_lists(fm, B, H_kv, max_pages):
    """Selections whose keys do not fit a CTA's shared memory, that a cluster shares, and in between, against a stable sort."""
    g = torch.Generator(device="cuda").manual_seed(B)
    src = shared_page_cache(fm, B, H_kv, 64, max_pages, 12, "int8", g, weight=True)
    src.weight.copy_(torch.floor(src.weight * 5000) / 5000)  # many ties
    cap, budget, recent = max_pages * PAGE, max_pages * PAGE // 5 + 3, 77
    lens = torch.randint(cap // 2, cap + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = cap
    dst_pages = -(-budget // PAGE)
    dst = fm.KVCache(*(torch.zeros((B * dst_pages, H_kv, PAGE, 64), dtype=torch.int8, device="cuda") for _ in range(2)),
                     *(torch.zeros((B * dst_pages, H_kv), device="cuda") for _ in range(2)),
                     torch.arange(B * dst_pages, dtype=torch.int32, device="cuda").view(B, dst_pages),
                     weight=torch.zeros((B, H_kv, dst_pages * PAGE), device="cuda"),
                     pos=torch.zeros((B, H_kv, dst_pages * PAGE), dtype=torch.int32, device="cuda"))
    new_len = fm.fm_cache_evict(src, dst, lens, budget, recent=recent)
    assert (new_len == budget).all() and fm.fm_get_device_status() == 0
    for b in {0, B // 2, B - 1}:
        for h in range(H_kv):
            n = int(lens[b])
            order = torch.sort(src.weight[b, h, :n - recent], descending=True, stable=True).indices[:budget - recent]
            kept = torch.cat([order.sort().values, torch.arange(n - recent, n, device="cuda")])
            assert torch.equal(dst.pos[b, h, :budget].long(), kept)
            assert torch.equal(dst.weight[b, h, :budget], src.weight[b, h, kept])
            page = src.page_table[b, kept // PAGE].long()
            want = src.k_codes[page, h, kept % PAGE].double() * src.k_scale[page, h].double()[:, None]
            to = torch.arange(budget, device="cuda")
            got = dst.k_codes[b * dst_pages + to // PAGE, h, to % PAGE].double() * dst.k_scale[b * dst_pages + to // PAGE, h].double()[:, None]
            step = dst.k_scale[b * dst_pages + to // PAGE, h].double()[:, None]
            assert ((got - want).abs() <= step / 2).all()  # one rounding of an int8 code


@pytest.mark.parametrize("max_pages", [10, 500])
def test_evict_captured_and_replayed(fm, max_pages):
    """The lengths in place (new_len is len), new weights before each replay: the same bits as calls made one by one."""
    g = torch.Generator(device="cuda").manual_seed(max_pages)
    src = shared_page_cache(fm, 2, 3, 64, max_pages, 9, "e4m3", g, weight=True)
    budget = max_pages * 16
    dst = [fm.fm_cache_alloc(2, 3, 64, budget, codes=torch.float8_e4m3fn) for _ in range(2)]
    lens = i32([max_pages * PAGE, max_pages * 20])
    ws = torch.empty(fm.fm_cache_evict_workspace_bytes(src, budget), dtype=torch.uint8, device="cuda")
    n, graph = lens.clone(), torch.cuda.CUDAGraph()
    fm.fm_cache_evict(src, dst[1], n, budget, recent=9, new_len=n, ws=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fm.fm_cache_evict(src, dst[1], n, budget, recent=9, new_len=n, ws=ws)
    for _ in range(3):
        src.weight.uniform_(generator=g)
        want = fm.fm_cache_evict(src, dst[0], lens, budget, recent=9)
        n.copy_(lens)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, want) and torch.equal(want, lens.clamp(max=budget))
        for a, b in zip((dst[0].weight, dst[0].pos, dst[0].k_codes.view(torch.uint8), dst[0].v_scale),
                        (dst[1].weight, dst[1].pos, dst[1].k_codes.view(torch.uint8), dst[1].v_scale)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_prompt_evict_decode(fm, code):
    """Prompt attention, key weights, cache, eviction, then tokens one by one, under a sliding-window mask."""
    B, H, H_kv, D, n, steps, budget, recent = 2, 8, 2, 128, 512, 70, 192, 32
    N = n + steps
    r = np.random.default_rng(8)
    qd, q = bf16(r.standard_normal((B, N, H, D)))
    kd, k = bf16(r.standard_normal((B, N, H_kv, D)))
    vd, v = bf16(r.standard_normal((B, N, H_kv, D)))
    j = np.arange(N)
    full = [np.broadcast_to(x, (B, 1, N)).astype(np.int32) for x in (np.minimum(j + 300, N), np.full(N, N), np.zeros(N), j)]
    part = [np.minimum(x[:, :, :n], n) for x in full]
    scale = 1 / math.sqrt(D)
    vt = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in part]
    meta = fm.fm_build_mask_meta(*vt, n_q=n)
    cut = lambda x, a, b: x[:, a:b].contiguous()  # noqa: E731
    o, lse = fm.fm_attn_fwd(cut(q, 0, n), cut(k, 0, n), cut(v, 0, n), meta, vt, scale)
    c = Pair(fm, B, H_kv, D, -(-n // PAGE), code)
    c.append(fm, kd[:, :n], vd[:, :n], np.zeros(B, int))
    fm.fm_attn_key_weight(cut(q, 0, n), cut(k, 0, n), lse, meta, vt, scale, weight=c.t.weight)
    check_key_weight(qd[:, :n], kd[:, :n], part, lse, c.t.weight.double().cpu().numpy(), scale)
    c.ref.weight[:] = c.t.weight.double().cpu().numpy()
    d = Pair(fm, B, H_kv, D, -(-(budget + steps) // PAGE), code, seed=5)
    lens = c.ref.evict(d.ref, np.full(B, n), budget, recent)
    length = fm.fm_cache_evict(c.t, d.t, i32(np.full(B, n)), budget, recent=recent)
    d.check(lens)
    vt = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in full]
    row = i32(np.full(B, n))
    for s in range(steps):
        at = n + s
        fm.fm_cache_append(d.t, cut(k, at, at + 1), cut(v, at, at + 1), length, row=row)
        d.ref.append(kd[:, at:at + 1], vd[:, at:at + 1], lens, row=np.full(B, at))
        length, lens = length + 1, lens + 1
        before = d.t.weight.double().cpu().numpy()
        o, lse = fm.fm_cache_attn(d.t, cut(q, at, at + 1), length, scale, row=row, vecs=vt, accumulate=True)
        if s % 23 == 0 or s == steps - 1:
            check_attention(d, lens, qd[:, at:at + 1], o, lse, scale, np.full(B, at), full, False, before)
        row += 1
    d.ref.weight[:] = d.t.weight.double().cpu().numpy()
    d.check(lens)
    assert fm.fm_get_device_status() == 0
