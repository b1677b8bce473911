"""Cases of the serving operators: the paged 8-bit K/V cache (its write, the attention that reads it, its
eviction) and the attention weight that a prompt's keys receive.

`own` false: every operator in elementary torch operations, fp32.  `own` true: the package's entry points.
`exact` computes the same from the definitions in 64 bits.

Cache layout: pages of 64 slots; K and V codes [page, H_kv, 64, D], one fp32 scale per (page, head) for each;
value = code * scale.  Scales are powers of two, so the codes (int8: whole numbers;
e4m3: 8-bit floats) are the same in 32 and in 64 bits, and come back as the numbers they are, next to their scales.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda" if torch.cuda.is_available() else "cpu"
NEG = -math.inf
QMAX = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences: one token each into the open block (latency; requantises the block
        # when the token exceeds its scale)
        dict(name="append token B64", op="append", B=64, H_kv=8, D=128, n_new=1, start=1000, ragged=True,
             code="int8"),
        # eight prompts of different lengths into empty caches, 8-bit floats
        dict(name="append prompts 8x4096", op="append", B=8, H_kv=8, D=128, n_new=4096, start=0, ragged=True,
             code="e4m3"),
        # one long prompt chunk behind an odd number of cached tokens
        dict(name="append chunk 32768", op="append", B=1, H_kv=16, D=128, n_new=32768, start=37, ragged=False,
             code="int8"),
        # the smallest call: one short conversation, one K/V head, one token
        dict(name="attend B1 517", op="attend", B=1, H=8, H_kv=1, D=64, n_q=1, len=517, ragged=False, code="int8",
             mask="none", window=0, accumulate=False, kept=False, mask_heads=False),
        # one long context, no batch to spread over the GPU
        dict(name="attend B1 131072", op="attend", B=1, H=32, H_kv=8, D=128, n_q=1, len=131072, ragged=False,
             code="int8", mask="none", window=0, accumulate=False, kept=False, mask_heads=False),
        # a serving batch of ragged lengths whose attention weights are kept for eviction; caches that were
        # evicted before (slots hold tokens with gaps between them)
        dict(name="attend B64 8192 weights", op="attend", B=64, H=32, H_kv=8, D=128, n_q=1, len=8192, ragged=True,
             code="e4m3", mask="none", window=0, accumulate=True, kept=True, mask_heads=False),
        # four drafted tokens checked at once under a sliding window with sink keys, head dimension 256
        dict(name="attend B16 n4 window", op="attend", B=16, H=8, H_kv=4, D=256, n_q=4, len=16384, ragged=True,
             code="int8", mask="window", window=1024, accumulate=True, kept=False, mask_heads=False),
        # a short causal prompt: few key tiles for 148 SMs
        dict(name="key weight 1024", op="key_weight", B=1, H=8, H_kv=2, D=128, n=1024, mask="causal"),
        # the benchmark's shortest sequence, packed documents
        dict(name="key weight 8192", op="key_weight", B=1, H=16, H_kv=16, D=128, n=8192, mask="document"),
        # a batch of odd length, shared K/V heads, bidirectional documents, head dimension 64
        dict(name="key weight 2x3996", op="key_weight", B=2, H=16, H_kv=4, D=64, n=3996, mask="blocks"),
        # a long prompt cut down to a sixteenth
        dict(name="evict B1 131072", op="evict", B=1, H_kv=8, D=128, len=131072, ragged=False, budget=8192, recent=1024,
             code="int8"),
        # a batch at its budget, some sequences over it and some not
        dict(name="evict B32 4200", op="evict", B=32, H_kv=8, D=128, len=4200, ragged=True, budget=2048, recent=100,
             code="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "key_weight", "key_weight", "evict"])
    D = rng.choice([64, 128, 128, 256])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    code = rng.choice(["int8", "e4m3"])
    if op == "append":
        one = rng.random() < 0.5
        B = _log(rng, 1, 96) if one else _log(rng, 1, 8)
        n_new = rng.randint(1, 5) if one else _log(rng, 6, 24000 // B)
        return dict(op=op, B=B, H_kv=H_kv, D=D, n_new=n_new, start=_log(rng, 1, 3000) - 1, ragged=rng.random() < 0.5,
                    code=code)
    if op == "attend":
        B = _log(rng, 1, 100)
        n = _log(rng, 8, min(120000, 330000000 // (B * H_kv * D)))
        return dict(op=op, B=B, H=H_kv * rng.choice([1, 2, 4, 7, 8, 16]), H_kv=H_kv, D=D, n_q=rng.choice([1, 1, 1, 2, 3, 5]),
                    len=n, ragged=rng.random() < 0.6, code=code,
                    mask=rng.choice(["none", "none", "causal", "window", "document"]), window=_log(rng, 16, 5000),
                    accumulate=rng.random() < 0.5, kept=rng.random() < 0.4, mask_heads=rng.random() < 0.3)
    if op == "key_weight":
        B = rng.choice([1, 1, 2, 3])
        G = rng.choice([1, 2, 4])
        H_kv = rng.choice([1, 2, 4])
        n = 4 * _log(rng, 8, int(2000 / math.sqrt(B * G * H_kv / 16.0)) if B * G * H_kv > 16 else 2000)
        return dict(op=op, B=B, H=H_kv * G, H_kv=H_kv, D=D, n=n, mask=rng.choice(["causal", "document", "blocks", "window"]))
    B = _log(rng, 1, 32)
    n = _log(rng, 100, 120000 // B)
    budget = max(1, int(n * rng.uniform(0.05, 0.9)))
    return dict(op=op, B=B, H_kv=H_kv, D=D, len=n, ragged=rng.random() < 0.6, budget=budget,
                recent=rng.randint(0, min(budget, 500)), code=code)


def _lengths(case, key, seed):
    """Host lengths [B]: the case's own, or spread over its last three quarters where it is ragged."""
    n, B = case[key], case["B"]
    r = np.random.RandomState(seed % (1 << 31))
    if not case["ragged"]:
        return np.full(B, n, np.int64)
    got = r.randint(max(1, n // 4), n + 1, size=B).astype(np.int64) if n > 0 else np.zeros(B, np.int64)
    got[r.randint(B)] = n
    return np.maximum(got, case.get("n_q", 0))


def work(case):
    op, D = case["op"], case["D"]
    H_kv, B = case["H_kv"], case["B"]
    if op == "append":
        n = float(_lengths(case, "n_new", 1).sum())
        return {"bytes": n * H_kv * D * 2 * (2 + 1) + n * H_kv * 8 + 8 * (n / PAGE + B) * H_kv, "flops": 0.0}
    if op == "attend":
        n = _lengths(case, "len", 1).astype(float)
        rows = case["n_q"] * case["H"]
        live = n.copy()
        if case["mask"] == "window":  # the keys that some row attends to: the window and the four sinks
            live = np.minimum(n, case["window"] / (2.0 if case["kept"] else 1.0) + case["n_q"] + 4)
        elif case["mask"] == "document":
            d = _doc(case["len"] * (3 if case["kept"] else 1))
            live = ((3 * n - 1) % d + 1) / 2.0 if case["kept"] else (n - 1) % d + 1
            live = np.minimum(n, live)
        keys = float(live.sum())
        vec = keys * 16.0 * (case["H"] if case["mask_heads"] else 1) if case["mask"] in ("window", "document") else 0.0
        pos = 4.0 * keys * H_kv if case["kept"] else 0.0
        return {"bytes": keys * H_kv * (2 * D + (8 if case["accumulate"] else 0)) + vec + pos + rows * B * (4 * D + 4),
                "flops": 4.0 * D * keys * rows}
    if op == "key_weight":
        n, H = case["n"], case["H"]
        pairs = _pairs(case)
        return {"bytes": B * n * (2.0 * D * (H + H_kv) + 4 * H + 4 * H_kv), "flops": 2.0 * D * pairs * H * B}
    n = _lengths(case, "len", 1).astype(float)
    kept = np.minimum(n, case["budget"])
    return {"bytes": float(n.sum()) * H_kv * 4 + float(kept.sum()) * H_kv * (4 * D + 8), "flops": 0.0}


# ------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _raw(codes):
    return codes.view(torch.uint8) if codes.dtype == torch.float8_e4m3fn else codes


def _scale_rule(amax, qmax):
    """0 for 0, else the smallest power of two s >= 2^-126 with qmax * s >= amax."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    qm, qe = math.frexp(qmax)
    k = torch.clamp(e - qe + (m > qm).to(e.dtype), min=-126)
    s = torch.ldexp(torch.ones_like(amax), k)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _code(x, code):
    """Nearest code (ties to even) of x, which is already in units of its scale; NaN becomes 0."""
    x = torch.where(torch.isnan(x), torch.zeros_like(x), x).clamp(-QMAX[code], QMAX[code])
    return torch.round(x).to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _quantise(x, code):
    """x [..., block values over the last two dimensions] -> codes, scale [...]."""
    fin = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    s = _scale_rule(fin.abs().amax((-1, -2)), QMAX[code])
    inv = torch.where(s > 0, 1.0 / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s))
    return _code(x * inv[..., None, None], code), s


def _pools(g, case, n_pages, filled=True):
    H_kv, D, code = case["H_kv"], case["D"], case["code"]
    if not filled:
        t = torch.int8 if code == "int8" else torch.float8_e4m3fn
        z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV).view(t)  # noqa: E731
        return dict(k_codes=z(n_pages, H_kv, PAGE, D), v_codes=z(n_pages, H_kv, PAGE, D),
                    k_scale=torch.zeros(n_pages, H_kv, device=DEV), v_scale=torch.zeros(n_pages, H_kv, device=DEV))
    k = _normal(g, n_pages, H_kv, PAGE, D)
    k *= 1.0 + 2.0 * (torch.arange(D, device=DEV) % 16 == 3)  # a few channels of K are larger, as in trained models
    kc, ks = _quantise(k, code)
    del k
    vc, vs = _quantise(_normal(g, n_pages, H_kv, PAGE, D), code)
    return dict(k_codes=kc, v_codes=vc, k_scale=ks, v_scale=vs)


def _table(g, B, max_pages):
    return torch.randperm(B * max_pages, generator=g, device=DEV).to(torch.int32).view(B, max_pages)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _doc(n):
    return max(16, n // 5)


def _vectors(mask, n, window, B, Hm):
    """Mask vectors LTS, LTE, UTS, UTE [B, Hm, n] over n rows and n keys, or None for each."""
    j = torch.arange(n, device=DEV, dtype=torch.int64)
    zero, end = torch.zeros_like(j), torch.full_like(j, n)
    h = torch.arange(Hm, device=DEV, dtype=torch.int64)[None, :, None]  # per-head masks differ by a few tokens
    if mask == "causal":
        v = (end, end, zero, j)
    elif mask == "window":  # the last `window` keys, and the first four always
        v = (torch.where(j < 4, end, torch.clamp(j + window - h, max=n)), end, zero, j)
    else:  # documents packed end to end: causal ("document") or seen in both directions ("blocks")
        d = _doc(n) + h
        v = (torch.clamp((j // d + 1) * d, max=n), end, zero, j if mask == "document" else (j // d) * d)
    return [x.expand(B, Hm, n).to(torch.int32).contiguous() for x in v]


def _pairs(case):
    n = case["n"]
    if case["mask"] == "causal":
        return n * (n + 1) / 2.0
    if case["mask"] == "window":
        w = min(n, max(16, n // 8))
        return w * (w + 1) / 2.0 + (n - w) * float(w)
    d = _doc(n)
    full, rest = divmod(n, d)
    if case["mask"] == "document":
        return full * d * (d + 1) / 2.0 + rest * (rest + 1) / 2.0
    return float(full * d * d + rest * rest)


def prepare(case, seed):
    g = _gen(seed)
    B, H_kv, D, op = case["B"], case["H_kv"], case["D"], case["op"]
    st = dict(case=case)
    if op == "key_weight":
        n, H = case["n"], case["H"]
        st["q"] = (1.5 * _normal(g, B, n, H, D)).to(torch.bfloat16)
        st["k"] = _normal(g, B, n, H_kv, D).to(torch.bfloat16)
        st["vecs"] = _vectors(case["mask"], n, max(16, n // 8), B, 1)
        st["scale"] = 1.0 / math.sqrt(D)
        s = _prompt_scores(st)
        st["lse"] = torch.logsumexp(s, -1).contiguous()  # [B, H, n], as the forward pass leaves it
        del s
        if own:
            import mask_aware_flash_b200 as fm
            st["meta"] = fm.fm_build_mask_meta(*st["vecs"], n_q=n)  # the forward pass's
        return st
    key = "n_new" if op == "append" else "len"
    lens = _lengths(case, key, seed)
    top = case[key] + (case["start"] if op == "append" else 0)
    max_pages = top // PAGE + 1
    st["table"] = _table(g, B, max_pages)
    cap = max_pages * PAGE
    if op == "append":
        st.update(_pools(g, case, B * max_pages))
        r = np.random.RandomState(seed % 997)
        start = np.full(B, case["start"], np.int64)
        if case["ragged"] and case["start"] > 0:
            start = r.randint(0, case["start"] + 1, size=B)
        first, last = start // PAGE, (start + lens - 1) // PAGE
        seqs = np.repeat(np.arange(B), last - first + 1)
        blocks = np.concatenate([np.arange(a, b + 1) for a, b in zip(first, last)])
        st["touched"] = (torch.as_tensor(seqs).to(DEV), torch.as_tensor(blocks).to(DEV))  # blocks that get tokens
        st["host_start"], st["host_count"] = start, lens
        st["start"], st["count"] = _i32(start), _i32(lens)
        st["row"] = _i32(start + 7)  # tokens were evicted before: positions run ahead of slots
        st["k"] = _normal(g, B, case["n_new"], H_kv, D).mul_(1.5).to(torch.bfloat16)
        st["v"] = _normal(g, B, case["n_new"], H_kv, D).mul_(1.5).to(torch.bfloat16)
        st["weight"] = torch.rand((B, H_kv, cap), generator=g, device=DEV)
        st["pos"] = torch.zeros((B, H_kv, cap), dtype=torch.int32, device=DEV)
    elif op == "attend":
        st.update(_pools(g, case, B * max_pages))
        n_q, H = case["n_q"], case["H"]
        st["len"] = _i32(lens)
        st["q"] = (1.5 * _normal(g, B, n_q, H, D)).to(torch.bfloat16)
        st["scale"] = 1.0 / math.sqrt(D)
        st["weight"] = torch.rand((B, H_kv, cap), generator=g, device=DEV) if case["accumulate"] else None
        last = torch.as_tensor(lens).to(DEV)  # position of the token after the newest
        if case["kept"]:  # half of the older tokens were evicted, others in each head; the newest 64 are together
            slot = torch.arange(cap, device=DEV)
            gap = torch.randint(0, 3, (B, H_kv, cap), generator=g, device=DEV)
            gap = torch.where(slot >= last[:, None, None] - PAGE, torch.zeros_like(gap), gap)
            raw = torch.cumsum(gap + 1, -1)
            at = raw.gather(-1, (last - 1)[:, None, None].expand(B, H_kv, 1))
            last = 3 * last
            st["pos"] = (raw - at + last[:, None, None] - 1).to(torch.int32).contiguous()
        else:
            st["pos"] = None
        st["row"] = (last - n_q).to(torch.int32).contiguous()  # the cache holds the queries' own tokens already
        st["vecs"], st["causal"] = None, case["mask"] == "causal"
        if case["mask"] in ("window", "document"):
            st["vecs"] = _vectors(case["mask"], case["len"] * (3 if case["kept"] else 1), case["window"], B,
                                  H if case["mask_heads"] else 1)
    else:
        st.update(_pools(g, case, B * max_pages))
        st["len"] = _i32(lens)
        # accumulated weights: few heavy keys, most of them light
        st["weight"] = torch.exp(1.5 * _normal(g, B, H_kv, cap))
        gap = torch.randint(0, 2, (B, H_kv, cap), generator=g, device=DEV)
        st["pos"] = (torch.cumsum(gap + 1, -1) - 1).to(torch.int32).contiguous()
        dst_pages = -(-case["budget"] // PAGE)
        st["dst"] = _pools(g, case, B * dst_pages, filled=False)
        st["dst"]["table"] = _table(g, B, dst_pages)
        st["dst"]["weight"] = torch.zeros((B, H_kv, dst_pages * PAGE), device=DEV)
        st["dst"]["pos"] = torch.zeros((B, H_kv, dst_pages * PAGE), dtype=torch.int32, device=DEV)
        st["new_len"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:
        _handles(st)
    return st


def _handles(st):
    """The cache objects, outputs and workspaces that a decode loop keeps between its calls."""
    import mask_aware_flash_b200 as fm
    of = lambda d: fm.KVCache(d["k_codes"], d["v_codes"], d["k_scale"], d["v_scale"], d["table"],  # noqa: E731
                              weight=d["weight"], pos=d["pos"])
    st["cache"] = of(st)
    if st["case"]["op"] == "evict":
        st["dst_cache"] = of(st["dst"])
        st["ws"] = torch.empty(fm.fm_cache_evict_workspace_bytes(st["cache"], st["case"]["budget"]), dtype=torch.uint8,
                               device=DEV)
    elif st["case"]["op"] == "attend":
        q = st["q"]
        st["o"] = torch.empty_like(q)
        st["lse"] = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=DEV)
        st["ws"] = torch.empty(fm.fm_cache_attn_workspace_bytes(st["cache"], q, accumulate=st["case"]["accumulate"]),
                               dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if not own:
        return {"append": _append, "attend": _attend, "key_weight": _key_weight, "evict": _evict}[op](st)
    import mask_aware_flash_b200 as fm
    if op == "append":
        fm.fm_cache_append(st["cache"], st["k"], st["v"], st["start"], count=st["count"], row=st["row"])
        return _cache_outputs(st)
    if op == "attend":
        fm.fm_cache_attn(st["cache"], st["q"], st["len"], st["scale"], row=st["row"], vecs=st["vecs"], causal=st["causal"],
                         accumulate=st["case"]["accumulate"], o=st["o"], lse=st["lse"], ws=st["ws"])
        return [st["o"], st["lse"], st["weight"]]
    if op == "key_weight":
        return fm.fm_attn_key_weight(st["q"], st["k"], st["lse"], st["meta"], st["vecs"], st["scale"])
    fm.fm_cache_evict(st["cache"], st["dst_cache"], st["len"], st["case"]["budget"], recent=st["case"]["recent"],
                      new_len=st["new_len"], ws=st["ws"])
    return _cache_outputs(st["dst"]) + [st["new_len"]]


def _cache_outputs(d):
    return [d["k_codes"], d["v_codes"], d["k_scale"], d["v_scale"], d["weight"], d["pos"]]


# ------------------------------------------------------------------------------------------------- plain forms
def _append(st):
    case = st["case"]
    code, n_new, H_kv = case["code"], case["n_new"], case["H_kv"]
    b, blk = st["touched"]
    page = st["table"][b, blk].long()
    slot = blk[:, None] * PAGE + torch.arange(PAGE, device=DEV)       # [touched, 64]
    start, count = st["start"].long()[b][:, None], st["count"].long()[b][:, None]
    t = slot - start
    fresh, old = (t >= 0) & (t < count), t < 0
    t = t.clamp(0, n_new - 1)
    for name, x in (("k", st["k"]), ("v", st["v"])):
        codes, scales = st[name + "_codes"], st[name + "_scale"]
        new = x[b[:, None], t].float().transpose(1, 2)                # [touched, H_kv, 64, D]
        was = _raw(codes)[page].view(codes.dtype).float()
        f4, o4 = fresh[:, None, :, None], old[:, None, :, None]
        amax = torch.where(f4 & torch.isfinite(new), new, torch.zeros_like(new)).abs().amax((-1, -2))
        s_old = torch.where(old.any(1)[:, None], scales[page], torch.zeros_like(amax))
        s = torch.maximum(s_old, _scale_rule(amax, QMAX[code]))
        inv = torch.where(s > 0, 1.0 / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s))[..., None, None]
        got = _code(torch.where(f4, new * inv, was * (s_old[..., None, None] * inv)), code)
        keep = f4 | o4
        _raw(codes)[page] = torch.where(keep, _raw(got), _raw(_code(was, code)))
        scales[page] = s
    h = torch.arange(H_kv, device=DEV)[None, :, None]
    bb, ss = b[:, None, None], slot[:, None, :]
    f3 = fresh[:, None, :]
    st["weight"][bb, h, ss] = torch.where(f3, torch.zeros((), device=DEV), st["weight"][bb, h, ss])
    row = st["row"].long()[b][:, None] + slot - start
    st["pos"][bb, h, ss] = torch.where(f3, row[:, None, :].to(torch.int32), st["pos"][bb, h, ss])
    return _cache_outputs(st)


def _values(d, name, dtype=torch.float32):
    """The cache's values in slot order, [B, H_kv, slots, D]."""
    codes, scale, table = d[name + "_codes"], d[name + "_scale"], d["table"].long()
    x = _raw(codes)[table].view(codes.dtype).to(dtype)                 # [B, pages, H_kv, 64, D]
    x = x * scale.to(dtype)[table][..., None, None]
    B, P, H_kv, _, D = x.shape
    return x.transpose(1, 2).reshape(B, H_kv, P * PAGE, D)


def _unmasked(st, S):
    """[B, H_kv, G, n_q, S] truth values: which slots each query attends to."""
    case = st["case"]
    B, H, H_kv, n_q = case["B"], case["H"], case["H_kv"], case["n_q"]
    slot = torch.arange(S, device=DEV)
    j = slot.expand(B, H_kv, S) if st["pos"] is None else st["pos"].long()
    i = st["row"].long()[:, None, None, None, None] + torch.arange(n_q, device=DEV)[:, None]
    ok = (slot < st["len"].long()[:, None])[:, None, None, None, :]
    if st["causal"]:
        ok = ok & (j[:, :, None, None, :] <= i)
    if st["vecs"] is not None:
        n = st["vecs"][0].shape[-1]
        inside = ((j >= 0) & (j < n))[:, :, None, None, :]
        Hm = st["vecs"][0].shape[1]
        b = torch.arange(B, device=DEV)[:, None, None, None]
        h = torch.zeros((1, 1, 1, 1), dtype=torch.long, device=DEV) if Hm == 1 else \
            torch.arange(H, device=DEV).view(1, H_kv, H // H_kv, 1)
        lts, lte, uts, ute = (v[b, h, j.clamp(0, n - 1)[:, :, None, :]][..., None, :] for v in st["vecs"])
        ok = ok & ~(inside & (((lts <= i) & (i < lte)) | ((uts <= i) & (i < ute))))
    return ok.expand(B, H_kv, H // H_kv, n_q, S)


def _attend(st):
    case = st["case"]
    B, H, H_kv, n_q, D = case["B"], case["H"], case["H_kv"], case["n_q"], case["D"]
    k = _values(st, "k")
    S = k.shape[2]
    q = st["q"].float().view(B, n_q, H_kv, H // H_kv, D).permute(0, 2, 3, 1, 4)   # [B, H_kv, G, n_q, D]
    s = torch.matmul(q.reshape(B, H_kv, -1, D), k.transpose(2, 3)).view(B, H_kv, H // H_kv, n_q, S) * st["scale"]
    del k
    s = torch.where(_unmasked(st, S), s, torch.full_like(s, NEG))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == NEG, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total))[..., 0].reshape(B, H, n_q)
    o = torch.matmul(p.view(B, H_kv, -1, S), _values(st, "v")).view(B, H_kv, H // H_kv, n_q, D)
    if case["accumulate"]:
        st["weight"] += p.sum((2, 3))
    return [o.permute(0, 3, 1, 2, 4).reshape(B, n_q, H, D).to(torch.bfloat16), lse, st["weight"]]


def _prompt_scores(st, dtype=torch.float32):
    """Scaled scores of a prompt, masked ones -inf: [B, H, n, n]."""
    q, k = st["q"].to(dtype), st["k"].to(dtype)
    G = q.shape[2] // k.shape[2]
    s = torch.matmul(q.permute(0, 2, 1, 3), k.repeat_interleave(G, 2).permute(0, 2, 3, 1)).mul_(st["scale"])
    i = torch.arange(q.shape[1], device=DEV)[:, None]
    lts, lte, uts, ute = (v.long()[:, :, None, :] for v in st["vecs"])
    return s.masked_fill_(((lts <= i) & (i < lte)) | ((uts <= i) & (i < ute)), NEG)


def _key_weight(st):
    s = _prompt_scores(st)
    B, H, n, _ = s.shape
    lse = st["lse"]
    p = s.sub_(torch.where(lse == NEG, torch.zeros_like(lse), lse)[..., None]).exp_()
    return p.sum(2).view(B, st["k"].shape[2], -1, n).sum(2)


def _evict(st):
    case, dst = st["case"], st["dst"]
    B, H_kv, D, budget = case["B"], case["H_kv"], case["D"], case["budget"]
    w, length = st["weight"], st["len"].long()[:, None, None]
    S = w.shape[2]
    slot = torch.arange(S, device=DEV).expand(B, H_kv, S)
    used = slot < length
    older = slot < length - case["recent"]
    order = torch.sort(torch.where(older, w, torch.full_like(w, NEG)), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.contiguous())
    keep = used & ((length <= budget) | ~older | (older & (rank < budget - case["recent"])))
    pages = dst["table"].shape[1]
    from_slot = torch.sort(torch.where(keep, slot, torch.full_like(slot, S)), dim=-1).values[..., :pages * PAGE]
    if from_slot.shape[-1] < pages * PAGE:
        from_slot = torch.nn.functional.pad(from_slot, (0, pages * PAGE - from_slot.shape[-1]), value=S)
    new_len = torch.clamp(st["len"], max=budget)
    live = torch.arange(pages * PAGE, device=DEV) < new_len[:, None, None]
    live = live & (from_slot < S)
    at = from_slot.clamp(max=S - 1)
    h = torch.arange(H_kv, device=DEV)[None, :, None]
    page = st["table"].long().gather(1, (at // PAGE).view(B, -1)).view(B, H_kv, -1)
    block_used = (torch.arange(pages, device=DEV) * PAGE < new_len[:, None])      # [B, pages]
    to = dst["table"].long()
    for name in ("k", "v"):
        x = _raw(st[name + "_codes"])[page, h, at % PAGE].view(st[name + "_codes"].dtype).float()
        x = x * st[name + "_scale"][page, h][..., None]
        x = torch.where(live[..., None], x, torch.zeros_like(x)).view(B, H_kv, pages, PAGE, D).transpose(1, 2)
        codes, s = _quantise(x, case["code"])                                     # [B, pages, H_kv, 64, D]
        out = _raw(dst[name + "_codes"])
        out[to] = torch.where(block_used[:, :, None, None, None], _raw(codes), out[to])
        dst[name + "_scale"][to] = torch.where(block_used[:, :, None], s, dst[name + "_scale"][to])
    dst["weight"].copy_(torch.where(live, w.gather(-1, at), dst["weight"]))
    dst["pos"].copy_(torch.where(live, st["pos"].gather(-1, at), dst["pos"]))
    st["new_len"].copy_(new_len)
    return _cache_outputs(dst) + [st["new_len"]]


# ------------------------------------------------------------------------------------------------- in 64 bits
def _scale_64(amax, qmax):
    """The scale rule in Python numbers."""
    if amax == 0:
        return 0.0
    e = -126
    guess = math.floor(math.log2(amax / qmax)) - 1
    e = max(e, guess)
    while math.ldexp(qmax, e) < amax:
        e += 1
    return math.ldexp(1.0, e)


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "key_weight": _exact_key_weight,
            "evict": _exact_evict}[case["op"]](case, st)


def _exact_append(case, st):
    """Scales of every page and the cleared weights (codes and positions are not floating-point results)."""
    out = []
    for name in ("k", "v"):
        scale = st[name + "_scale"].double().cpu().numpy()
        x = st[name].double().abs()
        table = st["table"].cpu().numpy()
        for b in range(case["B"]):
            start, count = int(st["host_start"][b]), int(st["host_count"][b])
            for blk in range(start // PAGE, (start + count - 1) // PAGE + 1):
                lo, hi = max(blk * PAGE, start) - start, min((blk + 1) * PAGE, start + count) - start
                amax = x[b, lo:hi].amax((0, 2)).cpu().numpy()
                for h in range(case["H_kv"]):
                    was = scale[table[b, blk], h] if start > blk * PAGE else 0.0
                    scale[table[b, blk], h] = max(was, _scale_64(float(amax[h]), QMAX[case["code"]]))
        out.append(torch.as_tensor(scale))
    weight = st["weight"].double().cpu()
    for b in range(case["B"]):
        weight[b, :, int(st["host_start"][b]):int(st["host_start"][b] + st["host_count"][b])] = 0.0
    return [None, None, out[0], out[1], weight, None]


def _exact_attend(case, st):
    B, H, H_kv, n_q, D = case["B"], case["H"], case["H_kv"], case["n_q"], case["D"]
    G = H // H_kv
    o = torch.zeros((B, n_q, H, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, n_q), NEG, dtype=torch.float64, device=DEV)
    weight = st["weight"].double() if case["accumulate"] else None
    for b in range(B):
        n = int(st["len"][b])
        pages = st["table"][b, :-(-n // PAGE)].long()
        for hk in range(H_kv):
            k = (_raw(st["k_codes"])[pages, hk].view(st["k_codes"].dtype).double()
                 * st["k_scale"].double()[pages, hk, None, None]).reshape(-1, D)[:n]
            v = (_raw(st["v_codes"])[pages, hk].view(st["v_codes"].dtype).double()
                 * st["v_scale"].double()[pages, hk, None, None]).reshape(-1, D)[:n]
            j = torch.arange(n, device=DEV) if st["pos"] is None else st["pos"][b, hk, :n].long()
            q = st["q"][b, :, hk * G:(hk + 1) * G].double()                      # [n_q, G, D]
            s = st["scale"] * torch.einsum("tgd,nd->tgn", q, k)
            i = (int(st["row"][b]) + torch.arange(n_q, device=DEV))[:, None, None]
            hidden = torch.zeros_like(s, dtype=torch.bool)
            if st["causal"]:
                hidden |= j > i
            if st["vecs"] is not None:
                N = st["vecs"][0].shape[-1]
                at = j.clamp(0, N - 1)
                many = st["vecs"][0].shape[1] > 1
                a, z, u, e = ((x[b, hk * G:(hk + 1) * G] if many else x[b, :1])[:, at].long()[None] for x in st["vecs"])
                hidden |= (((i >= a) & (i < z)) | ((i >= u) & (i < e))) & (j >= 0) & (j < N)
            s = s.masked_fill(hidden, NEG)
            row = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(row == NEG, torch.zeros_like(row), row)[..., None])
            o[b, :, hk * G:(hk + 1) * G] = torch.einsum("tgn,nd->tgd", p, v)
            lse[b, hk * G:(hk + 1) * G] = row.T
            if weight is not None:
                weight[b, hk, :n] += p.sum((0, 1))
    return [o, lse, weight]


def _exact_key_weight(case, st):
    B, H, H_kv, n = case["B"], case["H"], case["H_kv"], case["n"]
    out = torch.zeros((B, H_kv, n), dtype=torch.float64, device=DEV)
    i = torch.arange(n, device=DEV)[:, None]
    for b in range(B):
        a, z, u, e = (x[b, 0].long()[None, :] for x in st["vecs"])
        seen = ~(((i >= a) & (i < z)) | ((i >= u) & (i < e)))
        for h in range(H):
            hk = h // (H // H_kv)
            s = st["scale"] * (st["q"][b, :, h].double() @ st["k"][b, :, hk].double().T)
            lse = st["lse"][b, h].double()[:, None]
            out[b, hk] += torch.where(seen, torch.exp(s - lse), torch.zeros_like(s)).sum(0)
    return out


def _exact_evict(case, st):
    """Scales and weights of the new cache (codes, positions and lengths are not floating-point results)."""
    B, H_kv, budget, recent = case["B"], case["H_kv"], case["budget"], case["recent"]
    dst, table = st["dst"], st["table"].cpu().numpy()
    to = dst["table"].cpu().numpy()
    weight = dst["weight"].double().cpu().numpy()
    scales = [dst[n + "_scale"].double().cpu().numpy() for n in ("k", "v")]
    # the largest magnitude of each slot, [page, H_kv, 64]
    big = [(st[n + "_codes"].float().abs().amax(3).double() * st[n + "_scale"].double()[:, :, None]).cpu().numpy()
           for n in ("k", "v")]
    w = st["weight"].double().cpu().numpy()
    for b in range(B):
        n = int(st["len"][b])
        for h in range(H_kv):
            if n <= budget:
                kept = np.arange(n)
            else:
                heavy = np.argsort(-w[b, h, :n - recent], kind="stable")[:budget - recent]
                kept = np.concatenate([np.sort(heavy), np.arange(n - recent, n)])
            weight[b, h, :len(kept)] = w[b, h, kept]
            for x, scale in zip(big, scales):
                mags = x[table[b, kept // PAGE], h, kept % PAGE]
                for blk in range(-(-len(kept) // PAGE)):
                    scale[to[b, blk], h] = _scale_64(float(mags[blk * PAGE:(blk + 1) * PAGE].max()), QMAX[case["code"]])
    return [None, None, torch.as_tensor(scales[0]), torch.as_tensor(scales[1]), torch.as_tensor(weight), None, None]
