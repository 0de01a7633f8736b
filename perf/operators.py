"""Measured calls of the paged KV-cache operators around a sliding-window layer.

Five operators, one ``kind`` each:

* ``append``  -- per-head RMS norm of queries and keys, position rotation and the
  write of keys and values into the page pool, in one pass;
* ``decode``  -- one query token per sequence over a sliding window and the first
  tokens of the sequence (sinks), through the block table;
* ``prefill`` -- the same for a packed batch of new tokens (causal);
* ``copy``    -- whole pages copied in the pools of all layers (forking a sequence);
* ``compact`` -- the kept rows of each sequence moved to its front, in place, in the
  pools of all layers (eviction, accepted tokens of a draft).

``own = False`` computes each in elementary torch operations (fp32, rounded once),
``own = True`` calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
# one scale per pool and tensor for e4m3 pools: N(0,1) values use the range of the codes well
SCALE8 = 0.02


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _append(name, T, hq, hkv, d, **k):
    c = dict(kind="append", T=T, hq=hq, hkv=hkv, d=d, ps=16, rot=d, interleaved=False, norm=True, dtype="bf16",
             packed=True, pad=0, max_pos=32768)
    c.update(k, name=name)
    return c


def _decode(name, B, lo, hi, window, sinks, **k):
    c = dict(kind="decode", B=B, lo=lo, hi=hi, window=window, sinks=sinks, hq=32, hkv=8, d=128, ps=16, dtype="bf16")
    c.update(k, name=name)
    return c


def _prefill(name, B, n_lo, n_hi, c_lo, c_hi, window, sinks, **k):
    c = dict(kind="prefill", B=B, n_lo=n_lo, n_hi=n_hi, c_lo=c_lo, c_hi=c_hi, window=window, sinks=sinks, hq=32,
             hkv=8, d=128, ps=16, dtype="bf16")
    c.update(k, name=name)
    return c


def listed():
    return [
        # one decode step of the 32-sequence batch: 32 new tokens, rows are slices of one qkv product
        _append("append_decode_b32", 32, 32, 8, 128),
        # the new tokens of the chunked-prefill batch (10,496), some rows padding
        _append("append_prefill_10496", 10496, 32, 8, 128, pad=37),
        # an e4m3 cache, half of each head rotated in interleaved pairs, an odd token count
        _append("append_e4m3_2047", 2047, 16, 8, 128, rot=64, interleaved=True, dtype="e4m3"),
        # decode batch of 32 sequences of 512-4096 keys, a window of 1024 and 4 sinks
        _decode("decode_b32_w1024", 32, 512, 4096, 1024, 4),
        # long contexts: 256 sequences of 1k-32k keys, a window of 4096 and 4 sinks; pages behind the window are freed
        _decode("decode_long_b256_w4096", 256, 1024, 32768, 4096, 4),
        # e4m3 cache, one KV head for all 32 query heads, odd window and sinks
        _decode("decode_mqa_e4m3_b64_w999", 64, 1, 16384, 999, 17, hkv=1, dtype="e4m3"),
        # chunked prefill after up to 8192 cached tokens, a window of 1024 and 4 sinks
        _prefill("prefill_b8_w1024", 8, 512, 2048, 0, 8192, 1024, 4),
        # short ragged chunks on an e4m3 cache, head_dim 64, odd window
        _prefill("prefill_e4m3_d64_w333", 5, 1, 300, 0, 3000, 333, 5, hq=16, hkv=4, d=64, dtype="e4m3"),
        # a fork: the last page of each of 32 sequences, in 32 layers
        dict(kind="copy", name="copy_fork_32x32", layers=32, n=32, ps=16, hkv=8, d=128, dtype="bf16", slack=8),
        # moving many pages of a few layers
        dict(kind="copy", name="copy_1900x4", layers=4, n=1900, ps=16, hkv=8, d=128, dtype="bf16", slack=50),
        # accepted draft tokens: the last few rows of 32 sequences, in 16 layers
        dict(kind="compact", name="compact_draft_b32x16", layers=16, B=32, lo=17, hi=300, tail=8, frac=0.5, ps=16,
             hkv=8, d=128, dtype="bf16"),
        # eviction of half of every sequence's keys, in 4 layers
        dict(kind="compact", name="compact_evict_b16x4", layers=4, B=16, lo=1024, hi=4096, tail=0, frac=0.5, ps=16,
             hkv=8, d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["append", "decode", "prefill", "copy", "compact"])
    hq, hkv, d = rng.choice([(32, 8, 128), (32, 8, 128), (16, 2, 64), (8, 8, 64), (32, 1, 128), (40, 8, 128), (16, 16, 128)])
    ps = rng.choice([8, 16, 16, 32, 64])
    if kind == "append":
        dtype = rng.choice(["bf16", "bf16", "f32", "e4m3"])
        # e4m3 pools come back whole as values, f32 rows are twice the bytes: fewer tokens there
        T = _log(rng, 1, {"bf16": 10000, "f32": 4000, "e4m3": 1500}[dtype])
        return dict(kind="append", T=T, hq=hq, hkv=hkv, d=d, ps=ps, rot=rng.choice([d, d, d // 2]),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.8, dtype=dtype, packed=rng.random() < 0.7,
                    pad=rng.randint(0, T // 8), max_pos=_log(rng, 4096, 131072))
    dtype = rng.choice(["bf16", "bf16", "e4m3"])
    window, sinks = _log(rng, 32, 4096), rng.choice([0, 1, 4, 4, 16, 33, 128])
    if kind == "decode":
        B = _log(rng, 1, 256)
        window = min(window, max(32, (1 << 30) // (B * hkv * d)))
        lo = _log(rng, 1, 4096)
        return dict(kind="decode", B=B, lo=lo, hi=lo + _log(rng, 1, 28000), window=window, sinks=sinks, hq=hq, hkv=hkv,
                    d=d, ps=ps, dtype=dtype)
    if kind == "prefill":
        n_hi = _log(rng, 2, 2000)
        return dict(kind="prefill", B=rng.randint(1, 8), n_lo=rng.randint(1, n_hi), n_hi=n_hi, c_lo=0,
                    c_hi=_log(rng, 1, 8192), window=min(window, 1024), sinks=min(sinks, 33), hq=hq, hkv=hkv, d=d, ps=ps,
                    dtype=dtype)
    if kind == "copy":
        page = ps * hkv * d * 2
        layers = _log(rng, 1, 32)
        n = _log(rng, 1, max(1, min(4000, 240_000_000 // (2 * layers * page))))
        return dict(kind="copy", layers=layers, n=n, ps=ps, hkv=hkv, d=d, dtype="bf16", slack=rng.randint(0, 40))
    layers, B = _log(rng, 1, 16), _log(rng, 1, 32)
    hi = max(4, min(4096, 240_000_000 // (2 * layers * B * hkv * d * 2)))
    hi = _log(rng, 4, hi)
    return dict(kind="compact", layers=layers, B=B, lo=rng.randint(1, hi), hi=hi, tail=rng.choice([0, 0, 8, 33]),
                frac=round(rng.uniform(0.1, 0.95), 2), ps=ps, hkv=hkv, d=d, dtype="bf16")


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    h = torch.Generator(device="cpu")
    h.manual_seed(seed * 104729 + 5)
    return g, h


def _randn(shape, g, dtype):
    out = torch.empty(shape, device=DEV, dtype=dtype)
    flat, step = out.view(-1), 1 << 28
    for s in range(0, flat.numel(), step):
        e = min(flat.numel(), s + step)
        flat[s:e] = torch.randn(e - s, device=DEV, generator=g).to(dtype)
    return out


def _codes(shape, g):
    """e4m3 codes of N(0,1) values at SCALE8."""
    out = torch.empty(shape, device=DEV, dtype=torch.uint8)
    flat, step = out.view(-1), 1 << 28
    for s in range(0, flat.numel(), step):
        e = min(flat.numel(), s + step)
        x = torch.randn(e - s, device=DEV, generator=g) / SCALE8
        flat[s:e] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out.view(torch.float8_e4m3fn)


def _pool(shape, g, dtype):
    return _codes(shape, g) if dtype == "e4m3" else _randn(shape, g, TYPES[dtype])


def _live_tables(L, first, sinks, ps, h):
    """Block tables in which only pages with a key in [0, sinks) or [first, L) exist; other entries are -1 (freed)."""
    B, mb = L.numel(), max(1, (int(L.max()) + ps - 1) // ps)
    m = torch.arange(mb)[None, :] * ps
    live = (m < L[:, None]) & ((m < sinks) | (m + ps > first[:, None]))
    n = int(live.sum())
    P = n + n // 10 + 1
    bt = torch.full((B, mb), -1, dtype=torch.int32)
    bt[live] = torch.randperm(P, generator=h)[:n].to(torch.int32)
    return bt, P


def _lens(case, what):
    """Lengths of a batch, uniform in [lo, hi]: part of the case, the same for every seed."""
    lo, hi = case[what + "lo"], case[what + "hi"]
    h = torch.Generator(device="cpu")
    h.manual_seed(1000 + 31 * lo + hi)
    return torch.randint(lo, hi + 1, (case["B"],), generator=h)


def _first_rows(case, L):
    """compact: rows in front that stay where they are (all but the tail, or the first 4)."""
    return (L - case["tail"]).clamp(min=0) if case["tail"] else L.clamp(max=4)


def _kept(case, L, base):
    return ((L - base) * case["frac"]).round().long()


def prepare(case, seed):
    g, h = _gen(case, seed)
    s = {"case": case}
    kind = case["kind"]
    if kind == "append":
        T, hq, hkv, d, ps = (case[k] for k in ("T", "hq", "hkv", "d", "ps"))
        row = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        P = (T + T // 8 + ps) // ps + 1
        if case["packed"]:  # q, k, v are slices of the rows of one product
            qkv = _randn((T, hq + 2 * hkv, d), g, row)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = (_randn((T, n, d), g, row) for n in (hq, hkv, hkv))
        slots = torch.randperm(P * ps, generator=h)[:T]
        if case["pad"]:
            slots[torch.randperm(T, generator=h)[:case["pad"]]] = -1
        s["slots"] = slots.to(DEV)
        s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=h).to(torch.int32).to(DEV)
        s["qw"], s["kw"] = (((1 + 0.2 * torch.randn(d, device=DEV, generator=g)).to(row) for _ in range(2))
                            if case["norm"] else (None, None))
        inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        ang = torch.arange(case["max_pos"], device=DEV, dtype=torch.float64)[:, None] * inv[None, :]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["kp"], s["vp"] = _pool((P, ps, hkv, d), g, case["dtype"]), _pool((P, ps, hkv, d), g, case["dtype"])
        s["out"] = torch.zeros(T, hq, d, device=DEV, dtype=row)
        return s
    if kind in ("decode", "prefill"):
        B, hq, hkv, d, ps, W, S = (case[k] for k in ("B", "hq", "hkv", "d", "ps", "window", "sinks"))
        if kind == "decode":
            L = _lens(case, "")
            n = torch.ones_like(L)
        else:
            n = _lens(case, "n_")
            L = _lens(case, "c_") + n
        first = (L - n + 1 - W).clamp(min=0)  # first key that some query of the sequence sees through the window
        bt, P = _live_tables(L, first, S, ps, h)
        qsl = torch.zeros(B + 1, dtype=torch.int64)
        qsl[1:] = n.cumsum(0)
        s.update(kp=_pool((P, ps, hkv, d), g, case["dtype"]), vp=_pool((P, ps, hkv, d), g, case["dtype"]),
                 q=_randn((int(n.sum()), hq, d), g, torch.bfloat16), bt=bt.to(DEV), L=L.to(torch.int32).to(DEV),
                 qsl=qsl.to(torch.int32).to(DEV), scale=d ** -0.5, n_max=int(n.max()), l_max=int(L.max()),
                 scales=SCALE8 if case["dtype"] == "e4m3" else 1.0)
        s["out"] = torch.empty_like(s["q"])
        if own and kind == "decode":
            from serving_slot_mapping_gb300 import capi
            s["ws"] = capi.decode_workspace(B, hq, s["kp"])
        return s
    LY, ps, hkv, d = (case[k] for k in ("layers", "ps", "hkv", "d"))
    if kind == "copy":
        n, P = case["n"], 2 * case["n"] + case["slack"]
        ids = torch.randperm(P, generator=h)[:2 * n].to(torch.int32).to(DEV)
        s["src"], s["dst"] = ids[:n].contiguous(), ids[n:].contiguous()
    else:
        B = case["B"]
        L = _lens(case, "")
        base = _first_rows(case, L)
        keep = []
        for b, m in enumerate(_kept(case, L, base).tolist()):  # rows kept of [base, L), in order
            keep.append(base[b] + torch.randperm(int(L[b] - base[b]), generator=h)[:m].sort().values)
        ptr = torch.zeros(B + 1, dtype=torch.int64)
        ptr[1:] = torch.tensor([k.numel() for k in keep]).cumsum(0)
        bt, P = _live_tables(L, torch.zeros_like(L), 0, ps, h)
        s.update(bt=bt.to(DEV), L=L.to(torch.int32).to(DEV), base=base.to(torch.int32).to(DEV),
                 ptr=ptr.to(torch.int32).to(DEV), keep=torch.cat(keep).to(torch.int32).to(DEV))
    s["pools"] = _randn((LY, 2, P, ps, hkv, d), g, TYPES[case["dtype"]])
    if own:
        from serving_slot_mapping_gb300 import capi
        s["set"] = capi.make_pools([(s["pools"][i, 0], s["pools"][i, 1]) for i in range(LY)])
    return s


# --------------------------------------------------------------------------
# the operators, plainly
# --------------------------------------------------------------------------

def _values(x, scale):
    """fp32 values of gathered pool rows (e4m3 codes times their scale)."""
    return x.float() * scale if x.dtype == torch.float8_e4m3fn else x.float()


def _rows(pool, slot):
    """Rows of a pool by slot, as stored."""
    flat = pool.view(-1, pool.shape[2], pool.shape[3])
    if pool.dtype == torch.float8_e4m3fn:
        return flat.view(torch.uint8)[slot].view(torch.float8_e4m3fn)
    return flat[slot]


def _norm_rope(x, w, eps, cs, rot, interleaved):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()
    c, sn = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x[..., :rot]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _store(pool, slot, ok, x):
    """Scatter rows into a pool; rows with ok false keep what the pool holds."""
    if pool.dtype == torch.float8_e4m3fn:
        x = (x / SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pool = pool.view(torch.uint8)
    flat = pool.view(-1, pool.shape[2], pool.shape[3])
    at = torch.nonzero(ok)[:, 0]
    flat[slot[at]] = x[at].to(flat.dtype)


def _plain_append(s):
    c = s["case"]
    cs = s["cos_sin"][s["pos"].long()]
    ok = s["slots"] >= 0
    q = _norm_rope(s["q"], s["qw"], 1e-6, cs, c["rot"], c["interleaved"])
    k = _norm_rope(s["k"], s["kw"], 1e-6, cs, c["rot"], c["interleaved"])
    s["out"].copy_(torch.where(ok[:, None, None], q.to(s["out"].dtype), s["out"]))
    _store(s["kp"], s["slots"], ok, k)
    _store(s["vp"], s["slots"], ok, s["v"].float())
    return s["out"], s["kp"], s["vp"]


def _plain_attend(s, qp, q, L):
    """q [B, n, Hq, D] at positions qp [B, n] (below 0: no query) over each sequence's visible keys."""
    c = s["case"]
    W, S, ps, hkv = c["window"], c["sinks"], c["ps"], c["hkv"]
    B, n, hq, d = q.shape
    p0 = qp.masked_fill(qp < 0, 1 << 30).amin(1).clamp(max=1 << 29)  # first query position
    fs = torch.minimum((p0 - W + 1).clamp(min=0), L)  # first key of the window of any query
    span = min(s["l_max"], min(W, s["l_max"]) + n)
    j = torch.cat([torch.arange(S, device=DEV)[None, :].expand(B, S), fs[:, None] + torch.arange(span, device=DEV)], 1)
    there = j < L[:, None]
    there[:, :S] &= torch.arange(S, device=DEV)[None, :] < fs[:, None]  # a sink inside the span counts once
    page = torch.gather(s["bt"].long(), 1, (j // ps).clamp(max=s["bt"].shape[1] - 1))
    there &= page >= 0
    slot = torch.where(there, page * ps + j % ps, 0)
    zero = ~there[:, :, None, None]
    K = _values(_rows(s["kp"], slot), s["scales"]).masked_fill(zero, 0.0)
    V = _values(_rows(s["vp"], slot), s["scales"]).masked_fill(zero, 0.0)
    jq, pq = j[:, None, :], qp[:, :, None]
    see = there[:, None, :] & (jq <= pq) & ((jq > pq - W) | (jq < S))  # [B, n, keys]
    x = torch.matmul(q.float().view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d),
                     K.permute(0, 2, 3, 1)).view(B, hkv, hq // hkv, n, -1)
    x = x.mul_(s["scale"]).masked_fill_(~see[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    x = x.div_(x.sum(-1, keepdim=True).clamp(min=1e-30))
    o = torch.matmul(x.view(B, hkv, -1, x.shape[-1]), V.permute(0, 2, 1, 3)).view(B, hkv, hq // hkv, n, d)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, hq, d)


def _plain_decode(s):
    L = s["L"].long()
    o = _plain_attend(s, (L - 1)[:, None], s["q"][:, None], L)
    s["out"].copy_(o[:, 0])
    return s["out"]


def _plain_prefill(s):
    L, qsl = s["L"].long(), s["qsl"].long()
    n = qsl[1:] - qsl[:-1]
    i = torch.arange(s["n_max"], device=DEV)[None, :]
    there = i < n[:, None]
    row = (qsl[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    qp = torch.where(there, (L - n)[:, None] + i, -1)
    o = _plain_attend(s, qp, s["q"][row], L)
    s["out"][row[there]] = o[there].to(s["out"].dtype)
    return s["out"]


def _plain_copy(s):
    s["pools"][:, :, s["dst"].long()] = s["pools"][:, :, s["src"].long()]
    return s["pools"]


def _plain_compact(s):
    ps, ptr = s["case"]["ps"], s["ptr"].long()
    i = torch.arange(s["keep"].numel(), device=DEV)
    b = torch.searchsorted(ptr[1:].contiguous(), i, right=True)
    old, new = s["keep"].long(), s["base"].long()[b] + i - ptr[b]
    bt = s["bt"].long()
    flat = s["pools"].flatten(2, 3)
    flat[:, :, bt[b, new // ps] * ps + new % ps] = flat[:, :, bt[b, old // ps] * ps + old % ps]
    return s["pools"], (s["base"].long() + ptr[1:] - ptr[:-1]).to(torch.int32)


# --------------------------------------------------------------------------
# the operators, by the library
# --------------------------------------------------------------------------

def _own(s):
    from serving_slot_mapping_gb300 import capi
    c = s["case"]
    if c["kind"] == "append":
        sc = SCALE8 if c["dtype"] == "e4m3" else 1.0
        q = capi.paged_qk_norm_rope_append(s["kp"], s["vp"], s["q"], s["k"], s["v"], s["slots"], s["pos"], s["cos_sin"],
                                           q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                                           interleaved=c["interleaved"], out=s["out"], k_scale=sc, v_scale=sc)
        return q, s["kp"], s["vp"]
    if c["kind"] == "decode":
        return capi.paged_attention_decode_window(s["kp"], s["vp"], s["q"], s["bt"], s["L"], s["scale"], c["window"],
                                                  c["sinks"], max_seq_len=s["l_max"], out=s["out"], workspace=s["ws"],
                                                  k_scale=s["scales"], v_scale=s["scales"])
    if c["kind"] == "prefill":
        return capi.paged_attention_prefill_window(s["kp"], s["vp"], s["q"], s["qsl"], s["bt"], s["L"], s["scale"],
                                                   s["n_max"], c["window"], c["sinks"], max_seq_len=s["l_max"],
                                                   out=s["out"], k_scale=s["scales"], v_scale=s["scales"])
    if c["kind"] == "copy":
        capi.paged_kv_copy_pages(s["set"], s["src"], s["dst"])
        return s["pools"]
    return s["pools"], capi.paged_kv_compact(s["set"], s["bt"], s["L"], s["ptr"], s["keep"], base=s["base"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill, "copy": _plain_copy,
            "compact": _plain_compact}[state["case"]["kind"]](state)


# --------------------------------------------------------------------------
# work, and the results in 64 bits
# --------------------------------------------------------------------------

def work(case):
    e = {"bf16": 2, "f32": 4, "e4m3": 1}[case["dtype"]]
    kind = case["kind"]
    if kind == "append":
        T, hq, hkv, d = (case[k] for k in ("T", "hq", "hkv", "d"))
        r = 4 if case["dtype"] == "f32" else 2
        n = T - case["pad"]
        rows = n * d * ((2 * hq + 2 * hkv) * r + 2 * hkv * e)
        table = min(n, case["max_pos"]) * case["rot"] * 4
        return {"bytes": rows + n * 12 + table, "flops": n * d * (hq + hkv) * 8}
    if kind in ("decode", "prefill"):
        hq, hkv, d, W, S = (case[k] for k in ("hq", "hkv", "d", "window", "sinks"))
        L = _lens(case, "") if kind == "decode" else _lens(case, "c_") + _lens(case, "n_")
        n = torch.ones_like(L) if kind == "decode" else _lens(case, "n_")
        first = (L - n + 1 - W).clamp(min=0)
        keys = int((L - first + first.clamp(max=S)).sum())
        pairs = 0
        for l, m in zip(L.tolist(), n.tolist()):
            p = torch.arange(l - m, l)
            w = (p + 1).clamp(max=W)
            pairs += int((w + (p + 1 - w).clamp(max=S)).sum())
        return {"bytes": keys * hkv * d * 2 * e + keys / case["ps"] * 4 + 2 * int(n.sum()) * hq * d * 2,
                "flops": pairs * hq * d * 4}
    row = case["hkv"] * case["d"] * e
    if kind == "copy":
        return {"bytes": case["layers"] * 2 * 2 * case["n"] * case["ps"] * row + 8 * case["n"], "flops": 0}
    L = _lens(case, "")
    kept = int(_kept(case, L, _first_rows(case, L)).sum())
    return {"bytes": case["layers"] * 2 * 2 * kept * row + 4 * kept + 16 * case["B"], "flops": 0}


def _f64(x, scale=1.0):
    return x.float().double() * scale if x.dtype == torch.float8_e4m3fn else x.double()


def _exact_append(s, c):
    T, hq, hkv, d, rot = (c[k] for k in ("T", "hq", "hkv", "d", "rot"))
    half = rot // 2
    # rotation as a complex product, angles by their table (an input)
    z = torch.complex(s["cos_sin"][:, :half].double(), s["cos_sin"][:, half:].double())[s["pos"].long()]

    def turned(x, w):
        x = x.double().clone()
        if w is not None:
            x /= (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt()
            x *= w.double()
        idx = torch.arange(half, device=x.device)
        lo, hi = (2 * idx, 2 * idx + 1) if c["interleaved"] else (idx, idx + half)
        r = torch.complex(x[..., lo], x[..., hi]) * z[:, None, :]
        x[..., lo], x[..., hi] = r.real, r.imag
        return x

    ok = (s["slots"] >= 0).nonzero()[:, 0]
    out = s["out"].double()
    out[ok] = turned(s["q"], s["qw"])[ok]
    pools = []
    for pool, x in ((s["kp"], turned(s["k"], s["kw"])), (s["vp"], s["v"].double())):
        flat = _f64(pool).view(-1, hkv, d)
        # an e4m3 pool is compared by its codes' values: one step of the scale is one step of the code
        flat[s["slots"][ok]] = x[ok] / SCALE8 if c["dtype"] == "e4m3" else x[ok]
        if c["dtype"] == "e4m3":
            flat.clamp_(-448, 448)
        pools.append(flat.view(pool.shape))
    return out, pools[0], pools[1]


def _exact_attend(s, c):
    W, S, ps, hkv, hq = (c[k] for k in ("window", "sinks", "ps", "hkv", "hq"))
    L, bt, qsl = s["L"].tolist(), s["bt"].cpu(), s["qsl"].tolist()
    out = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    for b in range(c["B"]):  # one sequence at a time
        n = qsl[b + 1] - qsl[b]
        start = max(0, L[b] - n + 1 - W)
        j = torch.tensor([x for x in range(min(S, start))] + list(range(start, L[b])), dtype=torch.int64)
        slot = (bt[b].long()[j // ps] * ps + j % ps).to(DEV)
        K, V = (_f64(_rows(p, slot), s["scales"]).transpose(0, 1) for p in (s["kp"], s["vp"]))
        j = j.to(DEV)
        for a in range(0, n, 512):  # rows of queries
            e = min(n, a + 512)
            p = torch.arange(L[b] - n + a, L[b] - n + e, device=DEV)[:, None]
            hide = (j[None] > p) | ((j[None] <= p - W) & (j[None] >= S))
            q = s["q"][qsl[b] + a:qsl[b] + e].double().view(e - a, hkv, hq // hkv, -1)
            x = torch.einsum("nhgd,hkd->hgnk", q, K) * s["scale"]
            o = torch.einsum("hgnk,hkd->nhgd", torch.softmax(x.masked_fill(hide, -math.inf), -1), V)
            out[qsl[b] + a:qsl[b] + e] = o.reshape(e - a, hq, -1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "append":
        return _exact_append(s, case)
    if kind in ("decode", "prefill"):
        return _exact_attend(s, case)
    pools = s["pools"].clone()
    if kind == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pools[:, :, b] = s["pools"][:, :, a]
        return pools.double()
    ps, ptr, keep, base, bt = case["ps"], s["ptr"].tolist(), s["keep"].tolist(), s["base"].tolist(), s["bt"].tolist()
    frm, to = [], []
    for b in range(case["B"]):
        for i, old in enumerate(keep[ptr[b]:ptr[b + 1]]):
            new = base[b] + i
            frm.append(bt[b][old // ps] * ps + old % ps)
            to.append(bt[b][new // ps] * ps + new % ps)
    flat = pools.flatten(2, 3)
    before = s["pools"].flatten(2, 3)
    flat.index_copy_(2, torch.tensor(to, device=DEV, dtype=torch.long),
                     before.index_select(2, torch.tensor(frm, device=DEV, dtype=torch.long)))
    return pools.double(), None
