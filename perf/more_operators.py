"""Measured calls of the operators around a long-context cache under a memory budget.

Five operators, one ``kind`` each:

* ``append``  -- new bf16 rows quantised into int8 pools with a scale for each block of
  tokens and KV head, kept up to date by the append itself;
* ``decode``  -- one query token per sequence over such pools, through the block table;
* ``prefill`` -- the same for a packed batch of new tokens (causal);
* ``mass``    -- a decode that also gives each key's attention weight, summed over the
  query heads and added to what the key had before (bf16, e4m3 and int8 pools);
* ``rows`` / ``pages`` -- eviction by that accumulated weight: the first and the last tokens
  and the heaviest of the others within a budget, row by row or page by page.

``own = False`` computes each in elementary torch operations (fp32, rounded once),
``own = True`` calls the library.  The append's codes come back as the whole numbers
that they are, with the scales that make values of them beside them: its arithmetic is
fp32 with one division and one rounding, so they are the same to the last one.
"""
import math

import torch

own = False

DEV = "cuda"
# one scale per pool and tensor for e4m3 pools: N(0,1) values use the range of the codes well
SCALE8 = 0.02
QMAX = 127.0
SCALE_MIN, SCALE_MAX = 2.0 ** -40, 2.0 ** 40


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _append(name, B, n_lo, n_hi, c_lo, c_hi, **k):
    c = dict(kind="append", B=B, n_lo=n_lo, n_hi=n_hi, c_lo=c_lo, c_hi=c_hi, hkv=8, d=128, ps=16, blk=16, pad=0,
             packed=True)
    c.update(k, name=name)
    return c


def _decode(name, B, lo, hi, **k):
    c = dict(kind="decode", B=B, lo=lo, hi=hi, hq=32, hkv=8, d=128, ps=16, blk=16, dtype="int8")
    c.update(k, name=name)
    return c


def _prefill(name, B, n_lo, n_hi, c_lo, c_hi, **k):
    c = dict(kind="prefill", B=B, n_lo=n_lo, n_hi=n_hi, c_lo=c_lo, c_hi=c_hi, hq=32, hkv=8, d=128, ps=16, blk=16,
             dtype="int8")
    c.update(k, name=name)
    return c


def _mass(name, B, lo, hi, dtype, **k):
    c = dict(kind="mass", B=B, lo=lo, hi=hi, hq=32, hkv=8, d=128, ps=16, blk=16, dtype=dtype, decay=1.0, first=False)
    c.update(k, name=name)
    return c


def _evict(name, kind, B, lo, hi, budget, sinks, recent, **k):
    c = dict(kind=kind, B=B, lo=lo, hi=hi, budget=budget, sinks=sinks, recent=recent, ps=16, fresh=0.1)
    c.update(k, name=name)
    return c


def listed():
    return [
        # one decode step of the 32-sequence batch: one new token in a block that holds earlier ones
        _append("int8_append_decode_b32", 32, 1, 1, 511, 4095),
        # the new tokens of a chunked-prefill batch, some rows padding; rows are slices of one qkv product
        _append("int8_append_prefill_b8", 8, 512, 2048, 0, 8192, pad=37),
        # decode batch of 32 sequences of 512-4096 keys
        _decode("int8_decode_b32", 32, 512, 4096),
        # long contexts: 64 sequences of 1k-32k keys
        _decode("int8_decode_long_b64", 64, 1024, 32768),
        # one KV head for all 32 query heads, pages of 64, scales for 32 tokens
        _decode("int8_decode_mqa_b64", 64, 1, 16384, hkv=1, ps=64, blk=32),
        # chunked prefill after up to 8192 cached tokens
        _prefill("int8_prefill_b8", 8, 512, 2048, 0, 8192),
        # short ragged chunks, head_dim 64
        _prefill("int8_prefill_d64_ragged", 5, 1, 300, 0, 3000, hq=16, hkv=4, d=64, ps=32, blk=32),
        # the decode batch with the weights of its keys, added to those of the steps before; bf16 pools
        _mass("mass_bf16_b32", 32, 512, 4096, "bf16"),
        # the same over int8 pools, sequences of 1-16k keys, earlier weights fading
        _mass("mass_int8_b64", 64, 1, 16384, "int8", hq=16, hkv=2, d=64, ps=32, decay=0.99),
        # a decode batch brought down to 1024 rows a sequence
        _evict("evict_rows_b32", "rows", 32, 512, 4096, 1024, 4, 256),
        # one very long sequence
        _evict("evict_rows_one_131072", "rows", 1, 131072, 131072, 8192, 4, 1024),
        # long contexts brought down to 256 pages of 16 tokens each; nothing is moved but the block table
        _evict("evict_pages_b256", "pages", 256, 1024, 32768, 256, 4, 512),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["append", "decode", "prefill", "mass", "rows", "pages"])
    hq, hkv, d = rng.choice([(32, 8, 128), (32, 8, 128), (16, 2, 64), (8, 8, 64), (32, 1, 128), (40, 8, 128), (16, 16, 128),
                             (12, 3, 64)])
    ps = rng.choice([16, 16, 32, 64, 128])
    blk = rng.choice([b for b in (16, 32, 64) if b <= ps])
    if kind == "append":
        n_hi = rng.choice([1, 1, _log(rng, 2, 2000)])
        return dict(kind=kind, B=rng.randint(1, 64) if n_hi == 1 else rng.randint(1, 6), n_lo=rng.randint(1, n_hi), n_hi=n_hi,
                    c_lo=0, c_hi=_log(rng, 1, 8192), hkv=hkv, d=d, ps=ps, blk=blk, pad=rng.randint(0, 40),
                    packed=rng.random() < 0.7)
    if kind in ("decode", "mass"):
        dtype = "int8" if kind == "decode" else rng.choice(["bf16", "e4m3", "int8"])
        B = _log(rng, 1, 128)
        most = max(64, min(30000, (1 << 28) // (B * hkv * d)))
        lo = _log(rng, 1, most)
        c = dict(kind=kind, B=B, lo=lo, hi=lo + _log(rng, 1, most), hq=hq, hkv=hkv, d=d, ps=ps, blk=blk, dtype=dtype)
        if kind == "mass":
            c.update(decay=rng.choice([1.0, 0.99, 0.5]), first=rng.random() < 0.3)
        return c
    if kind == "prefill":
        n_hi = _log(rng, 2, 1500)
        return dict(kind=kind, B=rng.randint(1, 6), n_lo=rng.randint(1, n_hi), n_hi=n_hi, c_lo=0, c_hi=_log(rng, 1, 6000),
                    hq=hq, hkv=hkv, d=d, ps=ps, blk=blk, dtype="int8")
    B = _log(rng, 1, 128)
    hi = _log(rng, 64, min(100000, 3000000 // B))
    sinks, recent = rng.choice([0, 1, 4, 33]), rng.choice([0, 1, 32, 257])
    if kind == "rows":
        budget = sinks + recent + _log(rng, 1, hi)
    else:
        budget = -(-sinks // ps) + (recent + ps - 2) // ps + 2 + _log(rng, 1, max(1, hi // ps))
    return dict(kind=kind, B=B, lo=rng.randint(0, hi), hi=hi, budget=budget, sinks=sinks, recent=recent, ps=ps,
                fresh=rng.choice([0.0, 0.1, 0.6]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 23)
    h = torch.Generator(device="cpu")
    h.manual_seed(seed * 104729 + 11)
    return g, h


def _lens(case, what=""):
    """Lengths of a batch, uniform in [lo, hi]: part of the case, the same for every seed."""
    lo, hi = case[what + "lo"], case[what + "hi"]
    h = torch.Generator(device="cpu")
    h.manual_seed(1000 + 31 * lo + hi)
    return torch.randint(lo, hi + 1, (case["B"],), generator=h)


def _tables(L, ps, h):
    """Block tables of sequences of L rows over distinct pages, -1 behind them, and the number of pages."""
    B, mb = L.numel(), max(1, (int(L.max()) + ps - 1) // ps)
    live = torch.arange(mb)[None, :] * ps < L[:, None]
    n = int(live.sum())
    P = n + n // 10 + 1
    bt = torch.full((B, mb), -1, dtype=torch.int32)
    bt[live] = torch.randperm(P, generator=h)[:n].to(torch.int32)
    return bt, P


def _rows_like(shape, g):
    """Key or value rows [..., heads, dims]: normal values, each row with a size of its own."""
    x = torch.randn(shape, device=DEV, generator=g)
    return x.mul_(torch.randn(shape[:-1] + (1,), device=DEV, generator=g).mul_(0.4).exp_())


def _int8_pool(P, ps, blk, hkv, d, g):
    """Codes of such rows and their scales, block by block."""
    codes = torch.empty((P * ps // blk, blk, hkv, d), device=DEV, dtype=torch.int8)
    scales = torch.empty((P * ps // blk, hkv), device=DEV)
    step = max(1, (1 << 27) // (blk * hkv * d))
    for s in range(0, codes.shape[0], step):
        e = min(codes.shape[0], s + step)
        x = _rows_like((e - s, blk, hkv, d), g)
        scales[s:e] = x.abs().amax((1, 3)) / QMAX
        codes[s:e] = (x / scales[s:e, None, :, None]).round().to(torch.int8)
    return codes.view(P, ps, hkv, d), scales.view(P, ps // blk, hkv)


def _pool(P, case, g):
    """A pool of the case's type and its scales (None but for int8)."""
    ps, hkv, d = case["ps"], case["hkv"], case["d"]
    if case["dtype"] == "int8":
        return _int8_pool(P, ps, case["blk"], hkv, d, g)
    x = torch.empty((P, ps, hkv, d), device=DEV, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float8_e4m3fn)
    step = max(1, (1 << 27) // (ps * hkv * d))
    for s in range(0, P, step):
        e = min(P, s + step)
        y = _rows_like((e - s, ps, hkv, d), g)
        x[s:e] = y.to(torch.bfloat16) if case["dtype"] == "bf16" else (y / SCALE8).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x, None


def prepare(case, seed):
    g, h = _gen(seed)
    s = {"case": case}
    kind = case["kind"]
    if kind in ("rows", "pages"):
        B, L, ps = case["B"], _lens(case), case["ps"]
        width = max(1, -(-case["hi"] // ps)) * ps
        m = torch.empty((B, width), device=DEV).exponential_(generator=g)
        # keys that no query has seen yet tie at 0
        s["mass"] = m.masked_fill_(torch.rand((B, width), device=DEV, generator=g) < case["fresh"], 0.0)
        s["L"] = L.to(torch.int32).to(DEV)
        s["new_mass"] = torch.zeros_like(m)
        if kind == "rows":
            s["ptr"] = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
            s["keep"] = torch.zeros(B * (case["budget"] - case["sinks"]), dtype=torch.int32, device=DEV)
            s["base"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        else:
            bt, _ = _tables(L, ps, h)
            full = torch.full((B, width // ps), -1, dtype=torch.int32)
            full[:, :bt.shape[1]] = bt
            s["bt"] = full.to(DEV)
            s["new_bt"], s["new_L"] = torch.zeros_like(s["bt"]), torch.zeros_like(s["L"])
        return s
    B, hkv, d, ps = (case[k] for k in ("B", "hkv", "d", "ps"))
    if kind == "append":
        n, L0 = _lens(case, "n_"), _lens(case, "c_")
        bt, P = _tables(L0 + n, ps, h)
        T = int(n.sum())
        b = torch.repeat_interleave(torch.arange(B), n)
        pos = L0[b] + torch.arange(T) - (n.cumsum(0) - n)[b]
        slots = torch.cat([bt[b, pos // ps].long() * ps + pos % ps, torch.full((case["pad"],), -1)])
        s["slots"] = slots.to(DEV)
        N = slots.numel()
        if case["packed"]:  # k, v are slices of the rows of one product
            kv = _rows_like((N, 2 * hkv, d), g).to(torch.bfloat16)
            s["k"], s["v"] = kv[:, :hkv], kv[:, hkv:]
        else:
            s["k"], s["v"] = (_rows_like((N, hkv, d), g).to(torch.bfloat16) for _ in range(2))
        (s["kp"], s["ks"]), (s["vp"], s["vs"]) = (_int8_pool(P, ps, case["blk"], hkv, d, g) for _ in range(2))
        return s
    hq = case["hq"]
    if kind == "prefill":
        n = _lens(case, "n_")
        L = _lens(case, "c_") + n
    else:
        L = _lens(case)
        n = torch.ones_like(L)
    bt, P = _tables(L, ps, h)
    qsl = torch.zeros(B + 1, dtype=torch.int64)
    qsl[1:] = n.cumsum(0)
    (s["kp"], s["ks"]), (s["vp"], s["vs"]) = (_pool(P, case, g) for _ in range(2))
    s.update(q=torch.randn((int(n.sum()), hq, d), device=DEV, generator=g).to(torch.bfloat16), bt=bt.to(DEV),
             L=L.to(torch.int32).to(DEV), qsl=qsl.to(torch.int32).to(DEV), scale=d ** -0.5, n_max=int(n.max()),
             l_max=int(L.max()), scales=SCALE8 if case["dtype"] == "e4m3" else 1.0)
    s["out"] = torch.empty_like(s["q"])
    if kind == "mass":
        width = bt.shape[1] * ps
        s["mass"] = None if case["first"] else torch.empty((B, width), device=DEV).exponential_(generator=g)
        s["new_mass"] = torch.zeros((B, width), device=DEV)
    if own and kind != "prefill":
        from serving_slot_mapping_gb300 import capi
        s["ws"] = (capi.decode_workspace(B, hq, s["kp"]) if kind == "decode"
                   else capi.decode_mass_workspace(B, hq, s["kp"], s["l_max"]))
    return s


# --------------------------------------------------------------------------
# the operators, plainly
# --------------------------------------------------------------------------

def _scale_of(rows, old, first):
    """New scales [blocks, heads] from the largest magnitudes of the written rows: those alone where the block's first
    slot is written, else no less than the scale that the block has."""
    new = (rows / torch.full((), QMAX, device=DEV)).clamp(SCALE_MIN, SCALE_MAX)
    return torch.where(first[:, None], new, torch.maximum(old.clamp(SCALE_MIN, SCALE_MAX), new))


def _plain_append(s):
    c = s["case"]
    blk, hkv, d = c["blk"], c["hkv"], c["d"]
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][at]
    blocks, of = torch.unique(slot // blk, return_inverse=True)
    first = torch.zeros(blocks.numel(), dtype=torch.bool, device=DEV)
    first[of[slot % blk == 0]] = True
    mine = torch.zeros((blocks.numel(), blk), dtype=torch.bool, device=DEV)
    mine[of, slot % blk] = True
    for pool, scales, x in ((s["kp"], s["ks"], s["k"]), (s["vp"], s["vs"], s["v"])):
        x = x[at].float()
        flat, sc = pool.view(-1, blk, hkv, d), scales.view(-1, hkv)
        most = torch.zeros((blocks.numel(), hkv), device=DEV)
        most.scatter_reduce_(0, of[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
        old = sc[blocks]
        new = _scale_of(most, old, first)
        had = flat[blocks].float()
        grown = (~first[:, None] & (new > old))[:, None, :] & ~mine[:, :, None]
        moved = (had * (old / new)[:, None, :, None]).round()
        rows = torch.where(grown[..., None], moved, had)
        rows[of, slot % blk] = (x / new[of][:, :, None]).round().clamp(-QMAX, QMAX)
        flat[blocks] = rows.to(torch.int8)
        sc[blocks] = new
    return s["kp"], s["vp"], s["ks"], s["vs"]


def _gather(s, pool, scales, slot, there):
    """fp32 values [B, keys, heads, dims] of the rows at `slot`, zeros where there is no key."""
    hkv, d = pool.shape[2:]
    if pool.dtype == torch.float8_e4m3fn:
        x = pool.view(torch.uint8).view(-1, hkv, d)[slot].view(torch.float8_e4m3fn).float().mul_(s["scales"])
    else:
        x = pool.view(-1, hkv, d)[slot].float()
    if scales is not None:
        x *= scales.view(-1, hkv)[slot // s["case"]["blk"]][..., None]
    return x.masked_fill_(~there[:, :, None, None], 0.0)


def _plain_attend(s, qp, q, want_weights=False):
    """q [B, n, Hq, D] at positions qp [B, n] (below 0: no query) over the keys up to its own."""
    c = s["case"]
    ps, hkv = c["ps"], c["hkv"]
    B, n, hq, d = q.shape
    L = s["L"].long()
    j = torch.arange(s["l_max"], device=DEV)[None, :].expand(B, -1)
    there = j < L[:, None]
    page = torch.gather(s["bt"].long(), 1, j // ps)
    slot = torch.where(there, page * ps + j % ps, 0)
    K = _gather(s, s["kp"], s["ks"], slot, there)
    see = there[:, None, :] & (j[:, None, :] <= qp[:, :, None])  # [B, n, keys]
    x = torch.matmul(q.float().view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d),
                     K.permute(0, 2, 3, 1)).view(B, hkv, hq // hkv, n, -1)
    del K
    x = x.mul_(s["scale"]).masked_fill_(~see[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    x = x.div_(x.sum(-1, keepdim=True).clamp(min=1e-30))
    V = _gather(s, s["vp"], s["vs"], slot, there)
    o = torch.matmul(x.view(B, hkv, -1, x.shape[-1]), V.permute(0, 2, 1, 3)).view(B, hkv, hq // hkv, n, d)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, hq, d)
    return (o, x.sum((1, 2, 3))) if want_weights else o


def _plain_decode(s):
    s["out"].copy_(_plain_attend(s, s["L"].long()[:, None] - 1, s["q"][:, None])[:, 0])
    return s["out"]


def _plain_mass(s):
    L, m = s["L"].long(), s["l_max"]
    o, w = _plain_attend(s, L[:, None] - 1, s["q"][:, None], True)
    s["out"].copy_(o[:, 0])
    if s["mass"] is not None:
        w = s["mass"][:, :m] * s["case"]["decay"] + w
    live = torch.arange(m, device=DEV)[None, :] < L[:, None]
    s["new_mass"][:, :m] = torch.where(live, w, s["new_mass"][:, :m])
    return s["out"], s["new_mass"]


def _plain_prefill(s):
    L, qsl = s["L"].long(), s["qsl"].long()
    n = qsl[1:] - qsl[:-1]
    i = torch.arange(s["n_max"], device=DEV)[None, :]
    there = i < n[:, None]
    row = (qsl[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    qp = torch.where(there, (L - n)[:, None] + i, -1)
    o = _plain_attend(s, qp, s["q"][row])
    s["out"][row[there]] = o[there].to(s["out"].dtype)
    return s["out"]


def _heaviest(score, may, count):
    """Of the entries that `may` be taken, the `count` [B, 1] highest of each row, ties by the lower index."""
    x = torch.where(may, score, -math.inf)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order)
    rank.scatter_(1, order, torch.arange(x.shape[1], device=DEV)[None, :].expand_as(order))
    return may & (rank < count)


def _moved(mass, kept, out):
    """The kept entries of each row in front, zeros behind."""
    b, i = torch.nonzero(kept, as_tuple=True)
    out.zero_()
    out[b, kept.cumsum(1)[b, i] - 1] = mass[b, i]
    return out


def _plain_rows(s):
    c, L = s["case"], s["L"].long()[:, None]
    j = torch.arange(s["mass"].shape[1], device=DEV)[None, :]
    over = L > c["budget"]
    middle = over & (j >= c["sinks"]) & (j < L - c["recent"])
    top = _heaviest(s["mass"], middle, c["budget"] - c["sinks"] - c["recent"])
    kept = (j < L) & (top | ~middle)
    listed_ = kept & over & (j >= c["sinks"])
    s["ptr"][1:] = listed_.sum(1).cumsum(0).to(torch.int32)
    at = torch.nonzero(listed_)[:, 1]
    s["keep"][:at.numel()] = at.to(torch.int32)
    s["base"].copy_(torch.where(over, c["sinks"], L)[:, 0])
    return s["ptr"], s["keep"], s["base"], _moved(s["mass"], kept, s["new_mass"])


def _plain_pages(s):
    c, L, ps = s["case"], s["L"].long()[:, None], s["case"]["ps"]
    B, width = s["mass"].shape
    j = torch.arange(width, device=DEV)[None, :]
    x = s["mass"].masked_fill(j >= L, 0.0).view(B, -1, ps)
    while x.shape[-1] > 1:  # a page's weight: halves added, again and again
        x = x[..., :x.shape[-1] // 2] + x[..., x.shape[-1] // 2:]
    pages, m = -(-L // ps), torch.arange(width // ps, device=DEV)[None, :]
    over = pages > c["budget"]
    front, back = -(-c["sinks"] // ps), torch.div(L - max(1, c["recent"]), ps, rounding_mode="floor").clamp(min=0)
    middle = over & (m >= front) & (m < back)
    top = _heaviest(x[..., 0], middle, c["budget"] - front - (pages - back))
    kept = (m < pages) & (top | ~middle)
    there = m < pages
    order = torch.where(kept, kept.cumsum(1) - 1, kept.sum(1, keepdim=True) + (there & ~kept).cumsum(1) - 1)
    order = torch.where(there, order, m)
    s["new_bt"].scatter_(1, order, s["bt"])
    s["new_L"].copy_((L - ps * (pages - kept.sum(1, keepdim=True)))[:, 0])
    rows = kept.repeat_interleave(ps, 1) & (j < L)
    return s["new_bt"], s["new_L"], _moved(s["mass"], rows, s["new_mass"])


# --------------------------------------------------------------------------
# the operators, by the library
# --------------------------------------------------------------------------

def _own(s):
    from serving_slot_mapping_gb300 import capi
    c = s["case"]
    kind = c["kind"]
    if kind == "append":
        capi.paged_kv_append_int8(s["kp"], s["vp"], s["ks"], s["vs"], s["k"], s["v"], s["slots"])
        return s["kp"], s["vp"], s["ks"], s["vs"]
    if kind == "decode":
        return capi.paged_attention_decode_int8(s["kp"], s["vp"], s["ks"], s["vs"], s["q"], s["bt"], s["L"], s["scale"],
                                                max_seq_len=s["l_max"], out=s["out"], workspace=s["ws"])
    if kind == "prefill":
        return capi.paged_attention_prefill_int8(s["kp"], s["vp"], s["ks"], s["vs"], s["q"], s["qsl"], s["bt"], s["L"],
                                                 s["scale"], s["n_max"], max_seq_len=s["l_max"], out=s["out"])
    if kind == "mass":
        out = capi.paged_attention_decode_mass(s["kp"], s["vp"], s["q"], s["bt"], s["L"], s["scale"], s["new_mass"],
                                               mass_in=s["mass"], decay=c["decay"], max_seq_len=s["l_max"], out=s["out"],
                                               workspace=s["ws"], k_scale=s["scales"], v_scale=s["scales"],
                                               key_scales=s["ks"], value_scales=s["vs"])
        return out, s["new_mass"]
    if kind == "rows":
        return capi.paged_kv_evict_rows(s["mass"], s["L"], c["budget"], c["sinks"], c["recent"], keep_indptr=s["ptr"],
                                        keep=s["keep"], base=s["base"], new_mass=s["new_mass"])
    return capi.paged_kv_evict_pages(s["mass"], s["bt"], s["L"], c["ps"], c["budget"], c["sinks"], c["recent"],
                                     new_block_table=s["new_bt"], new_seq_lens=s["new_L"], new_mass=s["new_mass"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill, "mass": _plain_mass,
            "rows": _plain_rows, "pages": _plain_pages}[state["case"]["kind"]](state)


# --------------------------------------------------------------------------
# work, and the results in 64 bits
# --------------------------------------------------------------------------

def work(case):
    kind, B = case["kind"], case["B"]
    if kind in ("rows", "pages"):
        L = _lens(case)
        width = max(1, -(-case["hi"] // case["ps"])) * case["ps"]
        b = 4 * int(L.sum()) + 4 * B * width + 4 * B
        if kind == "rows":
            n = int((L > case["budget"]).sum()) * (case["budget"] - case["sinks"])
            return {"bytes": b + 4 * n + 8 * B, "flops": 0}
        return {"bytes": b + 8 * B * (width // case["ps"]) + 4 * B, "flops": 0}
    hkv, d, ps = case["hkv"], case["d"], case["ps"]
    if kind == "append":
        n, L0 = _lens(case, "n_"), _lens(case, "c_")
        T, blk = int(n.sum()), case["blk"]
        blocks = int(((L0 + n + blk - 1) // blk - L0 // blk).sum())
        kept = int((L0 % blk > 0).sum())  # blocks whose scale is read
        return {"bytes": 2 * T * hkv * d * 3 + 8 * (T + case["pad"]) + 8 * hkv * (blocks + kept), "flops": 2 * T * hkv * d * 2}
    e = {"bf16": 2, "e4m3": 1, "int8": 1}[case["dtype"]]
    hq = case["hq"]
    n = _lens(case, "n_") if kind == "prefill" else torch.ones(B, dtype=torch.int64)
    L = _lens(case, "c_") + n if kind == "prefill" else _lens(case)
    keys = int(L.sum())
    pairs = int((n * (L - n) + n * (n + 1) // 2).sum())
    b = keys * hkv * d * 2 * e + keys / ps * 4 + 2 * int(n.sum()) * hq * d * 2
    if case["dtype"] == "int8":
        b += keys / case["blk"] * hkv * 8
    if kind == "mass":
        b += keys * (4 if case["first"] else 8)
    return {"bytes": b, "flops": pairs * hq * d * 4}


def _exact_append(s, c):
    blk, hkv, d = c["blk"], c["hkv"], c["d"]
    slots = s["slots"].cpu()
    tokens = {}
    for t, slot in enumerate(slots.tolist()):
        if slot >= 0:
            tokens.setdefault(slot // blk, []).append((t, slot % blk))
    outs = []
    for scales, x in ((s["ks"], s["k"]), (s["vs"], s["v"])):
        sc = scales.double().cpu().view(-1, hkv).clone()
        most = x.abs().amax(-1).double().cpu()
        for block, rows in tokens.items():
            new = (most[[t for t, _ in rows]].amax(0) / QMAX).clamp(SCALE_MIN, SCALE_MAX)
            fresh = any(o == 0 for _, o in rows)
            sc[block] = new if fresh else torch.maximum(sc[block].clamp(SCALE_MIN, SCALE_MAX), new)
        outs.append(sc.view(scales.shape).to(DEV))
    return None, None, outs[0], outs[1]


def _exact_rows(s, pool, scales, slot):
    """64-bit values [heads, keys, dims] of the rows at `slot`."""
    hkv, d = pool.shape[2:]
    if pool.dtype == torch.float8_e4m3fn:
        x = pool.view(torch.uint8).view(-1, hkv, d)[slot].view(torch.float8_e4m3fn).float().double() * s["scales"]
    else:
        x = pool.view(-1, hkv, d)[slot].double()
    if scales is not None:
        x = x * scales.view(-1, hkv)[torch.div(slot, s["case"]["blk"], rounding_mode="floor")].double()[:, :, None]
    return x.transpose(0, 1)


def _exact_attend(s, c):
    ps, hkv, hq = c["ps"], c["hkv"], c["hq"]
    L, bt, qsl = s["L"].tolist(), s["bt"].cpu().long(), s["qsl"].tolist()
    out = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    mass = s["new_mass"].double() if "new_mass" in s else None
    for b in range(c["B"]):  # one sequence at a time
        n = qsl[b + 1] - qsl[b]
        j = torch.arange(L[b])
        slot = (bt[b][j // ps] * ps + j % ps).to(DEV)
        K, V = _exact_rows(s, s["kp"], s["ks"], slot), _exact_rows(s, s["vp"], s["vs"], slot)
        j = j.to(DEV)
        for a in range(0, n, 256):  # rows of queries
            e = min(n, a + 256)
            q = s["q"][qsl[b] + a:qsl[b] + e].double().view(e - a, hkv, hq // hkv, -1)
            x = torch.einsum("nhgd,hkd->hgnk", q, K) * s["scale"]
            hide = j[None] > torch.arange(L[b] - n + a, L[b] - n + e, device=DEV)[:, None]
            w = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            out[qsl[b] + a:qsl[b] + e] = torch.einsum("hgnk,hkd->nhgd", w, V).reshape(e - a, hq, -1)
            if mass is not None:
                before = 0.0 if s["mass"] is None else s["mass"][b, :L[b]].double() * c["decay"]
                mass[b, :L[b]] = before + w.sum((0, 1, 2))
    return out if mass is None else (out, mass)


def _exact_evict(s, c):
    pages, ps = c["kind"] == "pages", c["ps"] if c["kind"] == "pages" else 1
    out = torch.zeros(s["mass"].shape, dtype=torch.float64)
    for b, (n, row) in enumerate(zip(s["L"].tolist(), s["mass"].double().cpu())):
        units = -(-n // ps)
        front = -(-c["sinks"] // ps)
        back = max(0, (n - max(1, c["recent"])) // ps) if pages else n - c["recent"]
        keep = list(range(units))
        if units > c["budget"]:
            padded = torch.zeros(units * ps, dtype=torch.float64)
            padded[:n] = row[:n]
            weight = padded.view(units, ps).sum(1)
            order = torch.sort(weight[front:back], descending=True, stable=True).indices + front
            best = order[:c["budget"] - front - (units - back)].tolist()
            keep = sorted(list(range(front)) + best + list(range(back, units)))
        at = (torch.tensor(keep, dtype=torch.int64)[:, None] * ps + torch.arange(ps)[None, :]).reshape(-1)
        at = at[at < n]
        out[b, :at.numel()] = row[at]
    out = out.to(DEV)
    return (None, None, out) if pages else (None, None, None, out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "append":
        return _exact_append(s, case)
    if case["kind"] in ("rows", "pages"):
        return _exact_evict(s, case)
    return _exact_attend(s, case)
