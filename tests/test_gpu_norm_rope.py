"""paged_qk_norm_rope_append against the oracle.

Tolerance: the arithmetic is fp32.  The sum of squares of a head takes at most
16 adds in a thread and 5 across lanes, then a division, an add, a root and a
reciprocal: its inverse root is off by at most (22 / 2 + 4) * 2^-24; two more
products give a normed value, the rotation adds three roundings of terms of
magnitude |a| + |b|: 24 * 2^-24 (|a| + |b|) bounds all of it.  Then one rounding
to the output: 2^-8 (bf16), 2^-24 (f32), 2^-4 relative or half of the least step
2^-9 (e4m3, on top of the quotient's 2^-24)."""
import numpy as np
import pytest
import torch

import oracle
from serving_slot_mapping_gb300 import build as build_mod
from serving_slot_mapping_gb300 import capi

from _parity import bits, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    build_mod.build()
    capi.lib()
    capi.device_error()  # clear


def _inputs(dev, T, hq, hkv, d, dtype, packed=True, rot=None, norm=True, pad=0, ps=16, seed=0, max_pos=4000, odd=0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    row = torch.float32 if dtype == "f32" else torch.bfloat16
    n = hq + 2 * hkv
    wide = torch.randn(T, n * d + odd, generator=g).to(row).to(dev)
    x = wide[:, :n * d].unflatten(1, (n, d))
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    P = (T + ps) // ps + 3
    pool_t = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[dtype]
    kp, vp = (torch.randn(P, ps, hkv, d, generator=g).to(pool_t).to(dev) for _ in range(2))
    slots = rng.permutation(P * ps)[:T].astype(np.int64)
    slots[rng.permutation(T)[:pad]] = -1
    rot = d if rot is None else rot
    s = dict(q=q, k=k, v=v, kp=kp, vp=vp, slots=torch.from_numpy(slots).to(dev), rot=rot)
    s["pos"] = torch.from_numpy(rng.integers(0, max_pos, T).astype(np.int32)).to(dev) if rot else None
    s["cs"] = torch.from_numpy(oracle.rope_table(max_pos, rot).astype(np.float32)).to(dev) if rot else None
    s["qw"], s["kw"] = (((1 + torch.randn(d, generator=g)).to(row).to(dev)) for _ in range(2)) if norm else (None, None)
    return s


def _call(s, out=None, interleaved=False, eps=1e-5, scale=1.0, **k):
    return capi.paged_qk_norm_rope_append(s["kp"], s["vp"], s["q"], s["k"], s["v"], s["slots"], s["pos"], s["cs"],
                                          q_weight=s["qw"], k_weight=s["kw"], eps=eps, interleaved=interleaved, out=out,
                                          k_scale=scale, v_scale=scale, **k)


def _f64(t):
    if t is None:
        return None
    return oracle.kv_fp8.e4m3_decode(bits(t)) if t.dtype == torch.float8_e4m3fn else to_f64(bits(t))


def _pairs(x, rot, interleaved):
    """|a| + |b| of each element's rotated pair (|a| where it is not rotated)."""
    x = np.abs(x)
    y, half = x.copy(), rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = y[..., b] = x[..., a] + x[..., b]
    return y


def _check(s, dtype, interleaved=False, eps=1e-5, scale=1.0):
    kp0, vp0 = s["kp"].clone(), s["vp"].clone()
    q_in, k_in, v_in = (x.contiguous().clone() for x in (s["q"], s["k"], s["v"]))
    out0 = torch.full(s["q"].shape, 3.0, dtype=s["q"].dtype, device=s["q"].device)
    out = _call(s, out=out0, interleaved=interleaved, eps=eps, scale=scale)
    torch.cuda.synchronize()
    assert capi.device_error() == (0, 0)
    slots = s["slots"].cpu().numpy()
    live = slots >= 0
    pos = s["pos"].cpu().numpy() if s["pos"] is not None else None
    cs = _f64(s["cs"])
    eq, ek = oracle.qk_norm_rope(_f64(q_in), _f64(k_in), pos, cs, _f64(s["qw"]), _f64(s["kw"]), eps, interleaved)
    step = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    nq = _pairs(oracle.rms_norm(_f64(q_in), _f64(s["qw"]), eps), s["rot"], interleaved)
    nk = _pairs(oracle.rms_norm(_f64(k_in), _f64(s["kw"]), eps), s["rot"], interleaved)
    got = _f64(out)
    assert (np.abs(got - eq) <= 24 * 2.0 ** -24 * nq + step * np.abs(eq) + 1e-37)[live].all()
    assert (got[~live] == 3.0).all()           # padding rows are left as they were
    # the key pool: written rows within the rounding, every other slot untouched
    hkv, d = s["k"].shape[1:]
    flat, old = _f64(s["kp"]).reshape(-1, hkv, d), _f64(kp0).reshape(-1, hkv, d)
    at = slots[live]
    want = ek[live] / scale
    slack = 24 * 2.0 ** -24 * nk[live] / scale
    if dtype == "e4m3":
        want = np.clip(want, -448, 448)
        tol = slack + 2.0 ** -24 * np.abs(want) + np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10)
    else:
        tol = slack + step * np.abs(want) + 1e-37
    assert (np.abs(flat[at] - want) <= tol).all()
    rest = np.setdiff1d(np.arange(flat.shape[0]), at)
    assert np.array_equal(flat[rest], old[rest], equal_nan=True)
    # the value pool: what the append writes, bit for bit
    if dtype == "e4m3":
        _, ev = oracle.kv_fp8.paged_kv_append_fp8(bits(kp0), bits(vp0), _f64(k_in), _f64(v_in), slots, scale, scale)
    else:
        _, ev = oracle.paged_kv_append(bits(kp0), bits(vp0), bits(k_in), bits(v_in), slots)
    assert bits(s["vp"]).tobytes() == ev.tobytes()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot", [(32, 8, 128, 128), (8, 8, 64, 64), (16, 2, 128, 64), (4, 1, 256, 64),
                                          (5, 1, 96, 96), (3, 3, 80, 32), (4, 2, 64, 8), (2, 1, 40, 24), (6, 2, 8, 8),
                                          (2, 2, 192, 128), (1, 1, 72, 72)])
def test_shapes(cuda_device, dtype, interleaved, hq, hkv, d, rot):
    s = _inputs(cuda_device, 37, hq, hkv, d, dtype, rot=rot, pad=5, seed=hq + d + rot)
    _check(s, dtype, interleaved, scale=0.02 if dtype == "e4m3" else 1.0)


@pytest.mark.parametrize("T", [1, 2, 31, 700, 3001])
@pytest.mark.parametrize("packed", [False, True])
def test_token_counts(cuda_device, T, packed):
    _check(_inputs(cuda_device, T, 32, 8, 128, "bf16", packed=packed, pad=T // 7, seed=T), "bf16")


@pytest.mark.parametrize("dtype,hq,hkv,d,rot,interleaved", [("bf16", 8, 2, 128, 128, False), ("bf16", 4, 4, 64, 32, True),
                                                            ("f32", 4, 2, 64, 64, False), ("f32", 2, 1, 40, 24, True),
                                                            ("e4m3", 6, 2, 96, 96, False), ("bf16", 3, 1, 256, 0, False)])
def test_many_tokens(cuda_device, dtype, hq, hkv, d, rot, interleaved):
    """Thousands of tokens: the kernel that copies token rows through shared
    memory, with padding tokens between."""
    s = _inputs(cuda_device, 6001, hq, hkv, d, dtype, rot=rot, pad=700, seed=d)
    _check(s, dtype, interleaved, scale=0.02 if dtype == "e4m3" else 1.0)


def test_many_tokens_in_place_and_all_padding(cuda_device):
    s = _inputs(cuda_device, 5000, 8, 2, 64, "bf16", packed=False, seed=4)
    expect = _call(s)
    got = _call(s, out=s["q"])
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), expect.view(torch.int16))
    before = s["kp"].clone()
    s["slots"][:] = -1
    out = _call(s, out=torch.full_like(expect, 3.0))
    torch.cuda.synchronize()
    assert torch.all(out == 3.0) and torch.equal(s["kp"].view(torch.int16), before.view(torch.int16))
    s["slots"][:5] = torch.arange(5)
    s["pos"][3] = -7
    _call(s)
    assert capi.device_error() == (6, -7)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_without_norm_or_rotation(cuda_device, dtype):
    scale = 0.02 if dtype == "e4m3" else 1.0
    _check(_inputs(cuda_device, 9, 8, 2, 64, dtype, norm=False), dtype, scale=scale)
    _check(_inputs(cuda_device, 9, 8, 2, 64, dtype, rot=0), dtype, scale=scale)
    s = _inputs(cuda_device, 9, 8, 2, 64, dtype)
    s["qw"] = None                               # only the keys are normed
    _check(s, dtype, scale=scale)
    # neither: the append
    _check(_inputs(cuda_device, 9, 8, 2, 64, dtype, rot=0, norm=False), dtype, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("odd", [1, 4, 8])
def test_odd_strides_and_addresses(cuda_device, dtype, odd):
    # rows that start on no vector boundary
    s = _inputs(cuda_device, 21, 4, 2, 64, dtype, odd=odd)
    _check(s, dtype, scale=0.02 if dtype == "e4m3" else 1.0)
    flat = torch.randn(21 * 4 * 64 + odd, device=cuda_device).to(s["q"].dtype)
    s = _inputs(cuda_device, 21, 4, 2, 64, dtype, packed=False)
    s["q"] = flat[odd:].view(21, 4, 64)
    _check(s, dtype, scale=0.02 if dtype == "e4m3" else 1.0)


@pytest.mark.parametrize("scale", [0.02, 1.0, 1 / 3, 0.0078125, 0.013824462890625, 3.7e-5, 1234.5, 1e-37, 1e37,
                                   float(np.float32(1) - np.float32(2 ** -24)), float(np.float32(0.5) - np.float32(2 ** -25))])
def test_codes_are_those_of_the_division(cuda_device, scale):
    """Every bf16 value (infinities and NaN too) as a value row: the code is that
    of the correctly rounded quotient, as paged_kv_append stores it."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(512, 1, 128).to(cuda_device)
    f8 = torch.float8_e4m3fn
    a = [torch.zeros(32, 16, 1, 128, device=cuda_device).to(f8) for _ in range(4)]
    slots = torch.arange(512, device=cuda_device)
    # keys without norm or rotation go through the same store
    capi.paged_qk_norm_rope_append(a[0], a[1], x, x, x, slots, k_scale=scale, v_scale=scale)
    capi.paged_kv_append(a[2], a[3], x, x, slots, k_scale=scale, v_scale=scale)
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(a[i].view(torch.uint8), a[2 + i].view(torch.uint8))


def test_in_place(cuda_device):
    s = _inputs(cuda_device, 50, 16, 4, 128, "bf16", packed=False, seed=3)
    expect = _call(s)
    got = _call(s, out=s["q"])
    torch.cuda.synchronize()
    assert got.data_ptr() == s["q"].data_ptr()
    assert torch.equal(got.view(torch.int16), expect.view(torch.int16))


def test_extreme_rows(cuda_device):
    s = _inputs(cuda_device, 4, 2, 1, 64, "bf16", packed=False, rot=0)
    s["q"][0] = 0.0                              # 0 / sqrt(0 + eps)
    s["q"][1] = 2.0 ** 100 / 2 ** 60             # squares of 2^80 sum within fp32
    s["q"][2] = 2.0 ** -60
    _check(s, "bf16")
    assert torch.all(_call(s)[0] == 0)


def test_far_positions_read_the_table(cuda_device):
    s = _inputs(cuda_device, 16, 4, 2, 64, "f32", max_pos=200_000, seed=8)
    s["pos"][:2] = torch.tensor([199_999, 0], dtype=torch.int32)
    _check(s, "f32")


def test_bad_slots_and_positions_are_recorded_and_skipped(cuda_device):
    s = _inputs(cuda_device, 6, 4, 2, 64, "bf16", seed=9)
    n_slots = s["kp"].shape[0] * s["kp"].shape[1]
    for bad, code in (("slot", 2), ("pos", 6), ("neg", 6)):
        t = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in s.items()}
        for name in ("q", "k", "v"):
            t[name] = s[name]
        if bad == "slot":
            t["slots"][3] = n_slots
        else:
            t["pos"][3] = 4000 if bad == "pos" else -1
        out = _call(t, out=torch.full((6, 4, 64), 5.0, dtype=torch.bfloat16, device=cuda_device))
        torch.cuda.synchronize()
        assert capi.device_error()[0] == code
        assert torch.all(out[3] == 5.0) and not torch.any(out[2] == 5.0)
        assert torch.equal(t["kp"].view(-1, 2, 64)[s["slots"][3]], s["kp"].view(-1, 2, 64)[s["slots"][3]])


def test_no_tokens(cuda_device):
    s = _inputs(cuda_device, 1, 4, 2, 64, "bf16")
    for k in ("q", "k", "v", "slots", "pos"):
        s[k] = s[k][:0]
    assert _call(s).shape == (0, 4, 64)


def test_captured_and_replayed(cuda_device):
    s = _inputs(cuda_device, 12, 8, 2, 128, "bf16", seed=10)
    eager = _call(s)
    out = torch.zeros_like(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(s, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
