"""The oracle of int8 pools, attention weights and eviction, pinned by hand-worked
values, invariants and another way of computing the same (no GPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import evict, kv_int8


def state(P=3, ps=32, blk=16, hkv=2, d=4, seed=0):
    rng = np.random.default_rng(seed)
    return (rng.integers(-127, 128, size=(P, ps, hkv, d), dtype=np.int8),
            rng.uniform(0.5, 2.0, size=(P, ps // blk, hkv)).astype(np.float32), rng)


def test_values_of_codes():
    codes, scales, _ = state()
    scales[0, 1, 0], scales[1, 0, 1], scales[2, 0, 0] = np.nan, np.inf, 0.0
    x = kv_int8.dequantize(codes, scales)
    for p, s, h in ((0, 3, 1), (0, 20, 0), (1, 5, 1), (2, 0, 0), (2, 31, 1)):
        sc = {(0, 20, 0): 2.0 ** -40, (1, 5, 1): 2.0 ** 40, (2, 0, 0): 2.0 ** -40}.get((p, s, h), float(scales[p, s // 16, h]))
        assert np.array_equal(x[p, s, h], codes[p, s, h].astype(np.float64) * sc)


def test_append_by_hand():
    codes, scales = np.zeros((1, 16, 1, 3), dtype=np.int8), np.full((1, 1, 1), 9.0, dtype=np.float32)
    c, s = kv_int8.append_int8(codes, scales, [[[127.0, -63.5, 0.5]]], [0])      # a new block: scale 1
    assert s[0, 0, 0] == 1 and c[0, 0, 0].tolist() == [127, -64, 0]
    c, s = kv_int8.append_int8(c, s, [[[2.0, 3.0, 2.5]]], [1])                   # smaller: the scale stays
    assert s[0, 0, 0] == 1 and c[0, 1, 0].tolist() == [2, 3, 2]
    c, s = kv_int8.append_int8(c, s, [[[254.0, 3.0, float("nan")]]], [2])        # larger: twice the scale
    assert s[0, 0, 0] == 2 and c[0, :3, 0].tolist() == [[64, -32, 0], [1, 2, 1], [127, 2, 0]]
    c, s = kv_int8.append_int8(c, s, [[[-1.0, 0.0, float("inf")]]], [3])         # infinities take the largest scale
    assert s[0, 0, 0] == 2.0 ** 40 and c[0, :4, 0].tolist() == [[0, 0, 0]] * 3 + [[0, 0, 127]]
    c, s = kv_int8.append_int8(c, s, [[[0.0, 0.0, 0.0]]], [0])                   # the first slot again
    assert s[0, 0, 0] == np.float32(2.0 ** -40) and c[0, 0, 0].tolist() == [0, 0, 0]


def test_append_is_within_half_a_step_and_touches_nothing_else():
    codes, scales, rng = state(P=4)
    rows = rng.standard_normal((40, 2, 4)).astype(np.float32)
    slots = [64 + i for i in range(32)] + [-1] * 3 + [5, 6, 7, 8, 9]
    c, s = kv_int8.append_int8(codes, scales, rows, slots)
    x = kv_int8.dequantize(c, s).reshape(-1, 2, 4)
    for t, slot in enumerate(slots):
        if slot >= 0:
            sc = s.reshape(-1, 2)[slot // 16][:, None]
            assert (np.abs(x[slot] - rows[t]) <= sc * 0.5 * (1 + 2.0 ** -20)).all()
    same = np.ones(codes.shape[:2], dtype=bool)
    same[2] = False                          # the new blocks
    same[0, :16] = False                     # a block in use
    assert np.array_equal(c[same], codes[same])
    assert np.array_equal(s[1], scales[1]) and np.array_equal(s[0, 1], scales[0, 1]) and np.array_equal(s[3], scales[3])
    assert (s[0, 0] >= scales[0, 0]).all()


def test_order_of_tokens_does_not_matter():
    codes, scales, rng = state()
    rows = rng.standard_normal((20, 2, 4)).astype(np.float32)
    slots = rng.permutation(60)[:20]
    a = kv_int8.append_int8(codes, scales, rows, slots)
    o = rng.permutation(20)
    b = kv_int8.append_int8(codes, scales, rows[o], slots[o])
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_weights_against_a_library_softmax():
    rng = np.random.default_rng(3)
    pool, q = rng.standard_normal((9, 8, 2, 16)), rng.standard_normal((2, 6, 16))
    table, lens = rng.permutation(9)[:8].reshape(2, 4), [27, 9]
    got = evict.key_weights(pool, q, table, lens, 0.25)
    for b in range(2):
        K = torch.from_numpy(pool[table[b]].reshape(-1, 2, 16)[:lens[b]]).repeat_interleave(3, 1)
        w = torch.softmax(0.25 * torch.einsum("hd,khd->hk", torch.from_numpy(q[b]), K), -1).sum(0).numpy()
        assert np.allclose(got[b], w, atol=1e-14) and abs(got[b].sum() - 6) < 1e-12


def test_rows_by_hand():
    m = np.array([[9, 1, 5, 5, 2, 5, 0, 7, 3, 1]], dtype=np.float32)
    assert evict.evict_rows(m, [10], 10, 1, 1) == [(10, [])]
    assert evict.evict_rows(m, [10], 5, 1, 1) == [(1, [2, 3, 7, 9])]       # 7, then the first two of the 5s
    assert evict.evict_rows(m, [10], 2, 1, 1) == [(1, [9])]
    assert evict.evict_rows(m, [8], 3, 0, 0) == [(0, [0, 2, 7])]
    m[0, 7] = np.nan
    assert evict.evict_rows(m, [10], 5, 1, 1) == [(1, [2, 3, 5, 9])]
    assert evict.moved(m[0], [0, 2, 9], 5).tolist() == [9, 5, 1, 0, 0]


def test_pages_by_hand():
    m = np.array([[1, 0, 4, 4, 2, 5, 0, 8, 3]], dtype=np.float32)           # pages of 2: 1 8 7 8 3
    assert evict.evict_pages(m, [9], 2, 5, 0, 0) == [([0, 1, 2, 3, 4], [])]
    assert evict.evict_pages(m, [9], 2, 3, 1, 1) == [([0, 1, 4], [2, 3])]   # page 1 and 3 tie: the lower
    assert evict.evict_pages(m, [9], 2, 3, 0, 2) == [([1, 3, 4], [0, 2])]   # two rows reach into page 3
    assert evict.evict_pages(m, [8], 2, 2, 0, 1) == [([1, 3], [0, 2])]
    assert evict.page_weight([1e8, 1, -1e8, 1]) == 2                        # halves: (1e8 - 1e8) + (1 + 1)


@pytest.mark.parametrize("seed", range(5))
def test_rows_are_the_pages_of_one_row(seed):
    rng = np.random.default_rng(seed)
    m = rng.integers(0, 6, size=(4, 50)).astype(np.float32)
    lens = rng.integers(0, 51, size=4)
    rows, pages = evict.evict_rows(m, lens, 20, 3, 4), evict.evict_pages(m, lens, 1, 20, 3, 4)
    for (base, kept), (stay, go) in zip(rows, pages):
        assert list(range(base)) + kept == stay


def test_rows_feed_the_compaction():
    rng = np.random.default_rng(1)
    lens, table = np.array([40, 12]), rng.permutation(6).reshape(2, 3)
    pool = rng.standard_normal((6, 16, 1, 2))
    m = rng.random((2, 48)).astype(np.float32)
    picked = evict.evict_rows(m, lens, 15, 2, 3)
    ptr = np.concatenate([[0], np.cumsum([len(k) for _, k in picked])])
    out = oracle.paged_kv_compact(pool, table, [b for b, _ in picked], ptr, sum((k for _, k in picked), []))
    assert [b + len(k) for b, k in picked] == [15, 12]
    for b, (base, kept) in enumerate(picked):
        for i, j in enumerate(list(range(base)) + kept):
            assert np.array_equal(out[table[b, i // 16], i % 16], pool[table[b, j // 16], j % 16])
