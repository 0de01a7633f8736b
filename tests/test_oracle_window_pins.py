"""Pins of the oracle's sliding-window attention and row moves: closed forms,
the plain attention where the window hides nothing, and invariants."""
import numpy as np
import pytest

import oracle


def _step(rng, lens, hq=4, hkv=2, d=8, ps=4, extra=3):
    B = len(lens)
    mb = max(1, max((n + ps - 1) // ps for n in lens))
    P = sum((n + ps - 1) // ps for n in lens) + extra
    ids = rng.permutation(P)
    bt = np.full((B, mb), -1)
    at = 0
    for b, n in enumerate(lens):
        k = (n + ps - 1) // ps
        bt[b, :k] = ids[at:at + k]
        at += k
    return (rng.standard_normal((P, ps, hkv, d)), rng.standard_normal((P, ps, hkv, d)),
            rng.standard_normal((B, hq, d)), bt)


def test_a_window_that_hides_nothing_is_plain_attention():
    rng = np.random.default_rng(1)
    lens = [0, 1, 5, 19]
    kp, vp, q, bt = _step(rng, lens)
    plain = oracle.paged_attention_decode(kp, vp, q, bt, lens, 0.3)
    for window, sinks in ((19, 0), (1, 19), (100, 7)):
        got = oracle.paged_attention_decode_window(kp, vp, q, bt, lens, 0.3, window, sinks)
        np.testing.assert_allclose(got, plain, rtol=0, atol=1e-12)


def test_window_is_plain_attention_over_the_visible_keys():
    rng = np.random.default_rng(2)
    lens = [23]
    kp, vp, q, bt = _step(rng, lens)
    K, V = oracle.gather_pages(kp, bt[0], 23), oracle.gather_pages(vp, bt[0], 23)
    for window, sinks in ((1, 0), (5, 2), (9, 11), (20, 4)):
        idx = [j for j in range(23) if j >= 23 - window or j < sinks]
        assert oracle.visible_keys(22, window, sinks) == idx
        exp = oracle.attend(q, K[idx], V[idx], [len(idx) - 1], 0.5)[0]
        got = oracle.paged_attention_decode_window(kp, vp, q, bt, lens, 0.5, window, sinks)[0]
        np.testing.assert_allclose(got, exp, rtol=0, atol=1e-12)


def test_window_one_without_sinks_is_the_last_value():
    rng = np.random.default_rng(3)
    kp, vp, q, bt = _step(rng, [9])
    got = oracle.paged_attention_decode_window(kp, vp, q, bt, [9], 0.7, 1, 0)[0]
    last = vp[bt[0, 2], 0]
    np.testing.assert_allclose(got, np.repeat(last, 2, axis=0), atol=1e-14)


def test_prefill_rows_are_decodes_of_shorter_sequences():
    rng = np.random.default_rng(4)
    lens = [14, 6]
    kp, vp, _, bt = _step(rng, lens)
    n = [5, 8]                     # the second sequence has rows below position 0
    q = rng.standard_normal((13, 4, 8))
    got = oracle.paged_attention_prefill_window(kp, vp, q, [0, 5, 13], bt, lens, 0.4, 4, 2)
    for b, s0 in ((0, 0), (1, 5)):
        for i in range(n[b]):
            L = max(0, lens[b] - n[b] + i + 1)
            exp = oracle.paged_attention_decode_window(kp, vp, q[s0 + i:s0 + i + 1], bt[b:b + 1], [L], 0.4, 4, 2)
            np.testing.assert_allclose(got[s0 + i], exp[0], atol=1e-13)


def test_hidden_pages_are_never_read():
    rng = np.random.default_rng(5)
    kp, vp, q, bt = _step(rng, [40])
    exp = oracle.paged_attention_decode_window(kp, vp, q, bt, [40], 0.4, 6, 3)
    bt2 = bt.copy()
    bt2[0, 1:8] = 10 ** 6          # pages between the sinks (page 0) and the window (pages 8, 9)
    np.testing.assert_array_equal(oracle.paged_attention_decode_window(kp, vp, q, bt2, [40], 0.4, 6, 3), exp)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_differences(interleaved):
    rng = np.random.default_rng(6)
    table = oracle.rope_table(50, 16)
    x, y = rng.standard_normal((2, 1, 1, 24))
    turned = lambda v, p: oracle.rotate(v[0], table[p, :8], table[p, 8:], interleaved)[0]
    for p in (0, 3, 49):
        assert np.isclose(np.linalg.norm(turned(x, p)), np.linalg.norm(x))
        np.testing.assert_array_equal(turned(x, p)[16:], x[0, 0, 16:])
    np.testing.assert_allclose(turned(x, 0), x[0, 0])
    # the product of two rotated rows depends on the difference of the positions alone
    assert np.isclose(turned(x, 7) @ turned(y, 3), turned(x, 44) @ turned(y, 40))


def test_rotation_closed_form():
    table = np.array([[0.0, 1.0, 1.0, 0.0]])   # quarter turn of pair 0, none of pair 1
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    q, k = oracle.qk_norm_rope(x, x, [0], table, None, None, 0.0, False)
    np.testing.assert_allclose(q[0, 0], [-3.0, 2.0, 1.0, 4.0])
    q, k = oracle.qk_norm_rope(x, x, [0], table, None, None, 0.0, True)
    np.testing.assert_allclose(q[0, 0], [-2.0, 1.0, 3.0, 4.0])


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(7).standard_normal((3, 2, 32)) * 9
    y = oracle.rms_norm(x, np.ones(32), 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1.0)
    np.testing.assert_allclose(oracle.rms_norm(x, 2 * np.ones(32), 0.0), 2 * y)
    np.testing.assert_array_equal(oracle.rms_norm(x, None, 0.0), x)


def test_compact_is_gathering_the_kept_rows():
    rng = np.random.default_rng(8)
    kp, _, _, bt = _step(rng, [13, 0, 7])
    base, ptr = [2, 0, 0], [0, 4, 4, 6]
    keep = [3, 4, 9, 12, 0, 6]
    out = oracle.paged_kv_compact(kp, bt, base, ptr, keep)
    old = oracle.gather_pages(kp, bt[0], 13)
    np.testing.assert_array_equal(oracle.gather_pages(out, bt[0], 6), old[[0, 1, 3, 4, 9, 12]])
    np.testing.assert_array_equal(oracle.gather_pages(out, bt[0], 13)[6:], old[6:])
    np.testing.assert_array_equal(oracle.gather_pages(out, bt[2], 2), oracle.gather_pages(kp, bt[2], 7)[[0, 6]])


def test_copy_pages_moves_whole_pages():
    kp = np.arange(24.0).reshape(6, 4)
    out = oracle.paged_kv_copy_pages(kp, [1, 5, -1, 2], [0, 3, 4, -1])
    np.testing.assert_array_equal(out, kp[[1, 1, 2, 5, 4, 5]])
