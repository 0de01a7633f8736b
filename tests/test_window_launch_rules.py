"""Launch rules of the windowed calls (host code, no GPU)."""
import ctypes

from serving_slot_mapping_gb300 import build as build_mod


def test_clusters_of_the_windowed_decode_are_resident_at_once():
    """The rule that picks the CTAs of a (sequence, KV head): where it picks more than
    one, the whole grid fits the GPU with the CTAs an SM that the kernel is built for
    (deep rings: two up to 16 query heads a KV head, one for more)."""
    build_mod.build()
    rule = ctypes.CDLL(build_mod.LIB_PATH)["_ZN2pa21decode_window_clusterEiiiil"]
    rule.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64]
    sms, split = 152, 0
    for group in (1, 4, 8, 9, 16, 17, 32):
        per_sm = 2 if group <= 16 else 1
        for hkv in (1, 2, 8):
            for batch in (1, 3, 9, 10, 12, 18, 19, 24, 28, 37, 38, 50, 76, 152, 153, 228, 304, 305):
                for keys in (1, 100, 129, 1028, 4100, 100_000):
                    c = rule(sms, batch, hkv, group, keys)
                    assert c in (1, 2, 4, 8)
                    if c > 1:
                        split += 1
                        assert batch * hkv * c <= per_sm * sms, (group, hkv, batch, keys, c)
                        assert (keys + 15) // 16 >= 4 * c
    assert split > 100
