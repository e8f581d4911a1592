"""The test of which keys a decode sums, on outputs of the oracle with and without a mistake; and the
cut of its tiles between warps."""
import ctypes

import numpy as np
import pytest

import gqa_inputs as gi
from tests import cache_edges as edges
from tests import cache_ref as ref


@pytest.fixture(scope="module")
def gqa():
    import grouped_query_softmax_b200 as m
    return m


@pytest.mark.parametrize("n,lo", [(257, 0), (4099, 0), (20001, 0), (7000, 2904)])
def test_one_key_off_is_seen_and_roundings_are_not(n, lo):
    """An output rounded to bf16, with each product of a probability and a step rounded to fp16, passes;
    with a key less or more it does not."""
    Hq, Hkv, D = 8, 2, 128
    q = gi.normal_bf16(121, gi.TENSOR_Q, (Hq, D))
    k, v = (ref.kv4_pack(gi.normal_bf16(122 + i, i, (n, Hkv, D)))[0] for i in range(2))
    keys = [lo, n // 2 + lo // 2, n - 1] + ([lo - 1] if lo else [])
    o, off = edges.one_key_off(q, k, v, lo, keys)
    rounded = lambda x: gi.bf16_bits_to_f32(ref.bf16_bits(x.astype(np.float32))).reshape(x.shape)
    edges.assert_sees(rounded(o), o, off, "right")
    for j in keys:
        with pytest.raises(AssertionError):
            edges.assert_sees(rounded(off[j]), o, off, "one key off")
    vc, vs, vm = ref.kv4_parts(v)
    narrow = np.zeros_like(o)
    for a in range(Hq):
        h = a // (Hq // Hkv)
        sc = ref.kv4_values(k)[lo:, h] @ ref.f64(q)[a] * D ** -0.5
        p = np.exp(sc - sc.max())
        top = vs[lo:, h].max() / 2 ** 10
        w = (p[:, None] * vs[lo:, h] / top).astype(np.float16).astype(np.float64) * top
        narrow[a] = (w * (vc[lo:, h] - 8) + p[:, None] * (vm[lo:, h] + 8 * vs[lo:, h])).sum(0) / p.sum()
    edges.assert_sees(rounded(narrow), o, off, "with products in fp16")


def test_decode_cut_covers_every_tile_once(gqa):
    f = ctypes.CDLL(gqa.library_path()).gqa_testing_decode_kv4_cut
    f.argtypes = [ctypes.c_ulonglong, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    runs, start = ctypes.c_int(), ctypes.c_ulonglong()
    rng = np.random.default_rng(5)
    totals = [1, 2, 3, 4095, (1 << 19) - 1, 1 << 19, (1 << 32) + 1, (1 << 52) - 1] + [int(x) for x in rng.integers(1, 1 << 40, 6)]
    for total in totals:
        for places in (1, 7, 148, 1776, 4096):
            want = min(places, -(-total // 2))     # no run is shorter than two tiles, but for a lone tile
            cuts = []
            for i in range(want + 1):
                assert f(total, places, i, ctypes.byref(runs), ctypes.byref(start)) == 0 and runs.value == want
                assert start.value == total * i // want
                cuts.append(start.value)
            assert cuts[0] == 0 and cuts[-1] == total and min(b - a for a, b in zip(cuts, cuts[1:])) >= min(total, 1)
            assert f(total, places, want + 1, ctypes.byref(runs), ctypes.byref(start)) == 1
    for bad in ((0, 4, 0), (1 << 52, 4, 0), (9, 0, 0), (9, 4097, 0), (9, 4, -1)):
        assert f(*bad, ctypes.byref(runs), ctypes.byref(start)) == 1
    assert f(9, 4, 0, None, ctypes.byref(start)) == 1
