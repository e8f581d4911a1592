"""Which keys a decode over 4-bit rows has summed, told from its outputs: the definition's output in 64
bits beside the outputs with one key left out or one too many."""
import numpy as np

from tests import cache_ref as ref


def one_key_off(q, k_rows, v_rows, lo, keys):
    """q [Hq, D] bf16 bits, one query a head that sees rows lo .. n - 1 of k_rows and v_rows [n, Hkv, bytes].
    (o, {key: o without that key, or with it where key < lo}), each [Hq, D] in 64 bits. Of a lone key there
    is no output without it."""
    n = len(k_rows)
    keys = [j for j in keys if j < lo or n - lo > 1]
    q, k, v = ref.f64(q), ref.kv4_values(k_rows), ref.kv4_values(v_rows)
    G = q.shape[0] // k.shape[1]
    o, off = np.zeros_like(q), {j: np.zeros_like(q) for j in keys}
    for a in range(q.shape[0]):
        sc = k[:, a // G] @ q[a] * q.shape[1] ** -0.5
        p = np.exp(sc - sc[lo:].max())
        total, sums = p[lo:].sum(), p[lo:] @ v[lo:, a // G]
        o[a] = sums / total
        for j in keys:
            sign = 1 if j < lo else -1
            off[j][a] = (sums + sign * p[j] * v[j, a // G]) / (total + sign * p[j])
    return o, off


def assert_sees(got, o, off, what):
    """got - o, projected on what key j would change, is under half of that change: 1 where the key is left
    out (or is one too many). Roundings are independent of the key, so of their length, |o| 2^-8 / sqrt(3)
    at most, only one part in the square root of the number of elements lies along it."""
    err = np.asarray(got, np.float64) - o
    for j, x in off.items():
        share = (err * (x - o)).sum() / ((x - o) ** 2).sum()
        assert abs(share) < 0.5, f"{what}: the output holds {share:.2f} of the change that key {j} makes"
