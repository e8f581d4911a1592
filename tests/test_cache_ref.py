"""The plain forms of tests/cache_ref.py against their definitions: gradients against
differences, the 4-bit rows' error bound, and the plan's bookkeeping."""
import numpy as np
import pytest

import gqa_inputs as gi
from tests import cache_ref as ref


@pytest.mark.parametrize("rot,interleaved,weighted", [(16, False, True), (8, True, True), (16, True, False), (0, False, True)])
def test_norm_rope_gradient_matches_differences(rot, interleaved, weighted):
    rng = np.random.default_rng(1)
    D, eps = 16, 1e-3
    x, dz = rng.normal(size=(3, 5, D)), rng.normal(size=(3, 5, D))
    w = 1 + 0.3 * rng.normal(size=D) if weighted else None
    cos, sin = ref.angles(5, rot) if rot else (None, None)
    cos, sin = (c.astype(np.float64) if c is not None else None for c in (cos, sin))
    f = lambda x, w: (ref.norm_rope(x, w, eps, cos, sin, interleaved)[0] * dz).sum()
    dx, dw, _, _ = ref.norm_rope_bwd(dz, x, w, eps, cos, sin, interleaved)
    h = 1e-6
    for i in range(40):
        at = tuple(rng.integers(0, n) for n in x.shape)
        hi, lo = x.copy(), x.copy()
        hi[at] += h
        lo[at] -= h
        assert abs((f(hi, w) - f(lo, w)) / (2 * h) - dx[at]) < 1e-7
    if weighted:
        for d in range(D):
            hi, lo = w.copy(), w.copy()
            hi[d] += h
            lo[d] -= h
            assert abs((f(x, hi) - f(x, lo)) / (2 * h) - dw[d]) < 1e-7


def test_kv4_rows_stay_within_their_bound():
    x = gi.normal_bf16(3, gi.TENSOR_K, (500, 64))
    x[7] = 0x3F80          # a constant row
    x[8] = 0               # zeros
    x[9, 5] = 0x7F80       # an infinity
    x[10, 5] = 0x7FC0      # a NaN
    rows, bad = ref.kv4_pack(x)
    v, s = ref.kv4_values(rows), ref.kv4_parts(rows)[1]
    assert bad.nonzero()[0].tolist() == [9, 10] and np.isnan(v[9:11]).all()
    ok = ~bad
    assert (np.abs(v - ref.f64(x))[ok] <= (0.5 + 15 / 512) * s[ok] + 1e-7).all()
    assert (v[7] == 1).all() and (v[8] == 0).all()
    c = ref.kv4_parts(rows)[0]
    assert c[ok].max() == 15 and (c[7] == 0).all()


def test_plan_keeps_every_page_once():
    rng = np.random.default_rng(2)
    S, page, max_pages, pages = 20, 16, 8, 160
    lens = rng.integers(0, 60, S)
    table = np.full((S, max_pages), -1, np.int32)
    order = rng.permutation(pages).astype(np.int32)
    used = 0
    for s in range(S):
        n = -(-lens[s] // page)
        table[s, :n] = order[used:used + n]
        used += n
    free = np.full(pages, -1, np.int32)
    free[:pages - used] = order[used:]
    count = pages - used
    for step in range(30):
        keep = np.where(rng.random(S) < 0.2, rng.integers(0, lens + 1), lens)
        new = np.minimum(rng.integers(0, 20, S), max_pages * page - keep)
        got = ref.plan(lens, keep, new, table, free, count, page, pages, 500)
        assert got is not None
        lens, cu, pos, slots, table, free, count = got
        held = [table[s, i] for s in range(S) for i in range(-(-lens[s] // page))]
        assert sorted(held + list(free[:count])) == list(range(pages))
        assert cu[-1] == new.sum() and (slots[:cu[-1]] >= 0).all() and (slots[cu[-1]:] == -1).all()
        assert len(set(slots[:cu[-1]])) == cu[-1]
