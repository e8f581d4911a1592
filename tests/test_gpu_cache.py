"""GPU parity of the operators around the paged cache against the 64-bit plain forms of
tests/cache_ref.py: the plan of a step (equal), norm and rotation with their gradients, rows in
4 bits (equal, byte for byte), decode over them, and a serving step that runs them together.

Tolerances count roundings: bf16 outputs 2^-8 of the value; fp32 sums of D squares or products
are off by at most D * 2^-24 <= 2^-17 of their terms, so norm and rotation get 2^-16 of the size
of the terms an element is the sum of; decode's are derived in cache_ref.decode_kv4.
"""
import numpy as np
import pytest

import gqa_inputs as gi
from tests import cache_ref as ref
from tests.gpu_util import assert_parity, bits_of, from_dev, to_dev, torch_mod

pytestmark = pytest.mark.gpu

NAN_BITS = np.uint16(0x7FC0)
STEP = 2.0 ** -8


@pytest.fixture(scope="module")
def gqa():
    torch_mod()
    import grouped_query_softmax_b200 as m
    return m


def _sync_ok(gqa):
    torch_mod().cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_OK


def _i32(x):
    return torch_mod().tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _near(got, want, tol, what):
    err = np.abs(np.asarray(got, np.float64) - want)
    assert np.isfinite(got).all(), f"{what}: non-finite"
    worst = np.unravel_index(np.argmax(err - tol), err.shape) if err.size else None
    assert (err <= tol).all(), f"{what}: {err[worst]:.3e} over {tol[worst]:.3e} at {worst}"


# ---------------------------------------------------------------- plan
def _plan_inputs(S, held, max_pages, page, spare, seed):
    pages_of = lambda n: -(-n // page)
    used = int(sum(pages_of(int(h)) for h in held))
    order = gi.permutation(seed, gi.STREAM_PAGES, used + spare).astype(np.int32)
    table = np.full((S, max_pages), -7, np.int32)
    at = 0
    for s, h in enumerate(held):
        n = pages_of(int(h))
        table[s, :n] = order[at:at + n]
        at += n
    free = np.full(used + spare, -9, np.int32)
    free[:spare] = order[used:]
    return table, free, spare, used + spare


PLANS = [
    # requests, longest held, longest new, page, roll back or end every n-th, padding tokens
    (1, 1, 1, 16, 0, 0), (1, 0, 5, 64, 0, 3), (3, 100, 70, 16, 2, 1), (64, 4096, 1, 64, 0, 5), (37, 300, 130, 32, 3, 0),
    (1000, 200, 20, 16, 4, 7), (1025, 64, 40, 128, 5, 2), (8192, 40, 9, 16, 3, 1), (5, 3000, 2500, 256, 2, 6),
]


@pytest.mark.parametrize("case", PLANS, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches(gqa, case, in_place):
    S, hi, new_hi, page, every, pad = case
    held = gi.uniform_ints(11, gi.STREAM_LEN, S, 0, hi)
    new = gi.uniform_ints(12, gi.STREAM_LEN, S, 0, new_hi)
    keep = held.copy()
    if every:
        keep[::every] = gi.uniform_ints(13, gi.STREAM_LEN, S, 0, hi)[::every] % (held[::every] + 1)
        keep[1::2 * every], new[1::2 * every] = 0, 0
    max_pages = -(-int(max((keep + new).max(), held.max(), 1)) // page)
    spare = int(sum(-(-int(k + n) // page) for k, n in zip(keep, new))) + 3
    table, free, count, pages = _plan_inputs(S, held, max_pages, page, spare, 14)
    tokens = int(new.sum()) + pad + (1 if new.sum() + pad == 0 else 0)
    want = ref.plan(held, keep, new, table, free, count, page, pages, tokens)
    td, fd, hd, cd = _i32(table), _i32(free), _i32(held), _i32([count])
    out = None
    if in_place:
        torch = torch_mod()
        e = lambda n: torch.full((n,), -3, dtype=torch.int32, device="cuda")
        out = gqa.PagedPlan(hd, e(S + 1), e(tokens), e(tokens), cd)
    p = gqa.paged_plan(hd, _i32(new), td, fd, cd, page_size=page, num_pages=pages, max_tokens=tokens,
                       keep=_i32(keep) if every else None, out=out)
    _sync_ok(gqa)
    after, cu, pos, slots, t2, f2, c2 = want
    for got, w, n in ((p.seqlens_k, after, "lengths"), (p.cu_seqlens, cu, "cu"), (p.positions, pos, "positions"),
                      (p.slots, slots, "slots"), (td, t2, "table"), (p.free_count, [c2], "count")):
        np.testing.assert_array_equal(got.cpu().numpy(), w, err_msg=n)
    np.testing.assert_array_equal(fd.cpu().numpy()[:c2], f2[:c2], err_msg="free list")
    if not in_place:
        np.testing.assert_array_equal(hd.cpu().numpy(), held)
        assert int(cd) == count


@pytest.mark.parametrize("what", ["pages", "tokens", "keep", "held", "new", "capacity", "count"])
def test_plan_refuses_and_changes_nothing(gqa, what):
    S, page, max_pages = 4, 16, 6
    held, keep, new = np.array([20, 33, 0, 90]), np.array([20, 33, 0, 90]), np.array([10, 3, 40, 5])
    table, free, count, pages = _plan_inputs(S, held, max_pages, page, 4, 15)
    tokens = 60
    if what == "pages":
        count = 2        # three are needed, all by request 2
    elif what == "tokens":
        tokens = 57
    elif what == "keep":
        keep = np.array([20, 34, 0, 90])
    elif what == "held":
        held = keep = np.array([20, 33, -1, 90])
    elif what == "new":
        new = np.array([10, -3, 40, 5])
    elif what == "capacity":
        new = np.array([10, 3, 40, 7])
    else:
        count = -1
    assert ref.plan(held, keep, new, table, free, count, page, pages, tokens) is None
    td, fd, cd = _i32(table), _i32(free), _i32([count])
    p = gqa.paged_plan(_i32(held), _i32(new), td, fd, cd, page_size=page, num_pages=pages, max_tokens=tokens, keep=_i32(keep))
    torch_mod().cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_ERR_INVALID_ARGUMENT
    np.testing.assert_array_equal(td.cpu().numpy(), table)
    np.testing.assert_array_equal(fd.cpu().numpy(), free)
    np.testing.assert_array_equal(p.seqlens_k.cpu().numpy(), held)
    assert int(p.free_count) == count and (p.cu_seqlens == 0).all() and (p.slots == -1).all() and (p.positions == 0).all()


def test_plan_full_free_list_is_refused(gqa):
    """Pages given back that do not fit the list: nothing changes."""
    table, free, count, pages = _plan_inputs(2, np.array([40, 40]), 3, 16, 2, 16)
    td, fd = _i32(table), _i32(free[:3])   # room for one more, six come back
    p = gqa.paged_plan(_i32([40, 40]), _i32([0, 0]), td, fd, _i32([count]), page_size=16, num_pages=pages, max_tokens=4,
                       keep=_i32([0, 0]))
    torch_mod().cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_ERR_INVALID_ARGUMENT
    assert int(p.free_count) == count and (fd.cpu().numpy() == free[:3]).all()


# ---------------------------------------------------------------- norm and rotation
ROPE = [
    # B, T, Hq, Hkv, D, rot (0: none), interleaved, weights, fp32 weights
    (1, 1, 4, 2, 64, 64, False, True, False), (2, 37, 6, 2, 64, 32, True, True, False), (1, 130, 8, 8, 128, 128, False, True, True),
    (3, 5, 32, 1, 128, 64, False, False, False), (2, 19, 7, 7, 128, 8, True, True, False), (1, 64, 4, 4, 64, 0, False, True, False),
    (1, 33, 16, 4, 64, 8, False, True, True), (2, 300, 32, 8, 128, 128, True, True, False), (1, 3, 9, 3, 128, 104, False, True, False),
    (1, 2, 2, 2, 64, 0, False, False, False),
]


def _rope_inputs(case, seed):
    """(q, k bits [B, H, T, D] cut from one [B, T, heads, D] projection, weights, cos, sin, positions)."""
    B, T, Hq, Hkv, D, rot, inter, weighted, fp32 = case
    qkv = gi.normal_bf16(seed, gi.TENSOR_Q, (B, T, Hq + 2 * Hkv, D))
    w = {}
    rng = np.random.default_rng(seed)
    for n in ("q_weight", "k_weight"):
        v = (1 + 0.3 * rng.normal(size=D)).astype(np.float32)
        w[n] = (v if fp32 else gi.bf16_bits_to_f32(ref.bf16_bits(v))) if weighted else None
    cos, sin = ref.angles(T + 50, rot) if rot else (None, None)
    pos = rng.integers(0, T + 50, size=(B, T)).astype(np.int32) if rot else None
    return qkv, w, cos, sin, pos


def _dev_weights(w, fp32):
    torch = torch_mod()
    up = lambda v: None if v is None else torch.tensor(v, device="cuda").to(torch.float32 if fp32 else torch.bfloat16)
    return {n: up(v) for n, v in w.items()}


def _dev(x):
    return None if x is None else torch_mod().tensor(x, device="cuda")


def _at(cos, sin, pos):
    """Tables at [B, 1, T, rot/2], in 64 bits."""
    return (None, None) if cos is None else (cos[pos][:, None].astype(np.float64), sin[pos][:, None].astype(np.float64))


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_norm_rope_matches(gqa, case):
    B, T, Hq, Hkv, D, rot, inter, weighted, fp32 = case
    qkv, w, cos, sin, pos = _rope_inputs(case, 21)
    d = to_dev(qkv).transpose(1, 2)
    how = dict(_dev_weights(w, fp32), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos), interleaved=inter, eps=1e-5)
    q, k = gqa.qk_norm_rope(d[:, :Hq], d[:, Hq:Hq + Hkv], **how)
    _sync_ok(gqa)
    x = ref.f64(qkv).transpose(0, 2, 1, 3)
    c, s = _at(cos, sin, pos)
    for got, lo, hi, n in ((q, 0, Hq, "q_weight"), (k, Hq, Hq + Hkv, "k_weight")):
        want, size = ref.norm_rope(x[:, lo:hi], w[n], 1e-5, c, s, inter)
        _near(from_dev(got), want, STEP * np.abs(want) + 2.0 ** -16 * size, n)
    # in place: the same bits, and the values between them untouched
    before = bits_of(d[:, Hq + Hkv:])
    gqa.qk_norm_rope(d[:, :Hq], d[:, Hq:Hq + Hkv], q_out=d[:, :Hq], k_out=d[:, Hq:Hq + Hkv], **how)
    _sync_ok(gqa)
    np.testing.assert_array_equal(bits_of(d[:, :Hq]), bits_of(q))
    np.testing.assert_array_equal(bits_of(d[:, Hq:Hq + Hkv]), bits_of(k))
    np.testing.assert_array_equal(bits_of(d[:, Hq + Hkv:]), before)


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_norm_rope_backward_matches(gqa, case):
    B, T, Hq, Hkv, D, rot, inter, weighted, fp32 = case
    qkv, w, cos, sin, pos = _rope_inputs(case, 22)
    dq = gi.normal_bf16(23, gi.TENSOR_DO, (B, Hq, T, D))
    dk = gi.normal_bf16(24, gi.TENSOR_DO, (B, Hkv, T, D))
    d = to_dev(qkv).transpose(1, 2)
    how = dict(_dev_weights(w, fp32), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos), interleaved=inter, eps=1e-5)
    args = (to_dev(dq), to_dev(dk), d[:, :Hq], d[:, Hq:Hq + Hkv])
    got = gqa.qk_norm_rope_bwd(*args, **how)
    again = gqa.qk_norm_rope_bwd(*args, **how)
    _sync_ok(gqa)
    x = ref.f64(qkv).transpose(0, 2, 1, 3)
    c, s = _at(cos, sin, pos)
    for i, (dz, lo, hi, n) in enumerate(((dq, 0, Hq, "q_weight"), (dk, Hq, Hq + Hkv, "k_weight"))):
        dx, dw, size, wsize = ref.norm_rope_bwd(ref.f64(dz), x[:, lo:hi], w[n], 1e-5, c, s, inter)
        _near(from_dev(got[i]), dx, STEP * np.abs(dx) + 2.0 ** -16 * size, n)
        np.testing.assert_array_equal(bits_of(got[i]), bits_of(again[i]))
        if weighted:
            # a chain of at most a few hundred fp32 additions, each 2^-24, after terms within 2^-16
            _near(got[2 + i].cpu().numpy(), dw, 2.0 ** -15 * wsize, "gradient of " + n)
            assert torch_mod().equal(got[2 + i], again[2 + i])
        else:
            assert got[2 + i] is None
    # in place over the gradients
    a, b = args[0].clone(), args[1].clone()
    gqa.qk_norm_rope_bwd(a, b, *args[2:], dq=a, dk=b, **how)
    _sync_ok(gqa)
    np.testing.assert_array_equal(bits_of(a), bits_of(got[0]))
    np.testing.assert_array_equal(bits_of(b), bits_of(got[1]))


def test_norm_rope_gradient_matches_differences_of_the_kernel(gqa):
    """<dz, f(x + h e)> - <dz, f(x - h e)> over a direction e, on the device's own forward."""
    torch = torch_mod()
    case = (2, 64, 8, 2, 128, 128, False, True, True)
    qkv, w, cos, sin, pos = _rope_inputs(case, 25)
    how = dict(_dev_weights(w, True), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos))
    d = to_dev(qkv).transpose(1, 2)
    q, k = d[:, :8].contiguous(), d[:, 8:10].contiguous()
    dq, dk = to_dev(gi.normal_bf16(26, gi.TENSOR_DO, (2, 8, 64, 128))), to_dev(gi.normal_bf16(27, gi.TENSOR_DO, (2, 2, 64, 128)))
    gq, gk, gwq, gwk = gqa.qk_norm_rope_bwd(dq, dk, q, k, **how)
    # weights: f is linear in them, so a large step is exact but for the outputs' rounding
    h = 2.0
    for name, g, i, dz in (("q_weight", gwq, 0, dq), ("k_weight", gwk, 1, dk)):
        e = torch.zeros(128, device="cuda")
        e[17] = h
        up = gqa.qk_norm_rope(q, k, **dict(how, **{name: how[name] + e}))[i].double()
        down = gqa.qk_norm_rope(q, k, **dict(how, **{name: how[name] - e}))[i].double()
        terms = (up - down) * dz.double() / (2 * h)
        # each output is off by at most half a step
        tol = (STEP * (up.abs() + down.abs()) * dz.double().abs()).sum() / (2 * h)
        assert abs(float(terms.sum()) - float(g[17])) <= float(tol)
    _sync_ok(gqa)


def test_norm_rope_bad_positions_leave_their_rows(gqa):
    torch = torch_mod()
    q, k = to_dev(gi.normal_bf16(28, 0, (1, 4, 6, 64))), to_dev(gi.normal_bf16(29, 1, (1, 2, 6, 64)))
    q[:, :, 4], k[:, :, 1] = float("nan"), float("inf")   # rows at bad positions: no part in any gradient
    cos, sin = ref.angles(10, 64)
    how = dict(cos=_dev(cos), sin=_dev(sin), q_weight=torch.ones(64, device="cuda"), k_weight=torch.ones(64, device="cuda"))
    good = gqa.qk_norm_rope(q, k, positions=_i32([0, 1, 2, 3, 4, 5]), **how)
    want = gqa.qk_norm_rope_bwd(q[:, :, [0, 2, 3, 5]], k[:, :, [0, 2, 3, 5]], q[:, :, [0, 2, 3, 5]], k[:, :, [0, 2, 3, 5]],
                                positions=_i32([0, 2, 3, 5]), **how)
    _sync_ok(gqa)
    qo, ko = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    bad = _i32([0, -1, 2, 3, 10, 5])
    gqa.qk_norm_rope(q, k, positions=bad, q_out=qo, k_out=ko, **how)
    torch.cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_ERR_INVALID_ARGUMENT
    for got, w in ((qo, good[0]), (ko, good[1])):
        assert torch.equal(got[:, :, [0, 2, 3, 5]], w[:, :, [0, 2, 3, 5]]) and (got[:, :, [1, 4]] == 3).all()
    dq, dk = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    got = gqa.qk_norm_rope_bwd(q, k, q, k, positions=bad, dq=dq, dk=dk, **how)
    torch.cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_ERR_INVALID_ARGUMENT
    assert (dq[:, :, [1, 4]] == 3).all() and torch.equal(dq[:, :, [0, 2, 3, 5]], want[0])
    assert torch.allclose(got[2], want[2], rtol=0, atol=1e-4) and torch.allclose(got[3], want[3], rtol=0, atol=1e-4)


APPEND = [(1, 4, 2, 64, 64, False, 16, "NHD"), (37, 32, 8, 128, 128, False, 64, "NHD"), (130, 6, 6, 64, 16, True, 32, "HND"),
          (2000, 8, 1, 128, 64, False, 128, "HND")]


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append_writes_the_rows_of_its_slots(gqa, case):
    torch = torch_mod()
    N, Hq, Hkv, D, rot, inter, page, layout = case
    qkv, w, cos, sin, pos = _rope_inputs((1, N, Hq, Hkv, D, rot, inter, True, False), 31)
    pages = -(-N // page) + 2
    slots = gi.permutation(32, gi.STREAM_PAGES, pages * page)[:N].astype(np.int32)
    slots[N // 2::7] = -1
    shape = (pages, page, Hkv, D) if layout == "NHD" else (pages, Hkv, page, D)
    pools = [torch.full(shape, 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    d = to_dev(qkv)[0]
    how = dict(_dev_weights(w, False), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos[0]), interleaved=inter)
    q = gqa.qk_norm_rope_append(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], *pools, _i32(slots), pool_layout=layout, **how)
    plain = gqa.qk_norm_rope(d[None, :, :Hq].transpose(1, 2), d[None, :, Hq:Hq + Hkv].transpose(1, 2), **how)
    _sync_ok(gqa)
    assert torch.equal(q, plain[0][0].transpose(0, 1))
    keys, values = plain[1][0].transpose(0, 1), d[:, Hq + Hkv:]
    ok = slots >= 0
    for pool, rows in zip(pools, (keys, values)):
        flat = (pool if layout == "NHD" else pool.transpose(1, 2)).reshape(-1, Hkv, D)
        want = torch.full_like(flat, 9.0)
        want[torch.tensor(slots[ok], device="cuda").long()] = rows[torch.tensor(ok, device="cuda")]
        assert torch.equal(flat, want)


def test_append_and_rows_report_slots_past_the_pool(gqa):
    torch = torch_mod()
    x = to_dev(gi.normal_bf16(33, 0, (3, 2, 64)))
    slots = _i32([0, 5 * 16, 7])
    pools = [torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gqa.qk_norm_rope_append(x, x, x, *pools, slots)
    torch.cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_ERR_INVALID_ARGUMENT
    assert torch.equal(pools[1][0, 7], x[2]) and int((pools[1] != 0).any(-1).any(-1).sum()) == 2
    p4 = [gqa.kv4_pool(5, 2, 16, 64) for _ in range(2)]
    gqa.kv4_append(x, x, *p4, slots)
    torch.cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_ERR_INVALID_ARGUMENT
    k, v = gqa.kv4_gather(*p4, slots)
    torch.cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_ERR_INVALID_ARGUMENT
    assert (k[1] == 0).all() and (k[0] != 0).any() and torch.equal(k, v)


# ---------------------------------------------------------------- rows in 4 bits
KV4 = [(1, 1, 64, 16), (37, 8, 128, 64), (500, 3, 64, 32), (1000, 1, 128, 128), (4097, 2, 128, 256)]


def _hard_rows(x):
    """Rows that quantising can get wrong, in place."""
    n = x.shape[0]
    x[n // 3] = 0x3FC0                                    # constant
    x[n // 4] = 0
    if n > 20:
        x[5, 0, 3], x[6, 0, 0], x[7, 0, -1] = 0x7F80, 0x7FC0, 0xFF80   # infinity, NaN, -infinity
        x[8, 0, :2] = 0x7F7F, 0xFF7F                      # max - min past fp32
        x[9, 0] = 0x0001                                   # a step below 2^-126
        x[9, 0, 0] = 0x0003
        x[10, 0] = np.where(np.arange(x.shape[-1]) % 2, 0x4170, 0x0000)  # codes on both ends: 15 and 0
        x[11, 0, 0], x[11, 0, 1] = 0x3F80, 0x3400         # far exponents
    return x


@pytest.mark.parametrize("case", KV4, ids=str)
def test_kv4_rows_are_byte_for_byte(gqa, case):
    torch = torch_mod()
    N, H, D, page = case
    k, v = _hard_rows(gi.normal_bf16(41, 1, (N, H, D))), _hard_rows(gi.normal_bf16(42, 2, (N, H, D)))
    pages = -(-N // page) + 2
    slots = gi.permutation(43, gi.STREAM_PAGES, pages * page)[:N].astype(np.int32)
    slots[N // 2::5] = -1
    pools = [torch.full((pages, H, page, D // 2 + 4), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(2)]
    # token-major k beside head-major v: strides of their own
    vd = to_dev(np.ascontiguousarray(v.transpose(1, 0, 2))).transpose(0, 1)
    gqa.kv4_append(to_dev(k), vd, *pools, _i32(slots))
    back = gqa.kv4_gather(*pools, _i32(slots))
    _sync_ok(gqa)
    ok = slots >= 0
    for pool, x, b in zip(pools, (k, v), back):
        rows, bad = ref.kv4_pack(x)
        got = pool.cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, H, D // 2 + 4)
        want = np.full_like(got, 0xAB)
        want[slots[ok]] = rows[ok]
        is_bad = np.zeros(got.shape[:2], bool)
        is_bad[slots[ok]] = bad[ok]
        np.testing.assert_array_equal(got[~is_bad], want[~is_bad])
        np.testing.assert_array_equal(got[is_bad][:, -4:], want[is_bad][:, -4:])  # NaN rows: codes do not matter
        vals = gi.bf16_bits_to_f32(ref.bf16_bits(ref.kv4_values(rows).astype(np.float32)))
        vals = vals.reshape(x.shape)
        vals[~ok] = 0
        np.testing.assert_array_equal(from_dev(b), vals)


# ---------------------------------------------------------------- decode over 4-bit rows
DECODE = [
    # Hq, Hkv, Tq, lengths, D, window, page
    (8, 2, 1, [1], 128, 0, 16), (4, 4, 1, [31, 32, 33], 64, 0, 16), (32, 8, 1, [4099], 128, 0, 64),
    (8, 2, 1, [0, 5, 0, 700], 128, 0, 32), (16, 4, 4, [3, 100, 2, 1025], 64, 0, 16), (16, 2, 1, [257, 2000], 128, 0, 128),
    (12, 2, 3, [40, 999, 16], 64, 100, 32), (32, 1, 1, [130, 1, 2500], 128, 0, 64), (6, 2, 16, [16, 17, 300], 128, 0, 256),
    (8, 1, 16, [15, 640], 64, 33, 128), (32, 8, 1, [5000, 64, 3333, 1], 128, 1000, 64), (8, 8, 2, [700, 4, 2048], 128, 1, 16),
    (4, 1, 16, [1000, 33], 128, 0, 384), (8, 2, 1, [100] * 300, 64, 0, 16),
    # more units than clusters fit at once: runs of tiles that cut units, and the merge; a long
    # sequence in many pieces among short ones
    (32, 8, 1, [(37 * i) % 700 for i in range(44)], 128, 0, 32), (32, 2, 1, [(91 * i) % 300 for i in range(160)], 128, 0, 64),
    (32, 1, 1, [(53 * i) % 200 for i in range(155)], 128, 90, 16), (8, 1, 4, [(29 * i) % 150 for i in range(160)], 64, 0, 128),
    (16, 2, 2, [7000] + [i % 60 for i in range(170)], 64, 0, 64), (4, 4, 1, [0] * 60 + [9000] + [0, 3] * 30, 128, 0, 16),
    (8, 1, 1, [1, 2500] * 160, 64, 2000, 32),
]


def _kv4_pools(lens, Hkv, D, page, seed, window=0, Tq=1):
    """Random rows in shuffled pages; bytes of no visible row are 0xFF (steps and minima NaN), table
    entries of pages that no query sees are -1 or far outside the pool."""
    n_pages = [-(-int(n) // page) for n in lens]
    total = sum(n_pages) + 3
    order = gi.permutation(seed, gi.STREAM_PAGES, total)
    pools = [np.full((total, Hkv, page, D // 2 + 4), 0xFF, np.uint8) for _ in range(2)]
    table = np.full((len(lens), max(n_pages + [1]) + 2), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(lens):
        if n == 0:
            continue
        rows = order[at:at + n_pages[b]]
        at += n_pages[b]
        table[b, :n_pages[b]] = rows
        lo = max(0, n - Tq - window + 1) if window else 0
        table[b, :lo // page] = -1
        t = np.arange(lo, n)
        for i, pool in enumerate(pools):
            x = gi.normal_bf16(seed + 1 + i, 1 + i, (n - lo, Hkv, D), start=b * 1000003)
            pool[rows[t // page], :, t % page] = ref.kv4_pack(x)[0]
    return pools[0], pools[1], table


@pytest.mark.parametrize("case", DECODE, ids=lambda c: str(c[:3] + (c[3][:4],) + c[4:]))
def test_decode_kv4_matches(gqa, case):
    torch = torch_mod()
    Hq, Hkv, Tq, lens, D, window, page = case
    kp, vp, table = _kv4_pools(lens, Hkv, D, page, 51, window, Tq)
    q = gi.normal_bf16(52, gi.TENSOR_Q, (len(lens), Hq, Tq, D))
    want, tol = ref.decode_kv4(q, kp, vp, lens, table, window)
    args = (to_dev(q), _dev(kp), _dev(vp), _i32(lens), _i32(table))
    o = gqa.attn_decode_kv4(*args, window=window, out=torch.full_like(args[0], float("nan")))
    again = gqa.attn_decode_kv4(*args, window=window, max_seqlen_k=max(max(lens), 1))
    _sync_ok(gqa)
    _near(from_dev(o), want, tol, str(case))
    _near(from_dev(again), want, tol, "with the longest length given")
    third = gqa.attn_decode_kv4(*args, window=window)
    np.testing.assert_array_equal(bits_of(third), bits_of(o))  # whatever the order in which CTAs run


def test_decode_kv4_strided_pools_scale_and_bad_pages(gqa):
    """Pools that are slices of a larger one; a page number outside the pool reads as zeros."""
    torch = torch_mod()
    lens, Hq, Hkv, D, page = [200, 90], 8, 2, 128, 32
    kp, vp, table = _kv4_pools(lens, Hkv, D, page, 53)
    q = gi.normal_bf16(54, gi.TENSOR_Q, (2, Hq, D))
    table[0, 3], table[1, 0] = -1, kp.shape[0]
    big = torch.full((kp.shape[0], 3, 2, Hkv, page, 68), 0xFF, dtype=torch.uint8, device="cuda")
    big[:, 1, 0], big[:, 1, 1] = _dev(kp), _dev(vp)
    o = gqa.attn_decode_kv4(to_dev(q), big[:, 1, 0], big[:, 1, 1], _i32(lens), _i32(table), scale=0.3)
    _sync_ok(gqa)
    want, tol = ref.decode_kv4(q[:, :, None], kp, vp, lens, table, scale=0.3)
    _near(from_dev(o), want[:, :, 0], 2 * tol[:, :, 0], "strided")   # scale 0.3: the scores' error is 3.4 times as large


@pytest.mark.parametrize("extra", [0, 230])
def test_decode_kv4_lengths_outside_their_range(gqa, extra):
    """Beside valid sequences, few (a cluster each) and many (runs of tiles)."""
    torch = torch_mod()
    lens, Hq, Hkv, D, page = [200, 90, 64] + [33] * extra, 8, 2, 64, 16
    kp, vp, table = _kv4_pools(lens, Hkv, D, page, 55)
    q = gi.normal_bf16(56, gi.TENSOR_Q, (len(lens), Hq, 1, D))
    want, tol = ref.decode_kv4(q, kp, vp, lens, table)
    others = [0] + list(range(2, len(lens)))
    for bad in (-1, 201):
        out = torch.full((len(lens), Hq, 1, D), 5.0, dtype=torch.bfloat16, device="cuda")
        gqa.attn_decode_kv4(to_dev(q), _dev(kp), _dev(vp), _i32([200, bad] + lens[2:]), _i32(table), max_seqlen_k=200, out=out)
        torch.cuda.synchronize()
        assert gqa.gqa_get_device_error() == gqa.GQA_ERR_INVALID_ARGUMENT
        got = from_dev(out)
        assert (got[1] == 5).all()
        _near(got[others], want[others], tol[others], "beside a bad length")


def test_decode_kv4_nan_stays_with_the_queries_that_see_it(gqa):
    lens, Hq, Hkv, D, page, Tq = [500], 4, 2, 64, 16, 4
    kp, vp, table = _kv4_pools(lens, Hkv, D, page, 57)
    vp[table[0, 498 // page], 0, 498 % page, -4:] = 0xFF    # value row of key 498, KV head 0
    kp[table[0, 499 // page], 1, 499 % page, -4:] = 0xFF    # key 499, KV head 1
    q = gi.normal_bf16(58, gi.TENSOR_Q, (1, Hq, Tq, D))
    got = from_dev(gqa.attn_decode_kv4(to_dev(q), _dev(kp), _dev(vp), _i32(lens), _i32(table)))
    _sync_ok(gqa)
    bad = np.isnan(got).all(-1)[0]
    assert bad[:2].tolist() == [[False, False, True, True]] * 2 and bad[2:].tolist() == [[False, False, False, True]] * 2
    assert np.isfinite(got[0][~bad]).all()


def test_offsets_past_32_bits(gqa):
    """Pools of more than 2^32 bytes (4-bit rows) and 2^31 elements (bf16): rows on the last pages."""
    torch = torch_mod()
    Hkv, D, page, N = 8, 128, 64, 200
    pages = (1 << 32) // (Hkv * page * 68) + 40
    slots = (pages - 1 - np.arange(N) // page) * page + np.arange(N) % page
    k, v = gi.normal_bf16(91, 1, (N, Hkv, D)), gi.normal_bf16(92, 2, (N, Hkv, D))
    pools = [torch.empty((pages, Hkv, page, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
    gqa.kv4_append(to_dev(k), to_dev(v), *pools, _i32(slots))
    back = gqa.kv4_gather(*pools, _i32(slots))
    lens, table = [N], np.array([[pages - 1 - i for i in range(4)]])
    q = gi.normal_bf16(93, 0, (1, 32, D))
    o = gqa.attn_decode_kv4(to_dev(q), *pools, _i32(lens), _i32(table))
    _sync_ok(gqa)
    for b, x in zip(back, (k, v)):
        want = gi.bf16_bits_to_f32(ref.bf16_bits(ref.kv4_values(ref.kv4_pack(x)[0]).astype(np.float32)))
        np.testing.assert_array_equal(from_dev(b), want.reshape(x.shape))
    tail = [p[-4:].cpu().numpy() for p in pools]
    want, tol = ref.decode_kv4(q[:, :, None], *tail, lens, table - (pages - 4))
    _near(from_dev(o), want[:, :, 0], tol[:, :, 0], "last pages")
    del pools
    pages = (1 << 31) // (Hkv * page * D) + 10
    pool = torch.empty((2, pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    slots = (pages - 1 - np.arange(N) // page) * page + np.arange(N) % page
    kd, vd = to_dev(k), to_dev(v)
    got = gqa.qk_norm_rope_append(kd, kd, vd, pool[0], pool[1], _i32(slots))
    _sync_ok(gqa)
    at = torch.tensor(slots, device="cuda")
    assert torch.equal(got, kd)
    assert torch.equal(pool[0][at // page, at % page], kd) and torch.equal(pool[1][at // page, at % page], vd)


# ---------------------------------------------------------------- together
def _pool_rows(pool, table, lens):
    """[B] lists of [L, H, D] rows of an NHD pool."""
    page = pool.shape[1]
    return [pool[table[b, np.arange(n) // page], np.arange(n) % page] for b, n in enumerate(lens)]


@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_from_lengths(gqa, captured):
    """Three steps of four requests (a ragged prefill, a decode step, a step behind a rejected draft
    with one request finished): plan, norm and rotation into the pages, attention over them, in
    bf16 and in 4 bits. The captured form replays one graph per step shape with lengths and tokens
    changed in place; two captures share no workspace."""
    torch = torch_mod()
    import oracle
    Hq, Hkv, D, page, S, pages, max_pages, tokens = 8, 2, 128, 16, 4, 60, 12, 40
    cos, sin = ref.angles(max_pages * page, D)
    w = [(1 + 0.2 * np.random.default_rng(i).normal(size=D)).astype(np.float32) for i in (1, 2)]
    how = dict(q_weight=_dev(w[0]), k_weight=_dev(w[1]), cos=_dev(cos), sin=_dev(sin))
    free = _i32(gi.permutation(61, gi.STREAM_PAGES, pages))
    table = torch.full((S, max_pages), -1, dtype=torch.int32, device="cuda")
    count, lens, keep, new = _i32([pages]), _i32([0] * S), _i32([0] * S), _i32([0] * S)
    pools = [torch.full((pages, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pools4 = [torch.full((pages, Hkv, page, D // 2 + 4), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    qkv = torch.zeros(tokens, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    e = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    p = gqa.PagedPlan(lens, e(S + 1), e(tokens), e(tokens), count)
    q_in, k_in, v_in = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    kept = {}

    def step():
        gqa.paged_plan(lens, new, table, free, count, page_size=page, num_pages=pages, max_tokens=tokens, keep=keep, out=p)
        q = gqa.qk_norm_rope_append(q_in, k_in, v_in, *pools, p.slots, positions=p.positions, **how)
        k = gqa.qk_norm_rope(q_in[None].transpose(1, 2), k_in[None].transpose(1, 2), positions=p.positions, **how)[1]
        gqa.kv4_append(k[0].transpose(0, 1), v_in, *pools4, p.slots)
        kept["q"] = q
        kept["o"] = gqa.attn_fwd_varlen(q, *pools, cu_seqlens_q=p.cu_seqlens, seqlens_k=p.seqlens_k, block_table=table,
                                        max_seqlen_q=tokens)
        last = (p.cu_seqlens[1:] - 1).clamp(min=0).long()
        kept["o4"] = gqa.attn_decode_kv4(q[last].contiguous(), *pools4, p.seqlens_k, table)
        kept["k4"], kept["v4"] = gqa.kv4_gather(*pools4, p.slots)

    run = step
    if captured:
        state = (lens, table, free, count)
        saved = [t.clone() for t in state]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, s in zip(state, saved):
            t.copy_(s)
        run = graph.replay
    have = [0] * S
    rng = np.random.default_rng(62)
    for n, (kp, nw) in enumerate([([0] * 4, [13, 1, 0, 22]), (None, [1, 1, 1, 1]), ([12, 0, 1, 23], [2, 0, 4, 1])]):
        kp = have if kp is None else kp
        keep.copy_(_i32(kp))
        new.copy_(_i32(nw))
        qkv.copy_(to_dev(gi.normal_bf16(63 + n, 0, tuple(qkv.shape))))
        run()
        _sync_ok(gqa)
        have = [a + b for a, b in zip(kp, nw)]
        assert lens.tolist() == have and int(count) == pages - sum(-(-h // page) for h in have)
        t = table.cpu().numpy()
        live = sum(nw)
        # the cache holds these tokens' rows; attention over it against the oracle
        cu = np.concatenate([[0], np.cumsum(nw)])
        rows_k, rows_v = (_pool_rows(bits_of(x).reshape(x.shape), t, have) for x in pools)
        q_bits = bits_of(kept["q"]).reshape(tokens, Hq, D)
        x = ref.f64(bits_of(qkv).reshape(qkv.shape))
        o, o4 = from_dev(kept["o"]), from_dev(kept["o4"])
        pos = np.concatenate([np.arange(k, h) for k, h in zip(kp, have)]).astype(int)
        c, s = cos[pos][:, None].astype(np.float64), sin[pos][:, None].astype(np.float64)
        for got, lo, hi, wt in ((ref.f64(q_bits)[:live], 0, Hq, w[0]),
                                (ref.f64(np.concatenate([r[k:] for r, k in zip(rows_k, kp)])), Hq, Hq + Hkv, w[1])):
            z, size = ref.norm_rope(x[:live, lo:hi], wt, 1e-6, c, s, False)
            _near(got, z, STEP * np.abs(z) + 2.0 ** -16 * size, "rows in the cache")
        np.testing.assert_array_equal(np.concatenate([r[k:] for r, k in zip(rows_v, kp)]),
                                      bits_of(qkv).reshape(qkv.shape)[:live, Hq + Hkv:])
        for b in range(S):
            if nw[b] == 0:
                continue
            qb, kb, vb = (r.transpose(1, 0, 2)[None].copy(order="C")
                          for r in (q_bits[cu[b]:cu[b + 1]], rows_k[b], rows_v[b]))
            want = oracle.attention(qb, kb, vb)[0].transpose(1, 0, 2)
            assert_parity(o[cu[b]:cu[b + 1]], want, f"step {n} request {b}")
        last = np.maximum(cu[1:] - 1, 0)
        want, tol = ref.decode_kv4(q_bits[last][:, :, None], pools4[0].cpu().numpy(), pools4[1].cpu().numpy(), have, t)
        _near(o4, want[:, :, 0], tol[:, :, 0], f"4-bit decode of step {n}")


def test_training_step_gradients(gqa):
    """norm and rotation, attention, and both backward passes, against differences in 64 bits."""
    torch = torch_mod()
    import oracle
    B, T, Hq, Hkv, D = 1, 48, 4, 2, 64
    case = (B, T, Hq, Hkv, D, D, False, True, True)
    qkv, w, cos, sin, _ = _rope_inputs(case, 71)
    do = gi.normal_bf16(72, gi.TENSOR_DO, (B, Hq, T, D))
    how = dict(_dev_weights(w, True), cos=_dev(cos), sin=_dev(sin))
    d = to_dev(qkv).transpose(1, 2)
    q0, k0, v0 = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:].contiguous()
    q, k = gqa.qk_norm_rope(q0, k0, **how)
    o, lse = gqa.attn_fwd(q, k, v0, return_lse=True)
    dq, dk, dv = gqa.attn_bwd(q, k, v0, o, to_dev(do), lse)
    got = gqa.qk_norm_rope_bwd(dq, dk, q0, k0, **how)
    _sync_ok(gqa)
    # the formula on the oracle's gradients of the same rotated rows
    rq, rk, _ = oracle.attention_bwd(bits_of(q).reshape(q.shape), bits_of(k).reshape(k.shape), bits_of(v0).reshape(v0.shape), do)
    x = ref.f64(qkv).transpose(0, 2, 1, 3)
    c, s = cos[:T].astype(np.float64), sin[:T].astype(np.float64)
    for i, (dz, lo, hi, n) in enumerate(((rq, 0, Hq, "q_weight"), (rk, Hq, Hq + Hkv, "k_weight"))):
        dx, dw, size, wsize = ref.norm_rope_bwd(dz, x[:, lo:hi], w[n], 1e-6, c, s, False)
        # attn_bwd's own bar is 2^-6 of the largest and 2^-8 of the mean gradient; norm and rotation are linear in it
        err = np.abs(from_dev(got[i]) - dx)
        assert err.max() <= 2.0 ** -5 * np.abs(dx).max() and err.mean() <= 2.0 ** -7 * np.abs(dx).mean()
        assert np.abs(got[2 + i].cpu().numpy() - dw).max() <= 2.0 ** -6 * wsize.max()


@pytest.mark.parametrize("B", [3, 90])
def test_decode_kv4_captured_and_replayed(gqa, B):
    """One graph, lengths and queries changed between replays (a cluster a unit; runs of tiles), beside
    a second graph with a workspace of its own on another stream."""
    torch = torch_mod()
    kp, vp, table = _kv4_pools([400] * B, 4, 64, 32, 85)
    q = torch.zeros(B, 8, 1, 64, dtype=torch.bfloat16, device="cuda")
    lens = _i32([400] * B)
    args = (_dev(kp), _dev(vp), lens, _i32(table))
    graphs = []
    side = torch.cuda.Stream()
    gqa.attn_decode_kv4(q, *args)   # before the capture
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = gqa.attn_decode_kv4(q, *args, max_seqlen_k=400)
        graphs.append((g, out))
    for step in range(3):
        n = gi.uniform_ints(86 + step, gi.STREAM_LEN, B, 0, 400)
        bits = gi.normal_bf16(87 + step, 0, (B, 8, 1, 64))
        lens.copy_(_i32(n))
        q.copy_(to_dev(bits))
        for g, out in graphs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        graphs[1][0].replay()
        _sync_ok(gqa)
        want, tol = ref.decode_kv4(bits, kp, vp, n, table)
        for g, out in graphs:
            _near(from_dev(out), want, tol, f"replay {step}")


def test_two_streams_at_once_and_foreign_operands(gqa):
    torch = torch_mod()
    lens = [3000, 1700]
    kp, vp, table = _kv4_pools(lens, 2, 128, 64, 81)
    qs = [to_dev(gi.normal_bf16(82 + i, 0, (2, 8, 1, 128))) for i in range(2)]
    args = (_dev(kp), _dev(vp), _i32(lens), _i32(table))
    want = [bits_of(gqa.attn_decode_kv4(q, *args)) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append([gqa.attn_decode_kv4(q, *args, stream=s) for q, s in zip(qs, streams)])
    _sync_ok(gqa)
    for pair in outs:
        for o, wt in zip(pair, want):
            np.testing.assert_array_equal(bits_of(o), wt)
    with pytest.raises(TypeError):
        gqa.attn_decode_kv4(qs[0], args[0], args[1], args[2], args[3].cpu())
