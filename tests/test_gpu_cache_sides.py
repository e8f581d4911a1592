"""GPU: the operators around the paged cache on both sides of the rules that choose their launches,
against the 64-bit plain forms: many tokens, heads that do not fill a team's last turn."""
import numpy as np
import pytest

import gqa_inputs as gi
from tests import cache_ref as ref
from tests.gpu_util import bits_of, from_dev, to_dev, torch_mod
from tests.test_gpu_cache import STEP, _at, _dev, _dev_weights, _i32, _near, _plan_inputs, _rope_inputs, _sync_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    torch_mod()
    import grouped_query_softmax_b200 as m
    return m


# B, T, Hq, Hkv, D, rot, interleaved, weights, fp32 weights: sixteen heads a team forward, eight backward
MANY = [(2, 811, 36, 12, 128, 128, False, True, False), (1, 1601, 35, 5, 128, 64, True, True, True),
        (3, 1700, 18, 18, 64, 64, False, True, False), (1, 2500, 20, 20, 128, 32, False, False, False)]


@pytest.mark.parametrize("case", MANY, ids=str)
def test_norm_rope_of_many_tokens(gqa, case):
    B, T, Hq, Hkv, D, rot, inter, weighted, fp32 = case
    qkv, w, cos, sin, pos = _rope_inputs(case, 161)
    dz = [gi.normal_bf16(162 + i, gi.TENSOR_DO, (B, h, T, D)) for i, h in enumerate((Hq, Hkv))]
    d = to_dev(qkv).transpose(1, 2)
    x = (d[:, :Hq], d[:, Hq:Hq + Hkv])
    how = dict(_dev_weights(w, fp32), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos), interleaved=inter, eps=1e-5)
    z = gqa.qk_norm_rope(*x, **how)
    grads = gqa.qk_norm_rope_bwd(to_dev(dz[0]), to_dev(dz[1]), *x, **how)
    _sync_ok(gqa)
    rows = ref.f64(qkv).transpose(0, 2, 1, 3)
    c, s = _at(cos, sin, pos)
    for i, (lo, hi, n) in enumerate(((0, Hq, "q_weight"), (Hq, Hq + Hkv, "k_weight"))):
        want, size = ref.norm_rope(rows[:, lo:hi], w[n], 1e-5, c, s, inter)
        _near(from_dev(z[i]), want, STEP * np.abs(want) + 2.0 ** -16 * size, n)
        dx, dw, size, wsize = ref.norm_rope_bwd(ref.f64(dz[i]), rows[:, lo:hi], w[n], 1e-5, c, s, inter)
        _near(from_dev(grads[i]), dx, STEP * np.abs(dx) + 2.0 ** -16 * size, "gradient under " + n)
        if weighted:  # chains of fp32 additions as long as a CTA's share of the rows, a few hundred
            _near(grads[2 + i].cpu().numpy(), dw, 2.0 ** -15 * wsize, "gradient of " + n)


@pytest.mark.parametrize("N,Hq,Hkv,D,layout", [(1700, 36, 12, 128, "NHD"), (6000, 9, 3, 64, "HND"), (1000, 20, 20, 128, "HND")])
def test_append_of_many_tokens(gqa, N, Hq, Hkv, D, layout):
    torch = torch_mod()
    case = (1, N, Hq, Hkv, D, D, False, True, False)
    qkv, w, cos, sin, pos = _rope_inputs(case, 171)
    d = to_dev(qkv)[0]
    how = dict(_dev_weights(w, False), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos[0]), eps=1e-5)
    pages = N // 32 + 3
    slots = gi.permutation(172, gi.STREAM_PAGES, pages * 32)[:N].astype(np.int32)
    pools = [torch.full((pages, 32, Hkv, D) if layout == "NHD" else (pages, Hkv, 32, D), 9.0, dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    q = gqa.qk_norm_rope_append(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], *pools, _i32(slots), pool_layout=layout, **how)
    _sync_ok(gqa)
    at = torch.tensor(slots, device="cuda").long()
    flat = [(p if layout == "NHD" else p.transpose(1, 2)).reshape(-1, Hkv, D) for p in pools]
    c, s = cos[pos[0]][:, None].astype(np.float64), sin[pos[0]][:, None].astype(np.float64)
    for got, lo, hi, n in ((q, 0, Hq, "q_weight"), (flat[0][at], Hq, Hq + Hkv, "k_weight")):
        want, size = ref.norm_rope(ref.f64(qkv)[0][:, lo:hi], w[n], 1e-5, c, s, False)
        _near(from_dev(got), want, STEP * np.abs(want) + 2.0 ** -16 * size, n)
    np.testing.assert_array_equal(bits_of(flat[1][at]), bits_of(d[:, Hq + Hkv:]))
    rest = torch.ones(len(flat[0]), dtype=torch.bool, device="cuda")
    rest[at] = False
    assert all((f[rest] == 9).all() for f in flat)


@pytest.mark.parametrize("N,H,D", [(4700, 10, 128), (5001, 9, 64), (9500, 3, 64)])
def test_kv4_rows_of_many_tokens(gqa, N, H, D):
    torch = torch_mod()
    x = [gi.normal_bf16(181 + i, 1 + i, (N, H, D)) for i in range(2)]
    pages = N // 64 + 2
    slots = gi.permutation(183, gi.STREAM_PAGES, pages * 64)[:N].astype(np.int32)
    pools = [torch.full((pages, H, 64, D // 2 + 4), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(2)]
    gqa.kv4_append(to_dev(x[0]), to_dev(x[1]), *pools, _i32(slots))
    back = gqa.kv4_gather(*pools, _i32(slots))
    _sync_ok(gqa)
    for pool, bits, b in zip(pools, x, back):
        rows = ref.kv4_pack(bits)[0]
        got = pool.cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, H, D // 2 + 4)
        want = np.full_like(got, 0xAB)
        want[slots] = rows
        np.testing.assert_array_equal(got, want)
        vals = gi.bf16_bits_to_f32(ref.bf16_bits(ref.kv4_values(rows).astype(np.float32))).reshape(bits.shape)
        np.testing.assert_array_equal(from_dev(b), vals)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,per,padding", [(3, 6000, 0), (256, 2100, 13), (200, 60, 400000), (257, 5, 0)])
def test_plan_of_many_tokens(gqa, in_place, S, per, padding):
    """Few requests with more tokens than two rounds of small blocks write, and padding of that size."""
    torch = torch_mod()
    page = 64
    held = gi.uniform_ints(191, gi.STREAM_LEN, S, 0, 300)
    new = gi.uniform_ints(192, gi.STREAM_LEN, S, per // 2, per)
    keep = held.copy()
    keep[::3], new[1::5] = keep[::3] // 2, 0
    max_pages = -(-int((keep + new).max()) // page) + 5
    spare = int(sum(-(-int(k + n) // page) for k, n in zip(keep, new)))
    table, free, count, pages = _plan_inputs(S, held, max_pages, page, spare, 193)
    tokens = int(new.sum()) + padding
    after, cu, pos, slots, t2, f2, c2 = ref.plan(held, keep, new, table, free, count, page, pages, tokens)
    td, fd, hd, cd = _i32(table), _i32(free), _i32(held), _i32([count])
    out = None
    if in_place:
        e = lambda n: torch.full((n,), -3, dtype=torch.int32, device="cuda")
        out = gqa.PagedPlan(hd, e(S + 1), e(tokens), e(tokens), cd)
    p = gqa.paged_plan(hd, _i32(new), td, fd, cd, page_size=page, num_pages=pages, max_tokens=tokens, keep=_i32(keep), out=out)
    _sync_ok(gqa)
    for got, want in ((p.seqlens_k, after), (p.cu_seqlens, cu), (p.positions, pos), (p.slots, slots), (td, t2), (p.free_count, [c2])):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    np.testing.assert_array_equal(fd.cpu().numpy()[:c2], f2[:c2])


@pytest.mark.parametrize("side", ["q_weight", "k_weight"])
@pytest.mark.parametrize("case", [(2, 37, 6, 2, 64, 32, True, True, False), (1, 1300, 32, 8, 128, 128, False, True, True)], ids=str)
def test_norm_on_one_side_only(gqa, case, side):
    """A weight for the queries or the keys alone: the other side is rotated as it is, and has no
    weight gradient; its inputs are not read by the backward pass."""
    torch = torch_mod()
    B, T, Hq, Hkv, D, rot, inter, _, fp32 = case
    qkv, w, cos, sin, pos = _rope_inputs(case, 201)
    w = {n: v if n == side else None for n, v in w.items()}
    dz = [gi.normal_bf16(202 + i, gi.TENSOR_DO, (B, h, T, D)) for i, h in enumerate((Hq, Hkv))]
    d = to_dev(qkv).transpose(1, 2)
    x = [d[:, :Hq], d[:, Hq:Hq + Hkv]]
    how = dict(_dev_weights(w, fp32), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos), interleaved=inter, eps=1e-5)
    z = gqa.qk_norm_rope(*x, **how)
    unread = [t if n == side else torch.full_like(t, float("nan")) for t, n in zip(x, ("q_weight", "k_weight"))]
    grads = gqa.qk_norm_rope_bwd(to_dev(dz[0]), to_dev(dz[1]), *unread, **how)
    _sync_ok(gqa)
    rows = ref.f64(qkv).transpose(0, 2, 1, 3)
    c, s = _at(cos, sin, pos)
    for i, (lo, hi, n) in enumerate(((0, Hq, "q_weight"), (Hq, Hq + Hkv, "k_weight"))):
        want, size = ref.norm_rope(rows[:, lo:hi], w[n], 1e-5, c, s, inter)
        _near(from_dev(z[i]), want, STEP * np.abs(want) + 2.0 ** -16 * size, n)
        dx, dw, size, wsize = ref.norm_rope_bwd(ref.f64(dz[i]), rows[:, lo:hi], w[n], 1e-5, c, s, inter)
        _near(from_dev(grads[i]), dx, STEP * np.abs(dx) + 2.0 ** -16 * size, "gradient under " + n)
        if n == side:
            _near(grads[2 + i].cpu().numpy(), dw, 2.0 ** -15 * wsize, "gradient of " + n)
        else:
            assert grads[2 + i] is None


def test_every_call_on_another_stream(gqa):
    """The calls on a stream of their own, behind work of the current one, with outputs allocated by them
    and dropped at once: nothing allocated for a call is given away before the stream has passed it."""
    torch = torch_mod()
    N, Hq, Hkv, D, page = 600, 8, 2, 128, 32
    qkv, w, cos, sin, pos = _rope_inputs((1, N, Hq, Hkv, D, D, False, True, True), 211)
    how = dict(_dev_weights(w, True), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos[0]))
    d = to_dev(qkv)[0]
    q, k, v = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]
    pages = N // page + 2
    held, new, count, lens = _i32([N]), _i32([1]), _i32([4]), _i32([N])
    table0 = torch.arange(pages + 4, dtype=torch.int32, device="cuda")[None]
    side = torch.cuda.Stream()

    def step(stream):
        pools = [torch.full((pages, page, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        pools4 = [torch.full((pages, Hkv, page, D // 2 + 4), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(2)]
        table, free = table0.clone(), torch.arange(pages, pages + 4, dtype=torch.int32, device="cuda")
        slots = torch.arange(N, dtype=torch.int32, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        got = []
        p = gqa.paged_plan(held, new, table, free, count, page_size=page, num_pages=pages + 4, max_tokens=40, stream=stream)
        z = gqa.qk_norm_rope(q[None].transpose(1, 2), k[None].transpose(1, 2), stream=stream, **how)
        g = gqa.qk_norm_rope_bwd(*z, q[None].transpose(1, 2), k[None].transpose(1, 2), stream=stream, **how)
        qa = gqa.qk_norm_rope_append(q, k, v, *pools, slots, stream=stream, **how)
        gqa.kv4_append(k, v, *pools4, slots, stream=stream)
        back = gqa.kv4_gather(*pools4, slots, stream=stream)
        o = gqa.attn_decode_kv4(qa[-1][None], *pools4, lens, table, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        for t in (*p, *z, *g, qa, *back, o, *pools, *pools4, table, free):
            got.append(t.clone())
        return got

    want = step(None)
    _sync_ok(gqa)
    for _ in range(3):
        got = step(side)
        noise = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(4)]  # takes what was given back too early
        _sync_ok(gqa)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
        del noise
