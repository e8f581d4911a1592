"""The operators around the paged cache without a GPU: what the C entry points and the torch
functions refuse, and the workspace sizes."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def gqa():
    import grouped_query_softmax_b200 as m
    return m


P = 1 << 20  # an aligned fake device address; never dereferenced on these paths


def plan(gqa, **kw):
    a = dict(seqlens=P, keep=None, new_tokens=P, block_table=P, free_list=P, free_count=P, seqlens_out=P, cu_seqlens=P,
             positions=P, slots=P, free_count_out=P, S=4, max_pages=8, page_size=64, num_pages=100, free_capacity=100,
             max_tokens=64)
    a.update(kw)
    return gqa.gqa_paged_plan(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(seqlens=None), 1), (dict(new_tokens=None), 1), (dict(block_table=None), 1), (dict(free_list=P + 2), 1),
    (dict(keep=P + 1), 1), (dict(positions=P + 4), 1), (dict(slots=P + 8), 1), (dict(free_count_out=None), 1),
    (dict(S=0), 1), (dict(S=8193), 2), (dict(max_pages=0), 1), (dict(max_tokens=0), 1), (dict(free_capacity=0), 1),
    (dict(page_size=48), 1), (dict(page_size=8), 1), (dict(num_pages=0), 1), (dict(num_pages=1 << 26), 2),
    (dict(max_pages=1 << 26), 2),
])
def test_plan_rejects_bad_arguments(gqa, kw, status):
    assert plan(gqa, **kw) == status


def rope(gqa, **kw):
    r = dict(q_weight=P, k_weight=P, cos=P, sin=P, positions=P, positions_sb=0, n_positions=100, rot=64, interleaved=0,
             weight_fp32=0, eps=1e-6)
    r.update({k: kw.pop(k) for k in list(kw) if k in r})
    return gqa.GqaRope(**r), kw


LAY_Q, LAY_K = (8 * 4 * 64, 64, 4 * 64), (8 * 2 * 64, 64, 2 * 64)


def fwd(gqa, **kw):
    r, kw = rope(gqa, **kw)
    a = dict(q=P, k=P, q_out=P, k_out=P, B=2, T=8, Hq=4, Hkv=2, D=64, q_layout=LAY_Q, k_layout=LAY_K, q_out_layout=LAY_Q,
             k_out_layout=LAY_K, rope=r)
    a.update(kw)
    return gqa.gqa_qk_norm_rope(**a)


ROPE = [
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(sin=None), 1),
    (dict(cos=P + 4), 1), (dict(rot=0), 1), (dict(rot=20), 1), (dict(rot=128), 1), (dict(n_positions=0), 1),
    (dict(positions=P + 2), 1), (dict(positions=None, n_positions=7), 1), (dict(q_weight=P + 1), 1),
    (dict(weight_fp32=1, k_weight=P + 2), 1), (dict(Hq=5), 1), (dict(Hkv=0), 1), (dict(D=96), 2), (dict(rope=None), 1),
]


@pytest.mark.parametrize("kw,status", ROPE + [
    (dict(q=None), 1), (dict(k_out=P + 8), 1), (dict(T=0), 1), (dict(B=0), 1), (dict(q_layout=(2048, 64, 100)), 1),
    (dict(k_layout=(0, 64, 128)), 1), (dict(q_out_layout=(2048, 64, 32)), 1), (dict(positions_sb=-8), 1),
])
def test_norm_rope_rejects_bad_arguments(gqa, kw, status):
    assert fwd(gqa, **kw) == status


def bwd(gqa, **kw):
    r, kw = rope(gqa, **kw)
    a = dict(dq_out=P, dk_out=P, q=P, k=P, dq=P, dk=P, dq_weight=P, dk_weight=P, B=2, T=8, Hq=4, Hkv=2, D=64,
             dq_out_layout=LAY_Q, dk_out_layout=LAY_K, q_layout=LAY_Q, k_layout=LAY_K, dq_layout=LAY_Q, dk_layout=LAY_K,
             rope=r, workspace=P, workspace_bytes=1 << 20)
    a.update(kw)
    return gqa.gqa_qk_norm_rope_bwd(**a)


@pytest.mark.parametrize("kw,status", ROPE + [
    (dict(dq_out=None), 1), (dict(dk=P + 8), 1), (dict(q=None), 1), (dict(dq_weight=None), 1),
    (dict(q_weight=None), 1), (dict(dk_weight=P + 2), 1), (dict(T=0), 1), (dict(q_layout=(2048, 64, 100)), 1),
    (dict(workspace=None), 3), (dict(workspace=P + 64), 3), (dict(workspace_bytes=16), 3),
])
def test_norm_rope_bwd_rejects_bad_arguments(gqa, kw, status):
    assert bwd(gqa, **kw) == status


def append(gqa, **kw):
    r, kw = rope(gqa, **kw)
    pool = (64 * 2 * 64, 64, 2 * 64)
    a = dict(q=P, k=P, v=P, q_out=P, k_pool=P, v_pool=P, slots=P, N=8, Hq=4, Hkv=2, D=64, page_size=64, num_pages=10,
             q_layout=LAY_Q, k_layout=LAY_K, v_layout=LAY_K, q_out_layout=LAY_Q, k_pool_layout=pool, v_pool_layout=pool,
             rope=r)
    a.update(kw)
    return gqa.gqa_qk_norm_rope_append(**a)


@pytest.mark.parametrize("kw,status", ROPE + [
    (dict(v=None), 1), (dict(slots=None), 1), (dict(k_pool=P + 8), 1), (dict(N=-1), 1), (dict(page_size=24), 1),
    (dict(num_pages=0), 1), (dict(num_pages=1 << 25), 2), (dict(k_pool_layout=(64 * 128, 64, 100)), 1),
    (dict(v_pool_layout=(0, 64, 128)), 1), (dict(N=0), 0), (dict(N=0, q=None, slots=None), 0),
])
def test_append_rejects_bad_arguments(gqa, kw, status):
    assert append(gqa, **kw) == status


def kv4(gqa, gather=False, **kw):
    pool = (2 * 64 * 36, 64 * 36)
    a = dict(k=P, v=P, k_pool=P, v_pool=P, slots=P, N=8, Hkv=2, D=64, page_size=64, num_pages=10, k_layout=LAY_K,
             v_layout=LAY_K, k_pool_layout=pool, v_pool_layout=pool)
    a.update(kw)
    return gqa.gqa_kv4_gather(**a) if gather else gqa.gqa_kv4_append(**a)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v_pool=P + 4), 1), (dict(slots=P + 1), 1), (dict(N=-1), 1), (dict(Hkv=0), 1), (dict(D=32), 2),
    (dict(page_size=40), 1), (dict(num_pages=1 << 25), 2), (dict(k_layout=(0, 64, 60)), 1),
    (dict(k_pool_layout=(2 * 64 * 36 + 8, 64 * 36)), 1), (dict(v_pool_layout=(2 * 64 * 36, 64 * 32)), 1), (dict(N=0), 0),
])
def test_kv4_rows_reject_bad_arguments(gqa, gather, kw, status):
    assert kv4(gqa, gather, **kw) == status


# enough work for runs of tiles that cut units, whose partial states need a workspace
MANY = dict(B=64, Hq=32, Hkv=8, max_seqlen_k=32768, max_pages=512, k_layout=(8 * 64 * 68, 64 * 68),
            v_layout=(8 * 64 * 68, 64 * 68))


def dec(gqa, **kw):
    pool = (2 * 64 * 68, 64 * 68)
    a = dict(q=P, k_pool=P, v_pool=P, o=P, seqlens_k=P, block_table=P, page_size=64, num_pages=100, max_pages=16, B=2,
             Hq=4, Hkv=2, Tq=1, max_seqlen_k=1024, D=128, k_layout=pool, v_layout=pool, workspace=P,
             workspace_bytes=1 << 24)
    a.update(kw)
    return gqa.gqa_attn_decode_kv4(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(o=P + 8), 1), (dict(k_pool=P + 8), 1), (dict(seqlens_k=None), 1), (dict(block_table=None), 1),
    (dict(Hq=5), 1), (dict(B=0), 1), (dict(Tq=0), 1), (dict(Tq=17), 2), (dict(D=96), 2), (dict(window=-1), 1),
    (dict(page_size=48), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(max_seqlen_k=0), 1),
    (dict(max_seqlen_k=(1 << 30) + 1), 2), (dict(softmax_scale=float("nan")), 1), (dict(softmax_scale=float("inf")), 1),
    (dict(v_layout=(2 * 64 * 68, 64 * 68 - 16)), 1), (dict(k_layout=(2 * 64 * 68 + 4, 64 * 68)), 1),
    (dict(MANY, workspace=None), 3), (dict(MANY, workspace=P + 64), 3), (dict(MANY, workspace_bytes=100), 3),
    (dict(B=1 << 20, Hq=1 << 10, Hkv=1 << 10, Tq=16), 2),
])
def test_decode_rejects_bad_arguments(gqa, kw, status):
    assert dec(gqa, **kw) == status


def test_workspace_sizes(gqa):
    size = gqa.gqa_attn_decode_kv4_workspace_bytes
    assert size(1, 4, 1, 1, 32, 128) == 0 and size(1, 32, 8, 1, 4099, 128) == 0  # merged through shared memory
    assert 0 < size(64, 32, 8, 1, 32768, 128) <= 64 << 20
    assert size(64, 32, 8, 17, 32768, 128) == 0
    assert gqa.gqa_qk_norm_rope_bwd_workspace_bytes(1, 16, 8, 2, 128) % 256 == 0
    assert gqa.gqa_qk_norm_rope_bwd_workspace_bytes(1, 16, 8, 3, 128) == 0


def test_torch_functions_refuse_wrong_operands(gqa):
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    with pytest.raises(TypeError):  # not on a GPU
        gqa.paged_plan(i32(2), i32(2), i32(2, 4), i32(9), i32(1), page_size=16, num_pages=9, max_tokens=8)
    with pytest.raises(TypeError):
        gqa.paged_plan(i32(2).long(), i32(2), i32(2, 4), i32(9), i32(1), page_size=16, num_pages=9, max_tokens=8)
    with pytest.raises(ValueError):
        gqa.paged_plan(i32(2), i32(3), i32(2, 4), i32(9), i32(1), page_size=16, num_pages=9, max_tokens=8)
    with pytest.raises(ValueError):
        gqa.paged_plan(i32(2), i32(2), i32(3, 4), i32(9), i32(1), page_size=16, num_pages=9, max_tokens=8)
    with pytest.raises(TypeError):
        gqa.qk_norm_rope(bf(1, 4, 3, 64), bf(1, 2, 3, 64))
    with pytest.raises(TypeError):
        gqa.qk_norm_rope(bf(1, 4, 3, 64).float(), bf(1, 2, 3, 64))
    with pytest.raises(ValueError):
        gqa.qk_norm_rope(bf(1, 4, 3, 64), bf(1, 2, 4, 64))
    with pytest.raises(ValueError):
        gqa.qk_norm_rope(bf(1, 4, 64, 3).transpose(2, 3), bf(1, 2, 3, 64))
    with pytest.raises(ValueError):
        gqa.qk_norm_rope(bf(1, 4, 3, 64), bf(1, 2, 3, 64), cos=torch.zeros(3, 32))
    with pytest.raises(TypeError):
        gqa.qk_norm_rope(bf(1, 4, 3, 64), bf(1, 2, 3, 64), q_weight=bf(64), k_weight=torch.zeros(64))
    with pytest.raises(ValueError):
        gqa.qk_norm_rope(bf(1, 4, 3, 64), bf(1, 2, 3, 64), cos=torch.zeros(3, 32), sin=torch.zeros(3, 32),
                         positions=i32(4))
    with pytest.raises(ValueError):
        gqa.qk_norm_rope_append(bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), bf(5, 16, 3, 64), bf(5, 16, 3, 64), i32(3))
    with pytest.raises(ValueError):
        gqa.qk_norm_rope_append(bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), bf(5, 16, 2, 64), bf(5, 16, 2, 64), i32(4))
    pool = lambda d: torch.zeros((5, 2, 16, d // 2 + 4), dtype=torch.uint8)
    with pytest.raises(ValueError):
        gqa.kv4_append(bf(3, 2, 64), bf(3, 2, 64), pool(128), pool(128), i32(3))
    with pytest.raises(ValueError):
        gqa.kv4_append(bf(3, 4, 64), bf(3, 4, 64), pool(64), pool(64), i32(3))
    with pytest.raises(TypeError):
        gqa.kv4_gather(bf(5, 2, 16, 36), bf(5, 2, 16, 36), i32(3))
    with pytest.raises(ValueError):
        gqa.attn_decode_kv4(bf(2, 4, 64), pool(64), pool(64), i32(3), i32(2, 4))
    with pytest.raises(ValueError):
        gqa.attn_decode_kv4(bf(2, 4, 64), pool(64), pool(64), i32(2), i32(3, 4))
    with pytest.raises(TypeError):
        gqa.attn_decode_kv4(bf(2, 4, 64).float(), pool(64), pool(64), i32(2), i32(2, 4))


def test_decode_runs_cover_every_tile_once():
    """The cut of the tiles between CTAs, restated: runs are disjoint, cover all, none is empty,
    and the CTA of a tile is found from the tile's number alone."""
    rng = np.random.default_rng(4)
    for _ in range(200):
        total, grid = int(rng.integers(1, 5000)), int(rng.integers(1, 300))
        ctas = min(grid, total)
        cuts = [total * i // ctas for i in range(ctas + 1)]
        assert cuts[0] == 0 and cuts[-1] == total and all(a < b for a, b in zip(cuts, cuts[1:]))
        for w in rng.integers(0, total, 50):
            c = ((int(w) + 1) * ctas - 1) // total
            assert cuts[c] <= w < cuts[c + 1]
