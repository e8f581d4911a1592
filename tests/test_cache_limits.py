"""What the operators around the paged cache refuse at the ends of their ranges, without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def gqa():
    import grouped_query_softmax_b200 as m
    return m


P = 1 << 20  # an aligned fake device address; never dereferenced on these paths


@pytest.mark.parametrize("S,max_pages,page", [(8192, 1 << 18, 16), (8192, 1 << 20, 64), (128, 1 << 24, 16)])
def test_plan_refuses_tables_of_more_pages_than_it_counts(gqa, S, max_pages, page):
    """Every request may give all its pages back at once: their number has to fit 32 bits."""
    st = gqa.gqa_paged_plan(P, P, P, P, P, P, 2 * P, 2 * P, 2 * P, 2 * P, 2 * P, S, max_pages, page, 1000, 1000, 64)
    assert st == gqa.GQA_ERR_UNSUPPORTED


def test_merge_hook_refuses_what_the_decode_refuses(gqa):
    f = ctypes.CDLL(gqa.library_path()).gqa_testing_decode_kv4_merge
    f.argtypes = [ctypes.c_void_p] * 2 + [ctypes.c_int] * 6 + [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]
    runs = ctypes.c_int()
    many = (64, 32, 8, 1, 32768, 128)
    assert f(P, P, *many, None, 0, ctypes.byref(runs), None) == gqa.GQA_ERR_WORKSPACE
    assert f(P, P, *many, P, 1 << 20, ctypes.byref(runs), None) == gqa.GQA_ERR_WORKSPACE
    assert f(None, P, *many, P, 1 << 30, ctypes.byref(runs), None) == gqa.GQA_ERR_INVALID_ARGUMENT
    assert f(P, P, *many, P, 1 << 30, None, None) == gqa.GQA_ERR_INVALID_ARGUMENT
    assert f(P, P, 1, 32, 8, 1, 4099, 128, P, 1 << 30, ctypes.byref(runs), None) == gqa.GQA_ERR_UNSUPPORTED


def test_workspaces_that_claim_more_bytes_than_they_have_are_refused(gqa):
    """An expanded tensor's elements share memory: its size is not what a kernel may write."""
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    pool = torch.zeros((5, 2, 16, 36), dtype=torch.uint8)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 30), torch.zeros(1 << 12, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            gqa.attn_decode_kv4(bf(2, 4, 64), pool, pool, i32(2), i32(2, 4), workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            gqa.qk_norm_rope_bwd(bf(1, 4, 3, 64), bf(1, 2, 3, 64), bf(1, 4, 3, 64), bf(1, 2, 3, 64), q_weight=bf(64),
                                 k_weight=bf(64), workspace=ws)


def test_largest_cluster_hook_takes_powers_of_two(gqa):
    f = ctypes.CDLL(gqa.library_path()).gqa_testing_decode_kv4_largest_cluster
    assert [f(n) for n in (0, 3, 32, -1)] == [gqa.GQA_ERR_INVALID_ARGUMENT] * 4 and f(8) == f(16) == 0
