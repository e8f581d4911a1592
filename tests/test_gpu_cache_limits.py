"""The operators around the paged cache at the ends of what their arguments allow."""
import ctypes

import pytest

import gqa_inputs as gi
from tests import cache_ref as ref
from tests.gpu_util import from_dev, to_dev, torch_mod
from tests.test_gpu_cache import _kv4_pools, _near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    torch_mod()
    import grouped_query_softmax_b200 as m
    return m


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_of_as_many_tokens_as_fit_32_bits(gqa, in_place):
    """2^31 - 16 tokens of one request and 15 of padding: token numbers up to 2^31 - 2, which a thread
    steps past by its stride."""
    torch = torch_mod()
    page, tokens = 16, 2 ** 31 - 1
    total, pages = tokens - 15, (tokens - 15) // page
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    held, count = i32([0]), i32([pages])
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(pages, dtype=torch.int32, device="cuda")
    out = None
    if in_place:
        e = lambda n: torch.full((n,), -3, dtype=torch.int32, device="cuda")
        out = gqa.PagedPlan(held, e(2), e(tokens), e(tokens), count)
    p = gqa.paged_plan(held, i32([total]), table, free, count, page_size=page, num_pages=pages, max_tokens=tokens, out=out)
    torch.cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_OK
    assert p.seqlens_k.tolist() == [total] and p.cu_seqlens.tolist() == [0, total] and int(p.free_count) == 0
    assert torch.equal(table[0], torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda"))  # the last page first
    step = 1 << 27
    for lo in range(0, total, step):
        hi = min(lo + step, total)
        want = torch.arange(lo, hi, device="cuda")
        assert torch.equal(p.positions[lo:hi].long(), want)
        assert torch.equal(p.slots[lo:hi].long(), (pages - 1 - want // page) * page + want % page)
    assert (p.positions[total:] == 0).all() and (p.slots[total:] == -1).all()


def test_decode_kv4_merge_follows_only_runs_of_its_workspace(gqa):
    """The merge over units whose pieces' runs are not what a decode leaves: numbers a workspace may
    hold where a wait ran out. Those rows stay as they are, the others are merged."""
    torch = torch_mod()
    B, Hq, Hkv, Tq, longest, D, rows = 64, 32, 8, 1, 32768, 128, 8
    lib = ctypes.CDLL(gqa.library_path())
    lib.gqa_testing_decode_kv4_merge.argtypes = ([ctypes.c_void_p] * 2 + [ctypes.c_int] * 6
                                                 + [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p])
    nbytes = gqa.gqa_attn_decode_kv4_workspace_bytes(B, Hq, Hkv, Tq, longest, D)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    lens = torch.full((B,), longest, dtype=torch.int32, device="cuda")
    out = torch.full((B, Hq, Tq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    runs = ctypes.c_int()

    def merge():
        return lib.gqa_testing_decode_kv4_merge(out.data_ptr(), lens.data_ptr(), B, Hq, Hkv, Tq, longest, D, ws.data_ptr(),
                                                nbytes, ctypes.byref(runs), torch.cuda.current_stream().cuda_stream)

    assert merge() == gqa.GQA_OK   # all pairs are (0, 0): nothing to merge
    torch.cuda.synchronize()
    assert (out == 7).all()
    n = runs.value
    ends = ws[nbytes - 8 * B * Hkv:].view(torch.int32).view(B, Hkv, 2)
    parts = ws[:2 * n * rows * D * 4].view(torch.float32).view(n, 2, rows, D)   # log-sum-exps of 0: equal weights
    for run, slot, value in ((3, 1, 1.0), (4, 0, 2.0), (5, 0, 6.0), (n - 2, 1, 4.0), (n - 1, 0, 5.0)):
        parts[run, slot] = value
    bad = [(-1, 3), (-2 ** 31, 2 ** 31 - 1), (5, 3), (n - 1, n), (0, 2 ** 31 - 1), (2 ** 31 - 1, 0), (n, n + 1), (-5, -2)]
    for h, pair in enumerate(bad):
        ends[1, h] = torch.tensor(pair, dtype=torch.int64).int()
    ends[0, 0], ends[2, 7] = torch.tensor([3, 5]), torch.tensor([n - 2, n - 1])
    lens[2] = longest + 1     # such a sequence has no output, whatever its pairs say
    ends[63, 0], lens[62], ends[62, 0] = torch.tensor([n - 2, n - 1]), -1, torch.tensor([3, 5])
    assert merge() == gqa.GQA_OK
    torch.cuda.synchronize()
    assert gqa.gqa_get_device_error() == gqa.GQA_OK
    want = torch.full_like(out, 7.0)
    want[0, :4], want[63, :4] = 3.0, 4.5
    assert torch.equal(out, want)


@pytest.mark.parametrize("pool_layout,rot", [("NHD", 64), ("HND", 32)])
def test_append_leaves_all_rows_of_a_bad_position(gqa, pool_layout, rot):
    """A token outside the angle tables: neither its key nor its value row is written, nor its query."""
    torch = torch_mod()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q, k, v = (to_dev(gi.normal_bf16(101 + i, i, (6, h, 64))) for i, h in enumerate((4, 2, 2)))
    cos, sin = (torch.tensor(t, device="cuda") for t in ref.angles(10, rot))
    shape = (3, 16, 2, 64) if pool_layout == "NHD" else (3, 2, 16, 64)
    new = lambda: [torch.full(shape, 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)] + [torch.full_like(q, 9.0)]
    slots = i32([5, 20, 40, 1, -1, 30])
    good, got = new(), new()
    for out, positions in ((good, [0, 1, 2, 3, 4, 5]), (got, [0, 10, 2, -1, 4, 5])):
        gqa.qk_norm_rope_append(q, k, v, out[0], out[1], slots, cos=cos, sin=sin, positions=i32(positions),
                                pool_layout=pool_layout, q_out=out[2])
        torch.cuda.synchronize()
        assert gqa.gqa_get_device_error() == (gqa.GQA_OK if out is good else gqa.GQA_ERR_INVALID_ARGUMENT)
    for want, have in zip(good[:2], got[:2]):
        for slot in (20, 1):
            want[(slot // 16, slot % 16) if pool_layout == "NHD" else (slot // 16, slice(None), slot % 16)] = 9.0
        assert torch.equal(want, have)
    good[2][[1, 3]] = 9.0
    assert torch.equal(good[2], got[2])


@pytest.mark.parametrize("largest", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("Hq,Hkv,Tq,D,lens,window", [(8, 2, 1, 128, [4099], 0), (16, 2, 2, 64, [3000, 0, 1, 777], 0),
                                                     (32, 1, 1, 128, [2500, 40], 1000)])
def test_decode_kv4_in_smaller_clusters(gqa, largest, Hq, Hkv, Tq, D, lens, window):
    """Cases that take clusters of 16 CTAs, on a device that would hold fewer."""
    torch = torch_mod()
    lib = ctypes.CDLL(gqa.library_path())
    kp, vp, table = _kv4_pools(lens, Hkv, D, 64, 111, window, Tq)
    q = gi.normal_bf16(112, gi.TENSOR_Q, (len(lens), Hq, Tq, D))
    dev = lambda x: torch.tensor(x, device="cuda")
    try:
        assert lib.gqa_testing_decode_kv4_largest_cluster(largest) == 0
        o = gqa.attn_decode_kv4(to_dev(q), dev(kp), dev(vp), torch.tensor(lens, dtype=torch.int32, device="cuda"), dev(table),
                                window=window)
        torch.cuda.synchronize()
    finally:
        assert lib.gqa_testing_decode_kv4_largest_cluster(16) == 0
    assert gqa.gqa_get_device_error() == gqa.GQA_OK
    want, tol = ref.decode_kv4(q, kp, vp, lens, table, window)
    _near(from_dev(o), want, tol, f"clusters of at most {largest}")
