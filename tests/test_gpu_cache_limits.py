"""The operators around the paged cache at the ends of what their arguments allow."""
import numpy as np
import pytest

from tests.gpu_util import torch_mod

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
