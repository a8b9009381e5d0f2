"""fdllm_plan_blocks and fdllm_release_blocks at the header's limit of pages,
one slot a page: steps of the grid past 2^31 - 114 k pages."""
import pytest
import torch

import kv_cache_attention_flash_b200 as fd

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 2


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(a, b):
    step = 1 << 28
    return all(torch.equal(a[i:i + step], b[i:i + step]) for i in range(0, a.numel(), step))


def test_as_many_pages_as_a_call_may_take_and_give_back():
    """17 GB: a table of 2^31 - 2 pages given back to an empty list (in the table's
    order), and taken again from its end."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    table = torch.arange(MOST - 1, -1, -1, dtype=torch.int32, device="cuda").view(1, -1)
    free = torch.full((MOST,), -3, dtype=torch.int32, device="cuda")
    status = i32(0)
    back = fd.fdllm_release_blocks(i32(MOST), i32(0), table, 1, free, i32(0), status=status)
    assert int(back["n_free"]) == MOST and back["seq_lens"].tolist() == [0] and int(status) == 0
    assert same(free, table[0])
    table.fill_(-7)
    plan = fd.fdllm_plan_blocks(i32(5), i32(MOST - 5), table, 1, free, i32(MOST - 5), capacity=4, status=status)
    assert plan["granted"].tolist() == [1] and int(plan["n_free"]) == 0
    assert plan["cu_rows"].tolist() == [0, MOST - 5] and int(status) == 4        # rows past the capacity
    assert plan["positions"].tolist() == [5, 6, 7, 8]
    # the list's entry k holds page MOST - 1 - k; the request's pages come from entry MOST - 6 on down
    assert bool((table[0, :5] == -7).all())
    free.copy_(table[0])
    want = torch.arange(5, MOST, dtype=torch.int32, device="cuda")
    assert same(free[5:], want)
