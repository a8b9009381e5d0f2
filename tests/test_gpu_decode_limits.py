"""fdllm_decode_attention over as many slots as the header allows, whose
rounding up to whole tiles leaves 31 bits."""
import pytest
import torch

import kv_cache_attention_flash_b200 as fd

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("ps,blocks", [(16, 2 ** 27 - 2), (1, 2 ** 31 - 2)])
def test_the_longest_sequence(ps, blocks):
    """A table that names 1000 pages over and over: each page's slots count as
    often as it is named. 2^31 slots in 2^25 tiles over at least 100 CTAs: a thread
    adds up at most 2^19 values, each addition cut by 2^-23 of the sum, 2^-4 in all
    for the sum and for its products with V (a bound; what is looked for is a lost
    or misplaced slot range)."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    pages, D = 1000, 32
    n = ps * blocks
    g = torch.Generator(device="cuda").manual_seed(ps)
    kp, vp = (torch.randn(1, pages, 1, ps, D, generator=g, device="cuda").to(BF) for _ in range(2))
    vp = (vp.abs() + 1).to(BF)
    q = torch.randn(1, D, generator=g, device="cuda").to(BF)
    table = torch.empty(1, blocks, dtype=torch.int32, device="cuda")
    line = torch.arange(pages, dtype=torch.int32, device="cuda")
    whole = blocks // pages * pages
    table[0, :whole].view(-1, pages).copy_(line.expand(blocks // pages, pages))
    table[0, whole:] = line[:blocks - whole]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    times = torch.full((pages,), blocks // pages, dtype=torch.float64, device="cuda")
    times[:blocks - whole] += 1
    for first in (0, n - 100):                  # everything, and the last slots alone
        starts = torch.tensor([first], dtype=torch.int32, device="cuda")
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        out, lse = fd.fdllm_decode_attention(q, kp, vp, 0, table, lens, starts=starts, with_lse=True, status=status)
        K, V = kp[0, :, 0].double(), vp[0, :, 0].double()
        s = (K @ q[0].double()) * D ** -0.5     # [pages, ps]
        e = torch.exp(s)
        if first == 0:
            w = e * times[:, None]
        else:
            slot = torch.arange(first, n, device="cuda")
            w = torch.zeros_like(e)
            w.index_put_((table[0, slot // ps].long(), slot % ps), e[table[0, slot // ps].long(), slot % ps],
                         accumulate=True)
        want = torch.einsum("ps,psd->d", w, V) / w.sum()
        tol = 2.0 ** -3 if first == 0 else 2.0 ** -12
        assert int(status) == 0
        assert bool(((out[0].double() - want).abs() <= tol * want.abs()).all()), (first, out, want)
        assert abs(float(lse[0, 0]) - float(w.sum().log())) <= tol
