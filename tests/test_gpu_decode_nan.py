"""A NaN that a query sees reaches its output and lse, in sequences that one
CTA answers whole and in those whose parts are joined, and nobody else's."""
import numpy as np
import pytest
import torch

from test_gpu_decode_attention import BF, F32, case, run

pytestmark = pytest.mark.gpu


def both(c):
    out, lse, _, _, status = run(c)
    assert status == 0
    return out.view(out.shape[0], lse.shape[1], -1), lse


# lengths: of whole units (many short sequences), and split over many shares, with few
# heads (eight warps join a head) and with many (one does)
BATCHES = [(700, 1, 1, [40] * 700), (2, 2, 3, [9000, 5000]), (1, 1, 11, [20000]), (40, 8, 1, [700] * 40)]


@pytest.mark.parametrize("B,hk,G,lens", BATCHES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ps", [6, 64])
def test_a_query_of_nan(B, hk, G, lens, dtype, ps):
    c = case(B, hk, G, 32, ps, lens, dtype, append=False, rope=False, seed=B)
    want, want_lse = both(c)
    c["q"] = c["q"].clone()
    head = hk * G - 1
    c["q"][0, head * 32 + 5] = float("nan")
    out, lse = both(c)
    assert bool(out[0, head].isnan().all()) and bool(lse[0, head].isnan())
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[0, head] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_keys_of_nan_over_a_whole_part(dtype):
    """Of 9000 slots the keys of 3000 are NaN: more than a share holds, so some
    parts have no other score. Each head that reads them answers NaN."""
    c = case(1, 2, 2, 64, 64, [9000], dtype, append=False, seed=3)
    for slot in range(3000, 6000):
        c["k_pool"][0, c["table"][0, slot // 64], 1, slot % 64] = float("nan")
    out, lse = both(c)
    assert bool(out[0, 2:].isnan().all()) and bool(lse[0, 2:].isnan().all())
    assert bool(out[0, :2].isfinite().all()) and bool(lse[0, :2].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_seen_is_still_zero(dtype):
    lens = [0, 5000, 0]
    c = case(3, 2, 2, 64, 64, lens, dtype, append=False, seed=4)
    c["q"] = c["q"].clone()
    c["q"][0] = float("nan")                   # sees nothing: zeros, whatever it is
    out, lse = both(c)
    for b in (0, 2):
        assert bool((out[b] == 0).all()) and bool((lse[b] == -np.inf).all())
    assert bool(out[1].isfinite().all())
