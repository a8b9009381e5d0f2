"""The bounded waits of the single-token kernels, made to run out from the host:
a tile that is there is not said to be. The call reports FDLLM_ERR_TIMEOUT, and
the next one gives what the calls before gave. Waits of 2 ms; nothing traps,
faults or spins without a bound."""
import pytest
import torch

import kv_cache_attention_flash_b200 as fd
from kv_cache_attention_flash_b200 import _lib

BF, F32 = torch.bfloat16, torch.float32
WAIT_NS = 2_000_000


def test_refusals_without_a_gpu():
    lib = _lib.load()
    for ns in (-1, 10 ** 9 + 1):
        assert lib.fdllm_inject_tile_timeout(ns) == _lib.FDLLM_ERR_INVALID_ARG
        assert b"inject_tile_timeout" in lib.fdllm_last_error()
    assert lib.fdllm_inject_tile_timeout(5) == _lib.FDLLM_OK
    assert lib.fdllm_inject_tile_timeout(0) == _lib.FDLLM_OK


def held_up(call):
    """call(status) -> tensors: right, then held up, then right again."""
    def once():
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = [t.clone() for t in call(status)]
        torch.cuda.synchronize()
        return out, int(status.item())

    want, status = once()
    assert status == 0
    fd.fdllm_inject_tile_timeout(WAIT_NS)
    _, status = once()
    assert status == _lib.FDLLM_ERR_TIMEOUT
    got, status = once()
    assert status == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# tiles and rows; one tile a CTA, rings that fill up, shares taken over from the grid
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ps", [6, 64])
@pytest.mark.parametrize("B,hk,n", [(1, 1, 5), (1, 4, 700), (2, 2, 60000), (60, 8, 600)])
def test_decode_attention(dtype, ps, B, hk, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    width = -(-n // ps)
    kp, vp = rnd(1, B * width, hk, ps, 64), rnd(1, B * width, hk, ps, 64)
    table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q, k, v = rnd(B, 2 * hk * 64), rnd(B, hk * 64), rnd(B, hk * 64)
    held_up(lambda status: (*fd.fdllm_decode_attention(q, kp, vp, 0, table, lens, k, v, slots=lens - 1,
                                                       with_lse=True, status=status), kp, vp))


# one CTA a tile, clusters, a second round of CTAs, pairs of CTAs
@pytest.mark.gpu
@pytest.mark.parametrize("rows,n_in,n_out", [(1, 64, 64), (1, 4096, 512), (12, 8192, 1024), (40, 1000, 20008),
                                             (130, 2048, 2048), (600, 512, 1032), (3000, 4096, 2056)])
@pytest.mark.parametrize("gate", [False, True])
def test_linear(rows, n_in, n_out, gate):
    g = torch.Generator(device="cuda").manual_seed(rows)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    x, w, r = rnd(rows, n_in), rnd(n_in, n_out), rnd(rows, n_out)
    wg = rnd(n_in, n_out) if gate else None
    held_up(lambda status: [fd.fdllm_linear(x, w, act="silu", w_gate=wg, residual=r, status=status)])


@pytest.mark.gpu
def test_check_raises_it():
    c = fd.FlashCache(1, 1, 128, 64, 4, 256, 10000.0, "bf16", 1, 256)
    i32 = dict(dtype=torch.int32, device="cuda")
    z = torch.zeros(1, 128, dtype=BF, device="cuda")
    call = lambda: c.decode(0, z, z, z, torch.tensor([70], **i32), torch.tensor([[1, 2]], **i32),  # noqa: E731
                            torch.tensor([71], **i32))
    fd.fdllm_inject_tile_timeout(WAIT_NS)
    call()
    with pytest.raises(fd.FdllmError) as e:
        c.check()
    assert e.value.status == _lib.FDLLM_ERR_TIMEOUT and "timed out" in str(e.value)
    call()
    c.check()
