"""What the decode calls meet on the device reaches FlashCache.check(), as the
layer step's errors do, unless the caller gives a status word of its own."""
import pytest
import torch

import kv_cache_attention_flash_b200 as fd
from kv_cache_attention_flash_b200 import _lib
from test_gpu_decode_stack import Server, rnd

pytestmark = pytest.mark.gpu


def server():
    s = Server(layers=2)
    s.prompt([70, 64, 3])
    return s, s.plan([1, 1, 1])


def attend(s, p, **kw):
    q, k, v = rnd(3, 3 * s.H, seed=1).split(s.H, 1)
    return s.cache.decode(0, q, k, v, p["seq_positions"], s.table, p["seq_lens"], p["seq_slots"], **kw)


def stack(s, p, **kw):
    return s.stack.decode(rnd(3, s.H, seed=2), p["seq_positions"], s.table, p["seq_lens"], p["seq_slots"], **kw)


def raises(s, code, stream=None):
    with pytest.raises(fd.FdllmError) as e:
        s.cache.check(stream)
    assert e.value.status == code
    s.cache.check(stream)                   # read and cleared


@pytest.mark.parametrize("call", [attend, stack])
@pytest.mark.parametrize("stream", [False, True])
def test_check_raises_what_decode_met(call, stream):
    s, p = server()
    st = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    call(s, p, stream=st)
    s.cache.check(st)
    s.table[1, 0] = 10 ** 6                 # a page outside the pool
    torch.cuda.synchronize()
    call(s, p, stream=st)
    raises(s, _lib.FDLLM_ERR_DEVICE_BOUNDS, st)
    s.table[1, 0] = 0
    p["seq_lens"][2] = 10 ** 6              # a length past the table
    torch.cuda.synchronize()
    call(s, p, stream=st)
    raises(s, _lib.FDLLM_ERR_DEVICE_BOUNDS, st)
    s.cache.check(st.cuda_stream if st else None)


@pytest.mark.parametrize("call", [attend, stack])
def test_a_status_of_the_callers_takes_the_error(call):
    s, p = server()
    s.table[1, 0] = -5
    call(s, p, status=s.status)
    s.cache.check()
    assert int(s.status.item()) == _lib.FDLLM_ERR_DEVICE_BOUNDS


def test_a_captured_call_reports_too():
    s, p = server()
    stack(s, p)
    s.cache.check()
    g = torch.cuda.CUDAGraph()
    x = rnd(3, s.H, seed=2)
    with torch.cuda.graph(g):
        s.stack.decode(x, p["seq_positions"], s.table, p["seq_lens"], p["seq_slots"])
    g.replay()
    s.cache.check()
    s.table[0, 0] = -1
    g.replay()
    raises(s, _lib.FDLLM_ERR_DEVICE_BOUNDS)
