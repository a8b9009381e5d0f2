"""The planner's entries of a request each (seq_positions, seq_slots) and the
decode calls that take them: a request without a row moves nobody else's."""
import ctypes

import numpy as np
import pytest
import torch

import kv_cache_attention_flash_b200 as fd
import serve_case as S
from kv_cache_attention_flash_b200 import _lib
from test_gpu_decode_stack import Server, rnd
from test_gpu_plan_blocks import buffers, dev, layout


def of_requests(lens, new, granted, top):
    """By definition: position and slot of the request's last row."""
    pos, slots = [], []
    for n, m, ok in zip(lens, new, granted):
        row = ok and 0 <= n <= top and 0 < m <= top - n
        pos.append(n + m - 1 if row else 0)
        slots.append(n + m - 1 if row else -1)
    return pos, slots


@pytest.mark.gpu
@pytest.mark.parametrize("B,ps,past,most,spare", [(1, 64, 10, 1, 1), (33, 16, 100, 1, 2), (300, 7, 60, 1, 20),
                                                  (1025, 4, 30, 3, 500)])
def test_entries_of_requests_equal_the_definition(B, ps, past, most, spare):
    rs = np.random.RandomState(B)
    lens, new = rs.randint(0, past + 1, B), rs.randint(0, most + 1, B)
    width = -(-past // ps) + 1
    lens[::5] = width * ps                      # at the table's end: a token more has no place
    if B > 3:
        lens[3] = -2
    table, free = layout(rs, np.maximum(lens, 0), ps, width, spare)
    want = S.plan_blocks(lens, new, table, ps, free, spare)
    out, t, status = buffers(B, int(new.sum())), dev(table), dev([0])
    fd.fdllm_plan_blocks(dev(lens), dev(new), t, ps, dev(free), dev([spare]), out=out, status=status)
    pos, slots = of_requests(lens.tolist(), new.tolist(), want["granted"], width * ps)
    assert out["seq_positions"].tolist() == pos and out["seq_slots"].tolist() == slots
    assert out["cu_rows"].tolist() == want["cu_rows"] and out["granted"].tolist() == want["granted"]
    n = len(want["positions"])
    assert out["slots"][:n].tolist() == want["slots"]
    assert int(status.item()) == (4 if want["bad"] else 0)


def full_and_idle():
    """Five requests of up to 192 tokens: 1 is at its table's end, 3 gets no token."""
    s = Server(batch=5, width=3)
    s.prompt([150, 192, 64, 10, 70])
    p = s.plan([1, 1, 1, 0, 1])
    assert p["cu_rows"].tolist() == [0, 1, 1, 2, 2, 3] and p["granted"].tolist() == [1, 0, 1, 1, 1]
    assert int(s.status.item()) == 4
    s.status.zero_()
    return s, p


@pytest.mark.gpu
def test_requests_without_a_row_leave_the_others_alone():
    s, p = full_and_idle()
    cos, sin = (t.cpu().numpy() for t in s.cache.rope_tables())
    qkv = rnd(5, 3 * s.H, seed=3).float()
    q, k, v = qkv.split(s.H, 1)
    before = s.cache.k_pool.cpu(), s.cache.v_pool.cpu()
    out, _ = s.cache.decode(1, q, k, v, p["seq_positions"], s.table, p["seq_lens"], p["seq_slots"],
                            status=s.status)
    torch.cuda.synchronize()
    slots = np.array([150, -1, 64, -1, 70])
    ref, _, kp, vp, tol, _ = S.decode_attention(q.cpu(), *before, 1, s.table.cpu().numpy(),
                                                [151, 192, 65, 10, 71], k.cpu(), v.cpu(),
                                                np.maximum(slots, 0), slots, cos, sin)
    for b in (0, 2, 4):
        assert np.all(np.abs(out[b].double().cpu().numpy() - ref[b]) <= tol[b] + 2.0 ** -24 * np.abs(ref[b])), b
    assert torch.equal(s.cache.k_pool.cpu().view(torch.int16), kp.view(torch.int16))
    assert torch.equal(s.cache.v_pool.cpu().view(torch.int16), vp.view(torch.int16))
    assert int(s.status.item()) == 0


@pytest.mark.gpu
def test_the_stack_writes_the_new_tokens_alone():
    s, p = full_and_idle()
    before = s.cache.k_pool.clone()
    x = rnd(5, s.H, seed=4)
    y = s.stack.decode(x.clone(), p["seq_positions"], s.table, p["seq_lens"], p["seq_slots"], status=s.status)
    torch.cuda.synchronize()
    changed = (s.cache.k_pool.view(torch.int16) != before.view(torch.int16)).nonzero()
    got = {(int(page), int(off)) for page, off in zip(changed[:, 1], changed[:, 3])}
    t = s.table.cpu()
    assert got == {(int(t[0, 2]), 22), (int(t[2, 1]), 0), (int(t[4, 1]), 6)}
    # the same step with the other requests' x of another kind: the three keep their bits
    s2, p2 = full_and_idle()
    x2 = x.clone()
    x2[1], x2[3] = 7.0, -3.0
    y2 = s2.stack.decode(x2, p2["seq_positions"], s2.table, p2["seq_lens"], p2["seq_slots"])
    assert all(torch.equal(y[b], y2[b]) for b in (0, 2, 4))


def test_refusals_of_the_two_outputs():
    """Misaligned, over an input, over another output (addresses are stand-ins)."""
    lib = _lib.load()
    MB, BAD = 1 << 24, _lib.FDLLM_ERR_INVALID_ARG

    def plan(**p):
        names = ["seq_lens", "new_lens", "block_table", "free_pages", "n_free", "cu_rows", "positions", "slots",
                 "row_seq", "slot_map", "seq_lens_out", "granted", "n_free_out", "headroom", "seq_positions",
                 "seq_slots", "status"]
        at = {n: (i + 1) * MB for i, n in enumerate(names)}
        at.update(p)
        return lib.fdllm_plan_step(2, 4, 16, 8, 10, *[at[n] for n in names], None)

    for n in ("seq_positions", "seq_slots"):
        assert plan(**{n: 60 * MB + 2}) == BAD and b"misaligned" in lib.fdllm_last_error()
        assert plan(**{n: MB + 4}) == BAD and b"overlaps" in lib.fdllm_last_error()
        assert plan(**{n: 8 * MB}) == BAD and b"overlaps" in lib.fdllm_last_error()
    assert plan(seq_slots=15 * MB) == BAD and b"overlaps" in lib.fdllm_last_error()
    assert lib.fdllm_plan_step(0, 4, 16, 8, 10, *[ctypes.c_void_p(MB)] * 17, None) == BAD


@pytest.mark.gpu
def test_buffers_are_for_exactly_their_batch():
    """Buffers of four requests are refused for three; slices of them serve."""
    lens, new, table, free = dev([3, 0, 8]), dev([1, 2, 0]), dev([[0, 9], [9, 9], [1, 2]]), dev([5, 4, 3])
    out = fd.fdllm_plan_buffers(4, 10)
    with pytest.raises(ValueError, match="shape"):
        fd.fdllm_plan_blocks(lens, new, table, 4, free, dev([2]), out=out)
    part = {k: v[:{"cu_rows": 4, "seq_lens": 3, "granted": 3, "seq_positions": 3, "seq_slots": 3}.get(k, len(v))]
            for k, v in out.items()}
    fd.fdllm_plan_blocks(lens, new, table, 4, free, dev([2]), out=part)
    assert out["cu_rows"][:4].tolist() == [0, 1, 3, 3] and out["seq_lens"][:3].tolist() == [4, 2, 8]
    assert out["seq_slots"][:3].tolist() == [3, 1, -1] and out["slots"][:3].tolist() == [3, 0, 1]
    # without the entries that may be left out
    few = {k: v for k, v in part.items() if k not in ("headroom", "seq_positions", "seq_slots")}
    table = dev([[0, 9], [9, 9], [1, 2]])
    assert fd.fdllm_plan_blocks(lens, new, table, 4, free, dev([2]), out=few)["seq_lens"].tolist() == [4, 2, 8]
