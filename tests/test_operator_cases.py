"""The timed cases of perf/operators.py: the plain form of block planning, the
framework's call and the definition (`exact`) give the same whole numbers,
also where a request that needs no page is granted after refused ones."""
import importlib.util
import os

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cases():
    spec = importlib.util.spec_from_file_location("operator_cases", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plan_state(lens, new, table, free, n_free, ps, cap, device="cpu"):
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=device)  # noqa: E731
    full = lambda n, dt=torch.int32: torch.full((n,), -7, dtype=dt, device=device)  # noqa: E731
    B = len(lens)
    return {"op": "blocks", "kind": "plan", "page": ps, "seq_lens": i32(lens), "new": i32(new),
            "table": i32(table), "free": i32(free), "n_free": i32([n_free]),
            "out": {"cu_rows": full(B + 1), "positions": full(cap), "slots": full(cap), "row_seq": full(cap),
                    "slot_map": full(cap, torch.int64), "seq_lens": full(B), "granted": full(B),
                    "n_free": full(1)}}


# lengths, new tokens, pages free, free pages left over; pages of 4 slots
PLANS = [
    # one page is taken, three are refused, none is needed, one is refused
    ([4, 0, 2, 8], [3, 12, 2, 1], 2, 1),
    # all refused but a request without need
    ([4, 4, 1], [5, 5, 0], 1, 1),
    # none refused
    ([0, 3, 5], [4, 2, 3], 5, 3),
    # the last ones refused
    ([0, 0, 0], [4, 4, 4], 2, 0),
]


def equal(got, want):
    for i, (g, w) in enumerate(zip(got, want)):
        g = g.cpu().numpy() if torch.is_tensor(g) else np.asarray(g)
        assert np.array_equal(g, np.asarray(w)), i


@pytest.mark.parametrize("lens,new,n_free,left", PLANS)
def test_the_plain_form_of_planning_is_the_definition(cases, lens, new, n_free, left):
    def state():
        table = np.full((len(lens), 5), -1)
        at = 10
        for b, n in enumerate(lens):
            for j in range(-(-n // 4)):
                table[b, j], at = at, at + 1
        return plan_state(lens, new, table.tolist(), [5, 3, 8, 1, 6, 2] + [-1] * 14, n_free, 4, sum(new) + 2)

    want = cases._exact_blocks(state())
    assert int(want[7][0]) == left
    equal(cases._plain_blocks(state()), want)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["blocks_step_b32", "blocks_prompts_b509", "blocks_release_b1000"])
@pytest.mark.parametrize("seed", [0, 1, 2, 16])
def test_the_frameworks_call_gives_the_definitions_numbers(cases, name, seed):
    case = next(c for c in cases.listed() if c["name"] == name)
    want = cases.exact(case, seed)
    cases.own = True
    try:
        equal(cases.run(cases.prepare(case, seed)), want)
    finally:
        cases.own = False
