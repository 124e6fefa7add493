"""GPU tests of page plans with more new tokens than places for them: the table, lengths and counts cover all tokens, listed or not."""

import numpy as np
import pytest
import torch

import mx_bit_quantized_amd as mxq
import oracle
from test_gpu_attn import DEV, I32, ints, say, table_of

pytestmark = pytest.mark.gpu

CASES = [  # cached, added, width, free, page
    ([0], [100], 7, 7, 16),
    ([5, 16, 0, 33], [40, 0, 33, 15], 5, 20, 16),
    ([15, 31], [1, 1], 2, 4, 16),                       # no new page
    ([16, 0, 0, 7], [17, 0, 1, 200], 9, 6, 16),         # the list is used up
    ([100, 0], [500, 77], 8, 30, 32),                   # past the table
    ([-3, 9], [20, -8], 3, 9, 16),
    ([0] * 300 + [7] * 300, [19, 0, 3] * 200, 3, 800, 16),
    ([i * 37 % 90 for i in range(4096)], [i * 13 % 70 for i in range(4096)], 11, 12000, 16),
    ([], [], 3, 2, 16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("listed", [0.0, 0.01, 0.5, 0.99, 1.0])
def test_page_plan_lists_a_part(case, listed):
    cached, added, width, free, page = CASES[case]
    table, pages = table_of(cached, width, page, free, case)
    tokens = int(listed * sum(max(n, 0) for n in added))
    say("plan in part", case, len(cached), tokens)
    t = torch.tensor(table, dtype=I32, device=DEV).view(len(cached), width)
    got = mxq.page_plan(ints(cached), ints(added), t, ints(pages), page, tokens)
    want = oracle.page_plan(cached, added, table, pages, page, tokens)
    for name, g, w in zip(mxq.PagePlan._fields, got, want):
        assert g.cpu().tolist() == list(w), name
    assert np.array_equal(t.cpu().numpy(), want[5])


def test_page_plan_most_tokens():
    """Nearly 2^31 new tokens, a few of them listed, of requests whose tables hold a few pages."""
    say("most tokens")
    requests, width, page, tokens = 3, 4, 16, 70
    added = [(1 << 29) + 5, 1 << 29, (1 << 30) - 100]
    table = torch.full((requests, width), -1, dtype=I32, device=DEV)
    free = list(range(100, 111))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    mxq.page_plan(ints([0]), ints([1]), torch.zeros(1, 1, dtype=I32, device=DEV), ints([1]), page, 1)
    cached, new, pages = ints([0, 20, 0]), ints(added), ints(free)
    torch.cuda.synchronize()
    begin.record()
    got = mxq.page_plan(cached, new, table, pages, page, tokens)
    end.record()
    torch.cuda.synchronize()
    assert table.tolist() == [[100, 101, 102, 103], [-1, -1, 104, 105], [106, 107, 108, 109]]
    assert got.slots.tolist() == [1600 + i for i in range(64)] + [-1] * 6 and got.positions.tolist() == list(range(70))
    assert got.starts.tolist() == [0, added[0], added[0] + added[1], sum(added)]
    assert got.lengths.tolist() == [added[0], added[1] + 20, added[2]]
    # request 1 has 12 tokens on an old page that its table lacks, 32 on new ones
    assert got.taken.tolist() == [10, added[0] - 64 + added[1] - 32 + added[2] - 64]
    # (token by token it took 1.7 s: the work goes by the listed tokens and the pages)
    assert begin.elapsed_time(end) < 100.0, "milliseconds"
