"""Tables of a step: lengths whose sum saturates, in batches that a block scans in
one turn and in several, with new lengths beside the old ones and in place."""

import numpy as np
import pytest
import torch

import fp8_w8a8_static_b200 as fw
from test_gpu_fp4_kv import DEV, ints

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


def plain(lens, new, width, free, page, n_slots):
    """(cu_q, kv_lens, slots, pool, table) from a table of -2, whole numbers."""
    table = np.full((len(lens), width), -2, np.int64)
    cu, slots, taken = [0], [], 0
    for b, (o, a) in enumerate(zip(lens, new)):
        o, a = max(o, 0), max(a, 0)
        for j in range(min(-(-o // page), width), min(-(-(o + a) // page), width)):
            table[b, j] = free[taken] if taken < len(free) else -1
            taken += 1
        for pos in range(o, o + min(a, n_slots - len(slots))):
            p = table[b, pos // page] if pos // page < width else -1
            slots.append(p * page + pos % page if p >= 0 else -1)
        cu.append(min(cu[-1] + a, TOP))
    kv = [min(max(o, 0) + max(a, 0), TOP) for o, a in zip(lens, new)]
    got = min(taken, len(free))
    return cu, kv, slots + [-1] * (n_slots - len(slots)), [got, taken - got], table


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch", [1, 300, 1024, 1025, 3000])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("old,add", [(5, TOP), (40, TOP - 2), (TOP, TOP), (5, 70), (-3, 20)])
def test_lengths_whose_sum_saturates(old, add, where, batch, in_place):
    page, width, n_slots = 16, 6, 4000 + batch
    lens = [i % 40 for i in range(batch)]
    new = [(i + 1) % 3 for i in range(batch)]
    at = 0 if where == "first" else batch - 1
    lens[at], new[at] = old, add
    free = np.random.default_rng(batch).permutation(3 * batch + 5)
    want = plain(lens, new, width, free, page, n_slots)
    table = torch.full((batch, width), -2, dtype=torch.int32, device=DEV)
    t_lens, pool = ints(lens), ints([0, 0])
    out = (torch.empty(batch + 1, dtype=torch.int32, device=DEV),
           t_lens if in_place else torch.empty_like(t_lens),
           torch.empty(n_slots, dtype=torch.int64, device=DEV), pool)
    fw.fp4_kv_tables(t_lens, ints(new), table, ints(free.tolist()), pool, page, n_slots, out=out)
    for got, w in zip(out, want):
        assert got.tolist() == w
    assert np.array_equal(table.cpu().numpy(), want[4])
    if not in_place:
        assert t_lens.tolist() == lens
