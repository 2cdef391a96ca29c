"""Page calls whose bookkeeping is out of step (jobs that break a rule are left out and
recorded) and tables without rows.  Whole numbers: no tolerance."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G
from test_gpu_pages import dev

pytestmark = pytest.mark.gpu


def host(*tensors):
    return [t.cpu().numpy() for t in tensors]


def free(table, counts, refs, rows, in_place, P):
    t, c, r = dev(table), dev(counts), dev(refs)
    ws = torch.zeros(G.gdn_pages_workspace_size(P, len(counts), len(rows)), dtype=torch.uint8,
                     device="cuda")
    kw = dict(table_out=t, counts_out=c, refs_out=r) if in_place else {}
    out = G.gdn_pages_free(t, c, r, dev(rows), workspace=ws, **kw)
    return host(*out), G.gdn_check_record(ws)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_more", [0, 1500])
@pytest.mark.parametrize("bad", ["count below zero", "count too large", "page below zero",
                                 "page too large", "free page"])
def test_free_leaves_a_bad_job_out(in_place, bad, n_more):
    """The row of such a job keeps its count, its pages and their references; the other
    jobs run (also when there are more of them than one pass of the CTA takes)."""
    P, R, M = 4000, 1600, 3
    table, counts, refs = np.full((R, M), -1), np.zeros(R, int), np.zeros(P, int)
    for r in range(R):
        counts[r] = 1 + r % M
        table[r, : counts[r]] = 2 * r + np.arange(counts[r])
        np.add.at(refs, table[r, : counts[r]], 1)
    which = 5                                             # three pages
    if bad == "count below zero":
        counts[which] = -2
    elif bad == "count too large":
        counts[which] = M + 1
    elif bad == "page below zero":
        table[which, 1] = -1
    elif bad == "page too large":
        table[which, 1] = P
    else:
        refs[table[which, 1]] = 0
    rows = [3, which, 9] + list(range(20, 20 + n_more))
    (t, c, r), (st, job, _, _) = free(table, counts, refs, rows, in_place, P)
    assert (st, job) == (7, 1)
    for row in rows:
        if row != which:
            refs[table[row, : counts[row]]] -= 1
            table[row], counts[row] = -1, 0
    assert np.array_equal(t, table) and np.array_equal(c, counts) and np.array_equal(r, refs)
    # a bad job that is listed twice stays left out
    (t, c, r), (st, _, _, _) = free(table, counts, refs, [which, which], in_place, P)
    assert st == 7
    assert np.array_equal(t, table) and np.array_equal(c, counts) and np.array_equal(r, refs)


@pytest.mark.parametrize("in_place", [False, True])
def test_references_do_not_fall_below_zero(in_place):
    """Two rows hold a page that counts one: both rows give it back and are empty, its
    count ends at zero and the call says that something was wrong."""
    table = np.array([[4, 1], [4, 2], [4, 3]])
    counts, refs = np.array([2, 2, 2]), np.array([0, 1, 1, 1, 1, 0])
    (t, c, r), (st, job, _, _) = free(table, counts, refs, [0, 2], in_place, 6)
    assert st == 7 and job in (0, 1)
    assert np.array_equal(t, [[-1, -1], [4, 2], [-1, -1]]) and np.array_equal(c, [0, 2, 0])
    assert np.array_equal(r, [0, 0, 1, 0, 0, 0])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P", [12, 6000])
def test_compact_drops_a_free_page_that_a_row_names(in_place, P):
    """Rows 0 and 1 name page 1, which is free: another page moves there, and they must
    not come to share it.  Their entries become -1 and the call records the rule."""
    pool = torch.arange(P, dtype=torch.float32, device="cuda")[:, None].repeat(1, 4)
    table = np.full((4, 2), -1)
    table[0], table[1], table[2, 0], table[3, 0] = (0, 1), (1, 3), P - 1, P - 4
    counts, refs = np.array([2, 2, 1, 1]), np.zeros(P, int)
    refs[[0, 3, P - 1, P - 4]] = 1
    t, c, r = dev(table), dev(counts), dev(refs)
    ws = torch.zeros(G.gdn_pages_workspace_size(P, 4, 0), dtype=torch.uint8, device="cuda")
    kw = dict(table_out=t, refs_out=r) if in_place else {}
    num, t, r = G.gdn_pages_compact(pool, t, c, r, workspace=ws, **kw)
    st, row, _, _ = G.gdn_check_record(ws)
    assert st == 7 and row in (0, 1)
    t, r = host(t, r)
    assert num.item() == 4
    assert np.array_equal(t, [[0, -1], [-1, 3], [2, -1], [1, -1]])
    assert np.array_equal(np.flatnonzero(r), [0, 1, 2, 3])
    assert pool[:4, 0].tolist() == [0, P - 4, P - 1, 3]


def test_a_table_without_rows():
    """The reference counts come out as they went in; a pool with pages that no row names
    is compacted all the same."""
    P = 300
    pool = torch.arange(P, dtype=torch.float32, device="cuda")[:, None].repeat(1, 4)
    refs = np.zeros(P, int)
    refs[[7, 299]] = 2, 1
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table, counts = none.view(0, 3), none
    for _ in range(3):
        # what the allocator hands out next has been used for something else
        junk = [torch.full((P,), 77, dtype=torch.int32, device="cuda") for _ in range(6)]
        del junk
        fresh, t, c, r = G.gdn_pages_fork(pool, table, counts, dev(refs), none, none, check=True)
        assert fresh.numel() == 0 and t.shape == (0, 3) and c.shape == (0,)
        assert np.array_equal(host(r)[0], refs)
        junk = [torch.full((P,), 77, dtype=torch.int32, device="cuda") for _ in range(6)]
        del junk
        t, c, r = G.gdn_pages_free(table, counts, dev(refs), none, check=True)
        assert t.shape == (0, 3) and np.array_equal(host(r)[0], refs)
    r = dev(refs)
    _, _, _, same = G.gdn_pages_fork(pool, table, counts, r, none, none, refs_out=r, check=True)
    assert same is r and np.array_equal(host(r)[0], refs)
    num, t, r = G.gdn_pages_compact(pool, table, counts, dev(refs), check=True)
    assert num.item() == 2 and t.shape == (0, 3)
    assert host(r)[0].tolist() == [2, 1] + [0] * (P - 2)   # 7 and 299 move to 0 and 1
    assert pool[:2, 0].tolist() == [7, 299]
