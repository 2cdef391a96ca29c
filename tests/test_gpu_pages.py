"""GPU tests of the pages of a state cache: every result equals the host
bookkeeping of oracle/lin.py (whole numbers and copied bytes: no tolerance)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G
from oracle import lin

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def state(P, R, M, live, seed=0, page=(3, 16), dtype=torch.float32):
    """A pool with ``live`` rows that share snapshots, pages in random order."""
    r = np.random.default_rng(seed)
    order = list(r.permutation(P))
    table, counts, refs = np.full((R, M), -1), np.zeros(R, int), np.zeros(P, int)
    rows = r.permutation(R)
    shared = []
    for i in range(live):
        if i % 3 == 0:
            shared = [order.pop() for _ in range(r.integers(0, M))]
        mine = shared[: r.integers(0, len(shared) + 1)] + [order.pop()]
        table[rows[i], : len(mine)] = mine
        counts[rows[i]] = len(mine)
        np.add.at(refs, mine, 1)
    pool = torch.from_numpy(r.standard_normal((P, *page))).to(dtype).cuda()
    return pool, table, counts, refs, rows


def same(host, table, counts, refs, pool=None):
    assert np.array_equal(table.cpu().numpy(), host.table)
    assert np.array_equal(counts.cpu().numpy(), host.counts)
    assert np.array_equal(refs.cpu().numpy(), host.refs)
    if pool is not None:
        assert np.array_equal(pool.float().cpu().numpy(), host.pool)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P,R,M,live,n", [(40, 12, 3, 5, 4), (300, 80, 5, 40, 30),
                                          (9000, 4000, 2, 1500, 1300), (5000, 3000, 8, 10, 2500)])
@pytest.mark.parametrize("dtype,page", [(torch.float32, (3, 16)), (torch.bfloat16, (8,))])
def test_fork(in_place, P, R, M, live, n, dtype, page):
    pool, table, counts, refs, rows = state(P, R, M, live, seed=P, page=page, dtype=dtype)
    r = np.random.default_rng(1)
    parents = rows[r.integers(0, live, n)].copy()
    children = rows[live: live + n].copy()
    parents[::7] = -1                                  # new rows
    parents[1] = rows[-1]                               # an empty parent
    if n > 20:
        seen = set()
        for i in range(2, n, 9):                        # snapshots
            if parents[i] >= 0 and parents[i] not in seen:
                seen.add(parents[i])
                children[i] = parents[i]
    host = lin.Pages(table, counts, refs, pool.float().cpu().numpy())
    fresh_ref = host.fork(parents.tolist(), children.tolist())
    t, c, rf = dev(table), dev(counts), dev(refs)
    ws = torch.zeros(G.gdn_pages_workspace_size(P, R, n), dtype=torch.uint8, device="cuda")
    kw = dict(table_out=t, counts_out=c, refs_out=rf) if in_place else {}
    fresh, t2, c2, r2 = G.gdn_pages_fork(pool, t, c, rf, dev(parents), dev(children), workspace=ws,
                                         **kw)
    st = G.gdn_check(ws)
    assert st == (8 if host.short else 7 if host.bad else 0) or (host.bad and host.short)
    assert np.array_equal(fresh.cpu().numpy(), fresh_ref)
    same(host, t2, c2, r2, pool)
    if not in_place:
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(rf.cpu().numpy(), refs)


def test_fork_leaves_bad_jobs_out():
    pool, table, counts, refs, rows = state(60, 20, 3, 8, seed=3)
    empty = rows[8:]
    full = next((r for r in rows[:8] if counts[r] == 3), None)
    parents = [rows[0], 99, -2, rows[1], rows[2], rows[3], rows[0]]
    children = [rows[1], empty[0], empty[1], 20, -1, empty[2], empty[2]]
    if full is not None:
        parents.append(full)
        children.append(full)
    host = lin.Pages(table, counts, refs, pool.cpu().numpy())
    ref = host.fork(parents, children)
    ws = torch.zeros(G.gdn_pages_workspace_size(60, 20, len(parents)), dtype=torch.uint8,
                     device="cuda")
    fresh, t, c, r = G.gdn_pages_fork(pool, dev(table), dev(counts), dev(refs), dev(parents),
                                      dev(children), workspace=ws)
    st, job, _, _ = G.gdn_check_record(ws)
    assert st == 7 and job in host.bad
    assert np.array_equal(fresh.cpu().numpy(), ref)
    same(host, t, c, r, pool)


def test_fork_without_enough_pages():
    pool, table, counts, refs, rows = state(16, 30, 1, 13, seed=4)
    parents, children = rows[:6].tolist(), rows[13:19].tolist()
    host = lin.Pages(table, counts, refs, pool.cpu().numpy())
    ref = host.fork(parents, children)
    assert host.short and (ref >= 0).sum() == 3
    ws = torch.zeros(G.gdn_pages_workspace_size(16, 30, 6), dtype=torch.uint8, device="cuda")
    fresh, t, c, r = G.gdn_pages_fork(pool, dev(table), dev(counts), dev(refs), dev(parents),
                                      dev(children), workspace=ws)
    assert G.gdn_check(ws) == 8
    assert np.array_equal(fresh.cpu().numpy(), ref)
    same(host, t, c, r, pool)
    with pytest.raises(G.GdnError) as e:
        G.gdn_pages_fork(pool, t, c, r, dev(parents[:1]), dev(children[-1:]), check=True)
    assert e.value.status == 8


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P,R,M,live,n", [(40, 12, 3, 8, 3), (900, 300, 4, 200, 200),
                                          (9000, 4000, 2, 2500, 1200), (70000, 3000, 3, 2000, 900)])
def test_free_and_compact(in_place, P, R, M, live, n):
    pool, table, counts, refs, rows = state(P, R, M, live, seed=P + 1)
    gone = np.random.default_rng(2).permutation(rows[:live])[:n].tolist()
    gone += gone[:1] + [rows[-1]]                       # listed twice; an empty row
    host = lin.Pages(table, counts, refs, pool.cpu().numpy())
    host.free(gone)
    t, c, r = dev(table), dev(counts), dev(refs)
    kw = dict(table_out=t, counts_out=c, refs_out=r) if in_place else {}
    t, c, r = G.gdn_pages_free(t, c, r, dev(gone), check=True, **kw)
    same(host, t, c, r)
    live_ref = host.compact()
    kw = dict(table_out=t, refs_out=r) if in_place else {}
    num, t, r = G.gdn_pages_compact(pool, t, c, r, check=True, **kw)
    assert num.item() == live_ref
    same(host, t, c, r, pool)
    before = pool.clone()
    num, t, r = G.gdn_pages_compact(pool, t, c, r, check=True)   # nothing left to move
    assert num.item() == live_ref and torch.equal(pool, before)
    same(host, t, c, r)


def test_free_reports_bad_rows():
    pool, table, counts, refs, rows = state(40, 12, 3, 8, seed=5)
    host = lin.Pages(table, counts, refs)
    host.free([rows[0], 12, -1])
    ws = torch.zeros(G.gdn_pages_workspace_size(40, 12, 3), dtype=torch.uint8, device="cuda")
    t, c, r = G.gdn_pages_free(dev(table), dev(counts), dev(refs), dev([rows[0], 12, -1]),
                               workspace=ws)
    st, job, _, _ = G.gdn_check_record(ws)
    assert st == 7 and job in host.bad
    same(host, t, c, r)


@pytest.mark.parametrize("page", [(4,), (5, 1024), (2, 70000)])
def test_copy(page):
    r = np.random.default_rng(6)
    pool = torch.randn(30, *page, device="cuda")
    order = r.permutation(30)
    src, dst = order[r.integers(0, 12, 15)], order[12:27]
    want = pool.clone()
    want[torch.tensor(dst.copy())] = want[torch.tensor(src.copy())]
    src2, dst2 = [*src, 30, 3, order[27]], [*dst, order[28], -1, order[27]]
    ws = torch.zeros(G.gdn_pages_workspace_size(30, 0, len(src2)), dtype=torch.uint8, device="cuda")
    G.gdn_pages_copy(pool, dev(src2), dev(dst2), workspace=ws)
    st, job, _, _ = G.gdn_check_record(ws)
    assert st == 7 and job in (15, 16)
    assert torch.equal(pool, want)
    G.gdn_pages_copy(pool, dev(src), dev(dst), check=True)
    assert torch.equal(pool, want)
    G.gdn_pages_copy(pool, dev([]), dev([]), check=True)


def test_past_32_bits():
    """Pages that start beyond 4 GB."""
    P, n = 72, 1 << 26
    pool = torch.empty(P, n, dtype=torch.uint8, device="cuda")
    pool[0], pool[70], pool[71] = 1, 2, 3
    G.gdn_pages_copy(pool, dev([70, 0]), dev([5, 71]), check=True)
    assert (pool[5] == 2).all() and (pool[71] == 1).all() and (pool[70] == 2).all()
    table, counts, refs = np.full((3, 1), -1), np.array([1, 0, 0]), np.zeros(P, int)
    table[0, 0] = 70
    refs[70] = 1
    num, t, r = G.gdn_pages_compact(pool, dev(table), dev(counts), dev(refs), check=True)
    assert num.item() == 1 and t[0, 0].item() == 0 and (pool[0] == 2).all()
