"""Free and compact over pools, tables and lists of odd sizes, some longer than one CTA
holds at a time; with new bookkeeping, in place, and partly in place.  Whole numbers
and copied bytes: no tolerance."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G
from oracle import lin
from test_gpu_pages import dev, same, state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("place", ["new", "all", "refs", "table"])
@pytest.mark.parametrize("P,R,M,live,n", [(7, 3, 1, 2, 1), (1023, 77, 5, 60, 41),
                                          (1025, 129, 3, 100, 99), (4097, 1001, 3, 700, 301),
                                          (10001, 2001, 3, 1500, 700), (4099, 5, 2, 5, 0)])
def test_free_then_compact(place, P, R, M, live, n):
    pool, table, counts, refs, rows = state(P, R, M, live, seed=P + R, page=(4,))
    gone = rows[:n].astype(int)
    host = lin.Pages(table, counts, refs, pool.cpu().numpy())
    host.free(gone.tolist())
    t, c, rf = dev(table), dev(counts), dev(refs)
    own = dict(table_out=t, counts_out=c, refs_out=rf)
    keep = {"new": (), "all": own, "refs": ("refs_out",), "table": ("table_out",)}[place]
    kw = {name: own[name] for name in keep}
    t, c, rf = G.gdn_pages_free(t, c, rf, dev(gone), check=True, **kw)
    same(host, t, c, rf)
    own = dict(table_out=t, refs_out=rf)
    kw = {name: own[name] for name in keep if name in own}
    want = host.compact()
    num, t, rf = G.gdn_pages_compact(pool, t, c, rf, check=True, **kw)
    assert int(num) == want
    same(host, t, c, rf)
    assert np.array_equal(pool[:want].cpu().numpy(), host.pool[:want])
