"""First calls of one kernel from several threads with different sizes, each of which
needs another amount of shared memory: every call, then and later, runs."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
from linear_attention_recurrence_gated_gb300 import gdn as G

def norm(C, groups):
    x = torch.randn(2, 64, C, device="cuda")
    y, mean, rstd = G.gdn_group_norm(x, None, None, groups)
    g = G.gdn_group_norm_bwd(x, None, None, groups, mean, rstd, x)
    return [y, *[t for t in g.values() if t is not None]]

def scan(d):
    q = torch.randn(1, 100, 2, d, device="cuda")
    return list(G.gdn_lin_fwd(q, q, q, torch.zeros(2, device="cuda")))

jobs = [lambda: norm(1024, 16), lambda: norm(8192, 16), lambda: norm(4096, 8), lambda: norm(64, 1),
        lambda: scan(160), lambda: scan(256), lambda: scan(192), lambda: scan(224)]
torch.zeros(1, device="cuda")
failed, start = [], threading.Barrier(len(jobs))

def work(job):
    try:
        start.wait()
        for _ in range(3):
            assert all(bool(torch.isfinite(t).all()) for t in job())
    except Exception as e:
        failed.append(repr(e))

threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
[t.start() for t in threads]
[t.join() for t in threads]
assert not failed, failed
"""


def test_threads_with_different_sizes():
    """In processes of their own: only a process's first calls set a limit."""
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True,
                           timeout=120, cwd=ROOT)
        assert r.returncode == 0, r.stderr[-1500:]
