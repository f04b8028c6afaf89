"""Page tables over the whole range of rows, and rows whose length is none."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from oracle import pages as oracle

from gpu_helpers import need_gpu
from test_gpu_pages import Pool, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


ROWS = """
from test_gpu_pages import Pool
for rows in (4061, 4062, 4096, 4097):
    p = Pool(20000, 4)
    p.step([20, 33, 48], parents=[-1] * 3, keep=[0] * 3)
    held = [(20, 33, 48)[i % 3] for i in range(rows)]
    p.step([n + i % 2 for i, n in enumerate(held)], parents=[i % 3 for i in range(rows)], keep=held)
    p.check_counts()
    p.step([n + 1 for n in p.lens])
    p.check_counts()
"""


def test_rows_about_the_shared_memory_a_launch_has_by_default():
    """Three numbers a row pass 48 KB with the kernel's own at 4062 rows, without them at 4097. In a
    process of its own: a call with more rows raises the limit for those that follow."""
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([here, os.path.dirname(here)])
    run = subprocess.run([sys.executable, "-c", ROWS], cwd=here, capture_output=True, text=True,
                         timeout=300, env={**os.environ, "PYTHONPATH": path})
    assert run.returncode == 0, run.stderr[-2000:]


@pytest.mark.parametrize("bad", [-1, 161, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("parents", [None, [1, 0, 1], [1, -1, 2]])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("window", [0, 8])
def test_rows_of_a_length_that_does_not_fit_keep_their_pages(bad, parents, given, window):
    """An old row whose own length is none: nothing of it is given back, nothing is added."""
    p = Pool(50, 10)
    p.step([40, 50, 30], parents=[-1] * 3, keep=[0] * 3)
    p.kv.seq_lens[1] = bad
    old = list(range(3)) if parents is None else parents
    keep = [0 if q < 0 else (40, 50, 30)[q] for q in old]
    want = [n + 20 for n in keep]
    # as the oracle sees it: the row is full to the end of its pages and does not grow. (The window
    # it would have given pages back for, row by row.)
    whole = [64 if q == 1 else n for q, n in zip(old, keep)]
    ref = oracle.update_pages(p.table, [40, 64, 30], p.refs.tolist(), 3, parents, whole,
                              [64 if q == 1 else n for q, n in zip(old, want)], 16)
    table, copies, left = skv.kv_update_pages(
        p.kv, p.refs, ints(want), window=window,
        keep_lens=ints(keep) if given or parents is not None else None,
        parents=None if parents is None else ints(parents))
    assert skv.kv_check_device_errors() == (-5, 2)
    got = table.cpu().numpy()
    for b, q in enumerate(old):
        if q == 1:
            assert np.array_equal(got[b], p.table[1]) and copies[b].tolist() == [-1, -1]
    used = got[got >= 0]
    assert np.array_equal(np.bincount(used, minlength=50), p.refs.cpu().numpy())
    if window == 0:
        assert np.array_equal(got, ref[0]) and p.refs.tolist() == ref[1]
        assert np.array_equal(copies.cpu().numpy(), ref[2]) and left.tolist() == [ref[3]]
