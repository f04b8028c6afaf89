"""Page tables over the whole range of rows, and rows whose length is none."""

import os
import random
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
for rows in (4061, 4062, 4096, 4097, 16384):
    p = Pool(5 * rows, 4)
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


@pytest.mark.parametrize("pages,stride,PS,seed", [(1000, 30, 16, 1), (5003, 130, 64, 2),
                                                  (129, 9, 32, 3), (70001, 1100, 16, 4)])
def test_random_steps_that_fork_drop_and_slide(pages, stride, PS, seed):
    """Steps that the pool has room for, but for a few, and of every kind."""
    rng = random.Random(seed)
    p = Pool(pages, stride, PS)
    p.step([min(stride * PS, 20 * PS) // 2] * 4, parents=[-1] * 4, keep=[0] * 4)
    kinds = {"refused": 0, "copied": 0, "dropped": 0, "slid": 0, "freed": 0}
    for n in range(30):
        grow = n % 3 != 2                            # every third step keeps the rows as they are
        rows = rng.choice((2, 5, 9)) if grow else len(p.lens)
        parents = [rng.randrange(len(p.lens)) for _ in range(rows)] if grow else None
        if grow and n % 5 == 0:
            parents[-1] = -1
        old = p.lens if parents is None else [p.lens[q] if q >= 0 else 0 for q in parents]
        keep = [max(0, x - rng.choice((0, 0, 1, 3, PS))) for x in old]
        most = min(stride * PS, max(PS, pages * PS // (2 * rows)))
        want = [min(stride * PS, max(k, min(most, k + rng.choice((1, 2, 7, 2 * PS))))) for k in keep]
        window, sinks = (3 * PS, 4) if n % 4 == 3 else (0, 0)
        args = (p.lens, p.refs.tolist(), rows, parents, keep, want, PS)
        out, _, copies, left = oracle.update_pages(p.table, *args, window, sinks)
        bare, *_ = oracle.update_pages(p.table, *args)
        kinds["refused"] += left < 0
        kinds["copied"] += bool((copies >= 0).any())
        kinds["dropped"] += any(-(-k // PS) < -(-x // PS) for k, x in zip(keep, old))
        kinds["slid"] += left >= 0 and bool(((out < 0) & (bare >= 0)).any())
        kinds["freed"] += parents is not None and len(set(parents)) < len(p.lens)
        p.step(want, keep=keep, parents=parents, window=window, sinks=sinks,
               flags=32 if left < 0 else 0)
        p.check_counts()
    assert kinds["refused"] <= 5, kinds
    assert min(kinds[k] for k in ("copied", "dropped", "slid", "freed")) >= 3, kinds
