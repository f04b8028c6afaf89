"""Page tables over the whole range of rows."""

import os
import subprocess
import sys

import pytest
import torch

from gpu_helpers import need_gpu

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
