"""Windows and sinks beyond 32 bits reach as far as the largest number that fits."""

import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from sparse_kv_cache_build_gb300 import binding

from gpu_helpers import assert_no_device_error, need_gpu
from test_gpu_masked_attn import Masked
from test_gpu_pages import Pool, ints

pytestmark = pytest.mark.gpu

FAR = [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70 + 5]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("far", FAR)
def test_windows_and_sinks_of_any_size(far):
    c = Masked((3, 2), (90, 40), window=5)
    whole = skv.kv_window_attn(c.kv, c.q, c.scale, 93, cu_tokens=c.cu)
    sinks = skv.kv_window_attn(c.kv, c.q, c.scale, 5, 93, cu_tokens=c.cu)
    for args, ref in (((far,), whole), ((5, far), sinks), ((far, far), whole)):
        out, lse = skv.kv_window_attn(c.kv, c.q, c.scale, *args, cu_tokens=c.cu)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    for args in ((-far,), (5, -far), (5 - 2 ** 32,)):
        with pytest.raises(binding.KVError):
            skv.kv_window_attn(c.kv, c.q, c.scale, *args, cu_tokens=c.cu)
    assert_no_device_error()


@pytest.mark.parametrize("far", FAR)
def test_tables_of_windows_of_any_size(far):
    for kw in (dict(window=far), dict(window=3, sinks=far)):
        p = Pool(30, 10)
        p.step([100], parents=[-1], keep=[0])
        table, _, left = skv.kv_update_pages(p.kv, p.refs, ints([101]), **kw)
        assert (table[0, :7] >= 0).all() and left.tolist() == [23]
    with pytest.raises(binding.KVError):
        skv.kv_update_pages(p.kv, p.refs, ints([101]), window=5 - 2 ** 32)
    assert_no_device_error()
