"""Calls with stream=: the buffers that a call makes for itself are the stream's, whatever the
current stream still has to do with the memory or takes next."""

import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from sparse_kv_cache_build_gb300 import inputs

from gpu_helpers import assert_no_device_error, need_gpu, workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


@pytest.fixture(scope="module")
def cache(_gpu):
    w = workload(num_q_heads=16, num_kv_heads=4, head_dim=128, page_size=16, dtype="bf16", seed=5,
                 seq_lens=(2000, 1500, 33), planted=8)
    c = inputs.make_cache(w, "cuda")
    kv = skv.PagedKV.from_cache(c)
    stats = skv.kv_build_page_stats(kv)
    scores = skv.kv_score_pages(kv, c.q, stats)
    k = 32
    idx, cnt = skv.kv_select_topk(scores, c.seq_lens, 16, budget_pages=k, k_max=k)
    moments = skv.kv_entmax_page_moments(kv, c.q, stats, w.sm_scale)
    part = skv.kv_sparse_decode_attn(kv, c.q, w.sm_scale, idx, cnt, num_splits=3)
    return dict(c=c, kv=kv, stats=stats, scores=scores, idx=idx, cnt=cnt, moments=moments,
                part=part, scale=w.sm_scale, k=k)


CALLS = {
    "build_page_stats": lambda x, s: skv.kv_build_page_stats(x["kv"], stream=s),
    "build_page_stats_fp8": lambda x, s: skv.kv_build_page_stats_fp8(x["kv"], stream=s),
    "score_pages": lambda x, s: skv.kv_score_pages(x["kv"], x["c"].q, x["stats"], stream=s),
    "select_topk": lambda x, s: skv.kv_select_topk(x["scores"], x["c"].seq_lens, 16,
                                                   budget_pages=x["k"], k_max=x["k"], stream=s),
    "score_select": lambda x, s: skv.kv_score_select(x["kv"], x["c"].q, x["stats"],
                                                     budget_pages=x["k"], k_max=x["k"], stream=s),
    "sparse_decode_attn": lambda x, s: skv.kv_sparse_decode_attn(
        x["kv"], x["c"].q, x["scale"], x["idx"], x["cnt"], num_splits=3, stream=s),
    "select_decode_attn": lambda x, s: skv.kv_select_decode_attn(
        x["kv"], x["c"].q, x["scale"], x["scores"], budget_pages=x["k"], num_splits=3, stream=s),
    "decode_attn_merge": lambda x, s: skv.kv_decode_attn_merge(x["kv"], x["c"].q, x["scale"],
                                                               num_splits=3, stream=s),
    "merge_splits": lambda x, s: skv.kv_merge_splits(*x["part"], stream=s),
    "dropped_mass": lambda x, s: skv.kv_dropped_mass(x["kv"], x["c"].q, x["scale"], x["idx"],
                                                     x["cnt"], stream=s),
    "decode_step": lambda x, s: skv.kv_decode_step(x["kv"], x["c"].q, x["scale"], x["stats"],
                                                   budget_pages=x["k"], stream=s),
    "decode_step dense": lambda x, s: skv.kv_decode_step(x["kv"], x["c"].q, x["scale"], stream=s),
    "entmax_page_moments": lambda x, s: skv.kv_entmax_page_moments(
        x["kv"], x["c"].q, x["stats"], x["scale"], stream=s),
    "entmax_select": lambda x, s: skv.kv_entmax_select(*x["moments"], x["c"].seq_lens, 16, 4,
                                                       stream=s),
    "entmax_decode_attn": lambda x, s: skv.kv_entmax_decode_attn(x["kv"], x["c"].q, x["scale"],
                                                                 stream=s),
    "entmax_decode_step": lambda x, s: skv.kv_entmax_decode_step(
        x["kv"], x["c"].q, x["scale"], x["stats"], stream=s),
}
# slots that a call leaves as they were made: pages of nobody, entries past the count
LEFT = {"build_page_stats", "build_page_stats_fp8", "score_pages", "score_select", "select_topk",
        "entmax_page_moments", "entmax_select"}


def tensors(got):
    return list(got) if isinstance(got, tuple) else [got]


def written(x, name, outs):
    """The part of a call's outputs that the call defines."""
    if name not in LEFT:
        return outs
    pages = [int(-(-n // 16)) for n in x["c"].seq_lens.tolist()]
    mapped = torch.cat([x["c"].page_table[b, :n] for b, n in enumerate(pages)]).long()
    keep = []
    for t in outs:
        if name.startswith("build"):
            keep.append(t[mapped])
        elif t.dim() == 3 and t.dtype == torch.int32:          # lists: up to their counts
            cnt = next(c for c in outs if c.dim() == 2 and c.dtype == torch.int32).tolist()
            keep.append(torch.cat([t[b, g, :n] for b, row in enumerate(cnt)
                                   for g, n in enumerate(row)]))
        elif t.dim() == 3:                                     # a value per page
            keep.append(torch.cat([t[b, :, :n].flatten() for b, n in enumerate(pages)]))
        else:
            keep.append(t)
    return keep


@pytest.mark.parametrize("name", CALLS)
def test_a_call_s_own_buffers_are_its_stream_s(cache, name):
    call = CALLS[name]
    first = tensors(call(cache, None))
    want = [t.clone() for t in written(cache, name, first)]
    sizes = [t.numel() * t.element_size() for t in first] + [1 << 16, 1 << 20, 1 << 21]
    del first
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        junk = [torch.empty((n,), dtype=torch.uint8, device="cuda") for n in sizes * 2]
        torch.cuda._sleep(6_000_000)
        for t in junk:                          # freed with this stream's writes still to come
            t.fill_(255)
        del junk, t
        got = tensors(call(cache, s))
        torch.cuda.synchronize()
        assert_no_device_error()
        got = written(cache, name, got)
        assert len(got) == len(want)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_a_step_graph_is_made_after_the_current_stream_s_writes():
    """Creation runs the step once: on the lengths that the current stream was about to write."""
    w = workload(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, dtype="bf16", seed=6,
                 seq_lens=(500, 300))
    c = inputs.make_cache(w, "cuda")
    kv = skv.PagedKV.from_cache(c)
    stats = skv.kv_build_page_stats(kv)
    want, _ = skv.kv_decode_step(kv, c.q, w.sm_scale, stats, budget_pages=8)
    lens = c.seq_lens.clone()
    for _ in range(3):
        c.seq_lens.fill_(-5)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        c.seq_lens.copy_(lens)
        g = skv.DecodeStepGraph(kv, c.q, w.sm_scale, stats, budget_pages=8)
        out, _ = g.launch()
        assert_no_device_error()
        assert torch.equal(out, want)
        g.close()


def test_a_call_on_the_capturing_stream_given_by_argument(cache):
    q, scale, kv = cache["c"].q, cache["scale"], cache["kv"]
    want = skv.kv_decode_step(kv, q, scale)
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    rows = skv.kv_prefill_attn(kv, q, scale, cu_tokens=cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = torch.cuda.current_stream()
        got = skv.kv_decode_step(kv, q, scale, stream=s)
        got_rows = skv.kv_prefill_attn(kv, q, scale, cu_tokens=cu, stream=s)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert_no_device_error()
        for a, b in zip(got + got_rows, want + rows):
            assert torch.equal(a, b)
