"""A speculative step captured as it is used: page table, page copies, append, verification,
compaction, the next page table, a token more and a window, each call launched while the one before
still runs. The same calls with a wait after each are the reference, bit by bit."""

import os
import random
import subprocess
import sys

import pytest
import torch

import sparse_kv_cache_build_gb300 as skv

from gpu_helpers import assert_no_device_error, need_gpu
from test_gpu_drafts_loop import tree_of
from test_gpu_pages import ints
from test_gpu_prompt import DT, freqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


class Step:
    """The state before a step of a batch whose rows fork, and everything the step writes."""

    def __init__(self, dtype, D, HKV, G, PS, rows, most, seed):
        rng = random.Random(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        old = max(1, rows // 2)
        past = [rng.randrange(1, 900) for _ in range(old)]
        parents = [rng.randrange(-1, old) for _ in range(rows)]
        keep = [max(0, past[p] - rng.choice((0, 0, 3))) if p >= 0 else 0 for p in parents]
        trees = [tree_of(rng, rng.randrange(1, most + 1)) for _ in range(rows)]
        drafts = [len(up) for up, _ in trees]
        T, D2 = sum(drafts), (HKV * G + 2 * HKV, D)
        stride = 1000 // PS + 2
        NP = (old + rows) * stride
        self.window, self.sinks, self.scale = 3 * PS + 5, 4, D ** -0.5

        def rand(*shape):
            return torch.randn(shape, generator=gen, device="cuda").to(DT[dtype])

        k, v = rand(NP, HKV, PS, D), rand(NP, HKV, PS, D)
        table = torch.full((old, stride), -1, dtype=torch.int32)
        order = torch.randperm(NP, generator=gen, device="cuda").cpu()
        refs, at = torch.zeros(NP, dtype=torch.int32), 0
        for b, n in enumerate(past):
            pages = -(-n // PS)
            table[b, :pages] = order[at:at + pages]
            refs[order[at:at + pages]] = 1
            at += pages
        table = table.cuda()
        first = skv.PagedKV(k, v, table, ints(past))
        verified = [a + n for a, n in zip(keep, drafts)]
        kept = [sorted(rng.sample(range(n), rng.randrange(n + 1))) for n in drafts]
        most_kept = max(1, max(map(len, kept)))
        self.after = [a + len(x) for a, x in zip(keep, kept)]
        stats = skv.kv_build_page_stats(first)
        new = torch.full((rows, stride), -1, dtype=torch.int32, device="cuda")
        # what the step changes, kept to start it again
        self.state = [k, v, refs.cuda(), stats, new]
        self.start = [x.clone() for x in self.state]
        k, v, self.refs, self.stats, self.table = self.state
        self.first, self.parents, self.keep = first, ints(parents), ints(keep)
        self.verified = skv.PagedKV(k, v, new, ints(verified))
        self.grown = skv.PagedKV(k, v, new, ints([n + 1 for n in self.after]))
        self.cu = ints([sum(drafts[:b]) for b in range(rows + 1)])
        self.up = ints([p for up, _ in trees for p in up])
        self.depths = ints([a + d for a, (_, depth) in zip(keep, trees) for d in depth])
        self.kept = ints([x + [0] * (most_kept - len(x)) for x in kept])
        self.cnt = ints([len(x) for x in kept])
        self.turns = skv.kv_rope_turns(freqs(D), device="cuda")
        self.x = rand(T, *D2).split((HKV * G, HKV, HKV), dim=1)
        self.y = rand(rows, *D2).split((HKV * G, HKV, HKV), dim=1)

    def restore(self):
        for x, x0 in zip(self.state, self.start):
            x.copy_(x0)

    def run(self, then=lambda: None):
        table, copies, left = skv.kv_update_pages(
            self.first, self.refs, self.verified.seq_lens, keep_lens=self.keep,
            parents=self.parents, table=self.table)
        then()
        skv.kv_copy_pages(self.verified, copies, self.stats)
        then()
        q = skv.kv_append_rope(self.verified, *self.x, self.stats, self.turns, cu_tokens=self.cu,
                               positions=self.depths)
        then()
        tree, tree_lse = skv.kv_tree_attn(self.verified, q, self.scale, self.up, cu_tokens=self.cu)
        then()
        lens = skv.kv_compact(self.verified, self.kept, self.cnt, self.stats, cu_tokens=self.cu)
        then()
        _, copies2, left2 = skv.kv_update_pages(
            self.verified, self.refs, self.grown.seq_lens, keep_lens=lens, window=self.window,
            sinks=self.sinks)
        then()
        skv.kv_copy_pages(self.grown, copies2, self.stats)
        then()
        q1 = skv.kv_append_rope(self.grown, *self.y, self.stats, self.turns)
        then()
        out, lse = skv.kv_window_attn(self.grown, q1, self.scale, self.window, self.sinks)
        then()
        return [copies, left, q, tree, tree_lse, lens, copies2, left2, q1, out, lse]


STEPS = [
    # dtype, D, KV heads, G, PS, rows, most nodes
    ("bf16", 128, 8, 4, 16, 24, 3),       # keys in the tensor core's rows
    ("bf16", 128, 8, 4, 16, 24, 26),
    ("bf16", 64, 2, 8, 64, 7, 40),
    ("bf16", 64, 16, 1, 32, 64, 8),
    ("fp32", 128, 2, 4, 16, 24, 9),
    ("fp32", 64, 8, 2, 32, 5, 70),
]


@pytest.mark.parametrize("dtype,D,HKV,G,PS,rows,most", STEPS)
def test_a_captured_step_equals_its_calls_one_by_one(dtype, D, HKV, G, PS, rows, most):
    s = Step(dtype, D, HKV, G, PS, rows, most, seed=rows + most)
    ref = [x.clone() for x in s.run(then=torch.cuda.synchronize)]
    assert_no_device_error()
    assert ref[5].tolist() == s.after
    end = [x.clone() for x in s.state]
    s.restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = s.run()
    for _ in range(100):
        s.restore()
        graph.replay()
        for x, r in zip(outs + s.state, ref + end):
            # a page that nobody wrote may hold anything, NaN too: compared as bits
            assert torch.equal(x.view(torch.uint8), r.view(torch.uint8))
    assert_no_device_error()


FIRST = """
import torch
torch.cuda.set_device(0)
from test_gpu_captured_steps import STEPS, Step
for which in (0, 1, 5):
    s = Step(*STEPS[which], seed=3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = s.run()
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in outs + s.state]
    s.restore()
    ref = s.run(then=torch.cuda.synchronize) + s.state
    assert all(torch.equal(x.view(torch.uint8), r.view(torch.uint8)) for x, r in zip(got, ref))
"""


def test_calls_that_are_captured_before_they_ever_ran():
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([here, os.path.dirname(here)])
    run = subprocess.run([sys.executable, "-c", FIRST], cwd=here, capture_output=True, text=True,
                         timeout=300, env={**os.environ, "PYTHONPATH": path})
    assert run.returncode == 0, run.stderr[-2000:]
