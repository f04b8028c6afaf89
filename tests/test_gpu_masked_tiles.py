"""Windows and trees of batches of few rows to a sequence on average (16 heads counted, 8 at D = 64),
in which one sequence has many: its rows are several tiles of 32, a cached token's tile is read for
each, and a tree's lines begin in later tiles and cross words of 32 nodes."""

import pytest
import torch

import test_gpu_masked_attn as masked
from gpu_helpers import assert_no_device_error, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


def batch(singles, many, place, before):
    """`singles` sequences of one row, and one of `many` rows at `place` over `before` tokens."""
    new = [1] * singles
    past = [(37 * i) % 700 for i in range(singles)]
    new.insert(place, many)
    past.insert(place, before)
    return tuple(new), tuple(past)


TILES = [
    # singles, rows, place, tokens before, D, G, PS, shares
    (60, 200, 60, 1400, 128, 1, 16, 0),
    (60, 200, 7, 127, 128, 2, 32, 5),
    (60, 200, 0, 0, 64, 1, 64, 0),
    (90, 200, 90, 900, 64, 2, 16, 9),
    (130, 97, 50, 333, 128, 8, 64, 0),
    (210, 33, 210, 31, 64, 8, 16, 3),
    (280, 1024, 100, 500, 128, 1, 16, 0),
    (280, 1024, 280, 0, 64, 1, 16, 0),
]


@pytest.mark.parametrize("singles,many,place,before,D,G,PS,shares", TILES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (300, 130), (10 ** 6, 0)])
def test_window_of_many_rows_among_single_ones(singles, many, place, before, D, G, PS, shares,
                                               window, sinks):
    new, past = batch(singles, many, place, before)
    masked.test_window(new, past, "bf16", D, G, PS, shares, window, sinks)


@pytest.mark.parametrize("singles,many,place,before,D,G,PS,shares", TILES)
def test_tree_of_many_nodes_among_single_rows(singles, many, place, before, D, G, PS, shares):
    new, past = batch(singles, many, place, before)
    masked.test_tree(new, past, "bf16", D, G, PS, shares)


@pytest.mark.parametrize("D,G", [(128, 2), (64, 1)])
def test_a_long_line_among_single_rows(D, G):
    """Every word of a row's ancestors full: each row sees all before it."""
    new, past = batch(130 * G, 600, 20, 77)
    c = masked.Masked(new, past, "bf16", D, G, parents=[masked.line(n) for n in new])
    out, lse = c.attend()
    assert_no_device_error()
    c.check_attn(c.q, out, lse)
    for _ in range(5):
        again, lse2 = c.attend()
        assert torch.equal(again, out) and torch.equal(lse2, lse)
