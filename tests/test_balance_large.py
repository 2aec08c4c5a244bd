"""The balance loss and its gradient at sizes where the work per CTA grows: more
tokens than the forward pass has chunks of the least size (592), more than the
backward pass has warps' least steps (9,472), and more chunks than the finishing
kernel adds in one pass (256)."""
import numpy as np
import pytest
import torch

import test_balance as tb

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_mixture_experts_top_b200 as m
    return m


def rel_tol(lg):
    """test_balance's bound, for all rows at once. Its chains: a lane adds at most
    32 exponentials, 5 more steps join the lanes; a warp adds chunk / 8 tokens
    (T / 4736 at most: 149 for 700,001, shared by its 16 groups), then 8 warps, 10
    chunks, 16 groups and 2 steps: fewer than 256 additions throughout."""
    x = lg.astype(np.float64)
    hi = np.where(np.isfinite(x), x, -np.inf).max(1)
    lo = np.where(np.isfinite(x), x, np.inf).min(1)
    spread = max(0.0, float((hi - lo).max()))
    return (2 * (2 + 1.7 * spread) + 128 + 8) * 2.0 ** -23


# narrow and wide rows, in vectors of four and in single values: T is past
# 592 and 9,472 least steps of that shape, and no multiple of a step
SIZES = [(65521, 256, 8), (700001, 8, 2), (80021, 64, 6), (40003, 33, 5), (20011, 511, 7),
         (10007, 1001, 3), (11003, 1024, 4)]


def test_the_sizes_are_past_the_least_chunks():
    for T, E, _ in SIZES:
        vec = 4 if E % 4 == 0 else 1
        lanes = min(32, max(1 << max(0, (-(-E // vec) - 1).bit_length()), 2 if vec == 4 else 8))
        if vec == 1:
            lanes = 8 if E <= 8 else 32
        n = vec
        while lanes * n < E:
            n *= 2
        un = 4 if n <= 8 else 2 if n <= 16 else 1
        least = 32 // lanes * un
        assert T > 592 * 8 * least and T > 148 * 8 * 8 * least, (T, E, least)


@gpu
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("seqs,masked", [(1, False), (13, True)])
def test_large_batches(moe, monkeypatch, T, E, k, seqs, masked):
    monkeypatch.setattr(tb, "rel_tol", rel_tol)
    tb.check(moe, *tb._with(tb.inputs(T, E, k, T + E, seqs, masked), 0.01),
             dloss=None if masked else -2.5)


@gpu
def test_a_sequence_in_the_middle_of_many_chunks(moe, monkeypatch):
    """Sequences that start and end inside chunks, some within one, some over
    hundreds, with empty ones between."""
    monkeypatch.setattr(tb, "rel_tol", rel_tol)
    T, E, k = 65521, 256, 8
    lg, idx, mask, _ = tb.inputs(T, E, k, 3, 1, True)
    off = torch.tensor([5, 6, 6, 117, 222, 41000, 41000, 41001, 65500], dtype=torch.int32)
    tb.check(moe, lg, idx, 0.5, mask, off)
