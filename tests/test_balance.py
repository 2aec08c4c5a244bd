"""The router's balance loss, its counts and its gradient: refusals on the CPU,
everything else against a plain 64-bit form on the GPU."""
import ctypes

import numpy as np
import pytest
import torch

import moe_inputs as mi

gpu = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_mixture_experts_top_b200 as m
    return m


def softmax64(x):
    with np.errstate(invalid="ignore"):
        m = x.max(1, keepdims=True)
        z = np.exp(x - np.where(np.isneginf(m), 0, m))
    s = z.sum(1, keepdims=True)
    return z / np.where(s == 0, 1, s)


def reference(logits, idx, coef, mask=None, off=None, dloss=1.0, counts=None):
    """loss, counts, probs, tokens and dlogits in fp64; `counts` given: held at
    those (the loss as a function of the logits alone)."""
    T, E = logits.shape
    k = idx.shape[1]
    off = [0, T] if off is None else list(off)
    B = len(off) - 1
    ok = np.ones(T, bool) if mask is None else mask
    c, P, n = np.zeros((B, E), np.int64), np.zeros((B, E)), np.zeros(B, np.int64)
    d, loss = np.zeros((T, E)), 0.0
    for b in range(B):
        t = np.arange(off[b], off[b + 1])
        t = t[ok[t]]
        n[b] = len(t)
        if not len(t):
            continue
        ids = idx[t].ravel()
        c[b] = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        cb = c[b] if counts is None else counts[b]
        p = softmax64(logits[t].astype(np.float64))
        P[b] = p.sum(0) / len(t)
        loss += coef / B * E / (k * len(t)) * (cb * P[b]).sum()
        f = dloss * coef / B * E / (k * len(t) ** 2)
        d[t] = f * p * (cb - (p @ cb)[:, None])
    return loss, c, P, n, d


def inputs(T, E, k, seed, seqs=1, masked=False):
    g = torch.Generator().manual_seed(seed)
    lg = torch.randn(T, E, generator=g) * 2 + torch.randn(1, E, generator=g)
    idx = lg.topk(k, 1).indices.int()
    mask = torch.rand(T, generator=g) < 0.7 if masked else None
    off = None
    if seqs > 1:
        off = torch.randint(0, T + 1, (seqs + 1,), generator=g).sort().values.int()
    return lg, idx, mask, off


def rel_tol(lg):
    """Relative error of a probability and of a sum of them. exp(x): its
    argument is rounded (|x| 2^-24) and the fast exponential is off by at most
    2 + 1.16 |x| units of 2^-23, |x| <= the row's spread; numerator and sum
    each have that; the sums over experts, tokens, warps and chunks are
    chains of fewer than 256 additions of values of one sign; 8 more for
    quotients and products."""
    spread = max([float(np.ptp(r[np.isfinite(r)])) for r in lg if np.isfinite(r).any()] or [0.0])
    return (2 * (2 + 1.7 * spread) + 128 + 8) * 2.0 ** -23


def check(moe, lg, idx, coef, mask=None, off=None, dloss=None):
    to = lambda t: None if t is None else t.to(DEV)      # noqa: E731
    gl, gi, gm, go = lg.to(DEV), idx.to(DEV), to(mask), to(off)
    s = moe.balance_loss(gl, gi, coef, gm, go)
    dl = None if dloss is None else torch.tensor(dloss, device=DEV)
    d = moe.balance_loss_backward(gl, s, idx.shape[1], coef, gm, go, dl)
    npy = lambda t: None if t is None else t.numpy()     # noqa: E731
    loss, c, P, n, rd = reference(lg.numpy(), idx.numpy(), coef, npy(mask), npy(off),
                                  1.0 if dloss is None else dloss)
    np.testing.assert_array_equal(s.counts.cpu().numpy(), c)
    np.testing.assert_array_equal(s.tokens.cpu().numpy(), n)
    used = lg.numpy() if mask is None else lg.numpy()[mask.numpy()]
    tol = rel_tol(used)
    assert (np.abs(s.probs.cpu().numpy() - P) <= tol * P + 1e-37).all()
    assert abs(float(s.loss) - loss) <= 2 * tol * abs(loss) + 1e-37
    # d = p (a - s): the difference of two values of at most max(a)
    got = d.double().cpu().numpy()
    for b in range(len(n)):
        lo, hi = (0, lg.shape[0]) if off is None else (int(off[b]), int(off[b + 1]))
        if not n[b]:
            assert (got[lo:hi] == 0).all()
            continue
        f = abs(1.0 if dloss is None else dloss) * coef / len(n) * lg.shape[1] / (idx.shape[1] * n[b] ** 2)
        p = softmax64(np.nan_to_num(lg.numpy()[lo:hi].astype(np.float64), nan=0.0))
        size = f * p * (c[b] + (p @ c[b])[:, None])
        assert (np.abs(got[lo:hi] - rd[lo:hi]) <= 3 * tol * size + 1e-37).all()
    if off is not None:                       # tokens of no sequence
        assert (got[:int(off[0])] == 0).all() and (got[int(off[-1]):] == 0).all()
    return s, d


# ------------------------------------------------------------------ CPU

def test_calls_refuse_bad_arguments_without_launching(moe):
    L, P = moe.lib, None
    p, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
    ARG, UNS = moe.ERR_INVALID_ARG, moe.ERR_UNSUPPORTED

    def f(lg=p, idx=p, off=P, T=4, E=8, k=2, B=1, loss=p, ws=p, n=1 << 30):
        return L.moe_balance_loss(lg, idx, P, off, T, E, k, B, 1.0, loss, p, p, p, ws, n, P)

    assert f(lg=P) == ARG and f(idx=P) == ARG and f(loss=P) == ARG and f(lg=odd) == ARG
    assert f(T=-1) == ARG and f(k=9) == ARG and f(k=0) == ARG and f(E=0) == ARG
    assert f(B=0) == ARG and f(B=2) == ARG            # several sequences without offsets
    assert f(E=2048) == UNS and f(E=64, k=33) == UNS and f(off=p, B=65537) == UNS
    assert f(T=9000, ws=P) == moe.ERR_WORKSPACE and f(T=9000, n=8) == moe.ERR_WORKSPACE
    assert f(T=9000, ws=odd) == moe.ERR_WORKSPACE and f(off=p, B=2, ws=P) == moe.ERR_WORKSPACE
    assert f(T=1 << 30, k=4) == UNS                   # T * k past 32 bits
    assert f(T=(1 << 30) + 1, k=1) == UNS
    assert L.moe_balance_loss_workspace(-1, 8, 1) == 0
    assert L.moe_balance_loss_workspace(4, 8, 1) == 0 < L.moe_balance_loss_workspace(4, 8, 2)

    def g(lg=p, c=p, n=p, d=p, T=4, B=1):
        return L.moe_balance_loss_backward(lg, P, P, T, 8, 2, B, 1.0, c, n, P, d, P)

    assert g(lg=P) == ARG and g(c=P) == ARG and g(n=P) == ARG and g(d=P) == ARG
    assert g(d=odd) == ARG and g(B=3) == ARG
    assert g(T=0, lg=P, c=P, n=P, d=P) == moe.OK


def test_reference_gradient_is_the_difference_quotient():
    lg, idx, mask, off = inputs(23, 7, 3, 1, seqs=3, masked=True)
    x, i, m, o = lg.double().numpy(), idx.numpy(), mask.numpy(), off.numpy()
    _, c, _, _, d = reference(x, i, 0.5, m, o)
    h = 1e-5
    for t in range(23):
        for e in range(7):
            y = x.copy()
            y[t, e] += h
            hi = reference(y, i, 0.5, m, o, counts=c)[0]
            y[t, e] -= 2 * h
            lo = reference(y, i, 0.5, m, o, counts=c)[0]
            assert abs((hi - lo) / (2 * h) - d[t, e]) < 1e-9


# ------------------------------------------------------------------ GPU

@gpu
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (16, 8, 2), (17, 33, 5), (64, 128, 8),
                                   (129, 100, 32), (1000, 256, 8), (513, 511, 7), (300, 1024, 16),
                                   (100, 1001, 3), (9000, 64, 6)])
@pytest.mark.parametrize("seqs,masked", [(1, False), (1, True), (5, True)])
def test_balance_loss_and_gradient(moe, T, E, k, seqs, masked):
    check(moe, *_with(inputs(T, E, k, T + E, seqs, masked), 0.01), dloss=None if masked else -2.5)


def _with(t, coef):
    return t[0], t[1], coef, t[2], t[3]


@gpu
def test_gradient_is_the_difference_quotient(moe):
    """The kernel's gradient against differences of the 64-bit loss."""
    lg, idx, mask, off = inputs(40, 12, 2, 4, seqs=2, masked=True)
    s = moe.balance_loss(lg.to(DEV), idx.to(DEV), 1.0, mask.to(DEV), off.to(DEV))
    d = moe.balance_loss_backward(lg.to(DEV), s, 2, 1.0, mask.to(DEV), off.to(DEV)).cpu().numpy()
    x, c, h = lg.double().numpy(), s.counts.cpu().numpy(), 1e-4
    for t in range(0, 40, 3):
        for e in range(12):
            v = []
            for sign in (1, -1):
                y = x.copy()
                y[t, e] += sign * h
                v.append(reference(y, idx.numpy(), 1.0, mask.numpy(), off.numpy(), counts=c)[0])
            # a central difference is off by h^2/6 times a third derivative below 1
            assert abs((v[0] - v[1]) / (2 * h) - d[t, e]) <= 2e-8 + 1e-5 * abs(d[t, e])


@gpu
def test_empty_masked_and_uncovered(moe):
    lg, idx, _, _ = inputs(50, 16, 4, 9)
    # nothing valid: zeros
    s, d = check(moe, lg, idx, 1.0, torch.zeros(50, dtype=torch.bool))
    assert float(s.loss) == 0 and (d == 0).all()
    # an empty sequence, tokens before the first and behind the last
    check(moe, lg, idx, 1.0, None, torch.tensor([3, 20, 20, 41], dtype=torch.int32))
    # every sequence empty
    s, d = check(moe, lg, idx, 1.0, None, torch.tensor([50, 50, 50], dtype=torch.int32))
    assert float(s.loss) == 0
    # as many sequences as tokens
    check(moe, lg, idx, 1.0, None, torch.arange(51, dtype=torch.int32))
    # no tokens
    s = moe.balance_loss(lg[:0].to(DEV), idx[:0].to(DEV), 1.0)
    assert float(s.loss) == 0 and (s.counts == 0).all() and (s.probs == 0).all()
    assert moe.balance_loss_backward(lg[:0].to(DEV), s, 4, 1.0).shape == (0, 16)


@gpu
def test_nan_behind_the_mask_dropped_slots_and_infinities(moe):
    lg, idx, mask, off = inputs(200, 24, 3, 5, seqs=3, masked=True)
    lg[~mask] = float("nan")
    idx[::7, 1] = -1                           # dropped slots are not counted
    idx[::11, 2] = 24
    lg[mask.nonzero()[0], 3] = -float("inf")   # an expert switched off for a token
    check(moe, lg, idx, 0.3, mask, off)
    # the type's lowest value in every place of a row, and a row of -inf
    lg, idx, _, _ = inputs(8, 24, 3, 6)
    lg[2] = torch.finfo(torch.float32).min
    lg[3] = -float("inf")
    s, d = check(moe, lg, idx, 1.0)
    assert (d[3] == 0).all()
    # a NaN that takes part shows
    lg[5, 5] = float("nan")
    s = moe.balance_loss(lg.to(DEV), idx.to(DEV), 1.0)
    assert torch.isnan(s.loss) and torch.isnan(
        moe.balance_loss_backward(lg.to(DEV), s, 3, 1.0)[5]).all()


@gpu
def test_same_bits_in_a_graph_and_with_a_shared_workspace(moe):
    lg, idx, mask, off = inputs(5000, 96, 6, 7, seqs=4, masked=True)
    a = [t.to(DEV) for t in (lg, idx, mask, off)]
    ref = moe.balance_loss(a[0], a[1], 0.1, a[2], a[3])
    rd = moe.balance_loss_backward(a[0], ref, 6, 0.1, a[2], a[3])
    ws = torch.full((moe.lib.moe_balance_loss_workspace(5000, 96, 4),), 255, dtype=torch.uint8,
                    device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):                         # two captured steps with one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s = moe.balance_loss(a[0], a[1], 0.1, a[2], a[3], ws=ws)
            d = moe.balance_loss_backward(a[0], s, 6, 0.1, a[2], a[3])
        graphs.append((g, s, d))
    for _ in range(3):
        for g, s, d in graphs:
            ws.fill_(170)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(s.loss, ref.loss) and torch.equal(s.probs, ref.probs)
            assert torch.equal(s.counts, ref.counts) and torch.equal(d, rd)
    with torch.cuda.stream(side):
        s = moe.balance_loss(a[0], a[1], 0.1, a[2], a[3], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(s.probs, ref.probs)


@gpu
@pytest.mark.parametrize("dloss", [float("inf"), float("nan")])
@pytest.mark.parametrize("E", [8, 33, 256])
def test_a_gradient_that_is_not_finite_stays_with_its_tokens(moe, E, dloss):
    """A loss scaled past the fp32 range: tokens that take no part keep a zero
    gradient, the others show it."""
    lg, idx, mask, off = (t.to(DEV) for t in inputs(90, E, 2, E, 3, True))
    st = moe.balance_loss(lg, idx, 1.0, mask, off)
    d = moe.balance_loss_backward(lg, st, 2, 1.0, mask, off,
                                  dloss=torch.tensor(dloss, device=DEV))
    t = torch.arange(90, device=DEV)
    part = mask & (t >= off[0]) & (t < off[-1])
    assert 0 < part.sum() < 90
    assert (d[~part] == 0).all() and not torch.isfinite(d[part]).all(1).any()


@gpu
def test_binding_refusals(moe):
    lg, idx, mask, off = (None if t is None else t.to(DEV) for t in inputs(10, 8, 2, 1, 2, True))
    for bad in (dict(logits=lg.double()), dict(topk_idx=idx.long()), dict(topk_idx=idx[:5]),
                dict(mask=mask[:5]), dict(mask=mask.float()), dict(seq_off=off.long()),
                dict(logits=lg.t().contiguous().t())):
        with pytest.raises(ValueError):
            moe.balance_loss(**{**dict(logits=lg, topk_idx=idx, coef=1.0, mask=mask, seq_off=off), **bad})
    s = moe.balance_loss(lg, idx, 1.0)
    with pytest.raises(ValueError):
        moe.balance_loss_backward(lg, s, 2, 1.0, mask, off)          # another number of sequences
    with pytest.raises(moe.MoeError):
        moe.balance_loss(lg, idx, 1.0, mask, off, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
