"""What the Python binding does around a launch: where it allocates, what it
refuses. CPU tests run the calls on meta tensors with the library faked; GPU
tests run what only shows there."""
import contextlib
import ctypes
import os
import subprocess
import sys
import types

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


class FakeLib:
    """Every launch succeeds and is noted; a workspace takes 64 bytes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            if name == "moe_forward_layout":
                args[-1]._obj.total = 64
            return 64 if name.endswith("workspace") else 0
        return call


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def f8_experts(E=8, d=256, F=128, **other):
    u8 = torch.uint8
    return types.SimpleNamespace(**{**dict(
        fmt="f8", E=E, d=d, F=F, act="swiglu", w_gu=meta(E, 2 * F, d, dtype=u8),
        s_gu=meta(E, 2 * F // 128, d // 128), b_gu=None, w_dn=meta(E, d, F, dtype=u8),
        s_dn=meta(E, d // 128, F // 128), b_dn=None), **other})


def sort_tables(moe, T, k, E, BM=128, **other):
    i32, u32 = torch.int32, torch.uint32
    return moe.SortTables(**{**dict(
        order=meta(T * k, dtype=u32), inv_order=meta(T * k, dtype=u32),
        row_map=meta(T * k, dtype=u32), counts=meta(E, dtype=i32),
        row_off=meta(E + 1, dtype=i32), tile_off=meta(E + 1, dtype=i32), BM=BM), **other})


@pytest.fixture
def fake(moe, monkeypatch):
    """The binding without a GPU: its device checks passed over, its launches
    noted. `fake.inside`: a stream was entered by torch.cuda.stream."""
    f = FakeLib()
    f.inside = None

    @contextlib.contextmanager
    def stream(s):
        before, f.inside = f.inside, s
        yield
        f.inside = before

    f.recorded = []
    f.caller = types.SimpleNamespace(cuda_stream=0xCA11)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: f.caller)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: f.recorded.append((id(t), s)))
    monkeypatch.setattr(moe, "lib", f)
    monkeypatch.setattr(moe, "_dev", lambda *ts: None)
    monkeypatch.setattr(moe, "_on", lambda *ts: f.inside)
    monkeypatch.setattr(moe, "_stream", lambda *s: f.inside)
    return f


# ------------------------------------------------------------------ stream=

def calls(moe):
    T, E, k, d, F = 4, 8, 2, 256, 128
    bf, f16, i32, u8 = torch.bfloat16, torch.float16, torch.int32, torch.uint8
    ex, st = f8_experts(), sort_tables(moe, T, k, E)
    x, w, idx, lg = meta(T, d, dtype=bf), meta(E, d, dtype=bf), meta(T, k, dtype=i32), meta(T, E)
    stats = moe.BalanceStats(meta(), meta(1, E, dtype=i32), meta(1, E), meta(1, dtype=i32))
    return dict(
        route=(x, w, None, k), topk=(lg, k), sort_rows=(idx, E, 128),
        grouped_swiglu=(x, st, k, ex), grouped_down=(meta(T * k, F), st, T, k, ex),
        combine=(meta(T * k, d, dtype=f16), st.inv_order, meta(T, k), T, k),
        quantize_fp8=(x,), fp8_matmul=(meta(T, d, dtype=u8), meta(T, 2), meta(E, d, dtype=u8),
                                       meta(1, 2)),
        grouped_swiglu_fp8=(meta(T, d, dtype=u8), meta(T, 2), st, k, ex),
        grouped_down_fp8=(meta(T * k, F, dtype=u8), meta(T * k, 1), st, T, k, ex),
        balance_loss=(lg, idx, 1.0), balance_loss_backward=(lg, stats, k, 1.0),
        forward=(x, w, None, ex, k),
        pack_gate_up=("f8", meta(E, F, d, dtype=u8), meta(E, F, d, dtype=u8), meta(E, 1, 2), None,
                      meta(E, 1, 2)))


CALLS = ("route", "topk", "sort_rows", "grouped_swiglu", "grouped_down", "combine", "quantize_fp8",
         "fp8_matmul", "grouped_swiglu_fp8", "grouped_down_fp8", "balance_loss",
         "balance_loss_backward", "forward", "pack_gate_up")


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_another_stream_allocates_there(moe, fake, monkeypatch, name):
    """A block from the current stream's pool may still be in use by that
    stream's kernels when another stream's write it."""
    args = calls(moe)[name]
    made = []

    def noting(make):
        def f(*a, **kw):
            made.append(fake.inside)
            return make(*a, **kw)
        return f

    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch, "empty_like", noting(torch.empty_like))
    monkeypatch.setattr(moe, "_empty", noting(moe._empty))
    side = types.SimpleNamespace(cuda_stream=0x51DE, device=0)
    out = getattr(moe, name)(*args, stream=side)
    assert made and all(m is side for m in made)
    launches = [a for n, a in fake.calls if n == "moe_" + name]
    assert len(launches) == 1 and launches[0][-1] is side
    assert fake.inside is None
    # outputs go back to that stream's pool only after the caller's reads
    outs = [out] if torch.is_tensor(out) else out if isinstance(out, tuple) else vars(out).values()
    outs = [t for t in outs if torch.is_tensor(t)]
    assert outs and sorted(fake.recorded, key=str) == \
        sorted([(id(t), fake.caller) for t in outs], key=str)


@gpu
def test_balance_loss_beside_one_still_pending(moe):
    """A call whose scratch has gone back to the current stream's pool while
    its kernels still run, and one on another stream that starts at once."""
    T, E, k = 200003, 64, 4
    g = torch.Generator(device=DEV).manual_seed(0)
    a, b = (torch.randn(T, E, generator=g, device=DEV) for _ in range(2))
    ia, ib = (t.topk(k, 1).indices.int() for t in (a, b))
    ra, rb = moe.balance_loss(a, ia, 1.0), moe.balance_loss(b, ib, 1.0)
    qa, qb = moe.quantize_fp8(a), moe.quantize_fp8(b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    for _ in range(5):
        for _ in range(8):
            busy.zero_()                       # the current stream falls behind
        s = [moe.balance_loss(a, ia, 1.0) for _ in range(3)]
        t = [moe.balance_loss(b, ib, 1.0, stream=side) for _ in range(3)]
        q = moe.quantize_fp8(a)
        r = moe.quantize_fp8(b, stream=side)
        torch.cuda.synchronize()
        for got, want in [(v, ra) for v in s] + [(v, rb) for v in t]:
            assert torch.equal(got.loss, want.loss) and torch.equal(got.probs, want.probs)
            assert torch.equal(got.counts, want.counts) and torch.equal(got.tokens, want.tokens)
        for got, want in ((q, qa), (r, qb)):
            assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))
            assert torch.equal(got[1], want[1])


# ------------------------------------------------------------------ refusals

BAD_F8 = dict(
    bf16_scales=lambda: dict(s_gu=meta(8, 2, 2, dtype=torch.bfloat16)),
    bf16_down_scales=lambda: dict(s_dn=meta(8, 2, 1, dtype=torch.bfloat16)),
    a_scale_per_row=lambda: dict(s_gu=meta(8, 256)),
    gate_scales_alone=lambda: dict(s_gu=meta(8, 1, 2)),
    no_expert_axis=lambda: dict(s_dn=meta(2, 1)),
    codes_of_16_bits=lambda: dict(w_gu=meta(8, 256, 256, dtype=torch.bfloat16)),
    gate_alone=lambda: dict(w_gu=meta(8, 128, 256, dtype=torch.uint8)),
    down_transposed=lambda: dict(w_dn=meta(8, 128, 256, dtype=torch.uint8)),
    fewer_experts=lambda: dict(w_dn=meta(7, 256, 128, dtype=torch.uint8)))


@pytest.mark.parametrize("fmt", ["f8", 6])
@pytest.mark.parametrize("name", ["forward", "grouped_swiglu_fp8", "grouped_down_fp8"])
@pytest.mark.parametrize("bad", BAD_F8)
def test_f8_experts_of_other_shapes_or_types_are_refused(moe, fake, name, bad, fmt):
    """By the whole-layer call as by its stages: the kernels would read past
    the end of such scales, or misread them."""
    args = list(calls(moe)[name])
    i = next(i for i, a in enumerate(args) if isinstance(a, types.SimpleNamespace))
    args[i] = f8_experts(fmt=fmt)
    getattr(moe, name)(*args)
    assert len(fake.calls) >= 1
    fake.calls.clear()
    args[i] = f8_experts(fmt=fmt, **BAD_F8[bad]())
    with pytest.raises((ValueError, TypeError)):
        getattr(moe, name)(*args)
    assert not fake.calls


def test_rows_and_routers_of_another_width_are_refused(moe, fake):
    x, w, _, ex, k = calls(moe)["forward"]
    bf = torch.bfloat16
    for bad in ((meta(4, 128, dtype=bf), w), (x, meta(8, 128, dtype=bf)), (x, meta(7, 256, dtype=bf)),
                (meta(2, 2, 256, dtype=bf), w)):
        with pytest.raises(ValueError):
            moe.forward(*bad, None, ex, k)
    assert not fake.calls


@pytest.mark.parametrize("bad", [dict(row_off=torch.int64), dict(tile_off=torch.int64),
                                 dict(row_off=torch.float32), dict(row_map=torch.int64),
                                 dict(tile_off=torch.int16)])
def test_tables_of_other_types_are_refused(moe, fake, bad):
    """Tables of the right length whose entries have another width: the kernels
    would read past their end, or rows that are not there."""
    T, E, k = 4, 8, 2
    n = dict(row_map=T * k, row_off=E + 1, tile_off=E + 1)
    for name in ("grouped_swiglu_fp8", "grouped_down_fp8"):
        if "row_map" in bad and name == "grouped_down_fp8":
            continue                                   # takes the rows as they stand
        args = list(calls(moe)[name])
        args[2] = sort_tables(moe, T, k, E, **{f: meta(n[f], dtype=t) for f, t in bad.items()})
        with pytest.raises(ValueError):
            getattr(moe, name)(*args)
    args = list(calls(moe)["grouped_swiglu_fp8"])
    args[2] = sort_tables(moe, T, k, E, row_map=meta(T * k, dtype=torch.int32))
    moe.grouped_swiglu_fp8(*args)
    assert len(fake.calls) == 1


@pytest.mark.parametrize("bad", [
    dict(w_u=(2, 128, 512)), dict(w_u=(2, 384, 256)), dict(w_u=(3, 256, 256)),
    dict(s_u=(2, 1, 2)), dict(s_u=(2, 256)), dict(s_g=(2, 2, 1), s_u=(2, 2, 1)),
    dict(s_g=(2, 256, 2), s_u=(2, 256, 2)), dict(s_g=torch.bfloat16, s_u=torch.bfloat16),
    dict(s_u=torch.bfloat16), dict(w_g=torch.float16, w_u=torch.float16), dict(w_u=torch.bfloat16),
    dict(s_g=None), dict(s_u=None)])
def test_pack_gate_up_refuses_f8_parts_that_do_not_fit(moe, fake, bad):
    good = dict(w_g=meta(2, 256, 256, dtype=torch.uint8), w_u=meta(2, 256, 256, dtype=torch.uint8),
                s_g=meta(2, 2, 2), s_u=meta(2, 2, 2))
    w, s, b = moe.pack_gate_up("f8", **good)
    assert w.shape == (2, 512, 256) and s.shape == (2, 4, 2) and b is None
    fake.calls.clear()
    for n, v in bad.items():
        good[n] = v if v is None else (good[n].to(v) if isinstance(v, torch.dtype)
                                       else meta(*v, dtype=good[n].dtype))
    with pytest.raises((ValueError, TypeError)):
        moe.pack_gate_up("f8", **good)
    assert not fake.calls


@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 32) + 8])
def test_balance_sizes_past_a_c_int_are_refused(moe, fake, n):
    """Not cut to their low bits: experts, slots and sequences as tokens are."""
    i32 = torch.int32
    lg, idx = meta(4, 8), meta(4, 2, dtype=i32)
    stats = moe.BalanceStats(meta(), meta(1, 8, dtype=i32), meta(1, 8), meta(1, dtype=i32))
    wide = moe.BalanceStats(meta(), meta(1, n, dtype=i32), meta(1, n), meta(1, dtype=i32))
    many = moe.BalanceStats(meta(), meta(n - 1, 8, dtype=i32), meta(n - 1, 8), meta(n - 1, dtype=i32))
    off = meta(n, dtype=i32)
    for call in (lambda: moe.balance_loss(meta(0, n), meta(0, 2, dtype=i32), 1.0),
                 lambda: moe.balance_loss(meta(0, 8), meta(0, n, dtype=i32), 1.0),
                 lambda: moe.balance_loss(lg, idx, 1.0, seq_off=off),
                 lambda: moe.balance_loss_backward(lg, stats, n, 1.0),
                 lambda: moe.balance_loss_backward(meta(0, n), wide, 2, 1.0),
                 lambda: moe.balance_loss_backward(lg, many, 2, 1.0, seq_off=off)):
        with pytest.raises(ValueError, match="2\\^30"):
            call()
    assert not fake.calls


# ------------------------------------------------------------------ gradients

def test_the_loss_is_a_node_of_the_graph_where_its_logits_are(moe, fake):
    """No gradient is lost without a word (the launches are noted, not made)."""
    lg, idx = meta(4, 8), meta(4, 2, dtype=torch.int32)
    assert not moe.balance_loss(lg, idx, 1.0).loss.requires_grad
    lg.requires_grad_()
    with torch.no_grad():
        assert not moe.balance_loss(lg, idx, 1.0).loss.requires_grad
    fake.calls.clear()
    s = moe.balance_loss(lg, idx, 1.0)
    assert s.loss.requires_grad and not s.counts.requires_grad and not s.tokens.requires_grad
    (d,) = torch.autograd.grad(s.loss * 2, lg)
    assert d.shape == lg.shape
    assert [n for n, _ in fake.calls if not n.endswith("workspace")] == \
        ["moe_balance_loss", "moe_balance_loss_backward"]
    fake.calls.clear()
    s = moe.balance_loss(lg, idx, 1.0)
    with pytest.raises(RuntimeError, match="probs"):
        torch.autograd.grad((s.loss + s.probs.sum()), lg)
    s = moe.balance_loss(lg, idx, 1.0)
    with pytest.raises(RuntimeError, match="once differentiable"):
        torch.autograd.grad(s.loss, lg, create_graph=True)
    s = moe.balance_loss(lg, idx, 1.0)
    s.counts.add_(1)                                    # what the gradient needs
    with pytest.raises(RuntimeError, match="inplace"):
        torch.autograd.grad(s.loss, lg)


def _router_step(seed=0, T=3000, E=48, k=3, d=64):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, d, generator=g, device=DEV)
    w = (torch.randn(E, d, generator=g, device=DEV) / 8).requires_grad_()
    mask = torch.rand(T, generator=g, device=DEV) < 0.8
    off = torch.tensor([10, 900, 900, T - 7], dtype=torch.int32, device=DEV)
    idx = (x @ w.detach().t()).topk(k, 1).indices.int()
    return x, w, idx, mask, off, k


@gpu
@pytest.mark.parametrize("T", [100, 3000])
def test_a_router_trains_through_the_loss(moe, T):
    """The gradient of the router's weight is that of balance_loss_backward, bit
    for bit, beside another loss and on another stream."""
    x, w, idx, mask, off, k = _router_step(T=T)
    off = off if T > 1000 else None
    with torch.no_grad():
        lg = x @ w.t()
        s = moe.balance_loss(lg, idx, 0.7, mask, off)
        d = moe.balance_loss_backward(lg, s, k, 0.7, mask, off,
                                      dloss=torch.tensor(3.0, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        lg = x @ w.t()
        side.wait_stream(torch.cuda.current_stream())
        t = moe.balance_loss(lg, idx, 0.7, mask, off, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(t.loss.detach(), s.loss) and torch.equal(t.counts, s.counts)
        (got,) = torch.autograd.grad(3 * t.loss, lg)
        assert torch.equal(got, d)
    lg = x @ w.t()
    t = moe.balance_loss(lg, idx, 0.7, mask, off)
    (both,) = torch.autograd.grad(3 * t.loss + (lg * lg).mean(), w)
    lg2 = x @ w.t()
    (other,) = torch.autograd.grad((lg2 * lg2).mean(), w)
    want = d.double().t() @ x.double() + other.double()
    # fp32 products of T addends
    size = d.abs().double().t() @ x.abs().double() + other.abs().double() + \
        (2 / lg.numel() * lg.abs()).double().t() @ x.abs().double()
    assert ((both.double() - want).abs() <= (T + 8) * 2.0 ** -23 * size).all()


@gpu
def test_a_training_step_in_a_graph(moe):
    """Forward and backward captured together, replayed on new logits."""
    x, w, idx, mask, off, k = _router_step(1)

    def step():
        lg = x @ w.t()
        s = moe.balance_loss(lg, idx, 0.7, mask, off)
        return s.loss.detach(), torch.autograd.grad(s.loss, w)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, grad = step()
    for seed in (2, 3):
        x.copy_(_router_step(seed)[0])
        g.replay()
        torch.cuda.synchronize()
        l2, g2 = step()
        assert torch.equal(loss, l2) and torch.equal(grad, g2)


# ------------------------------------------------------------------ alignment

def test_scales_off_a_float_boundary_are_refused(moe):
    L, P, ARG = moe.lib, None, moe.ERR_INVALID_ARG
    p, off = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)
    assert L.moe_quantize_fp8(p, moe.BF16, 4, 128, 1, p, off, P) == ARG
    for i in (1, 3):
        a = [p, p, p, p]
        a[i] = off
        assert L.moe_fp8_matmul(*a, 4, 8, 128, moe.BF16, p, P) == ARG
    e = ctypes.byref(moe.Experts(moe.W_F8, 8, 256, 128, 0x10000, 0x10000, None, 0x10000, 0x10000,
                                 None))
    assert L.moe_grouped_swiglu_fp8(p, off, p, p, p, 128, 4, 2, e, p, p, 0, P) == ARG
    assert L.moe_grouped_swiglu_fp8(p, p, p, p, p, 128, 4, 2, e, p, off, 0, P) == ARG
    assert L.moe_grouped_down_fp8(p, off, p, p, 128, 4, 2, e, p, 0, P) == ARG
    for lg, E in ((off, 33), (ctypes.c_void_p(0x10004), 32)):
        assert L.moe_balance_loss(lg, p, P, P, 4, E, 2, 1, 1.0, p, p, p, p, p, 1 << 20, P) == ARG
        assert L.moe_balance_loss_backward(lg, P, P, 4, E, 2, 1, 1.0, p, p, P, p, P) == ARG
        assert L.moe_balance_loss_backward(p, P, P, 4, E, 2, 1, 1.0, p, p, P, lg, P) == ARG


def _floats(t):
    """A copy of fp32 t that starts 4 bytes into an allocation."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    return buf[1:].view(t.shape).copy_(t)


@gpu
@pytest.mark.parametrize("M,N,K", [(5, 256, 384), (40, 640, 2064), (1000, 2100, 768)])
def test_products_of_views(moe, M, N, K):
    """Rows of a batch, one expert of a stack: views whose scales start at any
    float give the bits of copies."""
    g = torch.Generator(device=DEV).manual_seed(M)
    a, sa = moe.quantize_fp8(torch.randn(M + 1, K, generator=g, device=DEV))
    Nb = -(-N // 128) * 128
    b, sb = moe.quantize_fp8(torch.randn(3, Nb, K, generator=g, device=DEV), 128)
    want = moe.fp8_matmul(a[1:].clone(), sa[1:].clone(), b[1, :N].clone(), sb[1].clone())
    assert torch.equal(moe.fp8_matmul(a[1:], sa[1:], b[1, :N], sb[1]), want)
    want = moe.fp8_matmul(a, sa, b[1, :N], sb[1].clone())
    assert torch.equal(moe.fp8_matmul(a, _floats(sa), b[1, :N], _floats(sb[1])), want)


@gpu
@pytest.mark.parametrize("regime", [1, 2])
def test_expert_stages_of_views(moe, regime):
    T, E, k, d, F = 70, 8, 2, 384, 128
    ex = mi.make_experts(mi.Workload("f8", 1, d, E, 1, F, "bf16", "f8"), 3, DEV)
    idx = mi.random_topk_idx(T, E, k, 1).to(DEV)
    st = moe.sort_rows(idx, E, 128)
    xq, xs = moe.quantize_fp8(torch.randn(T + 1, d, device=DEV))
    want = moe.grouped_swiglu_fp8(xq[1:].clone(), xs[1:].clone(), st, k, ex, regime)
    hq, hs = moe.grouped_swiglu_fp8(xq[1:], xs[1:], st, k, ex, regime)
    assert torch.equal(hq.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(hs, want[1])
    ys = moe.grouped_down_fp8(hq, hs, st, T, k, ex, regime)
    assert torch.equal(moe.grouped_down_fp8(hq, _floats(hs), st, T, k, ex, regime), ys)
    # scales written at such a place through the C calls
    s = torch.cuda.current_stream().cuda_stream
    e = moe.experts_struct(ex)
    buf = torch.full((hs.numel() + 2,), -1.0, device=DEV)
    h2 = torch.empty_like(hq)
    assert moe.lib.moe_grouped_swiglu_fp8(
        xq[1:].data_ptr(), xs[1:].data_ptr(), st.row_map.data_ptr(), st.row_off.data_ptr(),
        st.tile_off.data_ptr(), 128, T, k, ctypes.byref(e), h2.data_ptr(), buf[1:].data_ptr(),
        regime, s) == moe.OK
    assert torch.equal(buf[1:-1].view_as(hs), hs) and buf[0] == -1 and buf[-1] == -1
    x = torch.randn(9, 384, device=DEV)
    q, sq = moe.quantize_fp8(x)
    buf = torch.full((sq.numel() + 2,), -1.0, device=DEV)
    assert moe.lib.moe_quantize_fp8(x.data_ptr(), moe.F32, 9, 384, 1, q.data_ptr(),
                                    buf[1:].data_ptr(), s) == moe.OK
    assert torch.equal(buf[1:-1].view_as(sq), sq) and buf[0] == -1 and buf[-1] == -1


@gpu
@pytest.mark.parametrize("T,E", [(40, 33), (9000, 65), (700, 510)])
def test_balance_loss_of_a_batch_s_rows(moe, T, E):
    """Logits from any row of a batch whose rows are no multiple of 16 bytes."""
    g = torch.Generator(device=DEV).manual_seed(E)
    lg = torch.randn(T + 1, E, generator=g, device=DEV)
    idx = lg.topk(3, 1).indices.int()
    want = moe.balance_loss(lg[1:].clone(), idx[1:].clone(), 1.0)
    got = moe.balance_loss(lg[1:], idx[1:], 1.0)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.probs, want.probs)
    assert torch.equal(got.counts, want.counts)
    d = moe.balance_loss_backward(lg[1:], got, 3, 1.0)
    assert torch.equal(d, moe.balance_loss_backward(lg[1:].clone(), want, 3, 1.0))


# ------------------------------------------------------------------ torch

NO_SHORTCUTS = """
import torch
had = {n: getattr(torch._C, n) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream")
       if hasattr(torch._C, n)}
for n in had:
    delattr(torch._C, n)
import sparse_mixture_experts_top_b200 as moe
for n in had:                  # (torch's public calls may use them themselves)
    setattr(torch._C, n, had[n])
"""


def _without_shortcuts(code):
    r = subprocess.run([sys.executable, "-c", NO_SHORTCUTS + code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr


def test_the_binding_needs_no_private_name_of_torch(moe):
    _without_shortcuts("assert callable(moe._device) and callable(moe._raw_stream)")


@gpu
def test_calls_without_private_names_of_torch(moe):
    _without_shortcuts("""
x = torch.randn(4, 256, device="cuda")
q, s = moe.quantize_fp8(x)
assert moe._raw_stream(0) == torch.cuda.current_stream().cuda_stream and moe._device() == 0
side = torch.cuda.Stream()
torch.cuda.synchronize()
q2, s2 = moe.quantize_fp8(x, stream=side)
torch.cuda.synchronize()
assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
""")
