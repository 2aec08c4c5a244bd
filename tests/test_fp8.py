"""The e4m3 operators with block scales: quantiser, dense product, grouped
experts, the whole layer with f8 experts; refusals on the CPU, everything else
against plain 64-bit forms on the GPU."""
import ctypes

import numpy as np
import pytest
import torch

import moe_inputs as mi
from fp8_util import E4M3, act64, dequantize, quantize_ref, round_e4m3, sum_bound, values
from parity_util import _act_and_slope, rms

gpu = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_mixture_experts_top_b200 as m
    return m


# ------------------------------------------------------------------ CPU

def test_reference_decoding_is_the_format():
    """The decode table against torch's own e4m3 type, and the rounding against
    the nearest table value."""
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(E4M3, t)
    v = np.random.default_rng(0).normal(size=2000) * 60
    fin = np.sort(E4M3[np.isfinite(E4M3)])
    near = np.abs(fin[:, None] - v[None]).min(0)
    np.testing.assert_array_equal(np.abs(round_e4m3(v) - v), near)


def test_calls_refuse_bad_arguments_without_launching(moe):
    L, P = moe.lib, None
    p, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
    ARG, UNS, OK = moe.ERR_INVALID_ARG, moe.ERR_UNSUPPORTED, moe.OK
    q = L.moe_quantize_fp8
    assert q(P, moe.BF16, 4, 128, 1, p, p, P) == ARG
    assert q(p, moe.BF16, 4, 128, 1, P, p, P) == ARG
    assert q(p, moe.BF16, 4, 128, 1, p, P, P) == ARG
    assert q(p, 3, 4, 128, 1, p, p, P) == ARG
    assert q(p, moe.BF16, -1, 128, 1, p, p, P) == ARG
    assert q(p, moe.BF16, 4, 0, 1, p, p, P) == ARG
    assert q(p, moe.BF16, 4, 128, 64, p, p, P) == ARG
    assert q(odd, moe.BF16, 4, 128, 1, p, p, P) == ARG
    assert q(p, moe.BF16, 4, 120, 1, p, p, P) == UNS
    assert q(P, moe.BF16, 0, 128, 1, P, P, P) == OK
    m = L.moe_fp8_matmul
    assert m(P, p, p, p, 4, 8, 128, moe.BF16, p, P) == ARG
    assert m(p, p, p, P, 4, 8, 128, moe.BF16, p, P) == ARG
    assert m(p, p, p, p, 4, 0, 128, moe.BF16, p, P) == ARG
    assert m(p, p, p, p, -4, 8, 128, moe.BF16, p, P) == ARG
    assert m(p, p, p, p, 4, 8, 128, 9, p, P) == ARG
    assert m(p, p, p, p, 4, 8, 128, moe.BF16, odd, P) == ARG
    assert m(p, p, p, p, 4, 8, 100, moe.BF16, p, P) == UNS
    assert m(P, P, P, P, 0, 8, 128, moe.BF16, P, P) == OK
    big = (1 << 30) + 16                    # a tile past it would leave 32-bit indices
    assert q(p, moe.BF16, big, 16, 128, p, p, P) == UNS
    assert q(p, moe.BF16, 4, big, 1, p, p, P) == UNS
    assert q(p, moe.BF16, 0x7fffffff, 16, 128, p, p, P) == UNS
    assert m(p, p, p, p, big, 8, 16, moe.BF16, p, P) == UNS
    assert m(p, p, p, p, 4, big, 16, moe.BF16, p, P) == UNS
    assert m(p, p, p, p, 4, 8, big, moe.BF16, p, P) == UNS

    def ex(fmt=moe.W_F8, E=8, d=256, F=128, w=0x10000, s=0x10000):
        return ctypes.byref(moe.Experts(fmt, E, d, F, w, s, None, w, s, None))

    up = lambda e, x=p, BM=128, T=4, k=2, rg=0: L.moe_grouped_swiglu_fp8(  # noqa: E731
        x, p, p, p, p, BM, T, k, e, p, p, rg, P)
    dn = lambda e, x=p, BM=128, T=4, k=2, rg=0: L.moe_grouped_down_fp8(    # noqa: E731
        x, p, p, p, BM, T, k, e, p, rg, P)
    for f in (up, dn):
        assert f(ex(), x=P) == ARG
        assert f(ex(), x=odd) == ARG
        assert f(ex(), BM=0) == ARG
        assert f(ex(), k=9) == ARG
        assert f(ex(), rg=7) == ARG
        assert f(None) == ARG
        assert f(ex(s=None)) == ARG
        assert f(ex(s=0x10008)) == ARG
        assert f(ex(d=192)) == UNS
        assert f(ex(F=64)) == UNS
        assert f(ex(fmt=moe.W_BF16)) == UNS
        assert f(ex(E=1025), k=2) == UNS
        assert f(ex(), T=0, x=P) == OK
    # the 16-bit stage calls refer to the fp8 ones; f32 activations have no f8 experts
    e = ex()
    assert L.moe_grouped_swiglu(p, moe.BF16, p, p, p, 128, 4, 2, e, p, p, 1 << 20, 0, P) == UNS
    assert L.moe_grouped_down(p, moe.BF16, p, p, 128, 4, 2, e, p, 0, P) == UNS
    assert L.moe_forward(p, moe.F32, p, P, e, 4, 2, p, p, 1 << 30, 0, P) == UNS
    assert L.moe_forward(p, moe.BF16, p, P, e, 4, 2, p, p, 16, 0, P) == moe.ERR_WORKSPACE
    assert L.moe_pack_gate_up(moe.W_F8, 2, 128, 128, p, P, P, p, p, P, p, p, P, P) == ARG
    assert L.moe_pack_gate_up(moe.W_F8, 2, 192, 128, p, p, P, p, p, P, p, p, P, P) == UNS


def test_forward_layout_holds_codes_and_scales(moe):
    up = lambda v: -(-v // 256) * 256        # noqa: E731
    for T in (1, 33, 4096):
        L = moe.forward_layout(T, 512, 16, 4, 384, torch.bfloat16, "f8")
        R = T * 4
        assert L.ys - L.h >= up(R * 384) + R * 3 * 4
        assert L.total - L.x16 >= up(T * 512) + T * 4 * 4


def test_binding_refuses_bad_tensors(moe):
    with pytest.raises(ValueError):
        moe.quantize_fp8(torch.zeros(4, 128))                     # not on the GPU
    with pytest.raises(ValueError):
        moe.fp8_matmul(*[torch.zeros(4, 128)] * 4)


@pytest.mark.parametrize("rows", [(1 << 30) + 1, 1 << 31, (1 << 32) + 4])
def test_binding_refuses_sizes_past_its_integers(moe, monkeypatch, rows):
    """A size that a C int cannot hold is refused, not cut to its low bits.
    (Meta tensors have such sizes without memory; the device check is passed over.)"""
    monkeypatch.setattr(moe, "_on", lambda *ts: 0)
    x = torch.empty(rows, 16, dtype=torch.bfloat16, device="meta")
    a = torch.empty(rows, 16, dtype=torch.uint8, device="meta")
    sa = torch.empty(rows, 1, device="meta")
    b, sb = a[:8], sa[:1]
    for call in (lambda: moe.quantize_fp8(x), lambda: moe.quantize_fp8(x, 128),
                 lambda: moe.quantize_fp8(x.view(1, rows, 16)),
                 lambda: moe.fp8_matmul(a, sa, b, sb),
                 lambda: moe.fp8_matmul(b, sa[:8], a, sa[:-(-rows // 128)])):
        with pytest.raises(ValueError, match="2\\^30"):
            call()
    idx = torch.empty(rows, 1, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="2\\^30"):
        moe.balance_loss(x.float(), idx, 1.0)


# ------------------------------------------------------------------ quantiser

@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (3, 144), (130, 272), (257, 2064), (5, 7168)])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_matches_the_definition(moe, dtype, rows, K, block):
    g = torch.Generator().manual_seed(rows * K + block)
    x = torch.randn(rows, K, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x[0, :16] = 0
    x = x.to(dtype)
    q, s = moe.quantize_fp8(x.to(DEV), block)
    rq, rs = quantize_ref(x.float().numpy(), block)
    assert q.dtype == torch.float8_e4m3fn and s.shape == rs.shape
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(values(q), rq)
    # and so every value is within half a step: 2^-4 of itself, or 2^-10 of
    # its scale among the subnormal codes (plus the two fp32 roundings)
    xe = x.double().numpy()
    d = np.abs(dequantize(q, s, block) - xe)
    each = np.repeat(rs if block == 1 else np.repeat(rs, 128, 0)[:rows], 128, 1)[:, :K]
    assert (d <= (2.0 ** -4 + 2.0 ** -21) * np.abs(xe) + 2.0 ** -10 * each).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantize_special_values(moe, dtype):
    """Infinities and NaN become NaN codes and leave the scale alone; zero and
    tiny groups take the floor's scale; negative zero stays a zero."""
    x = torch.randn(6, 256)
    x[0, 3], x[0, 130], x[1, 5] = float("inf"), float("nan"), -float("inf")
    x[2] = 0
    x[3, :128] = 1e-38
    x[4, :128] = float("nan")
    x[5, 0], x[5, 1] = torch.finfo(dtype).max, -0.0
    gx = x.to(dtype).to(DEV)
    x = x.to(dtype).float()
    q, s = moe.quantize_fp8(gx)
    rq, rs = quantize_ref(x.numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(values(q), rq)
    assert np.isnan(values(q)[0, 3]) and np.isfinite(rs).all()
    # one bad element in a block spoils only itself
    q, s = moe.quantize_fp8(gx, 128)
    rq, rs = quantize_ref(x.numpy(), 128)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(values(q), rq)


@gpu
def test_quantize_stack_and_empty(moe):
    w = torch.randn(3, 256, 160)
    q, s = moe.quantize_fp8(w.to(DEV), 128)
    assert s.shape == (3, 2, 2)
    for e in range(3):
        rq, rs = quantize_ref(w[e].numpy(), 128)
        np.testing.assert_array_equal(values(q[e]), rq)
        np.testing.assert_array_equal(s[e].cpu().numpy(), rs)
    with pytest.raises(ValueError):
        moe.quantize_fp8(torch.zeros(2, 100, 128, device=DEV), 128)
    q, s = moe.quantize_fp8(torch.zeros(0, 128, device=DEV))
    assert q.shape == (0, 128) and s.shape == (0, 1)


# ------------------------------------------------------------------ dense product

def _operands(moe, M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    b = torch.randn(N, K, generator=g) / K ** 0.5
    return moe.quantize_fp8(a.to(DEV)) + moe.quantize_fp8(b.to(DEV), 128)


def _check_matmul(y, a, sa, b, sb, dtype):
    A, B = dequantize(a, sa), dequantize(b, sb, 128)
    ref, mag = A @ B.T, np.abs(A) @ np.abs(B).T
    u = torch.finfo(dtype).eps / 2
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    err = np.abs(y.double().cpu().numpy() - ref)
    bound = sum_bound(A.shape[1]) * mag + u * np.abs(ref) * (1 + 1e-3) + sub
    assert np.isfinite(err).all() and (err <= bound).all(), float((err / bound).max())


MATMUL_SIZES = [(1, 1, 16), (33, 20, 16), (1, 128, 128), (2, 17, 48), (7, 200, 272), (8, 512, 7168),
                (9, 256, 384), (33, 1000, 2064), (64, 96, 128), (100, 333, 656), (128, 256, 256),
                (129, 640, 1024), (300, 257, 512), (511, 1024, 1152),
                (40, 640, 4112), (1030, 2100, 400), (700, 4096, 256), (2000, 1300, 128),
                (900, 5000, 320), (3000, 1100, 1040)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", MATMUL_SIZES)
def test_matmul(moe, dtype, M, N, K):
    a, sa, b, sb = _operands(moe, M, N, K, M + N + K)
    # a guard behind the result: nothing past [M][N] is written
    buf = torch.full((M * N + 64,), 7.0, dtype=dtype, device=DEV)
    y = moe.fp8_matmul(a, sa, b, sb, dtype, out=buf[:M * N].view(M, N))
    _check_matmul(y, a, sa, b, sb, dtype)
    assert (buf[M * N:] == 7).all()
    assert moe.device_status() == moe.OK


@gpu
def test_matmul_refusals_and_status(moe):
    a, sa, b, sb = _operands(moe, 4, 32, 128, 0)
    assert moe.fp8_matmul(a[:0], sa[:0], b, sb).shape == (0, 32)
    with pytest.raises(TypeError):
        moe.fp8_matmul(a.float(), sa, b, sb)
    with pytest.raises(ValueError):
        moe.fp8_matmul(a, sa[:, :0], b, sb)
    with pytest.raises(ValueError):
        moe.fp8_matmul(a, sa, b.t().contiguous().t(), sb)       # strides
    with pytest.raises(ValueError):
        moe.fp8_matmul(a, sa, b[:, :64].contiguous(), sb)
    moe.device_status()
    y = moe.fp8_matmul(a, sa * 1e6, b, sb, torch.float16)
    assert torch.isinf(y).any() and moe.device_status() == moe.ERR_RANGE
    # a NaN token row is NaN in its own row only
    x = torch.randn(4, 128, device=DEV)
    x[2, 7] = float("nan")
    y = moe.fp8_matmul(*moe.quantize_fp8(x), b, sb, torch.float32)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3]]).all()


# ------------------------------------------------------------------ experts

def _experts(E, d, F, seed, act="swiglu"):
    wl = mi.Workload("f8", 1, d, E, 1, F, "bf16", "f8")
    return mi.make_experts(wl, seed, DEV).with_act(act)


def _dense(ex, e):
    gu = dequantize(ex.w_gu[e], ex.s_gu[e], 128)
    return gu[:ex.F], gu[ex.F:], dequantize(ex.w_dn[e], ex.s_dn[e], 128)


def _run_stages(moe, T, E, k, d, F, regime, BM, skew, act, seed):
    ex = _experts(E, d, F, seed, act)
    idx = mi.random_topk_idx(T, E, k, seed, skew).to(DEV)
    st = moe.sort_rows(idx, E, BM)
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, d, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).bfloat16()
    xq, xs = moe.quantize_fp8(x.to(DEV))
    hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, k, ex, regime)
    ys = moe.grouped_down_fp8(hq, hs, st, T, k, ex, regime)
    return ex, st, xq, xs, hq, hs, ys


def _check_stages(ex, st, xq, xs, hq, hs, ys):
    X, H = dequantize(xq, xs), dequantize(hq, hs)
    off = st.row_off.cpu().numpy()
    tok = st.row_map.cpu().view(torch.int32).numpy()
    Y = ys.double().cpu().numpy()
    S = np.repeat(hs.cpu().numpy().astype(np.float64), 128, 1)
    bd, bf = sum_bound(ex.d), sum_bound(ex.F)
    for e in range(ex.E):
        r = slice(off[e], off[e + 1])
        if r.start == r.stop:
            continue
        wg, wu, wd = _dense(ex, e)
        x = X[tok[r]]
        g, u = x @ wg.T, x @ wu.T
        a, da = _act_and_slope(g, ex.act)
        h = act64(g, ex.act) * u
        # h before it is quantised: the products' sums, and 2^-18 for the
        # activation's exp (error up to 2 + 1.16 |g| units of 2^-23), division
        # and products
        dh = (np.abs(u * da) * (bd * (np.abs(x) @ np.abs(wg).T)) +
              np.abs(a) * (bd * (np.abs(x) @ np.abs(wu).T))) * 1.01 + 2.0 ** -18 * np.abs(h) + 1e-30
        # then half a step of e4m3 (2^-4 of the value; 2^-10 of the scale among
        # the subnormal codes) on a value dh away
        err = np.abs(H[r] - h)
        bound = dh + (2.0 ** -4 + 2.0 ** -20) * (np.abs(h) + dh) + 2.0 ** -10 * S[r]
        assert (err <= bound).all(), ("h", e, float((err / bound).max()))
        # the scale is that of the block's largest magnitude
        top = np.abs(h).reshape(h.shape[0], -1, 128).max(-1)
        dtop = dh.reshape(h.shape[0], -1, 128).max(-1)
        sc = hs.cpu().numpy()[r].astype(np.float64)
        assert (np.abs(sc * 448 - top) <= dtop + 2.0 ** -22 * top + 2.0 ** -99).all(), ("hs", e)
        y, mag = H[r] @ wd.T, np.abs(H[r]) @ np.abs(wd).T
        err = np.abs(Y[r] - y)
        bound = bf * mag + 2.0 ** -11 * np.abs(y) * 1.001 + 2.0 ** -25
        assert (err <= bound).all(), ("ys", e, float((err / bound).max()))


STAGES = [  # T, E, k, d, F, BM, skew
    (1, 8, 2, 128, 128, 16, 0.0), (1, 128, 8, 512, 256, 16, 0.0), (5, 4, 3, 256, 384, 7, 0.0),
    (32, 16, 4, 384, 128, 16, 0.0), (40, 8, 2, 256, 256, 32, 0.6), (300, 6, 2, 256, 128, 128, 0.0),
    (200, 32, 4, 128, 256, 128, 0.2), (17, 1, 1, 128, 128, 128, 0.0)]


@gpu
@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("T,E,k,d,F,BM,skew", STAGES)
def test_expert_stages_streaming(moe, T, E, k, d, F, BM, skew, act):
    out = _run_stages(moe, T, E, k, d, F, moe.REGIME_GEMV, BM, skew, act, T + E)
    _check_stages(*out)
    assert moe.device_status() == moe.OK


STAGES_TC = [  # T, E, k, d, F, skew
    (1, 8, 2, 128, 128, 0.0), (5, 4, 3, 256, 384, 0.0), (33, 16, 4, 384, 128, 0.0),
    (300, 6, 2, 256, 128, 0.0), (200, 32, 4, 128, 256, 0.2), (129, 1, 1, 640, 256, 0.0),
    (400, 3, 2, 1152, 640, 0.3), (37, 64, 8, 256, 128, 0.05), (70, 2, 1, 2176, 128, 0.0),
    (1000, 16, 4, 256, 640, 0.1), (600, 40, 4, 128, 512, 0.02), (500, 24, 6, 2048, 128, 0.0),
    # many rows to an expert: pairs of tiles, one expert of few rows
    (2000, 3, 2, 640, 640, 0.0), (1500, 5, 2, 768, 512, 2.0), (3333, 1, 1, 512, 384, 0.0)]


@gpu
@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("T,E,k,d,F,skew", STAGES_TC)
def test_expert_stages_tensor_cores(moe, T, E, k, d, F, skew, act):
    out = _run_stages(moe, T, E, k, d, F, moe.REGIME_TC, 128, skew, act, T + E)
    _check_stages(*out)
    assert moe.device_status() == moe.OK


@gpu
@pytest.mark.parametrize("regime", [1, 2])
def test_expert_stages_nan_rows_stay_their_own(moe, regime):
    T, E, k, d, F = 6, 4, 2, 256, 128
    ex = _experts(E, d, F, 3)
    idx = mi.random_topk_idx(T, E, k, 3).to(DEV)
    st = moe.sort_rows(idx, E, 128)
    x = torch.randn(T, d, device=DEV)
    x[4, 9] = float("inf")
    xq, xs = moe.quantize_fp8(x)
    hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, k, ex, regime)
    bad = (st.row_map.view(torch.int32) == 4).cpu().numpy()
    H = values(hq)
    assert np.isnan(H[bad]).all() and np.isfinite(H[~bad]).all()
    assert np.isfinite(hs.cpu().numpy()).all()
    ys = moe.grouped_down_fp8(hq, hs, st, T, k, ex, regime).cpu().numpy()
    assert np.isnan(ys[bad]).all() and np.isfinite(ys[~bad]).all()
    assert moe.device_status() == moe.ERR_RANGE          # as any ys that is not finite


@gpu
@pytest.mark.parametrize("M,N,K", [(20, 512, 384), (900, 2048, 256)])
def test_results_at_any_16_byte_boundary(moe, M, N, K):
    """An output that starts 16 but not 32 bytes into an allocation, for the
    split and the persistent tensor-core form; nothing beside it is written."""
    a, sa, b, sb = _operands(moe, M, N, K, 9)
    buf = torch.full((M * N + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = moe.fp8_matmul(a, sa, b, sb, out=buf[8:8 + M * N].view(M, N))
    _check_matmul(y, a, sa, b, sb, torch.bfloat16)
    assert (buf[:8] == 7).all() and (buf[8 + M * N:] == 7).all()
    # gate|up codes through the C call
    T, E, k, d, F = 700, 4, 2, 256, 2048
    ex = _experts(E, d, F, 1)
    idx = mi.random_topk_idx(T, E, k, 1).to(DEV)
    st = moe.sort_rows(idx, E, 128)
    xq, xs = moe.quantize_fp8(torch.randn(T, d, device=DEV))
    hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, k, ex, moe.REGIME_TC)
    h2 = torch.full((T * k * F + 32,), 9, dtype=torch.uint8, device=DEV)
    s2 = torch.empty_like(hs)
    e = moe.experts_struct(ex)
    assert moe.lib.moe_grouped_swiglu_fp8(
        xq.data_ptr(), xs.data_ptr(), st.row_map.data_ptr(), st.row_off.data_ptr(),
        st.tile_off.data_ptr(), 128, T, k, ctypes.byref(e), h2.data_ptr() + 16, s2.data_ptr(),
        moe.REGIME_TC, torch.cuda.current_stream().cuda_stream) == moe.OK
    assert torch.equal(h2[16:-16], hq.view(torch.uint8).flatten()) and torch.equal(s2, hs)
    assert (h2[:16] == 9).all() and (h2[-16:] == 9).all()


@gpu
def test_pack_gate_up_f8(moe):
    E, d, F = 3, 256, 128
    ex = _experts(E, d, F, 5)
    g, u = ex.w_gu[:, :F].contiguous(), ex.w_gu[:, F:].contiguous()
    sg, su = ex.s_gu[:, :1].contiguous(), ex.s_gu[:, 1:].contiguous()
    w, s, b = moe.pack_gate_up("f8", g, u, s_g=sg, s_u=su)
    assert torch.equal(w, ex.w_gu) and torch.equal(s, ex.s_gu) and b is None


@gpu
def test_waits_that_run_out(moe):
    """With a bound of one cycle the first wait of a tensor-core kernel that is
    not met gives up, the status says so, and the next call is as before."""
    a, sa, b, sb = _operands(moe, 100, 640, 4096, 1)          # the split form
    a2, sa2, b2, sb2 = _operands(moe, 1000, 3000 // 8 * 8, 512, 2)   # the persistent one
    ex = _experts(16, 512, 256, 7)
    idx = mi.random_topk_idx(300, 16, 4, 1).to(DEV)
    st = moe.sort_rows(idx, 16, 128)
    xq, xs = moe.quantize_fp8(torch.randn(300, 512, device=DEV))
    hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, 4, ex, moe.REGIME_TC)
    calls = [lambda: (moe.fp8_matmul(a, sa, b, sb),), lambda: (moe.fp8_matmul(a2, sa2, b2, sb2),),
             lambda: moe.grouped_swiglu_fp8(xq, xs, st, 4, ex, moe.REGIME_TC),
             lambda: (moe.grouped_down_fp8(hq, hs, st, 300, 4, ex, moe.REGIME_TC),)]
    for f in calls:
        ref = f()
        assert moe.device_status() == moe.OK
        moe.set_wait_cycles(1)
        try:
            f()
            assert moe.device_status() == moe.ERR_TIMEOUT
        finally:
            moe.set_wait_cycles(0)
        for got, want in zip(f(), ref):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
        assert moe.device_status() == moe.OK


@gpu
def test_same_bits_every_time(moe):
    """25 runs on the same inputs, the large forms among them."""
    a, sa, b, sb = _operands(moe, 700, 1500, 1168, 3)
    y = moe.fp8_matmul(a, sa, b, sb)
    z = moe.fp8_matmul(a[:90].contiguous(), sa[:90].contiguous(), b, sb)
    for _ in range(25):
        assert torch.equal(moe.fp8_matmul(a, sa, b, sb), y)
        assert torch.equal(moe.fp8_matmul(a[:90].contiguous(), sa[:90].contiguous(), b, sb), z)
    ex = _experts(24, 768, 640, 7)
    idx = mi.random_topk_idx(500, 24, 4, 1, 0.05).to(DEV)
    st = moe.sort_rows(idx, 24, 128)
    xq, xs = moe.quantize_fp8(torch.randn(500, 768, device=DEV))
    for rg in (moe.REGIME_TC, moe.REGIME_GEMV):
        hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, 4, ex, rg)
        ys = moe.grouped_down_fp8(hq, hs, st, 500, 4, ex, rg)
        for _ in range(25):
            h2, s2 = moe.grouped_swiglu_fp8(xq, xs, st, 4, ex, rg)
            assert torch.equal(h2.view(torch.uint8), hq.view(torch.uint8)) and torch.equal(s2, hs)
            assert torch.equal(moe.grouped_down_fp8(hq, hs, st, 500, 4, ex, rg), ys)


@gpu
def test_two_streams_at_once(moe):
    """The same calls on two streams that overlap give the bits of one."""
    a, sa, b, sb = _operands(moe, 200, 1024, 2048, 4)
    ex = _experts(16, 512, 256, 8)
    idx = mi.random_topk_idx(64, 16, 4, 2).to(DEV)
    st = moe.sort_rows(idx, 16, 128)
    x = torch.randn(64, 512, device=DEV)

    def step(stream=None):
        xq, xs = moe.quantize_fp8(x, stream=stream)
        hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, 4, ex, stream=stream)
        return [moe.fp8_matmul(a, sa, b, sb, stream=stream), xq, xs, hq, hs,
                moe.grouped_down_fp8(hq, hs, st, 64, 4, ex, stream=stream)]

    ref = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                out.append(step())
            out.append(step(s))
    torch.cuda.synchronize()
    for o in out:
        for g, w in zip(o, ref):
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


# ------------------------------------------------------------------ whole layer

@gpu
@pytest.mark.parametrize("T,E,k,d,F,act", [(1, 32, 8, 512, 256, "bf16"), (48, 16, 4, 256, 128, "f16"),
                                           (700, 8, 2, 512, 384, "bf16")])
def test_forward_with_f8_experts(moe, T, E, k, d, F, act):
    """The layer is its stages, bit for bit, eagerly and in a replayed graph;
    and near the 64-bit layer of the same quantised operands."""
    wl = mi.Workload("f8", T, d, E, k, F, act, "f8", "normal0.5")
    L = mi.make_layer(wl, 1, DEV)
    if E == 8:            # experts quantised by the library from bf16 weights, packed from gate and up
        g = torch.Generator(device=DEV).manual_seed(5)
        mk = lambda n, m: (torch.randn(E, n, m, generator=g, device=DEV) / m ** 0.5).bfloat16()  # noqa: E731
        (wg, sg), (wu, su), (wd, sd) = (moe.quantize_fp8(mk(n, m), 128)
                                        for n, m in ((F, d), (F, d), (d, F)))
        w_gu, s_gu, _ = moe.pack_gate_up("f8", wg, wu, s_g=sg, s_u=su)
        L.experts = mi.Experts("f8", E, d, F, w_gu, wd, s_gu, None, sd, None)
    y = moe.forward(L.x, L.w_router, L.router_bias, L.experts, k)
    lay = moe.forward_layout(T, d, E, k, F, L.x.dtype, "f8")
    logits, idx, w = moe.route(L.x, L.w_router, L.router_bias, k)
    st = moe.sort_rows(idx, E, lay.BM)
    xq, xs = moe.quantize_fp8(L.x)
    hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, k, L.experts)
    ys = moe.grouped_down_fp8(hq, hs, st, T, k, L.experts)
    y2 = moe.combine(ys, st.inv_order, w, T, k, L.x.dtype)
    assert torch.equal(y, y2)
    _check_stages(L.experts, st, xq, xs, hq, hs, ys)
    # the router's statistics of the same step count what the sort dispatched
    b = moe.balance_loss(logits, idx, 1.0)
    assert torch.equal(b.counts[0], st.counts)

    ws = moe.forward_workspace(L.x, L.experts, k)
    out = torch.empty_like(L.x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.forward(L.x, L.w_router, L.router_bias, L.experts, k, ws=ws, out=out)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        moe.forward(L.x, L.w_router, L.router_bias, L.experts, k, ws=ws, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)

    X = dequantize(xq, xs)
    ii, ww = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    ref = np.zeros((T, d))
    for e in range(E):
        t, j = np.nonzero(ii == e)
        if not len(t):
            continue
        wg, wu, wd = _dense(L.experts, e)
        h = act64(X[t] @ wg.T, "swiglu") * (X[t] @ wu.T)
        hq64, hs64 = quantize_ref(h.astype(np.float32))
        H = hq64 * np.repeat(hs64.astype(np.float64), 128, 1)
        np.add.at(ref, t, ww[t, j][:, None] * (H @ wd.T))
    assert np.abs(y.double().cpu().numpy() - ref).max() <= 2e-2 * rms(ref)
    assert moe.device_status() == moe.OK
