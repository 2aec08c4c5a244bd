"""gate|up of e4m3 experts where the gate activation is small: blocks of 128
features whose gates are all strongly negative, against 64-bit forms that do not
cancel there."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
from fp8_util import dequantize, sum_bound

gpu = pytest.mark.gpu
DEV = "cuda"
C = np.sqrt(2 / np.pi)
BLOCKS = ((-3.2, -3.0), (-4.5, -4.0), (-6.0, -5.0), (-6.0, -3.0), (-9.0, -7.0))   # gates of each


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_mixture_experts_top_b200 as m
    return m


def act_slope_error(g, act):
    """The activation, its slope and the relative error of its fp32 form, in
    fp64: g s(x) with s the logistic function, x = g for SwiGLU and 2z for the
    tanh form of GELU. Error: the argument's roundings, for GELU four of them
    (|x| 2^-24 each); the fast exponential's 2 + 1.16 |x| units of 2^-23; the
    division's two; sum and product."""
    x = g if act == "swiglu" else 2 * C * (g + 0.044715 * g ** 3)
    dx = 1.0 if act == "swiglu" else 2 * C * (1 + 3 * 0.044715 * g ** 2)
    s = 1 / (1 + np.exp(-x))
    err = (8 + (1.16 + (0 if act == "swiglu" else 2)) * np.abs(x)) * 2.0 ** -23
    return g * s, s + g * s / (1 + np.exp(x)) * dx, err


def test_the_activation_is_the_tanh_form():
    g = np.linspace(-4, 4, 81)
    a, da, _ = act_slope_error(g, "geglu")
    np.testing.assert_allclose(a, 0.5 * g * (1 + np.tanh(C * (g + 0.044715 * g ** 3))), rtol=1e-9,
                               atol=1e-15)
    h = 1e-5
    d = (act_slope_error(g + h, "geglu")[0] - act_slope_error(g - h, "geglu")[0]) / (2 * h)
    np.testing.assert_allclose(da, d, atol=1e-8)


def experts(moe, E, d, seed):
    """Experts whose gates lie in BLOCKS for token rows of values 1 .. 1.1."""
    g = torch.Generator().manual_seed(seed)
    F = 128 * len(BLOCKS)
    target = torch.cat([lo + (hi - lo) * torch.rand(E, 128, generator=g) for lo, hi in BLOCKS], 1)
    wg = target[..., None] / (1.05 * d) * (0.95 + 0.1 * torch.rand(E, F, d, generator=g))
    wu = torch.randn(E, F, d, generator=g) / d ** 0.5
    w_gu, s_gu = moe.quantize_fp8(torch.cat([wg, wu], 1).to(DEV), 128)
    w_dn, s_dn = moe.quantize_fp8(torch.randn(E, d, F, generator=g).to(DEV), 128)
    return mi.Experts("f8", E, d, F, w_gu, w_dn, s_gu, None, s_dn, None)


@gpu
@pytest.mark.parametrize("act", ["geglu", "swiglu"])
@pytest.mark.parametrize("T,E,k,d,regime", [(3, 4, 2, 256, 1), (3, 4, 2, 256, 2), (40, 2, 1, 1152, 2),
                                            (2000, 4, 2, 256, 2), (700, 4, 2, 128, 1)])
def test_gates_far_below_zero(moe, act, T, E, k, d, regime):
    ex = experts(moe, E, d, T + d).with_act(act)
    idx = mi.random_topk_idx(T, E, k, T).to(DEV)
    st = moe.sort_rows(idx, E, 128)
    x = 1 + 0.1 * torch.rand(T, d, generator=torch.Generator().manual_seed(T))
    xq, xs = moe.quantize_fp8(x.to(DEV))
    hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, k, ex, regime)
    X, H, S = dequantize(xq, xs), dequantize(hq, hs), hs.cpu().numpy().astype(np.float64)
    off, tok = st.row_off.cpu().numpy(), st.row_map.cpu().view(torch.int32).numpy()
    F, b = ex.F, sum_bound(d)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if r.start == r.stop:
            continue
        w = dequantize(ex.w_gu[e], ex.s_gu[e], 128)
        xr = X[tok[r]]
        g, u = xr @ w[:F].T, xr @ w[F:].T
        assert g.max() < -2.7 and g.min() > -9.7
        a, da, err = act_slope_error(g, act)
        h = a * u
        # the products' sums, then the activation and its product
        dh = (np.abs(u * da) * b * (np.abs(xr) @ np.abs(w[:F]).T) +
              np.abs(a) * b * (np.abs(xr) @ np.abs(w[F:]).T)) * 1.01 + err * np.abs(h)
        each = np.repeat(S[r], 128, 1)
        # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale among the
        # subnormal codes
        bound = dh + (2.0 ** -4 + 2.0 ** -20) * (np.abs(h) + dh) + 2.0 ** -10 * each
        off_by = np.abs(H[r] - h)
        assert (off_by <= bound).all(), (e, float((off_by / bound).max()))
        top = np.abs(h).reshape(len(h), -1, 128).max(-1)
        dtop = dh.reshape(len(h), -1, 128).max(-1)
        assert (np.abs(S[r] * 448 - top) <= dtop + 2.0 ** -22 * top).all(), \
            float((np.abs(S[r] * 448 / top - 1) / (dtop / top)).max())
        # every block keeps its largest code
        assert (np.abs(H[r]).reshape(len(h), -1, 128).max(-1) >= 447 * S[r]).all()
    assert moe.device_status() == moe.OK
