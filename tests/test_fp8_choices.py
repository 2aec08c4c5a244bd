"""Calls of the e4m3 operators that take a kernel, or two, which the sizes of the
other tests do not: a K shorter than one block on the tensor cores, and a layer
whose gate|up streams weights while its down product does not."""
import pytest
import torch

import moe_inputs as mi
import test_fp8 as tf

gpu = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_mixture_experts_top_b200 as m
    return m


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(3000, 3000, 16), (2000, 2000, 112), (9, 700000, 48)])
def test_a_single_partial_block_on_the_tensor_cores(moe, dtype, M, N, K):
    """(Past 8 rows, the choice goes by 32-row passes over the weights: these
    have 2^21 bytes of them or more.)"""
    assert M > 8 and -(-M // 32) * N * K > 1 << 21
    a, sa, b, sb = tf._operands(moe, M, N, K, M + N + K)
    y = moe.fp8_matmul(a, sa, b, sb, dtype)
    rows = torch.randperm(N, generator=torch.Generator().manual_seed(1))[:2000].sort().values
    rows[-1] = N - 1
    blocks = rows // 128
    A, B = tf.dequantize(a, sa), tf.values(b[rows.to(DEV)]) * sb.cpu().numpy()[blocks].astype("f8")
    ref, mag = A @ B.T, abs(A) @ abs(B).T
    u = torch.finfo(dtype).eps / 2
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    err = abs(y[:, rows.to(DEV)].double().cpu().numpy() - ref)
    assert (err <= tf.sum_bound(K) * mag + u * abs(ref) * (1 + 1e-3) + sub).all()
    assert moe.device_status() == moe.OK


@gpu
@pytest.mark.parametrize("T,E,k,d,F,up,down", [(1, 128, 8, 2048, 768, 1, 2), (2, 16, 2, 256, 4096, 2, 1)])
def test_forward_takes_a_kernel_for_each_product(moe, T, E, k, d, F, up, down):
    """One token: 384 CTAs of gate|up, one wave, and 1,024 of down; and the other
    way round."""
    wl = mi.Workload("f8", T, d, E, k, F, "bf16", "f8", "normal0.5")
    L = mi.make_layer(wl, 1, DEV)
    y = moe.forward(L.x, L.w_router, L.router_bias, L.experts, k)
    assert moe.forward_layout(T, d, E, k, F, L.x.dtype, "f8").regime == up
    logits, idx, w = moe.route(L.x, L.w_router, L.router_bias, k)
    st = moe.sort_rows(idx, E, moe.sort_block_m())
    xq, xs = moe.quantize_fp8(L.x)
    hq, hs = moe.grouped_swiglu_fp8(xq, xs, st, k, L.experts, up)
    ys = moe.grouped_down_fp8(hq, hs, st, T, k, L.experts, down)
    assert torch.equal(y, moe.combine(ys, st.inv_order, w, T, k, L.x.dtype))
    for a, b in zip(moe.grouped_swiglu_fp8(xq, xs, st, k, L.experts), (hq, hs)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(moe.grouped_down_fp8(hq, hs, st, T, k, L.experts), ys)
    tf._check_stages(L.experts, st, xq, xs, hq, hs, ys)
    assert moe.device_status() == moe.OK
