"""The few-token layer (bf16 and MXFP8, two kernels) on a B200 against the float64 oracle."""

import numpy as np
import pytest
import torch

from gpu_common import SMALL, check_routing, device_weights, require_gpu, to_np, weights
from mixture_experts_transformer_b200 import binding as B
from mixture_experts_transformer_b200 import block, inputs
from oracle import moe_oracle as mo
from oracle import sandwich as sw
from test_gpu_mxfp8 import check_block, dequant

pytestmark = pytest.mark.gpu

ODD = inputs.Dims(embed_dim=320, num_experts=24, expert_dim=64, hidden_dim=448)
TINY = inputs.Dims(embed_dim=64, num_experts=8, expert_dim=64, hidden_dim=64)
TALL = inputs.Dims(embed_dim=4096, num_experts=8, expert_dim=192, hidden_dim=64)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def ok():
    st = B.moe_get_device_status()
    assert st == B.MOE_OK, B.moe_status_string(st)


def ffn_bound(x, wg, wu, wd):
    """(y, bound): fp32 sums (K 2^-24 of the products' absolute sum), a GeGLU good to 2^-19, rows held to 2^-16
    (two bf16 values), whatever the order of the sums."""
    x, wg, wu, wd = (mo.f64(a) for a in (x, wg, wu, wd))
    eps = 2.0**-24
    z, u = x @ wg, x @ wu
    dz, du = x.shape[1] * eps * (np.abs(x) @ np.abs(wg)), x.shape[1] * eps * (np.abs(x) @ np.abs(wu))
    g = mo.gelu_tanh(z)
    h = g * u
    dh = 1.13 * dz * (np.abs(u) + du) + np.abs(g) * du + (2.0**-19 + 2.0**-16) * np.abs(h)
    aw = np.abs(wd)
    return h @ wd, dh @ aw + 2 * h.shape[1] * eps * ((np.abs(h) + dh) @ aw)


def layer_bound(w, x, idx, wts, lo=0, hi=None, hidden=None):
    h0, h1 = hidden or (0, w.sg.shape[1])
    out, tol = ffn_bound(x, w.sg[:, h0:h1], w.su[:, h0:h1], w.sd[h0:h1])
    for e in np.unique(idx):
        if not lo <= e < (hi or w.wg.shape[0]):
            continue
        t, k = np.nonzero(idx == e)
        y, d = ffn_bound(x[t], w.wg[e], w.wu[e], w.wd[e])
        wk = wts[t, k][:, None].astype(np.float64)
        out[t] += wk * y
        tol[t] += wk * d + 2.0**-22 * np.abs(wk * y)
    # up to 150 parts of a sum, added in fp32
    return out, tol + 150 * 2.0**-24 * np.abs(out).max(-1, keepdims=True)


def check(w, xb, res, k, bias=None, xin=None):
    xin = xb if xin is None else xin
    idx, wts = to_np(res.idx), to_np(res.w)
    ref_idx, ref_w, logits = mo.route(xin, w.w_router, k, bias)
    check_routing(logits, ref_idx, ref_w, idx, wts, k)
    np.testing.assert_allclose(to_np(res.logits), logits, atol=1e-5 * max(1.0, np.abs(logits).max()))
    out, tol = layer_bound(w, xin, idx, wts)
    got = to_np(res.out_f32).astype(np.float64)
    assert np.all(np.abs(got - out) <= tol), np.max(np.abs(got - out) / tol)
    np.testing.assert_array_equal(to_np(res.out.float()), to_np(res.out_f32.bfloat16().float()))
    np.testing.assert_array_equal(to_np(res.cnt), np.bincount(idx.reshape(-1), minlength=w.w_router.shape[1]))


CASES = [(TINY, 1, 1), (TINY, 3, 8), (SMALL, 1, 4), (SMALL, 7, 4), (SMALL, 8, 2), (SMALL, 9, 4), (SMALL, 16, 16),
         (ODD, 2, 8), (ODD, 13, 3), (ODD, 16, 24), (TALL, 5, 2), (TALL, 16, 8)]


@pytest.mark.parametrize("dims,T,k", CASES)
def test_few_against_oracle(dims, T, k):
    w, dw = weights(dims), device_weights(dims)
    xb = inputs.make_x(T, dims.embed_dim, seed=T)
    bias = inputs.zipf_router_bias(dims.num_experts) if T == 9 else None
    bt = None if bias is None else torch.from_numpy(bias).cuda()
    res = block.forward_few(dw, block.bf16_tensor(xb), top_k=k, router_bias=bt, debug=True)
    ok()
    assert B.moe_last_launch_count() == 2
    check(w, xb, res, k, bias)


@pytest.mark.parametrize("dims,T,k", CASES)
@pytest.mark.parametrize("fed", [False, True])
def test_few_mxfp8_against_oracle(dims, T, k, fed):
    w, dw = weights(dims), device_weights(dims)
    mw = block.quantize_mxfp8(dw)
    xb = inputs.make_x(T, dims.embed_dim, seed=T)
    xq = xs = xv = None
    if fed:
        xq, xs = block.quantize_mxfp8_rows(block.bf16_tensor(inputs.make_x(T, dims.embed_dim, seed=T + 1)))
        xv = dequant(xq, xs)
    bias = inputs.zipf_router_bias(dims.num_experts) if T == 9 else None
    bt = None if bias is None else torch.from_numpy(bias).cuda()
    res = block.forward_mxfp8(mw, block.bf16_tensor(xb), xq=xq, xs=xs, top_k=k, router_bias=bt, debug=True)
    ok()
    assert B.moe_last_launch_count() == 2
    check_block(w, xb, res, k, bias, xv)


@pytest.mark.parametrize("T", [1, 8, 16])
def test_few_gemma_shapes(T):
    w, dw = weights(), device_weights()
    xb = inputs.make_x(T, seed=100 + T)
    x = block.bf16_tensor(xb)
    res = block.forward_few(dw, x, debug=True)
    ok()
    check(w, xb, res, 8)
    # the whole block within its own rounding of the few-token form
    whole = block.forward(dw, x, debug=True)
    ok()
    rms = float(whole.out_f32.square().mean().sqrt())
    assert float((whole.out_f32 - res.out_f32).abs().max()) <= 2e-2 * rms
    assert torch.equal(whole.idx, res.idx)
