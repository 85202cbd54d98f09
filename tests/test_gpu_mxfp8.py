"""The residual-add norm and the MXFP8 block on a B200 against float64."""

import numpy as np
import pytest
import torch

from gpu_common import SMALL, check_routing, device_weights, require_gpu, to_np, w_args, weights
from mixture_experts_transformer_b200 import binding as B
from mixture_experts_transformer_b200 import block, inputs
from oracle import moe_oracle as mo
from oracle import mxfp8 as mx
from oracle import sandwich as sw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def ok():
    assert B.moe_get_device_status() == B.MOE_OK


def dequant(q: torch.Tensor, scale: torch.Tensor) -> np.ndarray:
    s = to_np(scale.float()).astype(np.float64)
    return to_np(q.float()).astype(np.float64) * np.repeat(s, 32, -1)


# ------------------------------------------------------------------ the norm

# fp32 arithmetic of a row: a sum of D squares in at most D / (8 lanes' order) steps, a square root, a divide and
# three products keep y within 2^-18 of |gamma| (|residual| + |x|) / rms for every D here (a thread adds at most 32
# squares in order, then 5 + 16 tree steps: 53 roundings of 2^-24 on the mean, half of that on its root; the rest a
# dozen roundings).
FP32 = 2.0**-18


@pytest.mark.parametrize("T,D", [(1, 8), (3, 40), (5, 256), (7, 264), (2, 1024), (9, 1032), (4, 2560), (65, 2816),
                                 (3, 4096), (2, 4104), (3, 8192), (2, 16384)])
@pytest.mark.parametrize("post,res,gam", [(True, True, True), (False, True, True), (False, False, False),
                                          (True, False, True)])
def test_add_norm(T, D, post, res, gam):
    rng = np.random.default_rng(T * 10007 + D)
    bits = lambda *s: inputs.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    xb, rb, gb, pb = bits(T, D), bits(T, D), bits(D), bits(D)
    x, r, g, p = (block.bf16_tensor(b) for b in (xb, rb, gb, pb))
    quant = D % 32 == 0
    out = block.add_rms_norm(x, g if gam else None, residual=r if res else None, gamma_post=p if post else None,
                             quantize=quant)
    ok()
    xv = mo.f64(xb)
    a = sw.rms_norm(xv, mo.f64(pb)) if post else xv
    rv = mo.f64(rb) if res else 0.0
    s = rv + a
    gv = mo.f64(gb) if gam else np.ones(D)
    rms = np.sqrt((s * s).mean(-1, keepdims=True) + 1e-6)
    y = gv * s / rms
    mag = np.abs(rv) + np.abs(a)
    es = FP32 * mag
    # an error of s moves its row's rms by at most the largest relative one
    ey = np.abs(gv) / rms * es + np.abs(y) * (FP32 + np.sqrt((es * es).mean(-1, keepdims=True)) / rms)
    assert np.all(np.abs(to_np(out.sum.double()) - s) <= 2.0**-8 * np.abs(s) + es)
    assert np.all(np.abs(to_np(out.y.double()) - y) <= 2.0**-8 * np.abs(y) + ey * 1.01)
    if not quant:
        return
    got = dequant(out.q, out.scale)
    q, j = mx.quantize(y)
    jr = np.log2(to_np(out.scale.float()).astype(np.float64))
    amax = np.abs(y).reshape(T, D // 32, 32).max(-1)
    border = np.abs(amax / (448 * np.exp2(j.astype(np.float64))) - 1) < 1e-4  # the fp32 amax may pass the border
    border |= np.abs(amax / (224 * np.exp2(j.astype(np.float64))) - 1) < 1e-4
    assert np.all((jr == j) | border)
    step = np.repeat(np.exp2(jr), 32, -1)
    assert np.all(np.abs(got - y) <= np.maximum(2.0**-4 * np.abs(y), 2.0**-10 * step) + 1.07 * ey)
    if gam:
        assert np.mean(got != q * np.repeat(np.exp2(j.astype(np.float64)), 32, -1)) < 1e-2


def test_add_norm_special_rows():
    """Zero rows, a zero group, infinities and NaN, the largest and smallest values."""
    T, D = 6, 256
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    x[1, 32:64] = 3.0
    x[2] = 1.0
    x[2, 40] = float("inf")
    x[3] = 1.0
    x[3, 100] = float("nan")
    x[4] = torch.finfo(torch.bfloat16).max / 2**70
    x[5] = 1e-30
    r = block.add_rms_norm(x, quantize=True)
    ok()
    y, q, s = r.y.float(), r.q.float(), r.scale.view(torch.uint8)
    assert torch.equal(y[0], torch.zeros(D, device="cuda")) and torch.all(q[0] == 0) and torch.all(s[0] == 0)
    assert torch.all(q[1, :32] == 0) and s[1, 0] == 0 and torch.all(q[1, 32:64] != 0) and torch.all(q[1, 64:] == 0)
    assert torch.isnan(y[2, 40]) and torch.all(y[2, :40] == 0)  # inf / inf, 1 / inf
    assert s[2, 1] == 0xFF and torch.isnan(q[2, 32:64]).all() and torch.all(q[2, :32] == 0)
    assert torch.isnan(y[3]).all() and torch.all(s[3] == 0xFF) and torch.isnan(q[3]).all()
    assert torch.all(y[4] == 1.0)
    ref = 1e-30 / np.sqrt(1e-6)
    np.testing.assert_allclose(to_np(y[5]), ref, rtol=2.0**-7)
    # 2^-127 scales: the row's values sit below 448 2^-127 only when tiny; here they round to the nearest e4m3
    assert torch.all(q[5] * r.scale.float()[5].repeat_interleave(32) > 0)


def test_add_norm_in_place_and_optional_outputs():
    T, D = 33, 2816
    x = block.bf16_tensor(inputs.make_x(T, D, seed=5))
    res = block.bf16_tensor(inputs.make_x(T, D, seed=6))
    g = block.bf16_tensor(inputs.make_x(1, D, seed=7)[0])
    ref = block.add_rms_norm(x, g, residual=res, gamma_post=g, quantize=True)
    x2, r2 = x.clone(), res.clone()
    got = block.add_rms_norm(x2, g, residual=r2, gamma_post=g, y=x2, sum_out=r2)
    ok()
    assert torch.equal(got.y, ref.y) and torch.equal(r2, ref.sum) and got.y.data_ptr() == x2.data_ptr()
    q = torch.empty((T, D), dtype=torch.uint8, device="cuda")
    s = torch.empty((T, D // 32), dtype=torch.uint8, device="cuda")
    p = B.MoeNormParams(T, D, 0.0, x.data_ptr(), res.data_ptr(), g.data_ptr(), g.data_ptr(), None, None, q.data_ptr(),
                        s.data_ptr())
    B.check(B.moe_add_rms_norm(p), "8 bits only")
    ok()
    assert torch.equal(q, ref.q.view(torch.uint8)) and torch.equal(s, ref.scale.view(torch.uint8))
    assert torch.equal(block.add_rms_norm(x[:0], g).y, x[:0])
    with pytest.raises(ValueError):
        block.add_rms_norm(x.t(), g)
    with pytest.raises(ValueError):
        block.add_rms_norm(x[:, ::2], None)
    with pytest.raises(ValueError):
        block.add_rms_norm(x.float(), g)
    with pytest.raises(ValueError):
        block.add_rms_norm(x, g[:-8])
    with pytest.raises(ValueError):
        block.add_rms_norm(x.cpu(), None)
    with pytest.raises(B.MoeError):
        block.add_rms_norm(x, g, y=x, sum_out=x)


# ------------------------------------------------------------- quantisers


def test_quantisers_bit_exact():
    rng = np.random.default_rng(11)
    G, K, N = 3, 320, 192
    w = (rng.standard_normal((G, K, N)) * np.exp2(rng.uniform(-30, 30, (G, 1, N)))).astype(np.float32)
    w[0, :32, 3] = 0
    w[1, 32:64, 5] = [448.0 * 2.0**i for i in range(-16, 16)]
    wb = inputs.f32_to_bf16_bits(w)
    lin = block.quantize_mxfp8_linear(block.bf16_tensor(wb))
    ok()
    q, j = mx.quantize(np.swapaxes(mo.f64(wb), 1, 2))
    np.testing.assert_array_equal(to_np(lin.q.float()), q)
    sf = to_np(lin.sf.view(torch.uint8)).reshape(G, -1)
    used = np.zeros(sf.shape[1], bool)
    for n in range(N):
        for c in range(K // 32):
            o = mx.scale_tile_offset(n, c, K)
            used[o] = True
            np.testing.assert_array_equal(sf[:, o], j[:, n, c] + 127)
    assert np.all(sf[:, ~used] == 0)
    x = block.bf16_tensor(wb[0].T.copy())  # [N, K]
    xq, xs = block.quantize_mxfp8_rows(x)
    ok()
    np.testing.assert_array_equal(to_np(xq.float()), q[0])
    np.testing.assert_array_equal(to_np(xs.view(torch.uint8)), j[0] + 127)


# ------------------------------------------------------------- the block


def hidden_slack(xv, wg, wu):
    """(MXFP8 GeGLU rows, how far the GPU's may be from them): an fp32 sum of K products p is within K 2^-24 sum|p| of
    the exact one, gelu adds 2^-20 of its value (its slope is below 1.13), and a value that close to a rounding
    border may take the neighbouring code."""
    z, u = xv @ wg, xv @ wu
    K = xv.shape[1]
    dz, du = K * 2.0**-24 * (np.abs(xv) @ np.abs(wg)), K * 2.0**-24 * (np.abs(xv) @ np.abs(wu))
    g = mo.gelu_tanh(z)
    h = g * u
    d = 1.13 * dz * (np.abs(u) + du) + np.abs(g) * du + 2.0**-19 * np.abs(h)
    ref = mx.values(h)
    near = np.maximum(np.abs(mx.values(h + d) - ref), np.abs(mx.values(h - d) - ref))
    q, j = mx.quantize(h)
    # a group whose largest value sits at the border of its scale may take the other scale
    grp = np.abs(h).reshape(*h.shape[:-1], -1, 32)
    dm = d.reshape(grp.shape).max(-1)
    top = 448 * np.exp2(j.astype(np.float64))
    flip = (top - grp.max(-1) < dm) | (grp.max(-1) - top / 2 < dm)
    near = np.where(np.repeat(flip, 32, -1), np.maximum(near, 2.0**-3 * np.abs(h)), near)
    return ref, near


def block_reference(w, x_bits, idx, wts, xv=None):
    """(out, bound) in float64 for a given routing. Beside the GeGLU rows' slack: fp32 sums of the down products and
    the bf16 storage of the routed outputs (2^-8 of each, weighted)."""
    xv = mx.values(mo.f64(x_bits)) if xv is None else xv

    def ffn(rows, wg, wu, wd):
        h, near = hidden_slack(rows, mx.weight_values(wg), mx.weight_values(wu))
        wd = mx.weight_values(wd)
        mag = np.abs(h) @ np.abs(wd)
        return h @ wd, near @ np.abs(wd) + h.shape[1] * 2.0**-24 * mag

    out, tol = ffn(xv, w.sg, w.su, w.sd)
    for e in np.unique(idx):
        t, k = np.nonzero(idx == e)
        y, d = ffn(xv[t], w.wg[e], w.wu[e], w.wd[e])
        wk = wts[t, k][:, None].astype(np.float64)
        out[t] += wk * y
        tol[t] += wk * (d + 2.0**-8 * (np.abs(y) + d) + 2.0**-20 * np.abs(y))
    return out, tol + 2.0**-20 * np.abs(out)


def check_block(w, x_bits, res, k, bias=None, xv=None):
    idx, wts = to_np(res.idx), to_np(res.w)
    ref_idx, ref_w, logits = mo.route(x_bits, w.w_router, k, bias)
    check_routing(logits, ref_idx, ref_w, idx, wts, k)
    out, tol = block_reference(w, x_bits, idx, wts, xv)
    got = to_np(res.out_f32).astype(np.float64)
    assert np.all(np.abs(got - out) <= tol), np.max(np.abs(got - out) / tol)
    rms = np.sqrt(np.mean(out**2))
    print("max err / rms", np.abs(got - out).max() / rms, "bound", tol.max() / rms)
    np.testing.assert_array_equal(to_np(res.out.float()), to_np(res.out_f32.bfloat16().float()))
    np.testing.assert_array_equal(to_np(res.cnt), np.bincount(idx.reshape(-1), minlength=w.w_router.shape[1]))


ODD = inputs.Dims(embed_dim=320, num_experts=24, expert_dim=64, hidden_dim=448)


@pytest.mark.parametrize("dims,T,k", [(SMALL, 17, 4), (SMALL, 130, 4), (SMALL, 300, 2), (ODD, 33, 8), (ODD, 129, 1),
                                      (ODD, 64, 24)])
@pytest.mark.parametrize("fed", [False, True])
def test_block_against_oracle(dims, T, k, fed):
    w, dw = weights(dims), device_weights(dims)
    mw = block.quantize_mxfp8(dw)
    xb = inputs.make_x(T, dims.embed_dim, seed=T)
    x = block.bf16_tensor(xb)
    xq = xs = xv = None
    if fed:  # rows of their own, as a norm's fp32 result would give
        rows = block.bf16_tensor(inputs.make_x(T, dims.embed_dim, seed=T + 1))
        xq, xs = block.quantize_mxfp8_rows(rows)
        xv = dequant(xq, xs)
    bias = None
    if T == 130:
        bias = inputs.zipf_router_bias(dims.num_experts)
    res = block.forward_mxfp8(mw, x, xq=xq, xs=xs, top_k=k, debug=True,
                              router_bias=None if bias is None else torch.from_numpy(bias).cuda())
    ok()
    check_block(w, xb, res, k, bias, xv)


@pytest.mark.parametrize("T,k", [(1100, 4), (2000, 2)])
def test_large_skewed_batches(T, k):
    """Experts with many and with no rows (Zipf bias): a sample of tokens against the oracle, root mean square: the
    routed outputs' bf16 storage alone (2^-8 of each at most) bounds it up to rare flipped codes of the GeGLU rows."""
    w, dw = weights(SMALL), device_weights(SMALL)
    mw = block.quantize_mxfp8(dw)
    xb = inputs.make_x(T, SMALL.embed_dim, seed=T)
    bias = 2 * inputs.zipf_router_bias(SMALL.num_experts)
    buf = torch.full((T + 3, SMALL.embed_dim), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = block.mxfp8_workspace(mw, T, k)
    res = block.forward_mxfp8(mw, block.bf16_tensor(xb), top_k=k, debug=True, out=buf[:T], workspace=ws,
                              router_bias=torch.from_numpy(bias).cuda())
    ok()
    assert torch.all(buf[T:] == 7.0)
    cnt = to_np(res.cnt)
    assert cnt.sum() == T * k and cnt.max() > T // 2
    tok = np.arange(0, T, 7)
    idx, wts = to_np(res.idx)[tok], to_np(res.w)[tok]
    out = mx.block(xb[tok], w.w_router, w.wg, w.wu, w.wd, w.sg, w.su, w.sd, k, routing=(idx, wts))
    err = to_np(res.out_f32)[tok] - out
    assert np.sqrt(np.mean(err**2)) <= 2.0**-8 * np.sqrt(np.mean(out**2))
    again = block.forward_mxfp8(mw, block.bf16_tensor(xb), top_k=k, router_bias=torch.from_numpy(bias).cuda())
    ok()
    assert torch.equal(again.out, res.out)


def test_large_batch_graph_and_refusals():
    dw = device_weights(SMALL)
    mw = block.quantize_mxfp8(dw)
    T = 100
    x = block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=3))
    ws = block.mxfp8_workspace(mw, T, 4)
    ref = block.forward_mxfp8(mw, x, top_k=4, workspace=ws).out.clone()
    out = torch.zeros_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        block.forward_mxfp8(mw, x, top_k=4, workspace=ws, out=out)
    g.replay()
    torch.cuda.synchronize()
    ok()
    assert torch.equal(out, ref)
    del g
    f = B.moe_block_forward_mxfp8
    assert f(block.mxfp8_params(mw, T, x, out, top_k=4, workspace=ws[:-256])) == B.MOE_ERR_WORKSPACE
    assert f(block.mxfp8_params(mw, T, x, out, top_k=4, workspace=ws[16:])) == B.MOE_ERR_ALIGNMENT
    assert f(block.mxfp8_params(mw, T, x, x, top_k=4, workspace=ws)) == B.MOE_ERR_INVALID_ARG
    q, sc = block.quantize_mxfp8_rows(x)
    with pytest.raises(B.MoeError):
        block.forward_mxfp8(mw, x, xq=q, top_k=4)
    with pytest.raises(ValueError):
        block.forward_mxfp8(mw, x, xq=q.float(), xs=sc, top_k=4)
    with pytest.raises(ValueError):
        block.forward_mxfp8(mw, x, xq=q, xs=sc[:, :-1], top_k=4)
    ok()


# -------------------------------------------- offsets that pass 32 bits


def test_rows_past_32_bit_offsets():
    """2.2e9 elements: the rows behind the 2^31 and 2^32 byte and element borders equal the same rows alone."""
    T, D = 134_500, 16384
    assert T * D > 2**31
    x = torch.empty((T, D), dtype=torch.bfloat16, device="cuda").normal_()
    gamma = torch.empty(D, dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1.5)
    res = torch.empty_like(x).normal_()
    big = block.add_rms_norm(x, gamma, residual=res, gamma_post=gamma, quantize=True)
    qx, sx = block.quantize_mxfp8_rows(x)
    ok()
    for r in (0, 2**31 // D - 1, 2**31 // D, 2**30 // D, T - 3):
        rows = slice(max(0, r - 1), r + 3)
        one = block.add_rms_norm(x[rows].clone(), gamma, residual=res[rows].clone(), gamma_post=gamma, quantize=True)
        for a, b in ((big.y, one.y), (big.sum, one.sum), (big.q, one.q), (big.scale, one.scale)):
            assert torch.equal(a[rows].view(torch.uint8), b.view(torch.uint8))
        q, s = block.quantize_mxfp8_rows(x[rows].clone())
        assert torch.equal(qx[rows].view(torch.uint8), q.view(torch.uint8))
        assert torch.equal(sx[rows].view(torch.uint8), s.view(torch.uint8))
    ok()


def test_batch_past_32_bit_offsets():
    """70000 tokens of 4096 on all 8 experts: 560000 routed rows, 2.3e9 elements."""
    dims = inputs.Dims(embed_dim=4096, num_experts=8, expert_dim=64, hidden_dim=64)
    w, dw = weights(dims), device_weights(dims)
    mw = block.quantize_mxfp8(dw)
    T = 70_000
    assert T * 8 * dims.embed_dim > 2**31
    x = torch.empty((T, dims.embed_dim), dtype=torch.bfloat16, device="cuda").normal_()
    res = block.forward_mxfp8(mw, x, top_k=8, debug=True)
    ok()
    tok = np.array([0, 1, 32767, 32768, 65535, 65536, T - 129, T - 1])
    xb = to_np(x[torch.from_numpy(tok)].view(torch.int16)).view(np.uint16)
    idx, wts = to_np(res.idx)[tok], to_np(res.w)[tok]
    out = mx.block(xb, w.w_router, w.wg, w.wu, w.wd, w.sg, w.su, w.sd, 8, routing=(idx, wts))
    err = to_np(res.out_f32)[tok] - out
    # the routed outputs' bf16 storage (2^-9 rms each) and rare flipped codes, per token
    assert np.all(np.sqrt(np.mean(err**2, -1)) <= 2.0**-8 * np.sqrt(np.mean(out**2, -1)))


def test_weights_past_32_bit_offsets():
    """128 experts of 4096 x 4160: 2.2e9 elements a matrix. The last eight equal the same eight alone, bit for bit:
    quantised, and in both few-token forms and the grouped GEMMs."""
    G, K, N, S = 128, 4096, 4160, 64
    assert G * K * N > 2**31

    def rand(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, 0.02)

    big = block.DeviceWeights(inputs.Dims(K, G, N, S), rand(K, G), rand(G, K, N), rand(G, K, N), rand(G, N, K), rand(K, S),
                              rand(K, S), rand(S, K))
    last = block.DeviceWeights(inputs.Dims(K, 8, N, S), big.w_router[:, -8:].contiguous(), big.wg[-8:], big.wu[-8:],
                               big.wd[-8:], big.sg, big.su, big.sd)
    mbig, mlast = block.quantize_mxfp8(big), block.quantize_mxfp8(last)
    ok()
    assert torch.equal(mbig.wg.q[-8:].view(torch.uint8), mlast.wg.q.view(torch.uint8))
    assert torch.equal(mbig.wd.q[-8:].view(torch.uint8), mlast.wd.q.view(torch.uint8))
    n = mlast.wu.sf.numel()
    assert torch.equal(mbig.wu.sf[-n:].view(torch.uint8), mlast.wu.sf.view(torch.uint8))
    bias = torch.full((G,), -1e30, device="cuda")
    bias[-8:] = 0
    for T in (1, 9, 20):
        x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").normal_()
        if T <= 16:
            a = block.forward_few(big, x, top_k=2, router_bias=bias, debug=True)
            b = block.forward_few(last, x, top_k=2, debug=True)
            assert torch.equal(a.idx - (G - 8), b.idx) and torch.equal(a.out_f32, b.out_f32)
        a = block.forward_mxfp8(mbig, x, top_k=2, router_bias=bias, debug=True)
        b = block.forward_mxfp8(mlast, x, top_k=2, debug=True)
        ok()
        assert torch.equal(a.idx - (G - 8), b.idx) and torch.equal(a.out_f32, b.out_f32)
        assert torch.isfinite(a.out_f32).all()


def test_more_choices_than_the_few_token_form_holds():
    """top_k 40: one token takes the grouped GEMMs."""
    dims = inputs.Dims(embed_dim=128, num_experts=64, expert_dim=64, hidden_dim=64)
    w, dw = weights(dims), device_weights(dims)
    mw = block.quantize_mxfp8(dw)
    for T in (1, 16, 33):
        xb = inputs.make_x(T, 128, seed=T)
        res = block.forward_mxfp8(mw, block.bf16_tensor(xb), top_k=40, debug=True)
        ok()
        assert B.moe_last_launch_count() > 2
        check_block(w, xb, res, 40)


@pytest.mark.parametrize("D,F,S", [(256, 192, 320), (320, 64, 448), (64, 64, 64), (192, 128, 256)])
@pytest.mark.parametrize("T,k", [(160, 8), (257, 8), (700, 3)])
@pytest.mark.parametrize("fed", [False, True])
def test_block_of_many_rows_per_expert(D, F, S, T, k, fed):
    """Experts with 160 routed rows and more on average, some with few or none."""
    dims = inputs.Dims(D, 8, F, S)
    w, dw = weights(dims), device_weights(dims)
    mw = block.quantize_mxfp8(dw)
    xb = inputs.make_x(T, D, seed=T)
    xq = xs = xv = bias = None
    if fed:
        xq, xs = block.quantize_mxfp8_rows(block.bf16_tensor(inputs.make_x(T, D, seed=T + 1)))
        xv = dequant(xq, xs)
    if k < 8:
        bias = 2 * inputs.zipf_router_bias(8)
    res = block.forward_mxfp8(mw, block.bf16_tensor(xb), xq=xq, xs=xs, top_k=k, debug=True,
                              router_bias=None if bias is None else torch.from_numpy(bias).cuda())
    ok()
    check_block(w, xb, res, k, bias, xv)


@pytest.mark.parametrize("T,D", [(700, 2816), (3000, 256), (300, 4096), (64, 16384)])
def test_add_norm_codes_are_those_of_64_bits(T, D):
    """Codes and scales of y are the float64 oracle's: where an fp32 y lies within a few units of the middle of two codes
    the kernel decides in 64 bits. What is left is the row's sum of squares: fp32 chains of at most 16 fused additions and
    one more, then 64 bits, so at most 17 2^-24 of it and half of that in y. s = residual + x is exact in fp32 here, or
    too small to move a code. (The first run: 2 codes of a million differ, 5e-9 from the middle.)"""
    rng = np.random.default_rng(T)
    xb, rb = inputs.make_x(T, D, seed=T), inputs.make_x(T, D, seed=T + 1)
    gb = inputs.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(D)).astype(np.float32))
    codes, q, j, scale, y = _codes(xb, rb, gb)
    np.testing.assert_array_equal(scale, j)
    other = codes != q
    w = np.abs(y / np.exp2(np.repeat(j, 32, -1).astype(np.float64)))[other]
    assert np.all(np.abs(w - (np.abs(codes) + np.abs(q))[other] / 2) <= 9 * 2.0**-24 * w)


def _codes(xb, rb, gb):
    res = block.add_rms_norm(block.bf16_tensor(xb), block.bf16_tensor(gb), residual=block.bf16_tensor(rb), quantize=True)
    ok()
    s = mo.f64(xb) + mo.f64(rb)
    y = mo.f64(gb) * s / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-6)
    q, j = mx.quantize(y)
    return to_np(res.q.float()).astype(np.float64), q, j, to_np(res.scale.view(torch.uint8)).astype(int) - 127, y


@pytest.mark.parametrize("T,D", [(700, 2816), (3000, 256), (300, 4096), (64, 16384)])
def test_add_norm_codes_of_whole_numbers(T, D):
    """Whole numbers up to 16: their sums of squares are exact in fp32 (at most 2^8 each, 2^14 of them), so every code
    and scale is the oracle's."""
    rng = np.random.default_rng(D)
    xb, rb = (inputs.f32_to_bf16_bits(rng.integers(-8, 9, (T, D)).astype(np.float32)) for _ in range(2))
    gb = inputs.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(D)).astype(np.float32))
    codes, q, j, scale, _ = _codes(xb, rb, gb)
    np.testing.assert_array_equal(scale, j)
    assert np.count_nonzero(codes != q) == 0
