"""The few-token layer (bf16 and MXFP8, two kernels) on a B200 against the float64 oracle."""

import dataclasses

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


# ------------------------------------------------------- norms and shards


@pytest.mark.parametrize("T", [1, 7, 16])
@pytest.mark.parametrize("pre,post,res", [(True, True, True), (True, False, False), (False, True, False),
                                          (False, False, True)])
def test_few_sandwich(T, pre, post, res):
    w, dw = weights(SMALL), device_weights(SMALL)
    D = SMALL.embed_dim
    xb = inputs.make_x(T, D, seed=T)
    rng = np.random.default_rng(T)
    gp, go = (inputs.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
    res_ = block.forward_few(dw, block.bf16_tensor(xb), top_k=4, debug=True, residual=res,
                             norm_pre=block.bf16_tensor(gp) if pre else None,
                             norm_post=block.bf16_tensor(go) if post else None)
    ok()
    xin = xb
    if pre:  # the layer's input is the normalised row in bf16; the GPU's fp32 norm may round an element the other way
        exact = sw.rms_norm(mo.f64(xb), mo.f64(gp))
        xin = sw.bf16_bits(sw.bf16_rne(exact))
    idx, wts = to_np(res_.idx), to_np(res_.w)
    f, tol = layer_bound(w, xin, idx, wts)
    if pre:
        # an element within 2^-18 of a rounding border may be the neighbouring bf16 value: one step of 2^-7
        step = np.exp2(np.floor(np.log2(np.abs(exact) + 1e-30))) * 2.0**-7
        border = np.abs(np.abs(exact / step - np.floor(exact / step)) - 0.5) < 2.0**-18 * np.abs(exact / step)
        for t in np.flatnonzero(border.any(-1)):
            up, dn = (layer_bound(w, sw.bf16_bits(sw.bf16_rne(exact[t : t + 1] * (1 + sgn * 2.0**-17))),
                                  idx[t : t + 1], wts[t : t + 1])[0][0] for sgn in (1, -1))
            tol[t] += np.abs(up - dn)
    out = f
    if post:
        rms = np.sqrt((f * f).mean(-1, keepdims=True) + 1e-6)
        out = mo.f64(go) * f / rms
        tol = np.abs(mo.f64(go)) * tol / rms + np.abs(out) * (2.0**-18 + np.sqrt((tol * tol).mean(-1, keepdims=True)) / rms)
    if res:
        out = out + mo.f64(xb)
        tol = tol + 2.0**-23 * np.abs(out)
    got = to_np(res_.out_f32).astype(np.float64)
    assert np.all(np.abs(got - out) <= 1.01 * tol), np.max(np.abs(got - out) / tol)
    np.testing.assert_array_equal(to_np(res_.out.float()), to_np(res_.out_f32.bfloat16().float()))


def _params(dw, x, out, ws=None, **kw):
    return B.make_params(x.shape[0], x, *dw.args(), out, dims=dw.dims, workspace=ws, **kw)


def test_few_expert_shards_add_up():
    """Four expert shards (a quarter of the experts and of the shared hidden units each), one of them untouched by
    a one-token batch's top 2, sum to the whole layer; bf16 output absent."""
    w = weights(SMALL)
    E, S, D = SMALL.num_experts, SMALL.hidden_dim, SMALL.embed_dim
    for T, k in ((1, 2), (11, 4)):
        xb = inputs.make_x(T, D, seed=20 + T)
        x = block.bf16_tensor(xb)
        whole = block.forward_few(device_weights(SMALL), x, top_k=k, debug=True)
        total = torch.zeros((T, D), dtype=torch.float64, device="cuda")
        tolerance = np.zeros((T, D))
        untouched = 0
        for g in range(5):  # S = 320 = 5 slices of 64
            e0, ec = (g * 4, 4) if g < 4 else (0, 4)
            h0, h1 = g * 64, (g + 1) * 64
            if g == 4:  # the fifth shard: the last hidden slice with experts nobody chooses (weights 0)
                zero = np.zeros_like(w.wg[:4])
                part = dataclasses.replace(w, wg=zero, wu=zero, wd=np.zeros_like(w.wd[:4]), sg=w.sg[:, h0:h1].copy(),
                                           su=w.su[:, h0:h1].copy(), sd=w.sd[h0:h1].copy())
            else:
                part = dataclasses.replace(w, wg=w.wg[e0 : e0 + 4], wu=w.wu[e0 : e0 + 4], wd=w.wd[e0 : e0 + 4],
                                           sg=w.sg[:, h0:h1].copy(), su=w.su[:, h0:h1].copy(), sd=w.sd[h0:h1].copy())
            dev = [block.bf16_tensor(a) for a in (part.w_router, part.wg, part.wu, part.wd, part.sg, part.su, part.sd)]
            dims = inputs.Dims(D, E, SMALL.expert_dim, 64)
            f32 = torch.full((T, D), float("nan"), device="cuda")
            cnt = torch.full((E,), -1, dtype=torch.int32, device="cuda")
            p = B.make_params(T, x, *dev, None, dims=dims, top_k=k, out_f32=f32, cnt_out=cnt, expert_begin=e0,
                              expert_count=ec)
            B.check(B.moe_block_forward_few(p), "shard")
            ok()
            total += f32.double()
            if g < 4:
                untouched += int(cnt.sum()) == 0
                assert int(cnt[:e0].sum()) == 0 and int(cnt[e0 + 4 :].sum()) == 0
        tolerance = layer_bound(w, xb, to_np(whole.idx), to_np(whole.w))[1]
        err = np.abs(to_np(total) - to_np(whole.out_f32))
        assert np.all(err <= 3 * tolerance), np.max(err / tolerance)
        if T == 1:
            assert untouched >= 2


# ------------------------------------------------- selection, special values


def test_few_ties_take_the_lower_expert():
    w = weights(SMALL)
    router = w.w_router.copy()
    router[:, 9] = router[:, 3]  # equal columns: equal logits, whatever the order of the sums
    router[:, 5] = 0x8000        # -0 weights: logits of either zero's sign
    router[:, 6] = 0
    router[:, 12:] = 0
    dw = dataclasses.replace(device_weights(SMALL), w_router=block.bf16_tensor(router))
    xb = inputs.make_x(16, SMALL.embed_dim, seed=4)
    for k in (3, 16):
        res = block.forward_few(dw, block.bf16_tensor(xb), top_k=k, debug=True)
        ok()
        ref = mo.route(xb, router, k)[0]
        idx = to_np(res.idx)
        for t in range(16):
            pos = {e: j for j, e in enumerate(idx[t])}
            if 9 in pos:
                assert 3 in pos and pos[3] < pos[9]
            zeros = [e for e in idx[t] if e in (5, 6) or e >= 12]
            assert zeros == sorted(zeros)
            assert sorted(idx[t]) == sorted(ref[t])


def test_few_special_values_stay_with_their_tokens():
    w = weights(SMALL)
    T, k = 12, 2
    xb = inputs.make_x(T, SMALL.embed_dim, seed=9)
    clean = block.forward_few(device_weights(SMALL), block.bf16_tensor(xb), top_k=k, debug=True)
    for mx in (False, True):
        # a NaN row: only its own output
        x2 = block.bf16_tensor(xb)
        x2[4, 7] = float("nan")
        dw = device_weights(SMALL)
        mw = block.quantize_mxfp8(dw)
        run = (lambda x, m=mw: block.forward_mxfp8(m, x, top_k=k, debug=True)) if mx else (
            lambda x, d=dw: block.forward_few(d, x, top_k=k, debug=True))
        ref, got = run(block.bf16_tensor(xb)), run(x2)
        ok()
        keep = [t for t in range(T) if t != 4]
        assert torch.isnan(got.out_f32[4]).all() and torch.equal(got.out_f32[keep], ref.out_f32[keep])
        assert sorted(set(to_np(got.idx)[4])) == sorted(to_np(got.idx)[4])
        # infinite and NaN weights of one expert: only the tokens routed to it
        e = int(clean.idx[0, 0])
        bad = [a.copy() for a in (w.wg, w.wu, w.wd)]
        bad[0][e, 3, 5] = 0x7F80
        bad[2][e, 2, 1] = 0x7FC0
        dwb = block.upload(dataclasses.replace(w, wg=bad[0], wu=bad[1], wd=bad[2]))
        run2 = (lambda x: block.forward_mxfp8(block.quantize_mxfp8(dwb), x, top_k=k, debug=True)) if mx else (
            lambda x: block.forward_few(dwb, x, top_k=k, debug=True))
        got = run2(block.bf16_tensor(xb))
        ok()
        hit = (to_np(got.idx) == e).any(1)
        assert hit.any() and not hit.all()
        assert not torch.isfinite(got.out_f32[torch.from_numpy(hit)]).all(1).any()
        keep = torch.from_numpy(~hit)
        # fewer or more experts in the list move the CTAs' shares, not which terms are added: nothing here changes them
        assert torch.equal(got.out_f32[keep], ref.out_f32[keep])


# --------------------------------------------- calls as a program makes them


def test_few_writes_its_rows_only_and_is_deterministic():
    dw = device_weights(ODD)
    mw = block.quantize_mxfp8(dw)
    for T in (1, 5, 16):
        x = block.bf16_tensor(inputs.make_x(T, ODD.embed_dim, seed=T))
        outs = []
        for call in (lambda o, w_: block.forward_few(dw, x, top_k=3, out=o, workspace=w_),
                     lambda o, w_: block.forward_mxfp8(mw, x, top_k=3, out=o, workspace=w_)):
            same = []
            for fill in (0.0, float("nan")):  # and whatever the workspace held before
                buf = torch.full((T + 2, ODD.embed_dim), 7.0, dtype=torch.bfloat16, device="cuda")
                ws = torch.full((max(block.few_workspace(dw, T, 3).numel(), block.mxfp8_workspace(mw, T, 3).numel()) // 4,),
                                fill, device="cuda").view(torch.uint8)
                call(buf[:T], ws)
                ok()
                assert torch.all(buf[T:] == 7.0)
                same.append(buf[:T].clone())
            assert torch.equal(same[0], same[1]) and torch.isfinite(same[0]).all()
            outs.append(same[0])


@pytest.mark.parametrize("mx", [False, True])
def test_few_graphs_streams_and_workspaces(mx):
    """Two captured graphs on workspaces of their own, replayed on two streams at once and with new inputs; a capture
    without a workspace is refused."""
    dw = device_weights(SMALL)
    mw = block.quantize_mxfp8(dw)

    def call(x, out, ws, stream=None):
        if mx:
            return block.forward_mxfp8(mw, x, top_k=4, out=out, workspace=ws, stream=stream)
        return block.forward_few(dw, x, top_k=4, out=out, workspace=ws, stream=stream)

    sizes = (3, 14)
    xs = [block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=T)) for T in sizes]
    outs = [torch.empty_like(x) for x in xs]
    wss = [block.mxfp8_workspace(mw, T, 4) if mx else block.few_workspace(dw, T, 4) for T in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    graphs = []
    for x, o, ws, st in zip(xs, outs, wss, streams):
        with torch.cuda.stream(st):
            call(x, o, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call(x, o, ws)
        graphs.append(g)
    for rnd in range(3):
        new = [block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=50 * rnd + T)) for T in sizes]
        refs = [call(n, torch.empty_like(n), None).out.clone() for n in new]
        for x, n in zip(xs, new):
            x.copy_(n)
        torch.cuda.synchronize()
        for _ in range(4):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        ok()
        for o, r in zip(outs, refs):
            assert torch.equal(o, r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        with pytest.raises(B.MoeError) as err:
            call(xs[0], outs[0], None)
        outs[0].zero_()  # (a graph needs a node)
    assert err.value.status == B.MOE_ERR_WORKSPACE
    del g, graphs


def test_few_guards_and_refusals():
    dw = device_weights(SMALL)
    x = block.bf16_tensor(inputs.make_x(16, SMALL.embed_dim, seed=1))
    out = torch.empty_like(x)
    ws = block.few_workspace(dw, 16, 4)
    B.check(B.moe_block_forward_few(_params(dw, x, out, ws, top_k=4, check_guards=True)), "guarded")
    ok()
    assert B.moe_last_launch_count() == 4
    f = B.moe_block_forward_few
    assert f(_params(dw, x, out, ws[:-256], top_k=4)) == B.MOE_ERR_WORKSPACE
    assert f(_params(dw, x, out, ws[16:], top_k=4)) == B.MOE_ERR_ALIGNMENT
    x17 = block.bf16_tensor(inputs.make_x(17, SMALL.embed_dim, seed=1))
    assert f(_params(dw, x17, torch.empty_like(x17), None, top_k=4)) == B.MOE_ERR_INVALID_ARG
    assert f(_params(dw, x, x, ws, top_k=4)) == B.MOE_ERR_INVALID_ARG
    f32 = torch.empty((16, SMALL.embed_dim), device="cuda")
    assert f(_params(dw, x, f32.view(torch.bfloat16)[:16], ws, top_k=4, out_f32=f32)) == B.MOE_ERR_INVALID_ARG
    assert block.forward_few(dw, x[:0]).out.shape == (0, SMALL.embed_dim)
    mw = block.quantize_mxfp8(dw)
    assert block.forward_mxfp8(mw, x[:0]).out.shape == (0, SMALL.embed_dim)
    for bad in (x.t(), x[:, ::2], x.float(), x[:, :-64]):
        with pytest.raises(ValueError):
            block.forward_few(dw, bad)
        with pytest.raises(ValueError):
            block.forward_mxfp8(mw, bad)
    with pytest.raises(ValueError):
        block.forward_few(dw, x.cpu())
    ok()


def test_mxfp8_forms_agree_where_they_meet():
    """16 tokens (two kernels) and 17 (grouped GEMMs): the shared rows differ by the second form's bf16 storage only."""
    w, dw = weights(), device_weights()
    mw = block.quantize_mxfp8(dw)
    xb = inputs.make_x(17, seed=77)
    a = block.forward_mxfp8(mw, block.bf16_tensor(xb[:16]), debug=True)
    b = block.forward_mxfp8(mw, block.bf16_tensor(xb), debug=True)
    ok()
    assert torch.equal(a.idx, b.idx[:16])
    rms = float(a.out_f32.square().mean().sqrt())
    # y is rounded to bf16 in the second (2^-9 rms each, eight of weight ~ 1/8 beside the shared branch): under 2^-8 rms
    assert float((a.out_f32 - b.out_f32[:16]).square().mean().sqrt()) <= 2.0**-8 * rms
    # a workspace for the larger batch serves the smaller
    ws = block.mxfp8_workspace(mw, 17)
    c = block.forward_mxfp8(mw, block.bf16_tensor(xb[:16]), workspace=ws)
    ok()
    assert torch.equal(c.out, a.out)


# ------------------------------------------------------------- together


@pytest.mark.parametrize("T", [1, 6, 40])
def test_a_decode_step_in_8_bits(T):
    """Norm, MXFP8 layer, norm, as a layer's second half runs: residual stream and next input against float64."""
    w, dw = weights(SMALL), device_weights(SMALL)
    mw = block.quantize_mxfp8(dw)
    D = SMALL.embed_dim
    rng = np.random.default_rng(T)
    attn, stream = inputs.make_x(T, D, seed=1), inputs.make_x(T, D, seed=2)
    gs = [inputs.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)) for _ in range(4)]
    g = [block.bf16_tensor(b) for b in gs]
    first = block.add_rms_norm(block.bf16_tensor(attn), g[1], residual=block.bf16_tensor(stream), gamma_post=g[0],
                               quantize=True)
    layer = block.forward_mxfp8(mw, first.y, xq=first.q, xs=first.scale, top_k=4, debug=True)
    last = block.add_rms_norm(layer.out, g[3], residual=first.sum, gamma_post=g[2], quantize=True, sum_out=first.sum)
    ok()
    # each stage from the previous one's values as the GPU holds them
    yb = to_np(first.y.view(torch.int16)).view(np.uint16)
    check_block(w, yb, layer, 4, None, dequant(first.q, first.scale))
    s0 = mo.f64(stream) + sw.rms_norm(mo.f64(attn), mo.f64(gs[0]))
    s0b = sw.bf16_rne(s0)
    f = to_np(layer.out.double())
    s1 = s0b + sw.rms_norm(f, mo.f64(gs[2]))
    # the stream was rounded once (its bf16 value may differ by a step at a border), then again
    assert np.all(np.abs(to_np(last.sum.double()) - s1) <= 2.0**-8 * np.abs(s1) + 2.0**-7 * np.abs(s0) * (
        np.abs(to_np(last.sum.double()) - s1) > 2.0**-8 * np.abs(s1)) + 2.0**-16)
    y1 = sw.rms_norm(to_np(last.sum.double()), mo.f64(gs[3]))
    assert np.sqrt(np.mean((to_np(last.y.double()) - y1) ** 2)) <= 2.0**-8 * np.sqrt(np.mean(y1**2))
    got = dequant(last.q, last.scale)
    assert np.sqrt(np.mean((got - y1) ** 2)) <= 2.0**-4 * np.sqrt(np.mean(y1**2))
