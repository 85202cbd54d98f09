"""Edges of the few-token layer and the MXFP8 block on a B200: selection, alignment, streams, limits."""

import dataclasses

import numpy as np
import pytest
import torch

from gpu_common import SMALL, device_weights, require_gpu, to_np, weights
from mixture_experts_transformer_b200 import binding as B
from mixture_experts_transformer_b200 import block, inputs
from test_gpu_few import check
from test_gpu_mxfp8 import check_block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def ok():
    st = B.moe_get_device_status()
    assert st == B.MOE_OK, B.moe_status_string(st)


# ------------------------------------------------------------- selection


@pytest.mark.parametrize("T", [1, 8, 16])
@pytest.mark.parametrize("k", [1, 4, 15, 16])
@pytest.mark.parametrize("where", ["router", "bias", "-bias"])
def test_a_nan_logit_never_wins(T, k, where):
    """Logits that are NaN: every entry counts them as minus infinity, as the whole block does (experts 3 and 11 are
    chosen only when all 16 are, last and in order)."""
    w, dw = weights(SMALL), device_weights(SMALL)
    x = block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=T))
    bias = None
    if where == "router":
        router = w.w_router.copy()
        router[5, 3], router[200, 11] = 0x7FC0, 0xFFC0
        dw = dataclasses.replace(dw, w_router=block.bf16_tensor(router))
    else:
        bias = torch.zeros(SMALL.num_experts, device="cuda")
        bias[[3, 11]] = float("nan")
        if where == "-bias":
            bias.view(torch.int32)[[3, 11]] = -4194304  # 0xFFC00000
    ref = block.forward(dw, x, top_k=k, router_bias=bias, debug=True)
    got = block.forward_few(dw, x, top_k=k, router_bias=bias, debug=True)
    mx = block.forward_mxfp8(block.quantize_mxfp8(dw), x, top_k=k, router_bias=bias, debug=True)
    ok()
    for res in (got, mx):
        assert torch.equal(res.idx, ref.idx)
        np.testing.assert_allclose(to_np(res.w), to_np(ref.w), rtol=2e-5, atol=1e-9)
        assert torch.isfinite(res.out_f32).all()
        assert torch.equal(res.cnt, ref.cnt)
    assert torch.equal(torch.isnan(got.logits), torch.isnan(ref.logits))
    hit = torch.isin(ref.idx, torch.tensor([3, 11], device="cuda"))
    assert bool(hit.any()) == (k > 14) and torch.all(ref.w[hit] == 0)


@pytest.mark.parametrize("T", [1, 16])
def test_infinite_logits_choose_as_the_whole_block(T):
    """+infinity first, -infinity and NaN last and in order; only NaN logits: the first k experts, weights NaN."""
    dw = device_weights(SMALL)
    x = block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=T))
    mw = block.quantize_mxfp8(dw)
    inf, nan = float("inf"), float("nan")
    for values in ({2: -inf, 5: nan, 9: -inf}, {7: inf}, {4: inf, 9: inf, 1: nan}, {e: nan for e in range(16)}):
        bias = torch.zeros(SMALL.num_experts, device="cuda")
        for e, v in values.items():
            bias[e] = v
        for k in (2, 16):
            ref = block.forward(dw, x, top_k=k, router_bias=bias, debug=True)
            got = block.forward_few(dw, x, top_k=k, router_bias=bias, debug=True)
            mx = block.forward_mxfp8(mw, x, top_k=k, router_bias=bias, debug=True)
            ok()
            for res in (got, mx):
                assert torch.equal(res.idx, ref.idx)
                np.testing.assert_allclose(to_np(res.w), to_np(ref.w), rtol=2e-5, atol=1e-9)


# ------------------------------------------------------- where tensors are


def test_weights_elsewhere_are_refused():
    """Weights in host memory: refused before anything is launched."""
    x = block.bf16_tensor(inputs.make_x(4, SMALL.embed_dim, seed=1))
    dw = block.upload(weights(SMALL), device="cpu")
    with pytest.raises(ValueError, match="w_router is on cpu"):
        block.forward_few(dw, x, top_k=4)
    for name in ("wg", "sd"):
        mixed = dataclasses.replace(device_weights(SMALL), **{name: getattr(dw, name)})
        with pytest.raises(ValueError, match=f"{name} is on cpu"):
            block.forward_few(mixed, x, top_k=4)
    mw = block.quantize_mxfp8(device_weights(SMALL))
    host = [block.Mxfp8Linear(lin.q.cpu(), lin.sf.cpu(), lin.groups, lin.K, lin.N)
            for lin in (mw.wg, mw.wu, mw.wd, mw.sg, mw.su, mw.sd)]
    with pytest.raises(ValueError, match="w_router is on cpu"):
        block.forward_mxfp8(block.Mxfp8Weights(mw.dims, mw.w_router.cpu(), *host), x, top_k=4)
    with pytest.raises(ValueError, match="wg: on cpu"):
        block.Mxfp8Weights(mw.dims, mw.w_router, *host)
    ok()


def _calls(T):
    """name -> (call(stream) -> result tensors): everything that makes its own outputs."""
    dw = device_weights(SMALL)
    mw = block.quantize_mxfp8(dw)
    x = block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=T))
    wf, wm = block.few_workspace(dw, min(T, 16), 4), block.mxfp8_workspace(mw, T, 4)

    def norm(st):
        r = block.add_rms_norm(x, residual=x, quantize=True, stream=st)
        return r.y, r.sum, r.q, r.scale

    def linear(st):
        lin = block.quantize_mxfp8_linear(dw.sg, stream=st)
        return lin.q, lin.sf

    def layer(r):
        return r.out, r.out_f32, r.idx, r.w, r.cnt

    calls = {
        "norm": norm,
        "rows": lambda st: block.quantize_mxfp8_rows(x, stream=st),
        "linear": linear,
        "mxfp8": lambda st: layer(block.forward_mxfp8(mw, x, top_k=4, workspace=wm, stream=st, debug=True)),
    }
    if T <= 16:
        calls["few"] = lambda st: layer(block.forward_few(dw, x, top_k=4, workspace=wf, stream=st, debug=True))
    return calls


@pytest.mark.parametrize("T", [7, 40])
def test_outputs_of_a_call_on_another_stream(T):
    """A call given a stream makes its outputs from memory that the current stream no longer writes, and a later call's
    outputs do not take memory that the current stream still reads."""
    calls = _calls(T)
    side = torch.cuda.Stream()
    for name, call in calls.items():
        ref = [t.clone() for t in call(None)]
        ok()
        torch.cuda.synchronize()
        # freed here, but to be written by this stream some 10 ms from now
        old = [torch.empty_like(t) for t in ref]
        torch.cuda._sleep(20_000_000)
        for t in old:
            t.view(torch.uint8).fill_(7)
        del old, t
        got = call(side)
        torch.cuda.synchronize()
        ok()
        for a, b in zip(got, ref):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
        # read by this stream some 10 ms from now, but freed at once
        torch.cuda._sleep(20_000_000)
        kept = [t.clone() for t in got]
        del got, a
        again = call(side)
        with torch.cuda.stream(side):
            for t in again:
                t.view(torch.uint8).fill_(9)
        torch.cuda.synchronize()
        for a, b in zip(kept, ref):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
        del again, t, a, b


@pytest.mark.parametrize("T", [3, 40])
def test_scales_of_a_slice_of_rows(T):
    """Rows of one batch whose scales start off a 16-byte boundary (embed 320: 10 bytes a row), on the current and on
    another stream, and in a captured graph."""
    dims = inputs.Dims(embed_dim=320, num_experts=24, expert_dim=64, hidden_dim=448)
    mw = block.quantize_mxfp8(device_weights(dims))
    x = block.bf16_tensor(inputs.make_x(T + 5, 320, seed=T))
    xq, xs = block.quantize_mxfp8_rows(x)
    ws = block.mxfp8_workspace(mw, T, 4)
    side = torch.cuda.Stream()
    for first in (1, 3, 5):
        rows = slice(first, first + T)
        assert xs[rows].data_ptr() % 16
        ref = block.forward_mxfp8(mw, x[rows], xq=xq[rows], xs=xs[rows].clone(), top_k=4).out
        got = block.forward_mxfp8(mw, x[rows], xq=xq[rows], xs=xs[rows], top_k=4).out
        ok()
        assert torch.equal(got, ref)
        torch.cuda.synchronize()
        got = block.forward_mxfp8(mw, x[rows], xq=xq[rows], xs=xs[rows], top_k=4, workspace=ws, stream=side).out
        torch.cuda.synchronize()
        assert torch.equal(got, ref)
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        block.forward_mxfp8(mw, x[rows], xq=xq[rows], xs=xs[rows], top_k=4, workspace=ws, out=out)
    new = block.bf16_tensor(inputs.make_x(T + 5, 320, seed=T + 1))
    x.copy_(new)
    for a, b in zip((xq, xs), block.quantize_mxfp8_rows(new)):
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    ref = block.forward_mxfp8(mw, x[rows], xq=xq[rows], xs=xs[rows].clone(), top_k=4).out
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    ok()
    assert torch.equal(out, ref)
    del g


# ------------------------------------------------------------------ limits


@pytest.mark.parametrize("S", [16320, 16384])
@pytest.mark.parametrize("T", [1, 16])
def test_few_with_the_widest_shared_mlp(S, T):
    """16384 hidden units of the shared MLP: 128 units of work, a CTA has parts of two at most."""
    dims = inputs.Dims(embed_dim=128, num_experts=8, expert_dim=64, hidden_dim=S)
    w, dw = weights(dims), device_weights(dims)
    xb = inputs.make_x(T, 128, seed=T)
    res = block.forward_few(dw, block.bf16_tensor(xb), top_k=2, debug=True)
    ok()
    assert B.moe_last_launch_count() == 2
    check(w, xb, res, 2)
    res = block.forward_mxfp8(block.quantize_mxfp8(dw), block.bf16_tensor(xb), top_k=2, debug=True)
    ok()
    assert B.moe_last_launch_count() == 2
    check_block(w, xb, res, 2)


@pytest.mark.parametrize("E,T", [(32, 1), (32, 16), (40, 1), (128, 16)])
def test_few_with_the_most_choices(E, T):
    """top_k 32, a warp's worth of slots: of 32 experts (all), 40 and 128."""
    dims = inputs.Dims(embed_dim=192, num_experts=E, expert_dim=64, hidden_dim=64)
    w, dw = weights(dims), device_weights(dims)
    xb = inputs.make_x(T, 192, seed=E + T)
    res = block.forward_few(dw, block.bf16_tensor(xb), top_k=32, debug=True)
    ok()
    check(w, xb, res, 32)
    res = block.forward_mxfp8(block.quantize_mxfp8(dw), block.bf16_tensor(xb), top_k=32, debug=True)
    ok()
    assert B.moe_last_launch_count() == 2
    check_block(w, xb, res, 32)


@pytest.mark.parametrize("T", [1, 16])
def test_few_with_the_widest_experts(T):
    dims = inputs.Dims(embed_dim=64, num_experts=8, expert_dim=16384, hidden_dim=64)
    w, dw = weights(dims), device_weights(dims)
    xb = inputs.make_x(T, 64, seed=T)
    res = block.forward_few(dw, block.bf16_tensor(xb), top_k=3, debug=True)
    ok()
    check(w, xb, res, 3)
    res = block.forward_mxfp8(block.quantize_mxfp8(dw), block.bf16_tensor(xb), top_k=3, debug=True)
    ok()
    assert B.moe_last_launch_count() == 2
    check_block(w, xb, res, 3)


@pytest.mark.parametrize("T", [1, 16, 17])
@pytest.mark.parametrize("D,F,S", [(4160, 64, 64), (128, 64, 16448), (64, 16448, 64)])
def test_past_the_few_token_forms_limits(T, D, F, S):
    """Wider than the few-token form holds: MXFP8 calls take the grouped GEMMs at any size, bf16 calls are refused."""
    dims = inputs.Dims(embed_dim=D, num_experts=8, expert_dim=F, hidden_dim=S)
    w, dw = weights(dims), device_weights(dims)
    xb = inputs.make_x(T, D, seed=T)
    x = block.bf16_tensor(xb)
    mw = block.quantize_mxfp8(dw)
    res = block.forward_mxfp8(mw, x, top_k=2, debug=True, workspace=block.mxfp8_workspace(mw, 40, 2))
    ok()
    assert B.moe_last_launch_count() > 2
    check_block(w, xb, res, 2)
    with pytest.raises(B.MoeError) as err:
        block.forward_few(dw, x, top_k=2)
    assert err.value.status == B.MOE_ERR_INVALID_ARG
    p = B.make_params(T, top_k=2, dims=dims)
    assert B.moe_few_workspace_bytes(p) == 0


# ------------------------------------------- the grouped form, in earnest


@pytest.mark.parametrize("T", [17, 40, 300])
def test_grouped_special_values_stay_with_their_tokens(T):
    """More than 16 tokens: a NaN and an infinite row touch their own output alone, bad weights of an expert the tokens
    routed to it alone."""
    w, dw = weights(SMALL), device_weights(SMALL)
    mw = block.quantize_mxfp8(dw)
    x = block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=T))
    ref = block.forward_mxfp8(mw, x, top_k=2, debug=True)
    x2 = x.clone()
    x2[4, 7], x2[T - 1, 255], x2[9] = float("nan"), float("inf"), float("-inf")
    got = block.forward_mxfp8(mw, x2, top_k=2, debug=True)
    ok()
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[4, 9, T - 1]] = True
    assert torch.isnan(got.out_f32[bad]).all() and torch.equal(got.out_f32[~bad], ref.out_f32[~bad])
    assert all(len(set(r)) == 2 for r in to_np(got.idx))
    e = int(ref.idx[0, 0])
    arrays = [a.copy() for a in (w.wg, w.wu, w.wd)]
    arrays[0][e, 3, 5] = 0x7F80
    arrays[1][e, 100, 6] = 0xFFC0
    arrays[2][e, 2, 1] = 0x7FC0
    mwb = block.quantize_mxfp8(block.upload(dataclasses.replace(w, wg=arrays[0], wu=arrays[1], wd=arrays[2])))
    got = block.forward_mxfp8(mwb, x, top_k=2, debug=True)
    ok()
    hit = (ref.idx == e).any(1)
    assert hit.any() and not hit.all()
    assert not torch.isfinite(got.out_f32[hit]).all(1).any() and torch.equal(got.out_f32[~hit], ref.out_f32[~hit])


def test_grouped_graphs_and_streams_at_once():
    """Two captured graphs of different batches on workspaces of their own, replayed on two streams at once, with new
    inputs each time."""
    mw = block.quantize_mxfp8(device_weights(SMALL))
    sizes = (40, 700)
    xs = [block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=T)) for T in sizes]
    outs = [torch.empty_like(x) for x in xs]
    wss = [block.mxfp8_workspace(mw, T, 4) for T in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    graphs = []
    for x, o, ws, st in zip(xs, outs, wss, streams):
        block.forward_mxfp8(mw, x, top_k=4, out=o, workspace=ws, stream=st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                block.forward_mxfp8(mw, x, top_k=4, out=o, workspace=ws)
        graphs.append(g)
    for rnd in range(3):
        new = [block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=50 * rnd + T)) for T in sizes]
        refs = [block.forward_mxfp8(mw, n, top_k=4).out.clone() for n in new]
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
    del graphs, g


def test_grouped_rows_behind_the_batch_and_what_the_workspace_held():
    """Ragged batches write their own rows, whatever the workspace held before."""
    mw = block.quantize_mxfp8(device_weights(SMALL))
    for T in (17, 129, 500):
        x = block.bf16_tensor(inputs.make_x(T, SMALL.embed_dim, seed=T))
        same = []
        for fill in (0.0, float("nan")):
            buf = torch.full((T + 2, SMALL.embed_dim), 7.0, dtype=torch.bfloat16, device="cuda")
            ws = torch.full((block.mxfp8_workspace(mw, T, 3).numel() // 4,), fill, device="cuda").view(torch.uint8)
            block.forward_mxfp8(mw, x, top_k=3, out=buf[:T], workspace=ws)
            ok()
            assert torch.all(buf[T:] == 7.0)
            same.append(buf[:T].clone())
        assert torch.equal(same[0], same[1]) and torch.isfinite(same[0]).all()
