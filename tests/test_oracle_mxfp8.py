"""The MXFP8 oracle pinned on the CPU: codec against torch's float8 types, the
quantiser against brute force, the block against the bf16 oracle; and the host
validation of the MXFP8 and add-norm entry points (no GPU)."""

import ctypes

import numpy as np
import pytest
import torch

from mixture_experts_transformer_b200 import binding as B
from mixture_experts_transformer_b200 import block
from mixture_experts_transformer_b200 import build as mbuild
from mixture_experts_transformer_b200 import inputs
from oracle import moe_oracle as mo
from oracle import mxfp8 as mx

SMALL = inputs.Dims(embed_dim=128, num_experts=8, expert_dim=64, hidden_dim=192)


def test_e4m3_round_matches_torch():
    """Every finite e4m3 value is a fixed point; halfway points and random values round as torch's conversion."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    fin = np.sort(codes[np.isfinite(codes)])
    np.testing.assert_array_equal(mx.e4m3_round(fin), fin)
    mid = (fin[1:] + fin[:-1]) / 2
    rng = np.random.default_rng(0)
    v = np.concatenate([mid, (rng.standard_normal(20000) * np.exp2(rng.uniform(-12, 7, 20000))).clip(-448, 448)])
    v = v.astype(np.float32)  # every value above is exact in fp32 or becomes so here
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(mx.e4m3_round(v), ref.astype(np.float64))


def test_scale_is_the_smallest_power_of_two():
    rng = np.random.default_rng(1)
    amax = np.concatenate([np.exp2(rng.uniform(-140, 126, 5000)), 448 * np.exp2(np.arange(-60.0, 60)),
                           np.nextafter(448 * np.exp2(np.arange(-60.0, 60)), np.inf)])
    j = mx.scale_exponent(amax)
    assert j.min() == -127
    assert np.all(amax <= 448 * np.exp2(j.astype(np.float64)))
    inner = j > -127
    assert np.all(amax[inner] > 448 * np.exp2(j[inner] - 1.0))
    assert mx.scale_exponent(0.0) == -127


def test_quantise_error_and_zero_group():
    rng = np.random.default_rng(2)
    v = rng.standard_normal((4, 96)) * np.exp2(rng.uniform(-20, 20, (4, 1)))
    v[1, 32:64] = 0
    q, j = mx.quantize(v)
    assert np.abs(q).max() <= 448 and j[1, 1] == -127 and np.all(q[1, 32:64] == 0)
    got = mx.values(v)
    step = np.repeat(np.exp2(j.astype(np.float64)), 32, -1)
    # e4m3 rounds by at most 2^-4 of the value, or half the subnormal step 2^-9
    assert np.all(np.abs(got - v) <= np.maximum(np.abs(v) * 2.0**-4, step * 2.0**-10))


def test_scale_tiles_cover_their_storage_once():
    N, K = 200, 320
    off = {mx.scale_tile_offset(n, c, K) for n in range(N) for c in range(K // 32)}
    assert len(off) == N * K // 32 and max(off) < B.moe_mxfp8_weight_bytes(1, K, N - N % 64 + 64)[1]


def test_block_with_exactly_representable_operands():
    """Weights and rows that MXFP8 holds exactly leave only the GeGLU rows' rounding: its bound is checked."""
    rng = np.random.default_rng(3)
    d, e, f, s = 128, 8, 64, 192
    grid = np.array([-1.0, -0.5, 0.0, 0.5, 1.0])

    def w(*shape):
        return inputs.f32_to_bf16_bits(rng.choice(grid, shape).astype(np.float32))

    ws = (w(e, d, f), w(e, d, f), w(e, f, d), w(d, s), w(d, s), w(s, d))
    wr = inputs.f32_to_bf16_bits(rng.standard_normal((d, e)).astype(np.float32))
    x = w(5, d)
    for a in ws[:3]:
        np.testing.assert_array_equal(mx.weight_values(a), mo.f64(a))
    idx, wt, _ = mo.route(x, wr, 2)
    got = mx.block(x, wr, *ws, 2)
    ref = mo.moe_block(x, wr, *ws, top_k=2)["out"]
    slack = 2.0**-4 * (np.abs(mo.geglu_hidden(mo.f64(x), ws[3], ws[4])) @ np.abs(mo.f64(ws[5])))
    for t in range(5):
        for k in range(2):
            g, u, dn = (mo.f64(a[idx[t, k]]) for a in ws[:3])
            h = mo.gelu_tanh(mo.f64(x[t]) @ g) * (mo.f64(x[t]) @ u)
            slack[t] += wt[t, k] * 2.0**-4 * (np.abs(h) @ np.abs(dn))
    # subnormal codes of the GeGLU rows round by half a step of 2^-9 of the group's scale (<= its maximum / 224)
    assert np.all(np.abs(got - ref) <= 1.02 * slack + 1e-3)
    assert np.abs(got - ref).max() > 0


# ------------------------------------------------------------- refusals


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return B.lib()


FAR = 1 << 40


def _norm(T=4, D=256, eps=0.0, x=FAR, residual=2 * FAR, gamma_post=0, gamma=3 * FAR, sum=4 * FAR, y=5 * FAR, q=0,
          scale=0):
    return B.MoeNormParams(T, D, eps, x, residual, gamma_post, gamma, sum, y, q, scale)


def test_add_norm_refusals(lib):
    f = lambda **k: lib.moe_add_rms_norm(ctypes.byref(_norm(**k)), None)  # noqa: E731
    bad, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_ALIGNMENT
    assert lib.moe_add_rms_norm(None, None) == bad
    assert f(T=0) == B.MOE_OK
    assert f(T=-1) == bad and f(D=252) == bad and f(D=16392) == bad and f(D=-8) == bad
    assert f(eps=-1.0) == bad and f(eps=float("nan")) == bad and f(eps=float("inf")) == bad
    assert f(x=0) == bad
    assert f(sum=0, y=0) == bad  # no output
    assert f(q=6 * FAR) == bad and f(scale=6 * FAR) == bad  # one without the other
    assert f(D=40, q=6 * FAR, scale=7 * FAR) == bad  # not whole groups
    for name in ("x", "residual", "gamma_post", "gamma", "sum", "y"):
        assert f(**{name: 8 * FAR + 8}) == mis, name
    assert f(q=8 * FAR + 8, scale=7 * FAR) == mis
    n = 4 * 256 * 2
    assert f(sum=FAR + 16) == bad and f(y=2 * FAR + n - 16) == bad  # shifted overlap with x, residual
    assert f(q=FAR, scale=7 * FAR) == bad  # 8-bit rows over x
    assert f(sum=5 * FAR) == bad  # two outputs in one place
    assert f(y=3 * FAR) == bad  # over gamma
    assert f(q=6 * FAR, scale=6 * FAR + 32) == bad


def _mxp(T=4, k=2, D=128, E=8, F=64, S=64, **kw):
    p = B.MoeMxfp8Params()
    p.T, p.top_k_experts, p.embed_dim, p.num_experts, p.expert_dim, p.hidden_dim = T, k, D, E, F, S
    p.x, p.w_router, p.out = FAR, 2 * FAR, 3 * FAR
    for i, name in enumerate(("wg", "wu", "wd", "sg", "su", "sd")):
        setattr(p, name, B.MoeMxfp8Linear((4 + i) * FAR, (10 + i) * FAR))
    for a, v in kw.items():
        setattr(p, a, v)
    return p


def test_mxfp8_block_refusals(lib):
    f = lambda **k: lib.moe_block_forward_mxfp8(ctypes.byref(_mxp(**k)), None)  # noqa: E731
    bad, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_ALIGNMENT
    assert lib.moe_block_forward_mxfp8(None, None) == bad
    assert f(T=0) == B.MOE_OK
    assert f(T=-1) == bad and f(k=0) == bad and f(k=9) == bad
    assert f(D=96) == bad and f(F=32) == bad and f(S=100) == bad and f(E=12) == bad and f(E=136) == bad
    assert f(T=1 << 30, k=2) == bad
    assert f(x=0) == bad and f(w_router=0) == bad and f(wg=B.MoeMxfp8Linear(0, FAR)) == bad
    assert f(sd=B.MoeMxfp8Linear(FAR, 0)) == bad
    assert f(out=0) == bad
    assert f(xq=20 * FAR) == bad and f(xs=20 * FAR) == bad
    assert f(x=FAR + 8) == mis and f(wd=B.MoeMxfp8Linear(FAR + 4, FAR)) == mis
    assert f(xq=20 * FAR, xs=21 * FAR + 4) == mis and f(out_f32=20 * FAR + 8) == mis and f(idx_out=20 * FAR + 2) == mis
    assert f(out=FAR) == bad  # over x
    assert f(out=20 * FAR, xq=20 * FAR, xs=21 * FAR) == bad
    assert f(out=20 * FAR, xq=22 * FAR, xs=20 * FAR + 512) == bad
    assert f(out_f32=3 * FAR + 16) == bad  # over out


def test_mxfp8_quantiser_refusals_and_sizes(lib):
    bad, mis = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_ALIGNMENT
    assert B.moe_mxfp8_weight_bytes(3, 320, 192) == (3 * 320 * 192, 3 * 2 * 3 * 512)
    for g, K, N in ((0, 64, 64), (1, 32, 64), (1, 64, 96), (1, 0, 64)):
        assert lib.moe_mxfp8_weight_bytes(g, K, N, None, None) == bad
        assert lib.moe_mxfp8_quantize_weight(FAR, g, K, N, 2 * FAR, 3 * FAR, None) == bad
    q = lib.moe_mxfp8_quantize_weight
    assert q(0, 1, 64, 64, 2 * FAR, 3 * FAR, None) == bad
    assert q(FAR + 2, 1, 64, 64, 2 * FAR, 3 * FAR, None) == mis
    assert q(FAR, 1, 64, 64, FAR + 64, 3 * FAR, None) == bad  # codes over the weight
    a = lib.moe_mxfp8_quantize_act
    assert a(FAR, 0, 64, 2 * FAR, 3 * FAR, None) == B.MOE_OK
    assert a(FAR, 2, 40, 2 * FAR, 3 * FAR, None) == bad and a(FAR, -1, 64, 2 * FAR, 3 * FAR, None) == bad
    assert a(FAR, 2, 64, 2 * FAR + 8, 3 * FAR, None) == mis
    assert a(FAR, 2, 64, FAR, 3 * FAR, None) == bad
    assert B.moe_mxfp8_workspace_bytes(_mxp(E=12)) == 0
    assert B.moe_mxfp8_workspace_bytes(_mxp(T=64)) > B.moe_mxfp8_workspace_bytes(_mxp(T=0)) > 0


@pytest.mark.parametrize("dims", [(2816, 128, 704, 2112), (8192, 128, 64, 64), (256, 16, 192, 320), (64, 8, 64, 64)])
@pytest.mark.parametrize("k", [1, 8])
def test_mxfp8_workspace_serves_smaller_batches(dims, k):
    for T in list(range(40)) + list(range(100, 12000, 61)) + [896, 897, 900, 1025, 1153, 9476]:
        p = B.MoeMxfp8Params()
        p.T, p.top_k_experts = T, k
        p.embed_dim, p.num_experts, p.expert_dim, p.hidden_dim = dims
        sizes = [B.moe_mxfp8_workspace_bytes(p)]
        for smaller in (max(0, T - 1), max(0, T - 61), T // 2, min(T, 16), min(T, 17)):
            p.T = smaller
            sizes.append(B.moe_mxfp8_workspace_bytes(p))
        assert sizes[0] == max(sizes)


def test_mxfp8_weights_of_other_sizes_are_refused(lib):
    def linear(G, K, N, cut=0, dtype=torch.uint8):
        qb, sfb = B.moe_mxfp8_weight_bytes(G, K, N)
        return block.Mxfp8Linear(torch.empty(qb - cut, dtype=dtype), torch.empty(sfb, dtype=torch.uint8), G, K, N)

    d = SMALL
    gu, dn = (d.num_experts, d.embed_dim, d.expert_dim), (d.num_experts, d.expert_dim, d.embed_dim)
    sgu, sdn = (1, d.embed_dim, d.hidden_dim), (1, d.hidden_dim, d.embed_dim)
    router = torch.empty((d.embed_dim, d.num_experts), dtype=torch.bfloat16)
    block.Mxfp8Weights(d, router, linear(*gu), linear(*gu), linear(*dn), linear(*sgu), linear(*sgu), linear(*sdn))
    with pytest.raises(ValueError, match="contiguous bytes"):
        linear(*gu, cut=1)
    with pytest.raises(ValueError, match="contiguous bytes"):
        linear(*gu, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="wd: 8 Linears"):
        block.Mxfp8Weights(d, router, linear(*gu), linear(*gu), linear(*gu), linear(*sgu), linear(*sgu), linear(*sdn))
    with pytest.raises(ValueError, match="wu: 8 Linears"):
        block.Mxfp8Weights(d, router, linear(*gu), linear(7, *gu[1:]), linear(*dn), linear(*sgu), linear(*sgu), linear(*sdn))
