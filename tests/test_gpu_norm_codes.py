"""MXFP8 codes of the residual-add norm next to their borders, on a B200 against 64 bits."""

import numpy as np
import pytest
import torch

from gpu_common import require_gpu, to_np
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


def bits(a):
    return inputs.f32_to_bf16_bits(np.asarray(a, np.float32))


def run(xb, rb=None, gb=None, pb=None, **kw):
    dev = [None if b is None else block.bf16_tensor(b) for b in (xb, rb, gb, pb)]
    res = block.add_rms_norm(dev[0], dev[2], residual=dev[1], gamma_post=dev[3], quantize=True, **kw)
    ok()
    return res


def oracle(xb, rb=None, gb=None, pb=None):
    s = mo.f64(xb) if pb is None else sw.rms_norm(mo.f64(xb), mo.f64(pb))
    s = s if rb is None else mo.f64(rb) + s
    y = s / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-6)
    return y if gb is None else mo.f64(gb) * y


@pytest.mark.parametrize("T,D", [(700, 2816), (3000, 256), (300, 4096), (64, 16384)])
@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC0, 0xFFC0])
def test_a_gamma_that_is_not_finite_takes_its_group_alone(T, D, bad):
    """One infinite or NaN gamma in every eighth group: that group is NaN in every row, whatever values its neighbours
    hold; the other groups' codes are those of a finite gamma."""
    rng = np.random.default_rng(T)
    xb, rb = inputs.make_x(T, D, seed=T), inputs.make_x(T, D, seed=T + 1)
    gb = bits(1 + 0.1 * rng.standard_normal(D))
    ref = run(xb, rb, gb)
    gx = gb.copy()
    gx[37::256] = bad
    got = run(xb, rb, gx)
    hit = np.zeros(D // 32, bool)
    hit[1::8] = True
    codes, scale = to_np(got.q.view(torch.uint8)), to_np(got.scale.view(torch.uint8))
    assert np.all(scale[:, hit] == 0xFF)
    assert np.all(codes.reshape(T, -1, 32)[:, hit] == 0x7F)
    np.testing.assert_array_equal(scale[:, ~hit], to_np(ref.scale.view(torch.uint8))[:, ~hit])
    np.testing.assert_array_equal(codes.reshape(T, -1, 32)[:, ~hit],
                                  to_np(ref.q.view(torch.uint8)).reshape(T, -1, 32)[:, ~hit])


# Codes are decided in 64 bits but for the row's sum of squares: of each eight squares at most 5 fp32 roundings, and what
# s's own (one; after a post-norm two) bring in, twice each: 9 2^-24 of the sum and half of that of y, relatively.
OPEN = 4.5 * 2.0**-24


def check_codes(res, y, open=OPEN):
    """Codes and scales of res are the 64-bit oracle's of y."""
    q, j = mx.quantize(y)
    codes = to_np(res.q.float()).astype(np.float64)
    scale = to_np(res.scale.view(torch.uint8)).astype(int) - 127
    other = scale != j
    if other.any():
        amax = np.abs(y).reshape(*j.shape, 32).max(-1)[other]
        top = 448 * np.exp2(np.minimum(scale, j)[other].astype(np.float64))
        assert np.all(np.abs(amax - top) <= open * top), np.count_nonzero(other)
    w = y / np.exp2(np.repeat(scale, 32, -1).astype(np.float64))
    q = mx.e4m3_round(np.clip(w, -448, 448))
    other = codes != q
    if other.any():
        mid = (codes + q)[other] / 2
        assert np.all(np.abs(w[other] - mid) <= open * np.abs(mid)), np.count_nonzero(other)


def split(s):
    """s (float64) as the sum of two bf16 values, to about 2^-17 of it."""
    hi = sw.bf16_rne(s)
    return sw.bf16_bits(hi), sw.bf16_bits(sw.bf16_rne(s - hi))


@pytest.mark.parametrize("T,D", [(3, 32), (200, 256), (64, 2816), (20, 4096), (8, 16384)])
def test_codes_below_the_normal_range(T, D):
    """Groups of one large value and 31 that lie by the middles of e4m3's subnormal codes (below 2^-6 of the scale, a
    fixed step of 2^-9)."""
    rng = np.random.default_rng(D)
    large = sw.bf16_rne(rng.uniform(1.5, 3, (T, 1, 1)))  # one magnitude a row, so the rest hardly moves its rms
    rms = np.sqrt(large**2 / 32 + 1e-6)
    unit = np.exp2(mx.scale_exponent(large / rms).astype(np.float64))
    mid = (rng.integers(0, 8, (T, D // 32, 32)) + 0.5) * 2.0**-9 * rng.choice([-1, 1], (T, D // 32, 32))
    s = mid * unit * rms
    s[:, :, 7] = (large * rng.choice([-1, 1], (T, D // 32, 1)))[:, :, 0]
    s = s.reshape(T, D)
    xb, rb = split(s)
    # a bf16 square is exact in fp32, and so is the sum of those of one magnitude, at most 2^9 of them; what may be lost
    # are the small ones: 31 (7.5 2^-9 / 362)^2 of the sum for each large one (362 = 448 2^-7 .. on the scale of 2^-6), 0.42
    # 2^-24 of y. The large value alone fills a code; the sum's own 5 roundings do not arise.
    check_codes(run(xb, rb), oracle(xb, rb), open=0.45 * 2.0**-24)


def by_the_middles(rng, T, D):
    """s whose y = s / sqrt(mean(s^2) + 1e-6) lies at the middles of normal codes: f 2^j, of a mean square m below one,
    is the y of s = f 2^j sqrt(1e-6 / (1 - m))."""
    grid = np.unique(np.abs(torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()))
    mids = ((grid[1:] + grid[:-1]) / 2)[8:]
    f = mids[rng.integers(0, len(mids), (T, D))] * rng.choice([-1, 1], (T, D))
    f.reshape(T, -1, 32)[:, :, 0] = 440.0
    rms = np.sqrt((f * f).mean(-1, keepdims=True))
    y = f * np.exp2(np.ceil(-np.log2(rms)) - 1)
    return y * np.sqrt(1e-6 / (1 - (y * y).mean(-1, keepdims=True)))


@pytest.mark.parametrize("T,D", [(200, 256), (64, 2816), (20, 4096), (8, 16384)])
def test_codes_by_the_middles(T, D):
    xb, rb = split(by_the_middles(np.random.default_rng(D + 1), T, D))
    check_codes(run(xb, rb), oracle(xb, rb))


@pytest.mark.parametrize("D", [256, 2816, 4096, 16384])
def test_codes_by_the_middles_after_a_post_norm(D):
    """The post-norm carries what the residual, in bf16, leaves of s: its gamma is made for the one row."""
    rng = np.random.default_rng(D + 2)
    for _ in range(8):
        s = by_the_middles(rng, 1, D)
        rb = sw.bf16_bits(sw.bf16_rne(s))
        xb = bits(rng.uniform(1, 2, (1, D)) * rng.choice([-1, 1], (1, D)))
        rest = (s - mo.f64(rb)) / sw.rms_norm(mo.f64(xb))
        pb = sw.bf16_bits(sw.bf16_rne(rest[0]))
        check_codes(run(xb, rb, None, pb), oracle(xb, rb, None, pb))


@pytest.mark.parametrize("T,D", [(700, 2816), (3000, 256), (300, 4096), (64, 16384), (90, 1024), (50, 1056)])
@pytest.mark.parametrize("post", [False, True])
def test_codes_of_ordinary_rows(T, D, post):
    rng = np.random.default_rng(T)
    xb, rb = bits(rng.standard_normal((T, D))), bits(2 * rng.standard_normal((T, D)))
    gb = bits(1 + 0.1 * rng.standard_normal(D))
    pb = bits(1 + 0.1 * rng.standard_normal(D)) if post else None
    check_codes(run(xb, rb, gb, pb), oracle(xb, rb, gb, pb))


@pytest.mark.parametrize("T,D", [(100, 2816), (300, 256), (20, 16384)])
def test_codes_where_the_residual_cancels(T, D):
    """residual = -(post-norm of x), rounded to bf16: s is what that rounding left, 2^-9 of either."""
    rng = np.random.default_rng(T)
    xb, pb = bits(rng.standard_normal((T, D))), bits(1 + 0.1 * rng.standard_normal(D))
    rb = sw.bf16_bits(sw.bf16_rne(-sw.rms_norm(mo.f64(xb), mo.f64(pb))))
    gb = bits(1 + 0.1 * rng.standard_normal(D))
    res = run(xb, rb, gb, pb)
    y = oracle(xb, rb, gb, pb)
    check_codes(res, y)
    # sum is rounded once, by half of bf16's step of 2^-7 at most, from an s good to a few 2^-24 of itself
    s = mo.f64(rb) + sw.rms_norm(mo.f64(xb), mo.f64(pb))
    assert np.all(np.abs(to_np(res.sum.double()) - s) <= (2.0**-8 + 2.0**-21) * np.abs(s) + 2.0**-130)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,D", [(900, 256), (400, 2816), (40, 16384)])
def test_codes_in_place(T, D, post):
    """With 8-bit output, sum and y over residual and x: everything as in separate buffers."""
    rng = np.random.default_rng(T)
    xb, rb = bits(rng.standard_normal((T, D))), bits(2 * rng.standard_normal((T, D)))
    gb = bits(1 + 0.1 * rng.standard_normal(D))
    pb = bits(1 + 0.1 * rng.standard_normal(D)) if post else None
    ref = run(xb, rb, gb, pb)
    for swap in (False, True):
        x, r = block.bf16_tensor(xb), block.bf16_tensor(rb)
        y, s = (r, x) if swap else (x, r)
        got = block.add_rms_norm(x, block.bf16_tensor(gb), residual=r, quantize=True, y=y, sum_out=s,
                                 gamma_post=None if pb is None else block.bf16_tensor(pb))
        ok()
        for a, b in ((got.y, ref.y), (got.sum, ref.sum), (got.q, ref.q), (got.scale, ref.scale)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("below", [0, 3, 7, 10])
def test_codes_of_tiny_values(below):
    """Groups whose scale is 2^-127, the smallest, and whose values lie by the middles of codes, partly where fp32 holds
    fewer than 24 bits: gamma, a power of two, brings them there."""
    rng = np.random.default_rng(below)
    D = 2816
    for _ in range(8):
        s = by_the_middles(rng, 1, D)
        xb, rb = split(s)
        _, j = mx.quantize(oracle(xb, rb))
        gb = bits(np.full(D, 2.0 ** (-127 - below - int(j.min()))))
        res = run(xb, rb, gb)
        assert np.all(to_np(res.scale.view(torch.uint8)) <= 1)
        check_codes(res, oracle(xb, rb, gb))


def test_codes_of_tiny_rows():
    rng = np.random.default_rng(5)
    T, D = 60, 256
    e = rng.integers(-130, -100, (T, D // 32, 1)).astype(np.float64)
    xb = bits(rng.standard_normal((T, D // 32, 32)) * np.exp2(e)).reshape(T, D)
    check_codes(run(xb), oracle(xb))
    gb = bits(np.exp2(rng.integers(-120, 1, D).astype(np.float64)))
    ub = bits(rng.standard_normal((T, D)))
    check_codes(run(ub, None, gb), oracle(ub, None, gb))


@pytest.mark.parametrize("above", [1, 2, 4, 8, 12])
def test_codes_of_values_that_fp32_holds_in_part(above):
    """Groups at the scales just above the smallest: their smaller values lie where fp32 holds fewer than 24 bits."""
    rng = np.random.default_rng(above)
    D = 2816
    for _ in range(8):
        xb, rb = split(by_the_middles(rng, 1, D))
        _, j = mx.quantize(oracle(xb, rb))
        gb = bits(np.full(D, 2.0 ** (-127 + above - int(j.min()))))
        res = run(xb, rb, gb)
        assert int(res.scale.view(torch.uint8).min()) == above
        check_codes(res, oracle(xb, rb, gb))


@pytest.mark.parametrize("D", [256, 2816, 4096, 16384])
def test_post_norm_of_special_rows(D):
    """Rows with an infinity (x / inf = 0, inf / inf = NaN), a NaN (all NaN), the largest and the smallest values, zeros."""
    rng = np.random.default_rng(D)
    T = 6
    xb, rb = bits(rng.standard_normal((T, D))), bits(rng.standard_normal((T, D)))
    pb, gb = bits(1 + 0.1 * rng.standard_normal(D)), bits(1 + 0.1 * rng.standard_normal(D))
    x, r = block.bf16_tensor(xb), block.bf16_tensor(rb)
    x[0, 7], x[1, 9] = float("-inf"), float("nan")
    x[2] *= 2.0**100  # squares far past fp32
    x[3] *= 2.0**-60
    x[4] = 0.0
    for kw in ({}, {"y": x.clone(), "sum_out": None}):
        src = kw.get("y", x)
        res = block.add_rms_norm(src, block.bf16_tensor(gb), residual=r, gamma_post=block.bf16_tensor(pb), quantize=True, **kw)
        ok()
        keep = torch.ones(D, dtype=torch.bool, device="cuda")
        keep[7] = False
        assert torch.equal(res.sum[0, keep], r[0, keep]) and torch.isnan(res.sum[0, 7])
        assert torch.isnan(res.sum[1]).all()
        for t in (0, 1):
            assert torch.isnan(res.y[t]).all() and torch.all(res.scale[t].view(torch.uint8) == 0xFF)
            assert torch.isnan(res.q[t].float()).all()
        finite = [2, 3, 4, 5]
        xv = xb.copy()
        xv[2], xv[3], xv[4] = sw.bf16_bits(mo.f64(xb[2]) * 2.0**100), sw.bf16_bits(mo.f64(xb[3]) * 2.0**-60), 0
        y = oracle(xv[finite], rb[finite], gb, pb)
        part = block.NormResult(None, None, res.q[finite], res.scale[finite])
        check_codes(part, y)
        assert np.all(np.abs(to_np(res.y[finite].double()) - y) <= (2.0**-8 + 2.0**-20) * np.abs(y))
