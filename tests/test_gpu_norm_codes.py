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


# What 64-bit arithmetic of a row (sums of up to 2^14 squares in order, 2^-53 each, a root, a few products) may leave
# open: 2^14 2^-53 of the sum at most, so anything within 2^-38 of a border may fall on either side.
OPEN = 2.0**-38


def check_codes(res, y):
    """Codes and scales of res are the 64-bit oracle's of y."""
    q, j = mx.quantize(y)
    codes = to_np(res.q.float()).astype(np.float64)
    scale = to_np(res.scale.view(torch.uint8)).astype(int) - 127
    other = scale != j
    if other.any():
        amax = np.abs(y).reshape(*j.shape, 32).max(-1)[other]
        top = 448 * np.exp2(np.minimum(scale, j)[other].astype(np.float64))
        assert np.all(np.abs(amax - top) <= OPEN * top), np.count_nonzero(other)
    w = y / np.exp2(np.repeat(scale, 32, -1).astype(np.float64))
    q = mx.e4m3_round(np.clip(w, -448, 448))
    other = codes != q
    if other.any():
        mid = (codes + q)[other] / 2
        assert np.all(np.abs(w[other] - mid) <= OPEN * np.abs(mid)), np.count_nonzero(other)


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
    check_codes(run(xb, rb), oracle(xb, rb))


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
