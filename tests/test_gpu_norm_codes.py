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
