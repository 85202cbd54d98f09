"""Checks that the Python layer of the MXFP8 block and the few-token layer makes before anything runs (no GPU)."""

import pytest
import torch

from mixture_experts_transformer_b200 import binding as B
from mixture_experts_transformer_b200 import block, build, inputs

DIMS = inputs.Dims(embed_dim=128, num_experts=8, expert_dim=64, hidden_dim=192)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def linear(G, K, N, device="cpu"):
    qb, sfb = B.moe_mxfp8_weight_bytes(G, K, N)
    return block.Mxfp8Linear(torch.empty(qb, dtype=torch.uint8, device=device),
                             torch.empty(sfb, dtype=torch.uint8, device=device), G, K, N)


def mxfp8_weights(router, device="cpu", last=None):
    d = DIMS
    gu, dn = (d.num_experts, d.embed_dim, d.expert_dim), (d.num_experts, d.expert_dim, d.embed_dim)
    sgu, sdn = (1, d.embed_dim, d.hidden_dim), (1, d.hidden_dim, d.embed_dim)
    return block.Mxfp8Weights(d, router, linear(*gu, device), linear(*gu, device), linear(*dn, device),
                              linear(*sgu, device), linear(*sgu, device), linear(*sdn, last or device))


def test_mxfp8_weights_check_the_router():
    d = DIMS
    router = torch.empty((d.embed_dim, d.num_experts), dtype=torch.bfloat16)
    mxfp8_weights(router)
    for bad in (router.float(), router[:, :-1], router[:-1], router.t(), router.reshape(-1),
                torch.empty((d.embed_dim, 2 * d.num_experts), dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(ValueError, match="w_router"):
            mxfp8_weights(bad)


def test_mxfp8_weights_are_on_one_device():
    router = torch.empty((DIMS.embed_dim, DIMS.num_experts), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="sd"):
        mxfp8_weights(router, last="meta")
    with pytest.raises(ValueError, match="wg"):
        mxfp8_weights(router.to("meta"))


def test_weights_on_another_device_are_refused():
    router = torch.empty((DIMS.embed_dim, DIMS.num_experts), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="w_router is on cpu"):
        block._weights_on(0, {"w_router": router})
    block._weights_on(-1, {"w_router": router})


def test_stream_handle_without_the_raw_stream_call(monkeypatch):
    """The handle of the current stream comes through torch's public call where the quicker internal one is missing."""

    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(B, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert B.stream_handle() == 1234
    assert B.stream_handle() == 1234
    assert B.stream_handle(Stream) == 1234
