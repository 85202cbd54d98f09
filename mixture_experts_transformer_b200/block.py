"""Device-side convenience around the C ABI: upload bf16 weights once, run the block.

Marshalling only. Every computation happens inside libmoeblock.so.
"""

from __future__ import annotations

import dataclasses

import numpy as np
import torch

from . import binding as B
from .inputs import BlockWeights, Dims


def bf16_tensor(bits: np.ndarray, device="cuda") -> torch.Tensor:
    """bf16 bit patterns (uint16 numpy) -> torch.bfloat16 tensor on `device`."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)
    return t.to(device) if device != "cpu" else t


@dataclasses.dataclass
class DeviceWeights:
    dims: Dims
    w_router: torch.Tensor
    wg: torch.Tensor
    wu: torch.Tensor
    wd: torch.Tensor
    sg: torch.Tensor
    su: torch.Tensor
    sd: torch.Tensor

    def args(self):
        return (self.w_router, self.wg, self.wu, self.wd, self.sg, self.su, self.sd)


def upload(w: BlockWeights, device="cuda") -> DeviceWeights:
    return DeviceWeights(
        w.dims, *(bf16_tensor(a, device) for a in (w.w_router, w.wg, w.wu, w.wd, w.sg, w.su, w.sd))
    )


@dataclasses.dataclass
class BlockResult:
    out: torch.Tensor
    out_f32: torch.Tensor | None = None
    idx: torch.Tensor | None = None
    w: torch.Tensor | None = None
    cnt: torch.Tensor | None = None
    logits: torch.Tensor | None = None


def forward(
    dw: DeviceWeights,
    x: torch.Tensor,
    *,
    top_k: int = B.TOP_K,
    router_bias: torch.Tensor | None = None,
    debug: bool = False,
    workspace: torch.Tensor | None = None,
    out: torch.Tensor | None = None,
    stream=None,
    norm_pre: torch.Tensor | None = None,
    norm_post: torch.Tensor | None = None,
    residual: bool = False,
) -> BlockResult:
    """Run one block; with debug=True also return out_f32, the routing, the router logits and the counts.
    norm_pre / norm_post (bf16 [embed_dim]) and residual add the normalisation
    sandwich: out = x + norm_post-RMSNorm(block(norm_pre-RMSNorm(x)))."""
    T = x.shape[0]
    dev = x.device
    if out is None:
        out = torch.empty((T, dw.dims.embed_dim), dtype=torch.bfloat16, device=dev)
    res = BlockResult(out=out)
    if debug:
        res.out_f32 = torch.empty((T, dw.dims.embed_dim), dtype=torch.float32, device=dev)
        res.idx = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        res.w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        res.cnt = torch.empty((dw.dims.num_experts,), dtype=torch.int32, device=dev)
        res.logits = torch.empty((T, dw.dims.num_experts), dtype=torch.float32, device=dev)
    p = B.make_params(
        T,
        x,
        *dw.args(),
        out,
        top_k=top_k,
        dims=dw.dims,
        router_bias=router_bias,
        out_f32=res.out_f32,
        idx_out=res.idx,
        w_out=res.w,
        cnt_out=res.cnt,
        workspace=workspace,
        norm_pre=norm_pre,
        norm_post=norm_post,
        residual=residual,
        logits_out=res.logits,
    )
    B.check(B.moe_block_forward_ex(p, stream), "moe_block_forward_ex")
    return res


def workspace_for(dims: Dims, T: int, top_k: int = B.TOP_K, device="cuda") -> tuple[torch.Tensor, B.MoeWsLayout]:
    """A caller-owned workspace (uint8) and its layout."""
    p = B.make_params(T, top_k=top_k, dims=dims)
    lay = B.moe_workspace_layout(p)
    return torch.empty(lay.total_bytes, dtype=torch.uint8, device=device), lay


# ----------------------------------------------------------------- NVFP4


@dataclasses.dataclass
class Nvfp4Linear:
    """One quantised Linear stack on the device: codes, scale atoms, tensor scales."""

    q: torch.Tensor
    sf: torch.Tensor
    g: torch.Tensor
    groups: int
    K: int
    N: int

    def struct(self) -> B.MoeNvfp4Linear:
        return B.MoeNvfp4Linear(self.q.data_ptr(), self.sf.data_ptr(), self.g.data_ptr())


def quantize_linear(w: torch.Tensor, stream=None) -> Nvfp4Linear:
    """w [G][K][N] (or [K][N]) bf16 on the device -> NVFP4 (the library's quantiser)."""
    w3 = w if w.dim() == 3 else w.unsqueeze(0)
    G, K, N = w3.shape
    qb, sfb = B.moe_nvfp4_weight_bytes(G, K, N)
    q = torch.empty(qb, dtype=torch.uint8, device=w.device)
    sf = torch.empty(sfb, dtype=torch.uint8, device=w.device)
    g = torch.empty(G, dtype=torch.float32, device=w.device)
    B.check(B.moe_nvfp4_quantize_weight(w3, G, K, N, q, sf, g, stream), "moe_nvfp4_quantize_weight")
    return Nvfp4Linear(q, sf, g, G, K, N)


@dataclasses.dataclass
class Nvfp4Weights:
    dims: Dims
    w_router: torch.Tensor
    wg: Nvfp4Linear
    wu: Nvfp4Linear
    wd: Nvfp4Linear
    sg: Nvfp4Linear
    su: Nvfp4Linear
    sd: Nvfp4Linear


def quantize_block(dw: DeviceWeights, stream=None) -> Nvfp4Weights:
    return Nvfp4Weights(
        dw.dims,
        dw.w_router,
        *(quantize_linear(t, stream) for t in (dw.wg, dw.wu, dw.wd, dw.sg, dw.su, dw.sd)),
    )


def forward_nvfp4(
    nw: Nvfp4Weights,
    x: torch.Tensor,
    act_scales,
    *,
    top_k: int = B.TOP_K,
    router_bias: torch.Tensor | None = None,
    rms_norm_out: bool = False,
    debug: bool = False,
    workspace: torch.Tensor | None = None,
    out: torch.Tensor | None = None,
    stream=None,
) -> BlockResult:
    """One NVFP4 block; act_scales = (g_x, g_h, g_hs)."""
    T = x.shape[0]
    if out is None:
        out = torch.empty((T, nw.dims.embed_dim), dtype=torch.bfloat16, device=x.device)
    res = BlockResult(out=out)
    if debug:
        res.out_f32 = torch.empty((T, nw.dims.embed_dim), dtype=torch.float32, device=x.device)
        res.idx = torch.empty((T, top_k), dtype=torch.int32, device=x.device)
        res.w = torch.empty((T, top_k), dtype=torch.float32, device=x.device)
        res.cnt = torch.empty((nw.dims.num_experts,), dtype=torch.int32, device=x.device)
    p = nvfp4_params(nw, T, x, out, act_scales, top_k=top_k, router_bias=router_bias, rms_norm_out=rms_norm_out,
                     res=res, workspace=workspace)
    B.check(B.moe_block_forward_nvfp4(p, stream), "moe_block_forward_nvfp4")
    return res


def nvfp4_params(nw, T, x, out, act_scales, *, top_k=B.TOP_K, router_bias=None, rms_norm_out=False, res=None,
                 workspace=None) -> B.MoeNvfp4Params:
    p = B.MoeNvfp4Params()
    p.T, p.top_k_experts = T, top_k
    d = nw.dims
    p.embed_dim, p.num_experts, p.expert_dim, p.hidden_dim = d.embed_dim, d.num_experts, d.expert_dim, d.hidden_dim
    p.x, p.w_router, p.router_bias = B.ptr(x), B.ptr(nw.w_router), B.ptr(router_bias)
    for name in ("wg", "wu", "wd", "sg", "su", "sd"):
        setattr(p, name, getattr(nw, name).struct())
    p.g_x, p.g_h, p.g_hs = (float(v) for v in act_scales)
    p.rms_norm_out = 1 if rms_norm_out else 0
    p.out = B.ptr(out)
    if res is not None:
        p.out_f32, p.idx_out, p.w_out, p.cnt_out = (B.ptr(res.out_f32), B.ptr(res.idx), B.ptr(res.w), B.ptr(res.cnt))
    if workspace is not None:
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.numel()
    return p


def calibrate(dw: DeviceWeights, x: torch.Tensor, top_k: int = B.TOP_K, router_bias=None, stream=None):
    """Static NVFP4 activation tensor scales (g_x, g_h, g_hs) from one calibration
    batch run through the bf16 block: the library's observer writes the amax
    values and the scales on the device; they are copied back here.
    Returns ((g_x, g_h, g_hs) as float32, amax [3] float32)."""
    ws, _ = workspace_for(dw.dims, x.shape[0], top_k, device=x.device)
    out = torch.empty((x.shape[0], dw.dims.embed_dim), dtype=torch.bfloat16, device=x.device)
    amax = torch.zeros(3, dtype=torch.float32, device=x.device)
    scales = torch.zeros(3, dtype=torch.float32, device=x.device)
    p = B.make_params(x.shape[0], x, *dw.args(), out, top_k=top_k, dims=dw.dims, router_bias=router_bias, workspace=ws)
    B.check(B.moe_nvfp4_calibrate(p, amax, scales, stream), "moe_nvfp4_calibrate")
    g = scales.cpu().numpy().astype(np.float32)
    return tuple(np.float32(v) for v in g), amax.cpu().numpy().astype(np.float32)


# ------------------------------------------------ weight-only SFP8 / Q4_0


@dataclasses.dataclass
class WqLinear:
    """G stacked [K, N] Linears in a weight-only format: the library's blocks
    (uint8) and, for SFP8, the fp32 matrix scales [G]."""

    q: torch.Tensor
    scale: torch.Tensor | None

    def struct(self) -> B.MoeWqLinear:
        return B.MoeWqLinear(B.ptr(self.q), B.ptr(self.scale))


@dataclasses.dataclass
class WqWeights:
    dims: Dims
    fmt: str
    w_router: torch.Tensor
    wg: WqLinear
    wu: WqLinear
    wd: WqLinear
    sg: WqLinear
    su: WqLinear
    sd: WqLinear


def quantize_wq_linear(w: torch.Tensor, fmt: str, stream=None) -> WqLinear:
    """w [G, K, N] or [K, N] bf16 (device) -> the library's format `fmt`."""
    w3 = w if w.dim() == 3 else w.unsqueeze(0)
    G, K, N = w3.shape
    code = B.WFORMATS[fmt]
    q = torch.empty(B.moe_wq_weight_bytes(code, G, K, N), dtype=torch.uint8, device=w.device)
    scale = torch.empty(G, dtype=torch.float32, device=w.device) if fmt == "sfp8" else None
    B.check(B.moe_wq_quantize_weight(code, w3, G, K, N, q, scale, stream), "moe_wq_quantize_weight")
    return WqLinear(q, scale)


def quantize_wq(dw: DeviceWeights, fmt: str, stream=None) -> WqWeights:
    return WqWeights(dw.dims, fmt, dw.w_router,
                     *(quantize_wq_linear(t, fmt, stream) for t in (dw.wg, dw.wu, dw.wd, dw.sg, dw.su, dw.sd)))


def wq_params(ww: WqWeights, T: int, x, out, *, top_k=B.TOP_K, router_bias=None, res=None,
              workspace=None) -> B.MoeWqParams:
    p = B.MoeWqParams()
    p.T, p.top_k_experts, p.format = T, top_k, B.WFORMATS[ww.fmt]
    d = ww.dims
    p.embed_dim, p.num_experts, p.expert_dim, p.hidden_dim = d.embed_dim, d.num_experts, d.expert_dim, d.hidden_dim
    p.x, p.w_router, p.router_bias = B.ptr(x), B.ptr(ww.w_router), B.ptr(router_bias)
    for name in ("wg", "wu", "wd", "sg", "su", "sd"):
        setattr(p, name, getattr(ww, name).struct())
    p.out = B.ptr(out)
    if res is not None:
        p.out_f32, p.idx_out, p.w_out, p.cnt_out = (B.ptr(res.out_f32), B.ptr(res.idx), B.ptr(res.w), B.ptr(res.cnt))
    if workspace is not None:
        p.workspace = workspace.data_ptr()
        p.workspace_bytes = workspace.numel()
    return p


def forward_wq(ww: WqWeights, x: torch.Tensor, *, top_k: int = B.TOP_K, router_bias=None, debug: bool = False,
               workspace: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> BlockResult:
    """One block with weight-only SFP8 / Q4_0 expert and shared Linears."""
    T = x.shape[0]
    if out is None:
        out = torch.empty((T, ww.dims.embed_dim), dtype=torch.bfloat16, device=x.device)
    res = BlockResult(out=out)
    if debug:
        res.out_f32 = torch.empty((T, ww.dims.embed_dim), dtype=torch.float32, device=x.device)
        res.idx = torch.empty((T, top_k), dtype=torch.int32, device=x.device)
        res.w = torch.empty((T, top_k), dtype=torch.float32, device=x.device)
        res.cnt = torch.empty((ww.dims.num_experts,), dtype=torch.int32, device=x.device)
    p = wq_params(ww, T, x, out, top_k=top_k, router_bias=router_bias, res=res, workspace=workspace)
    B.check(B.moe_block_forward_wq(p, stream), "moe_block_forward_wq")
    return res


# ----------------------------------- few tokens, MXFP8 and the add-norm


def _rows(name: str, t: torch.Tensor, shape, dtypes, device: int) -> int:
    """t's address, after checking that it is a contiguous [shape] tensor of one of `dtypes` on CUDA device `device`."""
    if t.shape != shape or t.dtype not in dtypes or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name}: needs a contiguous {tuple(shape)} tensor of {' or '.join(map(str, dtypes))} on "
                         f"cuda:{device}, got {tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _on_current_device(x: torch.Tensor) -> int:
    """The index of x's device, which has to be the current one: the library launches there."""
    index = x.get_device()
    if index < 0 or index != torch.cuda.current_device():
        raise ValueError(f"x is on {x.device}: the library runs on the current CUDA device")
    return index


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory that `stream` (None: the current one) is to write: from that stream's pool, as other streams may still be
    using what the current one's holds, and not to be taken for another tensor while the current stream reads it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _weights_on(device: int, tensors: dict) -> None:
    """Refuses weights that are not on CUDA device `device` (where the library runs)."""
    for name, t in tensors.items():
        if t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}: the call runs on cuda:{device}")


_BF16, _E4M3, _E8M0 = (torch.bfloat16,), (torch.float8_e4m3fn, torch.uint8), (torch.float8_e8m0fnu, torch.uint8)


def few_workspace(dw: DeviceWeights, T: int, top_k: int = B.TOP_K) -> torch.Tensor:
    """A workspace (uint8) for forward_few calls of T tokens."""
    need = B.moe_few_workspace_bytes(B.make_params(T, top_k=top_k, dims=dw.dims))
    return torch.empty(need, dtype=torch.uint8, device=dw.w_router.device)


def forward_few(
    dw: DeviceWeights,
    x: torch.Tensor,
    *,
    top_k: int = B.TOP_K,
    router_bias: torch.Tensor | None = None,
    debug: bool = False,
    workspace: torch.Tensor | None = None,
    out: torch.Tensor | None = None,
    stream=None,
    norm_pre: torch.Tensor | None = None,
    norm_post: torch.Tensor | None = None,
    residual: bool = False,
) -> BlockResult:
    """forward() in two kernels for at most B.FEW_MAX_TOKENS tokens, unrounded between x and the output."""
    dev = _on_current_device(x)
    T, D = x.shape[0], dw.dims.embed_dim
    _rows("x", x, (T, D), _BF16, dev)
    _weights_on(dev, {n: getattr(dw, n) for n in ("w_router", "wg", "wu", "wd", "sg", "su", "sd")})
    for name, t in (("norm_pre", norm_pre), ("norm_post", norm_post)):
        if t is not None:
            _rows(name, t, (D,), _BF16, dev)
    if router_bias is not None:
        _rows("router_bias", router_bias, (dw.dims.num_experts,), (torch.float32,), dev)
    if workspace is not None:
        _rows("workspace", workspace, workspace.shape, (torch.uint8,), dev)
    if out is None:
        out = _empty((T, D), torch.bfloat16, x.device, stream)
    _rows("out", out, (T, D), _BF16, dev)
    res = _result(out, dw.dims, top_k, debug, stream)
    if debug:
        res.logits = _empty((T, dw.dims.num_experts), torch.float32, x.device, stream)
    d, ptr = dw.dims, B.ptr
    p = B.MoeParams(T, top_k, D, d.num_experts, d.expert_dim, d.hidden_dim, ptr(x), ptr(dw.w_router), ptr(router_bias),
                    ptr(dw.wg), ptr(dw.wu), ptr(dw.wd), ptr(dw.sg), ptr(dw.su), ptr(dw.sd), ptr(out), ptr(res.out_f32),
                    ptr(res.idx), ptr(res.w), ptr(res.cnt), ptr(workspace),
                    0 if workspace is None else workspace.numel(), ptr(norm_pre), ptr(norm_post), int(residual),
                    ptr(res.logits))
    B.check(B.moe_block_forward_few(p, stream), "moe_block_forward_few")
    return res


@dataclasses.dataclass
class NormResult:
    y: torch.Tensor | None
    sum: torch.Tensor | None
    q: torch.Tensor | None = None
    scale: torch.Tensor | None = None


def add_rms_norm(
    x: torch.Tensor,
    gamma: torch.Tensor | None = None,
    *,
    residual: torch.Tensor | None = None,
    gamma_post: torch.Tensor | None = None,
    quantize: bool = False,
    y: torch.Tensor | None = None,
    sum_out: torch.Tensor | None = None,
    q: torch.Tensor | None = None,
    scale: torch.Tensor | None = None,
    eps: float = 1e-6,
    stream=None,
) -> NormResult:
    """s = residual + (gamma_post-RMSNorm(x) with gamma_post, else x); y = gamma-RMSNorm(s), in one kernel.

    x, residual [T, D] bf16; gamma, gamma_post [D] bf16. Returns y and sum = s
    in bf16 and, with quantize=True or q and scale given, y in MXFP8: q [T, D]
    e4m3 and scale [T, D/32] e8m0. Outputs may be passed in; y and sum_out may
    each be x or residual itself (in place)."""
    dev = _on_current_device(x)
    shape = x.shape
    T, D = shape
    px = _rows("x", x, shape, _BF16, dev)
    pres = None if residual is None else _rows("residual", residual, shape, _BF16, dev)
    pgam = None if gamma is None else _rows("gamma", gamma, (D,), _BF16, dev)
    ppost = None if gamma_post is None else _rows("gamma_post", gamma_post, (D,), _BF16, dev)
    if y is None:
        y = _empty(shape, torch.bfloat16, x.device, stream)
    if sum_out is None:
        sum_out = _empty(shape, torch.bfloat16, x.device, stream)
    py, psum = _rows("y", y, shape, _BF16, dev), _rows("sum_out", sum_out, shape, _BF16, dev)
    pq = pscale = None
    if quantize or q is not None or scale is not None:
        if q is None:
            q = _empty(shape, torch.float8_e4m3fn, x.device, stream)
        if scale is None:
            scale = _empty((T, D // B.MXFP8_GROUP), torch.float8_e8m0fnu, x.device, stream)
        pq = _rows("q", q, shape, _E4M3, dev)
        pscale = _rows("scale", scale, (T, D // B.MXFP8_GROUP), _E8M0, dev)
    p = B.MoeNormParams(T, D, eps, px, pres, ppost, pgam, psum, py, pq, pscale)
    B.check(B.moe_add_rms_norm(p, stream), "moe_add_rms_norm")
    return NormResult(y, sum_out, q, scale)


@dataclasses.dataclass
class Mxfp8Linear:
    """G stacked [K, N] Linears in MXFP8 on the device: codes [G, N, K] e4m3 and the scale tiles."""

    q: torch.Tensor
    sf: torch.Tensor
    groups: int
    K: int
    N: int

    def __post_init__(self):
        sizes = B.moe_mxfp8_weight_bytes(self.groups, self.K, self.N)
        for name, t, n in (("q", self.q, sizes[0]), ("sf", self.sf, sizes[1])):
            if t.numel() != n or t.element_size() != 1 or not t.is_contiguous():
                raise ValueError(f"{name}: {self.groups} Linears [{self.K}, {self.N}] need {n} contiguous bytes, got "
                                 f"{tuple(t.shape)} {t.dtype}, strides {t.stride()}")

    def struct(self) -> B.MoeMxfp8Linear:
        return B.MoeMxfp8Linear(self.q.data_ptr(), self.sf.data_ptr())


def quantize_mxfp8_linear(w: torch.Tensor, stream=None) -> Mxfp8Linear:
    """w [G, K, N] (or [K, N]) bf16 on the device -> MXFP8 along K (the library's quantiser)."""
    w3 = w if w.dim() == 3 else w.unsqueeze(0)
    G, K, N = w3.shape
    _rows("w", w3, (G, K, N), _BF16, _on_current_device(w3))
    _, sfb = B.moe_mxfp8_weight_bytes(G, K, N)
    q = _empty((G, N, K), torch.float8_e4m3fn, w.device, stream)
    sf = _empty(sfb, torch.float8_e8m0fnu, w.device, stream)
    B.check(B.moe_mxfp8_quantize_weight(w3, G, K, N, q, sf, stream), "moe_mxfp8_quantize_weight")
    return Mxfp8Linear(q, sf, G, K, N)


def quantize_mxfp8_rows(x: torch.Tensor, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """x [T, D] bf16 -> (q [T, D] e4m3, scale [T, D/32] e8m0)."""
    T, D = x.shape
    dev = _on_current_device(x)
    _rows("x", x, (T, D), _BF16, dev)
    q = _empty((T, D), torch.float8_e4m3fn, x.device, stream)
    scale = _empty((T, D // B.MXFP8_GROUP), torch.float8_e8m0fnu, x.device, stream)
    B.check(B.moe_mxfp8_quantize_act(x, T, D, q, scale, stream), "moe_mxfp8_quantize_act")
    return q, scale


@dataclasses.dataclass
class Mxfp8Weights:
    dims: Dims
    w_router: torch.Tensor
    wg: Mxfp8Linear
    wu: Mxfp8Linear
    wd: Mxfp8Linear
    sg: Mxfp8Linear
    su: Mxfp8Linear
    sd: Mxfp8Linear

    def __post_init__(self):
        d = self.dims
        for name, G, K, N in (("wg", d.num_experts, d.embed_dim, d.expert_dim), ("wu", d.num_experts, d.embed_dim, d.expert_dim),
                              ("wd", d.num_experts, d.expert_dim, d.embed_dim), ("sg", 1, d.embed_dim, d.hidden_dim),
                              ("su", 1, d.embed_dim, d.hidden_dim), ("sd", 1, d.hidden_dim, d.embed_dim)):
            lin = getattr(self, name)
            if (lin.groups, lin.K, lin.N) != (G, K, N):
                raise ValueError(f"{name}: {G} Linears [{K}, {N}] expected, got {lin.groups} of [{lin.K}, {lin.N}]")
            if lin.q.device != self.w_router.device or lin.sf.device != self.w_router.device:
                raise ValueError(f"{name}: on {lin.q.device} and {lin.sf.device}, the router on {self.w_router.device}")
        r = self.w_router
        if r.shape != (d.embed_dim, d.num_experts) or r.dtype != torch.bfloat16 or not r.is_contiguous():
            raise ValueError(f"w_router: needs a contiguous {(d.embed_dim, d.num_experts)} tensor of torch.bfloat16, got "
                             f"{tuple(r.shape)} {r.dtype}, strides {r.stride()}")


def quantize_mxfp8(dw: DeviceWeights, stream=None) -> Mxfp8Weights:
    return Mxfp8Weights(dw.dims, dw.w_router,
                        *(quantize_mxfp8_linear(t, stream) for t in (dw.wg, dw.wu, dw.wd, dw.sg, dw.su, dw.sd)))


def mxfp8_params(mw: Mxfp8Weights, T: int, x=None, out=None, *, xq=None, xs=None, top_k=B.TOP_K, router_bias=None,
                 res=None, workspace=None) -> B.MoeMxfp8Params:
    d = mw.dims
    res = res or BlockResult(out=out)
    return B.MoeMxfp8Params(
        T, top_k, d.embed_dim, d.num_experts, d.expert_dim, d.hidden_dim, B.ptr(x), B.ptr(xq), B.ptr(xs),
        B.ptr(mw.w_router), B.ptr(router_bias), mw.wg.struct(), mw.wu.struct(), mw.wd.struct(), mw.sg.struct(),
        mw.su.struct(), mw.sd.struct(), B.ptr(out), B.ptr(res.out_f32), B.ptr(res.idx), B.ptr(res.w), B.ptr(res.cnt),
        B.ptr(workspace), 0 if workspace is None else workspace.numel())


def mxfp8_workspace(mw: Mxfp8Weights, T: int, top_k: int = B.TOP_K) -> torch.Tensor:
    """A workspace (uint8) for forward_mxfp8 calls of T tokens."""
    need = B.moe_mxfp8_workspace_bytes(mxfp8_params(mw, T, top_k=top_k))
    return torch.empty(need, dtype=torch.uint8, device=mw.w_router.device)


def forward_mxfp8(
    mw: Mxfp8Weights,
    x: torch.Tensor,
    *,
    xq: torch.Tensor | None = None,
    xs: torch.Tensor | None = None,
    top_k: int = B.TOP_K,
    router_bias: torch.Tensor | None = None,
    debug: bool = False,
    workspace: torch.Tensor | None = None,
    out: torch.Tensor | None = None,
    stream=None,
) -> BlockResult:
    """One block with MXFP8 weights and activations. x [T, D] bf16 feeds the
    router; xq / xs are the same rows in MXFP8 (as add_rms_norm writes them),
    without them the call quantises x. (xs off a 16-byte boundary, as a slice of
    a batch's rows may be, is copied to one first.)"""
    dev = _on_current_device(x)
    T, D = x.shape[0], mw.dims.embed_dim
    _rows("x", x, (T, D), _BF16, dev)
    _weights_on(dev, {"w_router": mw.w_router})  # (the others are where it is)
    if xq is not None:
        _rows("xq", xq, (T, D), _E4M3, dev)
    if xs is not None and _rows("xs", xs, (T, D // B.MXFP8_GROUP), _E8M0, dev) % 16:
        xs, part = _empty(xs.shape, xs.dtype, xs.device, stream), xs  # (rows of a batch may start anywhere)
        with torch.cuda.stream(stream):
            xs.view(torch.uint8).copy_(part.view(torch.uint8))
    if router_bias is not None:
        _rows("router_bias", router_bias, (mw.dims.num_experts,), (torch.float32,), dev)
    if workspace is not None:
        _rows("workspace", workspace, workspace.shape, (torch.uint8,), dev)
    if out is None:
        out = _empty((T, D), torch.bfloat16, x.device, stream)
    _rows("out", out, (T, D), _BF16, dev)
    res = _result(out, mw.dims, top_k, debug, stream)
    p = mxfp8_params(mw, T, x, out, xq=xq, xs=xs, top_k=top_k, router_bias=router_bias, res=res, workspace=workspace)
    B.check(B.moe_block_forward_mxfp8(p, stream), "moe_block_forward_mxfp8")
    return res


def _result(out: torch.Tensor, dims: Dims, top_k: int, debug: bool, stream) -> BlockResult:
    res = BlockResult(out=out)
    if debug:
        T, dev = out.shape[0], out.device
        res.out_f32 = _empty((T, dims.embed_dim), torch.float32, dev, stream)
        res.idx = _empty((T, top_k), torch.int32, dev, stream)
        res.w = _empty((T, top_k), torch.float32, dev, stream)
        res.cnt = _empty((dims.num_experts,), torch.int32, dev, stream)
    return res


# ---------------------------------------------------------------- dense FFN


def dense_forward(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, wd: torch.Tensor, *, debug: bool = False,
                  workspace: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> BlockResult:
    """The dense GeGLU FFN: out = (gelu_tanh(x wg) * (x wu)) wd; wg, wu [D, S], wd [S, D] bf16."""
    T, D = x.shape
    S = wg.shape[1]
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=x.device)
    res = BlockResult(out=out)
    if debug:
        res.out_f32 = torch.empty((T, D), dtype=torch.float32, device=x.device)
    p = B.make_dense_params(T, x, wg, wu, wd, out, embed_dim=D, hidden_dim=S, out_f32=res.out_f32,
                            workspace=workspace)
    B.check(B.moe_dense_ffn_forward(p, stream), "moe_dense_ffn_forward")
    return res
