"""Cases of three operators of the library, with their plain forms.

* ``norm``: the seam between two sub-layers of the normalisation sandwich:
  ``s = residual + x`` (or ``residual + gamma_post x / rms(x)``),
  ``y = gamma s / rms(s)``, with ``s`` and ``y`` in bf16 and ``y`` also in
  MXFP8 (e4m3 values under one power-of-two scale for each 32 of a row);
* ``few``: the whole MoE layer in bf16 for at most 16 tokens;
* ``mx``: the MoE layer with MXFP8 weights and activations, for any number of
  tokens, from bf16 rows or from the rows that ``norm`` wrote in 8 bits.

MXFP8 of 32 values v: the scale is the smallest 2^j >= max|v| / 448 with
j in [-127, 127], the values are v / 2^j rounded to e4m3 (nearest, ties to
even). The routed weights of a layer are quantised along the reduction; the
GeGLU rows between its two products are quantised again, the router stays bf16.
"""

import math

import torch

own = False

EMBED, EXPERTS, EXPERT_DIM, HIDDEN, TOP_K = 2816, 128, 704, 2112, 8  # the Gemma-4-26B-A4B block
E4B_EMBED = 2560  # the dense sibling's width
EPS = 1e-6
STD = 0.02  # the checkpoint's initializer_range


def listed():
    norm = dict(op="norm", D=EMBED, post=True, quant=True)
    layer = dict(D=EMBED, E=EXPERTS, F=EXPERT_DIM, S=HIDDEN, k=TOP_K, bias=False)
    few = dict(layer, op="few", sandwich=False)
    mx = dict(layer, op="mx", fed=False)
    return [
        # eight requests decoding: the seam before an MXFP8 layer, launch latency
        dict(norm, name="norm decode 8", T=8),
        # a ragged prefill of the dense sibling's width, bf16 only, no post-norm
        dict(norm, name="norm ragged 777", T=777, D=E4B_EMBED, post=False, quant=False),
        # a prefill batch before an MXFP8 layer
        dict(norm, name="norm prefill 4096", T=4096, post=False),
        # the largest batch of the block's workloads, every output
        dict(norm, name="norm batch 16384", T=16384),
        # one user decoding
        dict(few, name="few 1", T=1),
        # a handful of requests, with the layer's norms and residual around it
        dict(few, name="few 5 sandwich", T=5, sandwich=True),
        # the most tokens of the call, e.g. a verified draft of 16
        dict(few, name="few 16", T=16),
        # one user decoding in 8 bits, the rows as the norm wrote them
        dict(mx, name="mx 1 fed", T=1, fed=True),
        # eight requests decoding, with a load-balancing bias on the router
        dict(mx, name="mx 8 bias", T=8, bias=True),
        # a decode batch: every expert is touched, the weights bound it
        dict(mx, name="mx 64 fed", T=64, fed=True),
        # a ragged prefill chunk
        dict(mx, name="mx 777", T=777),
        # a prefill batch: the tensor cores bound it
        dict(mx, name="mx 4096", T=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "few", "mx"))
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 16384), D=64 * rng.randint(1, 44), post=rng.random() < 0.5,
                    quant=rng.random() < 0.7)
    whole = rng.random() < 0.5  # the block's own widths, or others
    case = dict(op=op, T=rng.randint(1, 16) if op == "few" else _log(rng, 1, 4096),
                D=EMBED if whole else 64 * rng.randint(2, 44), E=EXPERTS if whole else 8 * rng.randint(2, 16),
                F=EXPERT_DIM if whole else 64 * rng.randint(1, 11), S=HIDDEN if whole else 64 * rng.randint(1, 33),
                k=rng.randint(1, 8), bias=rng.random() < 0.3)
    case["sandwich" if op == "few" else "fed"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs


def _randn(g, shape, std):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).bfloat16()


def _weight(g, shape, mx):
    """bf16 [G, K, N], or its MXFP8 form: e4m3 [G, N, K] with the scales of 128 rows x 4 groups of 32 in one
    512-byte tile, row r and group c at byte 16 (r % 32) + 4 (r // 32) + c."""
    if not mx:
        return _randn(g, shape, STD)
    G, K, N = shape
    q, s = _mx(_randn(g, (G, N, K), STD).float())
    nb, kb = -(-N // 128), -(-K // 128)
    tile = torch.zeros((G, nb * 128, kb * 4), dtype=torch.uint8, device="cuda")
    tile[:, :N, : K // 32] = s.view(torch.uint8)
    tile = tile.view(G, nb, 4, 32, kb, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(torch.float8_e8m0fnu)
    return q, tile


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, D = case["T"], case["D"]
    st = dict(case)
    if case["op"] == "norm":
        st["x"] = _randn(g, (T, D), 1.0)
        st["residual"] = _randn(g, (T, D), 2.0)
        st["gamma"] = (1.0 + _randn(g, (D,), 0.1).float()).bfloat16()
        st["gamma_post"] = (1.0 + _randn(g, (D,), 0.1).float()).bfloat16() if case["post"] else None
        st["sum"], st["y"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        if case["quant"]:
            st["q"] = torch.empty((T, D), dtype=torch.float8_e4m3fn, device="cuda")
            st["scale"] = torch.empty((T, D // 32), dtype=torch.float8_e8m0fnu, device="cuda")
        return st
    mx = case["op"] == "mx"
    E, F, S, k = case["E"], case["F"], case["S"], case["k"]
    st["w_router"] = _randn(g, (D, E), STD)
    for name, shape in (("wg", (E, D, F)), ("wu", (E, D, F)), ("wd", (E, F, D)), ("sg", (1, D, S)), ("su", (1, D, S)),
                        ("sd", (1, S, D))):
        st[name] = _weight(g, shape, mx)
    st["bias"] = torch.randn(E, generator=g, device="cuda") * 0.5 if case["bias"] else None
    st["gamma_pre"] = st["gamma_post"] = None
    if case.get("sandwich"):
        st["gamma_pre"], st["gamma_post"] = ((1.0 + _randn(g, (D,), 0.1).float()).bfloat16() for _ in range(2))
    # Twice the rows, of which the first T stay whose k-th and next logit lie apart: nearer than the rounding of a
    # 32-bit sum (or of a normalised row to bf16) the order of the sum decides which expert such a row takes.
    x = _randn(g, (2 * T + 16, D), 1.0)
    if k < E:
        r = x.double()
        if st["gamma_pre"] is not None:
            r = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * st["gamma_pre"].double()
        logits = r @ st["w_router"].double() + (0.0 if st["bias"] is None else st["bias"].double())
        top = logits.topk(k + 1, dim=-1).values
        gap = top[:, k - 1] - top[:, k]
        x = x[torch.argsort((gap < 5e-4).int(), stable=True)]
    st["x"] = x[:T].contiguous()
    st["out"] = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    if case.get("fed"):
        st["xq"], st["xs"] = _mx(st["x"].float())
    st["held"] = {}  # what a user's program keeps beside its weights: their handle and a workspace
    return st


# ------------------------------------------------------------ the plain forms


def _mx(v):
    """MXFP8 of the last dimension of v: (e4m3 values, power-of-two scales)."""
    b = v.unflatten(-1, (v.shape[-1] // 32, 32))
    m, e = torch.frexp(b.abs().amax(-1))
    j = (e - 9 + (m > 0.875).int()).clamp(-127, 127)
    j = torch.where(m == 0, -127, j)
    q = torch.ldexp(b, -j.unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)
    return q, (j + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _value(q, s):
    return (q.float().unflatten(-1, (s.shape[-1], 32)) * s.float().unsqueeze(-1)).flatten(-2)


def _plain_weight(w, rows=None):
    """fp32 [G, K, N] of a bf16 or MXFP8 weight, of the given groups."""
    if not isinstance(w, tuple):
        return (w if rows is None else w[rows]).float()
    q, tile = w
    if rows is not None:
        q, tile = q[rows], tile.view(torch.uint8)[rows].view(torch.float8_e8m0fnu)
    G, N, K = q.shape
    s = tile.view(torch.uint8).permute(0, 1, 4, 3, 2, 5).reshape(G, tile.shape[1] * 128, -1)[:, :N, : K // 32]
    return _value(q, s.contiguous().view(torch.float8_e8m0fnu)).transpose(1, 2)


def _rms(x, gamma):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()


def _gelu(z):
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _plain_norm(st):
    x = st["x"].float()
    s = st["residual"].float() + (x if st["gamma_post"] is None else _rms(x, st["gamma_post"]))
    y = _rms(s, st["gamma"])
    out = dict(sum=s.bfloat16(), y=y.bfloat16())
    if st["quant"]:
        out["q"], out["scale"] = _mx(y)
    return out


def _route(st, x):
    logits = x.double() @ st["w_router"].double()
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    val, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
    k = st["k"]
    return idx[:, :k], torch.softmax(val[:, :k], -1).float()


def _ffn(x, wg, wu, wd, mx):
    h = _gelu(x @ wg) * (x @ wu)
    return (_value(*_mx(h)) if mx else h) @ wd


def _plain_layer(st):
    mx = st["op"] == "mx"
    raw = st["x"].float()
    x = raw if st["gamma_pre"] is None else _rms(raw, st["gamma_pre"]).bfloat16().float()
    idx, w = _route(st, x)
    if mx:
        x = _value(st["xq"], st["xs"]) if st["fed"] else _value(*_mx(x))
    out = _ffn(x.unsqueeze(0), *(_plain_weight(st[n]) for n in ("sg", "su", "sd")), mx)[0]
    T, k = idx.shape
    if T * k <= st["E"]:  # few rows: the experts of each row
        e = idx.reshape(-1)
        y = _ffn(x.repeat_interleave(k, 0).unsqueeze(1), *(_plain_weight(st[n], e) for n in ("wg", "wu", "wd")), mx)
        y = y.view(T, k, -1)
    else:  # many: each expert's rows together
        e, order = torch.sort(idx.reshape(-1), stable=True)
        count = torch.bincount(e, minlength=st["E"])
        at = torch.arange(T * k, device=e.device) - (count.cumsum(0) - count)[e]
        rows = x.new_zeros((st["E"], int(count.max()), x.shape[1]))
        rows[e, at] = x[order // k]
        y = _ffn(rows, *(_plain_weight(st[n]) for n in ("wg", "wu", "wd")), mx)[e, at]
        y = torch.empty_like(y).index_copy_(0, order, y).view(T, k, -1)
    out = out + (w.unsqueeze(-1) * y).sum(1)
    if st["gamma_post"] is not None:
        out = raw + _rms(out, st["gamma_post"])
    return out.bfloat16()


# ---------------------------------------------------------- the library's calls


def _own_layer(st):
    from mixture_experts_transformer_b200 import block
    from mixture_experts_transformer_b200.inputs import Dims

    held = st["held"]
    if not held:
        dims = Dims(st["D"], st["E"], st["F"], st["S"])
        names = ("wg", "wu", "wd", "sg", "su", "sd")
        if st["op"] == "few":
            held["w"] = block.DeviceWeights(dims, st["w_router"], *(st[n] if n[0] == "w" else st[n][0] for n in names))
            held["ws"] = block.few_workspace(held["w"], st["T"], st["k"])
        else:
            lin = [block.Mxfp8Linear(*st[n], st[n][0].shape[0], st[n][0].shape[2], st[n][0].shape[1]) for n in names]
            held["w"] = block.Mxfp8Weights(dims, st["w_router"], *lin)
            held["ws"] = block.mxfp8_workspace(held["w"], st["T"], st["k"])
    if st["op"] == "few":
        return block.forward_few(held["w"], st["x"], top_k=st["k"], router_bias=st["bias"], workspace=held["ws"],
                                 out=st["out"], norm_pre=st["gamma_pre"], norm_post=st["gamma_post"],
                                 residual=st["sandwich"]).out
    return block.forward_mxfp8(held["w"], st["x"], xq=st.get("xq"), xs=st.get("xs"), top_k=st["k"],
                               router_bias=st["bias"], workspace=held["ws"], out=st["out"]).out


def run(state):
    if state["op"] == "norm":
        if own:
            from mixture_experts_transformer_b200 import block

            r = block.add_rms_norm(state["x"], state["gamma"], residual=state["residual"],
                                   gamma_post=state["gamma_post"], y=state["y"], sum_out=state["sum"],
                                   q=state.get("q"), scale=state.get("scale"))
            out = dict(sum=r.sum, y=r.y)
            if state["quant"]:
                out["q"], out["scale"] = r.q, r.scale
            return out
        return _plain_norm(state)
    if own:
        return _own_layer(state)
    return _plain_layer(state)


# ------------------------------------------------------------------- work


def work(case):
    T, D = case["T"], case["D"]
    if case["op"] == "norm":
        b = T * D * 2 * 4 + D * 2 * (2 if case["post"] else 1) + (T * D + T * D // 32 if case["quant"] else 0)
        return dict(bytes=b, flops=T * D * (12 if case["post"] else 8))
    E, F, S, k = case["E"], case["F"], case["S"], case["k"]
    touched = E * (1.0 - (1.0 - k / E) ** T)
    per = (1.0 + 1.0 / 32) if case["op"] == "mx" else 2.0
    b = (touched * 3 * D * F + 3 * D * S) * per + D * E * 2 + T * D * 4
    return dict(bytes=b, flops=2.0 * T * (D * E + 3 * D * (k * F + S)))


# ------------------------------------------------------------- in 64 bits


def _exact_round(v):
    """v rounded to e4m3 (nearest, ties to even), for |v| <= 448."""
    ex = torch.frexp(v)[1] - 1
    step = torch.pow(2.0, (ex.clamp(min=-6) - 3).double())
    return torch.round(v / step) * step


def _exact_mx(v):
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    j = torch.ceil(torch.log2(top / 448.0)).clamp(-127, 127)
    j = torch.where(top > 448.0 * torch.pow(2.0, j), j + 1, j)
    j = torch.where(448.0 * torch.pow(2.0, j - 1) >= top, j - 1, j).clamp(-127, 127)
    scale = torch.pow(2.0, j)
    return _exact_round(b / scale).reshape(v.shape), scale.squeeze(-1)


def _exact_norm(x, gamma):
    return gamma.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _exact_weight(w, e):
    if not isinstance(w, tuple):
        return w[e].double()
    q, tile = w[0][e].double(), w[1][e].float().double()
    N, K = q.shape
    n, c = torch.arange(N, device=q.device)[:, None], torch.arange(K // 32, device=q.device)[None, :]
    s = tile[n // 128, c // 4, n % 32, n % 128 // 32, c % 4]
    return (q * s.repeat_interleave(32, 1)).T


def _exact_ffn(st, names, e, x):
    g, u, d = (_exact_weight(st[n], e) for n in names)
    z = x @ g
    h = z / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3))) * (x @ u)
    if st["op"] == "mx":
        q, s = _exact_mx(h)
        h = q * s.repeat_interleave(32, -1)
    return h @ d


def exact(case, seed):
    st = prepare(case, seed)
    x = st["x"].double()
    if st["op"] == "norm":
        s = st["residual"].double() + (_exact_norm(x, st["gamma_post"]) if case["post"] else x)
        y = _exact_norm(s, st["gamma"])
        out = dict(sum=s, y=y)
        if case["quant"]:
            out["q"], out["scale"] = _exact_mx(y)
        return out
    xin = x if st["gamma_pre"] is None else _exact_norm(x, st["gamma_pre"]).bfloat16().double()
    logits = xin @ st["w_router"].double() + (0 if st["bias"] is None else st["bias"].double())
    val, idx = logits.topk(st["k"], dim=-1)
    w = torch.exp(val - val[:, :1])
    w = w / w.sum(-1, keepdim=True)
    if st["op"] == "mx":
        q, s = (st["xq"].double(), st["xs"].float().double()) if st["fed"] else _exact_mx(xin)
        xin = q * s.repeat_interleave(32, -1)
    out = _exact_ffn(st, ("sg", "su", "sd"), 0, xin)
    for e in range(st["E"]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            out[t] += w[t, j][:, None] * _exact_ffn(st, ("wg", "wu", "wd"), e, xin[t])
    return out if st["gamma_post"] is None else x + _exact_norm(out, st["gamma_post"])
