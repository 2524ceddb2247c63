"""Cases that measure the operators around and inside one MoE block.

Three families, each in the form a block of a model calls them:

* the norms before and after the block, fused with the combine, the gate and the
  residual add, and their gradients;
* 8-bit checkpoints of the block's activations and their use in the backward pass;
* the SwiGLU experts on 4-bit weights with group scales, for few tokens (decoding).

``run`` computes a case either with the package's operators (``own``) or in plain
form: elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # decoding one token at the drafter's hidden size: pure latency
        dict(name="norm_in_one_token", op="norm_in", T=1, d=4096),
        # the drafter workload's batch: a training or prefill pass at HBM speed
        dict(name="norm_in_drafter", op="norm_in", T=32768, d=4096),
        # end of the block for a decoding batch: combine of 8 experts, norm, residual
        dict(name="norm_out_decode", op="norm_out", T=16, d=2048, E=128, K=8, shared=False,
             gain=True, gate="none"),
        # end of the block in training, with a learned gate per channel (qwen3 shape)
        dict(name="norm_out_qwen3", op="norm_out", T=8192, d=2048, E=128, K=8, shared=False,
             gain=True, gate="channel"),
        # gradient of the norm before the block joined with the residual's gradient
        dict(name="norm_in_backward_drafter", op="norm_in_backward", T=32768, d=4096),
        # gradient of the norm after the block at sizes off every tile, one gate vector per
        # sequence of 1000 tokens (adaptive norms), the last sequence cut short
        dict(name="norm_out_backward_ragged", op="norm_out_backward", T=16383, d=2056,
             gain=True, gate="sequence", span=1000),
        # token rows kept in 8 bits and dispatched again in the backward (dsv2lite shape)
        dict(name="ckpt8_rows_dsv2lite", op="ckpt8_rows", T=16384, d=2048, E=64, K=6),
        # gate and up projections kept in 8 bits, H made again from them (qwen3 shape)
        dict(name="ckpt8_swiglu_qwen3", op="ckpt8_swiglu", M=65536, I=768),
        # the combine's gradient from expert outputs kept in 8 bits, an odd number of tokens
        dict(name="ckpt8_combine_backward_odd", op="ckpt8_combine_backward", T=8191, d=2048,
             E=128, K=8),
        # decoding one token (qwen3 shape): 8 of 128 experts are read
        dict(name="w4_one_token_qwen3", op="w4_ffn", T=1, d=2048, E=128, K=8, I=768, group=128),
        # a small decoding batch (dsv2lite shape), finer groups
        dict(name="w4_batch16_dsv2lite", op="w4_ffn", T=16, d=2048, E=64, K=6, I=1408, group=64),
        # a full decoding batch (qwen3 shape): nearly every expert is read for a few rows
        dict(name="w4_batch64_qwen3", op="w4_ffn", T=64, d=2048, E=128, K=8, I=768, group=32),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _routing_sizes(rng, most_e):
    E = _spread(rng, 4, most_e)
    return E, rng.randint(1, min(8, E))


def _drawn(rng):
    op = rng.choice(["norm_in", "norm_out", "norm_in_backward", "norm_out_backward", "ckpt8_rows",
                     "ckpt8_swiglu", "ckpt8_combine_backward", "w4_ffn", "w4_ffn"])
    if op == "norm_in":
        return dict(op=op, T=_spread(rng, 1, 32768), d=8 * _spread(rng, 16, 1024))
    if op == "norm_in_backward":
        return dict(op=op, T=_spread(rng, 64, 32768), d=8 * _spread(rng, 16, 1024))
    if op == "norm_out":
        E, K = _routing_sizes(rng, 128)
        return dict(op=op, T=_spread(rng, 1, 16384), d=8 * _spread(rng, 16, 512), E=E, K=K,
                    shared=rng.random() < 0.5, gain=rng.random() < 0.75,
                    gate=rng.choice(["none", "token", "channel", "sequence"]))
    if op == "norm_out_backward":
        T = _spread(rng, 64, 32768)
        gate = rng.choice(["none", "token", "channel", "sequence"])
        return dict(op=op, T=T, d=8 * _spread(rng, 16, 512), gain=rng.random() < 0.75, gate=gate,
                    span=_spread(rng, 1, T))
    if op == "ckpt8_swiglu":
        return dict(op=op, M=_spread(rng, 128, 65536), I=8 * _spread(rng, 16, 256))
    if op in ("ckpt8_rows", "ckpt8_combine_backward"):
        E, K = _routing_sizes(rng, 128)
        return dict(op=op, T=_spread(rng, 64, 16384), d=8 * _spread(rng, 16, 512), E=E, K=K)
    E, K = _routing_sizes(rng, 128)
    return dict(op=op, T=_spread(rng, 1, 64), d=128 * _spread(rng, 2, 32), E=E, K=K,
                I=128 * _spread(rng, 2, 16), group=rng.choice([32, 64, 128]))


def draw(rng):
    cost = lambda c: work(c)["bytes"] / 6.8e12 + work(c)["flops"] / 1.8e15   # noqa: E731
    most = {op: max(cost(c) for c in listed() if c["op"] == op) for op in {c["op"] for c in listed()}}
    while True:
        case = _drawn(rng)
        if cost(case) <= most[case["op"]]:
            return case


def _gate_shape(case):
    """(rows, columns, tokens per row) of the gate, or None."""
    T, d, kind = case["T"], case["d"], case["gate"]
    if kind == "none":
        return None
    if kind == "token":
        return T, 1, 1
    if kind == "channel":
        return 1, d, T
    span = case.get("span", max(1, (T + 3) // 4))
    return -(-T // span), d, span


def work(case):
    op = case["op"]
    if op == "w4_ffn":
        T, d, E, K, I, g = (case[k] for k in ("T", "d", "E", "K", "I", "group"))
        active = E * (1.0 - (1.0 - K / E) ** T)   # experts with a row, on average
        weights = active * 3 * d * I * (0.5 + 2.0 / g)
        return {"bytes": int(weights + 2 * T * d + T * K * (2 * I + 2 * d)),
                "flops": 6 * T * K * d * I}
    if op == "ckpt8_swiglu":
        n = case["M"] * 2 * case["I"]
        # read to be packed, kept and read again, written restored with H
        return {"bytes": int(2 * n + 2 * n * 17 / 16 + 2 * n + n), "flops": 12 * n}
    T, d = case["T"], case["d"]
    n = T * d
    if op == "norm_in":
        return {"bytes": 4 * n + 4 * d + 4 * T, "flops": 5 * n}
    if op == "norm_in_backward":
        return {"bytes": 8 * n + 8 * d + 4 * T, "flops": 12 * n}
    gate = _gate_shape(case) if "gate" in case else None
    gate_bytes = 4 * gate[0] * gate[1] if gate else 0
    if op == "norm_out":
        K = case["K"]
        return {"bytes": 2 * n * (K + 3 + case["shared"]) + 8 * T * K + 4 * T + 4 * d + gate_bytes,
                "flops": n * (2 * K + 8)}
    if op == "norm_out_backward":
        return {"bytes": 6 * n + 8 * d + 4 * T + 2 * gate_bytes, "flops": 14 * n}
    K = case["K"]
    if op == "ckpt8_rows":
        return {"bytes": int(2 * n + 2 * n * 17 / 16 + 2 * n * K + 4 * T * K), "flops": 4 * n}
    return {"bytes": int(2 * n + n * K * 17 / 16 + 2 * n * K + 12 * T * K), "flops": 4 * n * K}


# ---------------------------------------------------------------- inputs
def _stream(g, T, d):
    """A residual stream: most channels of unit size, a few percent twenty times that."""
    x = torch.randn(T, d, generator=g, device="cuda")
    wide = torch.rand(d, generator=g, device="cuda") < 0.02
    return (x * torch.where(wide, 20.0, 1.0)).to(torch.bfloat16)


def _bf(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _routing(g, T, E, K):
    """Expert-major order of a router's top-k: (weights [T, K], perm, inv_perm, offsets)."""
    logits = torch.randn(T, E, generator=g, device="cuda")
    top, idx = torch.topk(logits, K, dim=1)
    w = torch.softmax(top, dim=1)
    flat = idx.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * K, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    return w, perm.to(torch.int32), inv.to(torch.int32), offsets.to(torch.int32)


def _codes4(g, E, N, K, group):
    """A 4-bit checkpoint: codes [E, N, K/2] (even k in the low half), scales [E, N, K/group]."""
    q = torch.randn(E, N, K, generator=g, device="cuda", dtype=torch.float16).mul_(2.6).round_()
    q = q.clamp_(-8, 7).add_(8).to(torch.uint8)
    codes = q[..., 0::2] | (q[..., 1::2] << 4)
    s = (0.005 + 0.006 * torch.rand(E, N, K // group, generator=g, device="cuda"))
    return codes.contiguous(), s.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    op, s = case["op"], {"case": case}
    if op == "w4_ffn":
        T, d, E, K, I, group = (case[k] for k in ("T", "d", "E", "K", "I", "group"))
        _, s["perm"], _, s["offsets"] = _routing(g, T, E, K)
        s["x"] = _bf(g, T, d)
        gate, up = _codes4(g, E, I, d, group), _codes4(g, E, I, d, group)
        down = _codes4(g, E, d, I, group)
        if own:   # a serving program lays its weights out once
            from grouped_gemm_moe_gb300 import binding as B
            s["wgu"] = B.moe_w4_pack_weights(*gate, *up)
            s["wd"] = B.moe_w4_pack_weights(*down)
            s["ws"] = B.new_workspace(B.workspace_size(B.MOE_OP_GROUPED_FFN_W4, T, E, K, 1, d, I),
                                      s["x"].device)
            s["out"] = (torch.empty(T * K, d, dtype=torch.bfloat16, device="cuda"),
                        torch.empty(T * K, I, dtype=torch.bfloat16, device="cuda"))
        else:
            s.update(gate=gate, up=up, down=down)
            # rows of the fullest expert, which a plain program needs to pad its segments
            s["cap"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        return s
    if op == "ckpt8_swiglu":
        s["gu"] = _bf(g, case["M"], 2 * case["I"], scale=1.3)
        return s
    T, d = case["T"], case["d"]
    if op == "norm_in":
        s["x"] = _stream(g, T, d)
        s["gain"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        return s
    if op == "norm_in_backward":
        s["x"] = _stream(g, T, d)
        s["gain"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
        s["dxn"], s["dres"] = _bf(g, T, d), _bf(g, T, d)
        if own:
            from grouped_gemm_moe_gb300 import binding as B
            s["ws"] = B.new_workspace(B.workspace_size(B.MOE_OP_NORM_BACKWARD, T, 1, 1, 1, d),
                                      s["x"].device)
        return s
    if op in ("norm_out", "norm_out_backward"):
        gate = _gate_shape(case)
        s["gate"] = s["span"] = None
        if gate:
            s["gate"] = 0.5 + 0.3 * torch.randn(gate[0], gate[1], generator=g, device="cuda")
            s["span"] = gate[2]
        s["gain"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda") if case["gain"] else None
        s["scale"] = 0.7
        if op == "norm_out":
            s["w"], _, s["inv_perm"], _ = _routing(g, T, case["E"], case["K"])
            s["y"] = _bf(g, T * case["K"], d, scale=0.4)
            s["shared"] = _bf(g, T, d, scale=0.4) if case["shared"] else None
            s["resid"] = _stream(g, T, d)
        else:
            s["dout"], s["z"] = _bf(g, T, d), _bf(g, T, d, scale=0.4)
            s["rstd"] = torch.rsqrt(s["z"].float().square().mean(1) + EPS)
            if own:
                from grouped_gemm_moe_gb300 import binding as B
                s["ws"] = B.new_workspace(
                    B.workspace_size(B.MOE_OP_NORM_BACKWARD, T, 1, 1, 1, d), s["z"].device)
        return s
    s["w"], _, s["inv_perm"], _ = _routing(g, T, case["E"], case["K"])
    if op == "ckpt8_rows":
        s["x"] = _stream(g, T, d)
    else:
        s["dout"] = _bf(g, T, d)
        s["q"], s["s"] = _pack8(_bf(g, T * case["K"], d, scale=0.4))
    return s


# ---------------------------------------------------------------- plain forms
def _pack8(x):
    """int8 codes and one bf16 scale per 32 elements of a row (the last block may be shorter)."""
    M, N = x.shape
    blocks = -(-N // 32)
    v = torch.zeros(M, blocks * 32, device=x.device)
    v[:, :N] = x.float()
    v = v.view(M, blocks, 32)
    fine = v.abs() < math.inf
    top = torch.where(fine, v.abs(), torch.zeros_like(v)).amax(2) / 127.0
    top = torch.clamp(top, min=2.0 ** -110)
    s = ((top.view(torch.int32) + 0xffff) >> 16 << 16).view(torch.float32)   # bf16, rounded up
    q = torch.where(fine, torch.round(v * (1.0 / s)[:, :, None]), torch.full_like(v, -128.0))
    return q.view(M, -1)[:, :N].to(torch.int8).contiguous(), s.to(torch.bfloat16)


def _unpack8(q, s):
    M, N = q.shape
    v = q.float() * torch.repeat_interleave(s.float(), 32, dim=1)[:, :N]
    return torch.where(q == -128, torch.full_like(v, math.nan), v)


def _unpack4(codes, s):
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float() - 8.0
    return (q.unflatten(-1, (s.shape[-1], -1)) * s.float()[..., None]).flatten(-2)


def _gate_rows(s, T):
    """The gate for each token: [T, 1], [T, d] or 1."""
    if s["gate"] is None:
        return 1.0
    return s["gate"][torch.arange(T, device=s["gate"].device) // s["span"]]


def _plain(s):
    case = s["case"]
    op = case["op"]
    bf = torch.bfloat16
    if op == "norm_in":
        x = s["x"].float()
        r = torch.rsqrt((x * x).mean(1) + EPS)
        return {"xn": (x * r[:, None] * s["gain"]).to(bf), "rstd": r}
    if op == "norm_in_backward":
        x, r = s["x"].float(), s["rstd"][:, None]
        dxn = s["dxn"].float()
        xh = x * r
        u = dxn * s["gain"]
        dx = s["dres"].float() + r * (u - xh * (u * xh).mean(1, keepdim=True))
        return {"dx": dx.to(bf), "dgain": (dxn * xh).sum(0)}
    if op == "norm_out":
        T, K = case["T"], case["K"]
        z = (s["y"][s["inv_perm"].view(T, K).long()].float() * s["w"][:, :, None]).sum(1)
        if s["shared"] is not None:
            z = z + s["shared"].float()
        out, r = z, None
        if s["gain"] is not None:
            r = torch.rsqrt((z * z).mean(1) + EPS)
            out = z * r[:, None] * s["gain"]
        out = s["resid"].float() + s["scale"] * _gate_rows(s, T) * out
        return {"out": out.to(bf), "z": z.to(bf), "rstd": r}
    if op == "norm_out_backward":
        T, d = case["T"], case["d"]
        dout, z = s["dout"].float(), s["z"].float()
        dn = s["scale"] * _gate_rows(s, T) * dout
        dgain = dgate = None
        n, dz = z, dn
        if s["gain"] is not None:
            r = s["rstd"][:, None]
            zh = z * r
            u = dn * s["gain"]
            dz = r * (u - zh * (u * zh).mean(1, keepdim=True))
            dgain = (dn * zh).sum(0)
            n = zh * s["gain"]
        if s["gate"] is not None:
            rows, cols = s["gate"].shape
            t = s["scale"] * dout * n
            if cols == 1:
                t = t.sum(1, keepdim=True)
            full = torch.zeros(rows * s["span"], cols, device=t.device)
            full[:T] = t
            dgate = full.view(rows, s["span"], cols).sum(1)
        return {"dz": dz.to(bf), "dgain": dgain, "dgate": dgate}
    if op == "ckpt8_rows":
        T, K = case["T"], case["K"]
        v = _unpack8(*_pack8(s["x"])).to(bf)
        xp = torch.empty(T * K, case["d"], dtype=bf, device=v.device)
        xp[s["inv_perm"].long()] = v[torch.arange(T * K, device=v.device) // K]
        return {"xp": xp}
    if op == "ckpt8_swiglu":
        v = _unpack8(*_pack8(s["gu"]))
        G, U = v[:, :case["I"]], v[:, case["I"]:]
        return {"gu": v.to(bf), "h": (G / (1.0 + torch.exp(-G)) * U).to(bf)}
    if op == "ckpt8_combine_backward":
        T, K = case["T"], case["K"]
        y = _unpack8(s["q"], s["s"])
        at = s["inv_perm"].view(T, K).long()
        dout = s["dout"].float()[:, None, :]
        dw = (dout * y[at]).sum(2)
        dy = torch.empty(T * K, case["d"], dtype=bf, device=y.device)
        dy[at] = (dout * s["w"][:, :, None]).to(bf)
        return {"dy": dy, "dtopk_w": dw}
    # 4-bit experts: the rows' own experts gathered, or segments padded to the fullest one
    M, E, cap = case["T"] * case["K"], case["E"], s["cap"]
    row = torch.arange(M, device=s["x"].device)
    e = (row[:, None] >= s["offsets"][None, 1:]).sum(1)
    xp = s["x"][s["perm"].long() // case["K"]].float()
    if M <= E:
        at, slot, span = e, torch.zeros_like(row), 1
        pick = lambda w: _unpack4(w[0][at], w[1][at])   # noqa: E731
        lead, slot = row, slot
    else:
        span = cap
        pick = lambda w: _unpack4(*w)   # noqa: E731
        lead, slot = e, row - s["offsets"][e]
    xs = torch.zeros(M if M <= E else E, span, case["d"], device=xp.device)
    xs[lead, slot] = xp
    G = torch.bmm(xs, pick(s["gate"]).transpose(1, 2))
    U = torch.bmm(xs, pick(s["up"]).transpose(1, 2))
    h = G / (1.0 + torch.exp(-G)) * U
    y = torch.bmm(h, pick(s["down"]).transpose(1, 2))
    return {"y": y[lead, slot].to(bf), "h": h[lead, slot].to(bf)}


# ---------------------------------------------------------------- the package's operators
def _own(s):
    from grouped_gemm_moe_gb300 import binding as B
    case = s["case"]
    op = case["op"]
    if op == "norm_in":
        xn, r = B.moe_norm_in(s["x"], s["gain"], EPS)
        return {"xn": xn, "rstd": r}
    if op == "norm_in_backward":
        dx, dgain = B.moe_norm_in_backward(s["dxn"], s["x"], s["gain"], s["rstd"], dres=s["dres"],
                                           ws=s["ws"])
        return {"dx": dx, "dgain": dgain}
    if op == "norm_out":
        out, z, r = B.moe_norm_out(s["y"], s["resid"], s["gain"], topk_w=s["w"],
                                   inv_perm=s["inv_perm"], shared_y=s["shared"], gate=s["gate"],
                                   span=s["span"], scale=s["scale"], eps=EPS)
        return {"out": out, "z": z, "rstd": r}
    if op == "norm_out_backward":
        dz, dgain, dgate = B.moe_norm_out_backward(s["dout"], s["z"], s["rstd"], s["gain"],
                                                   gate=s["gate"], span=s["span"],
                                                   scale=s["scale"], ws=s["ws"])
        return {"dz": dz, "dgain": dgain, "dgate": dgate}
    if op == "ckpt8_rows":
        return {"xp": B.moe_ckpt8_dispatch(*B.moe_ckpt8_pack(s["x"]), s["inv_perm"], case["K"])}
    if op == "ckpt8_swiglu":
        gu, h = B.moe_ckpt8_swiglu(*B.moe_ckpt8_pack(s["gu"]))
        return {"gu": gu, "h": h}
    if op == "ckpt8_combine_backward":
        dy, dw = B.moe_ckpt8_combine_backward(s["dout"], s["q"], s["s"], s["w"], s["inv_perm"])
        return {"dy": dy, "dtopk_w": dw}
    y, h = B.moe_grouped_ffn_w4(s["x"], s["offsets"], s["wgu"], s["wd"], perm=s["perm"],
                                K=case["K"], ws=s["ws"], out=s["out"])
    return {"y": y, "h": h}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _restored8(x):
    """The values an 8-bit checkpoint of x stands for, from the definition, in 64 bits."""
    x = x.double()
    out = torch.empty_like(x)
    N = x.shape[1]
    for c in range(0, N, 32):
        b = x[:, c:c + 32]
        top = (b.abs().amax(1, keepdim=True) / 127).clamp(min=2.0 ** -110)
        unit = torch.exp2(torch.floor(torch.log2(top)) - 7)   # spacing of bf16 at the scale
        s = torch.ceil(top / unit) * unit
        out[:, c:c + 32] = torch.round(b / s) * s
    return out


def _weights4(w, e):
    codes, s = w[0][e], w[1][e].double()
    N, half = codes.shape
    q = torch.empty(N, 2 * half, dtype=torch.float64, device=codes.device)
    q[:, 0::2] = (codes % 16).double()
    q[:, 1::2] = (codes // 16).double()
    return (q - 8) * s.repeat_interleave(2 * half // s.shape[1], dim=1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    f = lambda k: s[k].double()   # noqa: E731
    if op == "norm_in":
        x = f("x")
        norm = torch.sqrt(x.pow(2).sum(1) / case["d"] + EPS)
        return {"xn": x / norm[:, None] * f("gain"), "rstd": 1 / norm}
    if op == "norm_in_backward":
        x, v, r = f("x"), f("dxn"), f("rstd")[:, None]
        dg = (v * x * r).sum(0)
        v = v * f("gain")
        dot = (v * x).sum(1, keepdim=True)
        return {"dx": f("dres") + r * v - x * (r ** 3 * dot / case["d"]), "dgain": dg}
    if op in ("norm_out", "norm_out_backward"):
        T, d = case["T"], case["d"]
        gate = torch.ones(T, 1, dtype=torch.float64, device="cuda")
        if s["gate"] is not None:
            gate = f("gate").repeat_interleave(s["span"], dim=0)[:T]
        gain = f("gain") if s["gain"] is not None else None
        if op == "norm_out":
            z = f("shared") if s["shared"] is not None else 0.0
            at = s["inv_perm"].view(T, case["K"]).long()
            for j in range(case["K"]):
                z = z + f("w")[:, j:j + 1] * s["y"][at[:, j]].double()
            n, r = z, None
            if gain is not None:
                r = 1 / torch.sqrt(z.pow(2).sum(1) / d + EPS)
                n = z * gain * r[:, None]
            return {"out": f("resid") + s["scale"] * gate * n, "z": z, "rstd": r}
        dout, z = f("dout") * s["scale"], f("z")
        dgain = dgate = None
        v = dout * gate
        n, dz = z, v
        if gain is not None:
            r = f("rstd")[:, None]
            dgain = (v * z * r).sum(0)
            n = z * r * gain
            v = v * gain
            dz = r * v - z * (r ** 3 * (v * z).sum(1, keepdim=True) / d)
        if s["gate"] is not None:
            rows, cols = s["gate"].shape
            t = dout * n
            t = t.sum(1, keepdim=True) if cols == 1 else t
            at = torch.arange(T, device="cuda") // s["span"]
            if rows == T:
                dgate = t
            elif rows == 1:
                dgate = t.sum(0, keepdim=True)
            else:
                dgate = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
                dgate.index_add_(0, at, t)
        return {"dz": dz, "dgain": dgain, "dgate": dgate}
    if op == "ckpt8_rows":
        v = _restored8(s["x"])
        at = torch.argsort(s["inv_perm"].long()) // case["K"]
        return {"xp": v[at]}
    if op == "ckpt8_swiglu":
        v = _restored8(s["gu"])
        G, U = v[:, :case["I"]], v[:, case["I"]:]
        return {"gu": v, "h": G * torch.sigmoid(G) * U}
    if op == "ckpt8_combine_backward":
        T, K, d = case["T"], case["K"], case["d"]
        at = s["inv_perm"].view(T, K).long()
        dy = torch.empty(T * K, d, dtype=torch.float64, device="cuda")
        dw = torch.empty(T, K, dtype=torch.float64, device="cuda")
        for j in range(K):
            scale = s["s"][at[:, j]].double().repeat_interleave(32, dim=1)[:, :d]
            dw[:, j] = (f("dout") * s["q"][at[:, j]].double() * scale).sum(1)
            dy[at[:, j]] = f("dout") * f("w")[:, j:j + 1]
        return {"dy": dy, "dtopk_w": dw}
    ends = s["offsets"].tolist()
    M = case["T"] * case["K"]
    y = torch.zeros(M, case["d"], dtype=torch.float64, device="cuda")
    h = torch.zeros(M, case["I"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if a < b:
            x = s["x"][s["perm"][a:b].long() // case["K"]].double()
            G, U = x @ _weights4(s["gate"], e).T, x @ _weights4(s["up"], e).T
            h[a:b] = G * torch.sigmoid(G) * U
            y[a:b] = h[a:b] @ _weights4(s["down"], e).T
    return {"y": y, "h": h}
