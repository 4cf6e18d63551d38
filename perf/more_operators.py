"""Cases of the operators on both sides of an expert: the norm before a block with its output in 8
bits, the gated projection of a shared expert with its gradients, and products with 4-bit weights.

``listed`` and ``draw`` give cases, ``prepare`` makes a case's inputs and output buffers on the GPU,
``run`` makes one pass: with ``own`` set through the library's entry points, else in a plain form of
elementary tensor operations in 32 bits.  ``exact`` restates each operator in 64 bits.

Sizes: hidden sizes 4096, 7168 and 2048, intermediate sizes 2048 and 14336, 256 experts, top-k 8 and
the token counts 64 and 8192 are those of the expert-layer workloads in
``moe_expert_layer_prepare_gb300/synthetic.py``.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
_binding = None


def _B():
    global _binding
    if _binding is None:
        from moe_expert_layer_prepare_gb300 import binding
        _binding = binding
    return _binding


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One token between two blocks: its residual sum, the norm, and the norm's 8-bit form for
        # the experts beside the 16-bit one for the router.
        dict(name="norm_single_token", op="norm", T=1, K=7168, dtype="bf16", wdtype="bf16",
             sf="ue8m0", z=True, y=True),
        # Prefill of the same.
        dict(name="norm_prefill", op="norm", T=8192, K=7168, dtype="bf16", wdtype="bf16",
             sf="ue8m0", z=True, y=True),
        # An odd number of tokens whose norm is wanted in 8 bits alone, with fp32 scales and fp32
        # norm weights.
        dict(name="norm_odd_fp32_scales", op="norm", T=2051, K=4096, dtype="fp16", wdtype="fp32",
             sf="fp32", z=True, y=False),
        # One token through a shared expert's gate and up projections.
        dict(name="gated_single_token", op="gated", T=1, K=7168, N=2048, dtype="bf16", act="silu",
             train=False),
        # A decode batch through a wide feed-forward block.
        dict(name="gated_decode", op="gated", T=64, K=4096, N=14336, dtype="bf16", act="silu",
             train=False),
        # Prefill through a shared expert.
        dict(name="gated_prefill", op="gated", T=8192, K=7168, N=2048, dtype="bf16", act="silu",
             train=False),
        # A training step: forward, then the gradients of tokens and weights.
        dict(name="gated_train", op="gated", T=4096, K=7168, N=2048, dtype="bf16", act="silu",
             train=True),
        # The same at sizes that fill no tile, in fp16, with the other activation.
        dict(name="gated_train_odd", op="gated", T=1031, K=2056, N=1403, dtype="fp16",
             act="gelu_tanh", train=True),
        # One token through one matrix of 4-bit integers.
        dict(name="w4_single_token", op="w4", T=1, k=0, E=0, K=7168, N=4096, dtype="bf16",
             fmt="int4", G=128, zeros=False, act="none", pad=0.0),
        # A decode batch through a wide gate and up projection with zero points.
        dict(name="w4_decode_gated", op="w4", T=16, k=0, E=0, K=4096, N=28672, dtype="fp16",
             fmt="int4", G=64, zeros=True, act="silu", pad=0.0),
        # One token through the gate and up projections of its eight experts.
        dict(name="w4_experts_single_token", op="w4", T=1, k=8, E=256, K=7168, N=4096,
             dtype="bf16", fmt="e2m1", G=32, zeros=False, act="silu", pad=0.0),
        # Sixteen tokens' routes (a row each) through the down projections of their experts.
        dict(name="w4_experts_down", op="w4", T=128, k=1, E=256, K=2048, N=7168, dtype="bf16",
             fmt="int4", G=32, zeros=False, act="none", pad=0.02),
    ]


def _spread(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm, odd."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))) | 1


def draw(rng):
    op = rng.choice(["norm", "gated", "w4"])
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        K = rng.choice([2048, 4096, 7168, 128 * _spread(rng, 1, 100), _spread(rng, 64, 9000)])
        return dict(op=op, T=_spread(rng, 1, max(2, min(16000, int(5.0e7 / K)))), K=K, dtype=dtype,
                    wdtype=rng.choice(["fp32", dtype]), sf=rng.choice(["ue8m0", "fp32"]),
                    z=rng.random() < 0.7, y=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "gated":
        K, N = rng.choice([(7168, 2048), (4096, 4096 + 128 * rng.randint(0, 80)),
                           (8 * _spread(rng, 8, 900), _spread(rng, 33, 5000))])
        train = rng.random() < 0.5
        most = (7.0e11 if train else 4.8e11) / (K * N * (12 if train else 4))
        return dict(op=op, T=_spread(rng, 1, max(2, min(8000, int(most)))), K=K, N=N, dtype=dtype,
                    act=rng.choice(["silu", "gelu_tanh"]), train=train)
    fmt = rng.choice(["int4", "int4", "e2m1"])
    G = rng.choice([32, 64, 128]) if fmt == "int4" else 32
    act = rng.choice(["none", "silu", "gelu_tanh"])
    experts = rng.random() < 0.5
    K = rng.choice([2048, 4096, 7168, G * _spread(rng, 2, 4000 // G)])
    N = 2 * rng.choice([1024, 2048, 3584, _spread(rng, 17, 3500)])
    k = rng.randint(1, 8) if experts else 0
    T = _spread(rng, 1, max(2, 128 // k)) if experts else _spread(rng, 1, 33)
    E = 0
    if experts:  # the plain form takes a matrix for each route
        T = max(1, min(T, 128 // k, int(1.9e9 / (k * N * K))))
        E = max(8, min(_spread(rng, 8, 256), int(7.6e9 / (N * K))))
    return dict(op=op, T=T, k=k, E=E, K=K, N=N, dtype=dtype,
                fmt=fmt, G=G, zeros=fmt == "int4" and rng.random() < 0.5, act=act,
                pad=rng.choice([0.0, 0.1]) if experts else 0.0)


# ------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    dev = dict(device="cuda")

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        return (torch.randn(shape, generator=g, **dev) * std + mean).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, **dev)

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, **dev)

    c, T, K, dt = case, case["T"], case["K"], _DTYPES[case["dtype"]]
    s = dict(case=dict(case))
    if c["op"] == "norm":
        # the stream of a few channels is far larger than that of the others
        x = normal(T, K, std=2.0) * torch.where(uniform(K) < 0.01, 20.0, 1.0)
        groups = (K + 127) // 128
        s.update(x=x.to(dt), z=normal(T, K, dtype=dt) if c["z"] else None,
                 weight=normal(K, dtype=_DTYPES[c["wdtype"]], mean=1.0, std=0.2),
                 q=empty(T, K, dtype=torch.uint8),
                 q_sf=(empty(T, groups, dtype=torch.float32) if c["sf"] == "fp32" else
                       empty(T, (groups + 3) // 4, dtype=torch.int32)),
                 x_out=empty(T, K, dtype=dt) if c["z"] else None,
                 y=empty(T, K, dtype=dt) if c["y"] else None, rstd=empty(T, dtype=torch.float32))
    elif c["op"] == "gated":
        N = c["N"]
        s.update(x=normal(T, K, dtype=dt), weight=normal(2 * N, K, dtype=dt, std=K ** -0.5),
                 out=empty(T, N, dtype=dt))
        if c["train"]:
            s.update(gate_up=empty(T, 2 * N, dtype=dt), d_out=normal(T, N, dtype=dt),
                     d_x=empty(T, K, dtype=dt), d_weight=empty(2 * N, K, dtype=dt))
    else:
        N, G, E, k = c["N"], c["G"], c["E"], c["k"]
        lead = (E, N) if E else (N,)
        s.update(x=normal(T, K, dtype=dt),
                 weight=torch.randint(0, 256, (*lead, K // 2), dtype=torch.uint8, generator=g, **dev))
        if c["fmt"] == "e2m1":
            # powers of two about those of weights of deviation K ** -0.5, as bytes 127 + log2
            mean = 127 - round(math.log2(3.0 * math.sqrt(K)))
            s["scales"] = (mean + torch.randint(-1, 2, (*lead, K // G), generator=g, **dev)).to(torch.uint8)
        else:
            s["scales"] = ((0.5 + uniform(*lead, K // G)) * (K ** -0.5 / 4.6)).to(dt)
        s["zeros"] = (torch.randint(5, 12, (*lead, K // G), dtype=torch.uint8, generator=g, **dev)
                      if c["zeros"] else None)
        s["ids"] = None
        if E:
            ids = uniform(T, E).argsort(dim=1)[:, :k].to(torch.int32)
            if c["pad"]:
                ids[uniform(T) < c["pad"]] = -1
            s["ids"] = ids.contiguous()
        s["out"] = empty(T * max(k, 1), N if c["act"] == "none" else N // 2, dtype=dt)
    return s


# ---------------------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "gated": _own_gated, "w4": _own_w4}[op](state)
    return {"norm": _plain_norm, "gated": _plain_gated, "w4": _plain_w4}[op](state)


def _norm_outputs(s, q, sf):
    """The 8-bit values as what they stand for: codes as e4m3, packed exponents as powers of two."""
    if sf.dtype is not torch.float32:
        sf = sf.view(torch.uint8).view(torch.float8_e8m0fnu)
    return dict(q=q.view(torch.float8_e4m3fn), q_sf=sf)


def _own_norm(s):
    B, c = _B(), s["case"]
    B.moe_norm_quant(s["x"], s["weight"], s["q"], s["q_sf"], z=s["z"], x_out=s["x_out"], y=s["y"],
                     rstd=s["rstd"], eps=EPS)
    return dict(**_norm_outputs(s, s["q"], s["q_sf"]), x_out=s["x_out"], y=s["y"], rstd=s["rstd"])


def _activation(B, name):
    return {"silu": B.MOE_ACT_SILU, "gelu_tanh": B.MOE_ACT_GELU_TANH, "none": B.MOE_ACT_NONE}[name]


def _own_gated(s):
    B, c = _B(), s["case"]
    act = _activation(B, c["act"])
    if not c["train"]:
        B.moe_gated_linear(s["x"], s["weight"], s["out"], activation=act)
        return dict(out=s["out"])
    B.moe_gated_linear(s["x"], s["weight"], s["out"], activation=act, gate_up=s["gate_up"])
    ws = s.get("workspace")
    if ws is None:  # kept beside the buffers, as a user's program does
        n = B.gated_linear_workspace_size(c["T"], c["K"], c["N"])
        ws = s["workspace"] = torch.empty(max(256, n), dtype=torch.uint8, device="cuda")
    B.moe_gated_linear_backward(s["d_out"], s["x"], s["weight"], s["gate_up"], d_x=s["d_x"],
                                d_weight=s["d_weight"], activation=act, workspace=ws)
    return dict(out=s["out"], gate_up=s["gate_up"], d_x=s["d_x"], d_weight=s["d_weight"])


def _own_w4(s):
    B, c = _B(), s["case"]
    B.moe_w4_linear(s["x"], s["weight"], s["scales"], s["out"], zeros=s["zeros"],
                    topk_ids=s["ids"], activation=_activation(B, c["act"]))
    return dict(out=s["out"])


# ------------------------------------------------------------------------------------- plain forms
def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    T, K = x.shape
    if c["z"]:
        x = x + s["z"].float()
    rstd = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    y = x * rstd * s["weight"].float()
    groups = torch.nn.functional.pad(y, (0, -K % 128)).view(T, -1, 128)
    scale = groups.abs().amax(dim=2).clamp_min(1e-4) / 448.0
    if c["sf"] == "fp32":
        sf, inverse = scale, 1.0 / scale
    else:  # the power of two at or above, as a byte 127 + log2, four to a word
        m, e = torch.frexp(scale)
        log2 = torch.where(m == 0.5, e - 1, e)
        inverse = torch.exp2(-log2.float())
        sf = torch.nn.functional.pad((log2 + 127).clamp(1, 254).to(torch.uint8),
                                     (0, -scale.shape[1] % 4)).view(torch.int32)
    q = (groups * inverse[:, :, None]).clamp(-448.0, 448.0).view(T, -1)[:, :K]
    q = q.contiguous().to(torch.float8_e4m3fn)
    dt = s["x"].dtype
    return dict(**_norm_outputs(s, q, sf), x_out=x.to(dt) if c["z"] else None,
                y=y.to(dt) if c["y"] else None, rstd=rstd[:, 0])


def _gelu_inner(g):
    return math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)


def _plain_act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(_gelu_inner(g)))


def _plain_gated(s):
    c, dt, N = s["case"], s["x"].dtype, s["case"]["N"]
    x, w = s["x"].float(), s["weight"].float()
    gu = x @ w.t()
    out = (_plain_act(gu[:, :N], c["act"]) * gu[:, N:]).to(dt)
    if not c["train"]:
        return dict(out=out)
    # the backward call has gate and up as the forward call wrote them
    gate_up = gu.to(dt)
    g, u, d = gate_up[:, :N].float(), gate_up[:, N:].float(), s["d_out"].float()
    if c["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        act, slope = g * sig, sig * (1.0 + g * (1.0 - sig))
    else:
        t = torch.tanh(_gelu_inner(g))
        inner = math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * g * g)
        act, slope = 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * inner
    d_gu = torch.cat([d * u * slope, d * act], dim=1)
    return dict(out=out, gate_up=gate_up, d_x=(d_gu @ w).to(dt), d_weight=(d_gu.t() @ x).to(dt))


def _plain_w4(s):
    c, x = s["case"], s["x"].float()
    T, K = x.shape
    N, G, k = c["N"], c["G"], c["k"]
    weight, scales, zeros = s["weight"], s["scales"], s["zeros"]
    routed = None
    if s["ids"] is not None:  # a matrix for each route
        ids = s["ids"].reshape(-1)
        routed = ids >= 0
        at = ids.clamp_min(0).long()
        weight, scales = weight[at], scales[at]
        zeros = zeros[at] if zeros is not None else None
    codes = torch.stack([weight & 15, weight >> 4], dim=-1).view(*weight.shape[:-1], K // G, G)
    if c["fmt"] == "e2m1":
        w = torch.tensor(_E2M1, device="cuda")[codes.int()]
        scale = torch.exp2(scales.float() - 127.0)
    else:
        w = codes.float() - (zeros.float()[..., None] if zeros is not None else 8.0)
        scale = scales.float()
    w = (w * scale[..., None]).view(*weight.shape[:-1], K)
    if routed is None:
        r = x @ w.t()
    else:
        rows = x[:, None, :].expand(T, k, K).reshape(T * k, K, 1)
        r = torch.where(routed[:, None], torch.bmm(w, rows)[:, :, 0], 0.0)
    if c["act"] != "none":
        r = _plain_act(r[:, :N // 2], c["act"]) * r[:, N // 2:]
    return dict(out=r.to(s["x"].dtype))


# ------------------------------------------------------------------------------------ bytes, flops
def work(case):
    c, T, K, b = case, case["T"], case["K"], _BYTES[case["dtype"]]
    if c["op"] == "norm":
        tensors = 1 + (2 if c["z"] else 0) + (1 if c["y"] else 0)
        scales = (K + 127) // 128 * (4 if c["sf"] == "fp32" else 1)
        return dict(bytes=T * (K * (tensors * b + 1) + scales + 4) + K * _BYTES[c["wdtype"]],
                    flops=8 * T * K)
    if c["op"] == "gated":
        N = c["N"]
        bytes_, flops = (T * K + 2 * N * K + T * N) * b, 4 * T * N * K
        if c["train"]:  # d_out in; gate_up, d_x and d_weight out
            bytes_, flops = bytes_ + (T * N + 2 * T * N + T * K + 2 * N * K) * b, 3 * flops
        return dict(bytes=bytes_, flops=flops)
    N, G, rows = c["N"], c["G"], T * max(c["k"], 1)
    matrix = N * K // 2 + N * (K // G) * ((1 if c["fmt"] == "e2m1" else b) + (1 if c["zeros"] else 0))
    # experts that a batch of routes names, on average over draws without preference
    used = c["E"] * (1.0 - (1.0 - 1.0 / c["E"]) ** (rows * (1.0 - c["pad"]))) if c["E"] else 1
    out = rows * (N if c["act"] == "none" else N // 2)
    return dict(bytes=int(used * matrix) + (T * K + out) * b, flops=2 * rows * N * K)


# ------------------------------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    c, s = case, prepare(case, seed)
    return {"norm": _exact_norm, "gated": _exact_gated, "w4": _exact_w4}[c["op"]](c, s)


def _exact_norm(c, s):
    x = s["x"].double()
    if c["z"]:
        x = x + s["z"].double()
    T, K = x.shape
    rstd = 1.0 / torch.sqrt(torch.einsum("tk,tk->t", x, x) / K + EPS)
    y = torch.einsum("tk,t,k->tk", x, rstd, s["weight"].double())
    q, scales = torch.empty_like(y), []
    for at in range(0, K, 128):
        part = y[:, at:at + 128]
        scale = part.abs().max(dim=1).values.clamp_min(1e-4) / 448.0
        if c["sf"] != "fp32":
            scale = torch.exp2(torch.ceil(torch.log2(scale)))
        scales.append(scale)
        v = (part / scale[:, None]).clamp(-448.0, 448.0)
        # e4m3: three bits behind the leading one, steps of 2^-9 at the smallest
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
        q[:, at:at + 128] = torch.round(v / step) * step
    if c["sf"] != "fp32":  # the bytes that fill the last word are zero: 2^-127
        scales += [torch.full_like(rstd, 2.0 ** -127)] * (-len(scales) % 4)
    return dict(q=q, q_sf=torch.stack(scales, dim=1), x_out=x if c["z"] else None,
                y=y if c["y"] else None, rstd=rstd)


def _exact_gated(c, s):
    x, w = s["x"].double(), s["weight"].double()
    if c["train"]:
        x.requires_grad_(True)
        w.requires_grad_(True)
    gate_up = torch.einsum("tk,nk->tn", x, w)
    g, u = gate_up.split(c["N"], dim=1)
    if c["act"] == "silu":
        a = g * torch.sigmoid(g)
    else:
        a = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))
    out = a * u
    if not c["train"]:
        return dict(out=out)
    out.backward(s["d_out"].double())
    return dict(out=out.detach(), gate_up=gate_up.detach(), d_x=x.grad, d_weight=w.grad)


def _exact_w4(c, s):
    x, k = s["x"].double(), max(c["k"], 1)
    K, N, rows = c["K"], c["N"], c["T"] * k
    out = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
    experts = s["ids"].reshape(-1).tolist() if c["E"] else [0] * rows
    for e in sorted({i for i in experts if i >= 0}):  # each matrix with the rows that name it
        bytes_, scales, zeros = (t if t is None or not c["E"] else t[e]
                                 for t in (s["weight"], s["scales"], s["zeros"]))
        w = torch.empty(N, K, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (bytes_ % 16).double(), (bytes_ // 16).double()
        if c["fmt"] == "e2m1":
            sign = 1.0 - 2.0 * (w >= 8)
            code = w % 8
            two, half = torch.div(code, 2, rounding_mode="floor"), code % 2
            w = sign * torch.where(two == 0, half / 2, torch.exp2(two - 1) * (1 + half / 2))
            factor = 2.0 ** (scales.double() - 127)
        else:
            factor = scales.double()
            w -= 8 if zeros is None else zeros.double().repeat_interleave(c["G"], dim=1)
        w *= factor.repeat_interleave(c["G"], dim=1)
        mine = [r for r in range(rows) if experts[r] == e]
        out[mine] = x[[r // k for r in mine]] @ w.t()
    if c["act"] == "none":
        return dict(out=out)
    g, u = out[:, :N // 2], out[:, N // 2:]
    if c["act"] == "silu":
        return dict(out=g * torch.sigmoid(g) * u)
    return dict(out=0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))) * u)
