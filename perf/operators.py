"""Cases of the operators around the experts of an MoE block: routing, sorting rows by expert and
back, the norms before and after the block, and a projection with low-rank adapters.

``listed`` and ``draw`` give cases, ``prepare`` makes a case's inputs and output buffers on the GPU,
``run`` makes one pass: with ``own`` set through the library's entry points, else in a plain form of
elementary tensor operations in 32 bits.  ``exact`` restates each operator in 64 bits.

Sizes: hidden sizes 4096, 7168 and 2048, 8 and 256 experts, top-k 2 and 8 and the token counts are
those of the expert-layer workloads in ``moe_expert_layer_prepare_gb300/synthetic.py``.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
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
        # The router of a small decode batch: 8 experts, two per token, softmax over the two.
        dict(name="route_decode", op="route", T=64, E=8, k=2, dtype="bf16", scoring="softmax",
             renorm=True, bias=False, groups=1, top_groups=1, scale=1.0, pad=0.0, train=False),
        # Prefill of a 256-expert layer: sigmoid scores, a selection bias that balances the
        # experts, the experts limited to 4 of 8 groups, 2% padding tokens.
        dict(name="route_prefill_groups", op="route", T=8192, E=256, k=8, dtype="fp32",
             scoring="sigmoid", renorm=True, bias=True, groups=8, top_groups=4, scale=2.5,
             pad=0.02, train=False),
        # A training step's router: weights of the full softmax and the gradient of the logits.
        dict(name="route_train", op="route", T=16384, E=256, k=8, dtype="fp32",
             scoring="softmax", renorm=False, bias=False, groups=1, top_groups=1, scale=1.0,
             pad=0.0, train=True),
        # A decode batch sorted by expert and combined again.
        dict(name="sort_decode", op="sort", T=64, E=8, k=2, K=4096, dtype="bf16", pad=0.0,
             train=False),
        # Prefill of a 256-expert layer: 65,536 routes of 7168 values there and back.
        dict(name="sort_prefill", op="sort", T=8192, E=256, k=8, K=7168, dtype="bf16", pad=0.0,
             train=False),
        # A training step with an odd number of tokens, some of them padding: both directions.
        dict(name="sort_train_odd", op="sort", T=2051, E=32, k=6, K=4096, dtype="fp16", pad=0.05,
             train=True),
        # One token between two blocks: the norm after one and the norm before the next.
        dict(name="norm_single_token", op="norm", T=1, K=7168, dtype="bf16", wdtype="bf16",
             post=True, gate="channel", train=False),
        # Prefill of the same, each token's block output gated by a number of its own.
        dict(name="norm_prefill", op="norm", T=8192, K=7168, dtype="bf16", wdtype="bf16",
             post=True, gate="token", train=False),
        # A training step: forward and all gradients, fp32 norm weights, a gate for every value.
        dict(name="norm_train_odd", op="norm", T=4099, K=4096, dtype="bf16", wdtype="fp32",
             post=True, gate="full", train=True),
        # One request's single token through a gate_up projection with its adapter.
        dict(name="lora_single_token", op="lora", T=1, K=7168, N=4096, S=8, R=16, dtype="bf16",
             mixed=True),
        # A decode batch of requests that each name one of 48 adapters, through a down projection.
        dict(name="lora_decode", op="lora", T=64, K=2048, N=7168, S=48, R=32, dtype="fp16",
             mixed=True),
        # Prefill: the tokens of a few long requests after one another.
        dict(name="lora_prefill", op="lora", T=8192, K=7168, N=4096, S=16, R=64, dtype="bf16",
             mixed=False),
    ]


def _spread(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm, odd."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))) | 1


def draw(rng):
    op = rng.choice(["route", "sort", "norm", "lora"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "route":
        scoring = rng.choice(["softmax", "sigmoid"])
        grouped = rng.random() < 0.4
        groups = rng.choice([4, 8]) if grouped else 1
        E = groups * rng.randint(3, 32) if grouped else _spread(rng, 5, 383)
        train = rng.random() < 0.5
        return dict(op=op, T=_spread(rng, 1, 16000), E=E,
                    k=rng.randint(1, 2 if E < 8 else 8), dtype=dtype, scoring=scoring,
                    renorm=rng.random() < 0.5, bias=grouped, groups=groups,
                    top_groups=groups // 2 if grouped else 1,
                    scale=round(rng.uniform(0.5, 3.0), 3),
                    pad=rng.choice([0.0, 0.1]), train=train)
    if op == "sort":
        K = rng.choice([2048, 4096, 7168, 8 * _spread(rng, 8, 900), _spread(rng, 64, 5000)])
        k = rng.randint(1, 8)
        train = rng.random() < 0.5
        T = _spread(rng, 1, max(2, min(8000, int((1.8e8 if train else 4.0e8) / (K * k)))))
        return dict(op=op, T=T, E=_spread(rng, 4, 300), k=k, K=K, dtype=dtype,
                    pad=rng.choice([0.0, 0.1]), train=train)
    if op == "norm":
        K = rng.choice([2048, 4096, 7168, 8 * _spread(rng, 8, 900), _spread(rng, 64, 9000)])
        train = rng.random() < 0.5
        T = _spread(rng, 1, max(2, min(16000, int((1.5e7 if train else 5.0e7) / K))))
        return dict(op=op, T=T, K=K, dtype=dtype,
                    wdtype=rng.choice(["fp32", dtype]), post=rng.random() < 0.8,
                    gate=rng.choice(["none", "channel", "token", "full"]), train=train)
    K, N = rng.choice([(7168, 4096), (2048, 7168), (8 * _spread(rng, 8, 600), _spread(rng, 64, 6000))])
    return dict(op=op, T=_spread(rng, 1, 4000), K=K, N=N, S=rng.randint(1, 24),
                R=8 * rng.randint(1, 8), dtype=rng.choice(["bf16", "fp16"]),
                mixed=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    dev = dict(device="cuda")

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        return (torch.randn(shape, generator=g, **dev) * std + mean).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, **dev)

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, **dev)

    c, T, dt = case, case["T"], _DTYPES[case["dtype"]]
    s = dict(case=dict(case))
    if c["op"] == "route":
        E, k = c["E"], c["k"]
        # an uneven router: some experts are liked by every token
        s["logits"] = (normal(T, E) + normal(1, E, std=0.5)).to(dt)
        s["bias"] = normal(E, std=0.02) if c["bias"] else None
        s["is_padding"] = (uniform(T) < c["pad"]).to(torch.uint8) if c["pad"] else None
        s["ids"] = empty(T, k, dtype=torch.int32)
        s["weights"] = empty(T, k, dtype=torch.float32)
        if c["train"]:
            s["d_weights"] = normal(T, k)
            s["d_logits"] = empty(T, E, dtype=dt)
    elif c["op"] == "sort":
        E, k, K = c["E"], c["k"], c["K"]
        k = min(k, E)
        logits = normal(T, E) + normal(1, E, std=0.7)
        ids = logits.argsort(dim=1, descending=True)[:, :k].to(torch.int32)
        w = torch.softmax(normal(T, k), dim=1)
        if c["pad"]:
            padding = uniform(T) < c["pad"]
            ids[padding] = -1
            w[padding] = 0.0
        s.update(ids=ids.contiguous(), weights=w.contiguous(), x=normal(T, K, dtype=dt),
                 expert_out=normal(T * k, K, dtype=dt))
        s.update(offsets=empty(E + 1, dtype=torch.int32), route_row=empty(T, k, dtype=torch.int32),
                 row_route=empty(T * k, dtype=torch.int32), rows=empty(T * k, K, dtype=dt),
                 out=empty(T, K, dtype=dt))
        if c["train"]:
            s.update(d_out=normal(T, K, dtype=dt), d_rows_in=normal(T * k, K, dtype=dt),
                     d_expert_out=empty(T * k, K, dtype=dt),
                     d_weights=empty(T, k, dtype=torch.float32), d_x=empty(T, K, dtype=dt))
    elif c["op"] == "norm":
        K, wt = c["K"], _DTYPES[c["wdtype"]]
        s.update(x=normal(T, K, dtype=dt, std=2.0), z=normal(T, K, dtype=dt),
                 post_w=normal(K, dtype=wt, mean=1.0, std=0.2) if c["post"] else None,
                 pre_w=normal(K, dtype=wt, mean=1.0, std=0.2), scale=0.7)
        shape = {"none": None, "channel": (K,), "token": (T,), "full": (T, K)}[c["gate"]]
        gt = wt if c["gate"] == "channel" else dt
        s["gate"] = normal(*shape, dtype=gt, mean=0.5, std=0.5) if shape else None
        s.update(x_out=empty(T, K, dtype=dt), y=empty(T, K, dtype=dt),
                 rstd_post=empty(T, dtype=torch.float32) if c["post"] else None,
                 rstd_pre=empty(T, dtype=torch.float32))
        if c["train"]:
            s.update(d_x_out=normal(T, K, dtype=dt), d_y=normal(T, K, dtype=dt),
                     d_x=empty(T, K, dtype=dt), d_z=empty(T, K, dtype=dt),
                     d_post_w=empty(K, dtype=wt) if c["post"] else None,
                     d_pre_w=empty(K, dtype=wt),
                     d_gate=empty(*shape, dtype=gt) if shape else None)
    else:
        K, N, S, R = c["K"], c["N"], c["S"], c["R"]
        s.update(x=normal(T, K, dtype=dt), weight=normal(N, K, dtype=dt, std=K ** -0.5),
                 lora_a=normal(S, R, K, dtype=dt, std=K ** -0.5),
                 lora_b=normal(S, N, R, dtype=dt, std=R ** -0.5),
                 lora_scale=0.25 + uniform(S))
        if c["mixed"]:  # every token belongs to a request of its own; some have no adapter
            ids = torch.floor(uniform(T) * (S + 0.1)).to(torch.int32)
            ids[ids >= S] = -1
        else:  # requests one after another
            n = min(T, S + 1)
            begin = torch.floor(torch.sort(uniform(n)).values * T)
            request = (torch.arange(T, **dev)[:, None] >= begin[None, :]).sum(dim=1)
            ids = torch.where(request < n, request - 1, -1).to(torch.int32)
        s.update(adapter_ids=ids.contiguous(), out=empty(T, N, dtype=dt))
    return s


# ---------------------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "sort": _own_sort, "norm": _own_norm, "lora": _own_lora}[op](state)
    return {"route": _plain_route, "sort": _plain_sort, "norm": _plain_norm,
            "lora": _plain_lora}[op](state)


def _workspace(s, size):
    """The workspace that a user's program keeps beside its buffers."""
    ws = s.get("workspace")
    if ws is None:
        ws = s["workspace"] = torch.empty(max(256, size()), dtype=torch.uint8, device="cuda")
    return ws


def _own_route(s):
    B, c = _B(), s["case"]
    scoring = B.MOE_SCORE_SIGMOID if c["scoring"] == "sigmoid" else B.MOE_SCORE_SOFTMAX
    B.moe_route(s["logits"], s["ids"], s["weights"], bias=s["bias"], is_padding=s["is_padding"],
                scoring=scoring, renormalize=c["renorm"], scale=c["scale"],
                num_groups=c["groups"], top_groups=c["top_groups"])
    if not c["train"]:
        return dict(ids=s["ids"], weights=s["weights"])
    B.moe_route_backward(s["logits"], s["ids"], s["d_weights"], s["d_logits"], scoring=scoring,
                         renormalize=c["renorm"], scale=c["scale"])
    return dict(ids=s["ids"], weights=s["weights"], d_logits=s["d_logits"])


def _own_sort(s):
    B, c = _B(), s["case"]
    ws = _workspace(s, lambda: B.sort_workspace_size(c["T"], s["ids"].shape[1], c["E"]))
    B.moe_sort_routes(s["ids"], s["offsets"], s["route_row"], s["row_route"], ws)
    B.moe_permute(s["x"], s["route_row"], s["offsets"], s["rows"])
    B.moe_unpermute(s["expert_out"], s["route_row"], s["weights"], s["out"])
    r = dict(offsets=s["offsets"], route_row=s["route_row"], row_route=s["row_route"],
             rows=s["rows"], out=s["out"])
    if c["train"]:
        B.moe_unpermute_backward(s["d_out"], s["expert_out"], s["route_row"], s["weights"],
                                 s["offsets"], s["d_expert_out"], s["d_weights"])
        B.moe_permute_backward(s["d_rows_in"], s["route_row"], s["d_x"])
        r.update(d_expert_out=s["d_expert_out"], d_weights=s["d_weights"], d_x=s["d_x"])
    return r


def _own_norm(s):
    B, c = _B(), s["case"]
    B.moe_block_norm(s["x"], z=s["z"], post_weight=s["post_w"], gate=s["gate"], scale=s["scale"],
                     pre_weight=s["pre_w"], eps=EPS, x_out=s["x_out"], y=s["y"],
                     rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"])
    r = dict(x_out=s["x_out"], y=s["y"], rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"])
    if c["train"]:
        ws = _workspace(s, lambda: B.block_norm_workspace_size(c["T"], c["K"]))
        B.moe_block_norm_backward(s["x"], z=s["z"], post_weight=s["post_w"], gate=s["gate"],
                                  scale=s["scale"], pre_weight=s["pre_w"],
                                  rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"],
                                  d_x_out=s["d_x_out"], d_y=s["d_y"], d_x=s["d_x"], d_z=s["d_z"],
                                  d_gate=s["d_gate"], d_post_weight=s["d_post_w"],
                                  d_pre_weight=s["d_pre_w"], workspace=ws)
        r.update(d_x=s["d_x"], d_z=s["d_z"], d_post_w=s["d_post_w"], d_pre_w=s["d_pre_w"],
                 d_gate=s["d_gate"])
    return r


def _own_lora(s):
    B, c = _B(), s["case"]
    ws = _workspace(s, lambda: B.lora_workspace_size(c["T"], c["K"], c["N"], c["S"], c["R"]))
    B.moe_lora_linear(s["x"], s["weight"], s["lora_a"], s["lora_b"], s["adapter_ids"],
                      s["lora_scale"], s["out"], ws)
    return dict(out=s["out"])


# ------------------------------------------------------------------------------------- plain forms
_NINF = float("-inf")


def _selection(l, bias, sigmoid, groups, top_groups):
    """Selection keys in 32 bits, the groups that lose set to -inf.  Without a bias experts are
    taken in the order of their logits; with one, of score + bias (softmax: logit + bias)."""
    key = l
    if bias is not None:
        key = (1.0 / (1.0 + torch.exp(-l)) if sigmoid else l) + bias
    key = torch.where(key > _NINF, key, _NINF) + 0.0
    if groups > 1:
        T, E = key.shape
        best = key.view(T, groups, E // groups).sort(dim=2, descending=True, stable=True).values
        group = best[:, :, 0]
        if bias is not None and best.shape[2] > 1:
            group = group + torch.where(best[:, :, 1] > _NINF, best[:, :, 1], 0.0)
        order = group.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        kept = torch.zeros_like(group, dtype=torch.bool).scatter(1, order, True)
        key = torch.where(kept[:, :, None], key.view(T, groups, -1), _NINF).view(T, E)
    return key


def _plain_route(s):
    c, l = s["case"], s["logits"].float()
    T, E = l.shape
    k, sigmoid = c["k"], c["scoring"] == "sigmoid"
    key = _selection(l, s["bias"], sigmoid, c["groups"], c["top_groups"])
    top = key.sort(dim=1, descending=True, stable=True)
    ids, placed = top.indices[:, :k], top.values[:, :k] > _NINF
    if s["is_padding"] is not None:
        placed = placed & (s["is_padding"] == 0)[:, None]
    chosen = l.gather(1, ids)
    if sigmoid:
        score = torch.where(placed, 1.0 / (1.0 + torch.exp(-chosen)), 0.0)
        total = score.sum(dim=1, keepdim=True) + 1e-20 if c["renorm"] else 1.0
    elif c["renorm"]:
        score = torch.where(placed, torch.exp(chosen - chosen.max(dim=1, keepdim=True).values), 0.0)
        total = score.sum(dim=1, keepdim=True).clamp_min(1e-20)
    else:
        m = l.max(dim=1, keepdim=True).values
        score = torch.where(placed, torch.exp(chosen - m), 0.0)
        total = torch.exp(l - m).sum(dim=1, keepdim=True)
    p = score / total
    r = dict(ids=torch.where(placed, ids, -1).to(torch.int32), weights=p * c["scale"])
    if c["train"]:
        dw = torch.where(placed, s["d_weights"], 0.0) * c["scale"]
        mean = (dw * p).sum(dim=1, keepdim=True)
        if sigmoid:
            up = (dw - mean) / total if c["renorm"] else dw
            d = torch.where(placed, up * score * (1.0 - score), 0.0)
            d = torch.zeros_like(l).scatter_add(1, ids, d)
        elif c["renorm"]:
            d = torch.zeros_like(l).scatter_add(1, ids, p * (dw - mean))
        else:
            d = torch.zeros_like(l).scatter_add(1, ids, p * dw) - torch.exp(l - m) / total * mean
        r["d_logits"] = d.to(s["logits"].dtype)
    return r


def _plain_sort(s):
    c, ids, x = s["case"], s["ids"], s["x"]
    (T, k), K, E = ids.shape, x.shape[1], c["E"]
    flat = torch.where(ids < 0, E, ids).reshape(-1)
    order = flat.sort(stable=True)  # unrouted last
    n = torch.searchsorted(order.values, torch.arange(E + 1, dtype=torch.int32, device="cuda"))
    routed = order.values < E
    row_route = torch.where(routed, order.indices, -1)
    at = torch.empty_like(order.indices)
    at[order.indices] = torch.arange(T * k, device="cuda")
    route_row = torch.where(ids < 0, -1, at.view(T, k))
    rows = torch.where(routed[:, None], x[order.indices // k], 0.0).to(x.dtype)
    w = torch.where(ids < 0, 0.0, s["weights"])
    picked = torch.where((ids < 0)[:, :, None], 0.0, s["expert_out"][at.view(T, k)].float())
    out = (picked * w[:, :, None]).sum(dim=1)
    r = dict(offsets=n.to(torch.int32), route_row=route_row.to(torch.int32),
             row_route=row_route.to(torch.int32), rows=rows, out=out.to(x.dtype))
    if c["train"]:
        up = s["d_out"].float()
        r["d_weights"] = (picked * up[:, None, :]).sum(dim=2)
        back = up[order.indices // k] * w.reshape(-1)[order.indices][:, None]
        r["d_expert_out"] = torch.where(routed[:, None], back, 0.0).to(x.dtype)
        got = torch.where((ids < 0)[:, :, None], 0.0, s["d_rows_in"][at.view(T, k)].float())
        r["d_x"] = got.sum(dim=1).to(x.dtype)
    return r


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    x, z = s["x"].float(), s["z"].float()
    pre = s["pre_w"].float()
    gate = 1.0
    if s["gate"] is not None:
        gate = s["gate"].float()[:, None] if c["gate"] == "token" else s["gate"].float()
    post = s["post_w"].float() if c["post"] else 1.0
    rz = torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS) if c["post"] else None
    zhat = z * rz if c["post"] else z
    n = zhat * post
    xo = x + s["scale"] * (gate * n)
    rx = torch.rsqrt((xo * xo).mean(dim=1, keepdim=True) + EPS)
    xhat = xo * rx
    r = dict(x_out=xo.to(dt), y=(xhat * pre).to(dt),
             rstd_post=rz[:, 0] if c["post"] else None, rstd_pre=rx[:, 0])
    if c["train"]:
        dy = s["d_y"].float()
        up = dy * pre
        d = s["d_x_out"].float() + rx * (up - xhat * (up * xhat).mean(dim=1, keepdim=True))
        dn = s["scale"] * (gate * d)
        dz = dn * post
        if c["post"]:
            dz = rz * (dz - zhat * (dz * zhat).mean(dim=1, keepdim=True))
        dg = None
        if s["gate"] is not None:
            dg = s["scale"] * (d * n)
            dg = dg.sum(dim=0) if c["gate"] == "channel" else dg.sum(dim=1) if c["gate"] == "token" else dg
            dg = dg.to(s["gate"].dtype)
        wt = s["pre_w"].dtype
        r.update(d_x=d.to(dt), d_z=dz.to(dt), d_pre_w=(dy * xhat).sum(dim=0).to(wt),
                 d_post_w=(dn * zhat).sum(dim=0).to(wt) if c["post"] else None, d_gate=dg)
    return r


def _plain_lora(s):
    S, R, K = s["lora_a"].shape
    N = s["weight"].shape[0]
    x = s["x"].float()
    out = x @ s["weight"].float().t()
    mine = s["adapter_ids"][:, None] == torch.arange(S, device="cuda")[None, :]
    h = (x @ s["lora_a"].float().view(S * R, K).t()).view(-1, S, R)
    h = h * (mine * s["lora_scale"])[:, :, None]
    out = out + h.view(-1, S * R) @ s["lora_b"].float().transpose(1, 2).reshape(S * R, N)
    return dict(out=out.to(s["x"].dtype))


# ------------------------------------------------------------------------------------ bytes, flops
def work(case):
    c, T, b = case, case["T"], _BYTES[case["dtype"]]
    if c["op"] == "route":
        E, k = c["E"], c["k"]
        read = T * E * b + (E * 4 if c["bias"] else 0) + (T if c["pad"] else 0)
        write = T * k * 8
        flops = T * E * 4
        if c["train"]:
            read += T * k * 4
            write += T * E * b
            flops += T * E * 4
        return dict(bytes=read + write, flops=flops)
    if c["op"] == "sort":
        k, K = min(c["k"], c["E"]), c["K"]
        routed = int(T * k * (1.0 - c["pad"]))
        plan = T * k * 4 * 4 + (c["E"] + 1) * 4
        rows = T * k * K * b
        read = T * K * b + routed * K * b
        write = rows + T * K * b
        flops = 2 * routed * K
        if c["train"]:
            read += T * K * b + routed * K * b
            write += rows + T * K * b + T * k * 4
            flops += 4 * routed * K
        return dict(bytes=plan + read + write, flops=flops)
    if c["op"] == "norm":
        K, w = c["K"], _BYTES[c["wdtype"]]
        gate = {"none": 0, "channel": K * w, "token": T * b, "full": T * K * b}[c["gate"]]
        weights = (2 if c["post"] else 1) * K * w
        bytes_ = 4 * T * K * b + gate + weights + T * 8
        flops = 11 * T * K
        if c["train"]:
            bytes_ += 4 * T * K * b + gate + weights
            flops += 25 * T * K
        return dict(bytes=bytes_, flops=flops)
    K, N, S, R = c["K"], c["N"], c["S"], c["R"]
    used = min(T, S)
    return dict(bytes=(T * K + N * K + T * N + used * R * (K + N)) * b + T * 4 + S * 4,
                flops=2 * T * (N * K + R * (K + N)))


# ------------------------------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] != "lora":
        return {"route": _exact_route, "sort": _exact_sort, "norm": _exact_norm}[c["op"]](c, s)
    x, ids = s["x"].double(), s["adapter_ids"].long()
    out = x @ s["weight"].double().t()
    for a in range(c["S"]):  # each adapter's tokens by themselves
        at = (ids == a).nonzero()[:, 0]
        h = x[at] @ s["lora_a"][a].double().t() * s["lora_scale"][a].double()
        out[at] += h @ s["lora_b"][a].double().t()
    return dict(out=out)


def _exact_route(c, s):
    # which experts are taken is decided by keys in 32 bits; the weights follow from that choice
    keys = _selection(s["logits"].float(), s["bias"], c["scoring"] == "sigmoid", c["groups"], c["top_groups"])
    ids = keys.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    l = s["logits"].double().requires_grad_(True)
    raw = torch.sigmoid(l) if c["scoring"] == "sigmoid" else torch.softmax(l, dim=1)
    w = raw.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    live = 1.0 if s["is_padding"] is None else 1.0 - s["is_padding"].double()[:, None]
    w = w * c["scale"] * live
    r = dict(ids=None, weights=w.detach())
    if c["train"]:
        (w * s["d_weights"].double()).sum().backward()
        r["d_logits"] = l.grad
    return r


def _exact_sort(c, s):
    ids = s["ids"].reshape(-1).long()
    T, k = s["ids"].shape
    routes = torch.arange(T * k, device="cuda")
    # a route's place: all routes of lower experts, then the earlier ones of its own
    place = torch.argsort(torch.where(ids < 0, c["E"], ids) * (T * k) + routes)
    live = place[ids[place] >= 0]
    n = live.numel()
    token, rank = live // k, live % k
    x, eo = s["x"].double(), s["expert_out"].double()
    w = s["weights"].double()[token, rank]
    rows = torch.zeros_like(eo)
    rows[:n] = x[token]
    out = torch.zeros_like(x).index_add_(0, token, eo[:n] * w[:, None])
    r = dict(offsets=None, route_row=None, row_route=None, rows=rows, out=out)
    if c["train"]:
        up = s["d_out"].double()
        d_eo = torch.zeros_like(eo)
        d_eo[:n] = up[token] * w[:, None]
        d_w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        d_w[token, rank] = torch.einsum("rk,rk->r", eo[:n], up[token])
        r.update(d_expert_out=d_eo, d_weights=d_w,
                 d_x=torch.zeros_like(x).index_add_(0, token, s["d_rows_in"][:n].double()))
    return r


def _exact_norm(c, s):
    leaf = {}

    def var(name):
        if s.get(name) is None:
            return None
        leaf[name] = s[name].double().requires_grad_(bool(c["train"]))
        return leaf[name]

    x, z, post, pre, gate = (var(n) for n in ("x", "z", "post_w", "pre_w", "gate"))

    def inv_rms(v):
        return 1.0 / torch.sqrt(torch.einsum("tk,tk->t", v, v) / v.shape[1] + EPS)

    branch, rp = z, None
    if post is not None:
        rp = inv_rms(z)
        branch = z * rp[:, None] * post
    if gate is not None:
        branch = branch * (gate.unsqueeze(1) if c["gate"] == "token" else gate)
    xo = x + s["scale"] * branch
    rq = inv_rms(xo)
    y = xo * rq[:, None] * pre
    r = dict(x_out=xo.detach(), y=y.detach(), rstd_post=None if rp is None else rp.detach(),
             rstd_pre=rq.detach())
    if c["train"]:
        torch.autograd.backward([xo, y], [s["d_x_out"].double(), s["d_y"].double()])
        r.update(d_x=x.grad, d_z=z.grad, d_pre_w=pre.grad,
                 d_post_w=None if post is None else post.grad,
                 d_gate=None if gate is None else gate.grad)
    return r
