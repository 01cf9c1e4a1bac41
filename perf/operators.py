"""The expert-side operators of the router, as cases to be measured.

The router picks K experts for each of T tokens, and its expert maps order the T K (token,
choice) rows by expert.  The operators here are what runs on those rows:

* ``matmul``: every expert's weight times its rows, read from the tokens through the maps or
  from rows already in the maps' order; ``matmul_bwd`` its gradients by rows and by weights;
* ``matmul_w4``: the same product for decoding, on 4-bit weights with a scale per group;
* ``combine``: each token's sum of its K experts' outputs, weighted; ``combine_bwd`` its
  gradients by outputs and by weights.

The plain forms compute in fp32 and round once to the output's type.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# the largest listed case's cost, which a drawn one does not pass
MOST_FLOPS = 4 * 8192 * 4 * 2048 * 2048
MOST_BYTES = 1.3e9


def matmul(name, T, E, K, D, N, dtype="bf16", out="bf16", gather=True, op="matmul"):
    return {"name": name, "op": op, "T": T, "E": E, "K": K, "D": D, "N": N, "dtype": dtype,
            "out": out, "gather": gather}


def listed():
    return [
        # one decoded token: four experts' weights, nothing to hide the latency behind
        matmul("matmul t1 e64 k4", 1, 64, 4, 1024, 1024),
        # a decode batch: most experts get one or two rows, the weights are all the traffic
        matmul("matmul t32 e256 k8", 32, 256, 8, 2048, 1024),
        # a prefill batch over many experts: 256 rows each, as much traffic as arithmetic
        matmul("matmul t8192 e256 k8", 8192, 256, 8, 2048, 1024),
        # the second product of an expert layer (rows already in the maps' order), odd sizes,
        # kept in fp32 for the weighted sum behind it
        matmul("matmul t1003 e512 k22", 1003, 512, 22, 504, 1000, out="f32", gather=False),
        # fp32 rows and weights, sizes that leave every row at another alignment
        matmul("matmul f32 t517 e64 k4", 517, 64, 4, 515, 333, dtype="f32", out="f32"),
        # a training step of one product: gradients by rows and by weights, fp32 weight
        # gradients as an optimizer accumulates them
        matmul("matmul bwd t8192 e64 k4", 8192, 64, 4, 2048, 2048, out="f32", op="matmul_bwd"),
        # the same on many small ragged experts, bf16 weight gradients
        matmul("matmul bwd t777 e256 k8", 777, 256, 8, 1000, 520, gather=False, op="matmul_bwd"),
        # 4-bit experts: one token, and a decode batch
        {"name": "w4 t1 e256 k8", "op": "matmul_w4", "T": 1, "E": 256, "K": 8, "D": 2048, "N": 1024,
         "group": 128, "zeros": False, "out": "bf16"},
        {"name": "w4 t33 e512 k22", "op": "matmul_w4", "T": 33, "E": 512, "K": 22, "D": 1056,
         "N": 1000, "group": 32, "zeros": True, "out": "f32"},
        # one token's sum, and a prefill batch's with its gradients
        {"name": "combine t1 k8", "op": "combine", "T": 1, "E": 256, "K": 8, "D": 2048, "dtype": "bf16",
         "weighted": True},
        {"name": "combine t8192 k8", "op": "combine", "T": 8192, "E": 256, "K": 8, "D": 2048,
         "dtype": "bf16", "weighted": True},
        {"name": "combine bwd t8192 k8", "op": "combine_bwd", "T": 8192, "E": 256, "K": 8, "D": 2048,
         "dtype": "bf16", "weighted": True},
    ]


def log_int(rng, low, high, step=1):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step))


def draw(rng):
    """One more case: tokens from one to thousands, experts up to the router's largest count,
    feature sizes in eighths (aligned rows) for bf16 and any for fp32."""
    while True:
        op = rng.choice(("matmul", "matmul", "matmul_bwd", "matmul_w4", "combine", "combine_bwd"))
        E = log_int(rng, 4, 2304)
        case = {"op": op, "T": log_int(rng, 1, 8192), "E": E, "K": min(E, log_int(rng, 1, 36))}
        if op in ("matmul", "matmul_bwd"):
            dtype = rng.choice(("bf16", "bf16", "bf16", "bf16", "f32"))
            step = 8 if dtype == "bf16" else 1
            case |= {"D": log_int(rng, 64, 4096, step), "N": log_int(rng, 64, 4096, step), "dtype": dtype,
                     "out": "f32" if dtype == "f32" else rng.choice(("bf16", "f32")),
                     "gather": rng.random() < 0.6}
        elif op == "matmul_w4":
            group = rng.choice((32, 64, 128))
            case |= {"T": log_int(rng, 1, 64), "D": log_int(rng, 2, 4096 // group) * group,
                     "N": log_int(rng, 64, 4096), "group": group, "zeros": rng.random() < 0.5,
                     "out": rng.choice(("bf16", "f32"))}
        else:
            case |= {"D": log_int(rng, 64, 4096), "dtype": rng.choice(("bf16", "f32")),
                     "weighted": rng.random() < 0.8}
        w = work(case)
        # fp32 products run at the vector rate: an eighth of the work for the same time
        share = 0.125 if case.get("dtype") == "f32" and "matmul" in op else 1.0
        # a decode batch: its weights are the cost, not its rows
        flops = 2.4e9 if op == "matmul_w4" else share * MOST_FLOPS
        if w["flops"] <= flops and w["bytes"] <= MOST_BYTES and case["T"] * case["K"] <= 200000:
            return case


def active(T, E, K):
    """Experts that T tokens reach, when each picks K of E at random."""
    return E * (1.0 - (1.0 - K / E) ** T)


def work(case):
    T, E, K, D = case["T"], case["E"], case["K"], case["D"]
    P = T * K
    size = {"f32": 4, "bf16": 2}
    if case["op"] in ("matmul", "matmul_bwd"):
        N, s, o = case["N"], size[case["dtype"]], size[case["out"]]
        x = (T if case["gather"] else P) * D * s
        maps = 4 * (E + 1) + (4 * P if case["gather"] else 0)
        weights = active(T, E, K) * N * D * s
        if case["op"] == "matmul":
            return {"bytes": x + maps + weights + P * N * o, "flops": 2.0 * P * N * D}
        # rows, weights and the incoming gradient in; gradients by rows and by all weights out
        return {"bytes": x + maps + weights + P * N * s + P * D * s + E * N * D * o, "flops": 4.0 * P * N * D}
    if case["op"] == "matmul_w4":
        N, G = case["N"], D // case["group"]
        per_expert = N * (D / 2 + G * (3 if case["zeros"] else 2))
        return {"bytes": T * D * 2 + 4 * (E + 1 + P) + active(T, E, K) * per_expert + P * N * size[case["out"]],
                "flops": 2.0 * P * N * D}
    s, w = size[case["dtype"]], 4 * P if case["weighted"] else 0
    if case["op"] == "combine":
        return {"bytes": P * D * s + 4 * P + w + T * D * s, "flops": 2.0 * P * D}
    read = P * D * s if case["weighted"] else 0
    return {"bytes": T * D * s + read + 4 * P + 2 * w + P * D * s, "flops": 3.0 * P * D}


def prepare(case, seed):
    """Tokens routed by logits whose experts are not equally liked, the router's maps of
    their choices, and the operator's own inputs."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(scale)

    T, E, K, D = case["T"], case["E"], case["K"], case["D"]
    P = T * K
    logits = normal(T, E) + normal(1, E, scale=0.5)
    weights, choice = logits.softmax(1).topk(K, dim=1)
    # choice (t, k) is the expanded row t + k T; permuted rows go by expert, then token
    expert = choice.t().reshape(-1)
    token = torch.arange(P, device=dev) % T
    expert_sorted, by = torch.sort(expert * T + token)
    place = torch.empty_like(by)
    place[by] = torch.arange(P, device=dev)
    first = torch.searchsorted(expert_sorted.div(T, rounding_mode="floor"), torch.arange(E + 1, device=dev))
    s = dict(case, offsets=first.int(), p2u=by.int(), u2p=place.int(), topk=(weights / weights.sum(1, keepdim=True)))
    s["capacity"] = int((first[1:] - first[:-1]).max())
    if case["op"] in ("matmul", "matmul_bwd"):
        dt = TYPES[case["dtype"]]
        s["x"] = normal(T if case["gather"] else P, D, dtype=dt)
        s["weight"] = normal(E, case["N"], D, dtype=dt, scale=D ** -0.5)
        if case["op"] == "matmul_bwd":
            s["grad_out"] = normal(P, case["N"], dtype=dt)
    elif case["op"] == "matmul_w4":
        s["x"] = normal(T, D, dtype=torch.bfloat16)
        s["qweight"] = torch.randint(0, 256, (E, case["N"], D // 2), generator=g, device=dev, dtype=torch.uint8)
        G = D // case["group"]
        s["scales"] = torch.rand(E, case["N"], G, generator=g, device=dev).add_(0.5).mul_(0.25 * D ** -0.5).bfloat16()
        s["qzeros"] = (torch.randint(4, 12, (E, case["N"], G), generator=g, device=dev, dtype=torch.uint8)
                       if case["zeros"] else None)
    else:
        dt = TYPES[case["dtype"]]
        s["expert_out"] = normal(P, D, dtype=dt)
        if case["op"] == "combine_bwd":
            s["grad_out"] = normal(T, D, dtype=dt)
        if not case["weighted"]:
            s["topk"] = None
    return s


def by_expert(s, rows):
    """[P, n] rows in the maps' order as [E, capacity, n] fp32, zero behind each expert's last,
    and where each expert's rows lie in it."""
    E, first = s["E"], s["offsets"].long()
    at = torch.arange(s["capacity"], device=rows.device)
    inside = at < (first[1:] - first[:-1])[:, None]
    src = (first[:-1, None] + at).clamp(max=rows.shape[0] - 1)
    return torch.where(inside[:, :, None], rows[src.reshape(-1)].float().view(E, s["capacity"], -1), 0.0), inside


def rows_of(s):
    return s["x"][s["p2u"].long() % s["T"]] if s["gather"] else s["x"]


def plain_matmul(s):
    x, inside = by_expert(s, rows_of(s))
    return torch.bmm(x, s["weight"].float().transpose(1, 2))[inside].to(TYPES[s["out"]])


def plain_matmul_bwd(s):
    x, inside = by_expert(s, rows_of(s))
    g, _ = by_expert(s, s["grad_out"])
    grad_x = torch.bmm(g, s["weight"].float())[inside].to(s["x"].dtype)
    return {"grad_x": grad_x, "grad_weight": torch.bmm(g.transpose(1, 2), x).to(TYPES[s["out"]])}


def plain_w4(s):
    p = torch.arange(s["p2u"].numel(), device=s["x"].device)
    expert = torch.searchsorted(s["offsets"].long(), p, right=True) - 1
    q = s["qweight"][expert]
    P, N, half = q.shape
    q = torch.stack((q & 15, q >> 4), dim=3).view(P, N, -1, s["group"]).float()
    q -= 8.0 if s["qzeros"] is None else s["qzeros"][expert].float()[..., None]
    w = (q * s["scales"][expert].float()[..., None]).view(P, N, 2 * half)
    x = s["x"][s["p2u"].long() % s["T"]].float()
    return torch.bmm(w, x[:, :, None])[:, :, 0].to(TYPES[s["out"]])


def plain_combine(s):
    z = s["expert_out"][s["u2p"].long()].float().view(s["K"], s["T"], -1)
    if s["topk"] is not None:
        z = z * s["topk"].t()[:, :, None]
    return z.sum(0).to(s["expert_out"].dtype)


def plain_combine_bwd(s):
    u = s["p2u"].long()
    g = s["grad_out"][u % s["T"]].float()
    if s["topk"] is None:
        return {"grad_expert_out": g.to(s["grad_out"].dtype)}
    w = s["topk"].t().reshape(-1)
    dots = (g * s["expert_out"].float()).sum(1)
    return {"grad_expert_out": (g * w[u][:, None]).to(s["grad_out"].dtype),
            "grad_weights": dots[s["u2p"].long()].view(s["K"], s["T"]).t().contiguous()}


def run(s):
    op = s["op"]
    if own:
        import score_top_expert_gb300.router as R
        if op == "matmul":
            return R.router_expert_matmul(s["x"], s["weight"], s["offsets"], s["p2u"] if s["gather"] else None,
                                          out_dtype=TYPES[s["out"]])
        if op == "matmul_bwd":
            grad_x = R.router_expert_matmul_bwd_input(s["grad_out"], s["weight"], s["offsets"])
            grad_w = R.router_expert_matmul_bwd_weight(s["grad_out"], s["x"], s["offsets"],
                                                       s["p2u"] if s["gather"] else None,
                                                       out_dtype=TYPES[s["out"]])
            return {"grad_x": grad_x, "grad_weight": grad_w}
        if op == "matmul_w4":
            return R.router_expert_matmul_w4(s["x"], s["qweight"], s["scales"], s["offsets"], s["p2u"],
                                             zeros=s["qzeros"], out_dtype=TYPES[s["out"]])
        if op == "combine":
            return R.router_combine_fwd(s["expert_out"], s["u2p"], s["K"], s["topk"])
        grad_z, grad_w = R.router_combine_bwd(s["grad_out"], s["u2p"], s["K"],
                                              s["expert_out"] if s["topk"] is not None else None, s["topk"])
        return {"grad_expert_out": grad_z} if grad_w is None else {"grad_expert_out": grad_z, "grad_weights": grad_w}
    return {"matmul": plain_matmul, "matmul_bwd": plain_matmul_bwd, "matmul_w4": plain_w4,
            "combine": plain_combine, "combine_bwd": plain_combine_bwd}[op](s)


def exact(case, seed):
    """The definitions, expert by expert or choice by choice, in 64 bits."""
    s = prepare(case, seed)
    T, E, K, D, P = s["T"], s["E"], s["K"], s["D"], s["T"] * s["K"]
    first = s["offsets"].tolist()
    dev = s["offsets"].device
    f64 = {"dtype": torch.float64, "device": dev}
    if s["op"] == "combine":
        out = torch.zeros(T, D, **f64)
        for k in range(K):
            z = s["expert_out"].index_select(0, s["u2p"][k * T:(k + 1) * T]).double()
            out += z if s["topk"] is None else z * s["topk"][:, k:k + 1].double()
        return out
    if s["op"] == "combine_bwd":
        grad_z, grad_w = torch.zeros(P, D, **f64), torch.zeros(T, K, **f64)
        for k in range(K):
            at, g = s["u2p"][k * T:(k + 1) * T].long(), s["grad_out"].double()
            if s["topk"] is not None:
                grad_w[:, k] = torch.einsum("td,td->t", g, s["expert_out"][at].double())
                g = g * s["topk"][:, k:k + 1].double()
            grad_z.index_copy_(0, at, g)
        return {"grad_expert_out": grad_z} if s["topk"] is None else {"grad_expert_out": grad_z, "grad_weights": grad_w}
    N = s["N"]
    out = torch.zeros(P, N, **f64)
    if s["op"] == "matmul_bwd":
        grad_x, grad_w = torch.zeros(P, D, **f64), torch.zeros(E, N, D, **f64)
    for e in range(E):
        a, b = first[e], first[e + 1]
        if a == b:
            continue
        token = s["p2u"][a:b].long().remainder(T)
        if s["op"] == "matmul_w4":
            w = torch.zeros(N, D, **f64)
            w[:, 0::2] = s["qweight"][e].bitwise_and(15).double()
            w[:, 1::2] = s["qweight"][e].bitwise_right_shift(4).double()
            zero = torch.full((N, D // s["group"]), 8.0, **f64) if s["qzeros"] is None else s["qzeros"][e].double()
            w = (w - zero.repeat_interleave(s["group"], 1)) * s["scales"][e].double().repeat_interleave(s["group"], 1)
        else:
            w = s["weight"][e].double()
        x = s["x"][token].double() if s.get("gather", True) else s["x"][a:b].double()
        if s["op"] == "matmul_bwd":
            g = s["grad_out"][a:b].double()
            grad_x[a:b] = g @ w
            grad_w[e] = g.t() @ x
        else:
            out[a:b] = x @ w.t()
    return {"grad_x": grad_x, "grad_weight": grad_w} if s["op"] == "matmul_bwd" else out
