"""The operators around the routed experts' path, as cases to be measured.

* ``balance``: the load-balancing loss of each sequence of a packed batch and the z loss, from the
  router's logits and its [T, K] choices, with the tokens per expert and the gradient by the
  logits (one training step's forward and backward);
* ``w8``: the experts' products on 8-bit integers, tokens quantised row by row at the call, a
  scale for each token and each output channel of each expert;
* ``norm``: the end of an expert block: the weighted sum of the experts' outputs, the norm behind
  the block, its gate, the residual scale and sum, and the norm before the next block;
  ``norm_bwd`` its gradients.

The plain forms compute in fp32 and round once to the output's type.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-6

# the largest listed cases' cost, which a drawn one does not pass
MOST_FLOPS = 2 * 65536 * 2048 * 1024
MOST_BYTES = 7.2e8


def balance(name, T, E, K, S, pad=0, score="softmax", z=0.0, dtype="f32"):
    return {"name": name, "op": "balance", "T": T, "E": E, "K": K, "S": S, "pad": pad, "score": score, "z": z,
            "dtype": dtype}


def w8(name, T, E, K, D, N, out="bf16", gather=True, dtype="bf16"):
    return {"name": name, "op": "w8", "T": T, "E": E, "K": K, "D": D, "N": N, "dtype": dtype, "out": out,
            "gather": gather}


def norm(name, T, K, D, dtype="bf16", gate="none", post=True, pre=True, save=False, op="norm"):
    return {"name": name, "op": op, "T": T, "K": K, "D": D, "dtype": dtype, "gate": gate, "post": post, "pre": pre,
            "save": save}


def listed():
    return [
        # the last, short sequences of a batch: launches are all that counts
        balance("balance t24 e64 k4", 24, 64, 4, 2),
        # a packed training batch of eight ragged sequences with padding behind them, sigmoid
        # scores (the z term left out, as with that score function)
        balance("balance t8192 e256 k8 s8", 8192, 256, 8, 8, pad=37, score="sigmoid"),
        # the router's headline shape, one sequence, z term
        balance("balance t8192 e2304 k36", 8192, 2304, 36, 1, z=1e-3),
        # a large batch of bf16 logits, sequence by sequence
        balance("balance t65536 e512 k22 s16", 65536, 512, 22, 16, z=1e-3, dtype="bf16"),
        # one decoded token, and a decode batch: the 8-bit weights are all the traffic
        w8("w8 t1 e256 k8", 1, 256, 8, 2048, 1024),
        w8("w8 t32 e256 k8", 32, 256, 8, 2048, 1024),
        # the second product of an expert layer (rows in the maps' order), odd sizes, kept in fp32
        w8("w8 t1003 e512 k22", 1003, 512, 22, 504, 1000, out="f32", gather=False),
        # a prefill batch over many experts
        w8("w8 t8192 e256 k8", 8192, 256, 8, 2048, 1024),
        # one token's end of a block, and a prefill batch's
        norm("norm t1 k8", 1, 8, 2048),
        norm("norm t8192 k8", 8192, 8, 2048, gate="token"),
        # a training step's gradients: a gate for each token; and fp32 rows of odd length with a
        # gate for each value, no norm before the next block
        norm("norm bwd t8192 d2048", 8192, 8, 2048, gate="token", op="norm_bwd"),
        norm("norm bwd f32 t1003 d1001", 1003, 1, 1001, dtype="f32", gate="value", pre=False, op="norm_bwd"),
    ]


def log_int(rng, low, high, step=1):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step))


def draw(rng):
    """One more case: tokens from one to tens of thousands, experts up to the router's largest
    count, rows of any length (8-bit operands mostly in whole 16-byte pieces)."""
    while True:
        op = rng.choice(("balance", "balance", "w8", "w8", "w8", "norm", "norm_bwd"))
        if op == "balance":
            T, E = log_int(rng, 1, 65536), log_int(rng, 4, 2304)
            # (a router that picks every expert has nothing to balance: its gradient is zero)
            case = {"op": op, "T": T, "E": E, "K": min(E - 1, log_int(rng, 1, 36)), "S": min(T, log_int(rng, 1, 64)),
                    "pad": rng.choice((0, rng.randint(0, T // 4))), "score": rng.choice(("softmax", "sigmoid")),
                    "z": rng.choice((0.0, 1e-3)), "dtype": rng.choice(("f32", "bf16"))}
        elif op == "w8":
            E = log_int(rng, 4, 2304)
            step = rng.choice((16, 16, 16, 1))
            case = {"op": op, "T": log_int(rng, 1, 8192), "E": E, "K": min(E, log_int(rng, 1, 36)),
                    "D": log_int(rng, 64, 4096, step), "N": log_int(rng, 64, 4096, rng.choice((8, 1))),
                    "dtype": rng.choice(("bf16", "bf16", "f32")), "out": rng.choice(("bf16", "bf16", "f32")),
                    "gather": rng.random() < 0.6}
        else:
            case = {"op": op, "T": log_int(rng, 1, 16384), "K": log_int(rng, 1, 36),
                    "D": log_int(rng, 64, 8192, rng.choice((8, 8, 1))), "dtype": rng.choice(("bf16", "bf16", "f32")),
                    "gate": rng.choice(("none", "token", "value")), "post": rng.random() < 0.8,
                    "pre": rng.random() < 0.8, "save": rng.random() < 0.5}
        w = work(case)
        if w["flops"] <= MOST_FLOPS and w["bytes"] <= MOST_BYTES and case["T"] * case["K"] <= 1500000 \
                and (op != "w8" or case["T"] * case["K"] <= 200000):
            return case


def active(T, E, K):
    """Experts that T tokens reach, when each picks K of E at random."""
    return E * (1.0 - (1.0 - K / E) ** T)


def work(case):
    T, K, s = case["T"], case["K"], SIZE[case["dtype"]]
    P = T * K
    if case["op"] == "balance":
        E, S = case["E"], case["S"]
        # logits once in each direction, the gradient out, the choices in, the counts out
        return {"bytes": 3 * T * E * s + 4 * P + 4 * S * E + 4 * (S + 1) + 16, "flops": 16.0 * T * E}
    if case["op"] == "w8":
        E, D, N = case["E"], case["D"], case["N"]
        x = (T if case["gather"] else P) * D * s
        maps = 4 * (E + 1) + (4 * P if case["gather"] else 0)
        return {"bytes": x + maps + active(T, E, K) * N * (D + 4) + P * N * SIZE[case["out"]],
                "flops": 2.0 * P * N * D}
    D = case["D"]
    gate = {"none": 0, "token": 4 * T, "value": T * D * s}[case["gate"]]
    weights = 4 * D * (case["post"] + case["pre"])
    stats = 4 * T * (case["post"] + case["pre"])
    rows = T * D * s
    if case["op"] == "norm":
        return {"bytes": P * D * s + 8 * P + gate + weights + rows * (2 + case["pre"]) +
                (rows + stats if case["save"] else 0), "flops": 2.0 * P * D + 8.0 * T * D}
    # the gradients of the sum and (pre) the normed rows, with the rows they belong to, in;
    # those by the residual, the block and the gate out
    reads = rows * (1 + 2 * case["pre"] + (case["post"] or case["gate"] != "none"))
    return {"bytes": reads + stats + 2 * rows + 2 * gate + 2 * weights, "flops": 20.0 * T * D}


class Maker:
    """Inputs from the seed alone."""

    def __init__(self, seed):
        self.dev = torch.device("cuda")
        self.g = torch.Generator(device=self.dev)
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=self.g, device=self.dev).mul_(scale).to(dtype)

    def routed(self, T, E, K):
        """Logits whose experts are not equally liked, and the choices and weights of each token."""
        logits = self.normal(T, E) + self.normal(1, E, scale=0.5)
        weights, choice = logits.softmax(1).topk(K, dim=1)
        return logits, (weights / weights.sum(1, keepdim=True)).contiguous(), choice

    def maps(self, choice, T, E, K):
        """The router's maps: choice (t, k) is the expanded row t + k T, permuted rows go by
        expert, then token."""
        P = T * K
        expert = choice.t().reshape(-1)
        token = torch.arange(P, device=self.dev) % T
        key, by = torch.sort(expert * T + token)
        place = torch.empty_like(by)
        place[by] = torch.arange(P, device=self.dev)
        first = torch.searchsorted(key.div(T, rounding_mode="floor"), torch.arange(E + 1, device=self.dev))
        return first.int(), by.int(), place.int()


def prepare(case, seed):
    m = Maker(seed)
    s = dict(case)
    T, K, dt = case["T"], case["K"], TYPES[case["dtype"]]
    if case["op"] == "balance":
        E, S = case["E"], case["S"]
        logits, _, choice = m.routed(T, E, K)
        s["logits"], s["choice"] = logits.to(dt), choice.int()
        # S sequences of random lengths (some may be empty), padding behind the last one
        cuts = torch.randint(0, T - case["pad"] + 1, (S - 1,), generator=m.g, device=m.dev).sort().values
        ends = torch.tensor([T - case["pad"]], device=m.dev)
        s["seq"] = torch.cat((ends * 0, cuts, ends)).int()
        s["grad_loss"] = torch.rand(2, generator=m.g, device=m.dev).add_(0.5)
        return s
    if case["op"] == "w8":
        E, D, N = case["E"], case["D"], case["N"]
        _, _, choice = m.routed(T, E, K)
        s["offsets"], s["p2u"], _ = m.maps(choice, T, E, K)
        s["capacity"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["x"] = m.normal(T if case["gather"] else T * K, D, dtype=dt)
        s["weight"] = torch.randint(-127, 128, (E, N, D), generator=m.g, device=m.dev, dtype=torch.int8)
        s["weight_scales"] = torch.rand(E, N, generator=m.g, device=m.dev).add_(0.5).mul_(D ** -0.5 / 64)
        return s
    D = case["D"]
    s["gate_values"] = {"none": lambda: None, "token": lambda: torch.rand(T, generator=m.g, device=m.dev),
                        "value": lambda: torch.rand(T, D, generator=m.g, device=m.dev).to(dt)}[case["gate"]]()
    s["post_weight"] = m.normal(D, scale=0.2).add_(1.0) if case["post"] else None
    s["pre_weight"] = m.normal(D, scale=0.2).add_(1.0) if case["pre"] else None
    s["scale"] = 0.5
    if case["op"] == "norm":
        E = max(64, K)
        _, s["topk"], choice = m.routed(T, E, K)
        _, _, s["u2p"] = m.maps(choice, T, E, K)
        s["expert_out"] = m.normal(T * K, D, dtype=dt)
        s["residual"] = m.normal(T, D, dtype=dt, scale=2.0)
        return s
    # what a training forward kept: the block's output, the sum behind it and both norms' factors
    y, residual = m.normal(T, D, dtype=dt, scale=0.7), m.normal(T, D, dtype=dt, scale=2.0)
    s["block"] = y if case["post"] or case["gate"] != "none" else None
    s["rstd"] = torch.ones(T, 2, device=m.dev)
    h = y.float()
    if case["post"]:
        s["rstd"][:, 0] = (h * h).mean(1).add_(EPS).rsqrt_()
        h = h * s["rstd"][:, :1] * s["post_weight"]
    if case["gate"] != "none":
        h = h * (s["gate_values"] if case["gate"] == "value" else s["gate_values"][:, None]).float()
    x = residual.float() + s["scale"] * h
    if case["pre"]:
        s["rstd"][:, 1] = (x * x).mean(1).add_(EPS).rsqrt_()
    s["sum"] = x.to(dt) if case["pre"] else None
    s["grad_sum"] = m.normal(T, D, dtype=dt)
    s["grad_normed"] = m.normal(T, D, dtype=dt) if case["pre"] else None
    return s


def plain_balance(s):
    T, E, K, S = s["T"], s["E"], s["K"], s["S"]
    x, seq = s["logits"].float(), s["seq"].long()
    t = torch.arange(T, device=x.device)
    member = ((t >= seq[:-1, None]) & (t < seq[1:, None])).float()  # [S, T]
    shifted = x - x.amax(1, keepdim=True)
    e = shifted.exp()
    total = e.sum(1, keepdim=True)
    soft = e / total
    sig = 1.0 / (1.0 + (-x).exp())
    norm = sig.sum(1, keepdim=True)
    q = soft if s["score"] == "softmax" else sig / norm
    inside = member.sum(0)
    # each token's choices go to its sequence's counts; those of padding to a row behind them
    row = torch.where(inside > 0, torch.searchsorted(seq[1:], t, right=True).clamp(max=S - 1), S)
    cell = row[:, None] * E + s["choice"].long()
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=x.device)
    counts = counts.index_add_(0, cell.reshape(-1), torch.ones_like(cell, dtype=torch.int32).reshape(-1))
    counts = counts.view(S + 1, E)[:S]
    n = (seq[1:] - seq[:-1]).float()
    factor = 0.01 * E / (S * K) / (n * n).clamp(min=1.0)  # of each sequence
    balance_loss = ((member @ q) * counts.float()).sum(1).mul(factor).sum()
    tokens = inside.sum().clamp(min=1.0)
    lse = (total.log() + x.amax(1, keepdim=True)) * inside[:, None]
    z_loss = s["z"] * (lse * lse).sum() / tokens
    # a constant taken off a row's counts changes nothing: its mean keeps the differences exact
    c = (counts.float() - n[:, None] * K / E) * factor[:, None] * s["grad_loss"][0]
    c = member.t() @ c
    c = c - (c * q).sum(1, keepdim=True)
    grad = c * q if s["score"] == "softmax" else c * sig * (1.0 - sig) / norm
    grad = grad + s["grad_loss"][1] * s["z"] * 2.0 / tokens * lse * soft
    return {"loss": torch.stack((balance_loss, z_loss)), "counts": counts, "grad": grad.to(s["logits"].dtype)}


def plain_quantize(x):
    """Rows in 8 bits: the quotients are rounded in 64 bits, since fp32 makes ties of what is next to one."""
    scales = (x.double().abs().amax(1) / 127.0).float()  # rounded once (a fp32 division by a number is a product)
    scales = torch.where(scales > 0, scales.clamp(min=2.0 ** -126), scales)
    q = torch.where(scales[:, None] > 0, x.double() / scales[:, None].double(), 0.0).round()
    return q.float(), scales


def plain_w8(s):
    q, scales = plain_quantize(s["x"])
    E, first = s["E"], s["offsets"].long()
    source = s["p2u"].long() % s["T"] if s["gather"] else torch.arange(s["p2u"].numel(), device=q.device)
    at = torch.arange(s["capacity"], device=q.device)
    inside = at < (first[1:] - first[:-1])[:, None]
    row = source[(first[:-1, None] + at).clamp(max=source.numel() - 1)]
    x = torch.where(inside[:, :, None], q[row.reshape(-1)].view(E, s["capacity"], -1), 0.0)
    out = torch.bmm(x, s["weight"].float().transpose(1, 2))
    out = out * scales[row][:, :, None] * s["weight_scales"][:, None, :]
    return out[inside].to(TYPES[s["out"]])


def gated(s, v):
    return v if s["gate"] == "none" else v * (s["gate_values"] if s["gate"] == "value" else s["gate_values"][:, None])


def plain_norm(s):
    dt = s["residual"].dtype
    z = s["expert_out"][s["u2p"].long()].float().view(s["K"], s["T"], -1)
    y = (z * s["topk"].t()[:, :, None]).sum(0)
    rstd = torch.ones(s["T"], 2, device=y.device)
    h = y
    if s["post"]:
        rstd[:, 0] = torch.rsqrt((y * y).mean(1) + EPS)
        h = h * rstd[:, :1] * s["post_weight"]
    x = s["residual"].float() + s["scale"] * gated(s, h)
    if s["pre"]:
        rstd[:, 1] = torch.rsqrt((x * x).mean(1) + EPS)
    out = {"sum": x.to(dt)}
    if s["pre"]:
        out["normed"] = (x * rstd[:, 1:] * s["pre_weight"]).to(dt)
    if s["save"]:
        out |= {"block": y.to(dt), "rstd": rstd}
    return out


def plain_norm_bwd(s):
    dt = s["grad_sum"].dtype
    gx, out = s["grad_sum"].float(), {}
    if s["pre"]:
        hat = s["sum"].float() * s["rstd"][:, 1:]
        gn = s["grad_normed"].float()
        u = gn * s["pre_weight"]
        gx = gx + s["rstd"][:, 1:] * (u - hat * (u * hat).mean(1, keepdim=True))
        out["grad_pre_weight"] = (gn * hat).sum(0)
    out["grad_residual"] = gx.to(dt)
    gh = s["scale"] * gated(s, gx)
    if s["block"] is not None:
        hat = s["block"].float() * s["rstd"][:, :1]
        h = hat * s["post_weight"] if s["post"] else hat
        if s["gate"] == "value":
            out["grad_gate"] = (s["scale"] * gx * h).to(dt)
        elif s["gate"] == "token":
            out["grad_gate"] = s["scale"] * (gx * h).sum(1)
    if s["post"]:
        out["grad_post_weight"] = (gh * hat).sum(0)
        v = gh * s["post_weight"]
        gh = s["rstd"][:, :1] * (v - hat * (v * hat).mean(1, keepdim=True))
    out["grad_block"] = gh.to(dt)
    return out


def run(s):
    op = s["op"]
    if own:
        import score_top_expert_gb300.router as R
        if op == "balance":
            loss, counts, stats = R.router_balance_loss_fwd(s["logits"], s["choice"], s["score"], 0.01, s["z"], s["seq"])
            grad = R.router_balance_loss_bwd(s["grad_loss"], s["logits"], counts, stats, s["K"], s["score"], 0.01,
                                             s["z"], s["seq"])
            return {"loss": loss, "counts": counts, "grad": grad}
        if op == "w8":
            q, scales = R.router_quantize_rows(s["x"])
            return R.router_expert_matmul_w8(q, scales, s["weight"], s["weight_scales"], s["offsets"],
                                             s["p2u"] if s["gather"] else None, out_dtype=TYPES[s["out"]])
        if op == "norm":
            x, normed, block, rstd = R.router_combine_norm_fwd(
                s["expert_out"], s["residual"], s["u2p"], s["topk"], post_weight=s["post_weight"],
                gate=s["gate_values"], residual_scale=s["scale"], pre_weight=s["pre_weight"], eps=EPS,
                save=s["save"])
            out = {"sum": x, "normed": normed} if s["pre"] else {"sum": x}
            return out | {"block": block, "rstd": rstd} if s["save"] else out
        grads = R.router_combine_norm_bwd(
            s["grad_sum"], s["grad_normed"], s["block"], s["sum"], s["rstd"], post_weight=s["post_weight"],
            gate=s["gate_values"], residual_scale=s["scale"], pre_weight=s["pre_weight"])
        names = ("grad_block", "grad_residual", "grad_gate", "grad_post_weight", "grad_pre_weight")
        return {name: g for name, g in zip(names, grads) if g is not None}
    return {"balance": plain_balance, "w8": plain_w8, "norm": plain_norm, "norm_bwd": plain_norm_bwd}[op](s)


def exact(case, seed):
    """The definitions, sequence by sequence, expert by expert or row by row, in 64 bits."""
    s = prepare(case, seed)
    return {"balance": exact_balance, "w8": exact_w8, "norm": exact_norm, "norm_bwd": exact_norm_bwd}[s["op"]](s)


def exact_balance(s):
    E, K, S, first = s["E"], s["K"], s["S"], s["seq"].tolist()
    x, g = s["logits"].double(), s["grad_loss"].double()
    grad, counts = torch.zeros_like(x), torch.zeros(S, E, dtype=torch.int32, device=x.device)
    loss = torch.zeros(2, dtype=torch.float64, device=x.device)
    n = max(first[-1] - first[0], 1)
    for i, (a, b) in enumerate(zip(first, first[1:])):
        if a == b:
            continue
        r = x[a:b]
        lse = r.logsumexp(1, keepdim=True)
        soft, sig = (r - lse).exp(), torch.sigmoid(r)
        q = soft if s["score"] == "softmax" else sig / sig.sum(1, keepdim=True)
        c = torch.bincount(s["choice"][a:b].reshape(-1).long(), minlength=E)
        counts[i] = c.int()
        factor = 0.01 * E / (S * K * (b - a) ** 2)
        loss[0] += factor * (q.sum(0) * c).sum()
        loss[1] += s["z"] / n * lse.square().sum()
        by_q = factor * c.double().expand_as(q)
        inner = (by_q * q).sum(1, keepdim=True)
        if s["score"] == "softmax":
            gr = q * (by_q - inner)
        else:
            gr = (by_q - inner) * sig * (1 - sig) / sig.sum(1, keepdim=True)
        grad[a:b] = g[0] * gr + g[1] * s["z"] * 2 / n * lse * soft
    return {"loss": loss, "counts": counts, "grad": grad}


def exact_w8(s):
    x = s["x"].double()
    scales = x.abs().amax(1).div(127).float()  # the operator's scales are fp32 numbers
    scales = torch.where(scales > 0, scales.clamp(min=2.0 ** -126), scales).double()
    q = torch.where(scales[:, None] > 0, torch.round(x / scales[:, None]), torch.zeros_like(x))
    x = q * scales[:, None]
    first = s["offsets"].tolist()
    out = torch.zeros(s["p2u"].numel(), s["N"], dtype=torch.float64, device=x.device)
    for e in range(s["E"]):
        a, b = first[e], first[e + 1]
        if a < b:
            rows = x[s["p2u"][a:b].long().remainder(s["T"])] if s["gather"] else x[a:b]
            w = s["weight"][e].double() * s["weight_scales"][e].double()[:, None]
            out[a:b] = rows @ w.t()
    return out


def exact_norm(s):
    T, K = s["T"], s["K"]
    y = torch.zeros(T, s["D"], dtype=torch.float64, device=s["residual"].device)
    for k in range(K):
        y += s["expert_out"].index_select(0, s["u2p"][k * T:(k + 1) * T]).double() * s["topk"][:, k:k + 1].double()
    r_post, r_pre = torch.ones_like(y[:, :1]), torch.ones_like(y[:, :1])
    h = y
    if s["post"]:
        r_post = 1 / torch.sqrt(y.square().mean(1, keepdim=True) + EPS)
        h = y * r_post * s["post_weight"].double()
    if s["gate"] != "none":
        h = h * s["gate_values"].double().view(T, -1)
    x = s["residual"].double() + s["scale"] * h
    out = {"sum": x}
    if s["pre"]:
        r_pre = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + EPS)
        out["normed"] = x * r_pre * s["pre_weight"].double()
    if s["save"]:
        out |= {"block": y, "rstd": torch.cat((r_post, r_pre), 1)}
    return out


def exact_norm_bwd(s):
    """From the kept rows and factors as they are."""
    T, D = s["grad_sum"].shape
    gx, out = s["grad_sum"].double(), {}
    r = s["rstd"].double()
    if s["pre"]:
        hat = s["sum"].double() * r[:, 1:]
        by_hat = s["grad_normed"].double() * s["pre_weight"].double()
        gx = gx + r[:, 1:] * (by_hat - hat * torch.einsum("td,td->t", by_hat, hat)[:, None] / D)
        out["grad_pre_weight"] = torch.einsum("td,td->d", s["grad_normed"].double(), hat)
    out["grad_residual"] = gx
    gate = s["gate_values"].double().view(T, -1) if s["gate"] != "none" else 1.0
    gh = s["scale"] * gate * gx
    if s["block"] is not None:
        hat = s["block"].double() * r[:, :1]
        h = hat * s["post_weight"].double() if s["post"] else hat
        if s["gate"] != "none":
            by_gate = s["scale"] * gx * h
            out["grad_gate"] = by_gate if s["gate"] == "value" else by_gate.sum(1)
    if s["post"]:
        out["grad_post_weight"] = torch.einsum("td,td->d", gh, hat)
        by_hat = gh * s["post_weight"].double()
        gh = r[:, :1] * (by_hat - hat * torch.einsum("td,td->t", by_hat, hat)[:, None] / D)
    out["grad_block"] = gh
    return out
