"""What is measured of the operators that follow the attention in a decoder layer.

Three operators, each in its plain form (elementary torch operations) and as the call of the
package's entry point:
  norm     r = x + residual; y = r / sqrt(mean(r^2) + eps) * weight; y also in 8 bits (e4m3),
           one scale per 128 channels
  route    scores of the experts from router logits (softmax, sigmoid or sqrt(softplus)), the
           choice of experts by score + bias within the best groups, and their weights
  experts  out[t] = sum_j weights[t,j] * W2_e (silu(W1_e x_t) * W3_e x_t), e = ids[t,j], with the
           gate and up products clamped where a limit is given
``own`` chooses between the two.
"""
import math

import torch

own = False

GROUP = 128          # channels that share a scale of the 8-bit form
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's norm of a single sequence: latency
        dict(name="norm_one_token", op="norm", T=1, hidden=4096, dtype="bf16", residual=True, y=True, q8=False),
        # a prompt of the output projection's width, the residual stream updated
        dict(name="norm_prompt", op="norm", T=16384, hidden=4096, dtype="bf16", residual=True, y=True, q8=False),
        # the same with the 8-bit form beside the 16-bit one, a ragged number of tokens
        dict(name="norm_prompt_8bit", op="norm", T=8191, hidden=4096, dtype="bf16", residual=True, y=True, q8=True),
        # float32 rows of an odd width, no residual
        dict(name="norm_f32_odd", op="norm", T=3001, hidden=1111, dtype="f32", residual=False, y=True, q8=False),
        # a decode batch of 64 sequences
        dict(name="route_decode", op="route", T=64, E=256, k=6, groups=1, groups_kept=1, fn="sqrt_softplus",
             bias=True, renorm=True, dtype="f32"),
        # a prompt, experts in eight groups of which four are kept
        dict(name="route_prompt_groups", op="route", T=16384, E=256, k=8, groups=8, groups_kept=4, fn="sigmoid",
             bias=True, renorm=True, dtype="f32"),
        # softmax scores of 16-bit logits over few experts, an odd number of tokens
        dict(name="route_softmax_odd", op="route", T=4097, E=60, k=4, groups=1, groups_kept=1, fn="softmax",
             bias=False, renorm=False, dtype="bf16"),
        # one token of one sequence: the chosen experts' weights are read once
        dict(name="experts_one_token", op="experts", T=1, hidden=4096, inter=2048, E=64, k=6, limit=10.0, x8=False),
        # a decode batch: nearly every expert has a few rows
        dict(name="experts_decode_batch", op="experts", T=64, hidden=4096, inter=2048, E=64, k=6, limit=10.0, x8=False),
        # a ragged prompt of a narrow layer whose rows arrive in 8 bits
        dict(name="experts_prompt_8bit", op="experts", T=1777, hidden=2048, inter=1408, E=32, k=4, limit=0.0, x8=True),
        # a prompt
        dict(name="experts_prompt", op="experts", T=8192, hidden=4096, inter=2048, E=64, k=6, limit=10.0, x8=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "route", "experts"))
    if op == "norm":
        T = _log_int(rng, 1, 16384)
        hidden = _log_int(rng, 64, 8192)
        if rng.random() < 0.8:
            hidden = -(-hidden // 16) * 16
        while T * hidden > 16384 * 4096:
            T = max(1, T // 2)
        q8 = rng.random() < 0.4
        return dict(op=op, T=T, hidden=hidden, dtype=rng.choice(("bf16", "bf16", "f32")), residual=rng.random() < 0.7,
                    y=not q8 or rng.random() < 0.5, q8=q8)
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        per = rng.randint(8, 64 if groups > 1 else 400)
        kept = rng.randint(1, groups)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=groups * per, k=rng.randint(1, min(12, kept * per)), groups=groups,
                    groups_kept=kept, fn=rng.choice(("softmax", "sigmoid", "sqrt_softplus")), bias=rng.random() < 0.6,
                    renorm=rng.random() < 0.6, dtype=rng.choice(("f32", "f32", "bf16")))
    E = rng.randint(8, 64)
    return dict(op=op, T=_log_int(rng, 1, 6000), hidden=128 * rng.randint(4, 32), inter=16 * rng.randint(16, 128), E=E,
                k=rng.randint(1, 6), limit=rng.choice((0.0, 7.0, 10.0)), x8=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _quantise(v):
    """Rows in e4m3 with a power-of-two scale per 128 channels (hidden is a multiple of 128)."""
    g = v.float().unflatten(1, (-1, GROUP))
    s = torch.exp2(torch.ceil(torch.log2(g.abs().amax(2, keepdim=True).clamp_min(1e-30) / E4M3_MAX)))
    return (g / s).flatten(1).to(torch.float8_e4m3fn), s.squeeze(2).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    s = dict(case=dict(case))
    if case["op"] == "norm":
        t, (T, h) = _dtype(case["dtype"]), (case["T"], case["hidden"])
        # a residual stream: a few channels much larger than the rest
        loud = 1 + 20 * (torch.rand(h, generator=g, device="cuda") < 0.01)
        s["x"] = normal(T, h).to(t)
        s["residual"] = (normal(T, h) * loud).to(t) if case["residual"] else None
        s["weight"] = (1 + normal(h, scale=0.2)).to(t)
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        s["logits"] = (normal(T, E, scale=1.5) + normal(E, scale=0.7)).to(_dtype(case["dtype"]))
        s["bias"] = normal(E, scale=0.1) if case["bias"] else None
    else:
        T, h, f, E, k = case["T"], case["hidden"], case["inter"], case["E"], case["k"]
        x = normal(T, h, dtype=torch.bfloat16)
        s["x"], s["x_scale"] = _quantise(x) if case["x8"] else (x, None)
        # some experts are asked for more often than others
        wanted = normal(T, E) + normal(E, scale=0.5)
        s["ids"] = wanted.topk(k, dim=1).indices.to(torch.int32)
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        s["weights"] = (w / w.sum(1, keepdim=True) * 1.5).contiguous()
        s["w13"] = normal(E, 2 * f, h, dtype=torch.bfloat16, scale=1.5 / math.sqrt(h))
        s["w2"] = normal(E, h, f, dtype=torch.bfloat16, scale=1 / math.sqrt(f))
    return s


# ------------------------------------------------------------------ plain forms

def _plain_norm(c, s):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    out = {}
    if s["residual"] is not None:
        out["res"] = r.to(s["x"].dtype)
    if c["y"]:
        out["y"] = y.to(s["x"].dtype)
    if c["q8"]:
        T, h = y.shape
        n = -(-h // GROUP)
        g = torch.nn.functional.pad(y, (0, n * GROUP - h)).view(T, n, GROUP)
        scale = g.abs().amax(2) / E4M3_MAX
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        q = (g / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        out["q"] = q.view(T, n * GROUP)[:, :h].to(torch.float8_e4m3fn)
        out["scale"] = scale
    return out


def _scores(fn, logits):
    """In 64 bits: the choice of experts hangs on which of two close scores is larger."""
    l = logits.double()
    if fn == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    if fn == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    return torch.sqrt(torch.log1p(torch.exp(-l.abs())) + l.clamp_min(0))


def _plain_route(c, s):
    score = _scores(c["fn"], s["logits"])
    T, E = score.shape
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        by_group = choice.view(T, c["groups"], -1)
        best = by_group.sort(2, descending=True).values[:, :, :2].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["groups_kept"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(keep[:, :, None], by_group, -math.inf).view(T, E)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return {"ids": ids.to(torch.int32), "weights": (w * 1.5).float()}


def _plain_experts(c, s):
    T, h, f, E, k = c["T"], c["hidden"], c["inter"], c["E"], c["k"]
    x = s["x"].float()
    if c["x8"]:
        x = (x.view(T, -1, GROUP) * s["x_scale"][:, :, None]).view(T, h)
    # the (token, choice) pairs sorted by expert, each expert's rows padded to the longest
    expert, order = s["ids"].flatten().long().sort(stable=True)
    count = torch.bincount(expert, minlength=E)
    place = torch.arange(T * k, device=x.device) - (count.cumsum(0) - count)[expert]
    rows = x.new_zeros(E, int(count.max()), h)
    rows[expert, place] = x[order // k]
    gate, up = torch.bmm(rows, s["w13"].float().transpose(1, 2)).split(f, dim=2)
    if c["limit"] > 0:
        gate, up = gate.clamp(max=c["limit"]), up.clamp(-c["limit"], c["limit"])
    act = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(act, s["w2"].float().transpose(1, 2))[expert, place]
    pairs = torch.empty_like(y)
    pairs[order] = y * s["weights"].flatten()[order, None]
    return {"out": pairs.view(T, k, h).sum(1).to(torch.bfloat16)}


# ------------------------------------------------------------------ the package's calls

_FN = {"softmax": 0, "sigmoid": 1, "sqrt_softplus": 2}


def _handle(c, s):
    """Parameters, outputs and workspace, which a program makes once and keeps."""
    from sparse_long_context_csa_b200 import abi
    dev = "cuda"
    p = abi.Dsv4MoeParams()
    p.T, p.eps, p.swiglu_limit, p.routed_scale = c["T"], 1e-6, c.get("limit", 0.0), 1.5
    p.hidden, p.inter, p.E, p.topk = c.get("hidden", 0), c.get("inter", 0), c.get("E", 0), c.get("k", 0)
    p.n_group, p.topk_group, p.score_fn = c.get("groups", 1), c.get("groups_kept", 1), _FN[c.get("fn", "softmax")]
    p.renorm, p.scale_pow2 = int(c.get("renorm", False)), 0
    p.dtype = p.logits_dtype = abi.F32 if c.get("dtype") == "f32" else abi.BF16
    o = {}
    if c["op"] == "norm":
        o["res"] = torch.empty_like(s["x"]) if s["residual"] is not None else None
        o["y"] = torch.empty_like(s["x"]) if c["y"] else None
        o["q"] = torch.empty(s["x"].shape, dtype=torch.float8_e4m3fn, device=dev) if c["q8"] else None
        o["scale"] = torch.empty(c["T"], -(-c["hidden"] // GROUP), device=dev) if c["q8"] else None
    elif c["op"] == "route":
        o["ids"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device=dev)
        o["weights"] = torch.empty(c["T"], c["k"], device=dev)
    else:
        p.dtype = abi.BF16
        o["out"] = torch.empty(c["T"], c["hidden"], dtype=torch.bfloat16, device=dev)
        s["workspace"] = torch.empty(abi.dsv4_expert_mlp_workspace_bytes(p), dtype=torch.uint8, device=dev)
    s["handle"] = (abi, p, o, {n: t for n, t in o.items() if t is not None})


def _own(c, s):
    if "handle" not in s:
        _handle(c, s)
    abi, p, o, out = s["handle"]
    if c["op"] == "norm":
        abi.dsv4_add_rms_norm(p, s["x"], s["residual"], s["weight"], o["res"], o["y"], o["q"], o["scale"])
    elif c["op"] == "route":
        abi.dsv4_route_experts(p, s["logits"], s["bias"], o["ids"], o["weights"])
    else:
        abi.dsv4_expert_mlp(p, s["x"], s["x_scale"], s["ids"], s["weights"], s["w13"], s["w2"], o["out"], s["workspace"])
    return out


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"norm": _plain_norm, "route": _plain_route, "experts": _plain_experts}[c["op"]](c, state)


# ------------------------------------------------------------------ work and 64-bit values

def work(case):
    T = case["T"]
    if case["op"] == "norm":
        n = T * case["hidden"]
        e = 2 if case["dtype"] == "bf16" else 4
        b = n * e * (1 + 2 * case["residual"] + case["y"]) + case["hidden"] * e
        if case["q8"]:
            b += n + T * -(-case["hidden"] // GROUP) * 4
        return {"bytes": b, "flops": 5 * n}
    if case["op"] == "route":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * case["E"] * e + case["E"] * 4 * case["bias"] + T * case["k"] * 8, "flops": 8 * T * case["E"]}
    h, f, E, k = case["hidden"], case["inter"], case["E"], case["k"]
    used = E * (1 - (1 - k / E) ** T)  # experts that someone asks for, were they asked for evenly
    x = T * h * (1 if case["x8"] else 2) + (T * h // GROUP * 4 if case["x8"] else 0)
    return {"bytes": used * 3 * h * f * 2 + x + T * h * 2 + T * k * 8, "flops": 6 * T * k * h * f}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = s["x"].double()
        out = {}
        if case["residual"]:
            r = r.add(s["residual"].double())
            out["res"] = r
        rms = torch.sqrt(torch.linalg.vector_norm(r, dim=1).square() / case["hidden"] + 1e-6)
        y = s["weight"].double() * (r / rms[:, None])
        if case["y"]:
            out["y"] = y
        if case["q8"]:
            scale = torch.stack([b.abs().amax(1) for b in y.split(GROUP, dim=1)], 1) / E4M3_MAX
            scale[scale == 0] = 1.0
            out["q"] = y / scale.repeat_interleave(GROUP, 1)[:, :case["hidden"]]  # before it is rounded to 8 bits
            out["scale"] = scale
        return out
    if case["op"] == "route":
        import numpy as np
        l = s["logits"].double().cpu().numpy()
        b = np.zeros(case["E"]) if s["bias"] is None else s["bias"].double().cpu().numpy()
        if case["fn"] == "softmax":
            score = np.exp(l - np.logaddexp.reduce(l, axis=1, keepdims=True))
        elif case["fn"] == "sigmoid":
            score = 0.5 * (1 + np.tanh(0.5 * l))
        else:
            score = np.sqrt(np.logaddexp(0, l))
        choice = score + b
        T, E = choice.shape
        if case["groups"] > 1:
            g = choice.reshape(T, case["groups"], -1)
            two = np.partition(g, g.shape[2] - 2, axis=2)[:, :, -2:].sum(2)
            rank = np.argsort(np.argsort(-two, axis=1, kind="stable"), axis=1, kind="stable")
            choice = np.where((rank < case["groups_kept"])[:, :, None], g, -np.inf).reshape(T, E)
        ids = np.argsort(-choice, axis=1, kind="stable")[:, :case["k"]]
        w = np.take_along_axis(score, ids, 1)
        if case["renorm"]:
            w = w / (w.sum(1, keepdims=True) + 1e-20)
        return {"ids": ids.astype(np.int32), "weights": torch.from_numpy(1.5 * w)}
    T, h, f = case["T"], case["hidden"], case["inter"]
    x = s["x"].double()
    if case["x8"]:
        x = x * s["x_scale"].double().repeat_interleave(GROUP, 1)
    out = torch.zeros(T, h, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        token, j = (s["ids"] == e).nonzero(as_tuple=True)
        if len(token):
            a = x[token] @ s["w13"][e].double().T
            g, u = a[:, :f], a[:, f:]
            if case["limit"] > 0:
                g, u = torch.clamp_max(g, case["limit"]), torch.clamp(u, -case["limit"], case["limit"])
            v = (g * torch.sigmoid(g) * u) @ s["w2"][e].double().T
            out.index_add_(0, token, v * s["weights"][token, j].double()[:, None])
    return {"out": out}
