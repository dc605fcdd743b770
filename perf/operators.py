"""The operators around the mixture-of-experts layer, as cases to be measured.

Three operators: routing (``route``), the norms before and after a block with
its gate and residual (``norm``), and the 8-bit linear product (``linear``).
Each case runs in its plain form (elementary torch operations, 32 bits or
more) or, with ``own`` set, through the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # the routing of one decoded token of the decode-shaped layer (latency)
        {"name": "route one token", "op": "route", "T": 1, "E": 128, "k": 8, "dtype": "f32", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "renormalize": True, "scale": 1.0,
         "masked": False},
        # a decode batch of the large layer: sigmoid scores, balance bias, half of eight groups
        {"name": "route decode groups", "op": "route", "T": 64, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "renormalize": True,
         "scale": 2.5, "masked": False},
        # a ragged chunk, many small experts, 16-bit logits with masked experts and one token without any
        {"name": "route ragged masked", "op": "route", "T": 1027, "E": 300, "k": 16, "dtype": "bf16",
         "score": "softmax", "bias": False, "groups": 6, "top_groups": 3, "group_best": 1, "renormalize": False,
         "scale": 1.0, "masked": True},
        # a prefill chunk of the large layer
        {"name": "route prefill groups", "op": "route", "T": 16384, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "renormalize": True,
         "scale": 2.5, "masked": False},
        # between two blocks, one decoded token of the large layer (latency)
        {"name": "norm one token", "op": "norm", "T": 1, "H": 7168, "dtype": "bf16", "residual": "bf16",
         "kind": "rms", "after": True, "before": True, "gate": "none", "sigmoid": False, "offset": 0.0,
         "norm_bias": False, "res_scale": 1.0, "out_scale": 1.0},
        # a decode batch: layer-scale gate for each channel, weights stored as an offset from one
        {"name": "norm decode channel gate", "op": "norm", "T": 64, "H": 2048, "dtype": "f16", "residual": "f16",
         "kind": "rms", "after": True, "before": True, "gate": "channel", "sigmoid": False, "offset": 1.0,
         "norm_bias": False, "res_scale": 1.0, "out_scale": 0.22},
        # a width that is no multiple of a vector: layer norms with biases, a sigmoid gate for each element
        {"name": "norm odd width", "op": "norm", "T": 1027, "H": 1001, "dtype": "f32", "residual": "f32",
         "kind": "layer", "after": True, "before": True, "gate": "element", "sigmoid": True, "offset": 0.0,
         "norm_bias": True, "res_scale": 0.7, "out_scale": 1.3},
        # a prefill chunk of the large layer with the residual stream kept in 32 bits
        {"name": "norm prefill", "op": "norm", "T": 16384, "H": 7168, "dtype": "bf16", "residual": "f32",
         "kind": "rms", "after": True, "before": True, "gate": "token", "sigmoid": True, "offset": 0.0,
         "norm_bias": False, "res_scale": 1.0, "out_scale": 1.0},
        # one decoded token through a projection of the large layer: a stream of weights
        {"name": "linear one token", "op": "linear", "M": 1, "N": 2048, "K": 7168, "dtype": "bf16",
         "quantize": True, "bias": False},
        # a decode batch, its codes shared by several projections
        {"name": "linear decode", "op": "linear", "M": 64, "N": 4096, "K": 2048, "dtype": "bf16",
         "quantize": False, "bias": False},
        # odd sizes in every direction
        {"name": "linear odd", "op": "linear", "M": 777, "N": 1003, "K": 1999, "dtype": "f16",
         "quantize": True, "bias": True},
        # a prefill chunk through a square projection of the large layer
        {"name": "linear prefill", "op": "linear", "M": 4096, "N": 7168, "K": 7168, "dtype": "bf16",
         "quantize": True, "bias": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, its logarithm even."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "norm", "linear"])
    if op == "route":
        E = rng.choice([8, 20, 64, 96, 128, 160, 256, 300, 512, 1000])
        groups = rng.choice([g for g in (1, 2, 4, 5, 8) if E % g == 0 and E // g >= 2])
        top_groups = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        return {"op": op, "T": min(_spread(rng, 1, 16384), 16384 * 256 // E), "E": E, "k": k,
                "dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups,
                "group_best": rng.choice([1, 2]), "renormalize": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.random() < 0.3}
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        H = rng.choice([_spread(rng, 64, 16384), 128 * rng.randint(1, 128)])
        kind = rng.choice(["rms", "rms", "layer"])
        after, before = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        gate = rng.choice(["none", "token", "channel", "element"])
        return {"op": op, "T": min(_spread(rng, 1, 16384), 16384 * 4096 // H), "H": H, "dtype": dtype,
                "residual": rng.choice([dtype, "f32"]), "kind": kind, "after": after, "before": before,
                "gate": gate, "sigmoid": gate != "none" and rng.random() < 0.5, "offset": rng.choice([0.0, 1.0]),
                "norm_bias": kind == "layer" and rng.random() < 0.5, "res_scale": rng.choice([1.0, 0.9]),
                "out_scale": rng.choice([1.0, 0.25])}
    N, K = _spread(rng, 16, 8192), _spread(rng, 64, 8192)
    if rng.random() < 0.5:
        N, K = -(-N // 64) * 64, -(-K // 64) * 64
    return {"op": op, "M": _spread(rng, 1, 3000), "N": N, "K": K, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
            "quantize": rng.random() < 0.6, "bias": rng.random() < 0.3}


def _rows(n, k):
    """int8 [n, k] whose rows start at multiples of 16 bytes, as the quantizer lays codes out."""
    return torch.zeros((n, -(-k // 16) * 16), dtype=torch.int8, device="cuda")[:, :k]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        # router logits of uneven experts
        logits = 1.5 * normal(T, E) + 0.7 * normal(E)
        if case["masked"]:
            logits[torch.rand((T, E), generator=gen, device="cuda") < 0.1] = -math.inf
            logits[T // 2] = -math.inf
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["bias"] = 0.1 * normal(E) if case["bias"] else None
    elif case["op"] == "norm":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        spread = torch.exp(0.5 * normal(H))  # some channels are larger than others
        s["y"] = (0.7 * spread * normal(T, H) + 0.05).to(dt)
        s["r"] = (2.0 * spread * normal(T, H)).to(DTYPES[case["residual"]])
        for name in ("after", "before"):
            s[name] = (1.0 - case["offset"] + 0.2 * normal(H)).to(dt) if case[name] else None
            s[name + "_bias"] = (0.1 * normal(H)).to(dt) if case[name] and case["norm_bias"] else None
        shape = {"none": None, "token": (T, 1), "channel": (H,), "element": (T, H)}[case["gate"]]
        s["gate"] = normal(*shape).to(dt) if shape else None
    else:
        M, N, K, dt = case["M"], case["N"], case["K"], DTYPES[case["dtype"]]
        w = _rows(N, K)
        w.copy_((40.0 * normal(N, K)).round().clamp_(-127, 127))
        s["w"], s["w_scale"] = w, 1e-4 * torch.exp(0.3 * normal(N))
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
        x = normal(M, K) * torch.exp(0.5 * normal(K))  # activations with larger channels
        if case["quantize"]:
            s["x"] = x.to(dt)
        else:
            a = _rows(M, K)
            scale = x.abs().amax(1) / 127
            a.copy_((x / scale[:, None]).round().clamp_(-127, 127))
            s["a"], s["a_scale"] = a, scale
    return s


# --- plain forms ---------------------------------------------------------------

def _route(s, c):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double()
    score = torch.sigmoid(l)
    if c["score"] == "softmax":
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        z = e.sum(1, keepdim=True)
        score = e / torch.where(z > 0, z, 1.0)
    value = score + s["bias"].double() if c["bias"] else score
    rank = value if c["bias"] else l
    open_ = l > -math.inf
    if G > 1:
        # the best one or two open values of each group; a group without any is last
        best = torch.where(open_, value, -math.inf).view(T, G, E // G).sort(dim=2, descending=True).values
        best = best[:, :, :c["group_best"]]
        total = torch.where(best > -math.inf, best, 0.0).sum(2)
        total = torch.where(best[:, :, 0] > -math.inf, total, -math.inf)
        kept = total.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        chosen = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        open_ = open_ & chosen.repeat_interleave(E // G, dim=1)
    ids = torch.where(open_, rank, -math.inf).sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids) * open_.gather(1, ids)
    if c["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return ids.int(), (w * c["scale"]).float()


def _normed(v, weight, bias, c):
    if c["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    v = v * (weight.float() + c["offset"])
    return v if bias is None else v + bias.float()


def _norm(s, c):
    d = s["y"].float()
    if c["after"]:
        d = _normed(d, s["after"], s["after_bias"], c)
    if s["gate"] is not None:
        g = s["gate"].float()
        d = d * (torch.sigmoid(g) if c["sigmoid"] else g)
    r = c["res_scale"] * s["r"].float() + c["out_scale"] * d
    h = _normed(r, s["before"], s["before_bias"], c).to(s["y"].dtype) if c["before"] else None
    return r.to(s["r"].dtype), h


def _linear(s, c):
    if c["quantize"]:
        x = s["x"].float()
        top = x.abs().amax(1, keepdim=True)
        some = top >= 2.0 ** -119
        most = torch.full_like(top, 127.0)  # a tensor: a number on either side of / may become a reciprocal
        top = torch.where(some, top, most)
        a = torch.where(some, (x * torch.div(most, top)).round(), 0.0)
        a_scale = torch.div(top, most)[:, 0]
    else:
        a, a_scale = s["a"], s["a_scale"]
    # the sum of products is a whole number past 24 bits: 64 bits hold it
    acc = a.double() @ s["w"].double().t()
    out = acc * a_scale.double()[:, None] * s["w_scale"].double()
    if c["bias"]:
        out = out + s["bias"].double()
    return out.to(DTYPES[c["dtype"]])


# --- the framework's calls -----------------------------------------------------

def _own(s, c):
    from nvfp4_token_quant_amd import binding
    # the router's rule and the norms' weights are objects that a program makes once and keeps
    if c["op"] == "route":
        if "router" not in s:
            s["router"] = binding.Router(score=c["score"], groups=c["groups"], top_groups=c["top_groups"],
                                         group_best=c["group_best"], renormalize=c["renormalize"], scale=c["scale"])
        return binding.route(s["logits"], c["k"], s["router"], bias=s["bias"])
    if c["op"] == "norm":
        if "norms" not in s:
            s["norms"] = {n: binding.Norm(s[n], s[n + "_bias"], kind=c["kind"], eps=1e-6, offset=c["offset"])
                          if c[n] else None for n in ("before", "after")}
        return binding.block_norm(s["r"], s["y"], before=s["norms"]["before"], after=s["norms"]["after"],
                                  gate=s["gate"], gate_sigmoid=c["sigmoid"], res_scale=c["res_scale"],
                                  out_scale=c["out_scale"])
    if c["quantize"]:
        return binding.int8_linear(s["x"], s["w"], s["w_scale"], bias=s["bias"])
    return binding.int8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], bias=s["bias"],
                               out_dtype=DTYPES[c["dtype"]])


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"route": _route, "norm": _norm, "linear": _linear}[c["op"]](state, c)


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * SIZES[case["dtype"]] + 4 * E * case["bias"] + 8 * T * k, "flops": 20 * T * E}
    if case["op"] == "norm":
        T, H, b, rb = case["T"], case["H"], SIZES[case["dtype"]], SIZES[case["residual"]]
        g = {"none": 0, "token": T, "channel": H, "element": T * H}[case["gate"]]
        weights = H * (case["after"] + case["before"]) * (1 + case["norm_bias"])
        return {"bytes": T * H * (b + 2 * rb + b * case["before"]) + b * (g + weights), "flops": 14 * T * H}
    M, N, K, b = case["M"], case["N"], case["K"], SIZES[case["dtype"]]
    return {"bytes": M * K * (b if case["quantize"] else 1) + 4 * M * (not case["quantize"]) + N * K + 4 * N
            + 4 * N * case["bias"] + M * N * b, "flops": 2 * M * N * K}


# --- the definitions in 64 bits ------------------------------------------------

def _exact_route(s, c):
    """Token by token in numpy: ids have no such value, the weights have."""
    l = s["logits"].double().cpu().numpy()
    b = s["bias"].double().cpu().numpy() if c["bias"] else None
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    out = np.zeros((T, k))
    for t in range(T):
        some = np.flatnonzero(np.isfinite(l[t]))
        if some.size == 0:
            continue
        p = np.zeros(E)
        if c["score"] == "softmax":
            p[some] = np.exp(l[t, some] - l[t, some].max())
            p /= p.sum()
        else:
            p[some] = 1.0 / (1.0 + np.exp(-l[t, some]))
        v = p if b is None else p + b
        if G > 1:
            group = some // (E // G)
            scores = {g: np.sort(v[some[group == g]])[::-1][:c["group_best"]].sum() for g in set(group.tolist())}
            keep = sorted(scores, key=lambda g: (-scores[g], g))[:c["top_groups"]]
            some = some[np.isin(group, keep)]
        order = l[t] if b is None else v
        ids = some[np.lexsort((some, -order[some]))][:k]
        w = p[ids]
        if c["renormalize"] and w.sum() > 0:
            w = w / w.sum()
        out[t, :ids.size] = c["scale"] * w
    return None, out


def _exact_norm(s, c):
    def one(v, w, b):
        mean = v.mean(1, keepdim=True) if c["kind"] == "layer" else 0.0
        var = torch.square(v - mean).mean(1, keepdim=True)
        v = (v - mean) * torch.rsqrt(var + 1e-6) * (c["offset"] + w.double())
        return v if b is None else v + b.double()

    y, r = s["y"].double(), s["r"].double()
    n = one(y, s["after"], s["after_bias"]) if c["after"] else y
    if c["gate"] != "none":
        g = s["gate"].double()
        g = 1.0 / (1.0 + torch.exp(-g)) if c["sigmoid"] else g
        n = n * g
    r = r * c["res_scale"] + n * c["out_scale"]
    return r, one(r, s["before"], s["before_bias"]) if c["before"] else None


def _exact_linear(s, c):
    w = s["w"].double() * s["w_scale"].double()[:, None]
    if c["quantize"]:
        # a code is the nearest whole number to x times the 32-bit number 127 / max|x|, that product in 32 bits
        x = s["x"].double()
        top = x.abs().max(dim=1, keepdim=True).values
        none = top < 2.0 ** -119
        factor = torch.where(none, 0.0, 127.0 / top.clamp(min=2.0 ** -119)).float().double()
        q = torch.round((x * factor).float().double())
        a = q * torch.where(none, 1.0, top / 127.0).float().double()
    else:
        a = s["a"].double() * s["a_scale"].double()[:, None]
    out = torch.mm(a, w.t())
    return out + s["bias"].double() if c["bias"] else out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "linear": _exact_linear}[case["op"]](s, case)
