"""Workloads of the operators around a quantised projection: low-rank adapters of many requests added to its
output, and the norms before and after a block fused with the block's gate and residual.

``run`` computes them in plain torch operations, or, with ``own`` set, through the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------------------------------------ cases

def _lora(name, tokens, d_in, d_out, n_adapters, rank, requests, dtype="bf16", mixed=False, none=False,
          y_in=True):
    return {"op": "lora", "name": name, "tokens": tokens, "d_in": d_in, "d_out": d_out, "n_adapters": n_adapters,
            "rank": rank, "requests": requests, "dtype": dtype, "mixed": mixed, "none": none, "y_in": y_in}


def _norm(name, rows, d, y="fp32", r="bf16", h="bf16", w="bf16", post="rms", pre="rms", gate="none",
          act="linear", residual_scale=1.0, branch_scale=1.0, weight_offset=0.0, bias=False):
    return {"op": "norm", "name": name, "rows": rows, "d": d, "y": y, "r": r, "h": h, "w": w, "post": post,
            "pre": pre, "gate": gate, "act": act, "residual_scale": residual_scale, "branch_scale": branch_scale,
            "weight_offset": weight_offset, "bias": bias}


def listed():
    return [
        # one request in decode beside the 3-bit 4096 x 4096 projection: latency only
        _lora("lora_1tok_4096_r16", 1, 4096, 4096, 8, 16, 1, dtype="fp16"),
        # a decode batch at the 3-bit projection's largest token count, every request with its own adapter,
        # adapters of several ranks in one pool, one request without an adapter
        _lora("lora_16tok_4096_r64_mixed", 16, 4096, 4096, 15, 64, 16, dtype="fp16", mixed=True, none=True),
        # a large decode batch beside the up projection, several requests on each adapter, in no order
        _lora("lora_200tok_12288_r32", 200, 4096, 12288, 48, 32, 200),
        # a short ragged prefill: odd token count, unequal request lengths, some without an adapter
        _lora("lora_777tok_5120_r48_ragged", 777, 5120, 4104, 12, 48, 13, mixed=True, none=True),
        # prefill beside the down projection: a long reduction, a middling rank
        _lora("lora_4096tok_down_r64", 4096, 12288, 4096, 8, 64, 24),
        # prefill beside the widest projection, the largest call: the output's traffic leads
        _lora("lora_8192tok_17408_r16", 8192, 5120, 17408, 16, 16, 40, none=True),
        # one token of decode through the close of a block and the norm of the next: latency only
        _norm("norm_1row_4096", 1, 4096),
        # a decode batch with a gate per channel and a scaled residual, feeding the 3-bit projection in fp16
        _norm("norm_16row_5120_gate", 16, 5120, r="fp16", h="fp16", w="fp16", gate="channel",
              residual_scale=0.5, branch_scale=1.5),
        # prefill: the up projection's input from the down projection's fp32 output, post- and pre-norm
        _norm("norm_4096row_4096_sandwich", 4096, 4096, weight_offset=1.0),
        # prefill, the norm before a block alone
        _norm("norm_8192row_5120_pre", 8192, 5120, y="none", post="none"),
        # layer norms with biases and a sigmoid gate per element, wide rows, fp32 stream
        _norm("norm_2048row_12288_layer", 2048, 12288, r="fp32", h="bf16", w="fp32", post="layer", pre="layer",
              gate="element", act="sigmoid", bias=True),
        # odd width and rows: no 16-byte alignment anywhere
        _norm("norm_1531row_4097_odd", 1531, 4097, y="bf16", r="bf16", gate="element", act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {"lora": max(_cost(c) for c in listed() if c["op"] == "lora"),
            "norm": max(_cost(c) for c in listed() if c["op"] == "norm")}
    while True:
        if rng.random() < 0.5:
            tokens = _log(rng, 1, 8192)
            n = _log(rng, 1, 64)
            c = _lora("", tokens, 32 * _log(rng, 8, 384), 8 * _log(rng, 32, 2176), n, 8 * rng.randint(1, 16),
                      min(tokens, tokens if tokens <= 64 else _log(rng, 1, tokens)), rng.choice(["bf16", "fp16"]),
                      rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.8)
        else:
            post = rng.choice(["none", "rms", "rms", "layer"])
            y = rng.choice(["none", "fp32", "fp32", "bf16", "fp16"])
            c = _norm("", _log(rng, 1, 8192), _log(rng, 64, 16384) if rng.random() < 0.4 else 64 * _log(rng, 1, 256),
                      y, rng.choice(["bf16", "fp16", "fp32"]), rng.choice(["bf16", "fp16", "fp32"]),
                      rng.choice(["bf16", "fp16", "fp32"]), post if y != "none" else "none",
                      rng.choice(["rms", "rms", "layer"]),
                      rng.choice(["none", "none", "channel", "element"]) if y != "none" else "none",
                      rng.choice(["linear", "sigmoid", "silu"]), rng.choice([1.0, 0.5, 0.22]),
                      rng.choice([1.0, 1.5, 0.3]), rng.choice([0.0, 1.0]), rng.random() < 0.4)
        if _cost(c) <= most[c["op"]]:
            c.pop("name")
            return c


def _ranks(case):
    """Rank of each adapter: all the pool's, or a mix of smaller ones beside it (never one alone below 1)."""
    r = case["rank"]
    if not case["mixed"]:
        return [r] * case["n_adapters"]
    return [max(1, v) for v in ([r, r // 2, r // 4, r - 3] * case["n_adapters"])[: case["n_adapters"]]]


def _request_adapters(case):
    """Adapter of each request: every adapter in turn, and -1 (the base model alone) as one more of them."""
    slots = list(range(case["n_adapters"])) + ([-1] if case["none"] else [])
    return [slots[i % len(slots)] for i in range(case["requests"])]


def work(case):
    if case["op"] == "lora":
        t, k, n = case["tokens"], case["d_in"], case["d_out"]
        ranks, req = _ranks(case), _request_adapters(case)
        used = sum(ranks[g] for g in set(req) if g >= 0)
        mean = sum(ranks[g] for g in req if g >= 0) / len(req)          # requests of equal length on average
        return {"bytes": 2 * t * k + (8 if case["y_in"] else 4) * t * n + 2 * used * (k + n) + 4 * t,
                "flops": 2 * t * mean * (k + n) + t * n}
    e = case["rows"] * case["d"]
    per = SIZE[case["r"]] + SIZE[case["h"]]
    flops = 5
    if case["y"] != "none":
        per += SIZE[case["y"]] + SIZE[case["r"]] + (SIZE[case["y"]] if case["gate"] == "element" else 0)
        flops += 10
    vectors = (case["post"] != "none") + 1
    return {"bytes": e * per + case["d"] * SIZE[case["w"]] * vectors * (2 if case["bias"] else 1), "flops": flops * e}


def _cost(case):
    """What bounds a drawn case: its traffic, and for adapters the plain form's product over all of the pool."""
    if case["op"] == "norm":
        return case["rows"] * case["d"]
    t, k, n = case["tokens"], case["d_in"], case["d_out"]
    return t * n * 8 + t * k * 2 + 2 * t * (k + n) * case["n_adapters"] * case["rank"] / 4000


# ------------------------------------------------------------------------------------------------ inputs

def _student(gen, *shape):
    """Student-t(3) values, the heavy tails of activations."""
    z = torch.randn((4,) + shape, generator=gen, device="cuda")
    return z[0] / ((z[1] ** 2 + z[2] ** 2 + z[3] ** 2) / 3).sqrt_().clamp_(min=1e-2)


def _activations(gen, rows, d):
    """Student-t values, one channel in a hundred 50 times as large."""
    x = _student(gen, rows, d)
    hot = torch.randperm(d, generator=gen, device="cuda")[: max(1, d // 100)]
    x[:, hot] *= 50
    return x.clamp_(-30000, 30000)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    if case["op"] == "lora":
        t, k, n, na, r = (case[x] for x in ("tokens", "d_in", "d_out", "n_adapters", "rank"))
        dt = DTYPES[case["dtype"]]
        # requests of unequal lengths, one after the other; each has its adapter
        req = torch.tensor(_request_adapters(case), dtype=torch.int32, device="cuda")
        order = torch.randperm(len(req), generator=gen, device="cuda")
        cuts = torch.randperm(t - 1, generator=gen, device="cuda")[: len(req) - 1].sort().values + 1 if t > 1 else \
            torch.empty(0, dtype=torch.int64, device="cuda")
        which = torch.searchsorted(cuts, torch.arange(t, device="cuda"), right=True)
        s = {"x": _activations(gen, t, k).to(dt),
             "adapter": req[order][which].contiguous(),
             "a": (torch.randn(na, r, k, generator=gen, device="cuda") / math.sqrt(k)).to(dt),
             "b": (torch.randn(na, n, r, generator=gen, device="cuda") * 0.05).to(dt),
             "ranks": torch.tensor(_ranks(case), dtype=torch.int32, device="cuda") if case["mixed"] else None,
             "scale": torch.rand(na, generator=gen, device="cuda") + 0.5,
             "y_in": torch.randn(t, n, generator=gen, device="cuda") * 4 if case["y_in"] else None,
             "y": torch.empty(t, n, device="cuda"), "workspace": None}
        return {"case": case, **s}
    rows, d = case["rows"], case["d"]
    w = lambda: (torch.rand(d, generator=gen, device="cuda") + 0.5 - case["weight_offset"]).to(DTYPES[case["w"]])  # noqa: E731
    b = lambda: (torch.randn(d, generator=gen, device="cuda") * 0.1).to(DTYPES[case["w"]])  # noqa: E731
    has = case["y"] != "none"
    s = {"y": (_student(gen, rows, d) * 3).to(DTYPES[case["y"]]) if has else None,
         "r": _activations(gen, rows, d).to(DTYPES[case["r"]]),
         "gate": None, "post_weight": None, "post_bias": None, "pre_weight": w(),
         "pre_bias": b() if case["bias"] else None}
    if case["gate"] != "none":
        s["gate"] = torch.randn(*((rows, d) if case["gate"] == "element" else (d,)), generator=gen,
                                device="cuda").to(DTYPES[case["y"]])
    if case["post"] != "none":
        s["post_weight"] = w()
        s["post_bias"] = b() if case["bias"] else None
    s["r_out"] = torch.empty_like(s["r"]) if has else None
    s["h"] = torch.empty(rows, d, dtype=DTYPES[case["h"]], device="cuda")
    return {"case": case, **s}


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    if s["case"]["op"] == "lora":
        return _run_lora_own(s) if own else _run_lora(s)
    return _run_norm_own(s) if own else _run_norm(s)


def _run_lora(s):
    """Every token meets the whole pool; what belongs to other adapters, or to padding, is masked out."""
    c = s["case"]
    na, r, k, n = c["n_adapters"], c["rank"], c["d_in"], c["d_out"]
    live = torch.arange(r, device="cuda") < (s["ranks"][:, None] if s["ranks"] is not None else r)     # [na | 1, r]
    live = live.expand(na, r)
    mine = s["adapter"][:, None, None] == torch.arange(na, device="cuda")[:, None]
    mine = (mine & live).reshape(-1, na * r)
    low = s["x"].float() @ s["a"].float().reshape(na * r, k).T
    low = torch.where(mine, low * s["scale"].repeat_interleave(r), 0.0)
    up = torch.where(live[:, None, :], s["b"].float(), 0.0).permute(0, 2, 1).reshape(na * r, n)
    y = low @ up
    return {"y": y + s["y_in"] if s["y_in"] is not None else y}


def _run_lora_own(s):
    import activation_quantization_b200 as aq
    c = s["case"]
    if s["workspace"] is None:
        size = aq.wush_lora_workspace_bytes(c["tokens"], c["d_in"], c["d_out"], c["n_adapters"], c["rank"])
        s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    aq.wush_lora_add(s["x"], s["adapter"], s["a"], s["b"], s["y_in"], s["y"], s["workspace"], ranks=s["ranks"],
                     scale=s["scale"])
    return {"y": s["y"]}


EPS = 1e-6


def _plain_norm(v, kind, weight, bias, offset):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * (weight.float() + offset)
    return v if bias is None else v + bias.float()


def _run_norm(s):
    c = s["case"]
    out = s["r"].float()
    if s["y"] is not None:
        u = _plain_norm(s["y"].float(), c["post"], s["post_weight"], s["post_bias"], c["weight_offset"])
        if s["gate"] is not None:
            g = s["gate"].float()
            if c["act"] != "linear":
                sg = 1 / (1 + torch.exp(-g))
                g = sg if c["act"] == "sigmoid" else g * sg
            u = u * g
        out = c["residual_scale"] * out + c["branch_scale"] * u
    h = _plain_norm(out, c["pre"], s["pre_weight"], s["pre_bias"], c["weight_offset"]).to(DTYPES[c["h"]])
    return {"h": h, "r_out": out.to(DTYPES[c["r"]])} if s["y"] is not None else {"h": h}


def _run_norm_own(s):
    import activation_quantization_b200 as aq
    c = s["case"]
    if s["y"] is None:
        aq.wush_norm(s["r"], s["h"], c["pre"], s["pre_weight"], s["pre_bias"], eps=EPS,
                     weight_offset=c["weight_offset"])
        return {"h": s["h"]}
    aq.wush_residual_norm(s["y"], s["r"], s["r_out"], s["h"], post=c["post"], post_weight=s["post_weight"],
                          post_bias=s["post_bias"], gate=s["gate"], gate_act=c["act"],
                          residual_scale=c["residual_scale"], branch_scale=c["branch_scale"], pre=c["pre"],
                          pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], eps=EPS,
                          weight_offset=c["weight_offset"])
    return {"h": s["h"], "r_out": s["r_out"]}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        x, adapter = s["x"].double(), s["adapter"].tolist()
        t, n = case["tokens"], case["d_out"]
        y = s["y_in"].double() if s["y_in"] is not None else torch.zeros(t, n, dtype=torch.float64, device="cuda")
        for g in sorted(set(adapter) - {-1}):
            rows = torch.tensor([i for i, v in enumerate(adapter) if v == g], device="cuda")
            k = case["rank"] if s["ranks"] is None else int(s["ranks"][g])
            delta = (x[rows] @ s["a"][g, :k].double().T) @ s["b"][g, :, :k].double().T
            y[rows] += s["scale"][g].double() * delta
        return {"y": y}

    def norm(v, kind, weight, bias):
        if kind == "none":
            return v
        m = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
        rms = ((v - m).square().sum(1, keepdim=True) / v.shape[1] + EPS).sqrt()
        v = (v - m) / rms * (weight.double() + case["weight_offset"])
        return v + bias.double() if bias is not None else v

    out = s["r"].double()
    if s["y"] is not None:
        u = norm(s["y"].double(), case["post"], s["post_weight"], s["post_bias"])
        if s["gate"] is not None:
            g = s["gate"].double()
            u = u * {"linear": g, "sigmoid": g.sigmoid(), "silu": g * g.sigmoid()}[case["act"]]
        out = case["residual_scale"] * out + case["branch_scale"] * u
    h = norm(out, case["pre"], s["pre_weight"], s["pre_bias"])
    return {"h": h, "r_out": out} if s["y"] is not None else {"h": h}
