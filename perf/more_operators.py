"""What a decoder layer needs between its 16-bit products and its routed experts, as measured cases.

Three operators that follow one another in a serving step:

  norm    the residual's addition and the root-mean-square norm of the sum, in 16 bits and/or in 8 bits
          (e4m3) with a scale a row (moe_rms_norm)
  linear  y = act(x W^T + bias) + residual for x and W in 8 bits with scales a row, x perhaps brought to
          8 bits on the way (moe_linear_8bit, moe_quantize_rows)
  route   the choice of experts: softmax or sigmoid scores, a bias for balance that only the choice sees,
          groups of experts, top-k, weights renormalised and scaled (moe_route_scored)

`run` computes them in elementary torch operations (own = False; in 32 bits, the choice of experts in 64)
or through the library (own = True); `exact` computes them in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-6
LEAST = 1e-30  # a row's largest magnitude counts as at least that much


# ------------------------------------------------------------------ cases

def _norm(name, T, H, dtype="bf16", x32=False, residual=True, y=True, q=False, pad=0):
    c = dict(op="norm", T=T, H=H, dtype=dtype, x32=x32, residual=residual, y=y, q=q, pad=pad)
    return dict(c, name=name) if name else c


def _linear(name, T, K, N, dtype="bf16", act="none", bias=False, residual=False, from16=False, pad=0):
    c = dict(op="linear", T=T, K=K, N=N, dtype=dtype, act=act, bias=bias, residual=residual, from16=from16, pad=pad)
    return dict(c, name=name) if name else c


def _route(name, T, E, k, scoring="sigmoid", bias=True, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0,
           coarse=False):
    c = dict(op="route", T=T, E=E, k=k, scoring=scoring, bias=bias, groups=groups, top_groups=top_groups,
             group_top=group_top, renorm=renorm, scale=scale, coarse=coarse)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the norm ahead of one token's experts (hidden size 4096): nothing but latency
        _norm("norm_decode_1", 1, 4096),
        # 32 users: the experts' fp32 result joins the residual stream, and the next layer's
        # projection reads the norm in 8 bits
        _norm("norm_8bit_decode_32", 32, 4096, x32=True, y=False, q=True),
        # a ragged batch in fp16 with an odd hidden size, rows inside wider buffers, both outputs
        _norm("norm_both_ragged_f16", 333, 2051, "f16", q=True, pad=24),
        # the experts' fp32 result of a batch of prompts: the bytes are all there is
        _norm("norm_8bit_prompt_8192", 8192, 4096, x32=True, y=False, q=True),
        # the fused q, k, v projection (32 query and 8 key heads of 128) of one user's next token
        _linear("linear8_qkv_decode_1", 1, 4096, 6144, bias=True),
        # the projection behind the attention for 32 users: its rows come in 16 bits and go to 8 on the way
        _linear("linear8_out_decode_32", 32, 4096, 4096, residual=True, from16=True),
        # a ragged batch in fp16 with an odd number of outputs, rows inside wider buffers
        _linear("linear8_gelu_ragged_f16", 333, 1424, 2051, "f16", "gelu_tanh", True, True, pad=32),
        # the fused projection of a 4096-token prompt batch: the matrix product is all there is
        _linear("linear8_qkv_prompt_4096", 4096, 4096, 6144, bias=True),
        # one token's choice among 256 experts in 8 groups, 4 of which stay: nothing but latency
        _route("route_decode_1", 1, 256, 8, groups=8, top_groups=4, group_top=2, scale=2.5),
        # softmax scores read at the chosen experts, groups of 20 by their best expert, logits with ties
        _route("route_softmax_ragged", 333, 160, 6, "softmax", False, 8, 3, 1, False, 16.0, coarse=True),
        # many experts, no groups
        _route("route_wide_1000", 1000, 512, 10),
        # a batch of prompts
        _route("route_prompt_8192", 8192, 256, 8, groups=8, top_groups=4, group_top=2, scale=2.5),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_NORM = 8192 * 4096
MOST_LINEAR = 4096 * 4096 * 6144
MOST_ROUTE = 8192 * 256


def draw(rng):
    op = rng.choice(("norm", "linear", "route"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "norm":
        H = _logu(rng, 64, 16384)
        H = rng.choice((H, H // 8 * 8, H // 8 * 8))
        T = min(_logu(rng, 1, 8192), MOST_NORM // H)
        y, q = rng.choice(((True, False), (False, True), (True, True)))
        return _norm(None, T, H, dtype, rng.random() < 0.5, rng.random() < 0.7, y, q, rng.choice((0, 0, 8, 24)))
    if op == "linear":
        T, K, N = _logu(rng, 1, 4096), 16 * _logu(rng, 16, 512), _logu(rng, 64, 8192)
        N = max(64, min(N, MOST_LINEAR // (T * K)))
        return _linear(None, T, K, N, dtype, rng.choice(ACTS), rng.random() < 0.5, rng.random() < 0.5,
                       rng.random() < 0.5, rng.choice((0, 0, 16, 48)))
    E = rng.choice((8, 16, 40, 60, 64, 72, 96, 128, 160, 256, 257, 320, 384, 512, 1000))
    parts = [g for g in range(2, 17) if E % g == 0 and E // g >= 2]
    groups = rng.choice(parts) if parts and rng.random() < 0.6 else 1
    top_groups = rng.randint(1, groups)
    group_top = rng.choice((1, 2)) if groups > 1 else 1
    k = rng.randint(1, min(16, top_groups * (E // groups)))
    T = min(_logu(rng, 1, 8192), MOST_ROUTE // E)
    return _route(None, T, E, k, rng.choice(("softmax", "sigmoid")), rng.random() < 0.6, groups, top_groups, group_top,
                  rng.random() < 0.7, rng.choice((1.0, 2.5)), rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _wide(t, pad):
    """`t` as the leading columns of rows that are `pad` elements longer (and then, in 8 bits, a
    whole number of 16 bytes)."""
    cols = t.shape[1] + pad
    if t.dtype == E4M3:
        cols = (cols + 15) // 16 * 16
    if cols == t.shape[1]:
        return t
    w = torch.zeros(t.shape[0], cols, dtype=t.dtype, device=t.device)
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def _rows8(v):
    """v [rows, n] in 8 bits: (values in e4m3, fp32 scales [rows])."""
    a = v.abs().amax(1, keepdim=True)
    a = torch.where(a < LEAST, torch.full_like(a, LEAST), a)
    return torch.clamp(v * 448 / a, -448, 448).to(E4M3), a[:, 0] / 448


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    s = dict(case=case)
    if case["op"] == "norm":
        T, H, pad, dt = case["T"], case["H"], case["pad"], TYPES[case["dtype"]]
        # the stream's rows differ in size, and a few of its channels stand out
        loud = torch.where(torch.rand(H, generator=g, device=dev) < 0.01, 20.0, 1.0)
        size = torch.exp(normal(T, 1, std=0.5))
        s.update(x=_wide((normal(T, H) * size).to(torch.float32 if case["x32"] else dt), pad),
                 residual=_wide((normal(T, H, std=2.0) * size * loud).to(dt), pad) if case["residual"] else None,
                 weight=(1 + normal(H, std=0.2)).to(dt),
                 h=_wide(torch.zeros(T, H, dtype=dt, device=dev), pad) if case["residual"] else None,
                 y=_wide(torch.zeros(T, H, dtype=dt, device=dev), pad) if case["y"] else None,
                 q=_wide(torch.zeros(T, H, dtype=E4M3, device=dev), pad) if case["q"] else None,
                 scales=torch.empty(T, dtype=torch.float32, device=dev) if case["q"] else None)
        return s
    if case["op"] == "linear":
        T, K, N, pad, dt = case["T"], case["K"], case["N"], case["pad"], TYPES[case["dtype"]]
        w, sw = _rows8(normal(N, K, std=K ** -0.5))
        s.update(w=_wide(w, pad), sw=sw, y=_wide(torch.zeros(T, N, dtype=dt, device=dev), pad),
                 bias=normal(N).to(dt) if case["bias"] else None,
                 residual=_wide(normal(T, N).to(dt), pad) if case["residual"] else None)
        x = normal(T, K) * torch.exp(normal(T, 1, std=0.5))
        if case["from16"]:
            s.update(x=_wide(x.to(dt), pad), x8=_wide(torch.zeros(T, K, dtype=E4M3, device=dev), pad),
                     sx=torch.empty(T, dtype=torch.float32, device=dev))
        else:
            x, sx = _rows8(x)
            s.update(x=_wide(x, pad), sx=sx)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    # some experts are liked more than others, and the bias leans against that
    liked = normal(E, std=0.5)
    logits = normal(T, E, std=1.5) + liked
    if case["coarse"]:
        logits = logits.to(torch.bfloat16).float()
    s.update(logits=logits, bias=(-0.1 * liked + normal(E, std=0.02)) if case["bias"] else None,
             ids=torch.empty(T, k, dtype=torch.int32, device=dev),
             weights=torch.empty(T, k, dtype=torch.float32, device=dev))
    return s


# ------------------------------------------------------------------ one pass

def _plain_norm(s):
    c, dt = s["case"], s["weight"].dtype
    v = s["x"].float()
    out = {}
    if c["residual"]:
        s["h"].copy_((v + s["residual"].float()).to(dt))
        v = s["h"].float()
        out["h"] = s["h"]
    y = v / torch.sqrt((v * v).sum(1, keepdim=True) / c["H"] + EPS) * s["weight"].float()
    if c["y"]:
        s["y"].copy_(y.to(dt))
        out["y"] = s["y"]
    if c["q"]:
        q, scales = _rows8(y)
        s["q"].copy_(q)
        s["scales"].copy_(scales)
        out["q"], out["scales"] = s["q"], s["scales"]
    return out


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_linear(s):
    x, sx = _rows8(s["x"].float()) if s["case"]["from16"] else (s["x"], s["sx"])
    z = (x.float() * sx[:, None]) @ (s["w"].float() * s["sw"][:, None]).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    z = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    s["y"].copy_(z.to(s["y"].dtype))
    return s["y"]


def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    v = s["logits"].double()
    if c["scoring"] == "sigmoid":
        score = 1 / (1 + torch.exp(-v))
    else:
        e = torch.exp(v - v.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        # (stable sorts: equal values in the order of their numbers)
        best = choice.view(T, G, E // G).sort(dim=2, descending=True, stable=True).values[:, :, :c["group_top"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=v.device)
        stays.scatter_(1, kept, True)
        choice = torch.where(stays[:, :, None], choice.view(T, G, E // G), -math.inf).view(T, E)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    s["ids"].copy_(ids)
    s["weights"].copy_(w * c["scale"])
    return s["ids"], s["weights"]


def _own(s):
    import bit_vq_routed_gb300 as bv
    c = s["case"]
    if c["op"] == "norm":
        bv.moe_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], h=s["h"], y=s["y"], q=s["q"],
                        scales=s["scales"])
        return {k: s[k] for k in ("h", "y", "q", "scales") if s[k] is not None}
    if c["op"] == "linear":
        if "ws" not in s:
            s["ws"] = torch.zeros(bv.moe_linear_8bit_workspace_size(c["T"], c["N"], c["K"]), dtype=torch.uint8,
                                  device="cuda")
        x = s["x"]
        if c["from16"]:
            x = s["x8"]
            bv.moe_quantize_rows(s["x"], x, s["sx"])
        act = (bv.MOE_ACT_NONE, bv.MOE_ACT_RELU, bv.MOE_ACT_GELU, bv.MOE_ACT_GELU_TANH, bv.MOE_ACT_SILU)
        bv.moe_linear_8bit(x, s["sx"], s["w"], s["sw"], s["y"], bias=s["bias"], act=act[ACTS.index(c["act"])],
                           residual=s["residual"], ws=s["ws"])
        return s["y"]
    bv.moe_route_scored(s["logits"], c["k"], s["ids"], s["weights"],
                        scoring=bv.MOE_SCORE_SIGMOID if c["scoring"] == "sigmoid" else bv.MOE_SCORE_SOFTMAX,
                        bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
                        renormalize=c["renorm"], scale=c["scale"])
    return s["ids"], s["weights"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "linear": _plain_linear, "route": _plain_route}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work and the 64-bit result

def work(case):
    T = case["T"]
    if case["op"] == "norm":
        H = case["H"]
        a_value = 2 + 2 * case["x32"] + 4 * case["residual"] + 2 * case["y"] + case["q"]
        return {"bytes": T * H * a_value + 2 * H + 4 * T * case["q"], "flops": 6 * T * H}
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        b = T * K * (1 + case["from16"]) + N * K + 2 * T * N * (1 + case["residual"]) + 2 * N * case["bias"]
        return {"bytes": b + 4 * N + 4 * T * (not case["from16"]), "flops": 2 * T * K * N}
    E, k = case["E"], case["k"]
    return {"bytes": 4 * T * E + 8 * T * k + 4 * E * case["bias"], "flops": 8 * T * E}


def _eighths(v):
    """Half-to-even rounding of |v| <= 448 to a sign, 4 exponent bits (smallest normal 2^-6) and 3
    fraction bits, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        v = s["x"].double()
        out = {}
        if case["residual"]:
            v = v + s["residual"].double()
            out["h"] = v
            # the norm is that of the stored sum: rounded once in 32 and once in 16 bits
            v = (s["x"].float() + s["residual"].float()).to(s["weight"].dtype).double()
        y = torch.rsqrt(torch.mean(v ** 2, -1, keepdim=True) + EPS) * v * s["weight"].double()
        if case["y"]:
            out["y"] = y
        if case["q"]:
            a = y.abs().amax(-1).clamp_min(LEAST)
            out["scales"], out["q"] = a / 448, y * 448 / a[:, None]
        return out
    if case["op"] == "linear":
        x, w = s["x"].double(), s["w"].double()
        if case["from16"]:
            a = x.abs().amax(-1).clamp_min(LEAST)
            x, sx = _eighths(x * 448 / a[:, None]), a / 448
        else:
            sx = s["sx"].double()
        f = torch.nn.functional
        z = (x @ w.t()) * sx[:, None] * s["sw"].double()
        if s["bias"] is not None:
            z = z + s["bias"].double()
        z = {"none": lambda t: t, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
             "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[case["act"]](z)
        return z if s["residual"] is None else z + s["residual"].double()
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    v = s["logits"].double().cpu()
    score = torch.sigmoid(v) if case["scoring"] == "sigmoid" else torch.softmax(v, -1)
    choice = (score if s["bias"] is None else score + s["bias"].double().cpu()).tolist()
    n = E // G
    ids = []
    for row in choice:
        rank = [sum(sorted(row[g * n:(g + 1) * n], reverse=True)[:case["group_top"]]) for g in range(G)]
        kept = sorted(range(G), key=lambda g: (-rank[g], g))[:case["top_groups"]]
        left = [e for g in kept for e in range(g * n, (g + 1) * n)]
        ids.append(sorted(left, key=lambda e: (-row[e], e))[:k])
    ids = torch.tensor(ids)
    w = torch.take_along_dim(score, ids, 1)
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return ids.to(torch.int32), w * case["scale"]
