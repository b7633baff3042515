"""The attention side of a decoder layer around the routed experts, as measured cases.

Three operators that follow one another in a serving step:

  linear     y = act(x W^T + bias) + residual: the projections before and after the attention
             (moe_linear)
  append     new keys and values into a paged cache, keys and queries turned by their positions on
             the way (moe_kv_append)
  attention  softmax(q K^T scale) V over that cache for a batch whose sequences share a prefix,
             kept in the cache once, each with its own causal suffix (moe_prefix_attention)

`run` computes them in elementary torch operations in 32 bits (own = False) or through the
library (own = True); `exact` computes them in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
STYLES = ("half", "pairs")  # dimension i turns with i + rot/2, or 2i with 2i + 1


# ------------------------------------------------------------------ cases

def _linear(name, T, K, N, dtype="bf16", act="none", bias=False, residual=False, pad=0):
    c = dict(op="linear", T=T, K=K, N=N, dtype=dtype, act=act, bias=bias, residual=residual, pad=pad)
    return dict(c, name=name) if name else c


def _append(name, T, heads, group, D, rot, style, page, dtype="bf16", skip=0.0, base=0):
    c = dict(op="append", T=T, heads=heads, group=group, D=D, rot=rot, style=style, page=page, dtype=dtype, skip=skip,
             base=base)
    return dict(c, name=name) if name else c


def _attention(name, B, nq, prefix, suffix, heads, group, D, page, dtype="bf16", mix=0):
    c = dict(op="attention", B=B, nq=nq, prefix=prefix, suffix=suffix, heads=heads, group=group, D=D, page=page,
             dtype=dtype, mix=mix)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the fused q, k, v projection (32 query and 8 key heads of 128, hidden size 4096) of one user's
        # next token: the weights' bytes are all there is
        _linear("linear_qkv_decode_1", 1, 4096, 6144, bias=True),
        # the projection after the attention for 32 users' next tokens, added to the residual stream
        _linear("linear_out_decode_32", 32, 4096, 4096, residual=True),
        # a ragged batch in fp16 with an odd number of outputs, rows inside wider buffers
        _linear("linear_gelu_ragged_f16", 333, 1416, 2051, "f16", "gelu_tanh", True, True, 24),
        # the fused projection of a 4096-token prompt batch: the matrix product is all there is
        _linear("linear_qkv_prompt_4096", 4096, 4096, 6144, bias=True),
        # one user's next token: the smallest call, nothing but its latency
        _append("append_decode_1", 1, 8, 4, 128, 128, "half", 16, base=3000),
        # 32 users' next tokens
        _append("append_decode_32", 32, 8, 4, 128, 128, "half", 64, base=20000),
        # a ragged batch in fp16: head size 80 of which 64 turn, in pairs, padding tokens between
        _append("append_ragged_f16", 1537, 5, 3, 80, 64, "pairs", 16, "f16", 0.1, 100),
        # a batch of prompts
        _append("append_prompt_8192", 8192, 8, 4, 128, 128, "half", 64),
        # one user behind a short system prompt
        _attention("attention_decode_1", 1, 1, 1000, 200, 8, 4, 128, 16),
        # 32 users behind one long document: its keys and values are read once for all of them
        _attention("attention_decode_32", 32, 1, 32768, 1024, 8, 4, 128, 64, mix=1),
        # a ragged batch in fp16: head size 80, three query heads to a key head, up to 40 new tokens
        # for a sequence and none for some
        _attention("attention_ragged_f16", 9, 40, 1501, 700, 5, 3, 80, 16, "f16", mix=2),
        # four users' prompts of up to 1024 tokens behind one document
        _attention("attention_prompt_4", 4, 1024, 8192, 1024, 8, 4, 128, 64, mix=3),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(c):
    """New tokens and cached suffix tokens (the new ones among them) of each sequence: a spread
    between a quarter of the case's largest and the largest itself, the first sequence at it; where
    a call has many new tokens for some, a few sequences have none."""
    r = random.Random(1000 + c["mix"])
    nq, lens = [], []
    for b in range(c["B"]):
        n = c["nq"] if b == 0 or c["nq"] == 1 else r.randint(max(1, c["nq"] // 4), c["nq"])
        if b and 1 < c["nq"] <= 64 and r.random() < 0.15:
            n = 0
        m = c["suffix"] if b == 0 else r.randint(max(1, c["suffix"] // 4), c["suffix"])
        nq.append(n)
        lens.append(max(m, n))
    return nq, lens


def _pairs(nq, lens):
    """(query, key) pairs of the suffixes: query i of n sees len - n + i + 1 keys."""
    return sum(n * m - n * (n - 1) // 2 for n, m in zip(nq, lens))


MOST_LINEAR = 4096 * 4096 * 6144
MOST_APPEND = 8192 * (8 * 4 + 2 * 8) * 128
MOST_ATTENTION = 4096 * 32 * 128 * 8192 * 0.6


def draw(rng):
    op = rng.choice(("linear", "append", "attention"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "linear":
        T, K, N = _logu(rng, 1, 4096), 8 * _logu(rng, 32, 1024), _logu(rng, 64, 8192)
        N = max(64, min(N, MOST_LINEAR // (T * K)))
        return _linear(None, T, K, N, dtype, rng.choice(ACTS), rng.random() < 0.5, rng.random() < 0.5,
                       rng.choice((0, 0, 8, 24)))
    heads, group, D = rng.choice((1, 2, 4, 5, 8)), rng.choice((1, 2, 3, 4, 5, 8, 16)), rng.choice((64, 80, 96, 128))
    page = rng.choice((8, 16, 32, 64, 128, 256))
    if op == "append":
        T = _logu(rng, 1, 8192)
        T = max(1, min(T, MOST_APPEND // ((group + 2) * heads * D)))
        return _append(None, T, heads, group, D, rng.choice((D, D // 2, 16)), rng.choice(STYLES), page, dtype,
                       rng.choice((0.0, 0.0, 0.1)), _logu(rng, 1, 100000))
    if rng.random() < 0.6:
        B, nq, suffix, prefix = _logu(rng, 1, 64), rng.choice((1, 1, 1, 2, 4)), _logu(rng, 1, 2048), _logu(rng, 1, 32768)
    else:
        B, nq, suffix, prefix = rng.randint(1, 5), _logu(rng, 8, 1024), _logu(rng, 8, 1024), _logu(rng, 1, 8192)
    prefix = rng.choice((prefix, prefix, prefix, 0))
    most = int(MOST_ATTENTION // (B * nq * heads * group * D))
    prefix = min(prefix, most)
    return _attention(None, B, nq, prefix, suffix, heads, group, D, page, dtype, rng.randrange(1 << 16))


# ------------------------------------------------------------------ inputs

def _wide(t, pad):
    """`t` as the leading columns of rows that are `pad` elements longer."""
    if not pad:
        return t
    w = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def _turns(n, rot, dev):
    """cos | sin of the angle p * 10000^(-2i/rot), fp32 [n, rot]."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    dt, dev = TYPES[case["dtype"]], "cuda"

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    s = dict(case=case)
    if case["op"] == "linear":
        T, K, N, pad = case["T"], case["K"], case["N"], case["pad"]
        s.update(x=_wide(normal(T, K), pad), w=_wide(normal(N, K, std=K ** -0.5), pad), y=_wide(normal(T, N), pad),
                 bias=normal(N) if case["bias"] else None,
                 residual=_wide(normal(T, N), pad) if case["residual"] else None)
        return s
    heads, group, D, page = case["heads"], case["group"], case["D"], case["page"]
    if case["op"] == "append":
        T = case["T"]
        # the rows that the fused projection left: q, k and v of a token side by side
        qkv = normal(T, (group + 2) * heads, D)
        pages = -(-T // page) + 3
        if case["base"]:  # tokens of many sequences, each at its own page's end
            slots = torch.randperm(pages * page, generator=g, device=dev)[:T]
        else:  # prompts: page after page, the pages in no order
            slots = torch.randperm(pages, generator=g, device=dev)[:, None] * page + torch.arange(page, device=dev)
            slots = slots.reshape(-1)[:T].contiguous()
        if case["skip"]:
            slots[torch.rand(T, generator=g, device=dev) < case["skip"]] = -1
        first = case["base"]
        last = first + T + host.randrange(16)
        pos = torch.arange(T, device=dev) + first if case["base"] == 0 else \
            torch.randint(first, last, (T,), generator=g, device=dev)
        s.update(q=qkv[:, :group * heads], k=qkv[:, group * heads:(group + 1) * heads], v=qkv[:, (group + 1) * heads:],
                 q_out=torch.empty(T, group * heads, D, dtype=dt, device=dev),
                 k_cache=normal(pages, page, heads, D), v_cache=normal(pages, page, heads, D),
                 positions=pos.to(torch.int32), slots=slots, cos_sin=_turns(last + 1, case["rot"], dev))
        return s
    nq, lens = _lengths(case)
    T = sum(nq)
    shared, each = -(-case["prefix"] // page), [-(-m // page) for m in lens]
    pages = shared + sum(each) + 2
    # the pages as a server has them after some time: in no order
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), max(each), dtype=torch.int32)
    at, perm = shared, order.cpu()
    for b, n in enumerate(each):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = torch.zeros(len(nq) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(nq).cumsum(0)
    s.update(q=normal(T, heads * group, D, std=2.0), k_cache=normal(pages, page, heads, D),
             v_cache=normal(pages, page, heads, D), prefix_pages=order[:shared].contiguous(), page_table=table.to(dev),
             cu_q=cu.to(dev), seq_lens=torch.tensor(lens, dtype=torch.int32).to(dev),
             out=torch.empty(T, heads * group, D, dtype=dt, device=dev),
             lse=torch.empty(T, heads * group, dtype=torch.float32, device=dev))
    return s


# ------------------------------------------------------------------ one pass

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
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    z = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(s["x"].dtype)


def _turn(x, cs, rot, style):
    x = x.float()
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if style == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(s):
    c, dt = s["case"], s["q"].dtype
    cs = s["cos_sin"][s["positions"].long()]
    s["q_out"].copy_(_turn(s["q"], cs, c["rot"], c["style"]).to(dt))
    k = _turn(s["k"], cs, c["rot"], c["style"]).to(dt)
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    s["k_cache"].view(-1, c["heads"], c["D"])[at] = k[kept]
    s["v_cache"].view(-1, c["heads"], c["D"])[at] = s["v"][kept]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attention(s):
    c, dt = s["case"], s["q"].dtype
    heads, group, D, page, prefix, B = c["heads"], c["group"], c["D"], c["page"], c["prefix"], c["B"]
    T = s["q"].shape[0]
    scale = D ** -0.5
    q = s["q"].float().view(T, heads, group, D)
    cu, lens = s["cu_q"].long(), s["seq_lens"].long()
    # the shared prefix, for all tokens at once: [heads, T * group, prefix]
    rows = q.permute(1, 0, 2, 3).reshape(heads, T * group, D)
    kp = s["k_cache"][s["prefix_pages"].long()].view(-1, heads, D)[:prefix].float().permute(1, 0, 2)
    vp = s["v_cache"][s["prefix_pages"].long()].view(-1, heads, D)[:prefix].float().permute(1, 0, 2)
    sp = (rows @ kp.transpose(1, 2)) * scale
    # the suffixes, sequences padded to the longest: [B, heads, n * group, L]
    n, L = c["nq"], s["page_table"].shape[1] * page
    i = torch.arange(n, device=q.device)
    tok = cu[:-1, None] + i
    real = tok < cu[1:, None]
    tok = torch.where(real, tok, torch.zeros_like(tok))
    qs = q[tok].permute(0, 2, 1, 3, 4).reshape(B, heads, n * group, D)
    ks = s["k_cache"][s["page_table"].long()].view(B, L, heads, D).float().permute(0, 2, 1, 3)
    vs = s["v_cache"][s["page_table"].long()].view(B, L, heads, D).float().permute(0, 2, 1, 3)
    ss = (qs @ ks.transpose(2, 3)) * scale
    at = lens[:, None] - (cu[1:] - cu[:-1])[:, None] + i
    seen = torch.arange(L, device=q.device) <= at[:, :, None]
    ss = ss.masked_fill(~seen.repeat_interleave(group, 1)[:, None], -math.inf)
    # one softmax over both
    ms = ss.amax(-1).view(B, heads, n, group).permute(0, 2, 1, 3)[real]
    mp = sp.amax(-1).view(heads, T, group).permute(1, 0, 2) if prefix else torch.full_like(ms, -math.inf)
    m = torch.maximum(mp, ms)
    mb = torch.zeros(B, n, heads, group, device=q.device)
    mb[real] = m
    ps = torch.exp(ss - mb.permute(0, 2, 1, 3).reshape(B, heads, n * group, 1))
    pp = torch.exp(sp - m.permute(1, 0, 2).reshape(heads, T * group, 1))
    o = (pp @ vp).view(heads, T, group, D).permute(1, 0, 2, 3) + \
        (ps @ vs).view(B, heads, n, group, D).permute(0, 2, 1, 3, 4)[real]
    den = pp.sum(-1).view(heads, T, group).permute(1, 0, 2) + \
        ps.sum(-1).view(B, heads, n, group).permute(0, 2, 1, 3)[real]
    return (o / den[..., None]).reshape(T, heads * group, D).to(dt), (m + torch.log(den)).reshape(T, heads * group)


def _own(s):
    import bit_vq_routed_gb300 as bv
    c = s["case"]
    if c["op"] == "linear":
        if "ws" not in s:
            s["ws"] = torch.zeros(bv.moe_linear_workspace_size(c["T"], c["N"], c["K"]), dtype=torch.uint8, device="cuda")
        act = (bv.MOE_ACT_NONE, bv.MOE_ACT_RELU, bv.MOE_ACT_GELU, bv.MOE_ACT_GELU_TANH, bv.MOE_ACT_SILU)
        bv.moe_linear(s["x"], s["w"], s["y"], bias=s["bias"], act=act[ACTS.index(c["act"])], residual=s["residual"],
                      ws=s["ws"])
        return s["y"]
    if c["op"] == "append":
        bv.moe_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["positions"], s["slots"], s["cos_sin"],
                         interleaved=c["style"] == "pairs", q=s["q"], q_out=s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if "ws" not in s:
        s["ws"] = torch.zeros(bv.moe_prefix_attention_workspace_size(s["q"].shape[0], c["heads"] * c["group"],
                                                                     c["heads"], c["D"]),
                              dtype=torch.uint8, device="cuda")
    bv.moe_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["cu_q"], s["prefix_pages"], c["prefix"],
                            s["page_table"], s["seq_lens"], c["D"] ** -0.5, s["out"], lse=s["lse"], ws=s["ws"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "append": _plain_append, "attention": _plain_attention}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work and the 64-bit result

def work(case):
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        n = T * K + N * K + T * N + N * case["bias"] + T * N * case["residual"]
        return {"bytes": 2 * n, "flops": 2 * T * K * N}
    heads, group, D = case["heads"], case["group"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        return {"bytes": 4 * T * (group + 2) * heads * D + T * (12 + 4 * case["rot"]),
                "flops": 3 * T * (group + 1) * heads * case["rot"]}
    nq, lens = _lengths(case)
    T, keys = sum(nq), case["prefix"] + sum(m for n, m in zip(nq, lens) if n)
    return {"bytes": 4 * keys * heads * D + T * heads * group * (4 * D + 4),
            "flops": 4 * D * heads * group * (T * case["prefix"] + _pairs(nq, lens))}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        y = torch.nn.functional.linear(s["x"].double(), s["w"].double(),
                                       None if s["bias"] is None else s["bias"].double())
        f = torch.nn.functional
        y = {"none": lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
             "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}[case["act"]](y)
        return y if s["residual"] is None else y + s["residual"].double()
    heads, group, D, page = case["heads"], case["group"], case["D"], case["page"]
    if case["op"] == "append":
        rot = case["rot"]
        cs = s["cos_sin"].double()[s["positions"].long()]
        turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]

        def turned(x):
            x = x.double().clone()
            half = case["style"] == "half"
            a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
            z = torch.complex(a.contiguous(), b.contiguous()) * turn
            a.copy_(z.real)
            b.copy_(z.imag)
            return x

        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k, v = turned(s["k"]), s["v"].double()
        t = torch.nonzero(s["slots"] >= 0).flatten()
        kc[s["slots"][t] // page, s["slots"][t] % page] = k[t]
        vc[s["slots"][t] // page, s["slots"][t] % page] = v[t]
        return turned(s["q"]), kc, vc
    nq, lens = _lengths(case)
    T = sum(nq)
    out = torch.zeros(T, heads * group, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, heads * group), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, m) in enumerate(zip(nq, lens)):
        if n == 0:
            continue
        at = [s["k_cache"], s["v_cache"]]
        own_pages = s["page_table"][b, :-(-m // page)].long()
        kv = [torch.cat((x[s["prefix_pages"].long()].reshape(-1, heads, D)[:case["prefix"]],
                         x[own_pages].reshape(-1, heads, D)[:m])).double() for x in at]
        seen = torch.arange(case["prefix"] + m, device="cuda")[None] <= \
            (case["prefix"] + m - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(heads * group):
            z = s["q"][t0:t0 + n, h].double() @ kv[0][:, h // group].t() / math.sqrt(D)
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            lse[t0:t0 + n, h] = torch.logsumexp(z, -1)
            out[t0:t0 + n, h] = torch.softmax(z, -1) @ kv[1][:, h // group]
        t0 += n
    return out, lse
