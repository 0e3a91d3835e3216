"""The serving and training operators next to the attention kernels, as measured workloads.

Five operators, each with its plain form (elementary torch operations in 32 bits, rounded once at
the end) and the call that a user of this library makes:

  plan     block table, slots, positions and offsets of a step, from the requests' lengths
  rope     the position rotation of part of each head
  fwd      norm of each query / key head and the rotation in one pass, keys and values into the paged cache
  bwd      the gradients of that norm and rotation
  decode   attention of one new token over paged K and V pools, under a sink + local window or unbounded

`own` selects the side: False the plain forms, True the library."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one decode step of a batch with long contexts: most requests append one token, some slots are idle
        {"name": "plan decode step", "op": "plan", "batch": 256, "page": 128, "ctx_lo": 1, "ctx_hi": 131072,
         "new_lo": 0, "new_hi": 1, "capacity": 256},
        # admission of prompts (and of chunks of prompts) into a cache of small pages, up to a budget of tokens
        {"name": "plan prefill", "op": "plan", "batch": 48, "page": 16, "ctx_lo": 0, "ctx_hi": 4096,
         "new_lo": 1, "new_hi": 32768, "capacity": 160037},
        # absorbed MLA queries of one decode step: the last 64 of 576 columns are rotated, far positions
        {"name": "rope absorbed decode", "op": "rope", "dtype": "bf16", "tokens": 64, "heads": 64, "d": 576,
         "rope_dim": 64, "rope_off": 512, "interleaved": True, "factor": 4.0, "pos_hi": 131072},
        # per-head MLA queries of a long prompt, 128 + 64 columns
        {"name": "rope per-head prefill", "op": "rope", "dtype": "bf16", "tokens": 16411, "heads": 64, "d": 192,
         "rope_dim": 64, "rope_off": 128, "interleaved": True, "factor": 1.0, "pos_hi": 32768},
        # one decode step of the absorbed path: queries rotated, the latent normed, rotated and written to its page
        {"name": "norm+rope latent decode", "op": "fwd", "dtype": "bf16", "tokens": 64, "heads": 64, "kv_heads": 1,
         "d": 576, "d_v": 0, "norm_dim": 512, "q_norm": False, "rope_dim": 64, "rope_off": 512, "interleaved": True,
         "factor": 4.0, "pos_hi": 131072, "page": 128, "pooled": True},
        # a prompt with grouped heads, straight from the fused projection's rows into the paged cache
        {"name": "norm+rope grouped prefill", "op": "fwd", "dtype": "fp16", "tokens": 16381, "heads": 32,
         "kv_heads": 8, "d": 128, "d_v": 128, "norm_dim": 128, "q_norm": True, "rope_dim": 128, "rope_off": 0,
         "interleaved": False, "factor": 1.0, "pos_hi": 32768, "page": 16, "pooled": True},
        # the gradient at the size of a small check (four heads of 64), in 32 bits
        {"name": "norm+rope backward small", "op": "bwd", "dtype": "fp32", "tokens": 2048, "heads": 4, "kv_heads": 4,
         "d": 64, "norm_dim": 64, "rope_dim": 64, "rope_off": 0, "interleaved": False, "factor": 1.0,
         "pos_hi": 2048},
        # the gradient of a packed training batch with grouped heads, half of each head rotated
        {"name": "norm+rope backward large", "op": "bwd", "dtype": "bf16", "tokens": 32749, "heads": 32,
         "kv_heads": 8, "d": 128, "norm_dim": 128, "rope_dim": 64, "rope_off": 0, "interleaved": False,
         "factor": 1.0, "pos_hi": 32768},
        # one request, short context: the latency of a decode step
        {"name": "decode one sequence", "op": "decode", "dtype": "bf16", "batch": 1, "len_lo": 2048, "len_hi": 2048,
         "heads": 32, "kv_heads": 8, "d": 128, "d_v": 128, "page": 16, "block": 128, "sink": 0, "local": -1},
        # an ordinary batch with ragged contexts
        {"name": "decode ragged batch", "op": "decode", "dtype": "fp16", "batch": 64, "len_lo": 64, "len_hi": 16384,
         "heads": 32, "kv_heads": 8, "d": 128, "d_v": 128, "page": 64, "block": 128, "sink": 0, "local": -1},
        # the sparse window (one sink block, seven local ones) with per-head K/V of 192 and 128, long contexts of
        # which only the window's pages are still held
        {"name": "decode window per-head", "op": "decode", "dtype": "bf16", "batch": 24, "len_lo": 65536,
         "len_hi": 131072, "heads": 64, "kv_heads": 64, "d": 192, "d_v": 128, "page": 128, "block": 128, "sink": 1,
         "local": 7},
        # long contexts in full
        {"name": "decode long contexts", "op": "decode", "dtype": "bf16", "batch": 32, "len_lo": 16384,
         "len_hi": 49152, "heads": 32, "kv_heads": 8, "d": 128, "d_v": 128, "page": 64, "block": 128, "sink": 0,
         "local": -1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rope_of(rng, d):
    """Rotated part and layout of a head of d columns."""
    rope_dim, rope_off = rng.choice([(d, 0), (d // 2, 0), (d // 2, d - d // 2), (d // 4, d - d // 4)])
    rope_dim -= rope_dim % 2
    return {"rope_dim": rope_dim, "rope_off": rope_off, "interleaved": rng.random() < 0.5,
            "factor": rng.choice([1.0, 1.0, 4.0, 32.0]), "pos_hi": _log(rng, 64, 1 << 20)}


def draw(rng):
    op = rng.choice(["plan", "rope", "fwd", "bwd", "decode", "decode"])
    if op == "plan":
        batch = _log(rng, 1, 512)
        if rng.random() < 0.5:
            return {"op": op, "batch": batch, "page": rng.choice([16, 32, 64, 128, 256]), "ctx_lo": 0,
                    "ctx_hi": _log(rng, 16, 131072), "new_lo": 0, "new_hi": 1, "capacity": batch + rng.randrange(64)}
        batch, new_hi = min(batch, 64), _log(rng, 2, 24000)
        return {"op": op, "batch": batch, "page": rng.choice([16, 32, 64, 128, 256]), "ctx_lo": 0,
                "ctx_hi": _log(rng, 16, 8192), "new_lo": 0, "new_hi": new_hi,
                "capacity": batch * new_hi // 4 + rng.randrange(1, 64)}
    if op in ("rope", "fwd", "bwd"):
        d = rng.choice([64, 80, 96, 100, 128, 192, 256, 576])
        heads, kv_heads = rng.choice([(1, 1), (4, 4), (16, 2), (32, 8), (64, 1), (28, 4), (15, 5)])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        tokens = _log(rng, 1, max(2, 40_000_000 // ((heads + 2 * kv_heads) * d)))
        case = {"op": op, "dtype": dtype, "tokens": tokens, "heads": heads, "d": d, **_rope_of(rng, d)}
        if op == "rope":
            return case
        norm_dim = d if case["rope_off"] == 0 or rng.random() < 0.5 else case["rope_off"]
        case.update(kv_heads=kv_heads, norm_dim=norm_dim)
        if op == "fwd":
            pooled = rng.random() < 0.7
            case.update(q_norm=rng.random() < 0.7, d_v=rng.choice([0, 64, 128]) if pooled else 0, pooled=pooled,
                        page=rng.choice([16, 64, 128]))
        return case
    d, d_v = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    heads, kv_heads = rng.choice([(8, 8), (32, 8), (16, 2), (28, 4), (40, 8), (64, 64), (32, 1), (71, 1)])
    batch = _log(rng, 1, 192)
    block, sink, local = rng.choice([(128, 0, -1), (128, 0, -1), (128, 1, 7), (1, 16, 1024), (64, 2, 5)])
    keys = max(64, min(131072, 1_000_000_000 // (kv_heads * (d + d_v) * batch)))
    hi = _log(rng, 32, keys) if local < 0 else _log(rng, 32, 200_000)
    return {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "batch": batch, "len_lo": rng.choice([0, 1, hi // 2]),
            "len_hi": hi, "heads": heads, "kv_heads": kv_heads, "d": d, "d_v": d_v,
            "page": rng.choice([16, 32, 64, 128]), "block": block, "sink": sink, "local": local}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _frequencies(rope_dim, factor):
    """Angles per position in 64 bits, and the factor on cos and sin: base 10,000; factor > 1 blends the
    frequencies between kept (more than 32 turns over 4,096 positions) and divided by the factor (less than
    one), with the usual 0.1 ln(factor) + 1 on cos and sin."""
    half = rope_dim // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    if factor == 1.0:
        return freq, 1.0
    def dim_of(turns):
        return rope_dim * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
    low, high = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), rope_dim - 1)
    ramp = ((torch.arange(half, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
    return freq / factor * ramp + freq * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _lengths(case, lo, hi, gen):
    """`batch` lengths between case[lo] and case[hi], spread over their logarithm."""
    a, b = case[lo], case[hi]
    u = torch.rand(case["batch"], generator=gen, dtype=torch.float64)
    if a == b:
        return torch.full((case["batch"],), a, dtype=torch.int64)
    if b - a < 16:
        return a + (u * (b - a + 1)).floor().long()
    return ((a + 1) * ((b + 1) / (a + 1)) ** u - 1).round().long().clamp(a, b)


def prepare(case, seed):
    dev = torch.device("cuda")
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": case}
    op = case["op"]

    def normal(*shape, dtype=None):
        dtype = dtype or DTYPES[case["dtype"]]
        out = torch.empty(shape, dtype=dtype, device=dev)
        flat, step = out.view(-1), 1 << 28
        for at in range(0, flat.numel(), step):
            n = min(step, flat.numel() - at)
            flat[at:at + n] = torch.randn(n, device=dev, generator=gen)
        return out

    if op == "plan":
        ctx, new = _lengths(case, "ctx_lo", "ctx_hi", host), _lengths(case, "new_lo", "new_hi", host)
        P, B = case["page"], case["batch"]
        new = torch.minimum(new, (case["capacity"] - new.cumsum(0) + new).clamp(min=0))  # what the step has room for
        have, total = (ctx + P - 1) // P, (ctx + new + P - 1) // P
        cols = (case["ctx_hi"] + case["new_hi"]) // P + 2
        order = torch.randperm(int(total.sum()) + 16, generator=host).to(torch.int32)
        table = torch.full((B, cols), -1, dtype=torch.int32)
        table[torch.arange(cols)[None, :] < have[:, None]] = order[: int(have.sum())]
        s.update(ctx=ctx.int().to(dev), new=new.int().to(dev), table=table.to(dev),
                 free=order[int(have.sum()):].contiguous().to(dev), tokens=int(new.sum()),
                 pages=int((total - have).sum()))
        return s
    if op == "decode":
        B, P, Hk = case["batch"], case["page"], case["kv_heads"]
        lens = _lengths(case, "len_lo", "len_hi", host)
        cols = max(1, (int(lens.max()) + P - 1) // P)
        col = torch.arange(cols)[None, :] * P
        live = col < lens[:, None]
        if case["local"] >= 0:  # pages outside the sink blocks and the local ones have been handed back
            i = lens[:, None] - 1
            lo = ((i // case["block"] - case["local"] + 1) * case["block"]).clamp(min=0)
            live &= (col < case["sink"] * case["block"]) | (col + P > lo)
        n = int(live.sum())
        table = torch.full((B, cols), -1, dtype=torch.int32)
        table[live] = torch.randperm(n, generator=host).to(torch.int32)
        s.update(q=normal(B, case["heads"], case["d"]), k_pool=normal(max(1, n), P, Hk, case["d"]),
                 v_pool=normal(max(1, n), P, Hk, case["d_v"]), table=table.to(dev), lens=lens.int().to(dev),
                 max_len=max(1, int(lens.max())), scale=case["d"] ** -0.5)
        return s
    freq, s["rope_scale"] = _frequencies(case["rope_dim"], case["factor"])
    T, d = case["tokens"], case["d"]
    s["freq"] = freq.to(dev)
    s["pos"] = torch.randint(case["pos_hi"], (T,), generator=host, dtype=torch.int32).to(dev)
    if op == "rope":
        s["x"] = normal(T, case["heads"], d)
        return s
    H, Hk = case["heads"], case["kv_heads"]
    d_v = case.get("d_v", 0)
    rows = normal(T, (H + Hk) * d + Hk * d_v)  # the projection's output: q, k and v side by side
    s["q"], s["k"] = rows[:, :H * d].view(T, H, d), rows[:, H * d:(H + Hk) * d].view(T, Hk, d)
    s["v"] = rows[:, (H + Hk) * d:].view(T, Hk, d_v) if d_v else None
    s["qw"] = (1 + 0.2 * torch.randn(case["norm_dim"], device=dev, generator=gen)).to(DTYPES[case["dtype"]])
    s["kw"] = (1 + 0.2 * torch.randn(case["norm_dim"], device=dev, generator=gen)).to(DTYPES[case["dtype"]])
    if op == "bwd":
        s["dq"], s["dk"] = normal(T, H, d), normal(T, Hk, d)
        return s
    if not case["q_norm"]:
        s["qw"] = None
    if case["pooled"]:
        P = case["page"]
        pages = T // P + 5
        s["slots"] = torch.randperm(pages * P, generator=host)[:T].to(dev)
        s["k_pool"] = normal(pages, P, Hk, d)
        s["v_pool"] = normal(pages, P, Hk, d_v) if d_v else None
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_plan(s):
    P, B = s["case"]["page"], s["case"]["batch"]
    ctx, new, dev = s["ctx"].long(), s["new"].long(), s["ctx"].device
    have = (ctx + P - 1) // P
    need = (ctx + new + P - 1) // P - have
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    cu, pu = torch.cat([zero, new.cumsum(0)]), torch.cat([zero, need.cumsum(0)])
    each = torch.arange(B, device=dev)
    at = torch.repeat_interleave(each, need, output_size=s["pages"])
    nth = torch.arange(s["pages"], device=dev)
    s["table"][at, have[at] + nth - pu[at]] = s["free"][nth]
    row = torch.repeat_interleave(each, new, output_size=s["tokens"])
    pos = ctx[row] + torch.arange(s["tokens"], device=dev) - cu[row]
    slots = s["table"][row, pos // P].long() * P + pos % P
    pad = s["case"]["capacity"] - s["tokens"]
    counts = torch.stack([cu[-1], pu[-1], torch.zeros_like(cu[-1])])
    return {"table": s["table"], "cu_seqlens": cu.int(), "seqlens": (ctx + new).int(),
            "positions": torch.cat([pos, zero.expand(pad)]).int(),
            "slots": torch.cat([slots, (zero - 1).expand(pad)]), "counts": counts.int()}


def _angles(s):
    a = s["pos"].double()[:, None, None] * s["freq"]
    return (a.cos() * s["rope_scale"]).float(), (a.sin() * s["rope_scale"]).float()


def _rotate(x, cos, sin, case):
    lo, n = case["rope_off"], case["rope_dim"]
    part = x[..., lo:lo + n]
    if case["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = part[..., : n // 2], part[..., n // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([x[..., :lo], turned, x[..., lo + n:]], -1)


def _normed(x, w, n):
    r = torch.rsqrt((x[..., :n] * x[..., :n]).mean(-1, keepdim=True) + EPS)
    return torch.cat([x[..., :n] * r * w, x[..., n:]], -1)


def _plain_fwd(s):
    case, dtype = s["case"], s["q"].dtype
    cos, sin = _angles(s)
    q, k = s["q"].float(), s["k"].float()
    if s["qw"] is not None:
        q = _normed(q, s["qw"].float(), case["norm_dim"])
    k = _normed(k, s["kw"].float(), case["norm_dim"])
    q, k = _rotate(q, cos, sin, case).to(dtype), _rotate(k, cos, sin, case).to(dtype)
    if not case["pooled"]:
        return {"q": q, "k": k}
    page, row = s["slots"] // case["page"], s["slots"] % case["page"]
    s["k_pool"][page, row] = k
    if s["v"] is not None:
        s["v_pool"][page, row] = s["v"]
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_side_bwd(x, dy, w, cos, sin, case):
    n = case["norm_dim"]
    x, dn, w = x.float(), _rotate(dy.float(), cos, -sin, case), w.float()
    r = torch.rsqrt((x[..., :n] * x[..., :n]).mean(-1, keepdim=True) + EPS)
    hat = x[..., :n] * r
    g = dn[..., :n] * w
    dx = r * (g - hat * (g * hat).mean(-1, keepdim=True))
    return torch.cat([dx, dn[..., n:]], -1), (dn[..., :n] * hat).sum((0, 1))


def _plain_bwd(s):
    cos, sin = _angles(s)
    dq, dqw = _plain_side_bwd(s["q"], s["dq"], s["qw"], cos, sin, s["case"])
    dk, dkw = _plain_side_bwd(s["k"], s["dk"], s["kw"], cos, sin, s["case"])
    return {"dq": dq.to(s["q"].dtype), "dk": dk.to(s["q"].dtype), "dq_weight": dqw, "dk_weight": dkw}


def _window_keys(case, lens, width):
    """Key positions [B, W] that each sequence's last token sees, and which of them exist."""
    i = lens.long()[:, None] - 1
    if case["local"] < 0:
        t = torch.arange(width, device=lens.device)[None, :]
        return t.expand(len(lens), -1), t <= i
    head = case["sink"] * case["block"]
    lo = ((torch.div(i, case["block"], rounding_mode="floor") - case["local"] + 1) * case["block"]).clamp(min=0)
    j = torch.arange(head + case["local"] * case["block"], device=lens.device)[None, :]
    t = torch.where(j < head, j, lo + j - head)
    return t, (t <= i) & ((j < head) | (t >= head))


def _plain_decode(s):
    case = s["case"]
    B, H, Hk, P = case["batch"], case["heads"], case["kv_heads"], case["page"]
    t, seen = _window_keys(case, s["lens"], s["max_len"])
    t = torch.where(seen, t, torch.zeros_like(t))
    page = s["table"].gather(1, t // P).long().clamp(min=0)
    k, v = s["k_pool"][page, t % P].float(), s["v_pool"][page, t % P].float()
    q = s["q"].float().view(B, Hk, H // Hk, case["d"]) * s["scale"]
    z = torch.matmul(q, k.permute(0, 2, 3, 1)).masked_fill(~seen[:, None, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": out.view(B, H, case["d_v"]).to(s["q"].dtype), "lse": (top + total.log()).view(B, H)}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import block_sparse_streaming_b200 as bss
    case = s["case"]
    op = case["op"]
    if op == "plan":
        cu, lens, pos, slots, counts = bss.loza_page_plan(s["ctx"], s["new"], s["free"], s["table"], case["page"],
                                                          case["capacity"])
        return {"table": s["table"], "cu_seqlens": cu, "seqlens": lens, "positions": pos, "slots": slots,
                "counts": counts}
    if op == "decode":
        params = bss.Params(s["scale"], case["block"], case["sink"], case["local"])
        out, lse = bss.loza_ssa_decode_paged_kv(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"],
                                                s["max_len"], params)
        return {"out": out, "lse": lse}
    rope = bss.RopeParams(case["rope_dim"], case["rope_off"], case["interleaved"], s["rope_scale"])
    if op == "rope":
        return bss.loza_rope(s["x"], s["pos"], s["freq"], rope)
    if op == "fwd":
        if not case["pooled"]:
            q, k = bss.loza_qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], rope, s["qw"], s["kw"], EPS)
            return {"q": q, "k": k}
        q, _ = bss.loza_qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], rope, s["qw"], s["kw"], EPS, v=s["v"],
                                     k_pool=s["k_pool"], v_pool=s["v_pool"], slots=s["slots"])
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    dq, dk, dqw, dkw = bss.loza_qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freq"], rope,
                                                      s["qw"], s["kw"], EPS)
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "plan":
        return _plain_plan(state)
    if op == "rope":
        cos, sin = _angles(state)
        return _rotate(state["x"].float(), cos, sin, state["case"]).to(state["x"].dtype)
    if op == "fwd":
        return _plain_fwd(state)
    if op == "bwd":
        return _plain_bwd(state)
    return _plain_decode(state)


# ---------------------------------------------------------------------------
# Work of a pass: inputs read once, outputs written once
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        if case["new_hi"] - case["new_lo"] < 16:
            tokens = case["batch"] * (case["new_lo"] + case["new_hi"]) / 2
        else:  # mean of a length spread over its logarithm
            a, b = case["new_lo"] + 1, case["new_hi"] + 1
            tokens = case["batch"] * ((b - a) / math.log(b / a) - 1)
        pages = min(tokens, case["capacity"]) / case["page"]
        return {"bytes": case["batch"] * 20 + case["capacity"] * 12 + pages * 8 + 16, "flops": 0}
    if op == "decode":
        if case["len_lo"] == case["len_hi"]:
            keys = case["len_hi"]
        elif case["len_hi"] - case["len_lo"] < 16:
            keys = (case["len_lo"] + case["len_hi"]) / 2
        else:
            a, b = case["len_lo"] + 1, case["len_hi"] + 1
            keys = (b - a) / math.log(b / a) - 1
        if case["local"] >= 0:  # at a full window: the sink blocks, whole local blocks and half of the own one
            keys = min(keys, (case["sink"] + case["local"] - 0.5) * case["block"] + 0.5)
        size, wide = 2, case["d"] + case["d_v"]
        return {"bytes": case["batch"] * (keys * case["kv_heads"] * wide * size + case["heads"] * (wide * size + 4)),
                "flops": case["batch"] * keys * case["heads"] * wide * 2}
    size = 4 if case["dtype"] == "fp32" else 2
    T = case["tokens"]
    half = case["rope_dim"] // 2
    if op == "rope":
        n = T * case["heads"] * case["d"]
        return {"bytes": 2 * n * size + 4 * T + 8 * half, "flops": T * case["heads"] * half * 6}
    H = case["heads"] + case["kv_heads"]
    n = T * H * case["d"]
    if op == "fwd":
        moved = 2 * n + (2 * T * case["kv_heads"] * case["d_v"])
        return {"bytes": moved * size + T * (12 if case["pooled"] else 4) + 8 * half + 2 * case["norm_dim"] * size,
                "flops": T * H * (case["norm_dim"] * 4 + half * 6)}
    return {"bytes": 3 * n * size + 4 * T + 8 * half + 2 * case["norm_dim"] * (size + 4),
            "flops": T * H * (case["norm_dim"] * 12 + half * 6)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _turn64(x, s, sign, case):
    """The rotation as complex products."""
    lo, half = case["rope_off"], case["rope_dim"] // 2
    w = torch.polar(torch.full_like(s["freq"], s["rope_scale"]).expand(len(s["pos"]), half).contiguous(),
                    sign * torch.outer(s["pos"].double(), s["freq"]))[:, None, :]
    out = x.clone()
    first = torch.arange(half, device=x.device) * (2 if case["interleaved"] else 1) + lo
    second = first + (1 if case["interleaved"] else half)
    z = torch.complex(x[..., first], x[..., second]) * w
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _norm64(x, w, n):
    out = x.clone()
    out[..., :n] = x[..., :n] / (x[..., :n].square().sum(-1, keepdim=True) / n + EPS).sqrt() * w.double()
    return out


def _grad64(x, dy, w, s, case):
    """Gradients of w . x / rms(x): with u = x / rms, dx = (g - u <g, u> / n) / rms."""
    n = case["norm_dim"]
    dx = _turn64(dy.double(), s, -1.0, case)
    xn = x[..., :n].double()
    rms = (xn.square().sum(-1, keepdim=True) / n + EPS).sqrt()
    u = xn / rms
    dw = torch.einsum("thn,thn->n", dx[..., :n], u)
    g = dx[..., :n] * w.double()
    dx[..., :n] = (g - u * ((g * u).sum(-1, keepdim=True) / n)) / rms
    return dx, dw


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "rope":
        return _turn64(s["x"].double(), s, 1.0, case)
    if op == "bwd":
        dq, dqw = _grad64(s["q"], s["dq"], s["qw"], s, case)
        dk, dkw = _grad64(s["k"], s["dk"], s["kw"], s, case)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    if op == "fwd":
        q = s["q"].double()
        q = _turn64(q if s["qw"] is None else _norm64(q, s["qw"], case["norm_dim"]), s, 1.0, case)
        k = _turn64(_norm64(s["k"].double(), s["kw"], case["norm_dim"]), s, 1.0, case)
        if not case["pooled"]:
            return {"q": q, "k": k}
        k_pool = s["k_pool"].double()
        k_pool.view(-1, *k_pool.shape[2:]).index_copy_(0, s["slots"], k)
        v_pool = None
        if s["v"] is not None:
            v_pool = s["v_pool"].double()
            v_pool.view(-1, *v_pool.shape[2:]).index_copy_(0, s["slots"], s["v"].double())
        return {"q": q, "k_pool": k_pool, "v_pool": v_pool}
    outs, lses = [], []
    group, lens = case["heads"] // case["kv_heads"], s["lens"].tolist()
    for n in range(case["batch"]):
        L = lens[n]
        if L == 0:
            outs.append(torch.zeros(case["heads"], case["d_v"], dtype=torch.float64, device="cuda"))
            lses.append(torch.full((case["heads"],), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        if case["local"] < 0:
            keys = torch.arange(L, device="cuda")
        else:
            first = max(0, ((L - 1) // case["block"] - case["local"] + 1) * case["block"])
            keys = torch.cat([torch.arange(min(L, first, case["sink"] * case["block"]), device="cuda"),
                              torch.arange(first, L, device="cuda")])
        pages, rows = s["table"][n].long()[keys // case["page"]], keys % case["page"]
        k, v = s["k_pool"][pages, rows].double(), s["v_pool"][pages, rows].double()
        q = s["q"][n].double().view(case["kv_heads"], group, case["d"])
        z = torch.einsum("hgd,khd->hgk", q, k) * s["scale"]
        lse = torch.logsumexp(z, -1)
        outs.append(torch.einsum("hgk,khd->hgd", torch.exp(z - lse[..., None]), v).reshape(case["heads"], -1))
        lses.append(lse.reshape(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
