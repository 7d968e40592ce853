"""What the decode-window operators are measured on.

Three operators of the skinny-matmul library around one decode window:

  w4    C = A . W for 1 .. 16 rows and a 4-bit weight with one scale (and, if
        the weight has them, one zero point) per group of 32, 64 or 128
        elements along k: W[j][kk] = scale[j][kk/g] * (code[j][kk] - zero[j][kk/g])
  moe   a whole mixture-of-experts layer for the window's rows: the router's
        logits, its top-k and softmax, the routed experts' gated products, the
        shared expert behind its sigmoid gate, and the weighted sum
  lp    log probabilities of given tokens from rows of logits, with the
        distribution's entropy, the token's rank and the top alternatives

`own` selects who computes: False, the plain form below (elementary torch
operations in 32 bits, rounded once at the end); True, the library's kernels.
"""
import math

import torch

own = False


# --- the cases ---------------------------------------------------------------
def _w4(name, m, n, k, group, dtype, out, zeros):
    return {"name": name, "op": "w4", "m": m, "n": n, "k": k, "group": group, "dtype": dtype, "out": out,
            "zeros": zeros}


def _moe(name, m, experts, topk, d, inter, shared, weight, group, zeros, dtype, out, renorm):
    return {"name": name, "op": "moe", "m": m, "experts": experts, "topk": topk, "d": d, "inter": inter,
            "shared": shared, "weight": weight, "group": group, "zeros": zeros, "dtype": dtype, "out": out,
            "renorm": renorm}


def _lp(name, m, vocab, dtype, topk, masked):
    return {"name": name, "op": "lp", "m": m, "vocab": vocab, "dtype": dtype, "topk": topk, "masked": masked}


def listed():
    return [
        # a short projection of four window rows: a small weight, latency counts
        _w4("w4 4x512x2560", 4, 512, 2560, 64, "f16", "f16", False),
        # one token through the k = 896 projection, the finest groups, fp32 out
        _w4("w4 1x4864x896", 1, 4864, 896, 32, "bf16", "f32", True),
        # a full window through a wide projection
        _w4("w4 16x7680x2560", 16, 7680, 2560, 128, "bf16", "bf16", True),
        # three rows through an output head over an odd vocabulary, fp32 logits
        _w4("w4 3x100003x5120", 3, 100003, 5120, 128, "bf16", "f32", False),
        # one token, a small layer with few experts: latency counts
        _moe("moe 1 of 64", 1, 64, 4, 1024, 512, 0, "w4", 64, False, "f16", "f16", True),
        # one token through the 256-expert layer in bf16 with a shared expert
        _moe("moe 1 of 256 bf16", 1, 256, 10, 5120, 896, 896, "full", 0, False, "bf16", "bf16", True),
        # a verify window of five rows, many small experts, weights not renormalised, fp32 out
        _moe("moe 5 of 512", 5, 512, 10, 2560, 672, 0, "w4", 32, True, "f16", "f32", False),
        # a full window through the 256-expert layer in 4 bits, a wider shared expert
        _moe("moe 16 of 256", 16, 256, 10, 5120, 896, 1792, "w4", 128, True, "bf16", "bf16", True),
        # one sampled token, five alternatives: latency counts
        _lp("lp 1x32000", 1, 32000, "f32", 5, 0.0),
        # a full verify window over a large odd vocabulary
        _lp("lp 16x131071", 16, 131071, "bf16", 20, 0.0),
        # scoring under a constrained vocabulary: a third of the logits is masked out
        _lp("lp 512x50021", 512, 50021, "f16", 1, 0.35),
        # scoring a long prompt, ten alternatives for each position
        _lp("lp 2048x100003", 2048, 100003, "f32", 10, 0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4", "moe", "lp"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "w4":
        group = rng.choice([32, 64, 128])
        k = group * max(1, _log(rng, 256, 8192) // group)
        n = _log(rng, 64, min(131072, 100003 * 5120 // k))
        c = _w4("", rng.randint(1, 16), n, k, group, dtype, rng.choice(["f32", dtype]), rng.random() < 0.5)
    elif op == "moe":
        weight = rng.choice(["full", "w4"])
        group = rng.choice([32, 64, 128]) if weight == "w4" else 0
        unit = max(32, group)
        m = _log(rng, 1, 16)
        experts = _log(rng, 8, 512)
        topk = rng.randint(1, min(10, experts))
        d = unit * (_log(rng, 512, 5120) // unit)
        # the listed cases' largest expert, and (16-bit weights) largest layer
        most = min(896 * 5120 // d, 256 * 896 * 5120 // (experts * d) if weight == "full" else 1 << 20)
        inter = unit * max(1, _log(rng, unit, max(unit, min(2048, most))) // unit)
        shared = rng.choice([0, inter, unit * max(1, inter // (2 * unit))])
        c = _moe("", m, experts, topk, d, inter, shared, weight, group, rng.random() < 0.5 and weight == "w4", dtype,
                 rng.choice(["f32", dtype]), rng.random() < 0.5)
    else:
        vocab = _log(rng, 1000, 152000)
        m = _log(rng, 1, min(2048, 2048 * 100003 // vocab))
        c = _lp("", m, vocab, rng.choice(["f32", "bf16", "f16"]), rng.randint(1, 32), rng.choice([0.0, 0.0, 0.35, 0.9]))
    del c["name"]
    return c


# --- inputs ------------------------------------------------------------------
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _normal(g, shape, sd, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sd, generator=g)


def _codes(g, shape, group, dtype, zeros, sd):
    """A 4-bit grouped weight [..][k] of about the standard deviation sd:
    packed codes, scales and zero points (uint8) or None."""
    *lead, k = shape
    codes = torch.randint(0, 256, (*lead, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.empty((*lead, k // group), dtype=torch.float32, device="cuda")
    scales = scales.uniform_(0.7 * sd / 4.6, 1.3 * sd / 4.6, generator=g).to(dtype)
    z = None
    if zeros:
        z = torch.randint(5, 11, (*lead, k // group), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales, z


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "w4":
        dt = DTYPE[case["dtype"]]
        s["a"] = _normal(g, (case["m"], case["k"]), 1.0, dt)
        s["w"] = _codes(g, (case["n"], case["k"]), case["group"], dt, case["zeros"], 0.02)
    elif case["op"] == "moe":
        dt, d = DTYPE[case["dtype"]], case["d"]
        # weights that keep the activations near 1 at every width
        sd1, sd2 = 1.4 / math.sqrt(d), 1.4 / math.sqrt(case["inter"])

        def weight(shape, sd):
            if case["weight"] == "full":
                return _normal(g, shape, sd, dt)
            return _codes(g, shape, case["group"], dt, case["zeros"], sd)

        s["x"] = _normal(g, (case["m"], d), 1.0, dt)
        s["router"] = _normal(g, (case["experts"], d), sd1, dt)
        s["w13"] = weight((case["experts"], 2 * case["inter"], d), sd1)
        s["w2"] = weight((case["experts"], d, case["inter"]), sd2)
        s["shared"] = None
        if case["shared"]:
            s["shared"] = (weight((2 * case["shared"], d), sd1), weight((d, case["shared"]), sd2),
                           _normal(g, (d,), sd1, dt))
    else:
        dt, shape = DTYPE[case["dtype"]], (case["m"], case["vocab"])
        x = _normal(g, shape, 3.0, torch.float32).to(dt)
        # the tokens that a sampler took from these rows
        u = torch.rand(shape, device="cuda", generator=g).clamp_(1e-20, 1.0 - 1e-7)
        if case["masked"]:
            off = torch.rand(shape, device="cuda", generator=g) < case["masked"]
            off[:, 0] = False
            x.masked_fill_(off, -math.inf)
            del off
        s["tokens"] = (x.float() - torch.log(-torch.log(u))).argmax(dim=1)
        s["logits"] = x
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program that uses the library keeps: weights in its types, the
    layer's handle."""
    import row_gemv_decode_amd as sk

    c = s["case"]
    if c["op"] == "w4":
        s["W"] = sk.W4(*s["w"])
    elif c["op"] == "moe":
        def as_w(w):
            return sk.W4(*w) if isinstance(w, tuple) else w

        shared = {}
        if s["shared"] is not None:
            w13, w2, gate = s["shared"]
            shared = {"shared13": as_w(w13), "shared2": as_w(w2), "shared_gate": gate}
        s["layer"] = sk.MoELayer(s["router"], as_w(s["w13"]), as_w(s["w2"]), topk=c["topk"], renorm=c["renorm"],
                                 out_dtype=DTYPE[c["out"]], max_m=16, **shared)


# --- the plain form ----------------------------------------------------------
def _dequant(codes, scales, zeros):
    """[..][k] fp32 from packed codes (element 2i in the low nibble of byte i)."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).float()
    q = q.view(*scales.shape, -1)  # [..][groups][g]
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q - z) * scales.float().unsqueeze(-1)).flatten(-2)


def _plain_w4(s):
    w = _dequant(*s["w"])
    return (s["a"].float() @ w.T).to(DTYPE[s["case"]["out"]])


def _pick(w, idx):
    if isinstance(w, tuple):
        return _dequant(*(None if t is None else t[idx] for t in w))
    return w[idx].float()


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _top(x, topk):
    """The topk largest of each row, equal values by lower index first."""
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    return v[..., :topk], i[..., :topk]


def _plain_moe(s):
    c = s["case"]
    x = s["x"].float()
    logits = x @ s["router"].float().T
    v, idx = _top(logits, c["topk"])
    e = torch.exp(v - v[:, :1])
    total = e.sum(1, keepdim=True) if c["renorm"] else torch.exp(logits - v[:, :1]).sum(1, keepdim=True)
    p = e / total
    flat = idx.flatten()
    xr = x.repeat_interleave(c["topk"], dim=0).unsqueeze(-1).contiguous()
    y = torch.bmm(_pick(s["w13"], flat), xr).squeeze(-1)
    h = _silu(y[:, :c["inter"]]) * y[:, c["inter"]:]
    o = torch.bmm(_pick(s["w2"], flat), h.unsqueeze(-1).contiguous()).squeeze(-1)
    out = (o.view(c["m"], c["topk"], -1) * p.unsqueeze(-1)).sum(1)
    if s["shared"] is not None:
        w13, w2, gate = s["shared"]
        w13, w2 = (_dequant(*w) if isinstance(w, tuple) else w.float() for w in (w13, w2))
        y = x @ w13.T
        h = _silu(y[:, :c["shared"]]) * y[:, c["shared"]:]
        out = out + (h @ w2.T) / (1.0 + torch.exp(-(x @ gate.float()))).unsqueeze(-1)
    return out.to(DTYPE[c["out"]])


def _plain_lp(s):
    x, t = s["logits"].float(), s["tokens"].unsqueeze(1)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    lp = torch.where(e > 0, x - lse, 0.0)
    entropy = -(e * lp).sum(1) / total.squeeze(1)
    xt = x.gather(1, t)
    col = torch.arange(x.shape[1], device=x.device)
    rank = 1 + ((x > xt) | ((x == xt) & (col < t))).sum(1)
    v, i = _top(x, s["case"]["topk"])
    return (xt - lse).squeeze(1), entropy, rank.to(torch.int32), i.to(torch.int32), v - lse


def run(state):
    op = state["case"]["op"]
    if own:
        if op == "w4":
            import row_gemv_decode_amd as sk

            return sk.mm_w4(state["a"], state["W"], out_dtype=DTYPE[state["case"]["out"]])
        if op == "moe":
            return state["layer"](state["x"])
        import row_gemv_decode_amd as sk

        return tuple(sk.token_logprobs(state["logits"], state["tokens"], topk=state["case"]["topk"]))
    return {"w4": _plain_w4, "moe": _plain_moe, "lp": _plain_lp}[op](state)


# --- what a pass cannot do without -------------------------------------------
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _weight_bytes(rows, k, case):
    if case.get("weight") == "full":
        return rows * k * SIZE[case["dtype"]]
    return rows * (k // 2 + (k // case["group"]) * (SIZE[case["dtype"]] + (1 if case["zeros"] else 0)))


def work(case):
    if case["op"] == "w4":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _weight_bytes(n, k, case) + m * k * SIZE[case["dtype"]] + m * n * SIZE[case["out"]],
                "flops": 2.0 * m * n * k}
    if case["op"] == "moe":
        m, d, inter, e, topk = case["m"], case["d"], case["inter"], case["experts"], case["topk"]
        distinct = e * (1.0 - (1.0 - topk / e) ** m)  # the experts that m tokens reach, on average
        expert = _weight_bytes(2 * inter, d, case) + _weight_bytes(d, inter, case)
        bytes_ = e * d * SIZE[case["dtype"]] + distinct * expert + m * d * (SIZE[case["dtype"]] + SIZE[case["out"]])
        flops = 2.0 * m * d * (e + 3 * inter * topk + 3 * case["shared"])
        if case["shared"]:
            bytes_ += _weight_bytes(2 * case["shared"], d, case) + _weight_bytes(d, case["shared"], case)
            bytes_ += d * SIZE[case["dtype"]]
        return {"bytes": bytes_, "flops": flops}
    n = case["m"] * case["vocab"]
    # per logit: a difference, an exponential, two sums, a product, a comparison
    return {"bytes": n * SIZE[case["dtype"]] + case["m"] * (20 + 8 * case["topk"]), "flops": 6.0 * n}


# --- the definition in 64 bits -----------------------------------------------
def _weight64(w, rows=slice(None)):
    """Rows of one weight in 64 bits, element by element from the definition."""
    if not isinstance(w, tuple):
        return w[rows].double()
    codes, scales, zeros = w
    codes, scales = codes[rows], scales[rows].double()
    out = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    out[:, 0::2] = (codes % 16).double()
    out[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    g = out.shape[1] // scales.shape[1]
    if zeros is None:
        out -= 8
    else:
        out -= zeros[rows].double().repeat_interleave(g, dim=1)
    out *= scales.repeat_interleave(g, dim=1)
    return out


def _expert64(x, w13, w2):
    inter = w13.shape[0] // 2
    gate, up = w13[:inter] @ x, w13[inter:] @ x
    return w2 @ (gate * torch.sigmoid(gate) * up)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "w4":
        a, n = s["a"].double(), case["n"]
        return torch.cat([a @ _weight64(s["w"], slice(j, min(n, j + 8192))).T for j in range(0, n, 8192)], dim=1)
    if case["op"] == "moe":
        of = (lambda w, e: tuple(None if t is None else t[e] for t in w) if isinstance(w, tuple) else w[e])
        router, rows = s["router"].double(), []
        for x in s["x"].double():
            p = torch.softmax(router @ x, dim=0)
            order = sorted(range(case["experts"]), key=lambda e, p=p.tolist(): (-p[e], e))[:case["topk"]]
            total = sum(p[e] for e in order) if case["renorm"] else 1.0
            row = torch.zeros_like(x)
            for e in order:
                row += p[e] / total * _expert64(x, _weight64(of(s["w13"], e)), _weight64(of(s["w2"], e)))
            if s["shared"] is not None:
                w13, w2, gate = s["shared"]
                row += torch.sigmoid(gate.double() @ x) * _expert64(x, _weight64(w13), _weight64(w2))
            rows.append(row)
        return torch.stack(rows)
    outs = []
    for x, t in zip(s["logits"].split(256), s["tokens"].split(256)):
        x = x.double()
        lp = x - torch.logsumexp(x, dim=1, keepdim=True)
        entropy = torch.special.entr(lp.exp()).sum(1)
        mine = x.gather(1, t[:, None])
        before = torch.arange(x.shape[1], device=x.device)[None] < t[:, None]
        rank = 1 + (x > mine).sum(1) + ((x == mine) & before).sum(1)
        ids = torch.argsort(x, dim=1, descending=True, stable=True)[:, :case["topk"]]
        outs.append((lp.gather(1, t[:, None])[:, 0], entropy, rank.to(torch.int32), ids.to(torch.int32),
                     lp.gather(1, ids)))
    return tuple(torch.cat(o) for o in zip(*outs))
