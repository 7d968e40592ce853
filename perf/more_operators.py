"""What the operators of a batch of requests are measured on.

Three operators of the skinny-matmul library around the projections of a decode
step that serves several requests at once:

  norm    the residual's addition and a root-mean-square norm, with an output
          in 16 bits or in 8 bits (e4m3) with a scale per row or per group
  adapt   low-rank adapters beside a shared projection: to each row of the
          projection's output, the product of its request's adapter is added
  adjust  penalties for repeated tokens, biases and grammar masks on logits

`own` selects who computes: False, the plain form below (elementary torch
operations in 32 bits, rounded once at the end); True, the library's kernels.
"""
import math

import torch

own = False


# --- the cases ---------------------------------------------------------------
def _norm(name, m, d, x, residual, out, group):
    """residual: its type or "" (none); out: the 16/32-bit output's type or ""
    (none); group: -1 no 8-bit output, 0 one scale per row, else columns per scale."""
    return {"name": name, "op": "norm", "m": m, "d": d, "x": x, "residual": residual, "out": out, "group": group}


def _adapt(name, m, requests, adapters, rank, mixed, none, k, n, dtype, base, out):
    """Rows of `requests` requests, each of one of `adapters` adapters (a share
    `none` without one), of rank `rank` or (mixed) a quarter, half or all of it."""
    return {"name": name, "op": "adapt", "m": m, "requests": requests, "adapters": adapters, "rank": rank, "mixed": mixed,
            "none": none, "k": k, "n": n, "dtype": dtype, "base": base, "out": out}


def _adjust(name, m, vocab, dtype, out, history, biases, masks):
    """history: room for a row's tokens (0: no penalties); biases per row; masks:
    the share of rows with a grammar mask; out "": in place (masks only)."""
    return {"name": name, "op": "adjust", "m": m, "vocab": vocab, "dtype": dtype, "out": out, "history": history,
            "biases": biases, "masks": masks}


def listed():
    return [
        # one token between two layers: latency counts
        _norm("norm 1x5120", 1, 5120, "bf16", "bf16", "bf16", -1),
        # a window's rows for a projection in 8 bits, a scale per 128 columns
        _norm("norm 16x2560 e4m3/128", 16, 2560, "f16", "f16", "", 128),
        # a ragged batch over a residual stream that is kept in 32 bits
        _norm("norm 1983x896 f32", 1983, 896, "bf16", "f32", "bf16", -1),
        # long prompts into projections in 8 bits, a scale per row
        _norm("norm 16384x5120 e4m3", 16384, 5120, "bf16", "bf16", "", 0),
        # one request's token: latency counts
        _adapt("adapt 1 of 8", 1, 1, 8, 16, False, 0.0, 2560, 7680, "bf16", "bf16", "bf16"),
        # a window of sixteen requests, some without an adapter, fp32 throughout
        _adapt("adapt 16 of 32", 16, 16, 32, 16, False, 0.2, 5120, 5120, "f16", "f32", "f32"),
        # a large decode batch over many adapters of several ranks, an odd width
        _adapt("adapt 250 of 64", 250, 250, 64, 64, True, 0.1, 4096, 5003, "bf16", "f32", "bf16"),
        # twelve prompts together through a wide projection
        _adapt("adapt 4096 in 12 of 8", 4096, 12, 8, 32, False, 0.1, 5120, 7680, "bf16", "bf16", "bf16"),
        # one request's next token, a short history: latency counts
        _adjust("adjust 1x32000", 1, 32000, "f32", "f32", 300, 8, 0.0),
        # sixteen requests with histories and grammars, 16-bit logits to 32 bits for the sampler
        _adjust("adjust 16x131071", 16, 131071, "bf16", "f32", 4096, 16, 0.5),
        # structured output: grammar masks alone, where the logits lie
        _adjust("adjust 256x50021 in place", 256, 50021, "f16", "", 0, 0, 0.9),
        # a large batch with all of it
        _adjust("adjust 512x100003", 512, 100003, "f32", "f32", 1024, 32, 0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "adapt", "adjust"])
    half = rng.choice(["bf16", "f16"])
    if op == "norm":
        d = _log(rng, 64, 16384)
        if rng.random() < 0.75:
            d = max(64, d // 64 * 64)
        residual = rng.choice(["", half, half, "f32"])
        group = rng.choice([-1, -1, 0, 32, 64, 128])
        out = rng.choice([half, half, "f32"]) if group < 0 or rng.random() < 0.25 else ""
        x = rng.choice([half, half, half, "f32"])
        row = d * (SIZE[x] + 2 * SIZE.get(residual, 0) + SIZE.get(out, 0) + 1)
        c = _norm("", _log(rng, 1, min(65536, 16384 * 5120 * 7 // row, 16384 * 5120 // d)), d, x, residual, out, group)
    elif op == "adapt":
        k, n = 8 * (_log(rng, 256, 8192) // 8), _log(rng, 64, 8192)
        rank = rng.choice([8, 16, 16, 32, 64, 128])
        adapters = _log(rng, 1, min(256, 4096 // rank))
        base, out = rng.choice([half, "f32"]), rng.choice([half, "f32"])
        # the largest listed case's rows and products
        row = 2 * k + (SIZE[base] + SIZE[out]) * n
        m = _log(rng, 1, min(4096, 4096 * (5120 + 2 * 7680) * 2 // row, 3600 * 32 * (5120 + 7680) // (rank * (k + n))))
        requests = m if m <= 64 or rng.random() < 0.4 else rng.randint(1, 32)
        c = _adapt("", m, requests, adapters, rank, rng.random() < 0.5, rng.choice([0.0, 0.1, 0.3]), k, n, half, base, out)
    else:
        vocab = _log(rng, 1000, 152000)
        m = _log(rng, 1, min(512, 512 * 100003 // vocab))
        history = rng.choice([0, _log(rng, 1, 16384)])
        biases = rng.choice([0, 0, _log(rng, 1, 300)])
        masks = rng.choice([0.0, 0.5, 1.0]) if history or biases else rng.choice([0.5, 1.0])
        dtype = rng.choice(["f32", half])
        out = rng.choice([dtype, "f32"]) if history or biases or rng.random() < 0.5 else ""
        c = _adjust("", m, vocab, dtype, out, history, biases, masks)
    del c["name"]
    return c


# --- inputs ------------------------------------------------------------------
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def _normal(g, shape, sd, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sd, generator=g)


def _uniform(g, shape, lo, hi):
    return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(lo, hi, generator=g)


def _ints(g, shape, lo, hi):
    return torch.randint(lo, hi, shape, dtype=torch.int32, device="cuda", generator=g)


def _prepare_norm(c, g, s):
    m, d = c["m"], c["d"]
    # activations whose size differs from row to row, with a few channels far above the rest
    sd = torch.exp(_normal(g, (m, 1), 0.5, torch.float32))
    x = _normal(g, (m, d), 1.0, torch.float32).mul_(sd)
    x[:, :: max(1, d // 4)] *= 20.0
    s["x"] = x.to(DTYPE[c["x"]])
    del x
    s["weight"] = _uniform(g, (d,), 0.5, 1.5).to(DTYPE[c["x"]])
    s["residual"] = _normal(g, (m, d), 2.0, DTYPE[c["residual"]]) if c["residual"] else None
    # the buffers that a step's program keeps
    s["residual_out"] = torch.empty_like(s["residual"]) if c["residual"] else None
    s["out"] = torch.empty((m, d), dtype=DTYPE[c["out"]], device="cuda") if c["out"] else None
    s["q"] = s["scales"] = None
    if c["group"] >= 0:
        groups = -(-d // c["group"]) if c["group"] else 1
        s["q"] = torch.empty((m, d), dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty((m, groups), dtype=torch.float32, device="cuda")


def _prepare_adapt(c, g, s):
    m, k, n, rank, dt = c["m"], c["k"], c["n"], c["rank"], DTYPE[c["dtype"]]
    s["x"] = _normal(g, (m, k), 1.0, dt)
    s["A"] = _normal(g, (c["adapters"], rank, k), 1.0 / math.sqrt(k), dt)
    s["B"] = _normal(g, (c["adapters"], n, rank), 0.5 / math.sqrt(rank), dt)
    s["scaling"] = _uniform(g, (c["adapters"],), 0.5, 2.0)
    s["ranks"] = torch.clamp(rank >> _ints(g, (c["adapters"],), 0, 3), min=1) if c["mixed"] else None
    which = _ints(g, (c["requests"],), 0, c["adapters"])
    which[_uniform(g, (c["requests"],), 0.0, 1.0) < c["none"]] = -1
    if c["requests"] < m:  # prompts of different lengths, one after another
        cuts = torch.sort(_ints(g, (c["requests"] - 1,), 1, m)).values
        s["ids"] = which[torch.searchsorted(cuts, torch.arange(m, dtype=torch.int32, device="cuda"), right=True)]
    else:
        s["ids"] = which
    s["base"] = _normal(g, (m, n), 1.0, DTYPE[c["base"]])
    s["out"] = torch.empty((m, n), dtype=DTYPE[c["out"]], device="cuda")


def _prepare_adjust(c, g, s):
    m, vocab = c["m"], c["vocab"]
    s["logits"] = _normal(g, (m, vocab), 3.0, DTYPE[c["dtype"]])
    s["history"] = s["bias_ids"] = s["mask"] = None
    if c["history"]:
        # text repeats itself: few tokens are many, and rows are as long as they are
        u = _uniform(g, (m, c["history"]), 0.0, 1.0)
        s["history"] = (u.pow_(4.0) * vocab).to(torch.int32).clamp_(max=vocab - 1)
        s["lengths"] = _ints(g, (m,), 0, c["history"] + 1)
        s["lengths"][0] = c["history"]
        s["prompt_lengths"] = (s["lengths"] * _uniform(g, (m,), 0.0, 1.0)).to(torch.int32)
        s["repetition"] = _uniform(g, (m,), 1.0, 1.5)
        s["frequency"] = _uniform(g, (m,), 0.0, 0.5)
        s["presence"] = _uniform(g, (m,), 0.0, 1.0)
    if c["biases"]:
        # lists of different lengths, filled up with -1
        s["bias_ids"] = _ints(g, (m, c["biases"]), 0, vocab)
        used = _ints(g, (m, 1), 0, c["biases"] + 1)
        s["bias_ids"][torch.arange(c["biases"], device="cuda")[None] >= used] = -1
        s["bias_values"] = _uniform(g, (m, c["biases"]), -10.0, 10.0)
    if c["masks"]:
        # one mask for each row that has a grammar: inside a text most tokens are
        # allowed, at a key word or a bracket very few
        on = _uniform(g, (m,), 0.0, 1.0) < c["masks"]
        on[0] = True
        rows, words = int(on.sum()), (vocab + 31) // 32
        share = torch.where(_uniform(g, (rows, 1), 0.0, 1.0) < 0.5, 0.002, 0.9)
        bits = (_uniform(g, (rows, 32 * words), 0.0, 1.0) < share).view(rows, words, 32)
        weight = (1 << torch.arange(32, dtype=torch.int64, device="cuda"))
        packed = torch.zeros((rows, words), dtype=torch.int64, device="cuda")
        for b in range(32):
            packed += bits[:, :, b] * weight[b]
        s["mask"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
        index = torch.cumsum(on.to(torch.int32), 0, dtype=torch.int32) - 1
        s["mask_rows"] = torch.where(on, index, -1).to(torch.int32)
    s["out"] = torch.empty((m, vocab), dtype=DTYPE[c["out"]], device="cuda") if c["out"] else None


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    {"norm": _prepare_norm, "adapt": _prepare_adapt, "adjust": _prepare_adjust}[case["op"]](case, g, s)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the library keeps beside its tensors: the pool of
    adapters, the rules' tensors that it fills from step to step."""
    import row_gemv_decode_amd as sk

    if s["case"]["op"] == "adapt":
        s["adapters"] = sk.Adapters(s["A"], s["B"], scaling=s["scaling"], ranks=s["ranks"])
    elif s["case"]["op"] == "adjust":
        more = {}
        if s["history"] is not None:
            more = {k: s[k] for k in ("history", "lengths", "prompt_lengths", "repetition", "frequency", "presence")}
        if s["bias_ids"] is not None:
            more |= {"bias_ids": s["bias_ids"], "bias_values": s["bias_values"]}
        if s["mask"] is not None:
            more |= {"mask": s["mask"], "mask_rows": s["mask_rows"]}
        s["rules"] = sk.LogitRules(s["case"]["m"], s["case"]["vocab"], **more)


# --- the plain form ----------------------------------------------------------
def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    outs = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        outs["residual"] = h.to(s["residual"].dtype)
    y = h * (1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)) * s["weight"].float()
    if c["out"]:
        outs["out"] = y.to(DTYPE[c["out"]])
    if c["group"] >= 0:
        d = c["d"]
        size = c["group"] or d
        groups = -(-d // size)
        padded = torch.nn.functional.pad(y, (0, groups * size - d)).view(-1, groups, size)
        scales = torch.clamp(padded.abs().amax(2) / 448.0, min=2.0 ** -126)
        q = torch.clamp(padded / scales.unsqueeze(2), -448.0, 448.0).to(torch.float8_e4m3fn)
        outs["q"] = q.view(-1, groups * size)[:, :d]
        outs["scales"] = scales
    return outs


def _plain_adapt(s):
    c = s["case"]
    ids, (count, rank, k) = s["ids"].long(), s["A"].shape
    # every adapter's product with every row, of which a row keeps its own adapter's
    h = (s["x"].float() @ s["A"].float().view(count * rank, k).T).view(-1, count, rank)
    keep = (ids[:, None] == torch.arange(count, device=ids.device)).unsqueeze(2)
    if s["ranks"] is not None:
        keep = keep & (torch.arange(rank, device=ids.device) < s["ranks"][:, None])
    h = torch.where(keep, h * s["scaling"][:, None], 0.0)
    b = s["B"].float().permute(0, 2, 1).reshape(count * rank, c["n"])
    return (s["base"].float() + h.view(-1, count * rank) @ b).to(DTYPE[c["out"]])


def _plain_adjust(s):
    c = s["case"]
    m, vocab = c["m"], c["vocab"]
    x = s["logits"].float()
    if s["history"] is not None:
        tokens = s["history"].long()
        place = torch.arange(c["history"], device=x.device)
        held = place < s["lengths"][:, None]
        made = held & (place >= s["prompt_lengths"][:, None])
        seen = torch.zeros_like(x).scatter_add_(1, tokens, held.float()) > 0
        count = torch.zeros_like(x).scatter_add_(1, tokens, made.float())
        theta = s["repetition"][:, None]
        x = torch.where(seen, torch.where(x > 0, x / theta, x * theta), x)
        x = x - (s["frequency"][:, None] * count + s["presence"][:, None] * (count > 0))
    if s["bias_ids"] is not None:
        ids = s["bias_ids"].long()
        x = x + torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, s["bias_values"], 0.0))
    if s["mask"] is not None:
        bits = (s["mask"].unsqueeze(2) >> torch.arange(32, dtype=torch.int32, device=x.device)) & 1
        allowed = bits.view(bits.shape[0], -1)[:, :vocab].bool()
        row = s["mask_rows"].long()
        x = torch.where(allowed[row.clamp(min=0)] | (row < 0)[:, None], x, -math.inf)
    if not c["out"]:
        return s["logits"].copy_(x)
    return x.to(DTYPE[c["out"]])


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import row_gemv_decode_amd as sk

        if op == "norm":
            group = s["case"]["group"]
            r = sk.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"], out=s["out"],
                            quant=None if group < 0 else group, q=s["q"], scales=s["scales"])
            return {k: v for k, v in r._asdict().items() if v is not None}
        if op == "adapt":
            return sk.add_adapters(s["x"], s["adapters"], s["ids"], s["base"], out=s["out"])
        return sk.adjust_logits(s["logits"], s["rules"], out=s["logits"] if s["out"] is None else s["out"])
    return {"norm": _plain_norm, "adapt": _plain_adapt, "adjust": _plain_adjust}[op](s)


# --- what a pass cannot do without -------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["m"] * c["d"]
        groups = 0 if c["group"] < 0 else -(-c["d"] // c["group"]) if c["group"] else 1
        each = SIZE[c["x"]] + 2 * SIZE.get(c["residual"], 0) + SIZE.get(c["out"], 0) + (1 if c["group"] >= 0 else 0)
        # per value: the addition, a product and a sum, two products, the scale's comparison and quotient
        return {"bytes": n * each + c["d"] * SIZE[c["x"]] + 4 * c["m"] * groups, "flops": 7.0 * n}
    if c["op"] == "adapt":
        m, k, n = c["m"], c["k"], c["n"]
        rank = c["rank"] * (7 / 12 if c["mixed"] else 1.0)
        # the adapters that the requests reach, on average
        distinct = c["adapters"] * (1.0 - (1.0 - (1.0 - c["none"]) / c["adapters"]) ** c["requests"])
        rows = m * (1.0 - c["none"])
        bytes_ = distinct * rank * (k + n) * SIZE[c["dtype"]] + rows * k * SIZE[c["dtype"]]
        bytes_ += m * n * (SIZE[c["base"]] + SIZE[c["out"]]) + 4 * m
        return {"bytes": bytes_, "flops": 2.0 * rows * rank * (k + n) + m * n}
    m, n = c["m"], c["m"] * c["vocab"]
    lists = 4 * m * (c["history"] / 2 + 5) * (c["history"] > 0) + 8 * m * c["biases"] + n * c["masks"] / 8
    if not c["out"]:  # the masked logits are written, half the masks leave 0.2 % and half 90 %
        return {"bytes": lists + n * c["masks"] * 0.549 * SIZE[c["dtype"]], "flops": float(n)}
    return {"bytes": lists + n * (SIZE[c["dtype"]] + SIZE[c["out"]]), "flops": 6.0 * n}


# --- the definition in 64 bits -----------------------------------------------
def _exact_norm(c, s):
    outs = {}
    h = s["x"].double()
    if s["residual"] is not None:
        h += s["residual"].double()
        outs["residual"] = h
    y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / c["d"] + EPS)
    y *= s["weight"].double()
    if c["out"]:
        outs["out"] = y
    if c["group"] >= 0:
        pieces = torch.split(y, c["group"] or c["d"], dim=1)
        scales = [torch.linalg.vector_norm(p, ord=math.inf, dim=1, keepdim=True) / 448 for p in pieces]
        # the values that the codes stand for, before they are rounded to 8 bits
        outs["q"] = torch.cat([p / t for p, t in zip(pieces, scales)], dim=1)
        outs["scales"] = torch.cat(scales, dim=1)
    return outs


def _exact_adapt(c, s):
    out = s["base"].double()
    for a in range(c["adapters"]):
        rows = torch.nonzero(s["ids"] == a).flatten()
        if rows.numel():
            r = c["rank"] if s["ranks"] is None else int(s["ranks"][a])
            inner = s["x"][rows].double() @ s["A"][a, :r].double().T
            out[rows] += float(s["scaling"][a]) * (inner @ s["B"][a, :, :r].double().T)
    return out


def _exact_adjust(c, s):
    vocab = c["vocab"]
    rows = []
    for i in range(c["m"]):
        x = s["logits"][i].double()
        if s["history"] is not None:
            held = s["history"][i, :int(s["lengths"][i])]
            made = torch.bincount(held[int(s["prompt_lengths"][i]):], minlength=vocab).double()
            some = torch.unique(held).long()
            theta = float(s["repetition"][i])
            x[some] = torch.minimum(x[some] / theta, x[some] * theta)  # theta >= 1: the smaller of the two
            x -= float(s["frequency"][i]) * made
            x -= float(s["presence"][i]) * made.clamp(max=1)
        if s["bias_ids"] is not None:
            used = s["bias_ids"][i] >= 0
            x.index_add_(0, s["bias_ids"][i][used].long(), s["bias_values"][i][used].double())
        if s["mask"] is not None and int(s["mask_rows"][i]) >= 0:
            word = s["mask"][int(s["mask_rows"][i])].long() & 0xFFFFFFFF
            j = torch.arange(vocab, device=x.device)
            x[(word[j // 32] // 2 ** (j % 32)) % 2 == 0] = -math.inf
        rows.append(x)
    return torch.stack(rows)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "adapt": _exact_adapt, "adjust": _exact_adjust}[case["op"]](case, s)
