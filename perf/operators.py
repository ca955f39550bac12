"""Cases of the decode-step operators that stand around the weight products: the paged
key/value cache (written, read back, attended over), the residual RMS norm in front of a
quantized product, and the verification of drafted tokens.

Every case is a dict of plain values with a "kind":

  kv            new keys and values go into the cache, then rows are read back
  attn          attention of each sequence's new tokens over its cached tokens
  norm          residual addition and RMS norm, float32 or 8-bit output
  norm_product  the same with 8-bit output, then the Q4_0 product that takes it
  verify        accept or reject drafted tokens, and draw the next token

`run` computes them with elementary torch operations where `own` is false, and through the
library's entry points where it is true.  Sizes follow the shapes of a 31B-class dense model:
5376 embedding, 21504 FFN, 262144 vocabulary, 32 query and 16 key/value heads of 128.
"""
import math

import torch

own = False

DEV = "cuda"
GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------------------
# cases

def _kv(name, B, n, ctx, heads, dim, page, fmt, read_all):
    return {"name": name, "kind": "kv", "B": B, "n": n, "ctx": ctx, "heads": heads, "dim": dim, "page": page,
            "fmt": fmt, "read_all": read_all}


def _attn(name, B, n, ctx, q_heads, heads, dim, page, window, fmt):
    return {"name": name, "kind": "attn", "B": B, "n": n, "ctx": ctx, "q_heads": q_heads, "heads": heads,
            "dim": dim, "page": page, "window": window, "fmt": fmt}


def listed():
    return [
        # one decoded token of one stream joins the cache and is read back: all latency
        _kv("kv_append_one", 1, 1, 777, 16, 128, 16, "q8", False),
        # four prompts' chunks are written, then the whole cached sequences are read back
        # (to move a cache elsewhere, or to check it): all bandwidth
        _kv("kv_chunk_read_all", 4, 1024, 8192, 16, 128, 64, "q8", True),
        # one stream decoding one token with about a thousand cached: latency
        _attn("attn_decode_one", 1, 1, 1001, 32, 16, 128, 16, 0, "q8"),
        # a serving batch of 32 streams of very different lengths, one token each
        _attn("attn_decode_batch", 32, 1, 16384, 32, 16, 128, 64, 0, "q8"),
        # eight drafted tokens of eight streams checked at once, a sliding-window layer
        _attn("attn_verify_window", 8, 8, 4099, 32, 16, 128, 32, 1024, "q8"),
        # two prompts' chunks over what is cached of them: matrix products bound it
        _attn("attn_prefill_chunk", 2, 1024, 6000, 32, 8, 128, 64, 0, "q8"),
        # a float16 cache with wide heads shared by eight query heads
        _attn("attn_decode_f16_wide", 16, 1, 8192, 16, 2, 256, 32, 0, "f16"),
        # the norm in front of the projections of one decoded token
        {"name": "norm_q8_one", "kind": "norm", "M": 1, "K": 5376, "out": "q8"},
        # the norm of a prefill chunk
        {"name": "norm_chunk", "kind": "norm", "M": 2048, "K": 5376, "out": "f32"},
        # norm and FFN projection of a batch of 16 rows
        {"name": "norm_product_16", "kind": "norm_product", "M": 16, "K": 5376, "N": 21504},
        # four drafted tokens of one stream
        {"name": "verify_one", "kind": "verify", "B": 1, "drafts": 4, "V": 262144, "temperature": 0.8, "softcap": 30.0,
         "ragged": False},
        # seven drafted tokens of 32 streams, some with fewer
        {"name": "verify_batch", "kind": "verify", "B": 32, "drafts": 7, "V": 262144, "temperature": 1.0, "softcap": 0.0,
         "ragged": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    # no drawn case costs more than the largest listed one, and its plain form's padded
    # float32 arrays stay within what the listed ones take
    most = max(_cost(c) for c in listed())
    while True:
        kind = rng.choice(["kv", "attn", "attn", "attn", "norm", "norm_product", "verify"])
        page = rng.choice([16, 32, 64, 128])
        fmt = rng.choice(["q8", "q8", "f16"])
        dim = rng.choice([64, 128, 128, 256])
        if kind == "kv":
            n = _spread(rng, 1, 1024)
            c = _kv("", _spread(rng, 1, 64), n, _spread(rng, n, 8192), rng.choice([1, 2, 3, 8, 16]), dim, page, fmt,
                    rng.random() < 0.5)
            padded = c["B"] * c["ctx"] * c["heads"] * dim
            limit = 4 * 8192 * 16 * 128
        elif kind == "attn":
            n = rng.choice([1, 1, _spread(rng, 2, 16), _spread(rng, 17, 1024)])
            heads = rng.choice([1, 2, 4, 8, 16])
            group = rng.choice([1, 2, 3, 4, 8])
            c = _attn("", _spread(rng, 1, 64), n, _spread(rng, max(n, 16), 16384), heads * group, heads, dim, page,
                      rng.choice([0, 0, 0, 128, 513, 1024]), fmt)
            padded = max(c["B"] * c["ctx"] * heads * dim, c["B"] * heads * group * n * c["ctx"])
            limit = 32 * 16384 * 16 * 128
        elif kind == "norm":
            c = {"name": "", "kind": kind, "M": _spread(rng, 1, 2048), "K": 32 * _spread(rng, 4, 672),
                 "out": rng.choice(["q8", "f32"])}
            padded, limit = c["M"] * c["K"], 2048 * 5376 * 2
        elif kind == "norm_product":
            c = {"name": "", "kind": kind, "M": _spread(rng, 1, 64), "K": 256 * _spread(rng, 2, 63),
                 "N": _spread(rng, 96, 21504)}
            padded, limit = c["N"] * c["K"], 21504 * 5376 * 2
        else:
            c = {"name": "", "kind": kind, "B": _spread(rng, 1, 32), "drafts": rng.randint(1, 8),
                 "V": _spread(rng, 1000, 262144), "temperature": rng.choice([0.6, 0.8, 1.0, 1.3]),
                 "softcap": rng.choice([0.0, 30.0]), "ragged": rng.random() < 0.5}
            padded, limit = c["B"] * (2 * c["drafts"] + 1) * c["V"], 32 * 15 * 262144
        del c["name"]
        if padded <= limit and _cost(c) <= most:
            return c


# ---------------------------------------------------------------------------------------
# the batch of a case, from the case alone: new tokens, cached tokens, rows

def _lengths(c):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    new, total = [], []
    for b in range(c["B"]):
        f = (b * GOLDEN) % 1.0
        n = max(1, round(c["n"] * (1.0 - 0.5 * f)))
        new.append(n)
        total.append(max(n, round(c["ctx"] * (1.0 - 0.875 * f))))
    return new, total


def _visible(c):
    """(row, key) pairs that a row may look at, and keys that any row looks at, over the batch."""
    pairs = keys = 0
    for n, total in zip(*_lengths(c)):
        w = c["window"] or total
        first = total - n
        keys += total - max(0, first - w + 1)
        # the rows' counts rise by one a row up to w, then stay
        a, b = min(first + 1, w), min(total, w)
        rising = b - a
        pairs += (a + b) * (rising + 1) // 2 + b * (n - rising - 1)
    return pairs, keys


def _drafts(c):
    return [c["drafts"] - (b * 3 % (c["drafts"] + 1) if c["ragged"] and b % 2 else 0) for b in range(c["B"])]


def work(case):
    c = case
    if c["kind"] == "kv":
        new, total = _lengths(c)
        width = c["heads"] * c["dim"]
        cell = width + 4 * c["heads"] if c["fmt"] == "q8" else 2 * width  # one token's keys, cached
        rows, back = sum(new), sum(total) if c["read_all"] else sum(new)
        return {"bytes": 2 * (rows * (4 * width + cell) + back * (cell + 4 * width)), "flops": 2 * rows * width * 3}
    if c["kind"] == "attn":
        pairs, keys = _visible(c)
        rows = sum(_lengths(c)[0])
        cell = c["dim"] + 4 if c["fmt"] == "q8" else 2 * c["dim"]
        return {"bytes": keys * c["heads"] * 2 * cell + 8 * rows * c["q_heads"] * c["dim"],
                "flops": 4 * pairs * c["q_heads"] * c["dim"]}
    if c["kind"] == "norm":
        return {"bytes": 16 * c["M"] * c["K"] + 4 * c["K"], "flops": 6 * c["M"] * c["K"]}
    if c["kind"] == "norm_product":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": 12 * M * K + N * K // 32 * 18 + 4 * M * N, "flops": 2 * M * N * K}
    rows = sum(2 * n + 1 for n in _drafts(c))
    return {"bytes": 4 * c["V"] * rows, "flops": 8 * c["V"] * rows}


# ---------------------------------------------------------------------------------------
# inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _cache(c, g, s):
    """A cache with every sequence's pages scattered over it, and the batch's tables."""
    new, total = _lengths(c)
    page, heads, dim = c["page"], c["heads"], c["dim"]
    pages = [-(-t // page) for t in total]
    count = sum(pages) + 3
    order = torch.randperm(count, generator=g, device=DEV).to(torch.int32)
    width = max(pages)
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (count, heads, page, dim)
    if c["fmt"] == "q8":
        for name in ("k", "v"):
            s["c" + name] = (_randn(g, *shape) * 42.0).round_().clamp_(-127, 127).to(torch.int8)
            s["c" + name + "_scale"] = (torch.rand(shape[:3], generator=g, device=DEV) + 0.5) * (3.0 / 127)
    else:
        for name in ("k", "v"):
            s["c" + name] = _randn(g, *shape).half()
            s["c" + name + "_scale"] = None
    s.update(table=table, row_start=_ints(_starts(new)), kv_len=_ints(total), rows=sum(new), n_max=max(new),
             len_max=max(total), total_rows=sum(total), all_start=_ints(_starts(total)))


def _q4_0(g, N, K):
    """Q4_0 weights as bytes [N][K / 32 * 18]: an fp16 scale and 16 code bytes a block."""
    nb = K // 32
    w = torch.randint(0, 256, (N, nb, 18), generator=g, device=DEV, dtype=torch.uint8)
    d = ((torch.rand(N, nb, generator=g, device=DEV) + 0.5) * (1.5 / (4.6 * math.sqrt(K)))).half()
    w[:, :, :2] = d.view(torch.uint8).view(N, nb, 2)
    return w.view(N, nb * 18)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["kind"] in ("kv", "attn"):
        _cache(c, g, s)
        T, width = s["rows"], c["heads"] * c["dim"]
        if c["kind"] == "kv":
            s["k"] = _randn(g, T, width) * 1.5
            s["v"] = _randn(g, T, width) * 0.7
            back = s["total_rows"] if c["read_all"] else T
            s["k_back"] = torch.empty(back, width, device=DEV)
            s["v_back"] = torch.empty(back, width, device=DEV)
        else:
            s["q"] = _randn(g, T, c["q_heads"] * c["dim"]) * 1.2
            s["out"] = torch.empty(T, c["q_heads"] * c["dim"], device=DEV)
            s["scale"] = 1.0 / math.sqrt(c["dim"])
    elif c["kind"] in ("norm", "norm_product"):
        M, K = c["M"], c["K"]
        s["x"] = _randn(g, M, K) * 0.8
        s["r"] = _randn(g, M, K) * 2.0
        s["w"] = 1.0 + 0.2 * _randn(g, K)
        s["z"] = torch.empty(M, K, device=DEV)
        if c["kind"] == "norm_product":
            s["W"] = _q4_0(g, c["N"], K)
            s["y"] = torch.empty(M, c["N"], device=DEV)
        elif c["out"] == "f32":
            s["y"] = torch.empty(M, K, device=DEV)
        s["codes"] = torch.empty(M, K, dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(M, K // 32, device=DEV)
    else:
        B, G, V = c["B"], c["drafts"], c["V"]
        s["target"] = _randn(g, B, G + 1, V) * 2.5
        s["draft"] = s["target"][:, :G] + _randn(g, B, G, V) * 1.0
        # the drafter's own draw: the largest of logit / T + Gumbel noise
        e = torch.empty(B, G, V, device=DEV).exponential_(generator=g)
        s["draft_tokens"] = (s["draft"] / c["temperature"] - e.log_()).argmax(dim=2).to(torch.int32)
        s["n_draft"] = _ints(_drafts(c))
        s["u"] = torch.rand(B, G + 1, generator=g, device=DEV)
        s["accepted"] = torch.empty(B, dtype=torch.int32, device=DEV)
        s["tokens"] = torch.empty(B, G + 1, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------
# plain forms

def _quantize(x):
    """Codes (as float32) and scales of the last axis.  A code is decided by x / d next to
    a border, so the quotients are taken in 64 bits and rounded to 32 once."""
    d = (x.abs().amax(dim=-1, keepdim=True).double() / 127.0).float()
    r = (x.double() / d.double()).float().double()
    q = (r.sign() * (r.abs() + 0.5).floor()).clamp(-127.0, 127.0).float()
    return torch.where(d > 0, q, torch.zeros_like(q)), d


def _places(s, start, rows):
    """Page, offset of `rows` rows that are the last positions of their sequences."""
    at = torch.arange(rows, device=DEV)
    b = torch.searchsorted(start.long(), at, right=True) - 1
    position = s["kv_len"].long()[b] - (start.long()[b + 1] - at)
    page = s["case"]["page"]
    return s["table"][b, position // page].long(), position % page


def _plain_kv(s):
    c = s["case"]
    heads, dim = c["heads"], c["dim"]
    page, at = _places(s, s["row_start"], s["rows"])
    back = (page, at) if not c["read_all"] else _places(s, s["all_start"], s["total_rows"])
    out = []
    for name in ("k", "v"):
        x = s[name].view(-1, heads, dim)
        cache, scale = s["c" + name], s["c" + name + "_scale"]
        if c["fmt"] == "q8":
            q, d = _quantize(x)
            cache[page, :, at] = q.to(torch.int8)
            scale[page, :, at] = d[..., 0]
            out.append((cache[back[0], :, back[1]].float() * scale[back[0], :, back[1]][..., None]).view(-1, heads * dim))
        else:
            cache[page, :, at] = x.half()
            out.append(cache[back[0], :, back[1]].float().view(-1, heads * dim))
    return out


def _plain_attn(s):
    c = s["case"]
    B, heads, dim, page = c["B"], c["heads"], c["dim"], c["page"]
    group, n_max = c["q_heads"] // heads, s["n_max"]
    start, length = s["row_start"].long(), s["kv_len"].long()
    table = s["table"].long().clamp_min(0)

    def sequences(name):  # [B, heads, positions, dim] in float32
        x = s["c" + name][table].float()
        if s["c" + name + "_scale"] is not None:
            x = x * s["c" + name + "_scale"][table][..., None]
        return x.transpose(1, 2).reshape(B, heads, -1, dim)

    n = start[1:] - start[:-1]
    i = torch.arange(n_max, device=DEV)
    row = (start[:-1, None] + i).clamp_max(s["rows"] - 1)
    real = i < n[:, None]
    position = (length - n)[:, None] + i
    q = s["q"].view(-1, heads, group, dim)[row].permute(0, 2, 1, 3, 4).reshape(B, heads, n_max * group, dim)
    k = sequences("k")
    scores = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    j = torch.arange(scores.shape[3], device=DEV)
    seen = (j <= position[..., None]) & real[..., None]
    if c["window"]:
        seen &= j > position[..., None] - c["window"]
    scores = scores.view(B, heads, n_max, group, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = scores.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(B, heads, n_max * group, -1), sequences("v")).view(B, heads, n_max, group, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(0, 2, 1, 3, 4)[real].reshape(-1, c["q_heads"] * dim)


def _plain_norm(s):
    z = s["x"] + s["r"]
    # 8-bit codes are decided next to a border by the last bit of the norm, so the mean
    # is taken in 64 bits and its root rounded to 32 once
    rstd = (1.0 / torch.sqrt(z.double().square().mean(dim=1, keepdim=True) + 1e-6)).float()
    return z, (z * rstd) * s["w"]


def _plain_norm_q8(s):
    z, y = _plain_norm(s)
    q, d = _quantize(y.view(y.shape[0], -1, 32))
    return z, (q * d).view_as(y)


def _plain_product(s):
    c = s["case"]
    z, x = _plain_norm_q8(s)
    w = s["W"].view(c["N"], c["K"] // 32, 18)
    d = w[:, :, :2].contiguous().view(torch.float16).float()
    codes = w[:, :, 2:]
    w = torch.cat([(codes & 15).float(), (codes >> 4).float()], dim=2).sub_(8.0).mul_(d).view(c["N"], c["K"])
    return z, torch.matmul(x, w.t())


def _plain_verify(s):
    """All in 64 bits: a drawn token changes where a running sum passes a border."""
    c = s["case"]
    B, G, V = c["B"], c["drafts"], c["V"]

    def softmax(y):
        y = y.double()
        if c["softcap"]:
            y = torch.tanh(y / c["softcap"]) * c["softcap"]
        y = (y - y.amax(dim=-1, keepdim=True)).div_(c["temperature"]).exp_()
        return y.div_(y.sum(dim=-1, keepdim=True))

    p, q = softmax(s["target"]), softmax(s["draft"])
    token = s["draft_tokens"].long()[..., None]
    u, n = s["u"].double(), s["n_draft"].long()
    i = torch.arange(G, device=DEV)
    yes = (u[:, :G] * q.gather(2, token)[..., 0] < p[:, :G].gather(2, token)[..., 0]) & (i < n[:, None])
    accepted = yes.long().cumprod(dim=1).sum(dim=1)
    b = torch.arange(B, device=DEV)
    weight = p[b, accepted]
    rest = (weight - q[b, accepted.clamp_max(G - 1)]).clamp_min(0.0)
    rest = torch.where(rest.sum(dim=1, keepdim=True) > 0, rest, weight)
    weight = torch.where((accepted < n)[:, None], rest, weight)
    run = weight.cumsum(dim=1)
    drawn = (run <= (u[:, G] * run[:, -1])[:, None]).sum(dim=1).clamp_max(V - 1)
    i = torch.arange(G + 1, device=DEV)
    padded = torch.cat([s["draft_tokens"].long(), drawn[:, None]], dim=1)
    tokens = torch.where(i < accepted[:, None], padded, torch.full_like(padded, -1))
    tokens[b, accepted] = drawn
    return accepted.to(torch.int32), tokens.to(torch.int32)


# ---------------------------------------------------------------------------------------
# one pass

def _handles(s):
    """What a serving program keeps beside its buffers: the cache and batch descriptions
    and the workspaces, none of which depends on the tensors' contents."""
    from quantized_dequant_matrix_amd import qmv

    c = s["case"]
    h = {"qmv": qmv}
    if c["kind"] in ("kv", "attn"):
        h["cache"] = qmv.KVCache(s["ck"], s["cv"], s["ck_scale"], s["cv_scale"])
        h["batch"] = qmv.KVBatch(s["table"], s["row_start"], s["kv_len"], s["rows"])
        if c["kind"] == "kv":
            h["all"] = qmv.KVBatch(s["table"], s["all_start"], s["kv_len"], s["total_rows"]) if c["read_all"] else h["batch"]
        else:
            h["bytes"] = qmv.attn_paged_ws_bytes(h["cache"], h["batch"], c["q_heads"])
    elif c["kind"] == "norm_product":
        h["bytes"] = qmv.qmm_q4_0_q8_ws_bytes(c["N"], c["K"], c["M"])
    elif c["kind"] == "verify":
        h["bytes"] = qmv.draft_verify_ws_bytes(c["B"], c["drafts"], c["V"])
    if "bytes" in h:
        h["ws"] = torch.empty(h["bytes"], dtype=torch.uint8, device=DEV)
    return h


def run(state):
    s = state
    c = s["case"]
    kind = c["kind"]
    if not own:
        if kind == "kv":
            return _plain_kv(s)
        if kind == "attn":
            return _plain_attn(s)
        if kind == "norm":
            return _plain_norm_q8(s) if c["out"] == "q8" else _plain_norm(s)
        return _plain_product(s) if kind == "norm_product" else _plain_verify(s)
    h = s.get("handles")
    if h is None:
        h = s["handles"] = _handles(s)
    qmv = h["qmv"]
    if kind == "kv":
        width = c["heads"] * c["dim"]
        qmv.kv_write(h["cache"], h["batch"], s["k"], width, s["v"], width)
        qmv.kv_read(h["cache"], h["all"], s["k_back"], width, s["v_back"], width)
        return [s["k_back"], s["v_back"]]
    if kind == "attn":
        width = c["q_heads"] * c["dim"]
        qmv.attn_paged(h["cache"], h["batch"], s["q"], width, s["out"], width, c["q_heads"], s["scale"], c["window"],
                       h["ws"], h["bytes"])
        return s["out"]
    if kind == "norm" and c["out"] == "f32":
        qmv.rmsnorm_add(s["x"], s["r"], s["w"], s["z"], s["y"], c["K"], c["M"], 1e-6)
        return s["z"], s["y"]
    if kind == "norm":
        qmv.rmsnorm_add_q8(s["x"], s["r"], s["w"], s["z"], s["codes"], s["scales"], c["K"], c["M"], 1e-6)
        values = s["codes"].view(c["M"], -1, 32) * s["scales"][..., None]
        return s["z"], values.view(c["M"], c["K"])
    if kind == "norm_product":
        qmv.rmsnorm_add_q8(s["x"], s["r"], s["w"], s["z"], s["codes"], s["scales"], c["K"], c["M"], 1e-6)
        qmv.qmm_q4_0_q8(s["W"], s["codes"], s["scales"], s["y"], c["N"], c["K"], c["M"], h["ws"], h["bytes"])
        return s["z"], s["y"]
    qmv.draft_verify(s["target"], c["V"], s["draft"], c["V"], s["draft_tokens"], s["n_draft"], s["u"], s["accepted"],
                     s["tokens"], c["B"], c["drafts"], c["V"], c["temperature"], c["softcap"], h["ws"], h["bytes"])
    return s["accepted"], s["tokens"]


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence

def _exact_codes(x):
    """The quantizer is defined by its float32 steps (scale, quotient, half away from zero)."""
    d = (x.abs().max(dim=-1).values.double() / 127.0).float().unsqueeze(-1)
    t = torch.nan_to_num((x.double() / d.double()).float().double(), nan=0.0)
    q = torch.trunc(t + torch.copysign(torch.full_like(t, 0.5), t))
    return q.clamp(-127, 127), d.double()


def _exact_cached(s, name, b, count):
    """Sequence b's first `count` cached keys or values, [count][heads][dim] in 64 bits."""
    c = s["case"]
    pages = s["table"][b, : -(-count // c["page"])].long()
    x = s["c" + name][pages].double()
    if c["fmt"] == "q8":
        x = x * s["c" + name + "_scale"][pages].double().unsqueeze(-1)
    return x.permute(0, 2, 1, 3).reshape(-1, c["heads"], c["dim"])[:count]


def exact(case, seed):
    c = case
    if c["kind"] == "verify":
        return None  # whole numbers only
    s = prepare(c, seed)
    if c["kind"] == "kv":
        new, total = _lengths(c)
        out = []
        for name in ("k", "v"):
            rows, at = [], 0
            for b in range(c["B"]):
                x = s[name][at:at + new[b]].view(new[b], c["heads"], c["dim"])
                at += new[b]
                if c["fmt"] == "q8":
                    q, d = _exact_codes(x)
                    x = q * d
                else:
                    x = x.half().double()
                if c["read_all"]:
                    x = torch.cat([_exact_cached(s, name, b, total[b])[: total[b] - new[b]], x])
                rows.append(x.reshape(x.shape[0], -1))
            out.append(torch.cat(rows))
        return out
    if c["kind"] == "attn":
        new, total = _lengths(c)
        group, at, rows = c["q_heads"] // c["heads"], 0, []
        for b in range(c["B"]):
            n, L = new[b], total[b]
            first = max(0, L - n + 1 - c["window"]) if c["window"] else 0
            k, v = (_exact_cached(s, name, b, L)[first:] for name in ("k", "v"))
            q = s["q"][at:at + n].view(n, c["heads"], group, c["dim"]).double()
            at += n
            p = torch.arange(L - n, L, device=DEV)[:, None]
            j = torch.arange(first, L, device=DEV)[None]
            hidden = j > p
            if c["window"]:
                hidden |= j <= p - c["window"]
            o = torch.empty_like(q)
            for h in range(c["heads"]):
                for e in range(group):
                    a = (q[:, h, e] @ k[:, h].t()) * s["scale"]
                    o[:, h, e] = torch.softmax(a.masked_fill(hidden, -math.inf), dim=1) @ v[:, h]
            rows.append(o.view(n, -1))
        return torch.cat(rows)
    z32 = s["x"] + s["r"]
    z = z32.double()
    y = z / torch.sqrt((z * z).sum(dim=1, keepdim=True) / c["K"] + 1e-6) * s["w"].double()
    if c["kind"] == "norm" and c["out"] == "f32":
        return z, y
    # the codes are defined by the float32 norm
    rstd = (1.0 / torch.sqrt((z * z).sum(dim=1, keepdim=True) / c["K"] + 1e-6)).float()
    q, d = _exact_codes(((z32 * rstd) * s["w"]).view(c["M"], -1, 32))
    x = (q * d).view(c["M"], c["K"])
    if c["kind"] == "norm":
        return z, x
    w = s["W"].view(c["N"], c["K"] // 32, 18)
    scale = w[:, :, :2].contiguous().view(torch.float16).double()
    low, high = (w[:, :, 2:] % 16).double(), (w[:, :, 2:] // 16).double()
    return z, x @ ((torch.cat([low, high], dim=2) - 8.0) * scale).view(c["N"], c["K"]).t()
