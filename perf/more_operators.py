"""Cases of the operators at the two ends of a serving step and of the adapters in its middle:
cache pages and row maps planned on the GPU, embedding rows of a quantized table, low-rank
adapters of many requests, and the filtered draw of a token.

Every case is a dict of plain values with a "kind":

  plan   sequences are cut to what they keep and grown by new rows: pages, row starts, positions, slots
  embed  tokens' rows of a quantized table, scaled
  lora   each request's own adapter added to a shared projection's output
  draw   temperature, top-k, top-p and min-p of each row, and a token from a given random number

`run` computes them with elementary torch operations where `own` is false, and through the
library's entry points where it is true.  Sizes follow the shapes of a 31B-class dense model:
5376 embedding, 21504 FFN, 4096 query width, 262144 vocabulary.
"""
import math

import torch

own = False

DEV = "cuda"
GOLDEN = 0.6180339887498949
BLOCK = {"q8_0": (32, 34), "q4_0": (32, 18), "q4_k": (256, 144), "q6_k": (256, 210)}  # weights, bytes


# ---------------------------------------------------------------------------------------
# cases

def _plan(name, B, rows, ctx, page, slack):
    return {"name": name, "kind": "plan", "B": B, "rows": rows, "ctx": ctx, "page": page, "slack": slack}


def _embed(name, fmt, M, V, K):
    return {"name": name, "kind": "embed", "fmt": fmt, "M": M, "V": V, "K": K}


def _lora(name, B, rows, K, N, rank, slots, fmt, ragged):
    return {"name": name, "kind": "lora", "B": B, "rows": rows, "K": K, "N": N, "rank": rank, "slots": slots, "fmt": fmt,
            "ragged": ragged}


def _draw(name, M, V, filters, softcap, masked):
    return {"name": name, "kind": "draw", "M": M, "V": V, "filters": filters, "softcap": softcap, "masked": masked}


def listed():
    return [
        # one decoded token of 32 streams, drafts cut away, a stream that ends: latency
        _plan("plan_decode", 32, 5, 8192, 16, 1.0),
        # 256 requests with prompt chunks beside decoding ones: 100,000 rows mapped
        _plan("plan_chunks", 256, 1024, 16384, 16, 1.0),
        # the token just drawn, looked up in the 8-bit table that the logits use too: latency
        _embed("embed_one", "q8_0", 1, 262144, 5376),
        # a prompt chunk's tokens: bandwidth
        _embed("embed_chunk", "q4_k", 8192, 262144, 5376),
        # one stream with its adapter beside the FFN projection: latency
        _lora("lora_one", 1, 1, 5376, 21504, 16, 8, "bf16", False),
        # a serving batch of 32 streams over 24 adapters of ranks up to 64
        _lora("lora_decode", 32, 1, 5376, 21504, 64, 24, "bf16", True),
        # four prompts' chunks, one without an adapter, beside the FFN projection: bandwidth
        _lora("lora_chunk", 4, 512, 5376, 21504, 16, 8, "bf16", False),
        # prompts' chunks of odd lengths beside the output projection, adapters of rank 128 in float16
        _lora("lora_chunk_wide", 6, 333, 4096, 5376, 128, 4, "f16", True),
        # the next token of one stream, top-p over the whole vocabulary: latency
        _draw("draw_one", 1, 262144, "top_p", 30.0, False),
        # a serving batch of 32 streams, each with filters of its own
        _draw("draw_batch", 32, 262144, "mixed", 0.0, False),
        # 128 streams under a grammar that forbids most tokens
        _draw("draw_grammar", 128, 262144, "mixed", 0.0, True),
        # many streams of a small vocabulary, top-k and min-p
        _draw("draw_small_vocabulary", 256, 32000, "top_k", 0.0, False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    # no drawn case costs more than the largest listed one, and its plain form's float32
    # arrays stay within what the listed ones take
    most = max(_cost(c) for c in listed())
    while True:
        kind = rng.choice(["plan", "embed", "lora", "lora", "draw", "draw"])
        if kind == "plan":
            page = rng.choice([16, 32, 64, 128])
            c = _plan("", _spread(rng, 1, 512), _spread(rng, 1, 1024), _spread(rng, 64, 32768), page, rng.choice([0.2, 1.0]))
            fits = c["B"] * (c["ctx"] // page + 2) <= 1 << 20
        elif kind == "embed":
            fmt = rng.choice(["q8_0", "q4_0", "q4_k", "q6_k"])
            weights = BLOCK[fmt][0]
            c = _embed("", fmt, _spread(rng, 1, 8192), _spread(rng, 1000, 262144),
                       weights * _spread(rng, 512 // weights, 8192 // weights))
            fits = c["V"] * c["K"] <= 262144 * 5376
        elif kind == "lora":
            c = _lora("", _spread(rng, 1, 64), rng.choice([1, 1, _spread(rng, 2, 1024)]), 32 * _spread(rng, 8, 672),
                      _spread(rng, 96, 21504), rng.choice([8, 16, 16, 32, 64, 128]), _spread(rng, 1, 32),
                      rng.choice(["bf16", "f16"]), rng.random() < 0.5)
            fits = c["B"] * c["rows"] <= 4096 and (c["B"] + c["slots"]) * c["rank"] * (c["K"] + c["N"]) <= 1 << 29
        else:
            c = _draw("", _spread(rng, 1, 256), _spread(rng, 1000, 262144), rng.choice(["none", "top_k", "top_p", "mixed", "mixed"]),
                      rng.choice([0.0, 30.0]), rng.random() < 0.25)
            fits = c["M"] * c["V"] <= 128 * 262144
        del c["name"]
        if fits and _cost(c) <= most:
            return c


# ---------------------------------------------------------------------------------------
# the batch of a case, from the case alone

def _sequences(c):
    """Cached tokens, kept ones and new ones of each sequence: some end, some are new, some
    drop drafts, the others decode or bring a prompt's chunk."""
    length, keep, new = [], [], []
    for b in range(c["B"]):
        f = (b * GOLDEN) % 1.0
        n = max(1, round(c["rows"] * (1.0 - 0.6 * f)))
        cached = max(1, round((c["ctx"] - n) * (1.0 - 0.875 * f)))
        if b % 16 == 5:  # ends
            kept, n = 0, 0
        elif b % 8 == 2:  # a new request
            cached = kept = 0
        elif b % 2:  # rejected drafts
            kept = max(0, cached - 1 - b % 7)
        else:
            kept = cached
        length.append(cached)
        keep.append(kept)
        new.append(n)
    return length, keep, new


def _pages(x, page):
    return -(-x // page)


def _rows(c):
    """Rows of each sequence, and its adapter (-1: none).  Neighbours share adapters now and then."""
    rows, slot = [], []
    for b in range(c["B"]):
        f = (b * GOLDEN) % 1.0
        rows.append(max(1, round(c["rows"] * (1.0 - 0.5 * f))))
        slot.append(-1 if b % 8 == 3 else (b * 7 // 2) % c["slots"])
    return rows, slot


def _ranks(c):
    return [max(1, c["rank"] >> (s % 4)) if c["ragged"] else c["rank"] for s in range(c["slots"])]


def work(case):
    c = case
    if c["kind"] == "plan":
        length, keep, new = _sequences(c)
        page = c["page"]
        moved = sum(abs(_pages(k + n, page) - _pages(l, page)) for l, k, n in zip(length, keep, new))
        return {"bytes": 4 * (3 * c["B"] + 2 * c["B"] + 4) + 8 * moved + 12 * sum(new), "flops": 0}
    if c["kind"] == "embed":
        weights, size = BLOCK[c["fmt"]]
        return {"bytes": c["M"] * (c["K"] // weights * size + 4 * c["K"] + 4), "flops": 3 * c["M"] * c["K"]}
    if c["kind"] == "lora":
        rows, slot = _rows(c)
        ranks = _ranks(c)
        K, N = c["K"], c["N"]
        weights = sum(ranks[s] for s in set(slot) if s >= 0)
        used = [(n, ranks[s]) for n, s in zip(rows, slot) if s >= 0]
        return {"bytes": 2 * weights * (K + N) + sum(n for n, _ in used) * 4 * K + 8 * sum(rows) * N,
                "flops": sum(2 * n * r * (K + N) for n, r in used)}
    return {"bytes": 4 * c["M"] * c["V"], "flops": 8 * c["M"] * c["V"]}


# ---------------------------------------------------------------------------------------
# inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _half_bytes(g, shape, low, high):
    """float16 numbers of [low, high] as byte pairs."""
    x = torch.rand(shape, generator=g, device=DEV) * (high - low) + low
    return x.half().view(torch.uint8).view(*shape, 2)


def _table(c, g):
    """Rows of blocks [V][K / weights * bytes], every code used, scales of a trained table's size."""
    weights, size = BLOCK[c["fmt"]]
    V, nb = c["V"], c["K"] // weights
    w = torch.randint(0, 256, (V, nb, size), generator=g, device=DEV, dtype=torch.uint8)
    if c["fmt"] == "q8_0":
        w[..., :2] = _half_bytes(g, (V, nb), 2e-4, 9e-4)
    elif c["fmt"] == "q4_0":
        w[..., :2] = _half_bytes(g, (V, nb), 3e-3, 9e-3)
    elif c["fmt"] == "q4_k":
        w[..., :2] = _half_bytes(g, (V, nb), 4e-5, 2e-4)
        w[..., 2:4] = _half_bytes(g, (V, nb), 4e-4, 1e-3)
    else:
        w[..., 208:] = _half_bytes(g, (V, nb), 5e-6, 3e-5)
    return w.view(V, nb * size)


def _prepare_plan(c, g, s):
    length, keep, new = _sequences(c)
    page = c["page"]
    grown = [max(_pages(l, page), _pages(k + n, page)) for l, k, n in zip(length, keep, new)]
    spare = sum(grown) - sum(_pages(l, page) for l in length)
    in_use = sum(_pages(l, page) for l in length)
    free = spare + 1 + int(c["slack"] * spare)
    order = torch.randperm(in_use + free, generator=g, device=DEV).to(torch.int32)
    width = max(grown)
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device=DEV)
    held = _ints([_pages(l, page) for l in length]).long()
    cells = torch.arange(width, device=DEV)[None] < held[:, None]
    table[cells] = order[:in_use]
    stack = torch.full((in_use + free,), -1, dtype=torch.int32, device=DEV)
    stack[:free] = order[in_use:]
    T = sum(new) + 3  # a row buffer a little longer than the step
    s.update(table=table, stack=stack, count=_ints([free]), kv_len=_ints(length), keep=_ints(keep), n_new=_ints(new), T=T,
             new_len=_ints(length), new_count=_ints([0]), row_start=_ints([0] * (c["B"] + 1)), status=_ints([0, 0]),
             position=torch.full((T,), -1, dtype=torch.int32, device=DEV),
             slot=torch.full((T,), -1, dtype=torch.int64, device=DEV))


def _filters(c, g, s):
    """Each row's temperature, top-k, top-p and min-p, as a server's requests bring them."""
    M = c["M"]

    def pick(values):
        return torch.tensor(values, device=DEV)[torch.randint(0, len(values), (M,), generator=g, device=DEV)]

    kind = c["filters"]
    s["temperature"] = pick([0.6, 0.7, 0.8, 1.0, 1.0, 1.3])
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if kind == "mixed":
        s["temperature"] = pick([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.3])  # 0: the largest
    if kind in ("top_k", "mixed"):
        s["top_k"] = pick([0, 20, 40, 50, 64, 200, 1000] if kind == "mixed" else [20, 40, 50, 64, 100]).to(torch.int32)
    if kind in ("top_p", "mixed"):
        s["top_p"] = pick([1.0, 0.8, 0.9, 0.95] if kind == "mixed" else [0.8, 0.9, 0.95])
    if kind in ("top_k", "mixed"):
        s["min_p"] = pick([0.0, 0.02, 0.05, 0.1])


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["kind"] == "plan":
        _prepare_plan(c, g, s)
    elif c["kind"] == "embed":
        s["W"] = _table(c, g)
        s["tokens"] = torch.randint(0, c["V"], (c["M"],), generator=g, device=DEV).to(torch.int32)
        s["y"] = torch.empty(c["M"], c["K"], device=DEV)
        s["scale"] = math.sqrt(c["K"])
    elif c["kind"] == "lora":
        rows, slot = _rows(c)
        dtype = torch.bfloat16 if c["fmt"] == "bf16" else torch.float16
        R, K, N, T = c["rank"], c["K"], c["N"], sum(rows)
        s["A"] = (torch.randn(c["slots"], R, K, generator=g, device=DEV) / math.sqrt(K)).to(dtype)
        s["Bm"] = (torch.randn(c["slots"], N, R, generator=g, device=DEV) * 0.3 / math.sqrt(R)).to(dtype)
        s["rank"] = _ints(_ranks(c)) if c["ragged"] else None
        s["scale"] = torch.rand(c["slots"], generator=g, device=DEV) + 0.5
        s["slot"], s["row_start"] = _ints(slot), _ints(_starts(rows))
        s["x"] = torch.randn(T, K, generator=g, device=DEV)
        s["base"] = torch.randn(T, N, generator=g, device=DEV)  # the projection's output
        s["y"] = torch.empty(T, N, device=DEV)
        s["T"], s["n_max"] = T, max(rows)
    else:
        M, V = c["M"], c["V"]
        y = torch.randn(M, V, generator=g, device=DEV) * 2.0
        # the few tokens that a trained model prefers
        top = torch.randint(0, V, (M, 48), generator=g, device=DEV)
        y.scatter_reduce_(1, top, torch.rand(M, 48, generator=g, device=DEV) * 9.0 + 3.0, "amax")
        if c["masked"]:
            y.masked_fill_(torch.rand(M, V, generator=g, device=DEV) < 0.97, -math.inf)
        s["logits"] = y
        _filters(c, g, s)
        s["u"] = torch.rand(M, generator=g, device=DEV)
        s["token"] = torch.empty(M, dtype=torch.int32, device=DEV)
        s["kept"] = torch.empty(M, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------
# plain forms

def _plain_plan(s):
    c = s["case"]
    page, T = c["page"], s["T"]
    table, stack, count = s["table"], s["stack"], s["count"].long()
    B, width = table.shape
    n, keep = s["n_new"].long(), s["keep"].long()
    length = keep + n
    had, has = (s["kv_len"].long() + page - 1) // page, (length + page - 1) // page
    freed, need = (had - has).clamp_min(0), (has - had).clamp_min(0)
    pushed, popped = freed.cumsum(0), need.cumsum(0)
    start = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)])
    full = count + pushed[-1]
    lacking = (popped[-1] - full).clamp_min(0)
    status = torch.cat([(lacking > 0).long() + 2 * (start[-1:] > T).long(), lacking]).to(torch.int32)
    yes = status[:1] == 0
    # freed pages onto the stack, in order of sequences and positions; one cell behind it takes the others
    j = torch.arange(width, device=DEV)[None]
    out = torch.cat([stack, stack[:1]])
    leaves = (j >= has[:, None]) & (j < had[:, None]) & yes
    at = count + (pushed - freed)[:, None] + j - has[:, None]
    out[torch.where(leaves, at, stack.shape[0])] = table
    s["stack"].copy_(out[:-1])
    enters = (j >= had[:, None]) & (j < has[:, None]) & yes
    at = full - 1 - ((popped - need)[:, None] + j - had[:, None])
    table.copy_(torch.where(enters, out[at.clamp(0, stack.shape[0] - 1)], table))
    s["new_len"].copy_(torch.where(yes, length, s["kv_len"].long()))
    s["new_count"].copy_(torch.where(yes, full - popped[-1], count))
    s["row_start"].copy_(torch.where(yes, start, torch.zeros_like(start)))
    s["status"].copy_(status)
    r = torch.arange(T, device=DEV)
    b = (torch.searchsorted(start, r, right=True) - 1).clamp(0, B - 1)
    mine = (r < start[-1]) & yes
    p = torch.where(mine, keep[b] + r - start[b], torch.zeros_like(r))
    place = table[b, (p // page).clamp_max(width - 1)].long() * page + p % page
    s["position"].copy_(torch.where(mine, p, s["position"].long()))
    s["slot"].copy_(torch.where(mine, place, s["slot"]))
    return _planned(s)


def _planned(s):
    return [s[k] for k in ("table", "stack", "new_len", "new_count", "row_start", "status", "position", "slot")]


def _float16(b):
    return b.contiguous().view(torch.float16).float()


def _plain_embed(s):
    c = s["case"]
    weights, size = BLOCK[c["fmt"]]
    w = s["W"][s["tokens"].long()].view(c["M"], -1, size)
    if c["fmt"] == "q8_0":
        w = w[..., 2:].contiguous().view(torch.int8).float() * _float16(w[..., :2])
    elif c["fmt"] == "q4_0":
        codes = w[..., 2:]
        w = (torch.cat([codes & 15, codes >> 4], dim=-1).float() - 8.0) * _float16(w[..., :2])
    elif c["fmt"] == "q4_k":
        p = w[..., 4:16]
        low, mid, high = p[..., :4], p[..., 4:8], p[..., 8:]
        scales = torch.cat([low & 63, (high & 15) | ((low >> 6) << 4)], dim=-1).float()
        mins = torch.cat([mid & 63, (high >> 4) | ((mid >> 6) << 4)], dim=-1).float()
        codes = w[..., 16:].view(c["M"], -1, 4, 1, 32)  # 64 weights: low nibbles, then high ones
        codes = torch.cat([codes & 15, codes >> 4], dim=-2).view(c["M"], -1, 8, 32).float()
        d, dmin = _float16(w[..., :2]), _float16(w[..., 2:4])
        w = codes * (d * scales)[..., None] - (dmin * mins)[..., None]
    else:
        ql, qh = w[..., :128].view(c["M"], -1, 2, 2, 32), w[..., 128:192].view(c["M"], -1, 2, 1, 32)
        codes = torch.cat([ql & 15, ql >> 4], dim=-2)
        codes = codes | torch.cat([((qh >> f) & 3) << 4 for f in (0, 2, 4, 6)], dim=-2)
        scales = w[..., 192:208].contiguous().view(torch.int8).float() * _float16(w[..., 208:])
        w = (codes.reshape(c["M"], -1, 16, 16).float() - 32.0) * scales[..., None]
    return w.reshape(c["M"], c["K"]) * s["scale"]


def _plain_lora(s):
    c = s["case"]
    start, slot = s["row_start"].long(), s["slot"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(s["n_max"], device=DEV)
    real = i < n[:, None]
    row = (start[:-1, None] + i).clamp_max(s["T"] - 1)
    a, on = slot.clamp_min(0), (slot >= 0).float()
    A = s["A"][a].float()
    if s["rank"] is not None:
        A = A * (torch.arange(c["rank"], device=DEV) < s["rank"][a][:, None])[..., None]
    v = torch.matmul(s["x"][row], A.transpose(1, 2).contiguous())
    del A
    d = torch.matmul(v, s["Bm"][a].float().transpose(1, 2).contiguous()) * (s["scale"][a] * on)[:, None, None]
    return s["base"] + d[real]


def _plain_draw(s):
    """All in 64 bits: a drawn token changes where a running sum passes a border."""
    c = s["case"]
    y, order = s["logits"].sort(dim=1, descending=True, stable=True)
    some = y > -math.inf
    y = y.double()
    if c["softcap"]:
        y = torch.tanh(y / c["softcap"]) * c["softcap"]
    T = s["temperature"].double()[:, None]
    greedy = ~(T > 0)
    w = ((y - y[:, :1]) / torch.where(greedy, torch.ones_like(T), T)).exp_()
    w = torch.where(some, w, torch.zeros_like(w))
    del y
    i = torch.arange(c["V"], device=DEV)[None]
    n = some.sum(dim=1, keepdim=True)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        n = torch.where(k > 0, torch.minimum(n, k), n)
    run = w.cumsum(dim=1)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        border = p * run.gather(1, n - 1)
        n = torch.where(p < 1, torch.minimum(n, (run < border).sum(dim=1, keepdim=True) + 1), n)
    if s["min_p"] is not None:
        m = s["min_p"].double()[:, None]
        n = torch.where(m > 0, torch.minimum(n, ((w >= m) & some).sum(dim=1, keepdim=True)), n)
    n = torch.where(greedy, torch.ones_like(n), n.clamp_min(1))
    point = s["u"].double()[:, None] * run.gather(1, n - 1)
    at = torch.minimum(((run <= point) & (i < n)).sum(dim=1, keepdim=True), n - 1)
    return order.gather(1, at)[:, 0].to(torch.int32), n[:, 0].to(torch.int32)


# ---------------------------------------------------------------------------------------
# one pass

def _handles(s):
    """What a serving program keeps beside its buffers: the descriptions and the
    workspaces, none of which depends on the tensors' contents."""
    from quantized_dequant_matrix_amd import qmv

    c = s["case"]
    h = {"qmv": qmv}
    if c["kind"] == "plan":
        h["pool"] = qmv.KVPool(s["table"], s["stack"], c["page"])
        h["bytes"] = qmv.kv_plan_ws_bytes(h["pool"])
    elif c["kind"] == "lora":
        h["lora"] = qmv.Lora(s["A"], s["Bm"], s["scale"], s["rank"])
        h["bytes"] = qmv.lora_add_ws_bytes(h["lora"], c["B"], s["T"])
    elif c["kind"] == "draw":
        h["bytes"] = qmv.logits_draw_ws_bytes(c["V"], c["M"])
    if "bytes" in h:
        h["ws"] = torch.empty(h["bytes"], dtype=torch.uint8, device=DEV)
    return h


def run(state):
    s = state
    c = s["case"]
    kind = c["kind"]
    if not own:
        return {"plan": _plain_plan, "embed": _plain_embed, "lora": _plain_lora, "draw": _plain_draw}[kind](s)
    h = s.get("handles")
    if h is None:
        h = s["handles"] = _handles(s)
    qmv = h["qmv"]
    if kind == "plan":
        qmv.kv_plan(h["pool"], s["kv_len"], s["keep"], s["n_new"], s["count"], s["new_len"], s["new_count"], s["row_start"],
                    s["position"], s["slot"], s["status"], s["T"], h["ws"], h["bytes"])
        return _planned(s)
    if kind == "embed":
        getattr(qmv, "embed_" + c["fmt"])(s["W"], s["tokens"], s["y"], c["V"], c["K"], c["M"], s["scale"])
        return s["y"]
    if kind == "lora":
        qmv.lora_add(h["lora"], s["slot"], s["row_start"], s["x"], c["K"], s["base"], c["N"], s["y"], c["N"], c["B"], s["T"],
                     h["ws"], h["bytes"])
        return s["y"]
    qmv.logits_draw(s["logits"], c["V"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["token"], s["kept"],
                    c["V"], c["M"], c["softcap"], h["ws"], h["bytes"])
    return s["token"], s["kept"]


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, by blocks and by sequences

def _exact_row_weights(fmt, w):
    """Weights [M][blocks][weights] of blocks [M][blocks][bytes], element by element of the format."""
    def half(at):
        return w[:, :, at:at + 2].contiguous().view(torch.float16).double()

    byte = w.long()
    if fmt == "q8_0":
        q = byte[:, :, 2:]
        return (q - 256 * (q > 127)).double() * half(0)
    if fmt == "q4_0":
        e = torch.arange(32, device=DEV)
        q = (byte[:, :, 2 + e % 16] // torch.where(e < 16, 1, 16)) % 16
        return (q - 8).double() * half(0)
    e = torch.arange(256, device=DEV)
    if fmt == "q4_k":
        sub = e // 32
        q = (byte[:, :, 16 + 32 * (sub // 2) + e % 32] // torch.where(sub % 2 == 0, 1, 16)) % 16
        low = sub % 4
        first = sub < 4
        scale = torch.where(first, byte[:, :, 4 + low] % 64, byte[:, :, 12 + low] % 16 + 16 * (byte[:, :, 4 + low] // 64))
        least = torch.where(first, byte[:, :, 8 + low] % 64, byte[:, :, 12 + low] // 16 + 16 * (byte[:, :, 8 + low] // 64))
        return half(0) * scale * q - half(2) * least
    part, quarter, at = e // 128, (e // 32) % 4, e % 32
    q = (byte[:, :, 64 * part + 32 * (quarter % 2) + at] // torch.where(quarter < 2, 1, 16)) % 16
    q = q + 16 * ((byte[:, :, 128 + 32 * part + at] // (4 ** quarter)) % 4)
    scale = byte[:, :, 192 + e // 16]
    return half(208) * (scale - 256 * (scale > 127)) * (q - 32)


def exact(case, seed):
    c = case
    if c["kind"] in ("plan", "draw"):
        return None  # whole numbers only
    s = prepare(c, seed)
    if c["kind"] == "embed":
        size = BLOCK[c["fmt"]][1]
        out = torch.empty(c["M"], c["K"], dtype=torch.float64, device=DEV)
        for r in range(0, c["M"], 512):
            w = s["W"][s["tokens"][r:r + 512].long()].view(-1, c["K"] // BLOCK[c["fmt"]][0], size)
            out[r:r + 512] = _exact_row_weights(c["fmt"], w).reshape(-1, c["K"])
        # the scale is an argument in float32
        return out * float(torch.tensor(s["scale"], dtype=torch.float32))
    out = s["base"].double()
    rows, slot = _rows(c)
    ranks, at = _ranks(c), 0
    for n, a in zip(rows, slot):
        if a >= 0:
            R = ranks[a]
            v = s["x"][at:at + n].double() @ s["A"][a, :R].double().t()
            out[at:at + n] += float(s["scale"][a]) * (v @ s["Bm"][a, :, :R].double().t())
        at += n
    return out
