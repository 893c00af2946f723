"""The products of a mixture-of-experts block, as they are measured.

Four operators, each in a plain form (elementary torch operations in 32 or 64
bits) and, where ``own`` is true, as calls of this package:

* ``linear``: y = x W^T in 8-bit integers.  Row i of x has the scale
  s_i = fp32(max_k |x_ik| / 127) and the integers q_ik = x_ik / s_i rounded to
  the nearest (ties to even), W is given as integers with one scale per output
  channel: y_io = s_i w_o sum_k q_ik Q_ok + b_o.
* ``group``: token t picks the experts ids[t][0..top_k); the picks are put in
  the order of their experts (inside one, of their tokens): ``offsets`` of the
  experts' groups, the token of each grouped row, the row of each pick.  Ids
  outside 0..n_experts-1 (padded tokens) get no row.
* ``experts``: y_r = x_src(r) W_e^T for the rows r of expert e's group, W_e =
  (C1[i1] + C2[i2]) s + t stored as bit-packed codebook indices.
* ``combine``: y_t = sum_j w_tj z_pos(t,j) over a token's picks.
"""
import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# The cases.
# ---------------------------------------------------------------------------
def _linear(name, m, n, k, dt="bf16", out="bf16", bias=False, fused=True):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "dt": dt, "out": out, "bias": bias, "fused": fused}


def _group(name, tokens, top_k, experts, pad):
    return {"name": name, "op": "group", "tokens": tokens, "top_k": top_k, "experts": experts, "pad": pad}


def _experts(name, tokens, top_k, experts, n, k, d, b1, b2, layout, gather=True, shared=False, pad=0, dt="bf16", out="bf16",
             bias=False):
    return {"name": name, "op": "experts", "tokens": tokens, "top_k": top_k, "experts": experts, "n": n, "k": k, "d": d,
            "b1": b1, "b2": b2, "layout": layout, "gather": gather, "shared": shared, "pad": pad, "dt": dt, "out": out,
            "bias": bias}


def _combine(name, tokens, top_k, n, pad, dt="bf16", out="bf16"):
    return {"name": name, "op": "combine", "tokens": tokens, "top_k": top_k, "n": n, "pad": pad, "dt": dt, "out": out}


def listed():
    return [
        # one token through a narrow 8-bit projection (key and value heads): the call's latency
        _linear("linear 1x1024x16384", 1, 1024, 16384),
        # a batch of decoding sequences through a square projection: the weights' bytes
        _linear("linear 24x8192x8192", 24, 8192, 8192, bias=True),
        # a ragged prompt, fp16, a width that is no multiple of a tile
        _linear("linear 333x4100x2000", 333, 4100, 2000, dt="fp16", out="fp16", bias=True, fused=False),
        # a long prompt through a square projection: integer throughput; the rows are quantised for several products
        _linear("linear 4096x8192x8192", 4096, 8192, 8192, fused=False),
        # routing of a decoding batch, the last tokens padding
        _group("group 16x8 of 64", 16, 8, 64, 2),
        # routing of a prefill chunk
        _group("group 8192x8 of 128", 8192, 8, 128, 77),
        # one token, two of eight 2.5-bit experts (12 + 8 bits for 8 weights), tiled order: decode
        _experts("experts 1x2 of 8", 1, 2, 8, 14336, 4096, 8, 12, 8, "tile4"),
        # a decoding batch over many narrow experts at 2.67 bits (d = 6), rows in order, a residual book of 16
        _experts("experts 48x4 of 64", 48, 4, 64, 2048, 2050, 6, 12, 4, "rows", pad=3, bias=True),
        # a short prompt over 2-bit experts with 2^16-entry books, already grouped (the down projection)
        _experts("experts 500x2 of 16", 500, 2, 16, 4096, 2048, 8, 16, 0, "rows", gather=False),
        # a long prompt, about a thousand rows for each of eight experts: tensor-core throughput
        _experts("experts 4096x2 of 8", 4096, 2, 8, 14336, 4096, 8, 12, 8, "tile4"),
        # the experts' results of a decoding batch back to their tokens
        _combine("combine 48x4x2048", 48, 4, 2048, 3),
        # the same for a prefill chunk
        _combine("combine 8192x8x4096", 8192, 8, 4096, 77),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["linear", "linear", "group", "experts", "experts", "experts", "combine"])
    if op == "linear":
        while True:
            m, n, k = _log(rng, 1, 4096), _log(rng, 1, 16384), _log(rng, 16, 16384)
            if n * k <= 1 << 27 and m * n * k <= 1 << 38:
                break
        c = _linear("", m, n, k, rng.choice(["bf16", "fp16"]), rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.5,
                    rng.random() < 0.5)
    elif op == "group":
        tokens, top_k = _log(rng, 1, 8192), rng.randint(1, 8)
        c = _group("", tokens, top_k, max(top_k, _log(rng, 2, 256)), rng.randint(0, tokens // 4))
    elif op == "combine":
        tokens = _log(rng, 1, 8192)
        c = _combine("", tokens, rng.randint(1, 8), _log(rng, 8, 4096), rng.randint(0, tokens // 4),
                     rng.choice(["bf16", "fp16"]), rng.choice(["bf16", "fp16"]))
    else:
        d, b1, b2 = rng.choice([(8, 16, 0), (8, 12, 8), (6, 12, 4), (8, 8, 8), (4, 8, 0), (8, 16, 8)])
        while True:
            tokens, top_k, experts = _log(rng, 1, 4096), rng.randint(1, 4), _log(rng, 2, 64)
            n, k = _log(rng, 64, 14336), _log(rng, 64, 8192)
            if top_k <= experts and experts * n * k <= 1 << 28 and tokens * top_k * n * k <= 1 << 38:
                break
        c = _experts("", tokens, top_k, experts, n, k, d, b1, b2, rng.choice(["rows", "tile4"]), rng.random() < 0.5,
                     rng.random() < 0.3, rng.randint(0, tokens // 4), rng.choice(["bf16", "fp16"]),
                     rng.choice(["bf16", "fp16"]), rng.random() < 0.5)
    del c["name"]
    return c


def _rows(c):
    return (c["tokens"] - c["pad"]) * c["top_k"]


def work(case):
    c = case
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        b = 2 * m * k + n * k + 4 * n + (2 * n if c["bias"] else 0) + m * n * (4 if c["out"] == "fp32" else 2)
        return {"bytes": b, "flops": 2 * m * n * k}
    if c["op"] == "group":
        picks = c["tokens"] * c["top_k"]
        return {"bytes": 12 * picks + 4 * (c["experts"] + 1), "flops": 0}
    if c["op"] == "combine":
        return {"bytes": 2 * _rows(c) * c["n"] + 8 * c["tokens"] * c["top_k"] + 2 * c["tokens"] * c["n"],
                "flops": 2 * _rows(c) * c["n"]}
    m, e = _rows(c), c["experts"]
    active = e * (1 - (1 - c["top_k"] / e) ** (c["tokens"] - c["pad"]))      # experts with a row, on average
    nvec = -(-c["k"] // c["d"])
    books = 2 * c["d"] * ((1 << c["b1"]) + ((1 << c["b2"]) if c["b2"] else 0))
    b = active * (c["n"] * nvec * (c["b1"] + c["b2"]) / 8 + c["n"] * (6 if c["bias"] else 4))
    b += books * (1 if c["shared"] else active)
    b += 2 * (c["tokens"] if c["gather"] else m) * c["k"] + 2 * m * c["n"] + 4 * m
    return {"bytes": b, "flops": 2 * m * c["n"] * c["k"]}


# ---------------------------------------------------------------------------
# Inputs, made on the GPU from the seed.
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _activations(g, rows, k):
    """N(0, 1) with 0.1 % of the columns twenty times as large (outlier channels)."""
    x = _normal(g, rows, k)
    x[:, torch.randperm(k, generator=g, device="cuda")[: round(0.001 * k)]] *= 20.0
    return x


def _routing(g, tokens, top_k, experts, pad):
    """Picks of a router that likes some experts better than others; the last tokens are padding."""
    score = _normal(g, tokens, experts) + 0.5 * _normal(g, experts)
    w, ids = score.topk(top_k, dim=1)
    ids = ids.to(torch.int32)
    if pad:
        ids[tokens - pad:] = -1
    return ids, torch.softmax(w, dim=1)


def _strided(t, ld):
    """t as the first columns of rows that are ld apart."""
    full = torch.zeros((t.shape[0], ld), dtype=t.dtype, device=t.device)
    full[:, : t.shape[1]] = t
    return full[:, : t.shape[1]]


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        s["x"] = _strided(_activations(g, m, k).to(_DT[c["dt"]]), -(-k // 8) * 8)
        w = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
        s["w"] = _strided(w, -(-k // 16) * 16)
        s["ws"] = (0.5 + _uniform(g, n)) * (0.06 / 127)
        s["b"] = _normal(g, n).to(torch.float16) if c["bias"] else None
        if own:
            from bit_packed_index_b200 import vq
            s["layer"] = vq.Int8Layer(s["w"], s["ws"], s["b"])
        return s
    if c["op"] == "group":
        s["ids"], _ = _routing(g, c["tokens"], c["top_k"], c["experts"], c["pad"])
        return s
    if c["op"] == "combine":
        e = max(64, c["top_k"])
        ids, s["wt"] = _routing(g, c["tokens"], c["top_k"], e, c["pad"])
        s["pos"] = _group_plain(ids, e)[2]
        s["z"] = _normal(g, max(1, _rows(c)), c["n"]).to(_DT[c["dt"]])
        return s
    e, n, k, d = c["experts"], c["n"], c["k"], c["d"]
    ids, _ = _routing(g, c["tokens"], c["top_k"], e, c["pad"])
    s["offsets"], rows, _ = _group_plain(ids, e)
    m = c["tokens"] * c["top_k"]
    s["rows"] = rows if c["gather"] else None
    x = _activations(g, c["tokens"] if c["gather"] else m, k)
    s["x"] = _strided(x.to(_DT[c["dt"]]), -(-k // 8) * 8)
    nvec = -(-k // d)
    s["idx"], s["books"] = [], []
    for b, std in ((c["b1"], 0.02), (c["b2"], 0.005)):
        if b:
            shape = ((e, n, -(-nvec * b // 128) * 4) if c["layout"] == "rows" else (e, -(-nvec // 4), -(-n * 4 * b // 128) * 4))
            s["idx"].append(torch.randint(-(1 << 31), 1 << 31, shape, generator=g, device="cuda", dtype=torch.int32))
            s["books"].append((_normal(g, 1 if c["shared"] else e, 1 << b, d) * std).to(torch.float16))
    s["scale"] = (0.5 + _uniform(g, e, n)).to(torch.float16)
    s["t"] = (_normal(g, e, n) * 1e-3).to(torch.float16)
    s["b"] = _normal(g, e, n).to(torch.float16) if c["bias"] else None
    s["y"] = torch.zeros((m, n), dtype=_DT[c["out"]], device="cuda")
    # which experts have rows, and the longest group: what a plain program plans its padded batch by
    count = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    s["active"] = torch.tensor([i for i, v in enumerate(count) if v], dtype=torch.int64, device="cuda")
    s["longest"] = max(count)
    if own:
        from bit_packed_index_b200 import vq
        s["layer"] = vq.Experts(n, k, d, [b for b in (c["b1"], c["b2"]) if b], s["idx"], s["books"], s["scale"], s["t"],
                                layout=c["layout"], out_bias=s["b"])
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(state):
    c = state["c"]
    if own:
        from bit_packed_index_b200 import vq
        if c["op"] == "linear":
            if c["fused"]:
                return vq.linear_i8(state["layer"], state["x"], out_dtype=_DT[c["out"]])
            q, scale = vq.quant_i8(state["x"])
            return vq.gemm_i8(state["layer"], q, scale, out_dtype=_DT[c["out"]])
        if c["op"] == "group":
            return vq.group_rows(state["ids"], c["experts"])
        if c["op"] == "combine":
            return vq.combine_rows(state["z"], state["pos"], state["wt"], out_dtype=_DT[c["out"]])
        return vq.gemm_experts(state["layer"], state["x"], state["offsets"], rows=state["rows"], out=state["y"])
    if c["op"] == "linear":
        return _linear_plain(state["x"], state["w"], state["ws"], state["b"], _DT[c["out"]])
    if c["op"] == "group":
        return _group_plain(state["ids"], c["experts"])
    if c["op"] == "combine":
        return _combine_plain(state["z"], state["pos"], state["wt"], _DT[c["out"]])
    return _experts_plain(state)


def _linear_plain(x, w, ws, b, out):
    top = x.float().abs().amax(dim=1, keepdim=True)
    s = (top.double() / 127.0).float()      # rounded once; fp32 by a number becomes a product with 1 / 127 on the GPU
    q = torch.round(x.double() / s.double()).clamp(-127, 127).float()       # 64 bits: quotients next to a half
    y = (q @ w.float().t()) * s * ws
    return (y if b is None else y + b.float()).to(out)


def _group_plain(ids, n_experts):
    flat = ids.reshape(-1)
    n = flat.numel()
    valid = (flat >= 0) & (flat < n_experts)
    hit = torch.arange(n_experts, dtype=torch.int32, device=flat.device)[:, None] == flat
    upto = hit.cumsum(dim=1, dtype=torch.int32)                              # picks of an expert so far
    offsets = torch.zeros(n_experts + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = upto[:, -1].cumsum(dim=0, dtype=torch.int32)
    at = flat.clamp(0, n_experts - 1).long()
    pos = offsets[at] + upto.gather(0, at[None, :])[0] - 1
    pos = torch.where(valid, pos, torch.full_like(pos, -1))
    rows = torch.full((n + 1,), -1, dtype=torch.int32, device=flat.device)
    token = torch.arange(n, dtype=torch.int32, device=flat.device) // ids.shape[1]
    rows.scatter_(0, torch.where(valid, pos, torch.full_like(pos, n)).long(), token)
    return offsets, rows[:n], pos.reshape(ids.shape)


def _combine_plain(z, pos, wt, out):
    live = pos >= 0
    picked = z[pos.clamp(min=0).long()].float()
    w = torch.where(live, wt, torch.zeros_like(wt))
    return (picked * w[:, :, None]).sum(dim=1).to(out)


def _fields(words, b, bit):
    """The b-bit fields that start at the given bits of the words' last dimension."""
    last = words.shape[-1] - 1
    lo = words[..., bit >> 5].long() & 0xFFFFFFFF
    hi = words[..., ((bit >> 5) + 1).clamp(max=last)].long() & 0xFFFFFFFF
    return ((lo | (hi << 32)) >> (bit & 31)) & ((1 << b) - 1)


def _indices(words, b, n, nvec, layout):
    """Indices [experts][n][nvec] of a stacked stream."""
    dev = words.device
    if layout == "rows":
        return _fields(words, b, torch.arange(nvec, device=dev) * b)
    f = _fields(words, b, torch.arange(4 * n, device=dev) * b)               # [experts][tiles][4 n]
    f = f.reshape(f.shape[0], f.shape[1], n, 4).permute(0, 2, 1, 3)
    return f.reshape(f.shape[0], n, -1)[:, :, :nvec]


def _centroids(st, which, active):
    """The centroids of book 0 or 1 that the active experts' indices select: [active][n][nvec][d]."""
    c, book = st["c"], st["books"][which]
    i = _indices(st["idx"][which][active], c["b2"] if which else c["b1"], c["n"], -(-c["k"] // c["d"]), c["layout"])
    if book.shape[0] == 1:
        return book[0].float()[i]
    return book[active].float()[torch.arange(i.shape[0], device=i.device)[:, None, None], i]


def _experts_plain(st):
    c, active = st["c"], st["active"]
    n, k, y = c["n"], c["k"], st["y"]
    m = y.shape[0]
    if not st["longest"]:
        return y
    w = _centroids(st, 0, active)
    if c["b2"]:
        w = w + _centroids(st, 1, active)
    w = w.reshape(w.shape[0], n, -1)[:, :, :k] * st["scale"][active].float()[:, :, None] + st["t"][active].float()[:, :, None]
    # the groups padded to the longest, one product for each active expert
    first, after = st["offsets"][active].long(), st["offsets"][active + 1].long()
    r = first[:, None] + torch.arange(st["longest"], device=y.device)
    live = r < after[:, None]
    r = torch.where(live, r, torch.full_like(r, m))
    src = r.clamp(max=m - 1) if st["rows"] is None else st["rows"][r.clamp(max=m - 1)].long().clamp(min=0)
    out = torch.bmm(st["x"].float()[src], w.transpose(1, 2))
    if st["b"] is not None:
        out = out + st["b"][active].float()[:, None, :]
    full = torch.zeros((m + 1, n), dtype=y.dtype, device=y.device)
    full[r.reshape(-1)] = out.reshape(-1, n).to(y.dtype)
    return full[:m]


# ---------------------------------------------------------------------------
# The definition in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "group":
        return None
    st = prepare(case, seed)
    if c["op"] == "linear":
        x = st["x"].double()
        s = np.abs(x.cpu().numpy()).max(axis=1) / 127.0
        s = torch.from_numpy(s.astype(np.float32).astype(np.float64)).cuda()[:, None]
        low = torch.floor(x / s)
        part = x - low * s                                                  # against half a step; ties to even
        up = (part > s / 2) | ((part == s / 2) & (low % 2 != 0))
        q = torch.clamp(low + up.double(), -127, 127)
        y = torch.einsum("mk,nk->mn", q, st["w"].double()) * s * st["ws"].double()[None, :]
        return y if st["b"] is None else y + st["b"].double()[None, :]
    if c["op"] == "combine":
        z = torch.cat([st["z"].double(), torch.zeros((1, c["n"]), dtype=torch.float64, device="cuda")])
        y = torch.zeros((c["tokens"], c["n"]), dtype=torch.float64, device="cuda")
        for j in range(c["top_k"]):
            y += st["wt"][:, j, None].double() * z[st["pos"][:, j].long()]  # row -1: the zeros
        return y
    y = torch.zeros((c["tokens"] * c["top_k"], c["n"]), dtype=torch.float64, device="cuda")
    nvec = -(-c["k"] // c["d"])
    off = st["offsets"].tolist()
    place = torch.arange(32, device="cuda", dtype=torch.int32)
    for e in range(c["experts"]):
        r0, r1 = off[e], off[e + 1]
        if r0 == r1:
            continue
        w = 0.0
        for words, book, b in zip(st["idx"], st["books"], (c["b1"], c["b2"])):
            bits = ((words[e][:, :, None] >> place) & 1).reshape(words.shape[1], -1)   # bit by bit, lowest first
            if c["layout"] == "rows":
                f = bits[:, : nvec * b].reshape(c["n"], nvec, b)
            else:
                f = bits[:, : 4 * c["n"] * b].reshape(-1, c["n"], 4, b).permute(1, 0, 2, 3).reshape(c["n"], -1, b)[:, :nvec]
            index = (f.int() << place[:b]).sum(dim=2)
            w = w + book[min(e, book.shape[0] - 1)].double()[index]
        w = w.reshape(c["n"], -1)[:, : c["k"]]
        w = w * st["scale"][e].double()[:, None] + st["t"][e].double()[:, None]
        x = st["x"][r0:r1] if st["rows"] is None else st["x"][st["rows"][r0:r1].long()]
        y[r0:r1] = x.double() @ w.t()
        if st["b"] is not None:
            y[r0:r1] += st["b"][e].double()
    return y
