"""Measured cases of a step of speculative decoding over the paged key-value cache: new rows that are
normed, rotated and appended to the pages, attention of a drafted tree over the pages, sampling from
logits, and a tree's bookkeeping (masks and positions, the accepted path, its rows' move in the pages).

A case is one call of one operator (an append to a quantised cache also reads the rows back, which is
what a prefill step does; the bookkeeping is the calls that a step makes, over its layers' caches).
`own` false: the operators in elementary torch operations; true: the library's entry points.
"""
import math

import torch

own = False

ROW_MAX = {"fp8": 448.0, "nvfp4": 2688.0}   # largest |value| / 2^e of a row
MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)   # midpoints between the e2m1 magnitudes
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
THETA, SSMAX_BASE, SSMAX_EXP, EPS = 10000.0, 2048.0, 0.1, 1e-6
MOST_NODES = 64
VOCAB = 201088   # of the repository's own LM head


# ---------------------------------------------------------------------------- cases ----

def listed():
    beam = {"n_q": 48, "n_kv": 8, "dim": 128}   # the repository's own head layout
    return [
        # a decode step of one sequence: one token, where latency counts
        {"name": "append_b1_bf16", "op": "append", "dtype": "bf16", "seqs": 1, "chunk": 1, "past": 700, "page": 64, "tree": False, "kind": "rope", "norm": True, "gate": True, **beam},
        # the drafted trees of a serving batch: slots apart from positions, quantised, read back
        {"name": "append_b32_tree16_fp8", "op": "append", "dtype": "fp8", "seqs": 32, "chunk": 16, "past": 5000, "page": 32, "tree": True, "kind": "ssmax", "norm": True, "gate": True, **beam},
        # the headline prefill chunk, 8 x 2048 tokens of a sliding-window layer
        {"name": "append_8x2048_bf16", "op": "append", "dtype": "bf16", "seqs": 8, "chunk": 2048, "past": 100, "page": 64, "tree": False, "kind": "rope", "norm": True, "gate": True, **beam},
        # a short conversation, a small tree: the smallest verification call
        {"name": "tree_b1_n5_ctx200_bf16", "op": "tree", "dtype": "bf16", "seqs": 1, "nodes": 5, "fewest": 5, "ctx": 200, "least": 200, "window": 0, "page": 16, "gate": True, **beam},
        # the headline context with the largest tree
        {"name": "tree_b1_n64_100k_bf16", "op": "tree", "dtype": "bf16", "seqs": 1, "nodes": 64, "fewest": 64, "ctx": 100000, "least": 100000, "window": 0, "page": 64, "gate": True, **beam},
        # a serving batch of unequal sequences with trees of unequal size
        {"name": "tree_b32_n16_8k_fp8", "op": "tree", "dtype": "fp8", "seqs": 32, "nodes": 16, "fewest": 1, "ctx": 16001, "least": 33, "window": 0, "page": 64, "gate": True, **beam},
        # a sliding-window layer, another head layout, 4 bits, odd sizes
        {"name": "tree_b48_n21_w512_nvfp4", "op": "tree", "dtype": "nvfp4", "seqs": 48, "nodes": 21, "fewest": 0, "ctx": 9001, "least": 1, "window": 512, "page": 32, "gate": False, "n_q": 32, "n_kv": 4, "dim": 64},
        # the next token of one sequence over the repository's vocabulary
        {"name": "sample_b1_top_p", "op": "sample", "rows": 1, "vocab": VOCAB, "rules": "p", "ties": False},
        # a tree's nodes, few candidates each, over an odd vocabulary
        {"name": "sample_b33_top_k", "op": "sample", "rows": 33, "vocab": 32003, "rules": "k", "ties": True},
        # a serving batch whose rows each have their own rules
        {"name": "sample_b128_mixed", "op": "sample", "rows": 128, "vocab": VOCAB, "rules": "mixed", "ties": False},
        # the bookkeeping of one sequence's tree over one layer's pages
        {"name": "step_b1_n16_bf16", "op": "step", "dtype": "bf16", "seqs": 1, "nodes": 16, "fewest": 16, "past": 300, "page": 64, "layers": 1, **beam},
        # of a serving batch with the largest trees, over a stack's six layers
        {"name": "step_b64_n64_fp8_l6", "op": "step", "dtype": "fp8", "seqs": 64, "nodes": 64, "fewest": 1, "past": 500, "page": 32, "layers": 6, **beam},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "tree", "sample", "sample", "step"])
    if op == "sample":
        rows = _log(rng, 1, 128)
        return {"op": op, "rows": rows, "vocab": _log(rng, 1, VOCAB), "rules": rng.choice(["p", "k", "min_p", "none", "greedy", "mixed", "mixed"]),
                "ties": rng.random() < 0.3}
    dtype = rng.choice(["bf16", "fp8", "nvfp4"])
    dim = rng.choice([64, 128, 128])
    n_kv = rng.choice([1, 2, 3, 4, 8, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 6, 7, 8, 12, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    if dtype == "nvfp4" and dim == 64:
        page = max(page, 32)
    c = {"op": op, "dtype": dtype, "n_q": min(n_kv * group, 48), "n_kv": n_kv, "dim": dim, "page": page}
    c["n_q"] -= c["n_q"] % n_kv
    if op == "append":
        seqs = _log(rng, 1, 64)
        tree = rng.random() < 0.4
        return {**c, "seqs": seqs, "chunk": _log(rng, 1, MOST_NODES if tree else 16000 // seqs), "past": _log(rng, 1, 2000), "tree": tree,
                "kind": rng.choice(["rope", "ssmax"]), "norm": rng.random() < 0.8, "gate": rng.random() < 0.7}
    nodes = _log(rng, 1, MOST_NODES)
    if op == "tree":
        seqs = _log(rng, 1, 64)
        ctx = _log(rng, 1, min(100000, 6000000 // (seqs * nodes), 500000 // seqs))
        return {**c, "seqs": seqs, "nodes": nodes, "fewest": rng.choice([nodes, rng.randint(0, nodes)]), "ctx": ctx, "least": _log(rng, 1, ctx),
                "window": rng.choice([0, 0, 0, 3, 100, 512, 1000]), "gate": rng.random() < 0.7}
    return {**c, "seqs": _log(rng, 1, 64), "nodes": nodes, "fewest": rng.choice([nodes, rng.randint(0, nodes)]), "past": _log(rng, 1, 500), "layers": rng.choice([1, 2, 6])}


# Sizes do not hang on the seed: sequences' lengths and trees' sizes go in even steps.

def _steps(n, most, least):
    return [most - (most - least) * i // max(1, n - 1) for i in range(n)]


def _nodes(c):
    """Each sequence's number of rows in the call."""
    if c["op"] == "append":
        return [c["chunk"]] * c["seqs"]
    sizes = _steps(c["seqs"], c["nodes"], c["fewest"])
    return [sizes[i * 5 % len(sizes)] if len(sizes) % 5 else sizes[i] for i in range(len(sizes))]


def _lengths(c):
    """Tokens that each sequence holds already."""
    if c["op"] == "tree":
        return _steps(c["seqs"], c["ctx"], c["least"])
    held = [1 + (i * 37) % c["past"] for i in range(c["seqs"])]
    if c["op"] == "append" and c["dtype"] != "bf16":   # read back into a ring of `chunk` rows: whole turns before it
        held = [x - x % c["chunk"] for x in held]
    return held


def _tree(i, n):
    """(parents, a path) of a drafted tree of n nodes: a main chain, then side branches of up to two nodes that
    leave it; parents come before their children. The path is the one that verification accepts."""
    main = (n + 1) // 2
    parent = [j - 1 for j in range(main)]
    leave = max(1, main - 2)
    for j in range(main, n):
        side, second = divmod(j - main, 2)
        parent.append(j - 1 if second else side % leave)
    if n > main and i % 3 < 2:
        side = i % ((n - main + 1) // 2)
        first = main + 2 * side
        path = list(range(side % leave + 1)) + [first]
        if first + 1 < n and len(path) < main:
            path.append(first + 1)
    else:
        path = list(range(1 + i % main)) if n else []
    return parent, path


def _row_bytes(c):
    d = c["dim"]
    return {"bf16": 2 * d, "fp8": d + 1, "nvfp4": d // 2 + d // 16 + 1}[c["dtype"]]


def work(case):
    c = case
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return {"bytes": 4 * n + 28 * c["rows"], "flops": 4 * n}
    d, n_kv, n_q, rows = c["dim"], c["n_kv"], c["n_q"], sum(_nodes(c))
    if c["op"] == "append":
        qg = n_q * (2 if c["gate"] else 1)
        back = rows * n_kv * 2 * 2 * d if c["dtype"] != "bf16" else 0   # the values that come back (the rows are on the chip)
        return {"bytes": rows * (2 * d * (2 * qg + 2 * n_kv) + 2 * n_kv * _row_bytes(c)) + back, "flops": 8 * rows * d * (n_q + n_kv)}
    if c["op"] == "step":
        moved = sum(sum(a != b for a, b in enumerate(_tree(i, n)[1])) for i, n in enumerate(_nodes(c)))
        return {"bytes": moved * 2 * n_kv * 2 * _row_bytes(c) * c["layers"] + rows * 48 + c["seqs"] * 24, "flops": rows * 16}
    keys = pairs = 0
    for i, (base, n) in enumerate(zip(_lengths(c), _nodes(c))):
        parent, depth, reach = _tree(i, n)[0], [], 0
        for j in range(n):
            depth.append(1 + (depth[parent[j]] if parent[j] >= 0 else 0))
            see = min(base + depth[j], c["window"]) if c["window"] else base + depth[j]
            pairs += see
            reach = max(reach, min(base, max(0, see - depth[j])))   # context keys that any row reads
        keys += reach + n
    io = rows * n_q * d * 2 * (3 if c["gate"] else 2)
    return {"bytes": keys * n_kv * 2 * _row_bytes(c) + io, "flops": 4 * n_q * d * pairs}


# ------------------------------------------------------------------- the pages' formats ----

def _exp2(e):
    """2^e in fp32, from its bits: pow() may be off by a step."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _row_exponent(x, most):
    """The least e >= -127 with amax <= most * 2^e, for each row of x (fp32, finite)."""
    m, e = torch.frexp(x.abs().amax(-1))
    top, te = math.frexp(most)
    return torch.where(m == 0, -127, e - te + (m > top).to(e.dtype)).clamp_min(-127)


def _scaled(x, e):
    """x * 2^-e, exact: in two steps, since 2^-e alone may leave the range of fp32."""
    h = torch.div(-e, 2, rounding_mode="floor")
    return x * _exp2(h)[..., None] * _exp2(-e - h)[..., None]


def _quantise(x, dtype):
    """x [..., D] bf16 -> (codes, row bytes, block scales) of the cache's formats."""
    x = x.float()
    e = _row_exponent(x, ROW_MAX[dtype])
    y = _scaled(x, e)
    row = (e + 127).to(torch.uint8)
    if dtype == "fp8":
        return y.to(torch.float8_e4m3fn).view(torch.uint8), row, None
    y = y.unflatten(-1, (-1, 16))
    # a tensor as the divisor: by a plain number torch multiplies with its reciprocal, which misses ties
    s = (y.abs().amax(-1) / torch.full((1,), 6.0, device=y.device)).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    a = y.abs()
    # number of midpoints below (a tie goes to the even code): products of few bits, exact in fp32
    code = (a > MID[0] * sf).to(torch.uint8) + (a >= MID[1] * sf) + (a > MID[2] * sf) + (a >= MID[3] * sf)
    code = code + (a > MID[4] * sf) + (a >= MID[5] * sf) + (a > MID[6] * sf)
    code = torch.where(sf > 0, code, torch.zeros_like(code)) + 8 * (y < 0).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), row, s.view(torch.uint8)


def _values(codes, row, block, dtype):
    """fp32 values that the cache's codes stand for."""
    if dtype == "bf16":
        return codes.float()
    scale = _exp2(row.to(torch.int32) - 127)[..., None]
    if dtype == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * scale
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * block.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2) * scale


def _places(s, seq, slot):
    """(page, offset) of slots (1-based) of sequences seq."""
    page = s["case"]["page"]
    at = (slot - 1).long()
    return s["table"][seq.long(), torch.div(at, page, rounding_mode="floor")].long(), at % page


def _fetch(s, seq, slot):
    """K and V [..., n_kv, D] in fp32 at slots of sequences seq."""
    p, o = _places(s, seq, slot)
    out = []
    for i, name in enumerate(("k", "v")):
        row = s["row"][p, :, i, o] if s["row"] is not None else None
        block = s["block"][p, :, i, o] if s["block"] is not None else None
        out.append(_values(s[name][p, :, o], row, block, s["case"]["dtype"]))
    return out


# ---------------------------------------------------------------------- plain forms ----

def _plain_append(s):
    """q' and k' = norm (per head), then rotation by the position (or, on a layer without it, the query scale);
    both rounded to bf16, which is what the pages quantise."""
    c = s["case"]
    d, n_q, n_kv, dtype = c["dim"], c["n_q"], c["n_kv"], c["dtype"]
    z = s["qkv"].view(s["qkv"].shape[0], -1, d)
    q, k, v = z[:, :n_q].float(), z[:, n_q:n_q + n_kv].float(), z[:, n_q + n_kv:n_q + 2 * n_kv]
    if c["norm"]:
        q = q / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS) * s["qn"].float()
        k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + EPS) * s["kn"].float()
    if c["kind"] == "rope":
        half = d // 2
        inv = torch.tensor([THETA ** (-2.0 * i / d) for i in range(half)], dtype=torch.float64, device=z.device)
        angle = (s["pos"].double() - 1)[:, None] * inv
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        q, k = (torch.cat((x[..., :half] * cos - x[..., half:] * sin, x[..., half:] * cos + x[..., :half] * sin), -1) for x in (q, k))
    else:
        q = q * torch.exp(SSMAX_EXP * torch.log(1 + s["pos"].double() / SSMAX_BASE)).float()[:, None, None]
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    p, o = _places(s, s["seq"], s["slot"])
    for i, (name, x) in enumerate((("k", k), ("v", v))):
        if dtype == "bf16":
            s[name][p, :, o] = x
            continue
        codes, row, block = _quantise(x, dtype)
        s[name][p, :, o] = codes
        s["row"][p, :, i, o] = row
        if block is not None:
            s["block"][p, :, i, o] = block
    out = {"q": q}
    if c["gate"]:
        out["g"] = z[:, n_q + 2 * n_kv:].reshape(z.shape[0], n_q * d)
    if dtype == "bf16":
        return {**out, "k": s["k"], "v": s["v"]}
    n = c["chunk"]
    for name, x in zip(("k", "v"), _fetch(s, s["seq"], s["slot"])):
        s["to_" + name].copy_(x.view(c["seqs"], n, n_kv, d).transpose(1, 2).to(torch.bfloat16))
    return {**out, "k": s["to_k"], "v": s["to_v"]}


def _plain_tree(s):
    """Row j of sequence b sees the context 1..base (with a window: positions above p - window, p = base + the bits of
    its mask) and the nodes of its mask (with a window: its nearest ancestors only)."""
    c = s["case"]
    d, n_kv, group = c["dim"], c["n_kv"], c["n_q"] // c["n_kv"]
    b, most, dev = c["seqs"], c["nodes"], s["q"].device
    bit = torch.arange(most, device=dev)
    n = (s["start"][1:] - s["start"][:-1]).long()
    row = (s["start"][:-1].long()[:, None] + bit).clamp_max(s["q"].shape[0] - 1)
    real = bit < n[:, None]                                                  # [b, most]
    mask = torch.where(real, s["mask"][row], 0)
    see = (mask[..., None] >> bit) & 1                                       # [b, row, node]
    rank = see.cumsum(-1)
    depth = rank[..., -1:]
    base = s["base"].long()[:, None, None]
    w = c["window"] if c["window"] else 1 << 40
    see = (see > 0) & (base + rank > base + depth - w)
    longest = min(c["ctx"], c["window"]) if c["window"] else c["ctx"]
    at = s["base"].long()[:, None] - longest + 1 + torch.arange(longest, device=dev)   # context positions
    ctx = (at[:, None] >= 1) & (at[:, None] > base + depth - w) & (mask != 0)[..., None]
    slots = torch.cat((at.clamp_min(1), torch.where(real, s["base"].long()[:, None] + 1 + bit, 1)), 1)
    k, v = _fetch(s, s["ids"].long()[:, None].expand_as(slots), slots)       # [b, keys, n_kv, d]
    q = s["q"].float()[row].view(b, most, n_kv, group, d).permute(0, 2, 1, 3, 4).reshape(b, n_kv, most * group, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(d)
    here = torch.cat((ctx, see), -1)[:, None, :, None]
    x = x.view(b, n_kv, most, group, -1).masked_fill_(~here, -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, n_kv, most * group, -1), v.transpose(1, 2)).view(b, n_kv, most, group, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 2, 1, 3, 4).reshape(b, most, c["n_q"], d)[real]
    if c["gate"]:
        o = o / (1 + torch.exp(-(s["g"].float().view(o.shape) + s["bias"].float()[None, :, None])))
    return o.to(torch.bfloat16).view(-1, c["n_q"] * d)


def _plain_sample(s):
    """Tokens in order of their logits (equal ones by index): the first top_k; of these the fewest that hold top_p of
    their weight; of these the ones of at least min_p of the largest weight. Then the first token, by index, at which the
    kept weights' running sum passes u times their sum. Sums in 64 bits: a border is met by one token or another."""
    z = s["logits"].double()
    n = z.shape[1]
    t = s["temperature"].double()[:, None]
    value, index = torch.sort(z, dim=-1, descending=True, stable=True)
    top = value[:, :1]
    w = torch.exp((value - top) / torch.where(t > 0, t, torch.ones_like(t)))
    place = torch.arange(n, device=z.device)
    keep = (place < torch.where(s["top_k"] > 0, s["top_k"], n)[:, None])
    w = w * keep
    before = w.cumsum(-1) - w
    p = s["top_p"].double()[:, None]
    keep &= (before < p * w.sum(-1, keepdim=True)) | (p >= 1) | (place == 0)
    keep &= (value >= top + t * torch.log(s["min_p"].double()[:, None])) | (s["min_p"] <= 0)[:, None]
    keep &= (t > 0) | (place == 0)
    w = torch.zeros_like(w).scatter_(-1, index, w * keep)
    run = w.cumsum(-1)
    total = run[:, -1:]
    token = (run > s["u"].double()[:, None] * total).to(torch.int32).argmax(-1, keepdim=True)
    prob = w.gather(-1, token) / total
    return {"token": token.view(-1).to(torch.int32), "logprob": torch.log(prob).view(-1).float()}


def _plain_step(s):
    c = s["case"]
    b, most, dev = c["seqs"], c["nodes"], s["start"].device
    at = torch.arange(most, device=dev)
    n = (s["start"][1:] - s["start"][:-1]).long()
    row = (s["start"][:-1].long()[:, None] + at).clamp_max(s["parent"].shape[0] - 1)
    real = at < n[:, None]
    parent, token, sampled = (torch.where(real, s[x][row], -2).long() for x in ("parent", "token", "sampled"))
    # masks: a node's parent's and its own bit
    mask = torch.zeros((b, most), dtype=torch.int64, device=dev)
    for j in range(most):
        up = mask.gather(1, parent[:, j:j + 1].clamp_min(0))[:, 0]
        mask[:, j] = torch.where(parent[:, j] >= 0, up, 0) | (1 << j if j < 63 else -(1 << 63))
    depth = ((mask[..., None] >> at) & 1).sum(-1)
    base = s["base"].long()[:, None]
    plan = {"mask": mask[real], "pos": (base + depth)[real].to(torch.int32), "slot": (base + 1 + at).expand(b, -1)[real].to(torch.int32),
            "seq": s["ids"][:, None].expand(b, most)[real]}
    # the walk from the root along the sampled tokens
    path = torch.full((b, most), -1, dtype=torch.int64, device=dev)
    cur, live = torch.zeros(b, dtype=torch.int64, device=dev), n > 0
    for d in range(most):
        path[:, d] = torch.where(live, cur, -1)
        want = sampled.gather(1, cur[:, None])
        child = (parent == cur[:, None]) & (token == want) & real & (at > cur[:, None])
        live = live & child.any(-1)
        cur = torch.where(live, child.to(torch.int32).argmax(-1), cur)
    count = (path >= 0).sum(-1)
    follow = torch.where(n > 0, sampled.gather(1, cur[:, None])[:, 0], -1)
    # the accepted rows move to the front
    move = path >= 0
    seq = s["ids"].long()[:, None].expand(b, most)[move]
    src, dst = (base + 1 + path)[move], (base + 1 + at).expand(b, -1)[move]
    ps, os_ = _places(s, seq, src)
    pd, od = _places(s, seq, dst)
    for layer in s["layers"]:
        for i, name in enumerate(("k", "v")):
            layer[name][pd, :, od] = layer[name][ps, :, os_]
            if layer["row"] is not None:
                layer["row"][pd, :, i, od] = layer["row"][ps, :, i, os_]
            if layer["block"] is not None:
                layer["block"][pd, :, i, od] = layer["block"][ps, :, i, os_]
    return {**plan, "count": count.to(torch.int32), "path": path.to(torch.int32), "next": follow.to(torch.int32), "pages": _pages(s)}


def _pages(s):
    """What the layers' pages hold: codes as the values they stand for, before the row's power of two."""
    out = []
    for layer in s["layers"]:
        if s["case"]["dtype"] == "bf16":
            out.append({"k": layer["k"], "v": layer["v"]})
            continue
        e4m3 = torch.float8_e4m3fn
        kind = e4m3 if s["case"]["dtype"] == "fp8" else torch.uint8
        out.append({"k": layer["k"].view(kind), "v": layer["v"].view(kind), "row": layer["row"].view(torch.float8_e8m0fnu)})
        if layer["block"] is not None:
            out[-1]["block"] = layer["block"].view(e4m3)
    return out


# ----------------------------------------------------------------------- framework ----

def _handle(s):
    """The cache handles and the layer configuration that a user's program keeps."""
    if "handle" not in s:
        from hybrid_attention_moe_gb300 import beam as B
        c = s["case"]
        caches = [B.PagedKVCache(x["k"], x["v"], s["table"], x["row"], x["block"], window=c.get("window", 0)) for x in s.get("layers", [s])]
        kind = B.BEAM_ATTN_SWA_ROPE if c.get("kind") == "rope" else B.BEAM_ATTN_NOPE_SSMAX
        cfg = B.LayerCfg(hidden=c["n_q"] * c["dim"], n_q=c["n_q"], n_kv=c["n_kv"], head_dim=c["dim"], kind=kind, n_experts=8, n_groups=1,
                         topk_groups=1, topk=1, d_ff_expert=128, d_ff_dense=128, rope_theta=THETA, ssmax_base=SSMAX_BASE, ssmax_exp=SSMAX_EXP, eps=EPS)
        to = B.KVCache(s["to_k"], s["to_v"]) if "to_k" in s else None
        s["handle"] = (B, caches, cfg, to)
    return s["handle"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"append": _plain_append, "tree": _plain_tree, "sample": _plain_sample, "step": _plain_step}[c["op"]](s)
    if c["op"] == "sample":
        from hybrid_attention_moe_gb300 import beam as B
        B.beam_sample(s["logits"], s["u"], s["token"], s["logprob"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
        return {"token": s["token"], "logprob": s["logprob"]}
    B, caches, cfg, to = _handle(s)
    if c["op"] == "append":
        B.beam_paged_append(cfg, s["qkv"], s["qn"], s["kn"], s["seq"], s["pos"], s["slot"], s["q_out"], s["g_out"], caches[0])
        out = {"q": s["q_out"], "g": s["g_out"]} if c["gate"] else {"q": s["q_out"]}
        if c["dtype"] == "bf16":
            return {**out, "k": s["k"], "v": s["v"]}
        B.beam_paged_kv_read(caches[0], s["ids"], s["first"], s["last"], c["chunk"], to)
        return {**out, "k": s["to_k"], "v": s["to_v"]}
    if c["op"] == "tree":
        B.beam_paged_tree_attn(cfg, s["q"], s["g"], s["bias"], caches[0], s["ids"], s["start"], s["base"], s["mask"], s["reach"], None, s["out"], s["scratch"])
        return s["out"]
    B.beam_tree_plan(s["parent"], s["start"], s["ids"], s["base"], s["mask"], s["pos"], s["slot"], s["seq"])
    B.beam_tree_accept(s["parent"], s["token"], s["sampled"], s["start"], s["count"], s["path"], s["next"])
    for cache in caches:
        B.beam_paged_kv_keep(cache, s["ids"], s["base"], s["count"], s["path"])
    return {**{x: s[x] for x in ("mask", "pos", "slot", "seq", "count", "path", "next")}, "pages": _pages(s)}


def _prepare_sample(c, s, gen, dev):
    """Logits as an LM head with a softcap of 30 gives them: a wide body and a few dozen likely tokens."""
    rows, n = c["rows"], c["vocab"]

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(rows, generator=gen, device=dev)

    z = 2.2 * torch.randn((rows, n), generator=gen, device=dev)
    likely = torch.randint(0, n, (rows, 40), generator=gen, device=dev)
    z.scatter_add_(1, likely, 14 * torch.rand((rows, 40), generator=gen, device=dev))
    z = 30 * torch.tanh(z / 30)
    s["logits"] = z.to(torch.bfloat16).float() if c["ties"] else z
    rule = torch.arange(rows, device=dev) % 5 if c["rules"] == "mixed" else torch.full((rows,), {"p": 0, "k": 1, "min_p": 2, "none": 3, "greedy": 4}[c["rules"]], device=dev)
    both = torch.rand(rows, generator=gen, device=dev) < 0.3   # some rows with top-k and top-p together
    s["temperature"] = torch.where(rule == 4, torch.zeros(rows, device=dev), uniform(0.6, 1.3))
    s["top_p"] = torch.where((rule == 0) | ((rule == 1) & both), uniform(0.7, 0.99), torch.ones(rows, device=dev))
    most = torch.randint(1, 101, (rows,), generator=gen, device=dev)
    s["top_k"] = torch.where(rule == 1, most, 0).to(torch.int32)
    s["min_p"] = torch.where(rule == 2, uniform(0.01, 0.2), torch.zeros(rows, device=dev))
    s["u"] = torch.rand(rows, generator=gen, device=dev)
    s["token"] = torch.empty(rows, dtype=torch.int32, device=dev)
    s["logprob"] = torch.empty(rows, dtype=torch.float32, device=dev)
    return s


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "sample":
        return _prepare_sample(c, s, gen, dev)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev).to(dtype)

    sizes, held = _nodes(c), _lengths(c)
    b, d, page, n_kv, n_q = c["seqs"], c["dim"], c["page"], c["n_kv"], c["n_q"]
    T = sum(sizes)
    # the calls' sequences are in an order of their own in the page table
    ids = torch.randperm(b, generator=gen, device=dev)
    s["ids"] = ids.to(torch.int32)
    s["base"] = torch.tensor(held, dtype=torch.int32, device=dev)
    s["start"] = torch.tensor([sum(sizes[:i]) for i in range(b + 1)], dtype=torch.int32, device=dev)
    grown = torch.zeros(b, dtype=torch.int64, device=dev)
    grown[ids] = torch.tensor([x + y for x, y in zip(held, sizes)], device=dev)
    per = -(-max(x + y for x, y in zip(held, sizes)) // page)     # page table entries of a sequence
    need = torch.div(grown + page - 1, page, rounding_mode="floor")
    pool = sum(-(-(x + y) // page) for x, y in zip(held, sizes)) + 3   # a few pages belong to nobody
    # the sequences' pages lie anywhere in the pool; entries past a sequence's end name no page
    order = torch.randperm(pool, generator=gen, device=dev)
    begin = torch.cumsum(need, 0) - need
    idx = torch.arange(per, device=dev)[None]
    s["table"] = torch.where(idx < need[:, None], order[(begin[:, None] + idx).clamp_max(pool - 1)], -1).to(torch.int32).contiguous()
    width = {"bf16": d, "fp8": d, "nvfp4": d // 2}[c["dtype"]]
    kind = torch.bfloat16 if c["dtype"] == "bf16" else torch.uint8

    def pages(full):
        x = {"row": None, "block": None}
        for name in ("k", "v"):
            x[name] = torch.zeros((pool, n_kv, page, width), dtype=kind, device=dev)
        if c["dtype"] != "bf16":
            x["row"] = torch.zeros((pool, n_kv, 2, page), dtype=torch.uint8, device=dev)
        if c["dtype"] == "nvfp4":
            x["block"] = torch.zeros((pool, n_kv, 2, page, d // 16), dtype=torch.uint8, device=dev)
        # what the sequences hold: normed keys (unit variance), values whose size varies by token
        step = max(1, (64 << 20) // (n_kv * page * d))
        for a in range(0, pool if full else 0, step):
            m = min(step, pool - a)
            for i, name in enumerate(("k", "v")):
                y = torch.randn((m, n_kv, page, d), generator=gen, device=dev)
                if name == "v":
                    y = y * torch.exp(0.7 * torch.randn((m, n_kv, page, 1), generator=gen, device=dev))
                y = y.to(torch.bfloat16)
                if c["dtype"] == "bf16":
                    x[name][a:a + m] = y
                    continue
                codes, row, block = _quantise(y, c["dtype"])
                x[name][a:a + m] = codes
                x["row"][a:a + m, :, i] = row
                if block is not None:
                    x["block"][a:a + m, :, i] = block
        return x

    tree = c["op"] != "append" or c["tree"]
    trees = [_tree(i, n) if tree else ([], []) for i, n in enumerate(sizes)]
    masks, depths = [], []
    for parent, _ in trees:
        m = []
        for j, up in enumerate(parent):
            m.append((m[up] if up >= 0 else 0) | 1 << j)
        masks += [x - (1 << 64) if x >> 63 else x for x in m]
        depths += [bin(x).count("1") for x in m]
    s["mask"] = torch.tensor(masks, dtype=torch.int64, device=dev)
    if c["op"] == "append":
        s.update(pages(False))
        node = torch.arange(c["chunk"], device=dev)
        depth = torch.tensor(depths, device=dev).view(b, -1) if c["tree"] else node + 1
        s["seq"] = s["ids"].repeat_interleave(c["chunk"])
        s["pos"] = (s["base"][:, None] + depth).expand(b, -1).flatten().to(torch.int32)
        s["slot"] = (s["base"][:, None] + 1 + node).flatten().to(torch.int32)
        x = normal(T, n_q * (2 if c["gate"] else 1) + 2 * n_kv, d, dtype=torch.float32)
        x[:, n_q + n_kv:n_q + 2 * n_kv] *= torch.exp(0.7 * normal(T, n_kv, 1, dtype=torch.float32))
        s["qkv"] = x.to(torch.bfloat16).view(T, -1)
        s["qn"], s["kn"] = ((1 + 0.1 * normal(d, dtype=torch.float32)).to(torch.bfloat16) if c["norm"] else None for _ in "qk")
        s["q_out"] = torch.empty((T, n_q, d), dtype=torch.bfloat16, device=dev)
        s["g_out"] = torch.empty((T, n_q * d), dtype=torch.bfloat16, device=dev) if c["gate"] else None
        if c["dtype"] != "bf16":
            s["first"], s["last"] = s["base"] + 1, s["base"] + c["chunk"]
            s["to_k"] = torch.zeros((b, n_kv, c["chunk"], d), dtype=torch.bfloat16, device=dev)
            s["to_v"] = torch.zeros_like(s["to_k"])
        return s
    if c["op"] == "tree":
        s.update(pages(True))
        s["reach"] = max(x + y for x, y in zip(held, sizes))
        s["q"] = normal(T, n_q, d)
        s["g"] = normal(T, n_q * d) if c["gate"] else None
        s["bias"] = normal(n_q) if c["gate"] else None
        s["out"] = torch.empty((T, n_q * d), dtype=torch.bfloat16, device=dev)
        s["scratch"] = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
        return s
    s["layers"] = [pages(True) for _ in range(c["layers"])]
    s["parent"] = torch.tensor(sum((t[0] for t in trees), []), dtype=torch.int32, device=dev)
    # siblings' tokens differ; the sampled ones lead along the path and then to a token that nobody drafted
    node = torch.cat([torch.arange(n, device=dev) for n in sizes]) if T else torch.zeros(0, dtype=torch.int64, device=dev)
    s["token"] = (torch.randint(0, VOCAB // 64, (T,), generator=gen, device=dev) * 64 + node).to(torch.int32)
    s["sampled"] = torch.randint(0, VOCAB // 64, (T,), generator=gen, device=dev).mul_(64).to(torch.int32)
    at, lead = [], []
    end = []
    for i, (_, path) in enumerate(trees):
        first = sum(sizes[:i])
        at += [first + x for x in path[:-1]]
        lead += [first + x for x in path[1:]]
        end += [first + x for x in path[-1:]]
    s["sampled"][torch.tensor(at, dtype=torch.long, device=dev)] = s["token"][torch.tensor(lead, dtype=torch.long, device=dev)]
    s["sampled"][torch.tensor(end, dtype=torch.long, device=dev)] = VOCAB - 1
    for name, kind in (("pos", torch.int32), ("slot", torch.int32), ("seq", torch.int32)):
        s[name] = torch.empty(T, dtype=kind, device=dev)
    s["count"], s["next"] = (torch.empty(b, dtype=torch.int32, device=dev) for _ in "cn")
    s["path"] = torch.empty((b, c["nodes"]), dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------------ in 64 bits ----

def _e4m3_table(dev):
    """The value of each of the 256 e4m3 codes, from the format's definition."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(math.nan if b & 127 == 127 else -x if b & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _two_to(e):
    """2^e in float64 for whole e in -160..140."""
    table = torch.tensor([math.ldexp(1.0, i - 160) for i in range(301)], dtype=torch.float64, device=e.device)
    return table[e.long() + 160]


def _nearest(y, grid):
    """Index of the grid value nearest to y >= 0 (float64); a tie goes to the even index."""
    mid = (grid[:-1] + grid[1:]) / 2
    low, high = torch.bucketize(y, mid), torch.bucketize(y, mid, right=True)   # differ where y is a midpoint
    return torch.where(low % 2 == 0, low, high)


def _exact_rows(codes, row, block, dtype):
    if dtype == "bf16":
        return codes.double()
    scale = _two_to(row.long() - 127)[..., None]
    table = _e4m3_table(codes.device)
    if dtype == "fp8":
        return table[codes.long()] * scale
    d = codes.shape[-1] * 2
    v = torch.empty(codes.shape[:-1] + (d,), dtype=torch.float64, device=codes.device)
    mag = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        nib = ((codes.long() >> (4 * half)) & 15)
        v[..., half::2] = torch.where(nib >= 8, -mag[nib & 7], mag[nib & 7])
    return v * table[block.long()].repeat_interleave(16, -1) * scale


def _exact_sequence(s, b, slots):
    """K and V [n][n_kv][D] in float64 of the page table's sequence b."""
    page, out = s["case"]["page"], []
    pg = s["table"][b].long()[(slots - 1) // page]
    off = (slots - 1) % page
    for i, name in enumerate(("k", "v")):
        out.append(_exact_rows(s[name][pg, :, off], None if s["row"] is None else s["row"][pg, :, i, off],
                               None if s["block"] is None else s["block"][pg, :, i, off], s["case"]["dtype"]))
    return out


def _exact_quantise(x, dtype):
    """The values that rows are stored as, in float64."""
    x = x.double()
    most = x.abs().amax(-1)
    e = torch.ceil(torch.log2(most / ROW_MAX[dtype])).clamp(-140, 130)
    e = torch.where(_two_to(e - 1) * ROW_MAX[dtype] >= most, e - 1, e)   # the logarithm may be a hair off
    e = torch.where(_two_to(e) * ROW_MAX[dtype] < most, e + 1, e).clamp_min(-127)
    two = _two_to(e)[..., None]
    grid = _e4m3_table(x.device)[:127]
    if dtype == "fp8":
        return torch.copysign(grid[_nearest(x.abs() / two, grid)], x) * two
    a = (x.abs() / two).unflatten(-1, (-1, 16))
    sc = grid[_nearest(a.amax(-1), 6 * grid)][..., None]
    mag = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    y = torch.where(sc > 0, mag[_nearest(a / sc.clamp_min(1e-9), mag)], torch.zeros_like(a)) * sc
    return torch.copysign(y.flatten(-2), x) * two


def _exact_append(s):
    c = s["case"]
    d, n_q, n_kv, T = c["dim"], c["n_q"], c["n_kv"], s["qkv"].shape[0]
    z = s["qkv"].double().view(T, -1, d)
    both = z[:, :n_q + n_kv].clone()
    if c["norm"]:
        gain = torch.cat((s["qn"].double().expand(n_q, d), s["kn"].double().expand(n_kv, d)))
        both = both * (both.square().mean(-1, keepdim=True) + EPS).rsqrt() * gain
    if c["kind"] == "rope":
        i = torch.arange(d // 2, dtype=torch.float64, device=z.device)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=z.device), (s["pos"].double() - 1)[:, None] * torch.pow(THETA, -2 * i / d))
        pair = torch.complex(both[..., :d // 2], both[..., d // 2:]) * turn[:, None]
        both = torch.cat((pair.real, pair.imag), -1)
    else:
        both[:, :n_q] *= torch.pow(1 + s["pos"].double() / SSMAX_BASE, SSMAX_EXP)[:, None, None]
    out = {"q": both[:, :n_q]}
    if c["gate"]:
        out["g"] = z[:, n_q + 2 * n_kv:].reshape(T, -1)
    k, v = both[:, n_q:], z[:, n_q + n_kv:n_q + 2 * n_kv]
    if c["dtype"] == "bf16":
        pg = s["table"][s["seq"].long(), (s["slot"].long() - 1) // c["page"]].long()
        off = (s["slot"].long() - 1) % c["page"]
        for name, x in (("k", k), ("v", v)):
            out[name] = s[name].double()
            out[name][pg, :, off] = x
        return out
    for name, x in (("k", k.to(torch.bfloat16)), ("v", v)):   # the pages quantise rows of bf16
        out[name] = _exact_quantise(x, c["dtype"]).view(c["seqs"], -1, n_kv, d).transpose(1, 2)
    return out


def _exact_tree(s):
    c = s["case"]
    d, n_kv, group = c["dim"], c["n_kv"], c["n_q"] // c["n_kv"]
    o = torch.zeros((s["q"].shape[0], c["n_q"], d), dtype=torch.float64, device="cuda")
    start, base, masks = s["start"].tolist(), s["base"].tolist(), s["mask"].tolist()
    for b in range(c["seqs"]):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        seen = torch.zeros((n, base[b] + n), dtype=torch.bool)
        for j in range(n):
            nodes = [a for a in range(n) if masks[start[b] + j] >> a & 1]
            if c["window"]:
                nodes, left = nodes[-c["window"]:], max(0, c["window"] - len(nodes))
            else:
                left = base[b]
            seen[j, max(0, base[b] - left):base[b]] = left > 0
            seen[j, [base[b] + a for a in nodes]] = True
        k, v = _exact_sequence(s, int(s["ids"][b]), torch.arange(1, base[b] + n + 1, device="cuda"))
        q = s["q"][start[b]:start[b + 1]].double().view(n, n_kv, group, d)
        for h in range(n_kv):
            x = torch.matmul(q[:, h], k[:, h].T) * d ** -0.5
            x = x.masked_fill(~seen.cuda()[:, None], -math.inf)
            o[start[b]:start[b + 1], h * group:(h + 1) * group] = torch.matmul(torch.softmax(x, -1), v[:, h])
    if c["gate"]:
        o = o * torch.sigmoid(s["g"].double().view(o.shape) + s["bias"].double()[None, :, None])
    return o.view(-1, c["n_q"] * d)


def _exact_sample(s):
    token, logprob = [], []
    for r in range(s["logits"].shape[0]):
        z = s["logits"][r].double()
        t, k, p, m, u = (s[x][r].item() for x in ("temperature", "top_k", "top_p", "min_p", "u"))
        order = torch.argsort(-z, stable=True)
        if t <= 0:
            token.append(int(order[0]))
            logprob.append(0.0)
            continue
        if k > 0:
            order = order[:k]
        weight = torch.exp((z[order] - z[order[0]]) / t)
        if p < 1:
            reached = torch.nonzero(torch.cumsum(weight, 0) >= p * weight.sum())
            order = order[:max(1, int(reached[0]) + 1 if len(reached) else len(order))]
        if m > 0:
            order = order[z[order] >= z[order[0]] + t * math.log(m)]
        order = torch.sort(order).values
        weight = torch.exp((z[order] - z[order].max()) / t)
        run = torch.cumsum(weight, 0)
        at = int(torch.nonzero(run > u * run[-1])[0])
        token.append(int(order[at]))
        logprob.append(math.log(float(weight[at] / run[-1])))
    return {"token": torch.tensor(token, dtype=torch.int32, device="cuda"), "logprob": torch.tensor(logprob, dtype=torch.float64, device="cuda")}


def _exact_step(s):
    c = s["case"]
    start, base, parent = s["start"].tolist(), s["base"].tolist(), s["parent"].tolist()
    token, sampled, ids, table = s["token"].tolist(), s["sampled"].tolist(), s["ids"].tolist(), s["table"].tolist()
    out = {x: [] for x in ("mask", "pos", "slot", "seq", "count", "path", "next")}
    src, dst = [], []
    for b in range(c["seqs"]):
        first, n = start[b], start[b + 1] - start[b]
        for j in range(n):
            chain = [j]
            while parent[first + chain[-1]] >= 0:
                chain.append(parent[first + chain[-1]])
            mask = sum(1 << x for x in chain)
            out["mask"].append(mask - (1 << 64) if mask >> 63 else mask)
            out["pos"].append(base[b] + len(chain))
            out["slot"].append(base[b] + 1 + j)
            out["seq"].append(ids[b])
        path = [0] if n else []
        while path:
            step = [j for j in range(path[-1] + 1, n) if parent[first + j] == path[-1] and token[first + j] == sampled[first + path[-1]]]
            if not step:
                break
            path.append(step[0])
        out["count"].append(len(path))
        out["path"].append(path + [-1] * (c["nodes"] - len(path)))
        out["next"].append(sampled[first + path[-1]] if path else -1)
        for a, x in enumerate(path):
            for to, at in ((src, base[b] + x), (dst, base[b] + a)):
                to.append((table[ids[b]][at // c["page"]], at % c["page"]))
    sp, so = torch.tensor(src, dtype=torch.long, device="cuda").view(-1, 2).T
    dp, do = torch.tensor(dst, dtype=torch.long, device="cuda").view(-1, 2).T
    e4m3, pages = _e4m3_table("cuda"), []
    for layer in s["layers"]:
        x = {}
        for i, name in enumerate(("k", "v")):
            y = layer[name].clone()
            y[dp, :, do] = layer[name][sp, :, so]
            x[name] = y.double() if c["dtype"] == "bf16" else e4m3[y.long()] if c["dtype"] == "fp8" else y
        for name in ("row", "block"):
            if layer[name] is not None:
                y = layer[name].clone()
                y[dp, :, :, do] = layer[name][sp, :, :, so]
                x[name] = _two_to(y.long() - 127) if name == "row" else e4m3[y.long()]
        pages.append(x)
    kind = {x: torch.int64 if x == "mask" else torch.int32 for x in out}
    return {**{x: torch.tensor(v, dtype=kind[x], device="cuda") for x, v in out.items()}, "pages": pages}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_tree, "sample": _exact_sample, "step": _exact_step}[case["op"]](s)
