"""The 8-bit operators of a decode step, as cases that can be timed and compared.

Operators (the framework's names): ``rms_norm`` (residual addition, RMS norm,
8-bit rows with scales), ``quantize_rows``, ``dualpath_linear_int8`` (the
dual-pathway linear on 8-bit integers), ``kv_append`` (rows into a paged 8-bit
cache) and ``block_attention`` (a drafted block or tree over that cache).

With ``own`` false ``run`` computes them from elementary torch operations in
float32; with ``own`` true it makes the calls a user of the framework makes.
``exact`` states each operator again in float64.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one token of one sequence: the norm before a layer's q/k/v projections
        {"name": "norm_1x4096", "op": "norm", "M": 1, "d": 4096, "dtype": "bf16", "residual": True},
        # 64 sequences x 17 rows (16 drafts and the bonus row) of a hidden size of 4096
        {"name": "norm_1088x4096", "op": "norm", "M": 1088, "d": 4096, "dtype": "bf16",
         "residual": True},
        # the attention output of a few sequences on its way into the o projection, odd width
        {"name": "quantize_85x4088", "op": "quantize", "M": 85, "d": 4088, "dtype": "f32"},
        # the MLP's activations of a prompt on their way into the down projection
        {"name": "quantize_8192x12288", "op": "quantize", "M": 8192, "d": 12288, "dtype": "bf16"},
        # k projection of a single token, AR weights only, float32 output
        {"name": "linear_1x4096x1024", "op": "linear", "M": 1, "d_in": 4096, "d_out": 1024,
         "r": 0, "out": "f32"},
        # LM head of one drafted block (16 drafts and the bonus row)
        {"name": "linear_17x4096x151936", "op": "linear", "M": 17, "d_in": 4096,
         "d_out": 151936, "r": 128, "out": "bf16"},
        # gate or up projection of the batched decode step, both paths
        {"name": "linear_1088x4096x12288", "op": "linear", "M": 1088, "d_in": 4096,
         "d_out": 12288, "r": 128, "out": "bf16"},
        # the accepted rows of 64 blocks of 17, part-filled pages
        {"name": "append_64x17", "op": "append", "B": 64, "T": 17, "Hkv": 8, "D": 128,
         "page": 64, "len": 1024, "counts": True},
        # a prompt of 4000 tokens for each of 4 sequences
        {"name": "append_4x4000", "op": "append", "B": 4, "T": 4000, "Hkv": 8, "D": 128,
         "page": 64, "len": 0, "counts": False},
        # single-token decode of a ragged batch
        {"name": "attend_32x1_ragged", "op": "attend", "B": 32, "T": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "lo": 1, "hi": 8191, "tree": False},
        # verification of 64 drafted blocks of 16 drafts and the bonus row
        {"name": "attend_64x17", "op": "attend", "B": 64, "T": 17, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "lo": 2040, "hi": 4100, "tree": False},
        # verification of one tree of the tree sampler (15 positions, 16 kept sequences)
        {"name": "attend_1x241_tree", "op": "attend", "B": 1, "T": 241, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "lo": 5001, "hi": 5001, "tree": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "append", "attend", "attend"])
    if op in ("norm", "quantize"):
        M, d = _log(rng, 1, 8192), _log(rng, 33, 12288)
        c = {"op": op, "M": M, "d": d, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "norm":
            c["residual"] = rng.random() < 0.7
        return c
    if op == "linear":
        M, d_in = _log(rng, 1, 1088), 16 * _log(rng, 4, 768)
        d_out = _log(rng, 17, 12288)
        r = rng.choice([0, 16, 40, 128, 256])
        return {"op": op, "M": M, "d_in": d_in, "d_out": d_out, "r": r,
                "out": "bf16" if r else rng.choice(["bf16", "f32"])}
    Hkv, D, page = rng.choice([1, 2, 3, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        B, T = _log(rng, 1, 64), _log(rng, 1, 300)
        return {"op": op, "B": B, "T": T, "Hkv": Hkv, "D": D, "page": page,
                "len": _log(rng, 1, 1500), "counts": rng.random() < 0.5}
    tree = rng.random() < 0.3
    hi = _log(rng, 1, 8000)
    T = rng.choice([17, 65, 241]) if tree else rng.choice([1, 1, 2, 5, 9, 17, 33])
    B = _log(rng, 1, max(1, min(48, 400000 // (T * hi + T))))
    return {"op": op, "B": B, "T": T, "Hq": Hkv * rng.choice([1, 2, 4, 5, 8]), "Hkv": Hkv, "D": D,
            "page": page, "lo": rng.choice([1, max(1, hi // 2), hi]), "hi": hi, "tree": tree}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _int8_rows(w):
    s = (w.abs().amax(1) / 127.0).contiguous()
    return torch.round(w / s[:, None]).clamp_(-127, 127).to(torch.int8), s


def _pow2_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s; 0 for amax = 0."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _codes(pages, Hkv, page, D, g):
    """Random pages [pages, Hkv, page, D] of codes and their scales; the spread of
    the values differs from page to page."""
    x = torch.randn(pages, Hkv, page, D, generator=g, device=DEV)
    x *= torch.rand(pages, Hkv, 1, 1, generator=g, device=DEV) + 0.5
    s = _pow2_scale(x.abs().amax((2, 3)))
    return (x / s[:, :, None, None]).to(FP8), s


def _cache(case, tokens, g):
    """A cache whose sequences hold up to `tokens` tokens each, pages in random order,
    a few pages of the pool unused. Slots behind a sequence's length hold old codes."""
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    width = -(-tokens // page)
    pool = B * width + 3
    k, ks = _codes(pool, Hkv, page, D, g)
    v, vs = _codes(pool, Hkv, page, D, g)
    order = torch.randperm(pool, generator=g, device=DEV)[: B * width]
    return {"k": k, "v": v, "ks": ks, "vs": vs,
            "table": order.view(B, width).to(torch.int32).contiguous()}


def _lens(case, g):
    """Lengths spread evenly from lo to hi, in an order of their own for each seed."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    n = torch.tensor([hi - (hi - lo) * i // max(1, B - 1) for i in range(B)], dtype=torch.int32)
    return n.to(DEV)[torch.randperm(B, generator=g, device=DEV)].contiguous()


def _parents(B, T, g):
    """Trees as the tree sampler lays them out: node 0 the root, then up to 16 nodes a
    depth, ordered by depth and parent; parents index earlier nodes."""
    par = torch.full((B, T), -1, dtype=torch.int64, device=DEV)
    first, width, at = 0, 1, 1
    while at < T:
        n = min(16, 4 * width, T - at)
        pick = torch.randint(0, width, (B, n), generator=g, device=DEV)
        par[:, at:at + n] = first + pick.sort(1).values
        first, width, at = at, n, at + n
    return par.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    op, s = case["op"], {"case": case}
    if op in ("norm", "quantize"):
        t = _dtype(case["dtype"])
        s["x"] = normal(case["M"], case["d"], dtype=t)
        if op == "norm":
            s["res"] = normal(case["M"], case["d"], std=2.0, dtype=t) if case["residual"] else None
            s["w"] = (1.0 + normal(case["d"], std=0.2, dtype=torch.float32)).to(t)
    elif op == "linear":
        M, K, N, r = case["M"], case["d_in"], case["d_out"], case["r"]
        s["xq"], s["xs"] = _int8_rows(normal(M, K, dtype=torch.float32))
        s["wq"], s["ws"] = _int8_rows(normal(N, K, std=0.02, dtype=torch.float32))
        if r:
            s["aq"], s["as"] = _int8_rows(normal(r, K, std=0.02, dtype=torch.float32))
            s["bm"] = normal(N, r, std=0.01)
            s["scale"] = 2.0
            # the first row of each block of 17 keeps the AR weights alone
            s["gate"] = (torch.arange(M, device=DEV) % 17 != 0).to(torch.uint8)
    elif op == "append":
        B, T = case["B"], case["T"]
        s["cache"] = _cache(case, case["len"] + T, g)
        s["k"] = normal(B, T, case["Hkv"], case["D"])
        s["v"] = normal(B, T, case["Hkv"], case["D"], std=1.5)
        lo = case["len"] // 2
        s["start"] = torch.randint(lo, case["len"] + 1, (B,), generator=g,
                                   device=DEV).to(torch.int32)
        s["count"] = (torch.randint(0, T + 1, (B,), generator=g, device=DEV).to(torch.int32)
                      if case["counts"] else None)
    else:
        B, T, D = case["B"], case["T"], case["D"]
        s["cache"] = _cache(case, case["hi"], g)
        s["lens"] = _lens(case, g)
        s["q"] = normal(B, T, case["Hq"], D)
        s["k"] = normal(B, T, case["Hkv"], D)
        s["v"] = normal(B, T, case["Hkv"], D)
        s["out"] = torch.zeros(B, T, case["Hq"], D, dtype=torch.bfloat16, device=DEV)
        s["parent"] = _parents(B, T, g) if case["tree"] else None
        # a tree that shares prefixes uses fewer than its node slots
        s["nodes"] = (torch.randint((T + 1) // 2, T + 1, (B,), generator=g,
                                    device=DEV).to(torch.int32) if case["tree"] else None)
    return s


# ---------------------------------------------------------------------------
# plain forms (float32, or float64 for exact())
# ---------------------------------------------------------------------------


def _values(q, scale):
    """bf16 values that 8-bit rows and their scales stand for."""
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    return torch.mul(q, scale[:, None], out=out)


def _quantize(y):
    scale = y.abs().amax(1) / 127.0
    q = torch.round(y / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-127, 127)
    return q.to(torch.int8), scale


def _norm_plain(s):
    x, res = s["x"], s["res"]
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hf = h.float()
    y = hf * torch.rsqrt((hf * hf).mean(1, keepdim=True) + EPS) * s["w"].float()
    q, scale = _quantize(y)
    return h, _values(q, scale), scale


def _linear_plain(s):
    t = _dtype(s["case"]["out"])
    x = s["xq"].float()
    y = (x @ s["wq"].float().t()) * s["xs"][:, None] * s["ws"]
    if not s["case"]["r"]:
        return y.to(t)
    a = (x @ s["aq"].float().t()) * s["xs"][:, None] * (s["as"] * s["scale"])
    a = a.to(torch.bfloat16).float() * s["gate"][:, None]
    return y.to(t), (y + a @ s["bm"].float().t()).to(t)


def _append_one(codes, scales, x, table, start, count):
    """Rows x [B, T, H, D] into codes [pages, H, page, D] and scales [pages, H], in place."""
    B, T, H, D = x.shape
    page = codes.shape[2]
    pos = start.long()[:, None] + torch.arange(T, device=x.device)
    n = count.long()[:, None] if count is not None else torch.full((B, 1), T, device=x.device)
    live = torch.arange(T, device=x.device) < n
    ids = table.long().gather(1, (pos // page).clamp(max=table.shape[1] - 1))
    b, t = live.nonzero(as_tuple=True)
    pid, slot, rows = ids[b, t], pos[b, t] % page, x[b, t].float()
    # the scale of each touched page: that of its earlier tokens, grown where needed
    amax = torch.zeros_like(scales).index_reduce_(0, pid, rows.abs().amax(2), "amax")
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=x.device)
    touched[pid] = True
    fresh = torch.zeros_like(touched)
    fresh[pid[slot == 0]] = True
    old = torch.where(fresh[:, None], 0.0, scales)
    new = torch.maximum(old, _pow2_scale(amax))
    pages = touched.nonzero()[:, 0]
    safe = torch.where(new > 0, new, 1.0)
    grow = (old / safe)[pages]
    kept = torch.where(grow[:, :, None, None] == 1, codes[pages].float(),
                       codes[pages].float() * grow[:, :, None, None])
    # slots from the first appended one on are not the page's earlier tokens: left as they are
    first = torch.full((scales.shape[0],), page, dtype=torch.int64, device=x.device)
    first.index_reduce_(0, pid, slot, "amin")
    earlier = torch.arange(page, device=x.device) < first[pages, None]
    codes[pages] = torch.where(earlier[:, None, :, None], kept.to(FP8).float(),
                               codes[pages].float()).to(FP8)
    scales[pages] = new[pages]
    codes[pid, :, slot] = (rows / safe[pid][:, :, None]).clamp(-448, 448).to(FP8)


def _append_plain(s):
    c = s["cache"]
    _append_one(c["k"], c["ks"], s["k"], c["table"], s["start"], s["count"])
    _append_one(c["v"], c["vs"], s["v"], c["table"], s["start"], s["count"])
    return c["k"], c["ks"], c["v"], c["vs"]


def _ancestors(parent):
    """[B, T, T]: whether column j is row i or one of its ancestors."""
    B, T = parent.shape
    up = (parent.long()[:, :, None] == torch.arange(T, device=parent.device)).float()
    up = up + torch.eye(T, device=parent.device)
    for _ in range(max(1, T.bit_length())):  # paths of length 1, 2, 4, ...
        up = (up @ up).clamp(max=1.0)
    return up > 0


def _gather(codes, scales, table, dtype):
    """[B, tokens, H, D] values of a cache's sequences."""
    t = table.long()
    x = codes[t].to(dtype) * scales[t].to(dtype)[:, :, :, None, None]  # [B, width, H, page, D]
    return x.permute(0, 1, 3, 2, 4).flatten(1, 2)


def _attend(s, dtype):
    c, q = s["cache"], s["q"].to(dtype)
    B, T, Hq, D = q.shape
    Hkv = s["k"].shape[2]
    k, v = (torch.cat([_gather(c[n], c[n + "s"], c["table"], dtype), s[n].to(dtype)], 1)
            for n in ("k", "v"))
    L = k.shape[1] - T
    q = q.view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = q @ k.permute(0, 2, 3, 1) / math.sqrt(D)  # [B, Hkv, G * T, L + T]
    old = torch.arange(L, device=q.device) < s["lens"].long()[:, None]
    if s["parent"] is None:
        new = torch.ones(T, T, dtype=torch.bool, device=q.device).tril().expand(B, T, T)
    else:
        new = _ancestors(s["parent"])
    see = torch.cat([old[:, None].expand(B, T, L), new], 2)[:, None, None]
    score = score.view(B, Hkv, -1, T, L + T).masked_fill_(~see, -math.inf)
    score = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    # (G * T) rows of weights against [L + T, D]; slots behind a sequence have weight 0
    o = (score.flatten(2, 3) @ v.permute(0, 2, 1, 3)).view(B, Hkv, -1, T, D) / total
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D)


def _attend_plain(s):
    o = _attend(s, torch.float32).to(torch.bfloat16)
    if s["nodes"] is None:
        return o
    used = torch.arange(o.shape[1], device=o.device) < s["nodes"].long()[:, None]
    return torch.where(used[:, :, None, None], o, s["out"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _run_own(s):
    from lossless_decoding_b200 import api

    op = s["case"]["op"]
    if op == "norm":
        r = api.rms_norm(s["x"], s["w"], EPS, residual=s["res"])
        return r.h, _values(r.q, r.scale), r.scale
    if op == "quantize":
        q, scale = api.quantize_rows(s["x"])
        return _values(q, scale), scale
    if op == "linear":
        t = _dtype(s["case"]["out"])
        if not s["case"]["r"]:
            return api.dualpath_linear_int8(s["xq"], s["xs"], s["wq"], s["ws"], out_dtype=t)[0]
        return api.dualpath_linear_int8(s["xq"], s["xs"], s["wq"], s["ws"], s["aq"], s["as"],
                                        s["bm"], s["scale"], gate=s["gate"], out_dtype=t)
    c = s["cache"]
    cache = api.KvCache(c["k"], c["v"], c["ks"], c["vs"], c["table"])
    if op == "append":
        api.kv_append(cache, s["k"], s["v"], s["start"], count=s["count"])
        return cache.k, cache.k_scale, cache.v, cache.v_scale
    return api.block_attention(s["q"], s["k"], s["v"], cache, s["lens"],
                               parent=s["parent"], num_new=s["nodes"], out=s["out"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _norm_plain(state)
    if op == "quantize":
        q, scale = _quantize(state["x"].float())
        return _values(q, scale), scale
    if op == "linear":
        return _linear_plain(state)
    if op == "append":
        return _append_plain(state)
    return _attend_plain(state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op in ("norm", "quantize"):
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["M"] * case["d"]
        moved = n * e + n + 4 * case["M"]  # x in, q and scales out
        if op == "norm":
            moved += case["d"] * e + n * e * (2 if case["residual"] else 0)  # w; residual in, h out
        return {"bytes": moved, "flops": (7 if op == "norm" else 3) * n}
    if op == "linear":
        M, K, N, r = case["M"], case["d_in"], case["d_out"], case["r"]
        e = 2 if case["out"] == "bf16" else 4
        moved = M * K + N * K + 4 * (M + N) + M * N * e
        flops = 2 * M * K * N
        if r:
            moved += r * K + 4 * r + 2 * N * r + M + M * N * e
            flops += 2 * M * r * (K + N)
        return {"bytes": moved, "flops": flops}
    B, T, Hkv, D, page = case["B"], case["T"], case["Hkv"], case["D"], case["page"]
    if op == "append":
        n = B * (T / 2 if case["counts"] else T)  # tokens
        return {"bytes": 2 * Hkv * D * n * 3 + 2 * 4 * Hkv * (n / page + B),
                "flops": 2 * Hkv * D * n * 3}
    Hq, lo, hi = case["Hq"], case["lo"], case["hi"]
    total = sum(hi - (hi - lo) * i // max(1, B - 1) for i in range(B))
    rows = T * 3 / 4 if case["tree"] else T
    depth = 1 + T / 16 if case["tree"] else (T + 1) / 2  # new tokens that a row sees
    return {"bytes": 2 * Hkv * D * total + 2 * 4 * Hkv * total / page
            + 2 * B * rows * D * (2 * Hq + 2 * Hkv),
            "flops": 4 * Hq * D * rows * (total + B * depth)}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        h = s["x"].double()
        if s["res"] is not None:
            # the sum is rounded to the rows' own type, as the layer that follows reads it
            h = (h + s["res"].double()).to(s["x"].dtype).double()
        y = h / (h.pow(2).sum(1, keepdim=True) / case["d"] + EPS).sqrt() * s["w"].double()
        scale = y.abs().max(1).values / 127
        return h, (y / scale[:, None]).round() * scale[:, None], scale
    if op == "quantize":
        x = s["x"].double()
        scale = x.abs().max(1).values / 127
        return (x / scale[:, None]).round() * scale[:, None], scale
    if op == "linear":
        x = s["xq"].double() * s["xs"].double()[:, None]
        w = s["wq"].double() * s["ws"].double()[:, None]
        y = torch.mm(x, w.t())
        del w
        if not case["r"]:
            return y
        a = s["aq"].double() * s["as"].double()[:, None]
        down = torch.mm(x, a.t()) * s["scale"] * s["gate"].double()[:, None]
        return y, y + torch.mm(down, s["bm"].double().t())
    if op == "append":
        return None, *_append_exact(s, "k"), None, *_append_exact(s, "v")
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        _attend_exact(s, b, o)
    return o


def _append_exact(s, name):
    """The scales that one half of an append leaves, page by page."""
    c, case = s["cache"], s["case"]
    page = case["page"]
    table, start = c["table"].tolist(), s["start"].tolist()
    count = s["count"].tolist() if s["count"] is not None else [case["T"]] * case["B"]
    scales = c[name + "s"].double().cpu()
    peak = s[name].double().abs().amax(3).cpu()  # [B, T, H]
    for b in range(case["B"]):
        at, end = start[b], start[b] + count[b]
        while at < end:
            stop = min(end, (at // page + 1) * page)
            top = peak[b, at - start[b]:stop - start[b]].amax(0) / 448
            grown = torch.where(top > 0, 2.0 ** torch.ceil(torch.log2(top)), top)
            p = table[b][at // page]
            scales[p] = grown if at % page == 0 else torch.maximum(scales[p], grown)
            at = stop
    return (scales.to(DEV),)


def _attend_exact(s, b, o):
    """One sequence's outputs into o[b], the cached tokens and the new ones side by side."""
    case, c = s["case"], s["cache"]
    n, T, D = int(s["lens"][b]), case["T"], case["D"]
    used = int(s["nodes"][b]) if s["nodes"] is not None else T
    group = case["Hq"] // case["Hkv"]
    if s["parent"] is None:
        see = torch.arange(T).view(1, T) <= torch.arange(T).view(T, 1)
    else:
        see, par = torch.zeros(T, T, dtype=torch.bool), s["parent"][b].tolist()
        for i in range(T):
            j = i
            while j >= 0:
                see[i, j] = True
                j = par[j]
    bias = torch.where(see, 0.0, -math.inf).double().to(DEV)
    pages = c["table"][b].long()
    for h in range(case["Hkv"]):
        k, v = ((c[x][pages, h].double() * c[x + "s"][pages, h].double()[:, None, None])
                .reshape(-1, D)[:n] for x in ("k", "v"))
        k, v = torch.cat([k, s["k"][b, :, h].double()]), torch.cat([v, s["v"][b, :, h].double()])
        for i in range(h * group, (h + 1) * group):
            z = s["q"][b, :, i].double() @ k.t() * D ** -0.5
            z[:, n:] += bias
            p = torch.softmax(z, 1)
            o[b, :used, i] = (p @ v)[:used]
