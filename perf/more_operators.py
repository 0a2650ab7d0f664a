"""Operators of the decode step, as they are measured: the append of rotated keys and of values to a paged cache
held in 4 bits, the attention of new tokens over that cache, and the low-rank adapters of many requests beside a
shared projection.

`own` False: elementary torch operations in 32 bits.  `own` True: the framework's calls on the same state.

The 4-bit cache: a head's row of d elements is d codes of -7 .. 7 in four groups of d / 4, and a record of a float32
scale and four 8-bit multipliers; an element is code * multiplier * scale.  Of eight elements, element e lies at bits
4 (e / 2) + 16 (e % 2) of a 32-bit word, as code + 8.
"""
import math

import torch

own = False

ROPE_BASE = 500000.0

# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------


def _append(B, n, ctx, page, Hq, Hkv, d, rot, layout):
    return {"op": "append", "B": B, "n": n, "ctx": ctx, "page": page, "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot,
            "layout": layout, "ragged": False}


def _attend(B, n, ctx, page, Hq, Hkv, d, blk, ragged):
    return {"op": "attend", "B": B, "n": n, "ctx": ctx, "page": page, "Hq": Hq, "Hkv": Hkv, "d": d, "blk": blk,
            "ragged": ragged}


def _lora(B, n, H, N, R, adapters, ragged):
    """B requests of n tokens (ragged: from a quarter of n on), each with one of the adapters or none."""
    return {"op": "lora", "B": B, "n": n, "H": H, "N": N, "R": R, "adapters": adapters, "ragged": ragged}


def listed():
    return [
        # four sequences with one new token each
        dict(_append(4, 1, 2000, 16, 16, 4, 128, 128, "half"), name="append4_token"),
        # sixteen refinement blocks, half of each head rotated, interleaved pairs
        dict(_append(16, 32, 8191, 64, 16, 4, 128, 64, "interleaved"), name="append4_block"),
        # the last 8192 tokens of a long prompt
        dict(_append(1, 8192, 131072, 64, 16, 4, 128, 128, "half"), name="append4_prompt"),
        # one sequence, one token, a short and odd context: latency
        dict(_attend(1, 1, 777, 16, 16, 4, 128, 1, False), name="attend4_token_short"),
        # a serving batch of single tokens with contexts of very different lengths, small pages
        dict(_attend(32, 1, 8192, 16, 16, 4, 128, 1, True), name="attend4_batch"),
        # refinement blocks of 32 tokens
        dict(_attend(16, 32, 4000, 64, 16, 4, 128, 32, True), name="attend4_block"),
        # the same with smaller heads and more of them
        dict(_attend(8, 32, 16384, 64, 32, 8, 64, 32, True), name="attend4_block_d64"),
        # few sequences, very long contexts: the split over the length carries everything
        dict(_attend(2, 1, 200000, 64, 32, 8, 128, 1, False), name="attend4_long"),
        # one request, one token: latency
        dict(_lora(1, 1, 2048, 2560, 16, 8, False), name="lora_token"),
        # a serving batch of single tokens of many users
        dict(_lora(64, 1, 4096, 5120, 16, 24, False), name="lora_batch"),
        # sixteen refinement blocks of 32 tokens
        dict(_lora(16, 32, 2048, 2560, 32, 12, False), name="lora_block"),
        # prompts of different lengths, large ranks
        dict(_lora(7, 2048, 4096, 5120, 64, 4, True), name="lora_prompt"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "lora", "lora"])
    if op == "lora":
        H = rng.choice([512, 1000, 1024, 1536, 2048, 2056, 2560, 4096, 5120])
        N = rng.choice([264, 512, 1024, 1280, 2048, 2560, 4096, 5000, 5120])
        R = rng.choice([8, 16, 16, 24, 32, 64, 128])
        ragged = rng.random() < 0.5
        n = rng.choice([1, 1, 32, _log_int(rng, 2, 2048)])
        B = _log_int(rng, 1, max(1, min(256, 8192 // n)))
        # no more adapters than the largest listed case's weights and tokens would take
        return _lora(B, n, H, N, R, _log_int(rng, 1, max(1, min(64, 8192 // R))), ragged)
    Hkv, group = rng.choice([(4, 4), (8, 4), (1, 8), (2, 5), (4, 1), (2, 16)])
    d = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 20, 32, 64, 128])
    if op == "append":
        n = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(64, 8192 // n)))
        ctx = n + _log_int(rng, 1, 200000)
        rot = rng.choice([d, d // 2, d // 4])
        return _append(B, n, ctx, page, Hkv * group, Hkv, d, rot, rng.choice(["half", "interleaved"]))
    n = rng.choice([1, 1, 1, 2, 7, 32, 32])
    ctx = n + _log_int(rng, 1, 100000)
    # at most half of the largest listed case's cache, and about its products
    room = min(200000 * 8 // (ctx * Hkv), 16 * 4096 * 16 * 32 // (ctx * Hkv * group * n))
    B = _log_int(rng, 1, max(1, min(128, room)))
    return _attend(B, n, ctx, page, Hkv * group, Hkv, d, rng.choice([1, 32]), rng.random() < 0.5)


def _spread(B, low, high):
    return [low + (high - low) * i // (B - 1) for i in range(B)] if B > 1 else [high]


def _lens(c):
    """Cached length of each sequence, its new tokens included: all `ctx`, or spread from a quarter of it."""
    return _spread(c["B"], max(c["n"], c["ctx"] // 4), c["ctx"]) if c["ragged"] else [c["ctx"]] * c["B"]


def _requests(c):
    """Tokens of each request."""
    return _spread(c["B"], max(1, c["n"] // 4), c["n"]) if c["ragged"] else [c["n"]] * c["B"]


def _touched(c):
    """Pages that an append's new tokens lie in."""
    return sum(-(-L // c["page"]) - (L - c["n"]) // c["page"] for L in _lens(c))


def work(case):
    c = case
    if c["op"] == "lora":
        T, used = sum(_requests(c)), min(c["adapters"], c["B"])
        return {"bytes": 2 * T * (c["H"] + 2 * c["N"]) + 2 * used * c["R"] * (c["H"] + c["N"]) + 4 * T,
                "flops": 2 * T * c["R"] * (c["H"] + c["N"])}
    row = c["d"] // 2 + 8  # bytes of one cached head row
    if c["op"] == "append":
        T, pages = c["B"] * c["n"], _touched(c)
        moved = T * (c["Hq"] * c["d"] * 4 + 2 * c["Hkv"] * (c["d"] * 2 + row))
        values = 2 * (pages + 1) * c["Hkv"] * c["page"] * (row + 2 * c["d"])  # the cache read back
        return {"bytes": moved + values + 4 * (pages + c["B"] + c["rot"] // 2),
                "flops": T * ((c["Hq"] + c["Hkv"]) * c["rot"] * 3 + c["rot"] * 20)}
    cached = sum(_lens(c))
    pairs = 0
    for L in _lens(c):
        pairs += sum(min(L, ((L - c["n"] + i) // c["blk"] + 1) * c["blk"]) for i in range(c["n"]))
    T = c["B"] * c["n"]
    return {"bytes": 2 * cached * c["Hkv"] * row + T * c["Hq"] * (c["d"] * 4 + 4) + 4 * cached // c["page"],
            "flops": 4 * pairs * c["Hq"] * c["d"]}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------


def _pack(codes):
    """Codes (int8, -8 .. 7) [..., d] as the cache's bytes [..., d / 2]."""
    u = (codes + 8).to(torch.uint8).view(*codes.shape[:-1], -1, 2, 2, 2)  # [word][half of the bits][low, high][parity]
    return (u[..., 0, :] | (u[..., 1, :] << 4)).transpose(-1, -2).reshape(*codes.shape[:-1], codes.shape[-1] // 2)


def _unpack(cache):
    """The cache's bytes [..., d / 2] as codes (int8) [..., d]."""
    b = cache.view(*cache.shape[:-1], -1, 2, 2).transpose(-1, -2)  # [word][half of the bits][parity]
    return (torch.stack((b & 15, b >> 4), -2).to(torch.int8) - 8).reshape(*cache.shape[:-1], cache.shape[-1] * 2)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    if c["op"] == "lora":
        H, N, R, n = c["H"], c["N"], c["R"], c["adapters"]
        counts = _requests(c)
        T = sum(counts)
        # every seventh request or so, but not the first, is one of the base model
        choice = torch.randint(0, n, (c["B"],), generator=g, device=dev)
        choice[1:][torch.rand(c["B"] - 1, generator=g, device=dev) < 0.15] = -1
        adapter = choice.to(torch.int32).repeat_interleave(torch.tensor(counts, device=dev))
        ranks = torch.randint(1, R // 8 + 1, (n,), generator=g, device=dev, dtype=torch.int32) * 8
        ranks[::2] = R
        s = {"case": c, "adapter": adapter, "ranks": ranks, "scale": 2.0 * torch.rand(n, generator=g, device=dev) + 0.5,
             "x": randn(T, H).bfloat16(), "y": randn(T, N).bfloat16(),
             "a": (randn(n, R, H) / H ** 0.5).bfloat16(), "b": (0.3 * randn(n, N, R) / R ** 0.5).bfloat16(),
             "out": torch.empty((T, N), dtype=torch.bfloat16, device=dev)}
        # the plain form's plan: each adapter's tokens
        used = set(choice.tolist())
        s["rows"] = [(i, r, torch.nonzero(adapter == i).flatten()) for i, r in enumerate(ranks.tolist()) if i in used]
        return s

    B, n, page, Hq, Hkv, d = c["B"], c["n"], c["page"], c["Hq"], c["Hkv"], c["d"]
    lens = torch.tensor(_lens(c), dtype=torch.int64, device=dev)
    lens = lens[torch.randperm(B, generator=g, device=dev)]
    most = -(-c["ctx"] // page)
    at = torch.arange(most, device=dev)
    if c["op"] == "append":
        # the pages before the new tokens' are a prefix that the sequences share (page 0): nothing reads them here
        mine = (at >= ((lens - n) // page)[:, None]) & (at < ((lens + page - 1) // page)[:, None])
    else:
        mine = at < ((lens + page - 1) // page)[:, None]
    count = int(mine.sum())
    n_pages = count + 1
    table = torch.zeros((B, most), dtype=torch.int32, device=dev)
    table[mine] = (1 + torch.randperm(count, generator=g, device=dev)).to(torch.int32)
    # the fused projection's output: q, k and v of a token side by side; some channels of q and k are larger
    gain = (0.5 + 1.5 * torch.rand(d, generator=g, device=dev)).repeat(Hq + 2 * Hkv, 1)
    gain[Hq + Hkv:] = 1.0
    qkv = (randn(B * n, Hq + 2 * Hkv, d) * gain).bfloat16()
    s = {"case": c, "lens": lens.to(torch.int32), "table": table,
         "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:]}
    shape = (n_pages, Hkv, page, d)
    for cache, record in (("kc", "ks"), ("vc", "vs")):
        z = torch.randn(shape, generator=g, device=dev, dtype=torch.float16)
        s[cache] = _pack(z.mul_(2.6).clamp_(-7, 7).round_().to(torch.int8))
        del z
        # the multipliers of a row's groups: the largest 255, the others somewhat below
        m = torch.randint(90, 256, shape[:3] + (4,), generator=g, device=dev, dtype=torch.int32)
        m.scatter_(3, torch.randint(0, 4, shape[:3] + (1,), generator=g, device=dev), 255)
        scale = (0.1 * randn(*shape[:3])).exp_().div_(2.6 * 170)
        s[record] = torch.cat((scale.unsqueeze(-1).view(torch.uint8), m.to(torch.uint8)), -1)
    if c["op"] == "append":
        f = ROPE_BASE ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
        s["inv_freq"] = f.to(torch.float32).to(dev)
        s["q_out"] = torch.empty((B * n, Hq, d), dtype=torch.bfloat16, device=dev)
        s["kv_values"] = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        import quantized_moe_expert_routed_gb300 as M
        return {"append": _own_append, "attend": _own_attend, "lora": _own_lora}[op](M, state)
    return {"append": _plain_append, "attend": _plain_attend, "lora": _plain_lora}[op](state)


def _own_append(M, s):
    c = s["case"]
    layout = M.ROPE_HALF if c["layout"] == "half" else M.ROPE_INTERLEAVED
    q = M.mnw_kv_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], inv_freq=s["inv_freq"],
                        layout=layout, k_scale=s["ks"], v_scale=s["vs"], q_out=s["q_out"])
    return [q, M.mnw_kv_values(s["kc"], s["ks"], out=s["kv_values"][0]),
            M.mnw_kv_values(s["vc"], s["vs"], out=s["kv_values"][1])]


def _own_attend(M, s):
    c = s["case"]
    return list(M.mnw_attn_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], c["blk"], c["d"] ** -0.5,
                                 k_scale=s["ks"], v_scale=s["vs"], want_lse=True))


def _own_lora(M, s):
    return M.mnw_lora_add(s["y"], s["x"], s["a"], s["b"], s["adapter"], scale=s["scale"], ranks=s["ranks"],
                          out=s["out"])


def _dequantise(cache, record):
    """float32 values [..., d] of cached rows."""
    codes = _unpack(cache).float()
    factor = record[..., :4].contiguous().view(torch.float32) * record[..., 4:].float()
    return (codes.unflatten(-1, (4, -1)) * factor.unsqueeze(-1)).flatten(-2)


def _quantise(x):
    """Bytes and records of rows (last dimension) of float32 values."""
    groups = x.unflatten(-1, (4, -1))
    top = groups.abs().amax(-1)
    # the smallest value of 8 significant bits that is not below max / 1785
    scale = ((top.amax(-1, keepdim=True) / 1785.0).view(torch.int32) + 0xFFFF & -0x10000).view(torch.float32)
    m = torch.where(scale > 0, torch.ceil(top / (7.0 * scale)), torch.ones_like(top)).clamp_(1.0, 255.0)
    step = (scale * m).unsqueeze(-1)
    codes = torch.where(step > 0, torch.round(groups / step), torch.zeros_like(groups)).to(torch.int8)
    return _pack(codes.flatten(-2)), torch.cat((scale.view(torch.uint8), m.to(torch.uint8)), -1)


def _rotate(x, cos, sin, rot, layout):
    x = x.float()
    if layout == "half":
        u, w = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((u * cos - w * sin, w * cos + u * sin), -1)
    else:
        u, w = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1).bfloat16()


def _plain_append(s):
    c = s["case"]
    B, n, page, rot = c["B"], c["n"], c["page"], c["rot"]
    pos = (s["lens"].long()[:, None] - n + torch.arange(n, device=s["lens"].device)).flatten()
    angle = pos[:, None].double() * s["inv_freq"].double()  # 32 bits would lose far positions' fractions of a turn
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, rot, c["layout"]))
    k = _rotate(s["k"], cos, sin, rot, c["layout"])
    seq = torch.arange(B, device=pos.device).repeat_interleave(n)
    pages, slots = s["table"][seq, pos // page].long(), pos % page
    s["kc"][pages, :, slots], s["ks"][pages, :, slots] = _quantise(k.float())
    s["vc"][pages, :, slots], s["vs"][pages, :, slots] = _quantise(s["v"].float())
    return [s["q_out"], s["kv_values"][0].copy_(_dequantise(s["kc"], s["ks"])),
            s["kv_values"][1].copy_(_dequantise(s["vc"], s["vs"]))]


def _dense(cache, record, table):
    """Every sequence's cached rows one after another: [B, Hkv, keys, d] float32."""
    return _dequantise(cache[table.long()], record[table.long()]).transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c = s["case"]
    B, n, Hq, Hkv, d, blk = c["B"], c["n"], c["Hq"], c["Hkv"], c["d"], c["blk"]
    G = Hq // Hkv
    k, v = _dense(s["kc"], s["ks"], s["table"]), _dense(s["vc"], s["vs"], s["table"])
    q = s["q"].float().reshape(B, n, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, n * G, d)
    scores = torch.matmul(q, k.transpose(2, 3)) * (d ** -0.5)
    pos = s["lens"].long()[:, None] - n + torch.arange(n, device=k.device)
    end = torch.minimum(s["lens"].long()[:, None], (pos // blk + 1) * blk)  # [B, n]
    end = end.repeat_interleave(G, 1)[:, None, :, None]
    scores.masked_fill_(torch.arange(k.shape[2], device=k.device) >= end, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (torch.matmul(p, v) / total).view(B, Hkv, n, G, d).transpose(1, 2).reshape(B * n, Hq, d).bfloat16()
    lse = (top + total.log()).view(B, Hkv, n, G).transpose(1, 2).reshape(B * n, Hq)
    return [out, lse]


def _plain_lora(s):
    out = s["out"].copy_(s["y"])
    for i, rank, rows in s["rows"]:
        v = torch.matmul(s["x"][rows].float(), s["a"][i, :rank].float().T)
        d = torch.matmul(v, s["b"][i, :, :rank].float().T)
        out[rows] = (s["y"][rows].float() + s["scale"][i] * d).bfloat16()
    return out


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "lora": _exact_lora}[case["op"]](case, s)


def _exact_values(cache, record):
    """Values of cached rows, element by element of each 32-bit word."""
    words = cache.contiguous().view(torch.int32).long()
    parts = [(words >> (4 * (e // 2) + 16 * (e % 2)) & 15) - 8 for e in range(8)]
    codes = torch.stack(parts, -1).flatten(-2).double()
    d = codes.shape[-1]
    unit = record[..., :4].contiguous().view(torch.float32).double()
    m = record[..., 4:].double().repeat_interleave(d // 4, -1)
    return codes * m * unit


def _exact_round(x):
    """The values that rows of doubles (of 8 significant bits) are held as."""
    d = x.shape[-1]
    size = x.abs()
    most = size.max(-1, keepdim=True).values
    bound = most / 1785
    power = torch.floor(torch.log2(bound.clamp_min(1e-300)))
    unit = torch.ceil(bound / 2.0 ** (power - 7)) * 2.0 ** (power - 7)
    unit = torch.where(most > 0, unit, torch.ones_like(unit))
    parts = []
    for g in range(4):
        y = x[..., g * (d // 4):(g + 1) * (d // 4)]
        m = torch.ceil(y.abs().max(-1, keepdim=True).values / 7 / unit).clamp(1, 255)
        parts.append(torch.round(y / (m * unit)) * m * unit)
    return torch.cat(parts, -1)


def _exact_append(c, s):
    n, half, page = c["n"], c["rot"] // 2, c["page"]
    freq = s["inv_freq"].double()
    kc, vc = _exact_values(s["kc"], s["ks"]), _exact_values(s["vc"], s["vs"])

    def turn(x, a):
        x = x.double()
        first = torch.arange(half, device=x.device) if c["layout"] == "half" else torch.arange(0, c["rot"], 2, device=x.device)
        second = first + (half if c["layout"] == "half" else 1)
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(a), a)
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y
    qs = []
    for b, L in enumerate(s["lens"].tolist()):
        rows = slice(b * n, (b + 1) * n)
        pos = torch.arange(L - n, L, device=freq.device)
        a = (pos.double()[:, None] * freq)[:, None, :]
        qs.append(turn(s["q"][rows], a))
        where = s["table"][b, pos // page].long()
        kc[where, :, pos % page] = _exact_round(turn(s["k"][rows], a).bfloat16().double())
        vc[where, :, pos % page] = _exact_round(s["v"][rows].double())
    return [torch.cat(qs), kc, vc]


def _exact_attend(c, s):
    if work(c)["flops"] > 4e12:
        return None
    n, page, d, G = c["n"], c["page"], c["d"], c["Hq"] // c["Hkv"]
    out = torch.empty((c["B"] * n, c["Hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.empty((c["B"] * n, c["Hq"]), dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-L // page)].long()
        ends = torch.tensor([min(L, ((L - n + i) // c["blk"] + 1) * c["blk"]) for i in range(n)], device="cuda")
        hidden = torch.arange(L, device="cuda")[None, :] >= ends[:, None]
        for h in range(c["Hkv"]):
            K = _exact_values(s["kc"][pages, h], s["ks"][pages, h]).reshape(-1, d)[:L]
            V = _exact_values(s["vc"][pages, h], s["vs"][pages, h]).reshape(-1, d)[:L]
            for j in range(h * G, (h + 1) * G):
                z = s["q"][b * n:(b + 1) * n, j].double() @ K.T / math.sqrt(d)
                z[hidden] = -math.inf
                total = torch.logsumexp(z, dim=1)
                lse[b * n:(b + 1) * n, j] = total
                out[b * n:(b + 1) * n, j] = torch.exp(z - total[:, None]) @ V
    return [out, lse]


def _exact_lora(c, s):
    out = s["y"].double()
    ids, ranks = s["adapter"].tolist(), s["ranks"].tolist()
    for i in sorted(set(ids) - {-1}):
        rows = torch.tensor([j == i for j in ids], device="cuda")
        b, a = s["b"][i].double()[:, :ranks[i]], s["a"][i].double()[:ranks[i]]
        for part in torch.nonzero(rows).flatten().split(1024):
            out[part] += s["scale"][i].double() * torch.einsum("nr,rh,th->tn", b, a, s["x"][part].double())
    return out
