"""The decode step's operators around the routed-expert layer, as they are measured: the root-mean-square norm
with the residual's addition (BF16 or INT8-group output), the append of rotated keys and of values to a paged
cache, and the attention of new tokens over that cache.

`own` False: elementary torch operations in 32 bits.  `own` True: the framework's calls on the same state.
"""
import math

import torch

own = False

NORM_EPS = 1e-6
ROPE_BASE = 500000.0

# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------


def _norm(T, H, out, residual=True):
    return {"op": "norm", "T": T, "H": H, "out": out, "residual": residual}


def _append(B, n, ctx, page, fmt, Hq, Hkv, d, rot, layout, factor=1.0):
    return {"op": "append", "B": B, "n": n, "ctx": ctx, "page": page, "fmt": fmt, "Hq": Hq, "Hkv": Hkv, "d": d,
            "rot": rot, "layout": layout, "factor": factor}


def _attend(B, n, ctx, page, fmt, Hq, Hkv, d, blk, ragged):
    return {"op": "attend", "B": B, "n": n, "ctx": ctx, "page": page, "fmt": fmt, "Hq": Hq, "Hkv": Hkv, "d": d,
            "blk": blk, "ragged": ragged}


def listed():
    return [
        # one sequence, one new token: the norm before the router; latency alone counts
        dict(_norm(1, 2048, "bf16"), name="norm_token"),
        # one 32-token refinement block, ahead of the INT8-activation experts
        dict(_norm(32, 2048, "int8"), name="norm_block_int8"),
        # a prompt batch of the larger model; the embedding's norm has no residual, odd row count and width
        dict(_norm(8192, 4096, "int8"), name="norm_prompt_int8"),
        dict(_norm(1027, 2176, "bf16", residual=False), name="norm_odd"),
        # four sequences with one new token each
        dict(_append(4, 1, 2000, 16, "bf16", 16, 4, 128, 128, "half"), name="append_token"),
        # sixteen refinement blocks into an INT8 cache, half of each head rotated, interleaved pairs
        dict(_append(16, 32, 8191, 64, "int8", 16, 4, 128, 64, "interleaved"), name="append_block_int8"),
        # the last 8192 tokens of a long prompt, frequencies scaled for it
        dict(_append(1, 8192, 131072, 64, "bf16", 16, 4, 128, 128, "half", 8.0), name="append_prompt"),
        # one sequence, one token, a short and odd context: latency
        dict(_attend(1, 1, 777, 16, "bf16", 16, 4, 128, 1, False), name="attend_token_short"),
        # a serving batch of single tokens with contexts of very different lengths, small pages
        dict(_attend(32, 1, 8192, 16, "bf16", 16, 4, 128, 1, True), name="attend_batch"),
        # refinement blocks of 32 tokens over an INT8 cache
        dict(_attend(16, 32, 4000, 64, "int8", 16, 4, 128, 32, True), name="attend_block_int8"),
        # the same over a BF16 cache with smaller heads and more of them
        dict(_attend(8, 32, 16384, 64, "bf16", 32, 8, 64, 32, True), name="attend_block_d64"),
        # few sequences, very long contexts: the split over the length carries everything
        dict(_attend(2, 1, 200000, 64, "bf16", 32, 8, 128, 1, False), name="attend_long"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "attend"])
    if op == "norm":
        out = rng.choice(["bf16", "int8"])
        H = rng.choice([512, 640, 896, 1024, 1280, 1664, 2048, 2176, 2560, 2944, 4096, 4480, 5120])
        T = max(1, min(_log_int(rng, 1, 8192), 8192 * 4096 // H))
        return _norm(T, H, out, rng.random() < 0.75)
    Hkv, group = rng.choice([(4, 4), (8, 4), (1, 8), (2, 5), (4, 1), (2, 16)])
    d = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 20, 32, 64, 128])
    fmt = rng.choice(["bf16", "int8"])
    if op == "append":
        n = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(64, 8192 // n)))
        ctx = n + _log_int(rng, 1, 200000)
        rot = rng.choice([d, d // 2, d // 4])
        return _append(B, n, ctx, page, fmt, Hkv * group, Hkv, d, rot, rng.choice(["half", "interleaved"]),
                       rng.choice([1.0, 1.0, 4.0]))
    n = rng.choice([1, 1, 1, 2, 7, 32, 32])
    ctx = n + _log_int(rng, 1, 100000)
    # at most half of the largest listed case's cache, and about its products
    room = min(200000 * 8 // (ctx * Hkv), 16 * 4096 * 16 * 32 // (ctx * Hkv * group * n))
    B = _log_int(rng, 1, max(1, min(128, room)))
    return _attend(B, n, ctx, page, fmt, Hkv * group, Hkv, d, rng.choice([1, 32]), rng.random() < 0.5)


def _lens(c):
    """Cached length of each sequence, its new tokens included: all `ctx`, or spread from a quarter of it."""
    B, ctx, n = c["B"], c["ctx"], c["n"]
    if not c.get("ragged", False) or B == 1:
        return [ctx] * B
    low = max(n, ctx // 4)
    return [low + (ctx - low) * i // (B - 1) for i in range(B)]


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        per = 2 + 2 + (4 if c["residual"] else 0) + (1 + 4 / 128 if c["out"] == "int8" else 0)
        return {"bytes": n * per + 2 * c["H"], "flops": n * (8 if c["out"] == "int8" else 5)}
    row = c["d"] * 2 if c["fmt"] == "bf16" else c["d"] + 4  # bytes of one cached head row
    if c["op"] == "append":
        T = c["B"] * c["n"]
        pages = sum(-(-L // c["page"]) - (L - c["n"]) // c["page"] for L in _lens(c))
        moved = T * (c["Hq"] * c["d"] * 4 + 2 * c["Hkv"] * (c["d"] * 2 + row))
        return {"bytes": moved + 4 * (pages + c["B"] + c["rot"] // 2),
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


def _inv_freq(c, device):
    """Frequencies base^(-2i/rot); scaled contexts (factor > 1) slow the low ones down by `factor`, keep the high
    ones, and blend those between, by how often each turns within the original context of ctx / factor tokens."""
    rot, factor = c["rot"], c["factor"]
    f = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor > 1.0:
        turns = f * (c["ctx"] / factor) / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f.to(torch.float32).to(device), (0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        s = {"case": c, "w": (1.0 + 0.1 * randn(H)).bfloat16()}
        # a layer's output, and a residual stream with a few channels much larger than the rest
        s["x"] = (0.3 * randn(T, H)).bfloat16()
        big = 1.0 + 20.0 * (torch.rand(H, generator=g, device=dev) < 0.005).float()
        s["r"] = (randn(T, H) * big).bfloat16() if c["residual"] else None
        s["values"] = torch.empty((T, H // 128, 128), dtype=torch.bfloat16, device=dev) if c["out"] == "int8" else None
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
    # the fused projection's output: q, k and v of a token side by side
    gain = 0.5 + 1.5 * torch.rand(d, generator=g, device=dev)
    qkv = randn(B * n, Hq + 2 * Hkv, d).bfloat16()
    s = {"case": c, "lens": lens.to(torch.int32), "table": table, "n_pages": n_pages,
         "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:]}
    shape = (n_pages, Hkv, page, d)
    if c["fmt"] == "bf16":
        s["kc"] = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16).mul_(gain.bfloat16())
        s["vc"] = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        s["ks"] = s["vs"] = None
    else:
        s["kc"] = torch.randn(shape, generator=g, device=dev, dtype=torch.float16).mul_(45 * gain.half()).clamp_(-127, 127).round_().to(torch.int8)
        s["vc"] = torch.randn(shape, generator=g, device=dev, dtype=torch.float16).mul_(45).clamp_(-127, 127).round_().to(torch.int8)
        s["ks"] = (0.1 * randn(*shape[:3])).exp_().div_(45)
        s["vs"] = (0.1 * randn(*shape[:3])).exp_().div_(45)
    if c["op"] == "append":
        s["inv_freq"], s["mscale"] = _inv_freq(c, dev)
        s["q_out"] = torch.empty((B * n, Hq, d), dtype=torch.bfloat16, device=dev)
        if c["fmt"] == "int8":
            s["kv_values"] = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        import quantized_moe_expert_routed_gb300 as M
        return {"norm": _own_norm, "append": _own_append, "attend": _own_attend}[op](M, state)
    return {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend}[op](state)


def _values(codes, scales, out):
    """What 8-bit codes stand for."""
    return torch.mul(codes, scales.unsqueeze(-1), out=out)


def _own_norm(M, s):
    int8 = s["case"]["out"] == "int8"
    y, r, codes, scales = M.mnw_rmsnorm(s["x"], s["w"], NORM_EPS, residual=s["r"], int8=int8)
    got = [y] + ([r] if s["r"] is not None else [])
    return got + [_values(codes.view(s["values"].shape), scales, s["values"])] if int8 else got


def _own_append(M, s):
    c = s["case"]
    layout = M.ROPE_HALF if c["layout"] == "half" else M.ROPE_INTERLEAVED
    q = M.mnw_kv_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], inv_freq=s["inv_freq"],
                        layout=layout, mscale=s["mscale"], k_scale=s["ks"], v_scale=s["vs"], q_out=s["q_out"])
    if c["fmt"] == "bf16":
        return [q, s["kc"], s["vc"]]
    return [q, _values(s["kc"], s["ks"], s["kv_values"][0]), _values(s["vc"], s["vs"], s["kv_values"][1])]


def _own_attend(M, s):
    c = s["case"]
    return list(M.mnw_attn_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], c["blk"], c["d"] ** -0.5,
                                 k_scale=s["ks"], v_scale=s["vs"], want_lse=True))


def _quantise(x):
    """INT8 codes and FP32 scales of rows (last dimension) of float32 values."""
    scale = x.abs().amax(-1) / 127.0
    codes = torch.where(scale[..., None] > 0, torch.round(x / scale[..., None]), torch.zeros_like(x))
    return codes.clamp(-127, 127).to(torch.int8), scale


def _plain_norm(s):
    c = s["case"]
    r = s["x"].float()
    got = []
    if s["r"] is not None:
        rounded = (r + s["r"].float()).bfloat16()
        got, r = [rounded], rounded.float()
    y = (r * torch.rsqrt(r.square().mean(-1, keepdim=True) + NORM_EPS) * s["w"].float()).bfloat16()
    got = [y] + got
    if c["out"] == "int8":
        codes, scales = _quantise(y.float().view(c["T"], c["H"] // 128, 128))
        got.append(_values(codes, scales, s["values"]))
    return got


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
    cos = (angle.cos() * s["mscale"]).float()[:, None]
    sin = (angle.sin() * s["mscale"]).float()[:, None]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, rot, c["layout"]))
    k = _rotate(s["k"], cos, sin, rot, c["layout"])
    seq = torch.arange(B, device=pos.device).repeat_interleave(n)
    pages, slots = s["table"][seq, pos // page].long(), pos % page
    if c["fmt"] == "bf16":
        s["kc"][pages, :, slots] = k
        s["vc"][pages, :, slots] = s["v"]
        return [s["q_out"], s["kc"], s["vc"]]
    s["kc"][pages, :, slots], s["ks"][pages, :, slots] = _quantise(k.float())
    s["vc"][pages, :, slots], s["vs"][pages, :, slots] = _quantise(s["v"].float())
    return [s["q_out"], _values(s["kc"], s["ks"], s["kv_values"][0]), _values(s["vc"], s["vs"], s["kv_values"][1])]


def _dense(cache, scale, table):
    """Every sequence's cached rows one after another: [B, Hkv, keys, d] float32."""
    x = cache[table.long()].float()
    if scale is not None:
        x *= scale[table.long()].unsqueeze(-1)
    return x.transpose(1, 2).flatten(2, 3)


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


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, s)


def _exact_int8(v):
    """The values that INT8 codes of each row stand for, at one scale a row."""
    step = v.abs().max(dim=-1, keepdim=True).values / 127
    return torch.round(v / step.clamp_min(1e-300)).clamp(-127, 127) * step


def _exact_norm(c, s):
    def rows(lo, hi):
        z = s["x"][lo:hi].double()
        first = None
        if s["r"] is not None:
            z = z + s["r"][lo:hi].double()
            first = z
            z = z.bfloat16().double()
        y = z / (z.pow(2).sum(dim=1, keepdim=True) / c["H"] + NORM_EPS).sqrt() * s["w"].double()
        q = _exact_int8(y.bfloat16().double().view(hi - lo, -1, 128)) if c["out"] == "int8" else None
        return y, first, q
    parts = [rows(i, min(i + 1024, c["T"])) for i in range(0, c["T"], 1024)]
    whole = [torch.cat([p[k] for p in parts]) for k in range(3) if parts[0][k] is not None]
    return whole


def _exact_append(c, s):
    n, half, page = c["n"], c["rot"] // 2, c["page"]
    freq = s["inv_freq"].double()
    int8 = c["fmt"] == "int8"
    kc, vc = s["kc"].double(), s["vc"].double()
    if int8:
        kc *= s["ks"].double()[..., None]
        vc *= s["vs"].double()[..., None]

    def turn(x, a):
        x = x.double()
        first = torch.arange(half, device=x.device) if c["layout"] == "half" else torch.arange(0, c["rot"], 2, device=x.device)
        second = first + (half if c["layout"] == "half" else 1)
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.full_like(a, s["mscale"]), a)
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y
    qs = []
    for b, L in enumerate(s["lens"].tolist()):
        rows = slice(b * n, (b + 1) * n)
        pos = torch.arange(L - n, L, device=freq.device)
        a = (pos.double()[:, None] * freq)[:, None, :]
        qs.append(turn(s["q"][rows], a))
        k, v = turn(s["k"][rows], a), s["v"][rows].double()
        if int8:
            k, v = _exact_int8(k.bfloat16().double()), _exact_int8(v)
        where = s["table"][b, pos // page].long()
        kc[where, :, pos % page] = k
        vc[where, :, pos % page] = v
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
            K = s["kc"][pages, h].double().reshape(-1, d)[:L]
            V = s["vc"][pages, h].double().reshape(-1, d)[:L]
            if s["ks"] is not None:
                K = K * s["ks"][pages, h].double().reshape(-1, 1)[:L]
                V = V * s["vs"][pages, h].double().reshape(-1, 1)[:L]
            for j in range(h * G, (h + 1) * G):
                z = s["q"][b * n:(b + 1) * n, j].double() @ K.T / math.sqrt(d)
                z[hidden] = -math.inf
                total = torch.logsumexp(z, dim=1)
                lse[b * n:(b + 1) * n, j] = total
                out[b * n:(b + 1) * n, j] = torch.exp(z - total[:, None]) @ V
    return [out, lse]
