"""Plain 64-bit forms of the decode step's operators, and paged caches to run them on."""
import math

import numpy as np
import torch

DEV = "cuda"


def quantise_rows(x):
    """INT8 codes and FP32 scales of rows (last dimension), each step one binary32 operation (numpy)."""
    x = np.asarray(x, np.float32)
    scale = (np.abs(x).max(-1) / np.float32(127.0)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((x / scale[..., None]).astype(np.float32))
    q = np.where(scale[..., None] > 0, np.clip(q, -127, 127), 0)
    return q.astype(np.int8), scale


class Cache:
    """A paged cache with pages handed out in random order; every slot that no sequence owns holds `stale`."""

    def __init__(self, lens, page, Hkv, d, fmt, seed, spare=3, stale=float("nan"), joint=False, shuffle=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.Hkv, self.d, self.fmt = list(lens), page, Hkv, d, fmt
        need = [-(-L // page) for L in lens]
        self.most = max(max(need), 1) + 1
        total = sum(need) + spare
        order = torch.randperm(total, generator=g) if shuffle else torch.arange(total)
        table = torch.full((len(lens), self.most), -7, dtype=torch.int32)  # entries past the length: never read
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.table_host = table
        self.table = table.to(DEV)
        self.cache_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        shape = (total, Hkv, page, d)
        self.rows = []  # per sequence (k, v) float64 [len, Hkv, d]: the values the cache stands for
        if joint:
            both = torch.empty((total, 2) + shape[1:], dtype=torch.bfloat16 if fmt == "bf16" else torch.int8)
            k, v = both[:, 0], both[:, 1]
        else:
            k = torch.empty(shape, dtype=torch.bfloat16 if fmt == "bf16" else torch.int8)
            v = torch.empty_like(k)
        if fmt == "bf16":
            k.fill_(stale)
            v.fill_(stale)
        else:
            k.fill_(55)
            v.fill_(-77)
            self.ks = torch.full(shape[:3], stale, dtype=torch.float32)
            self.vs = torch.full(shape[:3], stale, dtype=torch.float32)
        for b, L in enumerate(lens):
            pos = torch.arange(L)
            pg, sl = table[b, pos // page].long(), pos % page
            kk = torch.randn((L, Hkv, d), generator=g) * torch.linspace(0.3, 2.0, d)
            vv = torch.randn((L, Hkv, d), generator=g)
            if fmt == "bf16":
                kk, vv = kk.bfloat16(), vv.bfloat16()
                k[pg, :, sl], v[pg, :, sl] = kk, vv
                self.rows.append((kk.double(), vv.double()))
            else:
                pair = []
                for x, codes, scales in ((kk, k, self.ks), (vv, v, self.vs)):
                    x = x * torch.exp(2.0 * torch.randn((L, Hkv, 1), generator=g)) if codes is v else x
                    c, s = quantise_rows(x.numpy()) if L else (np.zeros((0, Hkv, d), np.int8), np.zeros((0, Hkv), np.float32))
                    c, s = torch.from_numpy(c), torch.from_numpy(s)
                    codes[pg, :, sl], scales[pg, :, sl] = c, s
                    pair.append(c.double() * s.double()[..., None])
                self.rows.append(tuple(pair))
        if joint:
            both = both.to(DEV)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = k.to(DEV), v.to(DEV)
        self.ks = self.ks.to(DEV) if fmt == "int8" else None
        self.vs = self.vs.to(DEV) if fmt == "int8" else None

    def kw(self):
        return {"k_scale": self.ks, "v_scale": self.vs}


def starts_of(counts):
    return [0] + list(np.cumsum(counts))


def attend_plain(q, counts, cache, blk, scale):
    """(out, lse, sum of w |v|, largest sum of |scale q k|, largest w_j |v_j| times the keys) in float64: [T, Hq, d],
    [T, Hq], [T, Hq, d], [T, Hq], [T, Hq]."""
    T, Hq, d = q.shape
    q = q.double()
    out = torch.zeros((T, Hq, d), dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    top = torch.zeros((T, Hq), dtype=torch.float64)
    peak = torch.zeros((T, Hq), dtype=torch.float64)
    G = Hq // cache.Hkv
    t = 0
    for b, n in enumerate(counts):
        k, v = cache.rows[b]
        L = cache.lens[b]
        for i in range(n):
            p = L - n + i
            end = min(L, (p // blk + 1) * blk) if p >= 0 else 0
            if end > 0:
                for h in range(Hq):
                    s = scale * (k[:end, h // G] @ q[t, h])
                    lse[t, h] = torch.logsumexp(s, 0)
                    w = torch.exp(s - lse[t, h])
                    out[t, h] = w @ v[:end, h // G]
                    mag[t, h] = w @ v[:end, h // G].abs()
                    peak[t, h] = (w * v[:end, h // G].abs().amax(1)).max() * end
                    top[t, h] = (scale * (k[:end, h // G].abs() @ q[t, h].abs())).max()
            t += 1
    return out, lse, mag, top, peak


def check_attention(out, lse, q, counts, cache, blk, scale, lost=0.0):
    """Each rounding counted once: the output's (2^-8 of the value), the probabilities' (2^-8 of each product in BF16,
    2^-11 in FP16), and the scores' FP32 sums of d products (d 2^-24 of their magnitudes, twice: numerator and sum).
    lost: share of the row's largest product below which a product may be lost."""
    ref, ref_lse, mag, top, peak = attend_plain(q.cpu(), counts, cache, blk, scale)
    got, got_lse = out.double().cpu(), lse.double().cpu()
    assert torch.isfinite(got).all()
    p_round = 2.0 ** -8 if cache.fmt == "bf16" else 2.0 ** -11
    score = 2.0 * cache.d * 2.0 ** -24 * top + 2.0 ** -18
    tol = 2.0 ** -8 * ref.abs() + (p_round + score[..., None]) * (1 + 2.0 ** -8) * mag + lost * peak[..., None] + 1e-30
    bad = ((got - ref).abs() > tol).nonzero()
    assert bad.numel() == 0, (bad[:4].tolist(), float((got - ref).abs().max()))
    empty = torch.isinf(ref_lse)
    assert (got_lse[empty] == -math.inf).all() and (got[empty] == 0).all()
    off = (got_lse - ref_lse)[~empty].abs()
    assert (off <= (score + 2.0 ** -16 + 2.0 ** -22 * ref_lse.abs())[~empty]).all(), float(off.max())


def rotate_plain(x, pos, inv_freq, rot, layout, mscale):
    """(rotated float64, |u| + |w| of each element's pair) of x [T, heads, d] at positions pos [T]."""
    x = x.double().cpu()
    a = torch.as_tensor(pos, dtype=torch.float64)[:, None] * inv_freq.double().cpu()
    c, s = (a.cos() * mscale)[:, None], (a.sin() * mscale)[:, None]
    i = torch.arange(rot // 2)
    first, second = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y, size = x.clone(), torch.zeros_like(x)
    u, w = x[..., first], x[..., second]
    y[..., first], y[..., second] = u * c - w * s, w * c + u * s
    size[..., first] = size[..., second] = (u.abs() + w.abs()) * mscale
    return y, size
