"""Plain forms of cached rows in 4 bits, and paged caches of them."""
import numpy as np
import torch

import paged_util as U

DEV = U.DEV


def pack(codes):
    """Codes (-8 .. 7) [..., d] as bytes [..., d / 2], word by word (numpy)."""
    u = (np.asarray(codes) + 8).astype(np.uint32).reshape(*codes.shape[:-1], -1, 8)
    word = sum(u[..., e] << np.uint32(4 * (e // 2) + 16 * (e % 2)) for e in range(8)).astype("<u4")
    return word.view(np.uint8).reshape(*codes.shape[:-1], codes.shape[-1] // 2)


def unpack(data):
    word = np.ascontiguousarray(data).view("<u4").astype(np.int64)
    codes = np.stack([((word >> (4 * (e // 2) + 16 * (e % 2))) & 15) - 8 for e in range(8)], -1)
    return codes.reshape(*data.shape[:-1], data.shape[-1] * 2)


def records(scale, m):
    """float32 scales [...] and multipliers [..., 4] as records uint8 [..., 8]."""
    s = np.ascontiguousarray(scale, np.float32)[..., None].view(np.uint8)
    return np.concatenate([s, np.asarray(m).astype(np.uint8)], -1)


def values(data, rec):
    """float64 values of cached rows."""
    codes = unpack(data).astype(np.float64)
    s = np.ascontiguousarray(rec[..., :4]).view("<f4")[..., 0].astype(np.float64)
    m = rec[..., 4:].astype(np.float64)
    g = codes.reshape(*codes.shape[:-1], 4, -1)
    return (g * (m * s[..., None])[..., None]).reshape(codes.shape)


def quantise(x):
    """(bytes, records) of rows of BF16 values: the rule with exact integers, a row at a time."""
    from fractions import Fraction
    x = np.asarray(x, np.float64)
    flat = x.reshape(-1, x.shape[-1])
    d = flat.shape[1]
    codes, scale, mult = np.zeros(flat.shape, np.int64), np.zeros(len(flat), np.float32), np.ones((len(flat), 4), np.int64)
    for i, row in enumerate(flat):
        if not np.isfinite(row).all():
            scale[i] = np.nan
            continue
        top = np.abs(row).max()
        if top < 2.0 ** -100:
            continue
        # the smallest value of 8 significant bits with 1785 S >= top
        e = int(np.floor(np.log2(top / 1785))) - 8
        S = next(Fraction(n) * Fraction(2) ** e2 for e2 in (e, e + 1, e + 2) for n in range(128, 256)
                 if 1785 * n * Fraction(2) ** e2 >= Fraction(top))
        scale[i] = np.float32(float(S))
        for g in range(4):
            part = row[g * d // 4:(g + 1) * d // 4]
            m = max(1, -(-Fraction(np.abs(part).max()) // (7 * S)))
            mult[i, g] = m
            codes[i, g * d // 4:(g + 1) * d // 4] = [round(Fraction(v) / (S * m)) for v in part]  # half way: to even
    return (pack(codes).reshape(*x.shape[:-1], d // 2),
            records(scale, mult).reshape(*x.shape[:-1], 8))


class Cache(U.Cache):
    """As paged_util's, in 4 bits; slots that no sequence owns hold codes of -8 and NaN scales."""

    def __init__(self, lens, page, Hkv, d, seed, joint=False, spread=2.0):
        super().__init__(lens, page, Hkv, d, "bf16", seed, shuffle=True)
        g = torch.Generator().manual_seed(seed + 1)
        self.fmt = "int4"
        total = self.k.shape[0]
        shape = (total, Hkv, page)
        # joint: keys and values side by side in one allocation
        both = torch.zeros((total, 2) + shape[1:] + (d // 2,), dtype=torch.uint8)
        k, v = (both[:, 0], both[:, 1]) if joint else (both[:, 0].contiguous(), both[:, 1].contiguous())
        stale = torch.from_numpy(records(np.full(shape, np.nan), np.full(shape + (4,), 255)))
        ks, vs = stale.clone(), stale.clone()
        self.rows = []
        for b, L in enumerate(lens):
            pos = torch.arange(L)
            pg, sl = self.table_host[b, pos // page].long(), pos % page
            pair = []
            for codes, recs, wide in ((k, ks, 0.0), (v, vs, spread)):
                c = (torch.randn((L, Hkv, d), generator=g) * 2.6).round().clamp(-8, 7).numpy().astype(np.int64)
                m = torch.randint(1, 256, (L, Hkv, 4), generator=g).numpy()
                s = torch.exp(0.3 * torch.randn((L, Hkv), generator=g) + wide * torch.randn((L, Hkv), generator=g)) / 300
                data, rec = pack(c), records(s.numpy(), m)
                codes[pg, :, sl], recs[pg, :, sl] = torch.from_numpy(data), torch.from_numpy(rec)
                pair.append(torch.from_numpy(values(data, rec)))
            self.rows.append(tuple(pair))
        if joint:
            both = both.to(DEV)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = k.to(DEV), v.to(DEV)
        self.ks, self.vs = ks.to(DEV), vs.to(DEV)
