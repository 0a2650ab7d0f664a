"""Paged caches in 4 bits made on the GPU, and attention over them in 64 bits there: for caches too long for int4_util's."""
import math

import torch

LOST = 2.0 ** -30
ORDER = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of a word (byte by byte, the lower one first) that element e is


class Cache:
    """Pages in random order; slots that no sequence owns hold codes of -8 and NaN scales.  rising: the values' scales grow
    by 2^rising along a sequence.  bad: table entries of whole tiles' pages that name no page (they read as zeros)."""
    fmt = "int4"

    def __init__(self, lens, page, Hkv, d, seed, rising=0.0, bad=(), wide=0.5):
        g = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.page, self.Hkv, self.d = list(lens), page, Hkv, d
        need = [-(-L // page) for L in lens]
        total = sum(need) + 3
        order = torch.randperm(total, generator=g, device="cuda")
        self.table = torch.full((len(lens), max(max(need), 1) + 1), -7, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].int()
            at += n
        self.cache_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        shape = (total, Hkv, page)
        owned = torch.zeros((total, page), dtype=torch.bool, device="cuda")
        level = torch.zeros((total, page), device="cuda")
        for b, L in enumerate(lens):
            pg, sl = self.places(b)
            owned[pg, sl] = True
            level[pg, sl] = torch.linspace(0.0, rising, max(L, 1), device="cuda")[:L]
        pair = []
        for grow in (0.0, 1.0):
            codes = torch.randint(0, 256, shape + (d // 2,), generator=g, dtype=torch.uint8, device="cuda")
            codes *= owned[:, None, :, None]
            s = torch.exp(wide * torch.randn(shape, generator=g, device="cuda")) / 300 * torch.exp2(level * grow)[:, None]
            s = torch.where(owned[:, None], s, float("nan"))
            m = torch.randint(1, 256, shape + (4,), generator=g, dtype=torch.uint8, device="cuda")
            pair.append((codes, torch.cat([s[..., None].contiguous().view(torch.uint8), m], -1).contiguous()))
        (self.k, self.ks), (self.v, self.vs) = pair
        for b, entry, value in bad:
            self.table[b, entry] = value

    def places(self, b):
        pos = torch.arange(self.lens[b], device="cuda")
        return self.table[b, pos // self.page].long(), pos % self.page

    def kw(self):
        return {"k_scale": self.ks, "v_scale": self.vs}

    def rows(self, b, data, rec):
        """float64 [len, Hkv, d] that the cached rows stand for."""
        pg, sl = self.places(b)
        good = (pg >= 0) & (pg < data.shape[0])
        pg = torch.where(good, pg, 0)
        byte, r = data[pg, :, sl], rec[pg, :, sl]
        nibble = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
        codes = nibble.unflatten(-1, (-1, 8))[..., ORDER].flatten(-2).double() - 8
        f = r[..., :4].contiguous().view(torch.float32).double() * r[..., 4:].double()
        x = (codes.unflatten(-1, (4, -1)) * f[..., None]).flatten(-2)
        return torch.where(good[:, None, None], x, 0.0)


def units_and_runs(counts, lens, G, Hkv):
    """Key tiles of all items, and the CTAs that share them: by the kernels' tiles of query rows and keys."""
    rows = -(-sum(counts) // len(counts)) * G
    rt = 8 if rows <= 8 else 16 if rows <= 16 else 32 if rows <= 32 else 128
    tk = 128 if rt == 128 else 256
    units = sum(Hkv * -(-n * G // rt) * max(1, -(-L // tk)) for n, L in zip(counts, lens))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return units, sms * {8: 3, 16: 2, 32: 2, 128: 1}[rt]


def check(out, lse, q, counts, cache, blk, scale, lost=LOST, some=None):
    """As paged_util.check_attention (each rounding counted once), on the GPU; of all sequences, or of some."""
    t = 0
    for b, n in enumerate(counts):
        at, L = slice(t, t + n), cache.lens[b]
        t += n
        if n == 0 or (some is not None and b not in some):
            continue
        G = q.shape[1] // cache.Hkv
        K, V = cache.rows(b, cache.k, cache.ks), cache.rows(b, cache.v, cache.vs)
        p = torch.arange(L - n, L, device="cuda")
        end = torch.minimum((p // blk + 1) * blk, torch.tensor(L, device="cuda"))
        hidden = torch.arange(L, device="cuda")[None, None] >= end[:, None, None]
        for h in range(cache.Hkv):
            x = q[at, h * G:(h + 1) * G].double()  # [n, G, d]
            s = (scale * (x @ K[:, h].T)).masked_fill(hidden, -math.inf)
            ref_lse = torch.logsumexp(s, -1)
            w = torch.exp(s - ref_lse[..., None])
            ref, mag = w @ V[:, h], w @ V[:, h].abs()
            peak = (w * V[:, h].abs().amax(1)).amax(-1) * L
            top = (abs(scale) * (x.abs() @ K[:, h].abs().T)).masked_fill(hidden, 0.0).amax(-1)
            score = 2.0 * cache.d * 2.0 ** -24 * top + 2.0 ** -18
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + score[..., None]) * (1 + 2.0 ** -8) * mag + lost * peak[..., None] + 1e-30
            got, got_lse = out[at, h * G:(h + 1) * G].double(), lse[at, h * G:(h + 1) * G].double()
            assert torch.isfinite(got).all(), (b, h)
            off = (got - ref).abs()
            assert (off <= tol).all(), (b, h, (off > tol).nonzero()[:4].tolist(), float(off.max()))
            off = (got_lse - ref_lse).abs()
            assert (off <= score + 2.0 ** -16 + 2.0 ** -22 * ref_lse.abs()).all(), (b, h, float(off.max()))
