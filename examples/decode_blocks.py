"""A small decoder that writes text in refinement blocks: the attention half
(norm, rotated append to a paged cache, attention over it) and the expert half
of the library run together, one CUDA graph per pass.

    python examples/decode_blocks.py

Each sequence's prompt is appended to its cache in one call.  Then a block of
32 tokens at a time is written: the block starts as mask tokens and is passed
through the decoder several times, each pass replacing its tokens by the
likeliest ones; the tokens of a block see each other and all earlier blocks.
A pass appends to the slots that the pass before wrote, so the cache holds the
last pass's keys and values when the next block begins.  Weights are random.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_moe_expert_routed_gb300 as M  # noqa: E402
import synth as S  # noqa: E402

BF16 = torch.bfloat16


class PagedCache:
    """INT8 keys and values of every layer in pages that the layers' tables share, handed out in order of need."""

    def __init__(self, layers, sequences, most_tokens, page, Hkv, d):
        most = -(-most_tokens // page)
        n = sequences * most
        codes = lambda: [torch.zeros((n, Hkv, page, d), dtype=torch.int8, device="cuda") for _ in range(layers)]  # noqa: E731
        scales = lambda: [torch.zeros((n, Hkv, page), device="cuda") for _ in range(layers)]  # noqa: E731
        self.k, self.v, self.k_scale, self.v_scale = codes(), codes(), scales(), scales()
        self.page, self.free = page, list(range(n))
        self.table_host = torch.full((sequences, most), -1, dtype=torch.int32)
        self.held = [0] * sequences
        self.table = self.table_host.cuda()
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.lens_host = [0] * sequences

    def grow(self, counts):
        """Room for counts[b] more tokens of each sequence b."""
        for b, n in enumerate(counts):
            self.lens_host[b] += n
            while self.held[b] * self.page < self.lens_host[b]:
                self.table_host[b, self.held[b]] = self.free.pop(0)
                self.held[b] += 1
        self.table.copy_(self.table_host)
        self.lens.copy_(torch.tensor(self.lens_host, dtype=torch.int32))


class Decoder:
    def __init__(self, layers=2, vocab=512, H=1024, I=512, E=16, k=4, Hq=8, Hkv=2, d=128, block=32, seed=1):
        self.H, self.k, self.Hq, self.Hkv, self.d, self.block, self.vocab = H, k, Hq, Hkv, d, block, vocab
        g = torch.Generator().manual_seed(seed)
        dense = lambda n, m: (torch.randn((n, m), generator=g) / m ** 0.5).to(BF16).cuda()  # noqa: E731
        gain = lambda: torch.ones(H, dtype=BF16, device="cuda")  # noqa: E731
        self.embed, self.last_gain = dense(vocab + 1, H), gain()  # the last token is the mask
        self.layers = []
        for i in range(layers):
            blob, header, _ = S.expert_blob(S.FMT_INT8_G128, E, H, I, seed + i, device="cuda")
            self.layers.append({"qkv": dense((Hq + 2 * Hkv) * d, H), "o": dense(H, Hq * d), "gain1": gain(),
                                "gain2": gain(), "router": S.router_weights(E, H, seed + i, device="cuda"),
                                "experts": M.Layer(blob, header)})
        self.inv_freq, self.mscale = M.mnw_rope_frequencies(d, base=1e6, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def attention(self, i, y, cache, q_start=None):
        """Layer i's attention of normed tokens y [T, H]: rotated queries and the heads' outputs, [T, Hq, d] each."""
        T = y.shape[0]
        qkv = (y @ self.layers[i]["qkv"].T).view(T, -1, self.d)
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], 1)
        kw = dict(k_scale=cache.k_scale[i], v_scale=cache.v_scale[i], q_start=q_start, err=self.err)
        q = M.mnw_kv_append(q, k, v, cache.k[i], cache.v[i], cache.table, cache.lens, self.inv_freq, mscale=self.mscale,
                            **kw)
        return q, M.mnw_attn_paged(q, cache.k[i], cache.v[i], cache.table, cache.lens, self.block, self.d ** -0.5, **kw)

    def forward(self, tokens, cache, q_start=None):
        """Logits [T, vocab] of new tokens [T]; their positions are the last ones of cache.lens."""
        x, residual = self.embed[tokens], None
        for i, p in enumerate(self.layers):
            if residual is None:
                residual, y = x, M.mnw_rmsnorm(x, p["gain1"])[0]
            else:
                y, residual, _, _ = M.mnw_rmsnorm(x, p["gain1"], residual=residual)
            _, o = self.attention(i, y, cache, q_start)
            x = o.view(len(tokens), -1) @ p["o"].T
            y, residual, _, _ = M.mnw_rmsnorm(x, p["gain2"], residual=residual)
            x, _, _ = M.mnw_moe_forward_routed(p["experts"], M.ACT_BF16, y, p["router"], self.k)
        y = M.mnw_rmsnorm(x, self.last_gain, residual=residual)[0]
        return y @ self.embed[:-1].T

    def check(self):
        word = M.mnw_moe_read_error(self.err)
        if word:
            raise RuntimeError(f"device error word {word:#x}")


def write(model, prompts, blocks=2, passes=4, page=64, graph=True):
    """Continues prompts (lists of tokens, whole blocks long) by `blocks` blocks; returns the new tokens [B, n]."""
    B, n = len(prompts), model.block
    assert all(len(p) % n == 0 for p in prompts)
    cache = PagedCache(len(model.layers), B, max(map(len, prompts)) + blocks * n, page, model.Hkv, model.d)
    lens = [len(p) for p in prompts]
    cache.grow(lens)
    starts = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    model.forward(torch.tensor(sum(prompts, []), device="cuda"), cache, starts)

    tokens = torch.empty(B * n, dtype=torch.int64, device="cuda")

    def one_pass():
        tokens.copy_(model.forward(tokens, cache).float().argmax(1))

    run, written = one_pass, []
    for _ in range(blocks):
        cache.grow([n] * B)
        if graph and run is one_pass:  # the pass reads table and lengths from the device, so one graph serves all blocks
            tokens.fill_(model.vocab)
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                one_pass()
            torch.cuda.current_stream().wait_stream(side)
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                one_pass()
            run = captured.replay
        tokens.fill_(model.vocab)
        for _ in range(passes):
            run()
        written.append(tokens.view(B, n).clone())
    model.check()
    return torch.cat(written, 1)


def main():
    model = Decoder()
    g = torch.Generator().manual_seed(7)
    prompts = [torch.randint(model.vocab, (n,), generator=g).tolist() for n in (96, 320, 32, 160)]
    out = write(model, prompts, blocks=8)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    out = write(model, prompts, blocks=8)
    b.record()
    b.synchronize()
    print(f"{out.numel()} tokens in {a.elapsed_time(b):.1f} ms; first of each sequence: {out[:, :8].tolist()}")


if __name__ == "__main__":
    main()
