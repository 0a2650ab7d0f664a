"""Low-rank adapters beside a shared projection on the GPU against 64 bits.

Tolerance: BF16's half step of the output (2^-8 of the value); the inner sums' FP32 (a step of at most 2^-22 of the sum of
magnitudes for each of H / 16 instructions and 20 joins), the inner value's two BF16 terms (2^-16), the outer sums' FP32."""
import pytest
import torch

from test_gpu_decode_ops import M, _randn

pytestmark = pytest.mark.gpu


def plain(y, x, a, b, ids, scale, ranks):
    """(out, bound of what FP32 and the split terms may lose), float64."""
    H, R = a.shape[2], a.shape[1]
    out, size = y.double().clone(), torch.zeros_like(y, dtype=torch.float64)
    for i in sorted(set(ids.tolist())):
        if not 0 <= i < a.shape[0]:
            continue
        rows = (ids == i).nonzero().flatten()
        r = max(0, min(R, int(ranks[i]))) if ranks is not None else R
        s = float(scale[i]) if scale is not None else 1.0
        A, B, X = a[i, :r].double(), b[i, :, :r].double(), x[rows].double()
        out[rows] += s * (X @ A.T @ B.T)
        size[rows] = abs(s) * (X.abs() @ A.abs().T @ B.abs().T)
    return out, size * ((H / 16 + 20) * 2.0 ** -22 + 2.0 ** -16 + (R / 16 + 4) * 2.0 ** -22)


def check(got, y, x, a, b, ids, scale=None, ranks=None):
    ref, lost = plain(y.cuda(), x, a, b, ids, scale, ranks)
    off = (got.double() - ref).abs()
    bad = off > 2.0 ** -8 * ref.abs() + lost
    assert not bad.any(), (bad.nonzero()[:4].tolist(), float(off.max()))


def inputs(T, H, N, R, n, seed, pattern="random"):
    g = torch.Generator().manual_seed(seed)
    x, y = _randn((T, H), seed), _randn((T, N), seed + 1)
    a, b = _randn((n, R, H), seed + 2, H ** -0.5), _randn((n, N, R), seed + 3)
    if pattern == "runs":
        ids = torch.sort(torch.randint(-1, n, (T,), generator=g))[0]
    elif pattern == "none":
        ids = torch.full((T,), -1)
    elif pattern == "one":
        ids = torch.full((T,), n - 1)
    else:
        ids = torch.randint(-1, n, (T,), generator=g)
    return y, x, a, b, ids.to(torch.int32).cuda()


SHAPES = [
    # T, H, N, R, adapters, pattern
    (1, 8, 8, 8, 1, "one"), (1, 2048, 2560, 16, 8, "one"), (1, 4096, 1032, 128, 3, "one"), (1, 512, 64, 8, 2, "none"),
    (2, 64, 40, 16, 1000, "random"), (3, 1000, 264, 24, 2, "random"), (16, 512, 512, 16, 4, "random"), (33, 2056, 1000, 40, 5, "runs"),
    (64, 4096, 2048, 16, 24, "random"), (127, 256, 128, 32, 2, "one"), (128, 264, 136, 64, 1, "one"), (129, 72, 520, 72, 1, "one"),
    (200, 1024, 1280, 128, 7, "runs"), (256, 512, 256, 8, 64, "random"), (257, 520, 248, 56, 3, "random"), (700, 640, 768, 32, 12, "runs"),
    (1024, 512, 512, 16, 16, "random"), (1025, 512, 512, 64, 16, "runs"), (3000, 256, 264, 16, 1024, "random"), (2500, 1536, 1000, 64, 4, "runs"), (40000, 64, 40, 8, 5, "random"), (600, 128, 2600, 128, 3, "random"),
    # around the limits of the one kernel and of its tiles' sizes
    (303, 136, 72, 128, 2, "random"), (304, 136, 72, 72, 1, "one"), (305, 136, 72, 128, 2, "random"), (607, 72, 136, 64, 3, "runs"),
    (608, 72, 136, 40, 1, "one"), (609, 72, 136, 64, 3, "random"), (608, 72, 136, 16, 1, "one"), (609, 72, 136, 16, 1, "one"),
    (1023, 72, 136, 32, 1024, "random"), (1024, 72, 136, 128, 1024, "random"),
]


@pytest.mark.parametrize("T,H,N,R,n,pattern", SHAPES)
def test_matches_plain(T, H, N, R, n, pattern):
    y, x, a, b, ids = inputs(T, H, N, R, n, T + H, pattern)
    g = torch.Generator().manual_seed(T)
    scale = (torch.rand(n, generator=g) * 4 - 2).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = M().mnw_lora_add(y, x, a, b, ids, scale=scale, err=err)
    assert int(err.item()) == 0
    check(got, y, x, a, b, ids, scale)
    assert torch.equal(got[ids == -1], y[ids == -1])
    # the same bits in place, and again with a dirty workspace
    ws = torch.full((M().mnw_lora_workspace_size(T, H, R, n),), 255, dtype=torch.uint8, device="cuda")
    mine = y.clone()
    assert M().mnw_lora_add(mine, x, a, b, ids, scale=scale, out=mine, ws=ws) is mine
    assert torch.equal(mine, got)


@pytest.mark.parametrize("T,R", [(7, 16), (40, 32), (300, 64), (2000, 128)])
def test_ranks_and_what_lies_past_them(T, R):
    """Rows and columns past an adapter's rank hold NaN; a rank of zero adds nothing."""
    n, H, N = 6, 520, 392
    y, x, a, b, ids = inputs(T, H, N, R, n, R)
    ranks = torch.tensor([0, 1, 5, 8, R - 1, R], dtype=torch.int32)
    for i, r in enumerate(ranks.tolist()):
        a[i, r:] = float("nan")
        b[i, :, r:] = float("nan")
    got = M().mnw_lora_add(y, x, a, b, ids, ranks=ranks.cuda())
    check(got, y, x, a, b, ids, ranks=ranks)
    assert torch.equal(got[ids == 0], y[ids == 0])


@pytest.mark.parametrize("T,R,r", [(7, 16, 1), (40, 32, 3), (300, 64, 9), (2000, 24, 1), (2000, 128, 70)])
def test_infinities_stay_what_the_formula_makes_of_them(T, R, r):
    """An infinite input, and finite ones whose inner sum passes BF16 or FP32: infinite outputs where the formula has
    those, in their rows alone."""
    H, N = 264, 136
    y, x, a, b, ids = inputs(T, H, N, R, 2, 900 + T, "one")
    ids[1] = 0  # (a tile of its own)
    a, b = a.abs() + 2.0 ** -6, b.abs() + 2.0 ** -6  # terms of one sign: no infinity meets another
    ranks = torch.tensor([r, r], dtype=torch.int32, device="cuda")
    x[1, 5] = float("inf")
    x[2, 0] = float("-inf")
    x[3] = 2.0 ** 127       # passes FP32 in the sum
    got = M().mnw_lora_add(y, x, a, b, ids, None, ranks)
    assert (got[1] == float("inf")).all() and (got[2] == float("-inf")).all() and (got[3] == float("inf")).all()
    rest = torch.arange(T, device="cuda")
    rest = rest[(rest == 0) | (rest > 3)]
    check(got[rest], y[rest], x[rest], a, b, ids[rest], None, ranks)


@pytest.mark.parametrize("T", [1, 5, 130, 1500])
def test_slices_of_wider_tensors(T):
    H, N, n = 512, 264, 3
    y, x, a, b, ids = inputs(T, H, N, 16, n, T)
    wide_x, wide_y = _randn((T, H + 64), 1), _randn((T, N + 80), 2)
    wide_x[:, 24:24 + H], wide_y[:, 40:40 + N] = x, y
    before = wide_y.clone()
    out = torch.full((T, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    got = M().mnw_lora_add(wide_y[:, 40:40 + N], wide_x[:, 24:24 + H], a, b, ids, out=out[:, 8:8 + N])
    want = M().mnw_lora_add(y, x, a, b, ids)
    assert torch.equal(got, want) and (out[:, :8] == 7).all() and (out[:, 8 + N:] == 7).all()
    M().mnw_lora_add(wide_y[:, 40:40 + N], wide_x[:, 24:24 + H], a, b, ids, out=wide_y[:, 40:40 + N])
    before[:, 40:40 + N] = want
    assert torch.equal(wide_y, before)


@pytest.mark.parametrize("T", [6, 1100])
def test_bad_adapters_and_ranks_are_reported(T):
    m = M()
    y, x, a, b, ids = inputs(T, 256, 128, 16, 4, 5)
    bad = ids.clone()
    bad[1], bad[T - 1], bad[3] = 4, -2, 2 ** 31 - 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = m.mnw_lora_add(y, x, a, b, bad, err=err)
    assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_ADAPTER
    plain_ids = ids.clone()
    plain_ids[1] = plain_ids[T - 1] = plain_ids[3] = -1
    assert torch.equal(got, m.mnw_lora_add(y, x, a, b, plain_ids))
    ids[:4] = torch.arange(4)
    for ranks, same in (([16, 16, 17, 16], [16] * 4), ([16, 16, 16, -3], [16, 16, 16, 0])):
        err.zero_()
        r = [torch.tensor(z, dtype=torch.int32, device="cuda") for z in (ranks, same)]
        got = m.mnw_lora_add(y, x, a, b, ids, ranks=r[0], err=err)
        assert m.mnw_moe_read_error(err) == m.DEVERR_BAD_ADAPTER
        assert torch.equal(got, m.mnw_lora_add(y, x, a, b, ids, ranks=r[1]))


def test_rows_past_32_bit_offsets():
    T, H, N = 9, 256, 512
    y, x, a, b, ids = inputs(T, H, N, 16, 2, 1)
    apart = 1 << 28  # 2^31 elements and more from the first row to the last
    pool = torch.zeros(apart * (T - 1) + H + N, dtype=torch.bfloat16, device="cuda")
    far_x = pool.as_strided((T, H), (apart, 1))
    far_y = pool.as_strided((T, N), (apart, 1), H)
    far_x.copy_(x)
    far_y.copy_(y)
    M().mnw_lora_add(far_y, far_x, a, b, ids, out=far_y)
    assert torch.equal(far_y, M().mnw_lora_add(y, x, a, b, ids))


@pytest.mark.parametrize("T", [5, 40, 600, 1500])
def test_streams_and_replayed_graphs(T):
    """Captured once on one assignment, replayed on others; two calls on two streams with a workspace each."""
    m = M()
    H, N, R, n = 512, 384, 32, 9
    y, x, a, b, ids = inputs(T, H, N, R, n, 3)
    out = torch.empty_like(y)
    ws = torch.empty(m.mnw_lora_workspace_size(T, H, R, n), dtype=torch.uint8, device="cuda")
    m.mnw_lora_add(y, x, a, b, ids, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mnw_lora_add(y, x, a, b, ids, out=out, ws=ws)
    for i in range(6):
        pattern = ("random", "runs", "none", "one")[i % 4]
        y2, x2, _, _, ids2 = inputs(T, H, N, R, n, 20 + i, pattern)
        for to, new in ((y, y2), (x, x2), (ids, ids2)):
            to.copy_(new)
        graph.replay()
        assert torch.equal(out, m.mnw_lora_add(y2, x2, a, b, ids2))
    want = out.clone()
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in side:
            got.append(m.mnw_lora_add(y, x, a, b, ids, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(z, want) for z in got)
