"""The norm's INT8 groups as the operand of the W8A8 / W4A8 GEMMs: gathered by
the permutation, they give what the norm's BF16 rows quantised there give."""
import pytest
import torch

import synth as S

pytestmark = pytest.mark.gpu


def M():
    import quantized_moe_expert_routed_gb300 as m
    return m


@pytest.mark.parametrize("wfmt,fn", [(S.FMT_INT8_G128, "mnw_moe_grouped_gemm_w8a8"),
                                     (S.FMT_INT4_G128, "mnw_moe_grouped_gemm_w4a8")])
def test_codes_gathered_by_expert_feed_the_gemm(wfmt, fn):
    m = M()
    T, E, H, I, k = 37, 8, 512, 256, 3
    blob, header, _ = S.expert_blob(wfmt, E, H, I, 11, device="cuda")
    layer = m.Layer(blob, header)
    g = torch.Generator().manual_seed(4)
    x, r = (torch.randn((T, H), generator=g).bfloat16().cuda() for _ in range(2))
    w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    y, _, codes, scales = m.mnw_rmsnorm(x, w, residual=r, int8=True)
    offsets, order, _, _ = m.mnw_moe_permute(ids, E)
    want_q, want_s = m.mnw_moe_quantize_act(m.ACT_INT8_G128, y, row_index=order, index_div=k)
    rows = (order // k).long()
    assert torch.equal(codes[rows], want_q) and torch.equal(scales[rows], want_s)
    got = getattr(m, fn)(layer, m.KIND_GATE_UP, codes[rows], scales[rows], offsets)
    assert torch.equal(got, getattr(m, fn)(layer, m.KIND_GATE_UP, want_q, want_s, offsets))


@pytest.mark.parametrize("T,H", [(1, 128), (33, 2048), (3000, 1152)])
def test_codes_without_the_rows(T, H):
    m = M()
    g = torch.Generator().manual_seed(5)
    x, r = (torch.randn((T, H), generator=g).bfloat16().cuda() for _ in range(2))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    _, ro, codes, scales = m.mnw_rmsnorm(x, w, residual=r, int8=True)
    y, ro2, codes2, scales2 = m.mnw_rmsnorm(x, w, residual=r, int8=True, want_y=False)
    assert y is None
    assert torch.equal(ro, ro2) and torch.equal(codes, codes2) and torch.equal(scales, scales2)
    with pytest.raises(m.MnwError):
        m.mnw_rmsnorm(x, w, want_y=False)  # nothing to write
