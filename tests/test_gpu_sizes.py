"""Tensors of more rows or columns than 32 bits count are refused (their low
32 bits would pass for a small size)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16 = torch.float16
BIG = 2 ** 32 + 4


def test_sizes_beyond_32_bits():
    from bit_quantized_moe_token_amd import moeq
    mem = torch.empty(BIG, dtype=F16, device="cuda")         # 8.6 GB, never read
    tall, wide = mem.view(BIG, 1), mem.view(1, BIG)
    one = torch.zeros((1, 1, 1), dtype=F16, device="cuda")
    off = torch.tensor([0, 1], dtype=torch.int32).cuda()
    codes = mem.view(torch.int8)[:BIG]
    s = torch.ones(1, device="cuda")
    for call in (lambda: moeq.grouped_gemm(tall, one, off),
                 lambda: moeq.grouped_gemm(wide, mem.view(1, 1, BIG), off),
                 lambda: moeq.grouped_gemm(one[0], mem.view(1, BIG, 1), off),
                 lambda: moeq.grouped_gemm(one[0], one, off, pairs=torch.zeros(1, dtype=torch.int32, device="cuda"), k=BIG),
                 lambda: moeq.grouped_wgrad(wide, one[0], off),
                 lambda: moeq.grouped_wgrad(one[0], wide, off),
                 lambda: moeq.quantize_i8(tall),
                 lambda: moeq.quantize_i8(wide),
                 lambda: moeq.linear_i8(wide, codes.view(1, BIG), s),
                 lambda: moeq.gemm_i8(codes.view(1, BIG), s, codes.view(1, BIG), s),
                 lambda: moeq.block_norm(wide),
                 lambda: moeq.block_norm(tall),
                 lambda: moeq.block_norm_grad(wide, wide)):
        with pytest.raises(ValueError, match="beyond 32 bits"):
            call()
