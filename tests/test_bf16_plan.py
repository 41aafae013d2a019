"""The choice of the bf16 products' kernel, at both sides of its borders (CPU)."""
import pytest

from bf16_plan import plan


@pytest.mark.parametrize("mode,G,M,N,K,want", [
    ("gemm", 64, 64 * 4, 4096, 7168, "mid"), ("gemm", 64, 64 * 128, 4096, 7168, "mid"),
    ("gemm", 64, 64 * 129, 4096, 7168, "wide"), ("gemm", 1, 1, 4096, 7168, "split16x16"),
    ("gemm", 1, 16, 4096, 7168, "split16x16"), ("gemm", 1, 17, 4096, 7168, "split64x16"),
    ("gemm", 1, 256, 4096, 7168, "split64x64"), ("gemm", 1, 257, 4096, 7168, "mid"),
    ("gemm", 1, 2048, 4096, 7168, "mid"), ("gemm", 1, 2049, 4096, 7168, "wide"),
    ("gemm", 1, 30, 8200, 256, "split64x32"), ("gemm", 8, 32, 4096, 256, "mid"), ("gemm", 4, 16, 4096, 256, "split16x64"),
    ("glu", 1, 1, 2048, 7168, "split16x16"), ("glu", 257, 1152, 2048, 7168, "mid"),
    ("glu", 1, 30, 2048, 256, "split64x16"), ("glu", 1, 30, 8192, 256, "split64x64"),
    ("glu", 65, 57344, 2048, 7168, "wide"), ("gemm", 257, 147456, 7168, 2048, "wide"),
    ("dgrad", 64, 64, 4096, 7168, "mid"), ("dgrad", 1, 1024, 4096, 7168, "mid"),
    ("dgrad", 1, 2048, 4096, 7168, "wide"), ("dgrad_glu", 65, 57344, 7168, 2048, "wide"),
    ("wgrad", 65, 57344, 4096, 7168, "wide"), ("wgrad", 1, 57344, 2048, 2048, "mid"),
    ("wgrad", 8, 100, 4096, 4096, "wide"),
])
def test_plan(mode, G, M, N, K, want):
    assert plan(mode, G, M, N, K) == want


def test_offsets_of_a_gathered_product_past_32_bits_go_elsewhere():
    for mode in ("gemm", "glu", "wgrad"):
        assert plan(mode, 64, 64 * 512, 4096, 4096, True, 524100) == "wide"
        assert plan(mode, 64, 64 * 512, 4096, 4096, True, 524200) == "mid"
        assert plan(mode, 64, 64 * 512, 4096, 4096, False, 524300) == "wide"
