"""The choice of the int8 products' kernel, at both sides of its borders (CPU)."""
import pytest

from int8_plan import plan


@pytest.mark.parametrize("G,M,N,K,swiglu,want", [
    (64, 64 * 17, 4096, 7168, 0, "wide"), (64, 64 * 16, 4096, 7168, 0, "flow"),
    (1, 16, 4096, 7168, 0, "split16x16"), (1, 17, 4096, 7168, 0, "split64x16"),
    (1, 64, 4096, 7168, 0, "split64x16"), (1, 256, 4096, 7168, 0, "split64x64"),
    (1, 257, 4096, 7168, 0, "mid"), (1, 1024, 4096, 7168, 0, "mid"),
    (1, 4096, 4096, 7168, 0, "wide"), (1, 4096, 4096, 128, 0, "mid"), (1, 4096, 4096, 144, 0, "wide"),
    (1, 30, 16384, 4096, 0, "split64x64"), (1, 30, 8200, 256, 0, "split64x32"),
    (1, 30, 8192, 256, 1, "split64x64"), (1, 30, 8200, 256, 1, "mid"), (1, 30, 2048, 256, 1, "split64x16"),
    (257, 1152, 7168, 2048, 0, "flow"), (257, 1152, 2048, 7168, 1, "flow"),
    (257, 147456, 7168, 2048, 0, "wide"), (65, 28693, 1416, 7152, 1, "wide"),
    (40, 160, 1040, 256, 0, "split16x64"),
])
def test_plan(G, M, N, K, swiglu, want):
    assert plan(swiglu, 0, M, G, M, N, K) == want


def test_offsets_of_a_gathered_product_past_32_bits_go_to_the_registers():
    assert plan(0, 1, 1048700, 1, 4096, 4096, 4096) == "split64x64"
    assert plan(0, 0, 1048700, 1, 4096, 4096, 4096) == "wide"
