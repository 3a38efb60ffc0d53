"""Sizes of the buffers of 4-bit weights (no GPU needed): those of the header's layout."""
import pytest

lib = pytest.importorskip("lora_expert_gemm_amd")


@pytest.mark.parametrize("mats,N,K,codes,scales", [
    (1, 1, 1, 1024, 256),
    (1, 16, 128, 1024, 256),
    (1, 17, 129, 2 * 2 * 1024, 2 * 256),
    (3, 33, 512, 3 * 3 * 4 * 1024, 3 * 3 * 256),
    (2, 771, 2050, 2 * 49 * 17 * 1024, 2 * 49 * 5 * 256),
    (0, 5, 5, 0, 0),
])
def test_weight_bytes(mats, N, K, codes, scales):
    assert lib.fp4_weight_bytes(mats, N, K) == (codes, scales)
