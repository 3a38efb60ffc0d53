"""Conversions of 4-bit weights whose rows are whole lines of 128 bytes and several fours of
tiles long, full and partial ones, bit for bit."""
import pytest

from test_fp4 import B, F, test_pack as pack, test_quantize_and_back as quantize_and_back

pytestmark = pytest.mark.gpu
SIZES = [(2, 33, 640), (1, 17, 1088), (1, 16, 1024), (2, 50, 1600), (1, 5, 2112)]


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("mats,N,K", SIZES)
def test_whole_lines(mats, N, K, dtype):
    assert K > 512 and K % 64 == 0
    quantize_and_back(mats, N, K, dtype)


@pytest.mark.parametrize("mats,N,K", SIZES)
def test_packed_whole_lines(mats, N, K):
    pack(mats, N, K)
