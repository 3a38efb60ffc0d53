"""The largest sizes that the conversions of 4-bit weights take: a launch holds fewer than
2^32 threads, a wave makes four tiles and a workgroup has four waves, so a launch holds
2^26 - 4 fours of tiles."""
import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")

A = 4096          # an aligned address that no call here may read
NOT, BAD = lib.ERR_UNSUPPORTED, lib.ERR_INVALID_ARG
# matrices x fours of tiles along N (one along K)
PAST = {1: (8193, 8191), 2: (37262, 1801)}    # by how many they miss 2^26
LAST = (16380, 4097)                          # 2^26 - 4


def calls(mats, nt, src):
    q = [getattr(lib._lib, f"moelora_{n}_weights_fp4") for n in ("quantize", "dequantize", "pack")]
    return [q[0](mats, nt * 16, 1, lib.BF16, src, A, A, 0), q[1](mats, nt * 16, 1, lib.BF16, A, A, src, 0),
            q[2](mats, nt * 16, 1, src, A, A, A, 0)]


@pytest.mark.parametrize("short", list(PAST))
def test_more_tiles_than_a_launch_holds_are_refused(short):
    mats, nt = PAST[short]
    assert mats * nt == 2 ** 26 - short
    assert calls(mats, nt, A) == [NOT] * 3


def test_as_many_tiles_as_a_launch_holds_are_not_refused():
    """(They get as far as the missing pointer.)"""
    assert LAST[0] * LAST[1] == 2 ** 26 - 4
    assert calls(*LAST, None) == [BAD] * 3


@pytest.mark.gpu
def test_as_many_tiles_as_a_launch_holds():
    """Values of four bits come back as they were, to the last row of the last matrix."""
    mats, N = LAST[0], LAST[1] * 16
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    print(f"[fp4] weights {mats} x {N} x 1", flush=True)
    # 6 times a power of two: the scale is that power, the code 7
    w = torch.full((mats, N, 1), 6.0, dtype=torch.bfloat16, device="cuda")
    w[-1] *= 4
    w[:, -1] = -0.75
    codes = torch.empty(mats * LAST[1] * 1024, dtype=torch.uint8, device="cuda")
    scales = torch.empty(mats * LAST[1] * 256, dtype=torch.uint8, device="cuda")
    lib.moelora_quantize_weights_fp4(mats, N, 1, lib.BF16, w, codes, scales)
    back = torch.zeros_like(w)
    lib.moelora_dequantize_weights_fp4(mats, N, 1, lib.BF16, codes, scales, back)
    assert torch.equal(back, w)
