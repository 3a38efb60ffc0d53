"""Elements near the ends of the types in the product on 4-bit weights.  A float32 element's
parts are its word cut into upper halves: the last is a multiple of 2^-133, the smallest bf16
step, so that an element below 2^-110, whose last bit is below that, counts as cut to such a
multiple; from 2^-110 on, and in bf16 rows always, elements count whole, also those below the
smallest normal number.  A result here is one element times one weight: three exact products of
at most 11 bits added in float32, so two roundings, each of half a step, of a value not larger than
the result (the parts have one sign): 2^-23 relative.  A bf16 result adds one rounding, 2^-8."""
import numpy as np
import pytest
import torch

from test_fp4 import DT, cu, lib, say, tiles, up, values

pytestmark = pytest.mark.gpu
F, B = lib.F32, lib.BF16
BOUND = {F: 2.0 ** -23, B: 2.0 ** -8}


def single_products(R, dtype, v, scale, K):
    """Rows with v at a place each, against all codes of one scale: results and weights."""
    c = np.tile(np.arange(16, dtype=np.uint8)[:, None], (1, 1, K)).reshape(1, 16, K)
    s = np.full((1, 16, up(K, 32) // 32), scale, np.uint8)
    x = torch.zeros(R, K, dtype=DT[dtype])
    x[torch.arange(R), torch.arange(R) * 7 % K] = v
    out = torch.zeros(R, 16, dtype=DT[dtype], device="cuda")
    tc, ts = tiles(c, s)
    lib.moelora_fp4_gemm(R, 16, K, 1, dtype, 0, x.cuda(), None, cu(tc), cu(ts), out)
    return out.double().cpu().numpy(), values(c, s)[0][:, 0]


@pytest.mark.parametrize("R,K", [(3, 300), (40, 300), (700, 130), (5000, 130), (9, 3)])
@pytest.mark.parametrize("dtype", [F, B])
def test_small_elements_of_large_weights(dtype, R, K):
    say(f"[fp4] small elements R={R} K={K} {DT[dtype]}")
    rng = np.random.default_rng(R)
    for ex in (-100, -109, -110, -111, -118, -126, -130, -133):
        v = torch.from_numpy((1 + rng.random(R)) * rng.choice([-1, 1], R) * 2.0 ** ex).to(DT[dtype])
        got, w = single_products(R, dtype, v, 227, K)
        x = v.double().numpy()
        # (rows shorter than 16 bytes are not cut into parts)
        if dtype == F and K >= 4:
            x = np.sign(x) * np.floor(np.abs(x) * 2.0 ** 133) * 2.0 ** -133
            assert ex < -110 or np.array_equal(x, v.double().numpy())
        want = x[:, None] * w
        assert (np.abs(got - want) <= BOUND[dtype] * np.abs(want)).all()


@pytest.mark.parametrize("R,K", [(3, 300), (40, 300), (700, 130)])
@pytest.mark.parametrize("dtype", [F, B])
def test_large_elements_of_small_weights(dtype, R, K):
    """Scales of 2^-127 to 2^-124: weights below the smallest normal number."""
    rng = np.random.default_rng(R)
    for scale in range(4):
        v = torch.from_numpy((1 + rng.random(R)) * 2.0 ** 100).to(DT[dtype])
        got, w = single_products(R, dtype, v, scale, K)
        want = v.double().numpy()[:, None] * w
        assert (np.abs(got - want) <= BOUND[dtype] * np.abs(want)).all()
