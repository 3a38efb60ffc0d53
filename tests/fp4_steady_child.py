"""Child program of tests/test_gpu_fp4_steady_state.py (run under rocprofv3): every kernel that
the product on 4-bit weights can take, named, and both ways of the weights' conversions (rows of
whole lines and others), between two marker calls (hipDriverGetVersion; the program makes no
other).  One small call of another operator runs before the first marker."""
import ctypes
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import lora_expert_gemm_amd as L  # noqa: E402
from test_fp4 import sizes  # noqa: E402
from test_fp4_kernels import FLAT, ROWS, kernel  # noqa: E402

BOTH = {"short", "stream2", "split1x1", "split2x2", "tile4x2"}
ONE = {L.F32: {"tile4x1"}, L.BF16: {"stream4_once", "tile2x2", "tile4x2_once", "tile4x4", "tile4x4_regs"}}


def main():
    u8 = dict(dtype=torch.uint8, device="cuda")
    types = {L.F32: torch.float32, L.BF16: torch.bfloat16}
    calls, names = [], set()
    for name, dt, silu, rows, N, K in FLAT:
        if (dt, silu, name) in names:
            continue
        assert kernel(rows, N, K, dt, silu) == name
        names.add((dt, silu, name))
        counts = ROWS[rows]
        R, E = sum(counts), len(counts)
        c, s = (torch.zeros(n, **u8) for n in sizes(E * (1 + silu), N, K))
        x, y = torch.zeros(R, K, dtype=types[dt], device="cuda"), torch.zeros(R, N, dtype=types[dt], device="cuda")
        start = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        calls.append(lambda a=(R, N, K, E, dt, silu, x, start, c, s, y): L.moelora_fp4_gemm(*a))
    assert names == {(dt, silu, n) for dt in ONE for silu in (0, 1) for n in BOTH | ONE[dt]}
    for dt, td in types.items():
        for N, K in ((40, 640), (40, 704), (40, 700)):   # whole lines of 128 bytes, and not
            whole = K * torch.zeros(0, dtype=td).element_size() % 128 == 0
            assert whole == (K != 700)
            w = torch.zeros(N, K, dtype=td, device="cuda")
            c, s = (torch.zeros(n, **u8) for n in sizes(1, N, K))
            rc, rs = torch.zeros(N, K // 2, **u8), torch.zeros(N, (K + 31) // 32, **u8)
            calls += [lambda a=(1, N, K, dt, w, c, s): L.moelora_quantize_weights_fp4(*a),
                      lambda a=(1, N, K, rc, rs, c, s): L.moelora_pack_weights_fp4(*a),
                      lambda a=(1, N, K, dt, c, s, w): L.moelora_dequantize_weights_fp4(*a)]
    logits, ids = torch.zeros(3, 4, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    weights = torch.zeros(3, 2, device="cuda")
    hip = ctypes.CDLL("libamdhip64.so")
    ver = ctypes.c_int()
    L.moelora_route(3, 4, 2, L.F32, 0, logits, None, ids, weights)
    torch.cuda.synchronize()
    hip.hipDriverGetVersion(ctypes.byref(ver))   # marker: steady state begins
    for c in calls:
        c()
    hip.hipDriverGetVersion(ctypes.byref(ver))   # marker: steady state ends
    torch.cuda.synchronize()
    print(f"[child] {len(names)} kinds of products", flush=True)
    print(f"[child] done: {len(calls)} calls after the first", flush=True)


if __name__ == "__main__":
    main()
