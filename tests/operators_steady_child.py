"""Child program of tests/test_gpu_operators_steady_state.py (run under
rocprofv3): every stand-alone operator at sizes that take each of its kernels,
between two marker calls (hipDriverGetVersion; the program makes no other).
One small call of one operator runs before the first marker."""
import ctypes
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import lora_expert_gemm_amd as L  # noqa: E402


def main():
    i32 = dict(dtype=torch.int32, device="cuda")
    calls = []
    for dt, td in ((L.F32, torch.float32), (L.BF16, torch.bfloat16)):
        for H in (136, 6, 5):
            for T in (8, 1500, 9000):
                k, E = 2, 8
                x, xs = torch.zeros(T, H, dtype=td, device="cuda"), torch.zeros(T * k, H, dtype=td, device="cuda")
                ids, start = torch.zeros(T, k, **i32), torch.zeros(E + 1, **i32)
                rows, pos = torch.zeros(T * k, **i32), torch.zeros(T, k, **i32)
                w, dw = torch.zeros(T, k, device="cuda"), torch.zeros(T, k, device="cuda")
                n = L.moelora_dispatch_workspace(T, E, k)
                ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
                calls += [
                    lambda a=(T, H, E, k, dt, x, ids, start, rows, pos, xs, ws, n): L.moelora_dispatch(*a),
                    lambda a=(T, H, k, dt, xs, pos, w, x): L.moelora_combine(*a),
                    lambda a=(T, H, k, dt, x, xs, pos, w, xs, dw): L.moelora_combine_backward(*a),
                    lambda a=(T, H, k, dt, xs, pos, x): L.moelora_dispatch_backward(*a)]
            c, s = torch.zeros(64, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 64, device="cuda")
            src = torch.zeros(64, H, dtype=td, device="cuda")
            calls += [lambda a=(64, H, dt, src, 64, None, 1, c, s): L.moelora_quantize_rows(*a),
                      lambda a=(1, 64, H, dt, src, c, s): L.moelora_quantize_weights(*a)]
        for silu in (0, 1):
            for R in (4, 20, 40, 200, 600, 1100, 2100):
                N = 10_000
                c, s = torch.zeros(R, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, R, device="cuda")
                wc = torch.zeros(2 * N, 128, dtype=torch.uint8, device="cuda")
                ws = torch.zeros(2 * 79, 1, device="cuda")
                y = torch.zeros(R, N, dtype=td, device="cuda")
                calls.append(lambda a=(R, N, 128, 1, dt, silu, c, s, None, wc, ws, y): L.moelora_fp8_gemm(*a))
            # eight experts, few to many rows each; short and long rows
            for R, K, N in ((4, 100, 900), (48, 100, 9000), (48, 1500, 900), (100, 300, 9000),
                            (300, 300, 9000), (700, 300, 9000), (2000, 300, 9000)):
                kb, nb = -(-K // 128), -(-N // 128)
                c, s = torch.zeros(R, kb * 128, dtype=torch.uint8, device="cuda"), torch.zeros(kb, R, device="cuda")
                wc = torch.zeros(16 * N, kb * 128, dtype=torch.uint8, device="cuda")
                ws = torch.zeros(16 * nb, kb, device="cuda")
                y = torch.zeros(R, N, dtype=td, device="cuda")
                start = (torch.arange(9, device="cuda") * R // 8).int()
                calls.append(lambda a=(R, N, K, 8, dt, silu, c, s, start, wc, ws, y): L.moelora_fp8_gemm(*a))
    hip = ctypes.CDLL("libamdhip64.so")
    ver = ctypes.c_int()
    calls[0]()
    torch.cuda.synchronize()
    hip.hipDriverGetVersion(ctypes.byref(ver))   # marker: steady state begins
    for c in calls:
        c()
    hip.hipDriverGetVersion(ctypes.byref(ver))   # marker: steady state ends
    torch.cuda.synchronize()
    print(f"[child] done: {len(calls)} calls after the first", flush=True)


if __name__ == "__main__":
    main()
