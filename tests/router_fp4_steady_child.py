"""Child program of tests/test_gpu_router_fp4_steady_state.py (run under
rocprofv3): the router's operators and the 4-bit weights and their product at
sizes that take each of their kernels, between two marker calls
(hipDriverGetVersion; the program makes no other).  One small call of one
operator runs before the first marker."""
import ctypes
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import lora_expert_gemm_amd as L  # noqa: E402


def main():
    i32 = dict(dtype=torch.int32, device="cuda")
    calls, names = [], set()
    for dt, td in ((L.F32, torch.float32), (L.BF16, torch.bfloat16)):
        for E in (16, 32, 64, 128, 256, 512, 1024):
            for T in (3, 3000):
                k = 2
                x = torch.zeros(T, E, dtype=td, device="cuda")
                ids, w = torch.zeros(T, k, **i32), torch.zeros(T, k, device="cuda")
                counts, sums = torch.zeros(E + 1, **i32), torch.zeros(E, device="cuda")
                loss = torch.zeros(2, device="cuda")
                n = L.moelora_balance_loss_workspace(T, E, k)
                ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
                d = torch.zeros_like(x)
                for flags in (0, L.ROUTE_SOFTMAX_ALL):
                    calls += [
                        lambda a=(T, E, k, dt, flags, x, None, ids, w): L.moelora_route(*a),
                        lambda a=(T, E, k, dt, flags, x, None, ids, w, w, counts, loss, d):
                            L.moelora_route_backward(*a)]
                calls.append(lambda a=(T, E, k, dt, x, None, ids, counts, sums, loss, ws, n):
                             L.moelora_balance_loss(*a))
        N, K = 40, 700
        v = torch.zeros(N, K, dtype=td, device="cuda")
        c = torch.zeros(3 * 6 * 1024, dtype=torch.uint8, device="cuda")
        s = torch.zeros(3 * 2 * 256, dtype=torch.uint8, device="cuda")
        rc = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
        calls += [lambda a=(1, N, K, dt, v, c, s): L.moelora_quantize_weights_fp4(*a),
                  lambda a=(1, N, K, rc, rc, c, s): L.moelora_pack_weights_fp4(*a),
                  lambda a=(1, N, K, dt, c, s, v): L.moelora_dequantize_weights_fp4(*a)]
        for silu in (0, 1):
            for R, E, N, K in ((9, 2, 300, 3), (3, 1, 300, 300), (100, 40, 1100, 300), (40, 1, 300, 300),
                               (300, 1, 4000, 300), (300, 8, 9000, 300), (300, 2, 9000, 301), (2000, 2, 9000, 300),
                               (2000, 2, 9000, 301), (500, 2, 3000, 300)):
                x = torch.zeros(R, K, dtype=td, device="cuda")
                mats, nt, kb = E * (1 + silu), -(-N // 16), -(-K // 128)
                wc = torch.zeros(mats * nt * kb * 1024, dtype=torch.uint8, device="cuda")
                ws = torch.zeros(mats * nt * -(-kb // 4) * 256, dtype=torch.uint8, device="cuda")
                y = torch.zeros(R, N, dtype=td, device="cuda")
                start = (torch.arange(E + 1, device="cuda") * R // E).int()
                names.add((dt, silu, L.moelora_fp4_gemm_info(R, N, K, E, dt, silu).split()[0]))
                calls.append(lambda a=(R, N, K, E, dt, silu, x, start, wc, ws, y): L.moelora_fp4_gemm(*a))
    hip = ctypes.CDLL("libamdhip64.so")
    ver = ctypes.c_int()
    calls[0]()
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
