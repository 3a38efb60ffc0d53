"""The workspace of moelora_dispatch: a size asked for once serves every
smaller batch."""
import numpy as np
import pytest
import torch

lib = pytest.importorskip("lora_expert_gemm_amd")


def test_size_for_the_largest_batch_serves_smaller_ones():
    for E in (1, 7, 32, 128, 129, 600, 1024):
        for k in (1, 3, 8):
            tokens = sorted({max(1, r // k + d) for r in (
                1, 2800, 2801, 16384, 16385, 20000, 65536, 65537, 76800, 76801, 100_000, 131_072, 131_073, 140_000,
                196_608, 196_609, 262_144, 262_145, 1 << 20, 3_000_000, 1 << 24) for d in (-1, 0, 1)
                if 1 <= (r // k + d) * k <= 1 << 24})
            sizes = [lib.moelora_dispatch_workspace(t, E, k) for t in tokens]
            assert sizes == sorted(sizes), (E, k, list(zip(tokens, sizes)))
            assert sizes[-1] <= 1024 * E


@pytest.mark.gpu
@pytest.mark.parametrize("E", [32, 1024])
def test_one_workspace_for_all_batches(E):
    """Sized once for 300000 rows, used down to the smallest."""
    k, most = 3, 100_000
    n = lib.moelora_dispatch_workspace(most, E, k)
    # (guard bytes behind it: nobody writes past what was asked for)
    ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    for T in (most, 65_537, 65_536, 43_691, 43_690, 21_846, 21_845, 5000, 1):
        print(f"[order] one workspace: E={E} T={T}", flush=True)
        ids = rng.integers(-1, E, (T, k)).astype(np.int32)
        d = dict(dtype=torch.int32, device="cuda")
        start, rows, pos = torch.zeros(E + 1, **d), torch.zeros(T * k, **d), torch.zeros(T, k, **d)
        lib.moelora_dispatch(T, 8, E, k, lib.F32, None, torch.from_numpy(ids).cuda(), start, rows, pos, None,
                             ws, n)
        flat = ids.reshape(-1)
        key = np.where(flat >= 0, flat, E)
        order, kept = np.argsort(key, kind="stable"), int((flat >= 0).sum())
        assert np.array_equal(start.cpu().numpy(), np.searchsorted(key[order], np.arange(E + 1)))
        assert np.array_equal(rows.cpu().numpy()[:kept], order[:kept])
        assert bool((rows[kept:] == T * k).all())
    assert bool((ws[n:] == 0xA5).all())
