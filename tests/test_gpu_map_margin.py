"""The helpers' workspaces that hold tensor maps end 64 KiB behind them."""
import pytest
import torch

from tests.grouped_helpers import normals, offsets_of

pytestmark = pytest.mark.gpu
tn = pytest.importorskip("dense_gemm_tn_gb300", reason="library not built")


def test_workspaces_with_maps_go_on_behind_them(monkeypatch):
    taken = []
    workspace = tn._workspace

    def record(device, stream, n):
        taken.append(n)
        return workspace(device, stream, n)
    monkeypatch.setattr(tn, "_workspace", record)
    E, T, M, K = 3, 300, 64, 128
    off = offsets_of([100, 50, 150])
    dC, x = normals(T, M, seed=1, dtype=torch.bfloat16), normals(T, K, seed=2, dtype=torch.bfloat16)
    dA = tn.tn_grouped_grad_a(dC, x, off)
    assert taken == [tn.gemm_grouped_workspace(tn.GEMM_GROUPED_GRAD_A, E, M, K, T, dC, M, 0, x, K) + 65536]
    assert taken[0] >= E * 256 + 65536
    taken.clear()
    A = normals(E, 2 * M, K, seed=3, dtype=torch.bfloat16)
    _, P = tn.tn_gated(A, x, off, keep=True)
    tn.tn_gated_grad(A, x, P, dC, off)
    need = tn.gemm_gated_workspace(1, 0, E, M, K, T, A, K, 2 * M * K, x, K)
    assert taken == [need + 65536] and need >= E * 256
    taken.clear()
    tn.tn_gated_grad(A[0], x, P, dC)                               # (no maps)
    assert taken == [tn.gemm_gated_workspace(1, 1, 1, M, K, T, A, K, 0, x, K)]
    tn.gemm_poll_device_status()
    assert bool(torch.isfinite(dA).all())
