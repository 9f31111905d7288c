"""Outputs and workspaces over what a call reads are refused before a launch, each pair of arrays on its own (no GPU needed)."""
import ctypes

import pytest

from weight_only_int4_05_b200 import _lib, build as libbuild


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return _lib.load()


def far(n):
    return [(i + 1) << 40 for i in range(n)]


def pairs(call, sizes, over, workspace):
    """Array `over` (of sizes[over] bytes) at the first and at the last 16 bytes of every other one, and each of them in its own
    last 16 bytes."""
    for i, n in enumerate(sizes):
        if i == over:
            continue
        for at in (far(len(sizes))[i], far(len(sizes))[i] + (n - 16) // 16 * 16):
            p = far(len(sizes))
            p[over] = at
            assert call([ctypes.c_void_p(v) for v in p], workspace) == 1, (i, over, at)
        p = far(len(sizes))
        p[i] = p[over] + (sizes[over] - 16) // 16 * 16
        assert call([ctypes.c_void_p(v) for v in p], workspace) == 1, (i, over)


@pytest.mark.parametrize("M,N,K", [(17, 32, 512), (64, 1000, 1040)])
def test_linear(L, M, N, K):
    need = L.w8a8_workspace_bytes(M, N, K)
    call = lambda p, ws: L.w8a8_linear(p[0], 1, p[1], p[2], p[3], M, N, K, p[4], ws, None)  # noqa: E731
    sizes = [M * K * 2, N * K, L.fp8_scale_bytes(N, K), M * N * 2, need]
    pairs(call, sizes, 3, need), pairs(call, sizes, 4, need)


@pytest.mark.parametrize("M,E,topk,K,I,N", [(4, 8, 2, 512, 256, 128), (300, 3, 3, 1040, 144, 260)])
def test_experts(L, M, E, topk, K, I, N):
    need = L.w8a8_moe_workspace_bytes(M, E, topk, K, I, N)
    def call(p, ws):
        return L.w8a8_moe(p[0], 2, p[1], p[2], p[3], p[4], p[5], p[6], p[7], M, E, topk, K, I, N, p[8], ws, None)
    sizes = [M * K * 2, M * topk * 4, M * topk * 4, E * 2 * I * K, L.fp8_scale_bytes(E * 2 * I, K), E * N * I,
             L.fp8_scale_bytes(E * N, I), M * N * 2, need]
    pairs(call, sizes, 8, need)
    for i in range(1, 7):  # y may be x (array 0)
        for at in (far(9)[i], far(9)[i] + (sizes[i] - 16) // 16 * 16):
            p = far(9)
            p[7] = at
            assert call([ctypes.c_void_p(v) for v in p], need) == 1, (i, at)
