"""What a linear layer asks of its handle's workspace, by the form that serves it (no GPU needed)."""
from __future__ import annotations

import pytest
import torch

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def need():
    from splat_rendering_gb300 import build, pulsar
    build.build()
    return pulsar.linear_workspace


@pytest.mark.parametrize("dtype,side", [(F32, 64), (BF16, 128)])
@pytest.mark.parametrize("rows", [9, 1000, 1 << 20, 1 << 28])
def test_narrow_layers_keep_parts_only(need, dtype, side, rows):
    """At most 160 SMs' sums of dW (in 32 bits two each) and of the bias."""
    for k, n in ((1, 1), (7, 33), (side, side), (side, 5)):
        assert need(rows, k, n, dtype) <= 160 * (2 * (4 * k * n + 16) + 4 * n) * 4 + 4096


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [9, 1 << 20, 1 << 26])
def test_few_outputs_keep_parts_only(need, dtype, rows):
    """Nothing that grows with rows x inputs."""
    for k in (1, 96, 500, 2048):
        for n in (1, 4):
            assert need(rows, k, n, dtype) <= 4 * 160 * 4 * (k * n + 8) * 2 + 160 * 4 * n * k + 65536


def test_wide_layers_keep_their_operands(need):
    """Gradients of a wide layer: planes of x, W and dz, three of 16 bits in 32, one in 16."""
    M, K, N = 5000, 1000, 600
    size = M * K + N * K + M * N
    for dtype, planes in ((F32, 3), (BF16, 1)):
        assert 2 * planes * size <= need(M, K, N, dtype) <= 2 * planes * size + (64 << 20)


def test_more_rows_never_need_less(need):
    for dtype in (F32, BF16):
        for k, n in ((64, 64), (300, 3), (300, 300), (65, 700)):
            sizes = [need(rows, k, n, dtype) for rows in (16, 1 << 10, 1 << 14, 1 << 18, 1 << 22)]
            if k <= 64 or n <= 4:
                assert sizes == sorted(sizes)
