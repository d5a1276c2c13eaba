"""Paths of sga_linear_grad that only certain sizes take, against a plain
implementation in 64 bits (tolerances: tests/test_linear.py): grad_x as a few-row
launch of its own, whose weight tiles have the summed dimension strided, and two
products in one launch with more tiles of grad_x than CTA pairs.  The forms named
beside the sizes are those of a GPU with 152 SMs."""
import pytest
import torch

from test_linear import ACTS, act64, check, mat, sum_tol

# (M, N, K): rows of x at once, parts of the sum over N, ring
FEW_ROWS = [
    (1, 9000, 520),      # 16, 8 parts, narrow
    (5, 9001, 520),      # 16, 8, narrow; N not a multiple of the 64-deep blocks
    (16, 20000, 512),    # 16, 8, wide
    (18, 4695, 88),      # 32, 4, wide; a part of a tile in K
    (20, 9001, 520),     # 32, 8, wide
    (40, 8100, 504),     # 64, 8, wide
    (35, 4881, 72),      # 64, 4, wide
    (100, 20003, 512),   # 128, 8, wide
    (134, 5804, 936),    # two blocks of 128, 8, narrow
    (250, 9999, 520),    # two blocks of 128, the second with 122 rows, wide
    (256, 8000, 512),    # the example draft head's size
    (700, 9000, 136),    # six blocks, the last of 60 rows
    (2000, 9000, 136),   # 16 blocks, 4 parts
]

# tiles of grad_x a pair of CTAs has at least; pairs with one more; tiles of grad_weight
# of these pairs and of the others, at most
TWO_PRODUCTS = [
    (2560, 700, 2568),   # 1; 34; 0 and 1
    (2600, 1300, 2600),  # 1; 45; 1 and 1
    (3800, 1100, 2064),  # 1; 59; 1 and 0
    (4100, 1000, 2600),  # 2; 35; 1 and 1
    (1000, 3001, 2504),  # 0; 40; 1 and 3
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", FEW_ROWS + TWO_PRODUCTS, ids=str)
def test_gradient_of_every_form(sga_lib, shape):
    M, N, K = shape
    i = (FEW_ROWS + TWO_PRODUCTS).index(shape)
    act = ACTS[i % 5]
    x, x64 = mat(i + 1, M, K, 1.0, (0, 8)[i % 2])
    w, w64 = mat(i + 101, N, K, K ** -0.5, (24, 0)[i % 2])
    g, g64 = mat(i + 201, M, N, 1.0, (1, 0, 8)[i % 3])
    z, z64 = mat(i + 301, M, N, 1.5, (0, 5)[i % 2])
    dz = g64 * act64(z64, act)[1]
    ws = torch.full((sga_lib.sga_linear_grad_workspace(M, N, K),), 255, dtype=torch.uint8,
                    device="cuda")
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    gb = torch.empty(N, device="cuda")
    z = None if act == "none" else z
    sga_lib.sga_linear_grad(g, x, w, ws, ACTS.index(act), z, gx, gw, gb)
    round_dz = 2.0 ** -8 + 2.0 ** -18
    for got, exp, size, k, name in (
            (gx, dz @ w64, dz.abs() @ w64.abs(), N, "grad_x"),
            (gw, dz.T @ x64, dz.abs().T @ x64.abs(), M, "grad_weight")):
        check(got, exp, sum_tol(k, size) + round_dz * size + 2.0 ** -8 * exp.abs() + 1e-30, name)
        rel = (got.double().cpu() - exp).norm() / exp.norm()
        assert rel < 4e-3, (name, float(rel))
    check(gb, dz.sum(0), (M * 2.0 ** -24 + 2.0 ** -18) * (g64.abs() * 1.2).sum(0) + 1e-30, "bias")
    assert sga_lib.sga_device_error() == 0
    # each output alone gives the same
    one, other = torch.empty_like(gx), torch.empty_like(gw)
    sga_lib.sga_linear_grad(g, x, w, ws, ACTS.index(act), z, grad_x=one)
    sga_lib.sga_linear_grad(g, x, w, ws, ACTS.index(act), z, grad_weight=other)
    assert torch.equal(one, gx) and torch.equal(other, gw)
