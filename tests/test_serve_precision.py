"""The bound of serve_precision.py holds for weights of two operands, and of
some rows does not hold for weights rounded once, nor for the first operand
alone, at the lengths and counts of rows that the GPU tests take (an emulation
on the CPU).
Queries are large, so that few keys have most of the weight: over many equal
ones the roundings level out."""
import pytest
import torch

import serve_precision as P
import serve_util as U

SIZES = [2, 16, 33, 300, 1000, 5000]


def _case(n, d, seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(m, d, generator=g).to(torch.bfloat16).double() for m in (1, n, n))
    return 4 * q[0], k, P.balanced(v)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", SIZES)
def test_two_operands_are_within_the_bound(n, d):
    for seed in range(16):
        q, k, v = _case(n, d, seed)
        U.within(P.emulated(q, k, v, d ** -0.5, "two"), *P.attend64(q, k, v, d ** -0.5), (n, seed))


@pytest.mark.parametrize("weights", ["once", "first"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", SIZES)
def test_other_weights_are_outside(n, d, weights):
    outside = 0
    for seed in range(16):
        q, k, v = _case(n, d, seed)
        out, bound = P.attend64(q, k, v, d ** -0.5)
        outside += bool(((P.emulated(q, k, v, d ** -0.5, weights).double() - out).abs() > bound).any())
    assert outside
