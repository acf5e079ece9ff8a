"""Infinities in the layer's inputs give the infinities of the formulas, also where ranks are
padded and where sums are kept in two parts.  Exact: only the pattern of infinities and NaN is
compared, on inputs whose finite sums stay far from overflow."""
import pytest
import torch

import sparse_rank_linear_b200 as salr

gpu = pytest.mark.gpu
INF = float("inf")


def pattern(x):
    """0 for finite values, 1 and 2 for the infinities, 3 for NaN."""
    return torch.isposinf(x).int() + 2 * torch.isneginf(x).int() + 3 * torch.isnan(x).int()


def product(a, b):
    """a b in 64 bits, term by term (a library product might add terms of its own)."""
    return (a.double()[:, :, None] * b.double()[None]).sum(1)


def same(got, want):
    assert torch.equal(pattern(got.double()), pattern(want))
    assert pattern(want).any()


def setup(M, R, kind, positive):
    """A layer 128 x 192 and its inputs; ``positive``: weight and adapters without sign, so that
    infinities do not meet their opposites."""
    g = torch.Generator(device="cuda").manual_seed(R)

    def bf16(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    W, A, B = bf16(128, 192), bf16(192, R), bf16(R, 128)
    if positive:
        W, A, B = W.abs() + 0.5, A.abs() + 0.5, B.abs() + 0.5
    w = salr.encode(W, 0.0) if kind == "bitmap" else salr.encode_q4(W, 64, symmetric=False)
    return w, w.decode(), bf16(M, 192), bf16(M, 128), A, B


@gpu
@pytest.mark.parametrize("R", [8, 24, 64, 72, 128])
@pytest.mark.parametrize("kind", ["bitmap", "q4"])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_gradient_of_the_result_in_dX(kind, R, sign):
    w, W, X, dY, A, B = setup(70, R, kind, True)
    dY[9, 5] = sign * INF
    dX = salr.linear_backward(dY, X, w, A, B, needs=(True, False, False))[0]
    same(dX, product(dY, W) + product(product(dY, B.t()), A.t()))


@gpu
@pytest.mark.parametrize("R", [8, 64, 72, 128])
@pytest.mark.parametrize("place", ["dY", "X"])
def test_infinite_inputs_in_dA_and_dB(R, place):
    w, W, X, dY, A, B = setup(70, R, "q4", False)
    if place == "dY":
        dY[9, 5], dY[33, 100] = INF, -INF
    else:
        X[9, 5], X[33, 100] = INF, -INF
    _, dA, dB = salr.linear_backward(dY, X, w, A, B, needs=(False, True, True))
    u, t = product(dY, B.t()), product(X, A)
    same(dA, product(X.t(), u))
    same(dB, product(t.t(), dY))


@gpu
@pytest.mark.parametrize("M", [4, 70, 300])
@pytest.mark.parametrize("R", [8, 16, 24, 40, 128])
def test_infinite_activation_over_a_4_bit_weight(M, R):
    w, W, X, _, A, B = setup(M, R, "q4", True)
    X[2, 7] = INF
    same(salr.linear(X, w, A, B), product(X, W.t()) + product(product(X, A), B))
