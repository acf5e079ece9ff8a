"""Outputs that overlap what a call reads or writes are refused before anything is queued."""
import pytest
import torch

import sparse_rank_linear_b200 as salr

gpu = pytest.mark.gpu


def flat(n):
    return torch.randn(n, device="cuda").bfloat16()


@gpu
@pytest.mark.parametrize("kind", ["bitmap", "q4"])
def test_gradients_refuse_outputs_that_overlap(kind):
    N = K = 128
    M, R = 16, 8
    W = flat(N * K).view(N, K)
    w = salr.encode(W, 0.5) if kind == "bitmap" else salr.encode_q4(W, 64)
    dY, X, A, B = flat(M * N).view(M, N), flat(M * K).view(M, K), flat(K * R).view(K, R), flat(R * N).view(R, N)
    pool = flat(M * K + 64)
    first, second = pool[:M * K].view(M, K), pool[64:].view(M, K)
    small = pool[64:64 + K * R]
    kept = [t.clone() for t in (dY, X, A, B, pool)]
    for out in (dict(dX=dY), dict(dX=X), dict(dA=A), dict(dB=B), dict(dA=B.view(K, R)), dict(dB=A.view(R, N)),
                dict(dX=first, dA=small.view(K, R)), dict(dX=first, dB=small.view(R, N)),
                dict(dA=pool[:K * R].view(K, R), dB=small.view(R, N))):
        with pytest.raises(salr.SalrError, match="INVALID"):
            salr.linear_backward(dY, X, w, A, B, **out)
    with pytest.raises(salr.SalrError, match="INVALID"):  # by one row's end
        salr.linear_backward(first, X, w, dX=second, needs=(True, False, False))
    assert all(torch.equal(a, b) for a, b in zip((dY, X, A, B, pool), kept))
    # side by side, and over an X that the call does not read
    want = salr.linear_backward(dY, X, w, A, B)
    both = flat(2 * K * R)
    got = salr.linear_backward(dY, X, w, A, B, dA=both[:K * R].view(K, R), dB=both[K * R:].view(R, N))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    over = salr.linear_backward(dY, None, w, A, B, dX=X, needs=(True, False, False))[0]
    assert over.data_ptr() == X.data_ptr() and torch.equal(X, want[0])


@gpu
@pytest.mark.parametrize("M", [1, 16, 100])
@pytest.mark.parametrize("kind", ["bitmap", "q4"])
def test_layer_refuses_a_result_that_overlaps(kind, M):
    N = K = 128
    W = flat(N * K).view(N, K)
    w = salr.encode(W, 0.5) if kind == "bitmap" else salr.encode_q4(W, 64)
    A, B = flat(K * 8).view(K, 8), flat(8 * N).view(8, N)
    pool = flat((M + 1) * K)
    X = pool[:M * K].view(M, K)
    kept = [t.clone() for t in (pool, A, B)]
    with pytest.raises(salr.SalrError, match="INVALID"):
        salr.linear(X, w, A, B, Y=X)
    with pytest.raises(salr.SalrError, match="INVALID"):
        salr.linear(X, w, Y=pool[64:64 + M * K].view(M, K))
    if M == 1:
        with pytest.raises(salr.SalrError, match="INVALID"):
            salr.linear(X, w, A, B, Y=B[:1])
    assert all(torch.equal(a, b) for a, b in zip((pool, A, B), kept))
    long = flat((2 * M) * K)
    long[:M * K] = pool[:M * K]
    Y = salr.linear(long[:M * K].view(M, K), w, A, B, Y=long[M * K:].view(M, N))  # side by side
    want = X.double() @ w.decode().double().t() + (X.double() @ A.double()) @ B.double()
    assert (Y.double() - want).norm() <= 4e-3 * want.norm()
