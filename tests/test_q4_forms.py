"""Every form of a 4-bit weight (group, zero points) at every token tile of the layer, and the
forms that apply it rounded to bf16 (more than 64 tokens, the gradients), all against the
codes' own weight s (q - z) in 64 bits."""
import pytest
import torch

import sparse_rank_linear_b200 as salr
from test_q4 import bf16, check_small, make

gpu = pytest.mark.gpu
FORMS = [(group, zeros) for group in (32, 64, 128) for zeros in (False, True)]
U = 2.0 ** -8  # half a step of bf16, relative


def adapters(g, N, K, R):
    return (bf16(g, K, R, scale=0.05), bf16(g, R, N, scale=0.05)) if R else (None, None)


@gpu
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("group,zeros", FORMS)
def test_every_form_at_every_token_tile(group, zeros, M):
    for N, K, R in ((256, 1152, 40), (384, 768, 0), (640, 640, 128), (128, 128, 8)):
        codes, s, z, W, g = make(N, K, group, zeros, seed=M)
        w = salr.pack_q4(codes, s, z)
        X = bf16(g, M, K)
        A, B = adapters(g, N, K, R)
        check_small(salr.linear(X, w, A, B), X, W, A, B, group)
        assert w.sync_status() == 0


def sums(n):
    """Relative error of an fp32 reduction of n products in parts: n / 16 accumulations of 16
    (at most 17 roundings of 2^-23 in one, each at its running size), at most 64 parts."""
    return 2.0 ** -23 * (n / 16 + 17 + 64)


@gpu
@pytest.mark.parametrize("M", [65, 128, 129, 256, 300])
@pytest.mark.parametrize("R", [0, 40])
@pytest.mark.parametrize("group,zeros", FORMS)
def test_more_than_64_tokens(group, zeros, R, M):
    """The weight is rounded once to bf16 (half a step of each product), t = X A is too, and Y."""
    N, K = 384, 640
    codes, s, z, W, g = make(N, K, group, zeros, seed=M + R)
    w = salr.pack_q4(codes, s, z)
    X = bf16(g, M, K)
    A, B = adapters(g, N, K, R)
    Y = salr.linear(X, w, A, B).double()
    Xd = X.double()
    want, S = Xd @ W.t(), Xd.abs() @ W.abs().t()
    tol = (U + sums(K) * (1 + U)) * S
    if R:
        Ad, Bd = A.double(), B.double()
        t, tS = Xd @ Ad, Xd.abs() @ Ad.abs()
        want = want + t @ Bd
        et = U * t.abs() + sums(K) * (1 + U) * tS
        tol = tol + et @ Bd.abs() + sums(R) * ((1 + U) * t.abs() @ Bd.abs())
    tol = tol * (1 + U) + U * want.abs()
    err = (Y - want).abs()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3f} of the tolerance"
    # and in norm what salr.h promises of the layer: independent roundings add up as squares
    assert (err.norm() / want.norm()).item() <= 4e-3
    assert w.sync_status() == 0


@gpu
@pytest.mark.parametrize("M", [1, 65, 300])
@pytest.mark.parametrize("group,zeros", FORMS)
def test_gradients_of_the_codes_own_weight(group, zeros, M):
    """dX applies the weight rounded once to bf16; dA and dB do not see the weight."""
    N, K, R = 384, 640, 24
    codes, s, z, W, g = make(N, K, group, zeros, seed=M)
    w = salr.pack_q4(codes, s, z)
    X, dY = bf16(g, M, K), bf16(g, M, N)
    A, B = adapters(g, N, K, R)
    dX = salr.linear_backward(dY, X, w, A, B)[0].double()
    D, Ad, Bd = dY.double(), A.double(), B.double()
    u, uS = D @ Bd.t(), D.abs() @ Bd.abs().t()
    want = D @ W + u @ Ad.t()
    eu = 2.0 ** -16 * u.abs() + sums(N) * uS
    S = D.abs() @ W.abs()
    tol = U * S + eu @ Ad.abs().t() + sums(N + 256) * (1 + U) * (S + uS @ Ad.abs().t())
    tol = tol * (1 + U) + U * want.abs()
    err = (dX - want).abs()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3f} of the tolerance"
    assert (err.norm() / want.norm()).item() <= 4e-3
    assert w.sync_status() == 0


@gpu
def test_calls_on_one_weight_at_a_time_with_more_tokens():
    """Three streams over one weight, with 100, 300 and 20 tokens: each right, whatever the others do."""
    N, K, R = 1024, 768, 40
    codes, s, z, W, g = make(N, K, 64, True)
    w = salr.pack_q4(codes, s, z)
    A, B = adapters(g, N, K, R)
    Xs = [bf16(g, m, K) for m in (100, 300, 20)]
    want = [X.double() @ W.t() + (X.double() @ A.double()) @ B.double() for X in Xs]
    streams = [torch.cuda.Stream() for _ in Xs]
    torch.cuda.synchronize()
    got = [[] for _ in Xs]
    for _ in range(10):
        for k, X in enumerate(Xs):
            with torch.cuda.stream(streams[k]):
                got[k].append(salr.linear(X, w, A, B))
    torch.cuda.synchronize()
    for ys, v in zip(got, want):
        assert all((y.double() - v).norm() <= 4e-3 * v.norm() for y in ys)
    assert w.sync_status() == 0
