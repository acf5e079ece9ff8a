"""The layer's gradients (salr_linear_backward, linear_backward): refusals on the host, and
on the GPU against the formulas in 64 bits, autograd in 64 bits, and differences."""
import ctypes

import pytest
import torch

import sparse_rank_linear_b200 as salr
from sparse_rank_linear_b200 import binding
from sparse_rank_linear_b200.build import build

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


def test_unknown_handles_rejected_on_host(lib):
    P = ctypes.c_void_p
    ok, null = P(0x10000), P(0)
    for bad in (null, ok):
        assert lib.salr_linear_backward(ok, ok, 1, bad, null, null, 0, ok, null, null, null) == 1


# ---------------------------------------------------------------- helpers


def bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def setup(N, K, M, R, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = bf16(g, N, K, scale=0.05)
    w = salr.encode(W, 0.5) if kind == "bitmap" else salr.encode_q4(W, 64, kind == "q4s")
    X, dY = bf16(g, M, K), bf16(g, M, N)
    A, B = (bf16(g, K, R, scale=0.05), bf16(g, R, N, scale=0.05)) if R else (None, None)
    return w, X, dY, A, B, g


def reference(w, X, dY, A, B):
    """(value, tolerance) of dX, dA and dB.

    A tolerance is half a bf16 step of the value and the error of the fp32 sums.  With S the
    same product of magnitudes, a reduction of n values takes n / 16 accumulations of 16
    products (at most 17 roundings of 2^-23 in one, but each at its running size: n / 16 + 17
    bounds them), its parts' sums at most 64 more, and the two bf16 parts of t and u leave
    2^-16 of them."""
    W = w.decode().double()
    Xd, D = X.double(), dY.double()
    M, (N, K) = X.shape[0], W.shape

    def tol(v, S, n, extra=0.0):
        return 2.0 ** -8 * v.abs() + 2.0 ** -23 * (n / 16 + 17 + 64) * S + extra

    if A is None:
        v = D @ W
        return ((v, tol(v, D.abs() @ W.abs(), N)),)
    Ad, Bd = A.double(), B.double()
    u, t = D @ Bd.t(), Xd @ Ad
    uS, tS = D.abs() @ Bd.abs().t(), Xd.abs() @ Ad.abs()
    # error of the stored u and t
    eu = 2.0 ** -16 * u.abs() + 2.0 ** -23 * (N / 16 + 17 + 64) * uS
    et = 2.0 ** -16 * t.abs() + 2.0 ** -23 * (K / 16 + 17 + 64) * tS
    dX = D @ W + u @ Ad.t()
    dA, dB = Xd.t() @ u, t.t() @ D
    return ((dX, tol(dX, D.abs() @ W.abs() + uS @ Ad.abs().t(), N + 256, eu @ Ad.abs().t())),
            (dA, tol(dA, Xd.abs().t() @ uS, M, Xd.abs().t() @ eu)),
            (dB, tol(dB, tS.t() @ D.abs(), M, et.t() @ D.abs())))


def check(got, want):
    for name, x, (v, tol) in zip(("dX", "dA", "dB"), got, want):
        assert x.dtype == torch.bfloat16 and x.shape == v.shape
        err = (x.double() - v).abs()
        assert (err <= tol).all(), f"{name}: worst {(err / tol).max().item():.3f} of the tolerance"


# ---------------------------------------------------------------- the gradients


@gpu
@pytest.mark.parametrize("M", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("R", [0, 8, 64, 72, 128])
def test_gradients_match_formulas(M, R):
    for N, K, kind in ((128, 64, "bitmap"), (384, 320, "q4"), (256, 576, "q4s")):
        w, X, dY, A, B, _ = setup(N, K, M, R, kind, seed=M + R)
        got = salr.linear_backward(dY, X, w, A, B)
        check(got, reference(w, X, dY, A, B))
        assert R or got[1:] == (None, None)
        again = salr.linear_backward(dY, X, w, A, B)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))
        assert w.sync_status() == 0


@gpu
@pytest.mark.parametrize("N,K,M,R,kind", [
    (128, 4096, 300, 80, "bitmap"),    # one column of weight tiles, many of dX
    (8192, 64, 500, 16, "bitmap"),     # a long reduction for few tiles of dX: parts
    (4096, 4096, 2048, 96, "bitmap"),  # more tiles than CTA pairs: a last round in parts
    (1024, 8192, 1500, 128, "q4"),
    (2048, 2048, 4500, 40, "q4"),      # parts of the token reduction
    (4096, 1472, 8100, 72, "q4"),      # tiles of 512 columns, the last of them short, some in parts
])
def test_gradients_of_larger_layers(N, K, M, R, kind):
    w, X, dY, A, B, _ = setup(N, K, M, R, kind, seed=5)
    check(salr.linear_backward(dY, X, w, A, B), reference(w, X, dY, A, B))
    assert w.sync_status() == 0


@gpu
def test_against_autograd_and_differences():
    w, X, dY, A, B, g = setup(256, 192, 90, 24, "bitmap")
    W = w.decode().double()
    x, a, b = (v.double().requires_grad_() for v in (X, A, B))

    def loss(x, a, b):
        return ((x @ W.t() + (x @ a) @ b) * dY.double()).sum()

    loss(x, a, b).backward()
    got = salr.linear_backward(dY, X, w, A, B)
    want = reference(w, X, dY, A, B)
    check(got, [(p.grad, tol) for p, (_, tol) in zip((x, a, b), want)])
    with torch.no_grad():
        for i, p in enumerate((x, a, b)):
            d = torch.randn(p.shape, generator=g, device="cuda", dtype=torch.float64)
            args = [x, a, b]
            h = 1e-3
            args[i] = p + h * d
            up = loss(*args)
            args[i] = p - h * d
            # the loss is linear in each argument: the difference is exact but for 64-bit sums
            slope = (up - loss(*args)) / (2 * h)
            bound = (want[i][1] * d.abs()).sum() + 1e-6 * slope.abs()
            assert ((got[i].double() * d).sum() - slope).abs() <= bound


@gpu
@pytest.mark.parametrize("needs", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1)])
def test_only_what_is_wanted(needs):
    w, X, dY, A, B, _ = setup(256, 320, 150, 32, "q4")
    full = salr.linear_backward(dY, X, w, A, B)
    got = salr.linear_backward(dY, X if needs[1] or needs[2] else None, w, A, B, needs=needs)
    for n, a, b in zip(needs, got, full):
        assert (torch.equal(a, b) if n else a is None)


@gpu
def test_rows_behind_the_last_stay_and_tokens_do_not_mix():
    M = 70
    w, X, dY, A, B, _ = setup(128, 192, M, 16, "bitmap")
    clean = salr.linear_backward(dY, X, w, A, B)[0]
    dY[9, 5] = float("nan")
    full = torch.full((M + 200, 192), 3.0, dtype=torch.bfloat16, device="cuda")
    salr.linear_backward(dY, X, w, A, B, dX=full[:M])
    rows = [m for m in range(M) if m != 9]
    assert torch.equal(full[rows], clean[rows]) and torch.isnan(full[9]).all()
    assert (full[M:] == 3).all()


@gpu
def test_captured_call_beside_an_eager_one():
    w, X, dY, A, B, g = setup(384, 256, 300, 48, "bitmap")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    out = [torch.empty_like(X), torch.empty_like(A), torch.empty_like(B)]
    with torch.cuda.graph(graph, stream=side):
        salr.linear_backward(dY, X, w, A, B, *out)
    for _ in range(2):
        X.copy_(bf16(g, *X.shape))
        dY.copy_(bf16(g, *dY.shape))
        torch.cuda.synchronize()
        graph.replay()  # on the current stream
        with torch.cuda.stream(side):  # a call of its own at the same time
            eager = salr.linear_backward(dY, X, w, A, B)
        torch.cuda.synchronize()
        check(out, reference(w, X, dY, A, B))
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    assert w.sync_status() == 0


@gpu
def test_input_that_is_not_needed_is_not_looked_at():
    w, X, dY, A, B, _ = setup(128, 192, 40, 8, "q4")
    odd = torch.empty(40 * 192 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(40, 192)
    want = salr.linear_backward(dY, X, w, A, B)[0]
    for x in (odd, X.cpu(), None):
        got = salr.linear_backward(dY, x, w, A, B, needs=(True, False, False))
        assert torch.equal(got[0], want) and got[1] is None and got[2] is None


@gpu
def test_refusals_on_device(lib):
    w, X, dY, A, B, _ = setup(128, 128, 4, 8, "q4")
    P = ctypes.c_void_p
    x, d, a, b = (P(t.data_ptr()) for t in (X, dY, A, B))
    o, null = P(torch.empty(1 << 16, device="cuda").data_ptr()), P(0)

    def call(dy=d, xx=x, M=4, aa=a, bb=b, R=8, dx=o, da=null, db=null):
        return lib.salr_linear_backward(dy, xx, M, w.handle, aa, bb, R, dx, da, db, null)

    assert call(dy=null) == 1 and call(M=0) == 1 and call(R=-8) == 1 and call(dx=null) == 1
    assert call(R=0, da=o) == 1 and call(aa=null) == 1 and call(bb=null) == 1
    assert call(xx=null, da=o) == 1 and call(xx=null, db=o) == 1
    assert call(R=4) == 2 and call(R=136) == 2 and call(M=(1 << 24) + 1) == 2
    assert call(dx=P(o.value + 8)) == 2 and call(dy=P(d.value + 2)) == 2
    with pytest.raises(ValueError, match="no gradient"):
        salr.linear_backward(dY, X, w, A, B, needs=(False, False, False))
    with pytest.raises(ValueError, match="X is needed"):
        salr.linear_backward(dY, None, w, A, B)
    with pytest.raises(ValueError, match="columns"):
        salr.linear_backward(dY[:, :64].contiguous(), X, w, A, B)
    with pytest.raises(ValueError, match="shape"):
        salr.linear_backward(dY, X[:3], w, A, B)


@gpu
def test_training_steps_of_the_adapters():
    """Forward, gradients and AdamW together, as a training loop uses them: two layers, a
    bitmap one over a 4-bit one, run; the gradients that reach the first layer's adapters
    through the second are those of autograd on the same rounded activations."""
    g = torch.Generator(device="cuda").manual_seed(0)
    w1 = salr.encode(bf16(g, 256, 128, scale=0.05), 0.5)
    w2 = salr.encode_q4(bf16(g, 128, 256, scale=0.05), 64)
    ads = [bf16(g, *s, scale=0.1) for s in ((128, 16), (16, 256), (256, 16), (16, 128))]
    X, target = bf16(g, 200, 128), bf16(g, 200, 128)
    opt = salr.AdamW(ads, lr=1e-3, state_bits=8, master=True)
    for _ in range(3):
        H = salr.linear(X, w1, ads[0], ads[1])
        Y = salr.linear(H, w2, ads[2], ads[3])
        dY = ((Y.float() - target.float()) / Y.numel() * 100).bfloat16()
        dH, dA2, dB2 = salr.linear_backward(dY, H, w2, ads[2], ads[3])
        _, dA1, dB1 = salr.linear_backward(dH, X, w1, ads[0], ads[1], needs=(False, True, True))
        check((dH, dA2, dB2), reference(w2, H, dY, ads[2], ads[3]))
        check((dA1, dB1), reference(w1, X, dH, ads[0], ads[1])[1:])
        before = [a.clone() for a in ads]
        opt.step([dA1, dB1, dA2, dB2])
        assert all(not torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(ads, before))
    assert opt.step_count.item() == 3


@gpu
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(monkeypatch):
    w, X, dY, A, B, _ = setup(384, 320, 150, 24, "bitmap")
    monkeypatch.setenv("SALR_WAIT_LIMIT_CYCLES", "400000")  # about 0.2 ms a wait
    monkeypatch.setenv("SALR_FAIL_T_WAIT", "1")
    for needs in ((True, False, False), (False, True, True)):
        salr.linear_backward(dY, X, w, A, B, needs=needs)
        assert w.sync_status() == binding.SALR_ERR_TIMEOUT
    monkeypatch.delenv("SALR_FAIL_T_WAIT")
    monkeypatch.delenv("SALR_WAIT_LIMIT_CYCLES")
    for _ in range(2):
        check(salr.linear_backward(dY, X, w, A, B), reference(w, X, dY, A, B))
        assert w.sync_status() == 0


@gpu
def test_two_calls_on_one_handle_at_a_time():
    # the scratch is the call's own: calls on two streams do not disturb each other
    w, X, dY, A, B, g = setup(1024, 768, 600, 32, "q4")
    other = bf16(g, *dY.shape)
    want = [salr.linear_backward(d, X, w, A, B) for d in (dY, other)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for k, d in enumerate((dY, other)):
            with torch.cuda.stream(streams[k]):
                got[k] = salr.linear_backward(d, X, w, A, B)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
