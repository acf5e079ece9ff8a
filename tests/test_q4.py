"""Weights held as 4-bit codes with group scales: refusals on the host, and on the GPU the
packing, the quantiser and the layer against 64 bits."""
import ctypes

import pytest
import torch

import oracle
import sparse_rank_linear_b200 as salr
from gpu_util import to_bits
from sparse_rank_linear_b200 import binding
from sparse_rank_linear_b200.build import build

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


# ---------------------------------------------------------------- refusals (no GPU)


def test_bad_arguments_rejected_on_host(lib):
    P = ctypes.c_void_p
    h, ok, null = P(), P(0x10000), P(0)
    out = ctypes.byref(h)
    for c, s, o, code in ((null, ok, out, 1), (ok, null, out, 1), (ok, ok, None, 1)):
        assert lib.salr_q4_pack(c, s, null, 128, 128, 64, null, o) == code
    for n, k, g in ((100, 128, 64), (128, 96, 32), (128, 64 * 513, 64), (128, 128, 16),
                    (128, 128, 256), (128, 192, 128), (128, 128, 0), (128, 128, -64)):
        assert lib.salr_q4_pack(ok, ok, null, n, k, g, null, out) == 2
        assert lib.salr_q4_encode(ok, n, k, g, 1, null, out) == 2
    assert lib.salr_q4_pack(P(0x10004), ok, null, 128, 128, 64, null, out) == 2
    assert lib.salr_q4_pack(ok, P(0x10001), null, 128, 128, 64, null, out) == 2
    assert lib.salr_q4_encode(null, 128, 128, 64, 1, null, out) == 1
    assert lib.salr_q4_encode(ok, 128, 128, 64, 1, null, None) == 1
    assert lib.salr_q4_encode(P(0x10008), 128, 128, 64, 1, null, out) == 2
    assert h.value is None


def test_python_checks():
    c = torch.zeros(128, 64, dtype=torch.uint8)
    s = torch.zeros(128, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        salr.pack_q4(c, s)
    with pytest.raises(TypeError, match="codes"):
        salr.pack_q4(c.int(), s)
    with pytest.raises(ValueError, match="CUDA"):
        salr.encode_q4(torch.zeros(128, 128, dtype=torch.bfloat16))


class Elsewhere:
    """What the checks look at, of a bf16 CUDA tensor on a given device."""
    dtype, is_cuda = torch.bfloat16, True

    def __init__(self, shape, index):
        self.shape, self.index, self.device = shape, index, f"cuda:{index}"

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index


class Square:
    def _shape(self):
        return 128, 128


def test_tensors_of_another_device_are_refused():
    X, Y, A, B = (Elsewhere(s, i) for s, i in (((4, 128), 0), ((4, 128), 1), ((128, 8), 0), ((8, 128), 0)))
    far = [Elsewhere(t.shape, 1) for t in (A, B)]
    for a, b, y, name in ((far[0], B, None, "A_cat"), (A, far[1], None, "B_cat"), (A, B, Y, "Y")):
        with pytest.raises(ValueError, match=f"{name} must be on cuda:0"):
            salr.linear(X, Square(), a, b, Y=y)
    for x, a, b, dx, name in ((Y, A, B, None, "X"), (X, far[0], B, None, "A_cat"), (X, A, far[1], None, "B_cat"),
                              (X, A, B, Y, "dX")):
        with pytest.raises(ValueError, match=f"{name} must be on cuda:0"):
            salr.linear_backward(X, x, Square(), a, b, dX=dx)


# ---------------------------------------------------------------- helpers


def make(N, K, group, zeros, seed=0):
    """Random codes, scales and zero points, and the weight they stand for in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(N, K // group, generator=g, device="cuda") * 0.01 + 0.001).bfloat16()
    s[::7] *= -1  # a scale may be negative
    z = torch.randint(0, 16, s.shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    zd = 8.0 if z is None else z.double().repeat_interleave(group, 1)
    W = (q.double() - zd) * s.double().repeat_interleave(group, 1)
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return codes, s, z, W, g


def bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def check_small(Y, X, W, A, B, group):
    """|Y - Y*| <= half a bf16 step + the fp32 sums' error.  With S the sum of |products|: 64
    columns (32, if the group is that) are at most 4 products of 16, 17 roundings each (2^-23:
    the tensor cores may truncate); their scaled sums are added one after another (2^-24
    each), K / 64 or K / 32 of them; the adapter adds 2 R / 16 products on top, its t (K / 16
    products) is kept to 2^-16, and the partial sums of a row's ranges are fewer than 64."""
    K, R = X.shape[1], 0 if A is None else A.shape[1]
    Xd = X.double()
    Y64, S = Xd @ W.t(), Xd.abs() @ W.abs().t()
    if R:
        Y64 = Y64 + (Xd @ A.double()) @ B.double()
        S = S + (Xd.abs() @ A.double().abs()) @ B.double().abs()
    n = 4 * 17 + K / min(group, 64) / 2 + 64
    tol = 2.0 ** -8 * Y64.abs() + n * 2.0 ** -23 * S
    if R:
        Sa = (Xd.abs() @ A.double().abs()) @ B.double().abs()
        tol = tol + (2.0 ** -16 + 2.0 ** -23 * (17 * (K / 16 + R / 8))) * Sa
    err = (Y.double() - Y64).abs()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3f} of the tolerance"


# ---------------------------------------------------------------- packing


SHAPES = [(128, 64, 32), (128, 64, 64), (256, 128, 128), (128, 320, 64), (384, 256, 32),
          (128, 1152, 128), (256, 4096, 64), (128, 32768, 128)]


@gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", SHAPES)
def test_pack_and_decode(N, K, group, zeros):
    codes, s, z, W, _ = make(N, K, group, zeros)
    w = salr.pack_q4(codes, s, z)
    assert torch.equal(w.decode(), W.bfloat16())  # s (q - z) is exact in fp32, rounded once
    assert w.info() == {"N": N, "K": K, "nnz": N * K,
                        "bytes": N * K // 2 + N * K // group * (3 if zeros else 2)}
    w.free()


@gpu
def test_zero_point_above_15_is_refused():
    codes, s, z, _, _ = make(128, 128, 64, True)
    z[77, 1] = 16
    with pytest.raises(salr.SalrError, match="INVALID"):
        salr.pack_q4(codes, s, z)


@gpu
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_scale_that_is_not_finite_is_refused(bad):
    codes, s, z, _, _ = make(256, 128, 32, True)
    s[200, 3] = bad
    with pytest.raises(salr.SalrError, match="INVALID"):
        salr.pack_q4(codes, s, z)


@gpu
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("N,K,group", SHAPES[:-1])
def test_encode_rounds_to_the_nearest_code(N, K, group, symmetric):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    W = bf16(g, N, K, scale=0.02)
    W[5] = 0
    W[6] = W[6].abs()
    W[7, :group] = -1.5
    got = salr.encode_q4(W, group, symmetric).decode().double()
    v = W.double().view(N, -1, group)
    if symmetric:
        s = (v.abs().amax(-1).float() / 7).bfloat16().double()
        lo, hi = -8 * s, 7 * s
        far = s
    else:
        lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
        s = ((hi - lo).float() / 15).bfloat16().double()
        # z s is within half a step of -lo, so the codes end within half a step of lo and hi
        lo, hi = lo - s / 2, hi + s / 2
        far = 1.5 * s
    d = (got.view(N, -1, group) - v).abs()
    inside = (v >= lo[..., None]) & (v <= hi[..., None])
    # half a step from the nearest code, at most one (the scale's own rounding moves the last
    # code by up to 15 * 2^-9 of a step) beyond the ends; half a bf16 step from the decode
    near = s[..., None] * 0.5 * (1 + 2.0 ** -20) + 2.0 ** -8 * v.abs() + s[..., None] * 2.0 ** -8 * 8
    assert (d <= torch.where(inside, torch.maximum(near, far[..., None] * 0.6), far[..., None])).all()
    assert not got[5].any()


@gpu
def test_encode_refuses_values_that_are_not_finite():
    for bad in (float("nan"), float("inf"), -float("inf")):
        W = torch.zeros(128, 192, dtype=torch.bfloat16, device="cuda")
        W[100, 191] = bad
        with pytest.raises(salr.SalrError, match="INVALID"):
            salr.encode_q4(W, 64)


# ---------------------------------------------------------------- the layer


@gpu
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64])
@pytest.mark.parametrize("R", [0, 8, 80, 128])
def test_linear_small_m(M, R):
    for N, K, group, zeros in ((256, 320, 64, False), (128, 1152, 128, True), (384, 4096, 32, True)):
        codes, s, z, W, g = make(N, K, group, zeros, seed=M + R)
        w = salr.pack_q4(codes, s, z)
        X = bf16(g, M, K)
        A, B = (bf16(g, K, R, scale=0.05), bf16(g, R, N, scale=0.05)) if R else (None, None)
        Y = salr.linear(X, w, A, B)
        check_small(Y, X, W, A, B, group)
        assert torch.equal(Y, salr.linear(X, w, A, B))  # bit for bit
        assert w.sync_status() == 0


@gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", SHAPES)
def test_linear_one_token_all_shapes(N, K, group, zeros):
    codes, s, z, W, g = make(N, K, group, zeros, seed=1)
    X = bf16(g, 1, K)
    check_small(salr.linear(X, salr.pack_q4(codes, s, z)), X, W, None, None, group)


@gpu
@pytest.mark.parametrize("M", [65, 128, 200, 257, 700])
@pytest.mark.parametrize("R", [0, 24])
def test_linear_through_the_dense_scratch(M, R):
    codes, s, z, W, g = make(384, 576, 64, True, seed=M)
    w = salr.pack_q4(codes, s, z)
    X = bf16(g, M, 576)
    A, B = (bf16(g, 576, R, scale=0.05), bf16(g, R, 384, scale=0.05)) if R else (None, None)
    Y = salr.linear(X, w, A, B)
    Wd = w.decode().double()  # checked above
    Xd = X.double()
    want, S = Xd @ Wd.t(), Xd.abs() @ Wd.abs().t()
    if R:
        want = want + (Xd @ A.double()) @ B.double()
        S = S + (Xd.abs() @ A.double().abs()) @ B.double().abs()
    ok, rel, worst = oracle.check_tolerance(to_bits(Y), want.cpu().numpy(), S.cpu().numpy())
    assert ok, (rel, worst)
    assert w.sync_status() == 0


@gpu
@pytest.mark.parametrize("M", [3, 20])
def test_other_tokens_and_rows_are_left_alone(M):
    # a token of Inf and NaN stays in its own row, and rows behind the last stay as they were
    codes, s, z, W, g = make(128, 512, 64, True)
    w = salr.pack_q4(codes, s, z)
    X = bf16(g, M, 512)
    A, B = bf16(g, 512, 16, scale=0.05), bf16(g, 16, 128, scale=0.05)
    full = torch.full((M + 5, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    clean = salr.linear(X, w, A, B)
    X[1, 3], X[1, 400] = float("inf"), float("nan")
    salr.linear(X, w, A, B, Y=full[:M])
    rows = [m for m in range(M) if m != 1]
    assert torch.equal(full[rows], clean[rows])
    assert torch.isnan(full[1]).all() and (full[M:] == 7).all()


@gpu
def test_infinite_activation_gives_the_formulas_infinities():
    codes, s, z, W, g = make(128, 256, 64, False)
    w = salr.pack_q4(codes, s, z)
    X = bf16(g, 1, 256)
    X[0, 77] = float("inf")
    Y = salr.linear(X, w).double()
    want = X.double() @ W.t()  # +-inf, or NaN where the weight is zero
    assert torch.equal(torch.isnan(Y), torch.isnan(want))
    assert torch.equal(torch.isposinf(Y), torch.isposinf(want))


@gpu
@pytest.mark.parametrize("N,K", [(256, 1024), (384, 512), (128, 192)])  # clusters, ranges, one range
@pytest.mark.parametrize("R", [0, 32])
def test_captured_calls_and_another_stream(N, K, R):
    codes, s, z, W, g = make(N, K, 64, True)
    w = salr.pack_q4(codes, s, z)
    A, B = (bf16(g, K, R, scale=0.05), bf16(g, R, N, scale=0.05)) if R else (None, None)
    X = bf16(g, 5, K)
    Y = torch.empty(5, N, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        salr.linear(X, w, A, B, Y=Y)
        salr.linear(X, w, A, B, Y=Y)
    for k in range(3):
        X.copy_(bf16(g, 5, K))
        graph.replay()
        torch.cuda.synchronize()
        check_small(Y, X, W, A, B, 64)
    side.wait_stream(torch.cuda.current_stream())
    Z = torch.empty_like(Y)
    salr.linear(X, w, A, B, Y=Z, stream=side)
    side.synchronize()
    assert torch.equal(Y, Z) and w.sync_status() == 0


@gpu
def test_linear_host():
    codes, s, z, W, g = make(128, 256, 64, True)
    w = salr.pack_q4(codes, s, z)
    X = bf16(g, 4, 256)
    Xh = X.cpu().pin_memory()
    Yh = torch.empty(4, 128, dtype=torch.bfloat16).pin_memory()
    salr.linear_host(Xh, w, None, None, Yh)
    torch.cuda.synchronize()
    check_small(Yh.cuda(), X, W, None, None, 64)


@gpu
def test_calls_about_the_bitmap_form_are_refused(lib):
    codes, s, z, _, g = make(128, 128, 64, False)
    w = salr.pack_q4(codes, s, z)
    W = bf16(g, 128, 128)
    for call in (w.to_bytes, w.format_view, lambda: salr.residual_adapter(W, w, 8)):
        with pytest.raises(salr.SalrError, match="UNSUPPORTED"):
            call()
    p = ctypes.c_void_p
    Y = torch.empty(1, 128, dtype=torch.bfloat16, device="cuda")
    assert lib.salr_linear_noalloc(p(W.data_ptr()), 1, w.handle, p(0), p(0), 0, p(Y.data_ptr()), p(0)) == 2


@gpu
@pytest.mark.parametrize("N,K,M,R", [(128, 512, 3, 0), (256, 4096, 3, 0), (256, 4096, 20, 16), (4096, 1024, 1, 8)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(monkeypatch, N, K, M, R):
    codes, s, z, W, g = make(N, K, 64, True)
    w = salr.pack_q4(codes, s, z)
    X = bf16(g, M, K)
    A, B = (bf16(g, K, R, scale=0.05), bf16(g, R, N, scale=0.05)) if R else (None, None)
    monkeypatch.setenv("SALR_WAIT_LIMIT_CYCLES", "400000")  # about 0.2 ms a wait
    monkeypatch.setenv("SALR_FAIL_T_WAIT", "1")
    salr.linear(X, w, A, B)
    assert w.sync_status() == binding.SALR_ERR_TIMEOUT
    monkeypatch.delenv("SALR_FAIL_T_WAIT")
    monkeypatch.delenv("SALR_WAIT_LIMIT_CYCLES")
    for _ in range(2):
        check_small(salr.linear(X, w, A, B), X, W, A, B, 64)
        assert w.sync_status() == 0


@gpu
@pytest.mark.parametrize("M", [1, 40])
def test_calls_one_behind_another_see_each_others_results(M):
    # the launches overlap at their ends: a chain through square layers must still be in order
    ws, Ws = [], []
    for i in range(3):
        codes, s, z, W, g = make(512, 512, 64, i == 1, seed=i)
        ws.append(salr.pack_q4(codes, (s.float() * 0.2).bfloat16(), z))
        Ws.append(ws[-1].decode().double())
    A, B = bf16(g, 512, 16, scale=0.05), bf16(g, 16, 512, scale=0.05)
    X = bf16(g, M, 512)
    for _ in range(20):
        H = X
        for i, w in enumerate(ws):
            H = salr.linear(H, w, A if i else None, B if i else None)
    steps, H = [], X
    for i, w in enumerate(ws):
        torch.cuda.synchronize()
        H = salr.linear(H, w, A if i else None, B if i else None)
        torch.cuda.synchronize()
        steps.append(H)
    H = X
    for i, w in enumerate(ws):
        H = salr.linear(H, w, A if i else None, B if i else None)
    assert torch.equal(H, steps[-1])
