"""The layer on a 4-bit weight where CTA ranges share row blocks and their fp32 sums meet in
memory: against 64 bits, and with several calls on one weight at a time."""
import pytest
import torch

import sparse_rank_linear_b200 as salr
from sparse_rank_linear_b200 import binding
from test_q4 import bf16, check_small, make

gpu = pytest.mark.gpu


def ranges_of_a_block(N, K, slots=280):
    """The CTA ranges that a row block is cut into at most, by the launch rule where no
    clusters are formed: short blocks (under 8 records of 128 columns), or ranges of 16
    records and more.  ``slots``: CTAs resident at once, 280 to 296 on 148 SMs."""
    records, blocks = -(-K // 128), N // 128
    total = records * blocks
    grid = max(1, min(slots, total // 4))
    assert records < 8 or total // grid >= 16, "may run as clusters"
    cut = [total * c // grid for c in range(grid + 1)]
    return max(sum(a < (b + 1) * records and z > b * records for a, z in zip(cut, cut[1:]))
               for b in range(blocks))


SHAPES = [(384, 768, 32), (640, 768, 128), (384, 704, 64), (1152, 896, 64), (512, 640, 32)]
LONG = (9600, 8192, 64)


def test_the_shapes_share_row_blocks():
    assert all(ranges_of_a_block(N, K) > 1 for N, K, _ in SHAPES)
    for slots in range(280, 297):
        assert ranges_of_a_block(*LONG[:2], slots) >= 5


def adapters(g, N, K, R):
    return (bf16(g, K, R, scale=0.05), bf16(g, R, N, scale=0.05)) if R else (None, None)


@gpu
@pytest.mark.parametrize("M", [1, 8, 9, 17, 33, 64])
@pytest.mark.parametrize("R", [0, 80])
@pytest.mark.parametrize("N,K,group", SHAPES)
def test_sums_over_ranges(N, K, group, R, M):
    for zeros in (False, True):
        codes, s, z, W, g = make(N, K, group, zeros, seed=M + R)
        w = salr.pack_q4(codes, s, z)
        X = bf16(g, M, K)
        A, B = adapters(g, N, K, R)
        full = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
        Y = salr.linear(X, w, A, B, Y=full[:M])
        check_small(Y, X, W, A, B, group)
        assert torch.equal(Y, salr.linear(X, w, A, B))  # bit for bit
        assert (full[M:] == 7).all() and w.sync_status() == 0


@gpu
@pytest.mark.parametrize("M,R", [(1, 0), (1, 80), (16, 80), (30, 0), (64, 128)])
def test_a_block_over_five_ranges(M, R):
    N, K, group = LONG
    codes, s, z, W, g = make(N, K, group, True, seed=M)
    w = salr.pack_q4(codes, s, z)
    X = bf16(g, M, K)
    A, B = adapters(g, N, K, R)
    check_small(salr.linear(X, w, A, B), X, W, A, B, group)
    assert w.sync_status() == 0


@gpu
@pytest.mark.parametrize("M,R", [(1, 0), (5, 16), (40, 80)])
def test_a_wait_that_runs_out_leaves_nothing_behind(monkeypatch, M, R):
    N, K, group = SHAPES[0]
    codes, s, z, W, g = make(N, K, group, True)
    w = salr.pack_q4(codes, s, z)
    X = bf16(g, M, K)
    A, B = adapters(g, N, K, R)
    monkeypatch.setenv("SALR_WAIT_LIMIT_CYCLES", "400000")  # about 0.2 ms a wait
    monkeypatch.setenv("SALR_FAIL_T_WAIT", "1")
    salr.linear(X, w, A, B)
    monkeypatch.delenv("SALR_FAIL_T_WAIT")
    monkeypatch.delenv("SALR_WAIT_LIMIT_CYCLES")
    Y = salr.linear(X, w, A, B)  # before the error is fetched: the calls share no state
    assert w.sync_status() == binding.SALR_ERR_TIMEOUT
    check_small(Y, X, W, A, B, group)
    check_small(salr.linear(X, w, A, B), X, W, A, B, group)
    assert w.sync_status() == 0


@gpu
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[3], LONG, (256, 1024, 64)])
@pytest.mark.parametrize("R", [0, 32])
def test_calls_on_one_weight_at_a_time(shape, R):
    """Two captured graphs, each replayed on a stream of its own, and eager calls on a third,
    all on one weight."""
    N, K, group = shape
    codes, s, z, W, g = make(N, K, group, True)
    w = salr.pack_q4(codes, s, z)
    A, B = adapters(g, N, K, R)
    streams = [torch.cuda.Stream() for _ in range(3)]
    Xs = [bf16(g, m, K) for m in (1, 6, 20)]
    want = [salr.linear(X, w, A, B) for X in Xs]
    for X, Y in zip(Xs, want):
        check_small(Y, X, W, A, B, group)
    outs = [[torch.zeros_like(Y) for _ in range(20)] for Y in want]
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k], stream=streams[k]):
            for Y in outs[k]:
                salr.linear(Xs[k], w, A, B, Y=Y)
    torch.cuda.synchronize()
    for _ in range(3):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        for Y in outs[2]:
            salr.linear(Xs[2], w, A, B, Y=Y, stream=streams[2])
        torch.cuda.synchronize()
        for ys, y in zip(outs, want):
            assert all(torch.equal(a, y) for a in ys)
            for a in ys:
                a.zero_()
        torch.cuda.synchronize()
    assert w.sync_status() == 0
