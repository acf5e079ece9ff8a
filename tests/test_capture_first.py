"""The first call of an operator in a process may be a captured one."""
import subprocess
import sys

import pytest

PRELUDE = """
import torch, sparse_rank_linear_b200 as salr
g = torch.Generator(device="cuda").manual_seed(0)
def bf16(*shape): return (torch.randn(*shape, generator=g, device="cuda") * 0.1).bfloat16()
K, N, R, M = 512, 384, 32, {M}
X, dY, A, B = bf16(M, K), bf16(M, N), bf16(K, R), bf16(R, N)
W = bf16(N, K)
graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
def captured(call):
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    graph.replay()
    torch.cuda.synchronize()
"""
LINEAR = """
w = {weight}
D = w.decode().double()
Y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
def check():
    x, a, b = X.double(), A.double(), B.double()
    want, S = x @ D.T + x @ a @ b, x.abs() @ D.abs().T + x.abs() @ a.abs() @ b.abs()
    err = (Y.double() - want).abs()
    assert err.norm() <= 4e-3 * want.norm() and (err <= 1e-2 * S).all()
    # up to 64 tokens the sums have one order
    assert M > 64 or torch.equal(Y, salr.linear(X, w, A, B))
    assert w.sync_status() == 0
captured(lambda: salr.linear(X, w, A, B, Y=Y))
check()
salr.linear(bf16(8 * M, K), w, A, B)  # more tokens move nothing that the graph uses
X.copy_(bf16(M, K))
graph.replay()
torch.cuda.synchronize()
check()
"""
BACKWARD = """
w = {weight}
out = [torch.full_like(t, 7.0) for t in (X, A, B)]
captured(lambda: salr.linear_backward(dY, X, w, A, B, *out))
again = salr.linear_backward(dY, X, w, A, B)
assert all(torch.equal(a, b) for a, b in zip(out, again)) and w.sync_status() == 0
"""
ADAMW = """
def make():
    p = [W.clone(), A.clone()]
    return p, salr.AdamW(p, lr=1e-2, state_bits=8)
p, opt = make()
q, ref = make()
grads = [bf16(*t.shape) for t in p]
captured(lambda: opt.step(grads))
ref.step(grads)
assert all(torch.equal(a, b) and not torch.equal(a, c) for a, b, c in zip(p, q, (W, A)))
"""
Q4 = "salr.encode_q4(W, 64)"
BITMAP = "salr.encode(W, 0.5)"


@pytest.mark.gpu
@pytest.mark.parametrize("body,weight,M", [
    (LINEAR, Q4, 1), (LINEAR, Q4, 60), (LINEAR, Q4, 100), (LINEAR, Q4, 300),
    (BACKWARD, Q4, 5), (BACKWARD, BITMAP, 300), (ADAMW, "", 1),
], ids=["q4 1", "q4 60", "q4 100", "q4 300", "backward q4 5", "backward bitmap 300", "adamw"])
def test_first_call_is_captured(body, weight, M):
    run = subprocess.run([sys.executable, "-c", PRELUDE.format(M=M) + body.format(weight=weight)],
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-3000:]
