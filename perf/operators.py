"""The operators around the compressed linear layer that fine-tuning and serving need, each
in a plain torch form and as the library's own calls, with the cases they are measured on.

* ``q4``: Y = X W^T + (X A) B with W held as 4-bit codes with group scales, for 1 to 256
  tokens: the decode steps of a served model (and short prompts).
* ``backward``: the gradients of the layer Y = X W^T + (X A) B for a frozen compressed W
  (bitmap or 4-bit): dX, dA and dB, for training the adapters.
* ``adamw``: one AdamW step over all adapter tensors of a model at once, with moments held
  in 32 bits or in 8 bits (e4m3 with one scale per 256 elements).

``own`` selects the library's calls; the plain forms compute in fp32 and round once.
"""
import math
import random

import torch

own = False

BLOCK = 256  # elements that share a scale of the 8-bit moments; tensors start on multiples
E4M3_MAX = 448.0
E4M3_TINY = 2.0 ** -9  # the smallest positive e4m3 value
FLUSH = 2.0 ** -100  # blocks whose largest magnitude is below this are held as zeros

# N, K and total adapter rank of the projections the repository is configured for
SHAPES = {
    "tiny": (256, 256, 8),
    "q_proj": (4096, 4096, 80),
    "up_proj": (11008, 4096, 96),
    "down_proj": (4096, 11008, 128),
    "large": (28672, 8192, 96),
}


def _shape(name):
    N, K, R = SHAPES[name]
    return {"N": N, "K": K, "R": R}


def listed():
    return [
        # one decode step of one 4096-wide projection without adapters: latency counts
        dict(name="q4 q_proj M=1", op="q4", **{**_shape("q_proj"), "R": 0}, M=1, group=64, zeros=False),
        # a batch of 16 decoding requests, adapters unmerged, a checkpoint with zero points
        dict(name="q4 down_proj M=16", op="q4", **_shape("down_proj"), M=16, group=128, zeros=True),
        # a single token through the widest projection: the weight's bytes are the whole cost
        dict(name="q4 large M=1", op="q4", **_shape("large"), M=1, group=64, zeros=False),
        # an odd number of draft tokens to verify, fine groups
        dict(name="q4 up_proj M=37", op="q4", **_shape("up_proj"), M=37, group=32, zeros=True),
        # the smallest layer and batch
        dict(name="backward tiny M=16", op="backward", **_shape("tiny"), M=16, weight="bitmap"),
        # one sequence of a fine-tuning batch
        dict(name="backward up_proj M=2048", op="backward", **_shape("up_proj"), M=2048, weight="bitmap"),
        # a ragged batch over a 4-bit base
        dict(name="backward down_proj M=1000", op="backward", **_shape("down_proj"), M=1000, weight="q4"),
        # the largest layer and token count
        dict(name="backward large M=8192", op="backward", **_shape("large"), M=8192, weight="bitmap"),
        # the two adapter matrices of one projection
        dict(name="adamw one projection", op="adamw", layers=0, count=2, longest=4096 * 80, sizes=-1,
             param="bf16", master=True, grad="bf16", bits=32),
        # all adapters of a 32-layer model, fp32 moments and master copies
        dict(name="adamw 32 layers 32 bits", op="adamw", layers=32, count=448, longest=0, sizes=0,
             param="bf16", master=True, grad="bf16", bits=32),
        # the same with 8-bit moments and no master copies: the small-memory setting
        dict(name="adamw 32 layers 8 bits", op="adamw", layers=32, count=448, longest=0, sizes=0,
             param="bf16", master=False, grad="bf16", bits=8),
        # tensors of odd sizes in fp32 (norm weights, biases, small adapters)
        dict(name="adamw ragged fp32", op="adamw", layers=0, count=301, longest=65537, sizes=7,
             param="fp32", master=False, grad="fp32", bits=8),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("q4", "backward", "adamw"))
    if op == "adamw":
        master = rng.random() < 0.4
        return dict(op=op, layers=0, count=_log_uniform(rng, 1, 600),
                    longest=_log_uniform(rng, 1, 400000), sizes=rng.randrange(1, 1 << 30),
                    param="bf16" if master or rng.random() < 0.5 else "fp32", master=master,
                    grad=rng.choice(("bf16", "fp32")), bits=rng.choice((8, 32)))
    N = 128 * _log_uniform(rng, 1, 224)
    R = 8 * rng.randrange(0, 17)
    if op == "q4":
        return dict(op=op, N=N, K=128 * _log_uniform(rng, 1, 86), R=R, M=_log_uniform(rng, 1, 256),
                    group=rng.choice((32, 64, 128)), zeros=rng.random() < 0.5)
    weight = rng.choice(("bitmap", "q4"))
    unit = 64 if weight == "bitmap" else 128
    K = unit * _log_uniform(rng, 1, 8192 // unit)
    return dict(op=op, N=N, K=K, R=R, M=_log_uniform(rng, 1, 8192), weight=weight)


# ---------------------------------------------------------------- inputs


def _tensor_sizes(case):
    """Elements of each tensor of an adamw case."""
    if case["layers"]:
        one = []
        for name in ("q_proj",) * 4 + ("up_proj",) * 2 + ("down_proj",):
            N, K, R = SHAPES[name]
            one += [K * R, R * N]
        return one * case["layers"]
    if case["sizes"] < 0:
        return [case["longest"]] * case["count"]
    r = random.Random(case["sizes"])
    return [_log_uniform(r, 1, case["longest"]) for _ in range(case["count"])]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * scale


def _quantised(W, group, zeros):
    """Round-to-nearest 4-bit codes (N x K/2 bytes, even column in the low nibble), bf16
    scales and zero points (N x K/group) of W: what a 4-bit checkpoint holds."""
    N, K = W.shape
    w = W.view(N, K // group, group)
    if zeros:
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).bfloat16()
        z = torch.round(-lo / s.float()).clamp(0, 15)
    else:
        s = (w.abs().amax(-1) / 7).bfloat16()
        z = torch.full_like(s, 8.0, dtype=torch.float32)
    q = (torch.round(w / s.float()[..., None]) + z[..., None]).clamp(0, 15).to(torch.uint8).view(N, K)
    return q[:, 0::2] | (q[:, 1::2] << 4), s, z.to(torch.uint8) if zeros else None


def _pruned(W, sparsity=0.5):
    """W with the smallest magnitudes of each row set to zero."""
    drop = int(sparsity * W.shape[1])
    a = W.abs().float()
    return torch.where(a > a.kthvalue(drop, dim=1, keepdim=True).values, W, torch.zeros_like(W))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "adamw":
        return _prepare_adamw(s, g)
    N, K, R, M = case["N"], case["K"], case["R"], case["M"]
    W = _randn(g, N, K, scale=0.02)
    s["X"] = _randn(g, M, K).bfloat16()
    s["A"] = _randn(g, K, R, scale=0.01).bfloat16() if R else None
    s["B"] = _randn(g, R, N, scale=0.01).bfloat16() if R else None
    if case["op"] == "backward":
        s["dY"] = _randn(g, M, N).bfloat16()
    if case.get("weight") == "bitmap":
        s["W"] = _pruned(W.bfloat16())
    else:
        s["codes"], s["scales"], s["zeros"] = _quantised(W, case.get("group", 64), case.get("zeros", True))
    if own:
        import sparse_rank_linear_b200 as salr
        s["weight"] = (salr.encode(s["W"], 0.5) if "W" in s else
                       salr.pack_q4(s["codes"], s["scales"], s["zeros"]))
    return s


def _prepare_adamw(s, g):
    """Tensors as slices of flat buffers, each starting on a multiple of BLOCK elements."""
    sizes = _tensor_sizes(s)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
    used = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, sizes):
        used[a:a + n] = True
    pt = torch.bfloat16 if s["param"] == "bf16" else torch.float32
    gt = torch.bfloat16 if s["grad"] == "bf16" else torch.float32
    master = _randn(g, total, scale=0.01) * used
    s["p"] = master.to(pt)
    s["master_flat"] = master if s["master"] else None
    s["grad_flat"] = (_randn(g, total, scale=1e-3) * used).to(gt)
    m = _randn(g, total, scale=3e-4) * used
    v = (_randn(g, total, scale=1e-3) * used).square_()
    s["m_scale"] = s["r_scale"] = None
    if s["bits"] == 8:
        s["m"], s["m_scale"] = _to_e4m3(m, False)
        s["v"], s["r_scale"] = _to_e4m3(v.sqrt_(), True)
    else:
        s["m"], s["v"] = m, v
    s.update(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    s["step"] = torch.full((), 100, dtype=torch.int64, device="cuda")  # steps done so far
    s["grad_scale"] = torch.full((), 0.5, device="cuda")  # from clipping the global norm
    if own:
        import sparse_rank_linear_b200 as salr
        slices = [s["p"][a:a + n] for a, n in zip(starts, sizes)]
        s["grads"] = [s["grad_flat"][a:a + n] for a, n in zip(starts, sizes)]
        o = salr.AdamW(slices, lr=s["lr"], betas=(s["beta1"], s["beta2"]), eps=s["eps"],
                       weight_decay=s["weight_decay"], state_bits=s["bits"], master=s["master"])
        for held, given in ((o.master, "master_flat"), (o.exp_avg, "m"), (o.exp_avg_sq, "v"),
                            (o.exp_avg_scale, "m_scale"), (o.exp_avg_sq_scale, "r_scale"),
                            (o.step_count, "step")):
            if held is not None:
                held.copy_(s[given])
        s["opt"] = o
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    if s["op"] == "adamw":
        return _adamw_own(s) if own else _adamw_plain(s)
    if s["op"] == "q4":
        if own:
            import sparse_rank_linear_b200 as salr
            return salr.linear(s["X"], s["weight"], s["A"], s["B"])
        return _linear_plain(s)
    if own:
        import sparse_rank_linear_b200 as salr
        return salr.linear_backward(s["dY"], s["X"], s["weight"], s["A"], s["B"])
    return _backward_plain(s)


def _weight_plain(s):
    """The dense weight in fp32."""
    if "W" in s:
        return s["W"].float()
    c = s["codes"]
    q = torch.stack((c & 15, c >> 4), dim=-1).view(c.shape[0], s["scales"].shape[1], -1).float()
    z = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    return ((q - z) * s["scales"].float()[..., None]).view(c.shape[0], -1)


def _linear_plain(s):
    X = s["X"].float()
    Y = X @ _weight_plain(s).t()
    if s["A"] is not None:
        Y = Y + (X @ s["A"].float()) @ s["B"].float()
    return Y.bfloat16()


def _backward_plain(s):
    X, dY = s["X"].float(), s["dY"].float()
    dX = dY @ _weight_plain(s)
    if s["A"] is None:
        return dX.bfloat16(), None, None
    A, B = s["A"].float(), s["B"].float()
    u = dY @ B.t()
    dX = dX + u @ A.t()
    return dX.bfloat16(), (X.t() @ u).bfloat16(), ((X @ A).t() @ dY).bfloat16()


def _to_e4m3(x, positive):
    """x in blocks of BLOCK as e4m3 codes and one fp32 scale a block: scale = max |x| / 448.
    Where `positive`, what is above zero stays above zero."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    live = top >= FLUSH
    top = torch.where(live, top, torch.ones_like(top))
    full = torch.full_like(top, E4M3_MAX)
    y = torch.where(live, b * (full / top), torch.zeros_like(b))
    q = y.to(torch.float8_e4m3fn)
    if positive:
        q = torch.where((y > 0) & (q.float() == 0), torch.full_like(y, E4M3_TINY), q.float()).to(torch.float8_e4m3fn)
    return q.view(-1), torch.where(live, top / full, torch.zeros_like(top)).view(-1)


def _adamw_plain(s):
    g = s["grad_flat"].float() * s["grad_scale"]
    p = s["p"].float() if s["master_flat"] is None else s["master_flat"]
    if s["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        r = (s["v"].float().view(-1, BLOCK) * s["r_scale"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    t = (s["step"] + 1).double()
    rate = (s["lr"] / (1 - s["beta1"] ** t)).float()
    root = (1 / (1 - s["beta2"] ** t).sqrt()).float()
    m = m * s["beta1"] + g * (1 - s["beta1"])
    v = v * s["beta2"] + (g * g) * (1 - s["beta2"])
    r = v.sqrt()
    p = p * (1 - s["lr"] * s["weight_decay"]) - rate * (m / (r * root + s["eps"]))
    if s["bits"] == 8:
        for x, c, k, positive in ((m, "m", "m_scale", False), (r, "v", "r_scale", True)):
            q, scale = _to_e4m3(x, positive)
            s[c].copy_(q)
            s[k].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if s["master_flat"] is not None:
        s["master_flat"].copy_(p)
    s["p"].copy_(p)
    s["step"] += 1
    return {"p": s["p"], "master": s["master_flat"], "m": s["m"], "v": s["v"],
            "m_scale": s["m_scale"], "v_scale": s["r_scale"]}


def _adamw_own(s):
    o = s["opt"]
    o.step(s["grads"], grad_scale=s["grad_scale"])
    return {"p": s["p"], "master": o.master, "m": o.exp_avg, "v": o.exp_avg_sq,
            "m_scale": o.exp_avg_scale, "v_scale": o.exp_avg_sq_scale}


# ---------------------------------------------------------------- cost and the exact result


def _weight_bytes(case):
    N, K = case["N"], case["K"]
    if case.get("weight") == "bitmap":
        return N * K / 8 + 2 * N * (K - K // 2)
    group = case.get("group", 64)
    return N * K / 2 + N * K / group * (3 if case.get("zeros", True) else 2)


def work(case):
    if case["op"] == "adamw":
        n = sum(_tensor_sizes(case))
        b = {"bf16": 2, "fp32": 4}
        per = b[case["grad"]] + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        per += 8 + 2 if case["master"] else 2 * b[case["param"]]
        return {"bytes": n * per, "flops": n * 16}
    N, K, R, M = case["N"], case["K"], case["R"], case["M"]
    data = _weight_bytes(case) + 2 * M * (K + N) + 2 * R * (K + N)
    if case["op"] == "q4":
        return {"bytes": data, "flops": 2 * M * (N * K + R * (K + N))}
    return {"bytes": data + 2 * M * K + 2 * R * (K + N),
            "flops": 2 * M * (N * K + R * (3 * K + 2 * N))}


def exact(case, seed):
    """What run() returns, in 64 bits and unrounded."""
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    N, K = case["N"], case["K"]
    X = s["X"].double()
    if "W" in s:
        W = s["W"].double()
    else:
        W = torch.empty(N, K, dtype=torch.float64, device="cuda")
        W[:, 0::2] = (s["codes"] % 16).double()
        W[:, 1::2] = (s["codes"] // 16).double()
        each = K // s["scales"].shape[1]
        W -= 8 if s["zeros"] is None else s["zeros"].double().repeat_interleave(each, 1)
        W *= s["scales"].double().repeat_interleave(each, 1)
    A = B = None
    if case["R"]:
        A, B = s["A"].double(), s["B"].double()
    if case["op"] == "q4":
        Y = torch.mm(X, W.T)
        return Y if A is None else Y.addmm_(torch.mm(X, A), B)
    dY = s["dY"].double()
    if A is None:
        return torch.mm(dY, W), None, None
    dX = torch.mm(dY, W).addmm_(torch.mm(dY, B.T), A.T)
    return dX, torch.mm(X.T, torch.mm(dY, B.T)), torch.mm(torch.mm(A.T, X.T), dY)


def _exact_adamw(s):
    eight = s["bits"] == 8
    m, v = s["m"].double(), s["v"].double()
    if eight:
        m *= s["m_scale"].double().repeat_interleave(BLOCK)
        v *= s["r_scale"].double().repeat_interleave(BLOCK)
        v *= v
    g = 0.5 * s["grad_flat"].double()
    t = 101
    m = 0.9 * m + 0.1 * g
    v = 0.999 * v + 0.001 * g ** 2
    p = (s["p"] if s["master_flat"] is None else s["master_flat"]).double()
    p = p - 1e-3 * 0.01 * p
    p -= 1e-3 * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
    out = {"p": p, "master": p if s["master"] else None, "m": m, "v": v, "m_scale": None, "v_scale": None}
    if eight:
        for name, x in (("m", m), ("v", v.sqrt())):
            scale = x.view(-1, BLOCK).abs().amax(1) / 448
            out[name + "_scale"] = scale
            out[name] = torch.where(scale[:, None] > 0, x.view(-1, BLOCK) / scale[:, None], 0.0).view(-1)
    return out
