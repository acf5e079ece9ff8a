"""AdamW over many tensors (salr_adamw, AdamW): refusals on the host, and on the GPU the step
against the formula in 64 bits.

Tolerances count roundings of u = 2^-24 relative each.  With S = |b1 m| + |ob1 g'|: m takes
g * scale, two products, two rounded constants and one sum, at most 4 u S.  v is a sum of
non-negative terms with at most 6 roundings a term (two of g' in its square), 7 u v with
second-order terms; r = sqrt(v) halves the 6 and adds 2 u (it is within 2^-23), 5 u r; d = r
root + eps adds three, 8 u d.  The quotient m / d is within 2 units in the last place, 4 u;
rate and the product with it add 2, and |m| <= S: error at most (4 + 8 + 4 + 2) u rate S / d.
p * decay has two (the product and the constant) and the difference one: in all, with room
for second-order terms,
    |p - p*| <= u (4 |p| + 20 rate S / d).
A bf16 parameter adds half a step, 2^-8 relative; a moment held as e4m3 is within 2^-4
relative of its value, or 2^-10 scale near zero (2^-9 scale where a positive root is kept from
becoming zero)."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_rank_linear_b200 as salr
from sparse_rank_linear_b200 import binding
from sparse_rank_linear_b200.build import build

U = 2.0 ** -24
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


# ---------------------------------------------------------------- refusals (no GPU)


def _table(**kw):
    t = (binding.AdamwTensor * 1)()
    for f in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "master"):
        setattr(t[0], f, 0x10000)
    t[0].n = 8
    for k, v in kw.items():
        setattr(t[0], k, v)
    return t


def _config(**kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=0x10000,
             param_type=0, grad_type=0, state_bits=8, master=1)
    d.update(kw)
    return binding.AdamwConfig(**d)


@pytest.mark.parametrize("table,config,code", [
    (dict(param=None), {}, 1), (dict(exp_avg=None), {}, 1), (dict(exp_avg_sq=None), {}, 1),
    (dict(exp_avg_scale=None), {}, 1), (dict(exp_avg_sq_scale=None), {}, 1),
    (dict(master=None), {}, 1), (dict(n=-1), {}, 1),
    ({}, dict(step=None), 1), ({}, dict(param_type=2), 1), ({}, dict(grad_type=-1), 1),
    ({}, dict(state_bits=16), 1), ({}, dict(param_type=1), 1), ({}, dict(beta1=1.0), 1),
    ({}, dict(beta2=-0.1), 1), ({}, dict(beta1=float("nan")), 1), ({}, dict(eps=-1.0), 1),
    ({}, dict(eps=float("inf")), 1), ({}, dict(lr=float("nan")), 1),
    ({}, dict(weight_decay=float("inf")), 1),
    (dict(param=0x10001), {}, 2), (dict(grad=0x10001), {}, 2), (dict(exp_avg=0x10008), {}, 2),
    (dict(master=0x10004), {}, 2), (dict(exp_avg_scale=0x10002), {}, 2),
    (dict(n=(1 << 38) + 1), {}, 2), ({}, dict(step=0x10004), 2), ({}, dict(lr_dev=0x10002), 2),
])
def test_bad_arguments_rejected_on_host(lib, table, config, code):
    c = _config(**config)
    assert lib.salr_adamw(_table(**table), 1, ctypes.byref(c), None) == code


def test_null_arrays_rejected_on_host(lib):
    c = _config()
    assert lib.salr_adamw(None, 1, ctypes.byref(c), None) == 1
    assert lib.salr_adamw(_table(), -1, ctypes.byref(c), None) == 1
    assert lib.salr_adamw(_table(), 1, None, None) == 1


def test_class_refuses_what_the_library_cannot_take():
    p = torch.zeros(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="empty"):
        salr.AdamW([])
    with pytest.raises(ValueError, match="CUDA"):
        salr.AdamW([p])
    with pytest.raises(TypeError):
        salr.AdamW([p.half()])


# ---------------------------------------------------------------- the step


SIZES = [1, 2, 7, 8, 9, 255, 256, 257, 511, 2048, 2049, 0, 5000, 31]


def _make(sizes, param, master, bits, seed=0, offset=0):
    """An optimizer with a state in full swing, and its inputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(n):
        return torch.randn(n, generator=g, device="cuda")

    params = [(randn(n + offset) * 0.1).to(param)[offset:] for n in sizes]
    opt = salr.AdamW(params, lr=3e-3, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1,
                     state_bits=bits, master=master)
    for s in opt.slices:
        n = s.stop - s.start
        if not n:
            continue
        m, r = randn(n) * 1e-3, randn(n).abs() * 1e-2
        if bits == 8:
            for x, codes, scales in ((m, opt.exp_avg, opt.exp_avg_scale),
                                     (r, opt.exp_avg_sq, opt.exp_avg_sq_scale)):
                k = -(-n // 256)
                b = torch.zeros(k * 256, device="cuda")
                b[:n] = x
                sc = b.view(k, 256).abs().amax(1) / 448
                codes[s.start:s.start + k * 256] = (b.view(k, 256) / sc[:, None]).view(-1).to(codes.dtype)
                scales[s.start // 256:s.start // 256 + k] = sc
        else:
            opt.exp_avg[s], opt.exp_avg_sq[s] = m, r * r
    if master:
        opt.master += 1e-4 * torch.randn(opt.master.shape, generator=g, device="cuda")
    opt.step_count.fill_(6)
    return opt, params, g


def _state(opt):
    """Flat m and sqrt(v) (8 bits) or v (32 bits) in 64 bits."""
    out = []
    for x, s in ((opt.exp_avg, opt.exp_avg_scale), (opt.exp_avg_sq, opt.exp_avg_sq_scale)):
        x = x.double()
        out.append(x if s is None else (x.view(-1, 256) * s.double()[:, None]).view(-1))
    return out


def _check(opt, params, before, grads, lr=3e-3, gscale=1.0, t=7):
    """The state after one step against the formula on the state `before`."""
    p0, m0, v0, master0 = before
    m1, v1 = _state(opt)
    for i, (p, s, g) in enumerate(zip(params, opt.slices, grads)):
        n = s.stop - s.start
        if n == 0:
            continue
        m, v = m0[s], v0[s]
        v = v * v if opt.state_bits == 8 else v
        if g is None:
            assert torch.equal(p.reshape(-1), p0[i])
            assert torch.equal(m1[s], m0[s]) and torch.equal(v1[s], v0[s])
            continue
        x = p0[i].double() if master0 is None else master0[s].double()
        gd = g.double().reshape(-1) * gscale
        S = 0.9 * m.abs() + (1 - 0.9) * gd.abs()
        m, v = 0.9 * m + (1 - 0.9) * gd, 0.99 * v + (1 - 0.99) * gd * gd
        rate, root = lr / (1 - 0.9 ** t), 1 / (1 - 0.99 ** t) ** 0.5
        d = v.sqrt() * root + 1e-6
        x = x * (1 - lr * 0.1) - rate * m / d
        tol = U * (4 * (x.abs() + (rate * m / d).abs()) + 20 * rate * S / d)
        if master0 is not None:
            assert ((opt.master[s].double() - x).abs() <= tol).all()
        if p.dtype == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * x.abs()
        assert ((p.double().reshape(-1) - x).abs() <= tol).all(), f"tensor {i}"
        if opt.state_bits == 32:
            assert ((m1[s] - m).abs() <= 4 * U * S).all()
            assert ((v1[s] - v).abs() <= 7 * U * v).all()
        else:
            k = -(-n // 256)
            for got, want, scales, near, err in (
                    (m1, m, opt.exp_avg_scale, 2.0 ** -10, 4 * U * S),
                    (v1, v.sqrt(), opt.exp_avg_sq_scale, 2.0 ** -9, 6 * U * v.sqrt())):
                sc = scales[s.start // 256:s.start // 256 + k].double()
                pad = torch.zeros(k * 256, dtype=torch.float64, device="cuda")
                pad[:n] = want
                top = pad.view(k, 256).abs().amax(1) / 448
                # the error of the block's largest value, 1 / 448 and the product with it
                assert ((sc - top).abs() <= 16 * U * top + 2 * U * sc).all()
                each = sc.repeat_interleave(256)[:n]
                # the product with 448 / max adds few roundings before the one to e4m3
                assert ((got[s] - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), near * each)
                        * (1 + 2.0 ** -20) + err).all()


def _before(opt, params):
    m, v = _state(opt)
    return ([p.detach().clone().reshape(-1) for p in params], m, v,
            None if opt.master is None else opt.master.clone())


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("param,master", [(torch.bfloat16, False), (torch.bfloat16, True),
                                          (torch.float32, False)])
def test_step_matches_formula(param, master, grad, bits):
    opt, params, g = _make(SIZES, param, master, bits)
    grads = [(torch.randn(p.shape, generator=g, device="cuda") * 1e-2).to(grad) for p in params]
    grads[4] = None
    before = _before(opt, params)
    opt.step(grads)
    _check(opt, params, before, grads)
    assert opt.step_count.item() == 7 and opt._step[1].item() == 0


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [1, 3, 4])
def test_unaligned_slices(offset, bits):
    opt, params, g = _make([300, 17, 2500], torch.bfloat16, False, bits, offset=offset)
    grads = [(torch.randn(p.numel() + 1, generator=g, device="cuda") * 1e-2)[1:] for p in params]
    before = _before(opt, params)
    guard = [p._base[:offset].clone() for p in params]
    opt.step(grads)
    _check(opt, params, before, grads)
    assert all(torch.equal(p._base[:offset], k) for p, k in zip(params, guard))


@gpu
@pytest.mark.parametrize("count", [1, 24, 25, 448, 449, 1000])
def test_tables_of_every_size(count):
    opt, params, g = _make([1 + (37 * i) % 600 for i in range(count)], torch.bfloat16, True, 8)
    grads = [(torch.randn(p.shape, generator=g, device="cuda") * 1e-2).bfloat16() for p in params]
    before = _before(opt, params)
    opt.step(grads)
    _check(opt, params, before, grads)
    assert opt.step_count.item() == 7


@gpu
def test_many_blocks_per_warp_and_scaled_gradients():
    # more blocks than the resident warps take in one pass
    opt, params, g = _make([3_000_001, 123, 4_000_000], torch.bfloat16, True, 8)
    grads = [(torch.randn(p.shape, generator=g, device="cuda") * 1e-2).bfloat16() for p in params]
    before = _before(opt, params)
    opt.step(grads, lr=torch.full((1,), 0.002, device="cuda"),
             grad_scale=torch.full((1,), 0.25, device="cuda"))
    _check(opt, params, before, grads, lr=float(np.float32(0.002)), gscale=0.25)


@gpu
def test_no_gradients_still_counts_the_step():
    opt, params, _ = _make([5], torch.float32, False, 32)
    before = _before(opt, params)
    opt.step([None])
    _check(opt, params, before, [None])
    assert opt.step_count.item() == 7


@gpu
def test_first_steps_from_zero_state():
    # m / sqrt(v) starts at sign(g): three steps on one gradient, in both state widths
    for bits in (32, 8):
        p = torch.full((300,), 0.5, device="cuda")
        g = torch.full((300,), 1e-3, device="cuda")
        g[::2] *= -1
        opt = salr.AdamW([p], lr=1e-2, weight_decay=0.0, eps=0.0, state_bits=bits)
        for _ in range(3):
            opt.step([g])
        want = 0.5 - 3e-2 * torch.sign(g).double()
        # every value is its block's largest, held exactly up to the scale's rounding: some
        # 20 roundings a step of the update 1e-2, and three of p
        assert ((p.double() - want).abs() <= 3 * U * (20 * 1e-2 + 2)).all()
        assert opt.step_count.item() == 3


@gpu
def test_non_finite_gradients_stay_in_their_element():
    p = torch.zeros(512, device="cuda")
    g = torch.full((512,), 1e-2, device="cuda")
    g[3], g[4] = float("nan"), float("inf")
    opt = salr.AdamW([p], state_bits=8)
    opt.step([g])
    bad = torch.zeros(512, dtype=torch.bool, device="cuda")
    bad[3] = bad[4] = True
    assert torch.equal(~torch.isfinite(p), bad)
    m, r = _state(opt)
    assert torch.equal(~torch.isfinite(m), bad) and torch.equal(~torch.isfinite(r), bad)


@gpu
def test_tiny_blocks_are_held_as_zeros():
    p = torch.zeros(256, device="cuda")
    g = torch.full((256,), 1e-37, device="cuda")
    opt = salr.AdamW([p], state_bits=8)
    opt.step([g])
    m, r = _state(opt)
    assert not m.any() and not r.any() and not opt.exp_avg_scale.any()
    assert torch.isfinite(p).all()


@gpu
def test_steps_repeat_bit_for_bit():
    got = []
    for _ in range(2):
        opt, params, g = _make(SIZES, torch.bfloat16, True, 8, seed=3)
        for _ in range(4):
            opt.step([(torch.randn(p.shape, generator=g, device="cuda") * 1e-2) for p in params])
        got.append([opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8), opt.master])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@gpu
def test_captured_step_replays_with_the_state_of_the_moment():
    opt, params, g = _make([700, 90], torch.bfloat16, True, 8)
    grads = [torch.zeros(p.shape, dtype=torch.bfloat16, device="cuda") for p in params]
    lr = torch.full((1,), 1e-3, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        opt.step(grads, lr=lr)
    assert opt.step_count.item() == 6  # capturing runs nothing
    for k in range(3):
        for x in grads:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda") * 1e-2)
        lr.fill_(1e-3 * (k + 1))
        before = _before(opt, params)
        graph.replay()
        torch.cuda.synchronize()
        _check(opt, params, before, grads, lr=float(np.float32(1e-3 * (k + 1))), t=7 + k)


@gpu
def test_step_on_another_stream():
    opt, params, g = _make([4000], torch.float32, False, 32)
    s = torch.cuda.Stream()
    grads = [torch.randn(4000, generator=g, device="cuda") * 1e-2]
    before = _before(opt, params)
    s.wait_stream(torch.cuda.current_stream())
    opt.step(grads, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    _check(opt, params, before, grads)


@gpu
def test_class_refusals_on_device():
    p = torch.zeros(4, 6, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        salr.AdamW([p.t()])
    with pytest.raises(ValueError, match="overlap"):
        salr.AdamW([p, p])
    with pytest.raises(ValueError, match="overlap"):
        salr.AdamW([p, p[1:]])
    with pytest.raises(TypeError, match="one type"):
        salr.AdamW([p, p.bfloat16()])
    with pytest.raises(ValueError, match="master"):
        salr.AdamW([p], master=True)
    with pytest.raises(ValueError, match="state_bits"):
        salr.AdamW([p], state_bits=16)
    opt = salr.AdamW([p, torch.zeros(3, device="cuda")])
    ok = torch.zeros(3, device="cuda")
    for bad in ([p.clone()], [p.t(), ok], [p[:2], ok], [p.cpu(), ok]):
        with pytest.raises(ValueError):
            opt.step(bad)
    for bad in ([p.half(), None], [p.clone(), ok.bfloat16()]):
        with pytest.raises(TypeError):
            opt.step(bad)
    with pytest.raises(ValueError, match="grad_scale"):
        opt.step([None, ok], grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(salr.SalrError):
        opt.step([None, ok], lr=float("nan"))
    assert opt.step_count.item() == 0


@gpu
def test_parameters_that_moved_are_found_again():
    p = [torch.zeros(300, device="cuda"), torch.zeros(5, device="cuda")]
    g = [torch.ones(300, device="cuda"), torch.ones(5, device="cuda")]
    opt = salr.AdamW(p, lr=0.1, weight_decay=0.0)
    opt.step(g)
    old = p[0].data
    p[0].data = torch.full((300,), 2.0, device="cuda")
    opt.step(g)
    torch.cuda.synchronize()
    assert (old == old[0]).all() and abs(old[0].item() + 0.1) < 1e-5  # one step, and left alone
    assert ((p[0] - 1.9).abs() < 1e-5).all()
    p[0].data = torch.zeros(299, device="cuda")
    with pytest.raises(ValueError, match="params"):
        opt.step(g)
    p[0].data = torch.zeros(300, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="params"):
        opt.step(g)
    assert opt.step_count.item() == 2


@gpu
def test_state_buffers_cannot_be_replaced():
    opt = salr.AdamW([torch.zeros(3, device="cuda")], state_bits=8)
    for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "master", "step_count"):
        with pytest.raises(AttributeError):
            setattr(opt, name, torch.zeros(256, device="cuda"))
