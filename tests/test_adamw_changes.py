"""AdamW between steps: gradients of another shape, parameters whose view changed, attributes
that are set, and what autograd learns of a step."""
import pytest
import torch

import sparse_rank_linear_b200 as salr

gpu = pytest.mark.gpu


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, device="cuda", dtype=dtype)


@gpu
@pytest.mark.parametrize("grad", [(6, 4), (24,), (4, 6, 1), (2, 12)])
def test_gradient_of_another_shape_is_refused(grad):
    p = [zeros(4, 6), zeros(3)]
    opt = salr.AdamW(p)
    ok = [torch.ones(4, 6, device="cuda"), torch.ones(3, device="cuda")]
    for other in (ok[1], None):
        with pytest.raises(ValueError, match="grads"):
            opt.step([torch.ones(grad, device="cuda"), other])
    opt.step(ok)
    with pytest.raises(ValueError, match="grads"):  # after a step too
        opt.step([torch.ones(grad, device="cuda"), ok[1]])
    opt.step(ok)
    assert opt.step_count.item() == 2


@gpu
def test_gradients_may_change_type_and_be_left_out_between_steps():
    p = [zeros(4, 6), zeros(3)]
    opt = salr.AdamW(p, lr=0.1, weight_decay=0.0)
    g = [torch.ones(4, 6, device="cuda"), torch.ones(3, device="cuda")]
    opt.step(g)
    opt.step([x.bfloat16() for x in g])
    opt.step([None, g[1]])
    opt.step(g)
    with pytest.raises(TypeError):
        opt.step([g[0], g[1].bfloat16()])
    with pytest.raises(TypeError):
        opt.step([x.half() for x in g])
    with pytest.raises(ValueError):
        opt.step([x.cpu() for x in g])
    assert opt.step_count.item() == 4
    # m / sqrt(v) is 1 in every step, but that the first tensor's moments miss one
    assert ((p[1] + 0.4).abs() < 1e-5).all() and (p[0] < -0.25).all() and (p[0] == p[0][0, 0]).all()


@gpu
def test_parameter_that_became_transposed_in_place_is_refused():
    p = zeros(4, 4)
    opt = salr.AdamW([p])
    g = torch.ones(4, 4, device="cuda")
    opt.step([g])
    p.data = p.data.t()
    with pytest.raises(ValueError, match="params"):
        opt.step([g])
    p.data = p.data.t()
    opt.step([g])
    assert opt.step_count.item() == 2


@gpu
def test_parameter_of_another_type_in_place_is_refused():
    p = zeros(40, dtype=torch.bfloat16)
    opt = salr.AdamW([p])
    g = torch.ones(40, device="cuda")
    opt.step([g])
    p.data = p.data.view(torch.float16)
    with pytest.raises(TypeError, match="params"):
        opt.step([g])


@gpu
def test_parameter_that_became_shorter_in_place_is_refused():
    p = zeros(300)
    opt = salr.AdamW([p])
    g = torch.ones(300, device="cuda")
    opt.step([g])
    p.data = p.data[:299]
    with pytest.raises(ValueError, match="params"):
        opt.step([g])


@gpu
def test_parameters_that_moved_onto_one_another_are_refused():
    p = [zeros(30), zeros(30)]
    opt = salr.AdamW(p)
    g = [torch.ones(30, device="cuda") for _ in p]
    opt.step(g)
    both = zeros(60)
    p[0].data, p[1].data = both[:30], both[20:50]
    with pytest.raises(ValueError, match="overlap"):
        opt.step(g)
    p[1].data = both[30:]
    opt.step(g)
    assert opt.step_count.item() == 2


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_eps_and_betas_take_effect_when_set(bits):
    g = torch.Generator(device="cuda").manual_seed(0)
    start = torch.randn(500, generator=g, device="cuda")
    grad = torch.randn(500, generator=g, device="cuda") * 1e-3
    got = []
    for given in (True, False):
        p = start.clone()
        kw = dict(betas=(0.5, 0.75), eps=1e-3) if given else {}
        opt = salr.AdamW([p], lr=0.1, state_bits=bits, **kw)
        if not given:
            opt.betas, opt.eps = (0.5, 0.75), 1e-3
        for _ in range(3):
            opt.step([grad])
        got.append(p)
    assert torch.equal(*got)
    for name, bad in (("betas", (1.0, 0.9)), ("betas", (0.9, -0.1)), ("eps", -1.0), ("eps", float("nan"))):
        good = getattr(opt, name)
        setattr(opt, name, bad)
        with pytest.raises(salr.SalrError, match="INVALID"):
            opt.step([grad])
        setattr(opt, name, good)
    assert opt.step_count.item() == 3


@gpu
def test_autograd_learns_that_a_step_changed_the_parameters():
    p = torch.ones(8, device="cuda", requires_grad=True)
    q = torch.ones(8, device="cuda", requires_grad=True)
    y, z = (p * p).sum(), (q * q).sum()  # both save their factors
    opt = salr.AdamW([p, q])
    opt.step([torch.ones(8, device="cuda"), None])
    z.backward()  # q was left alone
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@gpu
def test_decode_and_host_results_count_as_written():
    g = torch.Generator(device="cuda").manual_seed(0)
    w = salr.encode_q4(torch.randn(128, 128, generator=g, device="cuda").bfloat16(), 64)
    out = torch.empty(128, 128, device="cuda", dtype=torch.bfloat16)
    host = torch.zeros(4, 128, dtype=torch.bfloat16).pin_memory()
    there = torch.empty(4, 128, dtype=torch.bfloat16).pin_memory()
    w.decode(out)
    salr.linear_host(host, w, None, None, there)
    torch.cuda.synchronize()
    assert out._version == 1 and there._version == 1 and host._version == 0


@gpu
def test_autograd_learns_that_results_were_written_into_a_tensor():
    g = torch.Generator(device="cuda").manual_seed(0)
    W = torch.randn(128, 128, generator=g, device="cuda").bfloat16()
    X = torch.randn(4, 128, generator=g, device="cuda").bfloat16()
    w = salr.encode_q4(W, 64)
    a = torch.ones(4, 128, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    for write in (lambda y: salr.linear(X, w, Y=y), lambda y: salr.linear_backward(X, X, w, dX=y)):
        buffer = torch.ones(4, 128, device="cuda", dtype=torch.bfloat16)
        s = (a * buffer).sum()  # saves the buffer
        write(buffer)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            s.backward()
