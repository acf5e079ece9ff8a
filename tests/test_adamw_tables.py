"""AdamW over as many tensors as one launch's table holds, one more, and several tables."""
import pytest
import torch

from test_adamw import _before, _check, _make

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [479, 480, 481, 961])
def test_tables_at_their_ends(count, bits):
    opt, params, g = _make([1 + (53 * i) % 400 for i in range(count)], torch.bfloat16, True, bits)
    grads = [(torch.randn(p.shape, generator=g, device="cuda") * 1e-2).bfloat16() for p in params]
    grads[0] = grads[-1] = None  # skipped entries move the tables' ends
    before = _before(opt, params)
    opt.step(grads)
    _check(opt, params, before, grads)
    grads = [(torch.randn(p.shape, generator=g, device="cuda") * 1e-2).bfloat16() for p in params]
    before = _before(opt, params)
    opt.step(grads)
    _check(opt, params, before, grads, t=8)
    assert opt.step_count.item() == 8
