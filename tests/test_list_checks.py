"""The whole-list check that AdamW takes between steps: it says yes only to tensors of the same
types, shapes, strides and devices (no GPU)."""
import pytest
import torch

from sparse_rank_linear_b200.optim import _Watch

TENSORS = [torch.zeros(4, 6), torch.zeros(3), torch.zeros(0), torch.zeros(5, 5)]


def watch():
    w = _Watch()
    w.learn(TENSORS)
    return w


def test_nothing_is_known_before_the_first_check():
    assert not _Watch().same(TENSORS)


def test_same_kinds_elsewhere_in_memory():
    assert watch().same([t.clone() for t in TENSORS])


@pytest.mark.parametrize("i,other", [
    (0, torch.zeros(6, 4)), (0, torch.zeros(24)), (0, torch.zeros(4, 6, 1)), (0, torch.zeros(4, 6).bfloat16()),
    (0, torch.zeros(6, 4).t()), (1, torch.zeros(2)), (1, torch.zeros(6)[::2]), (2, torch.zeros(1)),
    (3, torch.zeros(5, 5).t()), (3, torch.zeros(5, 5, dtype=torch.int32)), (3, torch.zeros(5, 5, device="meta")),
    (3, None), (3, [[0.0] * 5] * 5),
])
def test_anything_else_is_looked_at_again(i, other):
    w = watch()
    assert not w.same(TENSORS[:i] + [other] + TENSORS[i + 1:])
    assert w.same(TENSORS)


def test_without_the_guards_every_list_is_looked_at(monkeypatch):
    monkeypatch.setattr(torch._C._dynamo, "guards", None)
    assert not watch().same(TENSORS)
