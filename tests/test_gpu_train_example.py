"""The operators together, as a training step uses them: the example model's
gradients against torch autograd in fp64 on the same rounded weights, and its
loss over a few steps."""
import importlib.util
import math
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_moe_lm", os.path.join(ROOT, "examples", "train_moe_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_match_autograd(lib, example):
    """Each of the chain's roundings to bf16 (7 of them from the table to the
    table's gradient, 2^-8 at most each) moves a gradient by a like share of
    its norm: 7 * 2^-8 = 2.7%, and 3% with the sums'."""
    vocab, dim, hidden, experts, tokens = 700, 72, 136, 5, 333
    model = example.MoeLm(vocab, dim, hidden, experts, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    targets = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    loss = model.gradients(ids, targets)

    table = model.table.double().requires_grad_()
    up, down, head = (x.to(BF16).double().requires_grad_() for x in (model.up, model.down, model.head))
    expert = ids * 2654435761 % 4294967291 % experts
    h = model.scale * table[ids]
    u = torch.einsum("thd,td->th", up[expert], h)
    x = h + torch.einsum("tdh,th->td", down[expert], torch.relu(u).square())
    want = torch.nn.functional.cross_entropy(x @ head.t(), targets)
    want.backward()
    assert abs(loss.item() - want.item()) < 2.0 ** -8 * want.item()
    for got, ref in ((model.d_table, table), (model.d_head, head), (model.d_up, up), (model.d_down, down)):
        rel = ((got.double() - ref.grad).norm() / ref.grad.norm()).item()
        assert rel < 0.03, rel


def test_loss_falls(lib, example):
    losses = example.train(steps=40, vocab=512, dim=128, hidden=192, experts=4, tokens=2048, log=lambda s: None)
    assert abs(losses[0] - math.log(512)) < 0.5
    assert losses[-1] < 0.25 * losses[0], losses
