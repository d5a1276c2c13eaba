"""The example draft head end to end: its proposals and its gradients against
the same computation in 64 bits, and a few steps of training."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(sga_lib):
    spec = importlib.util.spec_from_file_location(
        "draft_head_example", os.path.join(ROOT, "examples", "draft_head.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def make(example, rows, hidden, vocab, org, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, sigma):
        return torch.empty(shape, device="cuda").normal_(0.0, sigma, generator=g)

    head = example.DraftHead(normal(hidden, hidden, sigma=hidden ** -0.5).bfloat16(),
                             normal(hidden, sigma=0.3),
                             normal(vocab, hidden, sigma=2 * hidden ** -0.5).bfloat16(), rows,
                             org_vocab=org)
    return head, normal(rows, hidden, sigma=1.0).bfloat16(), g


def forward64(head, x, weight, bias, org):
    z = x.double() @ weight.T + bias
    h = x.double() + z * torch.sigmoid(z)
    return h @ head.lm_weight.double()[:org].T


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 24, 200])
def test_proposals(example, rows):
    hidden, vocab, org = 256, 4096, 4000
    head, x, _ = make(example, rows, hidden, vocab, org, rows)
    token, ids, logprobs, entropy = head.propose(x)
    logits = forward64(head, x, head.weight.double(), head.bias.double(), org)
    lp = torch.log_softmax(logits, 1)
    # logits of size up to about 8 went through two roundings to bf16
    # (2^-8 of 8 each, and 2^-8 of h summed over the LM head): 0.1 covers both
    best = logits.max(1).values
    assert (torch.gather(logits, 1, token.long()[:, None])[:, 0] >= best - 0.1).all()
    assert torch.equal(token, ids[:, 0])
    assert ((torch.gather(lp, 1, ids.long()) - logprobs).abs() <= 0.1).all()
    assert ((-(lp.exp() * lp).sum(1) - entropy).abs() <= 0.1).all()
    assert (ids < org).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bonus", [0.0, 0.05])
def test_gradients_against_autograd_in_64_bits(example, bonus):
    rows, hidden, vocab, org = 150, 256, 1000, 990
    head, x, g = make(example, rows, hidden, vocab, org, 3)
    tokens = torch.randint(0, org, (rows,), generator=g, device="cuda", dtype=torch.int32)
    tokens[::10] = -1
    loss, gw, gb = head.loss_and_grads(x, tokens, bonus)
    weight = head.weight.double().requires_grad_()
    bias = head.bias.double().requires_grad_()
    lp = torch.log_softmax(forward64(head, x, weight, bias, org), 1)
    live = tokens >= 0
    at = torch.gather(lp, 1, tokens.clamp(min=0).long()[:, None])[:, 0]
    exp = torch.where(live, -at + bonus * (lp.exp() * lp).sum(1), 0.0)
    exp.mean().backward()
    assert ((loss.double() - exp).abs() <= 0.1).all()
    # h, the logits, their gradient, dh and dz are each rounded to bf16 (about
    # 2e-3 of the value in the 2-norm), the logits' rounding also moves p by up
    # to 2^-8 * 8: together below 3 %
    for got, want in ((gw, weight.grad), (gb, bias.grad)):
        rel = (got.double() - want).norm() / want.norm()
        assert rel < 0.03, float(rel)


@pytest.mark.gpu
def test_training_lowers_the_loss(example):
    losses = example.main(steps=8, rows=128, hidden=256, vocab=2000)
    assert losses[-1] < 0.8 * losses[0]
