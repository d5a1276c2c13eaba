"""A draft head on the library's operators: proposing tokens and training.

A draft head is one residual block in front of the LM head,

    h = x + silu(W x + b),    logits = h . E^T,

x the target model's hidden states, E the LM head's weight.  Serving
(`propose`): the block, the logits, and per row the greedy token with its log
probability, the row's entropy and the best alternatives.  Training
(`loss_and_grads`): the mean negative log probability of given tokens, less an
entropy bonus, and its gradients with respect to W and b, through the logits,
the LM head (frozen) and the block; or (`distill_and_grads`) the same of the mean
divergence from the target model's top logits.

    python examples/draft_head.py        (needs a GB300; trains a small head)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import greedy_spec_decode_gb300 as sga  # noqa: E402


class DraftHead:
    """weight: bf16 [H, H], bias: float32 [H], lm_weight: bf16 [V, H] (ids past
    org_vocab are padding); at most max_rows rows a call.  Buffers are kept, so
    the calls can be captured in a CUDA graph; what a call returns lies in them
    and holds until the next call."""

    def __init__(self, weight, bias, lm_weight, max_rows, top_k=5, org_vocab=None):
        self.weight, self.bias, self.lm_weight = weight, bias, lm_weight
        V, H = lm_weight.shape
        self.org_vocab = org_vocab or V

        def bf16(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

        def f32(*shape):
            return torch.empty(shape, device="cuda")

        n = max_rows
        self.h, self.preact, self.grad_h = bf16(n, H), bf16(n, H), bf16(n, H)
        self.logits = bf16(n, V)
        self.logprob, self.entropy, self.lse = f32(n), f32(n), f32(n)
        self.top_ids = torch.empty((n, top_k), dtype=torch.int32, device="cuda")
        self.top_logprobs = f32(n, top_k)
        self.grad_weight, self.grad_bias = torch.empty_like(weight), torch.empty_like(bias)
        self.workspace = torch.empty(max(sga.sga_linear_grad_workspace(n, H, H),
                                         sga.sga_linear_grad_workspace(n, V, H)),
                                     dtype=torch.uint8, device="cuda")

    def _logits(self, x, preact=None):
        n = x.size(0)
        sga.sga_linear(x, self.weight, self.h[:n], bias=self.bias, act=sga.SGA_ACT_SILU,
                       residual=x, out_preact=preact)
        return sga.sga_linear(self.h[:n], self.lm_weight, self.logits[:n])

    def propose(self, x):
        """x: bf16 [n, H].  Per row: the greedy tokens int32 [n], the best
        tokens and their log probabilities [n, top_k] (the greedy token first,
        equal logits by ascending id), and the entropy [n]."""
        n = x.size(0)
        sga.sga_token_logprobs(self._logits(x), self.org_vocab, None, None, self.entropy[:n],
                               self.lse[:n], self.top_ids[:n], self.top_logprobs[:n])
        return self.top_ids[:n, 0], self.top_ids[:n], self.top_logprobs[:n], self.entropy[:n]

    def loss_and_grads(self, x, tokens, entropy_bonus=0.0):
        """tokens: int32 [n], -1 where a row has none.  The loss of each row
        ([n]; 0 without a token), and the gradients of their mean with respect
        to weight and bias."""
        n = x.size(0)
        logits = self._logits(x, self.preact[:n])
        logprob, entropy, lse = self.logprob[:n], self.entropy[:n], self.lse[:n]
        sga.sga_token_logprobs(logits, self.org_vocab, tokens, logprob, entropy, lse)
        live = (tokens >= 0).float()
        g_logprob = -live / n
        g_entropy = -entropy_bonus * live / n if entropy_bonus else None
        # the logits are not needed again: their gradient takes their place
        sga.sga_token_logprobs_grad(logits, 0, self.org_vocab, tokens, lse, entropy, g_logprob,
                                    logits, grad_entropy=g_entropy)
        self._block_grads(x, logits)
        return -logprob - entropy_bonus * entropy * live, self.grad_weight, self.grad_bias

    def distill_and_grads(self, x, teacher_ids, teacher_logits, teacher_lse=None,
                          temperature=1.0):
        """teacher_ids / teacher_logits: int32 / float32 [n, k], the target's top
        logits (-1: no entry), teacher_lse [n] the log-sum-exp of all of them over
        the temperature, or None for the list by itself.  The divergence of each row
        ([n]), and the gradients of their mean with respect to weight and bias."""
        n = x.size(0)
        logits = self._logits(x, self.preact[:n])
        mean = torch.full((n,), 1.0 / n, device="cuda")
        # loss and gradient in one pass; the gradient takes the logits' place
        sga.sga_distill(logits, self.org_vocab, teacher_ids, teacher_logits, self.logprob[:n],
                        teacher_lse=teacher_lse, temperature=temperature, grad_loss=mean,
                        out_grad=logits)
        self._block_grads(x, logits)
        return self.logprob[:n], self.grad_weight, self.grad_bias

    def _block_grads(self, x, grad_logits):
        n = x.size(0)
        sga.sga_linear_grad(grad_logits, self.h[:n], self.lm_weight, self.workspace,
                            grad_x=self.grad_h[:n])
        sga.sga_linear_grad(self.grad_h[:n], x, self.weight, self.workspace, sga.SGA_ACT_SILU,
                            self.preact[:n], grad_weight=self.grad_weight,
                            grad_bias=self.grad_bias)


def main(steps=30, rows=256, hidden=512, vocab=8000):
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def normal(*shape, sigma):
        return torch.empty(shape, device="cuda").normal_(0.0, sigma, generator=g)

    master = normal(hidden, hidden, sigma=hidden ** -0.5)      # fp32 copy that is trained
    head = DraftHead(master.bfloat16(), torch.zeros(hidden, device="cuda"),
                     normal(vocab, hidden, sigma=hidden ** -0.5).bfloat16(), rows)
    x = normal(rows, hidden, sigma=1.0).bfloat16()
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    losses = []
    for _ in range(steps):
        loss, gw, gb = head.loss_and_grads(x, tokens)
        losses.append(float(loss.mean()))
        master -= 100.0 * gw.float()
        head.bias -= 100.0 * gb
        head.weight.copy_(master)
    token, ids, logprobs, entropy = head.propose(x)
    hit = (token == tokens).float().mean()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps; the target is the greedy "
          f"token in {100 * float(hit):.0f} % of the rows; mean entropy {float(entropy.mean()):.2f}")
    return losses


if __name__ == "__main__":
    main()
