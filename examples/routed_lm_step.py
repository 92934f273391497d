"""A post-training step of a small routed language model with the library's losses.

One model, four kinds of data in each step, each with its loss and its gradient with
respect to the logits straight from the library:

  distillation   a teacher's eight best entries and the mass it leaves to the rest
  policy         rollouts with advantages, clipped, with a KL term to the starting model
  preference     pairs of answers, chosen and rejected
  balance        the router's choices on all of these, with per-expert counts

The library writes gradients with respect to logits, torch carries them on to the
weights:  torch.autograd.backward([logits, ...], [grad, ...]).

  python examples/routed_lm_step.py [--steps 40]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sinkhorn_point_cloud_gb300 as sot  # noqa: E402

VOCAB, WIDTH, EXPERTS, CHOICES = 4000, 128, 8, 2


class RoutedLM(torch.nn.Module):
    """Embedding, one routed layer, output head: next-token logits from the current token."""

    def __init__(self, seed: int):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        w = lambda *n: torch.nn.Parameter(torch.randn(*n, generator=g) * n[-1] ** -0.5)  # noqa: E731
        self.embed, self.head = w(VOCAB, WIDTH), w(VOCAB, WIDTH)
        self.router, self.experts = w(EXPERTS, WIDTH), w(EXPERTS, WIDTH, WIDTH)
        self.lean = torch.nn.Parameter(torch.tensor([0.5] * 2 + [0.0] * (EXPERTS - 2)))  # a router that starts out uneven

    def forward(self, tokens):
        """(logits [T, VOCAB] bf16, router logits [T, EXPERTS] fp32, experts chosen [T, CHOICES])"""
        x = self.embed[tokens]
        r = x @ self.router.T + self.lean
        gate, ids = torch.softmax(r, 1).topk(CHOICES, 1)
        y = torch.einsum("td,tkde->tke", x, self.experts[ids])
        h = x + (gate[..., None] * torch.tanh(y)).sum(1)
        return (h @ self.head.T).bfloat16(), r, ids.to(torch.int32)


def batch(T, g, dev):
    return torch.randint(0, VOCAB, (T,), generator=g, device=dev)


def train(steps=40, lr=1e-3, seed=0, report=True):
    """Runs the steps; returns one dict of losses per step."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    model, teacher = RoutedLM(1).to(dev), RoutedLM(2).to(dev)
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    # fixed data: text to distil on, rollouts with advantages, pairs of answers of different lengths
    text, prompts, actions = batch(512, g, dev), batch(256, g, dev), batch(256, g, dev)
    advantage = torch.randn(256, generator=g, device=dev)
    lens = torch.tensor([20, 31, 9, 17, 40, 12, 26, 33], device=dev)
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0)])
    said, answers = batch(int(lens.sum()), g, dev), batch(int(lens.sum()), g, dev)
    answers[::7] = -100  # tokens of the prompt take no part
    with torch.no_grad():
        top, ids = torch.log_softmax(16.0 * teacher(text)[0].float(), 1).topk(8, 1)
        ids = ids.to(torch.int32)
        before = sot.sot_token_logprob(model(prompts)[0], actions)[0]  # the starting model's
        answered = sot.sot_token_logprob(model(said)[0], answers)[0]
    history = []
    for step in range(steps):
        with torch.no_grad():
            old = sot.sot_token_logprob(model(prompts)[0], actions)[0]  # the model that made the rollouts
        logits, routers, chosen = zip(*(model(t) for t in (text, prompts, said)))
        router, choices = torch.cat(routers), torch.cat(chosen)
        distil, d_text = sot.sot_distill_topk(logits[0].detach(), ids, top, tail=True)
        policy, _, kl, d_roll = sot.sot_policy_loss(logits[1].detach(), actions, old, advantage, ref_logp=before, kl_coef=0.05)
        logp, lse = sot.sot_token_logprob(logits[2].detach(), answers)
        prefer, margin, d_logp = sot.sot_preference_loss(logp, offsets, ref_logp=answered, target=answers, beta=0.1)
        d_pairs = sot.sot_token_logprob_grad(logits[2].detach(), answers, lse, d_logp)
        counts, balance, d_router = sot.sot_balance_loss(router.detach(), choices, balance_coef=0.2, z_coef=1e-3)
        opt.zero_grad()
        torch.autograd.backward([*logits, router], [d_text, d_roll, d_pairs, d_router])
        opt.step()
        history.append(dict(distil=distil.sum().item(), policy=policy.sum().item(), kl=kl.mean().item(),
                            prefer=prefer.mean().item(), margin=margin.mean().item(), balance=balance[0].item(),
                            busiest=counts.max().item() / max(1, counts.sum().item())))
        if report and (step % 10 == 0 or step == steps - 1):
            print("step %3d  " % step + "  ".join("%s %.4f" % kv for kv in history[-1].items()))
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    train(ap.parse_args().steps)
