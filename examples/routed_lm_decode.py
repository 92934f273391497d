"""Decoding with a routed language model: the rollouts that a post-training step scores.

A few sequences at a time, one token each per step: embedding lookup, routed layers, output head, then the
sampled tokens' log-probabilities with the entropies and the best alternatives, which is what a
policy step or a distillation takes later.  The routers' scores and choices of all steps go to the balance
loss's counts.

  python examples/routed_lm_decode.py [--tokens 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sinkhorn_point_cloud_gb300 as sot  # noqa: E402

VOCAB, WIDTH, HIDDEN, EXPERTS, CHOICES, LAYERS = 8000, 512, 256, 16, 4, 2


class Decoder:
    """Next-token logits from the current token: embedding, routed layers with their residuals, output head."""

    def __init__(self, seed: int):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *n: (torch.randn(*n, generator=g, device="cuda") * n[-1] ** -0.5).bfloat16()  # noqa: E731
        self.table, self.head = w(VOCAB, WIDTH), w(VOCAB, WIDTH)
        self.layers = [(w(EXPERTS, WIDTH), w(EXPERTS, 2 * HIDDEN, WIDTH), w(EXPERTS, WIDTH, HIDDEN)) for _ in range(LAYERS)]

    def step(self, tokens):
        """(logits [T, VOCAB] bf16, one (router scores, choices) a layer) for tokens [T]"""
        x = sot.sot_embed(self.table, tokens, scale=WIDTH ** 0.5)
        routed = []
        for router, gate_up, down in self.layers:
            y, scores, choices, _ = sot.sot_routed_layer(x, router, gate_up, down, CHOICES)
            x = x + y
            routed.append((scores, choices))
        return x @ self.head.T, routed


def decode(tokens=32, sequences=4, alternatives=8, seed=0, temperature=0.8):
    """Samples `tokens` tokens for each sequence; returns tokens, log-probabilities and entropies [tokens, sequences],
    alternatives [tokens, sequences, alternatives] and the experts' counts of each layer."""
    model = Decoder(1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    now = torch.randint(0, VOCAB, (sequences,), generator=g, device="cuda")
    said, logps, entropies, best, scores, choices = [], [], [], [], [[] for _ in range(LAYERS)], [[] for _ in range(LAYERS)]
    for _ in range(tokens):
        logits, routed = model.step(now)
        noise = -torch.empty(logits.shape, device="cuda").exponential_(generator=g).log()  # the largest of y + noise is a sample
        now = (logits.float() / temperature + noise).argmax(1)
        logp, _, entropy, ids, _ = sot.sot_token_topk(logits, alternatives, target=now, temperature=temperature)
        said.append(now)
        logps.append(logp)
        entropies.append(entropy)
        best.append(ids)
        for layer, (r, c) in enumerate(routed):
            scores[layer].append(r)
            choices[layer].append(c)
    counts = [sot.sot_balance_loss(torch.cat(r), torch.cat(c), grad=False)[0] for r, c in zip(scores, choices)]
    return torch.stack(said), torch.stack(logps), torch.stack(entropies), torch.stack(best), counts


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=32)
    said, logps, entropies, _, counts = decode(ap.parse_args().tokens)
    print("tokens", tuple(said.shape), " mean log-probability %.4f  mean entropy %.4f" % (logps.mean().item(), entropies.mean().item()))
    print("choices of each expert, by layer:", [c.tolist() for c in counts])
