"""One round of reinforcement learning at the language-model head, on synthetic hidden states.

    python examples/rl_step.py [--sequences 16] [--length 256] [--hidden 1024] [--vocab 32000] [--steps 20]

The chain a trainer runs around the head, each step one call of the library:

1. rollout, in 8 bits: residual add + RMS norm to e4m3, the head's product for one token of every
   sequence at a time, a token drawn from the logits;
2. scoring by the frozen reference policy (``flce_score_valid``) and by the policy itself: ref_logp, old_logp;
3. training: norm (with gradient), per-token log-probabilities without the logits, the clipped policy loss with a
   KL term, and its backward into the head and the norm;
4. a preference step on the same sequences, taken in pairs.

The "reward" is the share of a sequence's tokens with an even id, so that a few steps visibly move the policy.
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import lm_head_linear_gb300 as flce

IGNORE = -100


class Head:
    """A final norm and a language-model head, the part of a policy that is trained here."""

    def __init__(self, hidden: int, vocab: int, dev, seed: int):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.norm = torch.ones(hidden, device=dev, requires_grad=True)
        self.W = (torch.randn(vocab, hidden, generator=g, device=dev) * hidden ** -0.5).bfloat16().requires_grad_(True)

    def frozen_fp8(self):
        """The head's weights in 8 bits, laid out once for a rollout."""
        return flce.flce_quantize_fp8(self.W.detach())

    def hidden(self, x, residual):
        return flce.add_rms_norm(x, self.norm, residual)

    def parameters(self):
        return [self.norm, self.W]


def rollout(head, x, residual, length: int, generator):
    """Draws `length` tokens for every sequence from the 8-bit logits.  x, residual [S, length, hidden]."""
    S = x.shape[0]
    Wq, Ws = head.frozen_fp8()
    ws = torch.empty(256, dtype=torch.uint8, device=x.device)
    logits = torch.empty(S, Wq.shape[0], dtype=torch.float32, device=x.device)
    tokens = torch.empty(S, length, dtype=torch.int64, device=x.device)
    for t in range(length):
        _, _, _, q, qs = flce.flce_add_rms_norm(x[:, t], head.norm.detach(), residual=residual[:, t], normed=False, fp8=True)
        flce.flce_linear_fp8(q, qs, Wq, Ws, dtype=torch.float32, workspace=ws, out={"y": logits})
        gumbel = -torch.empty_like(logits).exponential_(generator=generator).log_()
        tokens[:, t] = (logits + gumbel).argmax(dim=1)
    assert flce.flce_read_device_status(ws) == 0
    return tokens


def run(sequences=16, length=256, hidden=1024, vocab=32000, steps=20, lr=0.5, prompt=0.25, seed=0, device="cuda"):
    """Returns a list of per-step metrics (floats)."""
    dev = torch.device(device)
    g = torch.Generator(device=dev).manual_seed(seed)
    S, T = sequences, sequences * length
    x = torch.randn(S, length, hidden, generator=g, device=dev).bfloat16()
    residual = torch.randn(S, length, hidden, generator=g, device=dev).bfloat16()
    flat_x, flat_r = x.view(T, hidden), residual.view(T, hidden)
    cu = torch.arange(S + 1, device=dev) * length
    policy, reference = Head(hidden, vocab, dev, seed + 1), Head(hidden, vocab, dev, seed + 1)
    log = []
    for step in range(steps):
        if step % 4 == 0:  # a new rollout every few updates
            tokens = rollout(policy, x, residual, length, g)
            y = tokens.clone()
            y[:, :int(prompt * length)] = IGNORE  # the prompt is not trained on
            reward = (tokens % 2 == 0).float().mean(dim=1)
            advantages = (reward - reward.mean()) / (reward.std() + 1e-6)
            y = y.view(T)
            with torch.no_grad():
                old_logp = flce.flce_score_valid(policy.hidden(flat_x, flat_r)[0], policy.W.detach(), y, IGNORE)[0]
                ref_logp = flce.flce_score_valid(reference.hidden(flat_x, flat_r)[0], reference.W.detach(), y, IGNORE)[0]
        h, _ = policy.hidden(flat_x, flat_r)
        logp = flce.linear_log_probs(h, policy.W, y, IGNORE)
        loss, stats = flce.policy_loss(logp, old_logp, advantages, y, ref_logp, cu, per_sequence=True,
                                       reduction="sequence_mean", clip_low=0.2, clip_high=0.28, kl_coef=0.01)
        loss.backward()
        with torch.no_grad():
            for p in policy.parameters():
                p -= (lr * p.grad / (p.grad.norm() + 1e-12)).to(p.dtype)
                p.grad = None
        log.append({"reward": float(reward.mean()), "policy_loss": float(loss.detach()), "kl": float(stats[0]),
                    "clipped": float(stats[1]), "ratio": float(stats[3])})
    # a preference step: of every two sequences the better-rewarded one is the chosen one
    order = torch.arange(S // 2 * 2, device=dev).view(-1, 2)
    swap = reward[order[:, 0]] < reward[order[:, 1]]
    order = torch.where(swap[:, None], order.flip(1), order).reshape(-1)
    px, pr, py = x[order].reshape(-1, hidden), residual[order].reshape(-1, hidden), y.view(S, length)[order].reshape(-1)
    pairs_cu = torch.arange(order.numel() + 1, device=dev) * length
    pref = ref_logp.view(S, length)[order].reshape(-1)
    for _ in range(3):
        h, _ = policy.hidden(px, pr)
        loss, chosen, rejected = flce.preference_loss(flce.linear_log_probs(h, policy.W, py, IGNORE), py, pairs_cu, pref, beta=0.05)
        loss.backward()
        with torch.no_grad():
            for p in policy.parameters():
                p -= (lr * p.grad / (p.grad.norm() + 1e-12)).to(p.dtype)
                p.grad = None
        log.append({"preference_loss": float(loss.detach()), "margin": float((chosen - rejected).mean())})
    return log


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("sequences", 16), ("length", 256), ("hidden", 1024), ("vocab", 32000), ("steps", 20), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=default)
    for i, m in enumerate(run(**vars(ap.parse_args()))):
        print(f"{i:3d}  " + "  ".join(f"{k} {v:9.5f}" for k, v in m.items()))


if __name__ == "__main__":
    main()
