"""Natural gradient steps of a token policy's output layer.

A linear head maps features to logits over a small vocabulary.  Each round draws
tokens from the policy, scores them (kfac_token_logprob), rewards them, and takes
K-FAC steps on the clipped policy loss: kfac_policy_loss writes the output gradients
[rows, vocab], which are the source of the factor G (kfac_factor_update) and give the
weight gradient; the preconditioned gradient is bounded in the Fisher metric and
applied by kfac_clip_norm (KfacStep).  --loss preference instead pairs the better and
the worse of two drawn sequences (kfac_preference_loss).

--drafts K: the policy's tokens are drafted K at a time by the policy of the round before,
and accepted or replaced under the present one (kfac_verify_draft).  --checkpoints: the
features and the output gradients are kept in 8 bits (kfac_checkpoint_store), and the
weight gradient and the factors are made from these.

    python examples/policy_step.py [--loss policy|preference] [--rounds N] [--drafts K] [--checkpoints]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from second_order_optimisation_gb300 import kfac  # noqa: E402
from second_order_optimisation_gb300.step import KfacStep  # noqa: E402
from second_order_optimisation_gb300.workloads import Layer  # noqa: E402


class Head:
    """The policy: logits = features @ weight^T, and its K-FAC state."""

    def __init__(self, din: int, vocab: int, rows: int, eta: float, max_norm: float, seed: int = 0, device="cuda",
                 drafts: int = 0, checkpoints: bool = False):
        self.gen = torch.Generator(device=device).manual_seed(seed)
        self.weight = torch.randn(vocab, din, device=device, generator=self.gen) * 0.02
        self.wanted = torch.randn(vocab, din, device=device, generator=self.gen)  # what the reward prefers
        self.step = KfacStep([Layer("head", din, vocab, 1, 1, 0, 1, 1)], rows, xi=0.5, gamma=1e-2, device=device,
                             weights=[self.weight], eta=eta, max_norm=max_norm)
        self.drafts, self.checkpoints = drafts, checkpoints
        self.drafter = self.weight.clone()

    def features(self, rows: int) -> torch.Tensor:
        return torch.randn(rows, self.weight.shape[1], device=self.weight.device, generator=self.gen).bfloat16()

    def logits(self, a: torch.Tensor) -> torch.Tensor:
        return a @ self.weight.bfloat16().t()

    def draw(self, logits: torch.Tensor) -> torch.Tensor:
        noise = torch.empty_like(logits, dtype=torch.float32).exponential_(generator=self.gen).log_()
        return (logits.float() - noise).argmax(1)

    def reward(self, a: torch.Tensor, tokens: torch.Tensor) -> torch.Tensor:
        """1 for a token whose wanted score is above most others', in 0 .. 1."""
        score = a.float() @ self.wanted.t()
        return (score <= score.gather(1, tokens[:, None])).float().mean(1)

    def logp(self, logits: torch.Tensor, tokens: torch.Tensor) -> torch.Tensor:
        out = torch.empty(len(tokens), device=logits.device)
        kfac.kfac_token_logprob(kfac.TokenLogprob(logits, tokens, out))
        return out

    def drafted(self, a: torch.Tensor, logits: torch.Tensor):
        """Tokens drafted by the policy of the round before and verified under this one, and their
        log-probabilities; -1 and 0 in the rows behind a sequence's last token."""
        rows, vocab = logits.shape
        draft = a @ self.drafter.bfloat16().t()
        self.drafter.copy_(self.weight)
        offsets = torch.arange(0, rows + 1, self.drafts + 1, dtype=torch.int32, device=a.device)
        offsets[-1] = rows
        seqs = len(offsets) - 1
        uniform = torch.rand(rows, device=a.device, generator=self.gen)
        noise = torch.empty(seqs, vocab, device=a.device).exponential_(generator=self.gen)
        accepted = torch.empty(seqs, dtype=torch.int32, device=a.device)
        tokens, logp = self.draw(draft), torch.empty(rows, device=a.device)
        kfac.kfac_verify_draft(kfac.VerifyDraft(logits, tokens, offsets, accepted, tokens, logp, draft=draft, uniform=uniform,
                                                noise=noise))
        return tokens, logp

    def keep(self, a: torch.Tensor):
        """What the backward pass needs of a: its checkpoint, or a itself."""
        return checkpoint(a) if self.checkpoints else a

    def update(self, a, dlogits: torch.Tensor) -> None:
        """One K-FAC step from the per-sample output gradients."""
        if self.checkpoints:
            self.step.run([a], [checkpoint(dlogits)])
        else:
            self.step.run([a], [dlogits], [(dlogits.t() @ a) / len(a)])


def checkpoint(x: torch.Tensor) -> kfac.Checkpoint:
    c = kfac.Checkpoint.empty(*x.shape, device=x.device)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(x, c)])
    return c


def policy_round(head: Head, rows: int, steps: int = 2) -> float:
    a = head.features(rows)
    logits, kept = head.logits(a), head.keep(a)
    if head.drafts:
        tokens, old = head.drafted(a, logits)
    else:
        tokens = head.draw(logits)
        old = head.logp(logits, tokens)
    live = tokens >= 0  # (rows without a token are ignored by the loss)
    reward = head.reward(a, tokens.clamp(min=0))
    mean, std = reward[live].mean(), reward[live].std()
    advantage = (reward - mean) / (std + 1e-6)
    stats = torch.empty(5, device=a.device)
    for _ in range(steps):
        logits = head.logits(a)
        dlogits = torch.empty_like(logits)
        # scaled by the number of rows: each row is one sample's gradient
        kfac.kfac_policy_loss(kfac.PolicyLoss(logits, tokens, advantage, old, stats, dlogits=dlogits, ref_logp=old,
                                              kl_coef=0.02, entropy_coef=0.001, grad_scale=float(rows)))
        head.update(kept, dlogits)
    return float(mean)


def preference_round(head: Head, rows: int, length: int = 4, steps: int = 2) -> float:
    """Pairs of sequences over the same features; the one with more reward is preferred."""
    pairs = rows // (2 * length)
    a = head.features(pairs * length).view(pairs, 1, length, -1).expand(-1, 2, -1, -1).reshape(2 * pairs * length, -1)
    a = a.contiguous()
    logits, kept = head.logits(a), head.keep(a)
    tokens = head.draw(logits)
    reward = head.reward(a, tokens)
    total = reward.view(pairs, 2, length).sum(2)
    swap = (total[:, 1] > total[:, 0])[:, None, None]
    t = tokens.view(pairs, 2, length)
    tokens = torch.where(swap, t.flip(1), t).reshape(-1).contiguous()
    ref = head.logp(logits, tokens).view(2 * pairs, length).sum(1).contiguous()
    offsets = torch.arange(0, len(tokens) + 1, length, dtype=torch.int32, device=a.device)
    loss = torch.empty(1, device=a.device)
    for _ in range(steps):
        logits = head.logits(a)
        dlogits = torch.empty_like(logits)
        kfac.kfac_preference_loss(kfac.PreferenceLoss(logits, tokens, offsets, loss, dlogits=dlogits, ref_logp=ref,
                                                      beta=0.5, grad_scale=float(pairs * length)))
        head.update(kept, dlogits)
    return float(reward.mean())


def train(loss: str = "policy", rounds: int = 20, din: int = 64, vocab: int = 256, rows: int = 2048, seed: int = 0,
          drafts: int = 0, checkpoints: bool = False):
    """Mean reward of each round."""
    head = Head(din, vocab, rows, eta=1.0, max_norm=1.0, seed=seed, drafts=drafts, checkpoints=checkpoints)
    one = policy_round if loss == "policy" else preference_round
    return [one(head, rows) for _ in range(rounds)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=("policy", "preference"), default="policy")
    ap.add_argument("--rounds", type=int, default=20)
    ap.add_argument("--drafts", type=int, default=0)
    ap.add_argument("--checkpoints", action="store_true")
    args = ap.parse_args()
    for i, r in enumerate(train(args.loss, args.rounds, drafts=args.drafts, checkpoints=args.checkpoints)):
        print(f"round {i:3d}  mean reward {r:.4f}")
