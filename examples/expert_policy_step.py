"""Policy-gradient training of an expert layer and a vocabulary head, on the library's training-step operators.

    rows sorted by expert --Experts.forward--> hidden --relu--> Experts.forward (one expert: a linear layer) --> logits
    PolicyLoss.forward_backward --> loss, dlogits
    Experts.backward_data / backward_weight --> gradients of both layers (fp32, added over inner steps)
    GradClip.clip --> clipped gradients --> SGD on fp32 masters, bf16 copies for the products

With ``--orthogonal`` (``ExpertPolicy(orthogonal=True)``) the step uses the operators around these as well:

    TokenLogp.forward --> log-probabilities of the sampled actions, entropy
    TokenLogp.backward --> gradient of an entropy bonus, added to the loss's
    Orthogonal.update --> momentum and an orthogonalised step on the masters, instead of SGD

The task: every row belongs to an expert and has a hidden right action; the policy samples actions and is rewarded for
the right one.  Each batch is used for a few inner steps, so the ratio to the sampling policy moves and is clipped.

    python examples/expert_policy_step.py [--steps 200] [--orthogonal]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from conv2d_backward_implicit_bwd_gb300 import train  # noqa: E402


class ExpertPolicy:
    def __init__(self, experts=4, width=64, hidden=128, vocab=64, rows=1024, seed=0, lr=2.0, max_norm=1.0, kl=0.01, orthogonal=False, bonus=0.01):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.vocab, self.rows, self.lr, self.max_norm = g, vocab, rows, lr, max_norm
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.masters = [normal(experts, hidden, width) / width ** 0.5, normal(1, vocab, hidden) / hidden ** 0.5]
        self.w = [m.bfloat16() for m in self.masters]
        self.grads = [torch.zeros_like(m) for m in self.masters]
        # the plans: kept for the program's life, one set per stream
        self.layer = train.Experts(experts, width, hidden)
        self.head = train.Experts(1, hidden, vocab)
        self.loss = train.PolicyLoss(vocab, clip_low=0.2, clip_high=0.2, kl=kl)
        self.clip = train.GradClip.like(self.grads)
        self.logp, self.bonus = None, bonus
        if orthogonal:
            self.lr = 0.02 if lr == 2.0 else lr
            self.logp = train.TokenLogp(vocab)
            self.step_plans = [train.Orthogonal(*m.shape, "f32") for m in self.masters]
            self.momenta = [torch.zeros_like(m) for m in self.masters]
        # the task: rows sorted by expert (ragged), each with a right action that is linear in the row
        share = torch.rand(experts, generator=g, device="cuda") + 0.2
        cuts = (share.cumsum(0) / share.sum() * rows).round().int()
        self.offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), cuts])
        self.one = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        self.x = normal(rows, width).bfloat16()
        self.right = (self.x.float() @ normal(width, vocab)).argmax(1).int()

    def logits(self):
        self.hidden = torch.relu(self.layer.forward(self.x, self.w[0], self.offsets))
        return self.head.forward(self.hidden, self.w[1], self.one)

    def gradients(self, actions, advantage, weight, old_logp, ref_logp):
        """Forward, loss, backward; adds to self.grads.  Returns (loss, logp)."""
        z = self.logits()
        if self.logp is None:
            loss, logp, dz = self.loss.forward_backward(z, actions, advantage, weight, old_logp, ref_logp, out=z)
        else:
            _, entropy, lse, _, _ = self.logp.forward(z)
            loss, logp, dz = self.loss.forward_backward(z, actions, advantage, weight, old_logp, ref_logp)
            dz += self.logp.backward(z, None, lse, entropy, grad_entropy=-self.bonus * weight, out=z)
        dh = self.head.backward_data(dz, self.w[1], self.one) * (self.hidden > 0)
        self.head.backward_weight(dz, self.hidden, self.one, out=self.grads[1], accumulate=True)
        self.layer.backward_weight(dh, self.x, self.offsets, out=self.grads[0], accumulate=True)
        return loss, logp

    def update(self):
        """Clips the gradients in place and steps; returns their norm before clipping."""
        norm, _ = self.clip.clip(self.grads, self.max_norm)
        if self.logp is not None:
            for plan, m, g, v, w in zip(self.step_plans, self.masters, self.grads, self.momenta, self.w):
                plan.update(m, g, v, self.lr, copy=w)
            torch._foreach_zero_(self.grads)
            return norm
        torch._foreach_add_(self.masters, self.grads, alpha=-self.lr)
        torch._foreach_copy_(self.w, self.masters)
        torch._foreach_zero_(self.grads)
        return norm

    def batch(self):
        """Samples actions; returns (actions, advantage, weight, old_logp, mean reward)."""
        z = self.logits()
        p = torch.softmax(z.float(), 1)
        actions = torch.multinomial(p, 1, generator=self.gen)[:, 0]
        old = torch.log(p.gather(1, actions[:, None])[:, 0]) if self.logp is None else self.logp.forward(z, actions.int())[0]
        reward = (actions == self.right).float()
        weight = torch.full((self.rows,), 1.0 / self.rows, device="cuda")
        return actions.int(), (reward - reward.mean()) / (reward.std() + 1e-4), weight, old, reward.mean()

    def step(self, inner=2):
        actions, advantage, weight, old, reward = self.batch()
        for _ in range(inner):
            loss, _ = self.gradients(actions, advantage, weight, old, old)
            norm = self.update()
        return dict(loss=loss, reward=reward, norm=norm)

    def check(self):
        for plan in (self.layer, self.head, self.loss, self.clip, *([] if self.logp is None else [self.logp, *self.step_plans])):
            status, detail = plan.status()
            if status != train.OK:
                raise train.ConvBwdError(status, f"device status {detail:#x}")


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--orthogonal", action="store_true", help="entropy bonus and orthogonalised updates")
    a = ap.parse_args()
    model = ExpertPolicy(orthogonal=a.orthogonal)
    for i in range(a.steps):
        out = model.step()
        if i % 20 == 0 or i == a.steps - 1:
            print("step %3d  reward %.3f  loss %+.4f  gradient norm %.3f" % (i, out["reward"], out["loss"], out["norm"]))
    model.check()


if __name__ == "__main__":
    main()
