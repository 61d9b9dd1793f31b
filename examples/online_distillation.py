"""Speculative rounds under sampling rules, with the drafter trained from what
the target computed for the verification.

A round: the drafter samples K tokens under temperature, top-k, top-p and min-p
(specv_sample, which also writes the rows it sampled from); the target's rows
are kept as their top logits (specv_top_logits), put under the same rules
(specv_filter_logits) and verified against the drafts (specv_verify); and the
drafter takes a step on the distillation loss (distill_loss) at the positions
whose context the target agreed with.  Both models are bigram tables of random
weights, the drafter's of lower rank, so that the example needs no data.

    python examples/online_distillation.py --rounds 200
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import speculative_decoding_verification_50_gb300 as sv  # noqa: E402


class Bigram(torch.nn.Module):
    """Logits of the next token from the last: a table of rank `dim`."""

    def __init__(self, vocab, dim, scale, device, seed):
        super().__init__()
        gen = torch.Generator(device=device).manual_seed(seed)

        def table(*shape):
            return torch.nn.Parameter(torch.randn(*shape, device=device, generator=gen))

        self.embed = table(vocab, dim)
        self.head = table(dim, vocab)
        self.scale = scale / dim ** 0.5

    def forward(self, tokens):
        x = self.embed[tokens.long()].bfloat16()
        return (x @ self.head.bfloat16()) * self.scale


def run(rounds=200, batch=64, drafts=4, vocab=2048, top=64, lr=0.02, temperature=0.8, top_k=50,
        top_p=0.95, min_p=0.02, device="cuda:0", seed=1):
    """Accepted drafts per entry and round (the mean), and the loss, per round."""
    gen = torch.Generator(device=device).manual_seed(seed)
    target = Bigram(vocab, 32, 4.0, device, seed + 1).requires_grad_(False)
    drafter = Bigram(vocab, 24, 1.0, device, seed + 2)
    adam = torch.optim.Adam(drafter.parameters(), lr=lr)
    rules = dict(top_k=torch.full((batch,), top_k, dtype=torch.int32, device=device),
                 top_p=torch.full((batch,), top_p, device=device),
                 min_p=torch.full((batch,), min_p, device=device))
    temp = torch.full((batch,), temperature, device=device)
    last = torch.randint(vocab, (batch,), device=device, generator=gen, dtype=torch.int32)
    q = torch.empty((batch, drafts, vocab), dtype=torch.bfloat16, device=device)
    accepted, losses = [], []
    for _ in range(rounds):
        # the drafter's tokens, and the rows that they were sampled from
        context = [last]
        with torch.no_grad():
            for k in range(drafts):
                u = torch.rand(batch, device=device, generator=gen)
                out = sv.specv_sample(drafter(context[-1]), temp, u, filtered=q[:, k], **rules)
                context.append(out["tokens"])
            context = torch.stack(context, dim=1)  # [batch, drafts + 1]
            p = target(context)                    # [batch, drafts + 1, vocab]
        # what the drafter learns from, before the rules cut the rows
        teacher = sv.specv_top_logits(p.view(-1, vocab), top)
        sv.specv_filter_logits(p, temp, filtered=p, **rules)
        u = torch.rand((batch, drafts + 1), device=device, generator=gen)
        out = sv.specv_verify(p, q, context[:, 1:].contiguous(), temp, u)
        n = out["accept_len"]
        # positions 0 .. n: their contexts are tokens that the target kept
        weights = (torch.arange(drafts + 1, device=device) <= n[:, None]).float().view(-1)
        loss = sv.distill_loss(drafter(context.view(-1)), teacher["ids"], teacher["values"],
                               teacher_lse=teacher["lse"], weights=weights, tail=True)
        loss = loss.sum() / weights.sum()
        adam.zero_grad(set_to_none=True)
        loss.backward()
        adam.step()
        last = out["out_tokens"].gather(1, n[:, None].long())[:, 0].contiguous()
        accepted.append(n.float().mean())
        losses.append(loss.detach())
    return torch.stack(accepted).tolist(), torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--rounds", type=int, default=200)
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--vocab", type=int, default=2048)
    a = ap.parse_args()
    accepted, losses = run(a.rounds, a.batch, vocab=a.vocab)
    step = max(1, a.rounds // 10)
    for i in range(0, a.rounds, step):
        part = slice(i, i + step)
        print(f"rounds {i:4d}-{min(i + step, a.rounds) - 1:4d}: accepted per round "
              f"{sum(accepted[part]) / len(accepted[part]):.2f}, loss {sum(losses[part]) / len(losses[part]):.3f}")


if __name__ == "__main__":
    main()
