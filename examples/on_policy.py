"""On-policy distillation in small: a student draws its own text through an 8-bit head, a
teacher scores the positions, and the student takes a step of the fused KL loss on them.

    python examples/on_policy.py [--steps 3] [--batch 8] [--length 64]

The "models" are random tables, one hidden state per previous token, so that the example shows
the calls and not a network: what a real trunk would compute is `hidden(tokens)`.  Each drawn
token is one `draw_token` (8-bit product of the LM head, then the sampler); the teacher's
top-K cache comes from `teacher_topk`, and `fused_kl` gives the loss and the gradients of the
student's hidden states and head.  After each step the head is brought to 8 bits again.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lm_head_top_tcgen05_gb300 as fkl  # noqa: E402


class Table:
    """A stand-in for a trunk: the hidden state after a token is the token's row."""

    def __init__(self, vocab, width, generator, device):
        self.rows = torch.randn(vocab, width, generator=generator, device=device).to(torch.bfloat16)
        self.head = (torch.randn(vocab, width, generator=generator, device=device) * 0.05).to(torch.bfloat16)

    def hidden(self, tokens):
        return self.rows[tokens.long()]


def generate(student, head8, start, length, generator, **settings):
    """Tokens [batch, length] drawn by the student from its 8-bit head, and the log-probabilities
    with which they were drawn."""
    token, out, logs = start, [], []
    logits = torch.empty(start.shape[0], head8[0].shape[0], device=start.device)
    for _ in range(length):
        u = torch.rand(start.shape[0], generator=generator, device=start.device)
        token, logprob = fkl.draw_token(student.hidden(token), *head8, u, logits=logits, **settings)
        out.append(token)
        logs.append(logprob)
    return torch.stack(out, 1), torch.stack(logs, 1)


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--steps", type=int, default=3)
    a.add_argument("--batch", type=int, default=8)
    a.add_argument("--length", type=int, default=64)
    a.add_argument("--vocab", type=int, default=8192)
    a.add_argument("--width", type=int, default=256)
    a.add_argument("--top-k", type=int, default=64)
    a.add_argument("--lr", type=float, default=20.0)
    a = a.parse_args(argv)
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(0)
    teacher, student = Table(a.vocab, a.width, g, device), Table(a.vocab, a.width, g, device)
    losses = []
    for step in range(a.steps):
        head8 = fkl.quantize_int8(student.head)
        start = torch.randint(0, a.vocab, (a.batch,), generator=g, device=device, dtype=torch.int32)
        tokens, logs = generate(student, head8, start, a.length, g, temperature=0.9, top_p=0.95)
        assert (tokens >= 0).all()  # -1: a row without a logit to draw from, as a failed product leaves
        seen = torch.cat([start[:, None], tokens[:, :-1]], 1).reshape(-1)  # the states the tokens came from
        ids, values = fkl.teacher_topk(teacher.hidden(seen).contiguous(), teacher.head, a.top_k)
        H = student.hidden(seen).contiguous().requires_grad_()
        W = student.head.clone().requires_grad_()
        loss = fkl.fused_kl(H, W, ids, values)
        loss.backward()
        assert fkl.read_status(device=device) == 0
        with torch.no_grad():
            student.head = (student.head.float() - a.lr * W.grad.float()).to(torch.bfloat16)
            student.rows.index_add_(0, seen.long(), (-a.lr * H.grad.float()).to(torch.bfloat16))
        losses.append(loss.item())
        print(f"step {step}: loss {losses[-1]:.4f}, drawn log-probability {logs.mean().item():.3f}")
    return losses


if __name__ == "__main__":
    main()
