"""The end of a training step, and the answer to single tokens, with the framework's operators.

Training: hidden states of a batch go through the language-model head in FP8, the log probabilities of the next tokens
and the mean entropy are the loss, its gradient goes back through the head, and AdamW updates the head (FP32 master,
8-bit moments, BF16 model copy), which is quantized again for the next step.  Serving: one token's hidden state, the
head, the likeliest alternatives.

    python examples/lm_head_step.py [--tokens 2048 --width 1024 --vocab 8001 --steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_quantized_pretraining_gb300 as F  # noqa: E402


class Head:
    """A vocab x width projection: FP32 master, BF16 copy, FP8 forms, 8-bit AdamW moments."""

    def __init__(self, vocab: int, width: int, generator):
        self.master = torch.randn((vocab, width), device="cuda", generator=generator) * 0.02
        self.model = self.master.bfloat16()
        self.grad = torch.empty((vocab, width), dtype=torch.bfloat16, device="cuda")
        m, v, m_scale, v_scale = F.AdamWTensors.moments(self.master)
        self.tensors = F.AdamWTensors([self.master], [self.grad], [m], [v], [m_scale], [v_scale], model=[self.model],
                                      weight_decay=0.01)
        self.q = F.fp4_fp8_quantize_dual(self.model, block_rows=128)

    def train(self, hidden, targets, step, lr, entropy_weight=0.0):
        """One step on hidden (T x width BF16) and targets (T).  Returns (loss, gradient of the hidden states)."""
        counted = (targets >= 0).sum().clamp(min=1)
        logits, saved = F.fp4_fp8_linear_fwd(hidden, self.q[0])
        r = F.fp4_token_logprobs(logits, targets)
        loss = (-r.logprob.sum() - entropy_weight * r.entropy.sum()) / counted
        g = torch.full_like(r.logprob, -1.0) / counted
        dlogits = F.fp4_token_logprobs_bwd(logits, r, targets, g_logprob=g,
                                           g_entropy=entropy_weight * g if entropy_weight else None, dlogits=logits)
        dhidden, _ = F.fp4_fp8_linear_bwd(dlogits, self.q[1], saved, dW=self.grad)
        F.fp4_adamw_step(self.tensors, step, lr, seed=1)
        F.fp4_fp8_quantize_dual(self.model, 128, *self.q)
        return loss, dhidden

    def answer(self, hidden, top_k=5, temperature=1.0):
        """The likeliest next tokens of each row of hidden (few rows)."""
        logits, _ = F.fp4_fp8_linear_fwd(hidden, self.q[0], save=False)
        return F.fp4_token_logprobs(logits, top_k=top_k, temperature=temperature)


def run(tokens=2048, width=1024, vocab=8001, steps=20, lr=3e-3, log=print):
    """Trains a head to recover a fixed map from hidden states to tokens; returns the losses and the share of tokens
    that it then answers rightly."""
    g = torch.Generator(device="cuda").manual_seed(0)
    centres = torch.randn((vocab, width), device="cuda", generator=g)
    head, losses = Head(vocab, width, g), []
    for step in range(1, steps + 1):
        targets = torch.randint(0, vocab // 8, (tokens,), device="cuda", generator=g)
        hidden = (centres[targets] + 0.3 * torch.randn((tokens, width), device="cuda", generator=g)).bfloat16()
        targets[::17] = -100  # prompt tokens do not count
        loss, _ = head.train(hidden, targets, step, lr)
        losses.append(float(loss))
        log(f"step {step}: loss {losses[-1]:.4f}")
    F.fp4_check_status()
    right = 0
    for i in range(16):
        token = i * (vocab // 8) // 16
        r = head.answer(centres[token:token + 1].bfloat16())
        right += int(r.top_index[0, 0]) == token
        if i == 0:
            log("alternatives:", [(int(t), round(float(p), 3)) for t, p in zip(r.top_index[0], r.top_logprob[0])])
    log(f"{right} of 16 tokens answered rightly")
    return losses, right


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("width", 1024), ("vocab", 8001), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    run(a.tokens, a.width, a.vocab, a.steps)
