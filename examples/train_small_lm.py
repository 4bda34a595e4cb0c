"""A small language model trained on next tokens, from lookup to updated weights.

    python examples/train_small_lm.py [steps]

One step, with what this package brings in capitals:

    x = EMBEDDING(tokens)                          bfloat16 activations, float32 table
    y0 = LAYER NORM(x);  z1, gate = y0 W1, y0 G1   (W1, G1, W2: torch matrix products)
    y1, s1 = BLOCK NORM(z1, x, gate);  z2 = y1 W2
    y2, s2 = BLOCK NORM(z2, s1)
    loss = LINEAR CROSS ENTROPY(y2, head, next tokens)      no logits in memory
    ... back through the same: every gradient ends in the float32 buffer of its
    parameter;  ADAMW clips them all together, steps the float32 weights (the two tables'
    moments in 8 bits) and writes the bfloat16 copies that the next step's products read.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import learned_optimizer_step_gb300 as L  # noqa: E402

VOCAB, WIDTH, SCALE = 5003, 256, 0.7
BF = torch.bfloat16


class Model:
    """Parameters, their gradients and moments, and the optimizer's list."""

    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda") * 0.02  # noqa: E731
        one, zero = torch.ones(WIDTH, device="cuda"), torch.zeros(WIDTH, device="cuda")
        self.params = {"table": normal(VOCAB, WIDTH), "head": normal(VOCAB, WIDTH), "w1": normal(WIDTH, WIDTH),
                       "g1": normal(WIDTH, WIDTH), "w2": normal(WIDTH, WIDTH), "n0.w": one.clone(), "n0.b": zero.clone(),
                       "n1.post": one.clone(), "n1.pre": one.clone(), "n2.post": one.clone(), "n2.pre": one.clone()}
        self.grads = {k: torch.zeros_like(p) for k, p in self.params.items()}
        tensors = []
        for k, p in self.params.items():
            matrix = p.dim() == 2
            tensors.append(L.AdamWTensor.zeros(p, self.grads[k], "8bit" if k in ("table", "head") else "float32",
                                               BF if matrix and k != "table" else None, decay=matrix))
        self.copies = {k: t.copy for k, t in zip(self.params, tensors) if t.copy is not None}
        self.optimizer = L.AdamW(tensors, weight_decay=0.01)
        self.steps = 0

    def loss_and_gradients(self, tokens, following):
        """The loss of every token (float32); the gradients of their mean go to self.grads."""
        p, g, c = self.params, self.grads, self.copies
        w = torch.full((tokens.numel(),), 1.0 / tokens.numel(), device="cuda")
        x = L.embedding_forward(p["table"], tokens, WIDTH ** 0.5, out_dtype=BF)
        y0, mean, rstd = L.layernorm_forward(x, p["n0.w"], p["n0.b"])
        z1, gate = y0 @ c["w1"], y0 @ c["g1"]
        y1, s1, a1, b1 = L.block_norm_forward(z1, x, p["n1.post"], p["n1.pre"], gate=gate, scale=SCALE)
        z2 = y1 @ c["w2"]
        y2, s2, a2, b2 = L.block_norm_forward(z2, s1, p["n2.post"], p["n2.pre"], scale=SCALE)
        loss, lse = L.linear_cross_entropy_forward(y2, c["head"], following, row_weight=w)

        dy2, _ = L.linear_cross_entropy_backward(y2, c["head"], following, lse, row_weight=w, grad_weight=g["head"])
        dz2, ds1, _, _, _ = L.block_norm_backward(dy2, z2, s2, a2, b2, p["n2.post"], p["n2.pre"], scale=SCALE,
                                                  grad_w_post=g["n2.post"], grad_w_pre=g["n2.pre"])
        g["w2"].copy_(y1.t() @ dz2)
        dz1, dx, dgate, _, _ = L.block_norm_backward(dz2 @ c["w2"].t(), z1, s1, a1, b1, p["n1.post"], p["n1.pre"], gate=gate,
                                                     scale=SCALE, grad_summed=ds1, grad_w_post=g["n1.post"],
                                                     grad_w_pre=g["n1.pre"])
        g["w1"].copy_(y0.t() @ dz1)
        g["g1"].copy_(y0.t() @ dgate)
        dx, _, _ = L.layernorm_backward(dz1 @ c["w1"].t() + dgate @ c["g1"].t(), x, mean, rstd, p["n0.w"], grad_residual=dx,
                                        grad_weight=g["n0.w"], grad_bias=g["n0.b"])
        L.embedding_backward(dx, tokens, VOCAB, WIDTH ** 0.5, out=g["table"])
        return loss * tokens.numel()

    def step(self, tokens, following, lr=3e-3):
        """(losses, the gradients' norm)"""
        loss = self.loss_and_gradients(tokens, following)
        self.steps += 1
        return loss, self.optimizer.step(self.steps, lr, max_norm=1.0)


class Text:
    """Sequences in which most tokens determine the next one."""

    def __init__(self, seed: int = 1):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.next = torch.randperm(VOCAB, generator=self.gen, device="cuda")

    def batch(self, count: int):
        u = torch.rand(count, generator=self.gen, device="cuda", dtype=torch.float64)
        tokens = ((VOCAB + 1.0) ** u - 1.0).long().clamp_(0, VOCAB - 1)
        other = torch.randint(0, VOCAB, (count,), generator=self.gen, device="cuda")
        following = torch.where(torch.rand(count, generator=self.gen, device="cuda") < 0.9, self.next[tokens], other)
        following[::50] = -1                  # the last token of a sequence has none
        return tokens, following


def main(steps: int = 60, batch: int = 4096, show: bool = True):
    """Losses (mean over the tokens that have a next one) of `steps` steps."""
    model, text = Model(), Text()
    losses = []
    for k in range(steps):
        tokens, following = text.batch(batch)
        loss, norm = model.step(tokens, following)
        losses.append(float(loss.sum() / (following >= 0).sum()))
        if show and (k % 10 == 0 or k == steps - 1):
            print("step %3d  loss %.4f  gradient norm %.3f" % (k, losses[-1], float(norm)))
    L.check_indices()
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
