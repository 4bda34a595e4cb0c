"""A small language model learns a teacher's next-token distribution, trained
by the learned optimizer.

    python examples/distill_small_lm.py [steps]

One step, with what this package brings in capitals:

    x = EMBEDDING(tokens)                      bfloat16 activations, float32 table
    y1 = LAYER NORM(x);  z = y1 W1             (W1, Wh: torch matrix products)
    y, s = LAYER NORM(z + x), z + x
    logits = y Wh
    loss, d logits = DISTILLATION(logits, the teacher's top logits)
    ... back through the same: every gradient ends in the float32 buffer of
    its parameter, which the LEARNED OPTIMIZER's step reads.

The learned optimizer runs with weights that route one feature, the momentum
m (decay 0.9) divided by sqrt(v), to its direction output: no meta-trained
weights are needed to see the loss fall.
"""

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import learned_optimizer_step_gb300 as L  # noqa: E402

VOCAB, WIDTH, TOP = 5003, 256, 32


def routing_weights(feature: int, hidden: int = 32) -> np.ndarray:
    """MLP weights with direction = the feature and magnitude = 0."""
    w1 = np.zeros((39, hidden))
    w1[feature, :2] = 1.0, -1.0              # ReLU keeps the sign's two halves apart
    w2 = np.zeros((hidden, hidden))
    w2[0, 0] = w2[1, 1] = 1.0
    w3 = np.zeros((hidden, 2))
    w3[:2, 0] = 1.0, -1.0
    zeros = np.zeros(hidden)
    return np.concatenate([w.ravel() for w in (w1, zeros, w2, zeros, w3, np.zeros(2))]).astype(np.float32)


class Model:
    """Parameters, their gradients and the optimizer's state, all float32."""

    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda") * 0.02  # noqa: E731
        one, zero = torch.ones(WIDTH, device="cuda"), torch.zeros(WIDTH, device="cuda")
        self.params = {"table": normal(VOCAB, WIDTH), "n1.w": one.clone(), "n1.b": zero.clone(),
                       "w1": normal(WIDTH, WIDTH), "n2.w": one.clone(), "n2.b": zero.clone(),
                       "head": normal(WIDTH, VOCAB)}
        self.grads = {k: torch.zeros_like(p) for k, p in self.params.items()}
        state = []
        for k, p in self.params.items():
            rows, cols = (1, p.numel()) if p.dim() == 1 else p.shape
            state.append(L.zeros_state(p, self.grads[k], rows, cols))
        self.optimizer = L.LearnedOptimizer(routing_weights(8), 32, "tc")
        self.state = self.optimizer.prepare(state)
        self.steps = 0

    def loss_and_gradients(self, tokens, top_logits, top_index, temperature=1.0):
        """The loss of every token (float32); the gradients go to self.grads."""
        p, g = self.params, self.grads
        bf = torch.bfloat16
        n = tokens.numel()
        w1, head = p["w1"].to(bf), p["head"].to(bf)
        x = L.embedding_forward(p["table"], tokens, WIDTH ** 0.5, out_dtype=bf)
        y1, mean1, rstd1 = L.layernorm_forward(x, p["n1.w"], p["n1.b"])
        y, s, mean2, rstd2 = L.layernorm_forward(y1 @ w1, p["n2.w"], p["n2.b"], residual=x)
        logits = y @ head
        weight = torch.full((n,), 1.0 / n, device="cuda")
        loss, d = L.distill_forward_backward(logits, top_logits, top_index, temperature, row_weight=weight,
                                             grad=logits)     # the gradient takes the logits' place
        g["head"].copy_(y.t() @ d)
        ds, _, _ = L.layernorm_backward(d @ head.t(), s, mean2, rstd2, p["n2.w"], grad_weight=g["n2.w"],
                                        grad_bias=g["n2.b"])
        g["w1"].copy_(y1.t() @ ds)
        dx, _, _ = L.layernorm_backward(ds @ w1.t(), x, mean1, rstd1, p["n1.w"], grad_residual=ds,
                                        grad_weight=g["n1.w"], grad_bias=g["n1.b"])
        L.embedding_backward(dx, tokens, VOCAB, WIDTH ** 0.5, out=g["table"])
        return loss * n

    def step(self, tokens, top_logits, top_index, lr=2.0):
        loss = self.loss_and_gradients(tokens, top_logits, top_index)
        self.steps += 1
        self.optimizer.step(self.state, self.steps, lr)
        return loss


class Teacher:
    """A fixed bigram model: the top logits that follow each token."""

    def __init__(self, seed: int = 1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        a, b = (torch.randn(*s, generator=g, device="cuda") for s in ((VOCAB, 24), (24, VOCAB)))
        self.top, self.index = torch.topk(a @ b, TOP, dim=1)
        self.gen = g

    def batch(self, count: int):
        """Text-like tokens and the teacher's list for each."""
        u = torch.rand(count, generator=self.gen, device="cuda", dtype=torch.float64)
        tokens = ((VOCAB + 1.0) ** u - 1.0).long().clamp_(0, VOCAB - 1)
        return tokens, self.top[tokens], self.index[tokens]


def main(steps: int = 60, batch: int = 4096, show: bool = True):
    """Losses (mean over the batch) of `steps` steps."""
    model, teacher = Model(), Teacher()
    losses = []
    for k in range(steps):
        loss = model.step(*teacher.batch(batch))
        losses.append(float(loss.mean()))
        if show and (k % 10 == 0 or k == steps - 1):
            print("step %3d  loss %.4f" % (k, losses[-1]))
    L.check_indices()
    model.optimizer.check()
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
