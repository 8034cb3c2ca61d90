"""A small language model on one MI355X: embedding, an expert layer, and a
classifier whose logits are never in memory; trained with Muon and AdamW, then
distilled into a narrower one, and asked for tokens' probabilities one by one.

    python examples/language_model.py [--steps 40] [--vocab 4000] [--tokens 2048]

The text repeats a fixed table: each token has four that may follow it.  Some
places are padding (target -1), which costs nothing and gets no gradient.
"""
import argparse
import importlib.util
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))

import matrix_orthogonalizing_optimizer_muon_amd as M  # noqa: E402

_spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(HERE, "expert_layer.py"))
expert_layer = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(expert_layer)


class LanguageModel:
    """Embedding and classifier (vocab x width, bf16) around one expert layer with a
    way past it."""

    def __init__(self, vocab, width, hidden, experts, k, seed, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.scale = width ** 0.5
        self.table = (torch.randn(vocab, width, generator=g, device=device) / self.scale).bfloat16()
        self.classifier = (torch.randn(vocab, width, generator=g, device=device) / self.scale).bfloat16()
        self.layer = expert_layer.ExpertLayer(experts, width, hidden, k, seed + 1, device)

    def hidden(self, tokens):
        """The classifier's inputs for these tokens, and what backward() needs."""
        h = M.embed(tokens, self.table, scale=self.scale)
        out, saved = self.layer.forward(h)
        return h + out, (tokens, saved)

    def backward(self, dx, saved):
        """Gradients of (table, router, gate_up, down) from that of the classifier's inputs."""
        tokens, layer = saved
        grads, dh = self.layer.backward(dx, layer)
        return (M.embed_backward(dx + dh, tokens, self.table.shape[0], scale=self.scale), *grads)

    def loss_and_grads(self, tokens, targets, teacher=None, temperature=2.0):
        """Mean loss over the places that count, and the gradients of (classifier, table, router, gate_up, down).
        teacher: (logits, ids) of another model's largest logits instead of targets."""
        x, saved = self.hidden(tokens)
        count = (targets >= 0).sum().clamp_min(1)
        dloss = (targets >= 0).float() / count
        if teacher is None:
            loss, _, dx, dw = M.classifier_loss_grads(dloss, x, self.classifier, targets)
        else:
            ids = torch.where(targets[:, None] >= 0, teacher[1], -1)
            loss, _, dx, dw = M.distill_loss_grads(dloss, x, self.classifier, teacher[0], ids, temperature=temperature)
        return loss.sum() / count, (dw, *self.backward(dx, saved))

    def top(self, tokens, k):
        """The k largest logits and their ids for these tokens."""
        logits = self.hidden(tokens)[0].float() @ self.classifier.float().t()
        return torch.topk(logits, k, dim=1)


class Trainer:
    """Muon for the experts' matrices, AdamW for the rest."""

    def __init__(self, model, lr=0.02):
        self.model, self.lr, self.steps = model, lr, 0
        layer = model.layer
        self.matrices = [*layer.gate_up, *layer.down]
        shapes = [tuple(m.shape) for m in self.matrices]
        self.muon = M.MuonPlan(shapes, "bf16", tune="off")
        self.momenta = [torch.zeros(s, device=model.table.device) for s in shapes]
        self.rest = [model.classifier, model.table, layer.router]
        self.adamw = M.AdamWPlan([t.numel() for t in self.rest], ["bf16", "bf16", "f32"])
        self.moments = [[torch.zeros(t.shape, device=t.device) for t in self.rest] for _ in range(2)]

    def step(self, grads):
        dw, dtable, d_router, d_gate_up, d_down = grads
        self.steps += 1
        self.muon.step(self.matrices, [*d_gate_up, *d_down], self.momenta, lr=self.lr, wd=0.0)
        self.adamw.step(self.rest, [dw, dtable, d_router.contiguous()], *self.moments, lr=self.lr / 4, wd=0.0,
                        step=self.steps)

    def close(self):
        self.muon.close()
        self.adamw.close()


def text(vocab, tokens, seed, device="cuda"):
    """Tokens and what follows each, a tenth of it padding."""
    g = torch.Generator(device=device).manual_seed(seed)
    follows = torch.randint(0, vocab, (vocab, 4), generator=torch.Generator(device=device).manual_seed(9), device=device)
    t = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    y = follows[t, torch.randint(0, 4, (tokens,), generator=g, device=device)]
    return t, torch.where(torch.rand(tokens, generator=g, device=device) < 0.1, -1, y)


def train(steps=40, vocab=4000, tokens=2048, width=256, hidden=192, experts=8, k=2, teacher=None, seed=1, report=None):
    """Losses of the steps, and the model.  teacher: a model whose 16 largest logits are learnt."""
    model = LanguageModel(vocab, width, hidden, experts, k, seed)
    trainer = Trainer(model)
    losses = []
    for step in range(steps):
        t, y = text(vocab, tokens, 100 + step)
        top = None if teacher is None else teacher.top(t, 16)
        loss, grads = model.loss_and_grads(t, y, top)
        trainer.step(grads)
        losses.append(loss)
        if report and (step == 0 or (step + 1) % 10 == 0):
            report(f"step {step + 1}: loss {float(loss):.4f}")
    trainer.close()
    return [float(v) for v in losses], model


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--vocab", type=int, default=4000)
    p.add_argument("--tokens", type=int, default=2048)
    a = p.parse_args()

    def say(s):
        print(s, flush=True)
    _, large = train(a.steps, a.vocab, a.tokens, report=say)
    say("distilled into half the width:")
    _, small = train(a.steps, a.vocab, a.tokens, width=128, teacher=large, seed=5, report=say)
    t, y = text(a.vocab, 8, 7)
    for name, model in (("large", large), ("small", small)):
        one = [float(M.classifier_loss(model.hidden(t[i:i + 1])[0], model.classifier, y[i:i + 1])[0]) for i in range(8)]
        say(f"{name}: log-probabilities of eight tokens " + " ".join(f"{-v:.2f}" for v in one))


if __name__ == "__main__":
    main()
