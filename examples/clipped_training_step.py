"""One training step as a user of the library writes it: Muon for the hidden matrices, AdamW for
what Muon does not take (embedding, head, gains), and all gradients clipped to a global norm.

The norm of every gradient is formed once; both optimizers take the clip scale from the device, so
that clipping costs no pass of its own over the gradients and no wait on the host. Parameters,
states and gradients stay where they are, so their lists are described to the library once.

The model is a small residual MLP language model that learns to follow a fixed permutation of its
tokens. Run as `python examples/clipped_training_step.py` (needs the built library and a GPU).
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_orthogonalizing_optimizer_gb300 as gns  # noqa: E402


class Model:
    """Leaf tensors of one kind and shape in one stack, as the optimizers take them."""

    def __init__(self, vocab, width, hidden, layers, seed, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def leaf(shape, std, dtype=torch.bfloat16):
            return (torch.randn(shape, generator=g, device=device) * std).to(dtype).requires_grad_()

        self.embedding = leaf((vocab, width), 0.5)
        self.head = leaf((vocab, width), 0.02)
        self.up = leaf((layers, hidden, width), width ** -0.5)
        self.down = leaf((layers, width, hidden), 0.1 * hidden ** -0.5)
        self.gains = [torch.ones(width, device=device).requires_grad_() for _ in range(layers + 1)]

    def loss(self, tokens, targets):
        x = F.embedding(tokens, self.embedding)
        for i in range(self.up.shape[0]):
            y = F.rms_norm(x, x.shape[-1:]) * self.gains[i].to(x.dtype)
            x = x + F.gelu(y @ self.up[i].t()) @ self.down[i].t()
        x = F.rms_norm(x, x.shape[-1:]) * self.gains[-1].to(x.dtype)
        return F.cross_entropy((x @ self.head.t()).float(), targets)


class ClippedStep:
    """Muon on the stacks of matrices, AdamW on the rest, with one clip scale for all of them."""

    def __init__(self, model, max_norm, muon_lr=0.02, adamw_lr=3e-3):
        matrices = [model.up, model.down]
        rest = [model.embedding, model.head] + model.gains
        for p in matrices + rest:
            p.grad = torch.zeros_like(p)  # gradients keep their memory: backward adds into it
        device = model.embedding.device
        data = lambda ps: [p.detach() for p in ps]  # noqa: E731
        f32 = lambda ps: [torch.zeros(p.shape, dtype=torch.float32, device=device) for p in ps]  # noqa: E731

        self.max_norm = max_norm
        self.gradients = [p.grad for p in matrices + rest]
        self.all = gns.tensor_list(self.gradients)
        self.result = torch.empty(2, dtype=torch.float32, device=device)
        self.norm_workspace = gns.alloc_workspace(gns.list_workspace_size(len(self.all)), device)

        self.muon = gns.MuonParams(lr=muon_lr, momentum=0.95)
        self.W, self.G = data(matrices), [p.grad for p in matrices]
        self.M = [torch.zeros_like(w) for w in self.W]
        self.muon_workspace = gns.alloc_workspace(gns.workspace_size(gns._lib.GNS_OP_MUON_STEP, self.M, muon=self.muon), device)

        masters = [p.detach().float() if p.dtype != torch.float32 else None for p in rest]
        self.adamw = gns.AdamWParams(lr=adamw_lr, beta2=0.99, weight_decay=0.0)
        self.lists = [gns.tensor_list(x) for x in (data(rest), [p.grad for p in rest], f32(rest), f32(rest))]
        self.masters = gns.tensor_list(masters)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def __call__(self, step):
        """Step number `step` (1 for the first); result[0] is then the norm before clipping."""
        gns.grad_norm(self.all, max_norm=self.max_norm, result=self.result, workspace=self.norm_workspace, status=self.status)
        scale = self.result[1:]
        gns.muon_step(self.W, self.G, self.M, params=self.muon, workspace=self.muon_workspace, grad_scale=scale, status=self.status)
        self.adamw.step = step
        gns.adamw_step(*self.lists, params=self.adamw, masters=self.masters, grad_scale=scale, status=self.status)
        torch._foreach_zero_(self.gradients)


def train(steps=40, vocab=512, width=128, hidden=512, layers=3, batch=2048, max_norm=0.5, seed=0, log=print):
    """Losses and gradient norms of `steps` steps."""
    model = Model(vocab, width, hidden, layers, seed)
    step = ClippedStep(model, max_norm)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    follow = torch.randperm(vocab, generator=g, device="cuda")
    losses, norms = [], []
    for t in range(1, steps + 1):
        tokens = torch.randint(vocab, (batch,), generator=g, device="cuda")
        loss = model.loss(tokens, follow[tokens])
        loss.backward()
        step(t)
        losses.append(loss.detach())
        norms.append(step.result[0].clone())
    gns.check_status(step.status, what="training")
    losses, norms = torch.stack(losses).tolist(), torch.stack(norms).tolist()
    for t in range(0, steps, max(1, steps // 8)):
        log(f"step {t + 1:4d}  loss {losses[t]:.4f}  gradient norm {norms[t]:.3f}")
    log(f"step {steps:4d}  loss {losses[-1]:.4f}  gradient norm {norms[-1]:.3f}")
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--max-norm", type=float, default=0.5)
    a = ap.parse_args()
    train(steps=a.steps, max_norm=a.max_norm)
