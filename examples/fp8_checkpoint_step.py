"""A residual network of gated blocks with norms before and behind them, trained with 8-bit products and 8-bit checkpoints: the
backward pass reads nothing of the forward pass but 8-bit matrices and a factor for each row and norm.

    python examples/fp8_checkpoint_step.py --steps 20

The model learns a fixed random linear map of normal inputs.  Of torch it takes memory, the loss and the loss's gradient.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_04_gb300 as muon  # noqa: E402


class Weight:
    """A bf16 matrix [out, in] with its 8-bit copies: by rows for the forward product, transposed for the data gradient."""

    def __init__(self, rows, cols, generator):
        self.master = (torch.randn(rows, cols, device="cuda", generator=generator) / cols ** 0.5).bfloat16()
        self.refresh()

    def refresh(self):
        self.rows, self.cols = muon.fp8_quantize(self.master, square=True, rows=True, cols=True)


class Block:
    """stream -> stream + sigmoid(gate(n)) scale rms(down(silu(branch(n)) up(n))) post, n the normalised stream."""

    def __init__(self, width, hidden, g):
        self.branch, self.up, self.down = Weight(hidden, width, g), Weight(hidden, width, g), Weight(width, hidden, g)
        self.gate = Weight(width, width, g)
        self.post, self.pre, self.scale = (torch.ones(width, device="cuda") for _ in range(3))
        self.weights = [self.branch, self.up, self.down, self.gate]
        self.vectors = [self.post, self.pre, self.scale]

    def forward(self, q, stream, last):
        a = muon.gated_activation(muon.fp8_matmul(q, self.branch.rows), muon.fp8_matmul(q, self.up.rows), fp8="e4m3", y=False,
                                  checkpoint="e4m3")
        r = muon.block_norm(muon.fp8_matmul(a.q, self.down.rows), stream, self.post, self.pre, gate=muon.fp8_matmul(q, self.gate.rows),
                            scale=self.scale, fp8="e4m3", y=last, checkpoint="e4m3")
        return r, (q, a.kept, r.kept)

    def backward(self, dy, dstream, kept):
        """(gradient of n, of the stream, of the matrices (bf16), of the vectors (fp32))."""
        q, branches, norms = kept
        n = muon.block_norm_backward(dy, norms, self.post, self.pre, scale=self.scale, dh=dstream)
        d, dt = muon.fp8_quantize(n.dx, "e5m2", cols=True)
        b = muon.gated_activation_backward(muon.fp8_matmul(d, self.down.cols), branches, dense=False, fp8="e5m2", y_fp8="e4m3")
        g, gt = muon.fp8_quantize(n.dgate, "e5m2", cols=True)
        qt = muon.fp8_transpose(q)
        matrices = [muon.fp8_matmul(b.dgate_cols, qt), muon.fp8_matmul(b.dup_cols, qt), muon.fp8_matmul(dt, b.y_cols),
                    muon.fp8_matmul(gt, qt)]
        dn = muon.fp8_matmul(g, self.gate.cols)
        dn = muon.fp8_matmul(b.dgate_rows, self.branch.cols, add=dn)
        dn = muon.fp8_matmul(b.dup_rows, self.up.cols, add=dn)
        return dn, n.dresidual, matrices, [n.dpost_weight, n.dpre_weight, n.dscale]


class Network:
    def __init__(self, layers, width, hidden, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks = [Block(width, hidden, g) for _ in range(layers)]
        self.norm = torch.ones(width, device="cuda")

    @property
    def weights(self):
        return [w for b in self.blocks for w in b.weights]

    @property
    def vectors(self):
        return [self.norm] + [v for b in self.blocks for v in b.vectors]

    def forward(self, x):
        first = muon.rms_norm(x, self.norm, fp8="e4m3", y=False)
        q, stream, kept = first.q, x, []
        for i, block in enumerate(self.blocks):
            r, k = block.forward(q, stream, last=i + 1 == len(self.blocks))
            q, stream = r.q, r.h
            kept.append(k)
        return r.y, (kept, x, first.rstd)

    def backward(self, dy, saved):
        """Gradients of the matrices (bf16, in the order of `weights`) and of the vectors (fp32, in that of `vectors`)."""
        kept, x, rstd = saved
        matrices, vectors, dstream = [], [], None
        for block, k in zip(reversed(self.blocks), reversed(kept)):
            dy, dstream, m, v = block.backward(dy, dstream, k)
            matrices, vectors = m + matrices, v + vectors
        _, dnorm = muon.rms_norm_backward(dy, x, self.norm, rstd, dresidual=dstream)
        return matrices, [dnorm] + vectors


def kept_bytes(saved):
    """Bytes that the forward pass left for the backward pass, without its input."""
    def size(t):
        if t is None:
            return 0
        if isinstance(t, muon.Fp8Tensor):
            return size(t.data) + size(t.scale)
        return t.numel() * t.element_size() if isinstance(t, torch.Tensor) else sum(size(u) for u in t)
    return size(saved[0]) + size(saved[2])


def train(steps=20, tokens=2048, layers=2, width=512, hidden=1024, lr=0.05, max_norm=0.1, seed=0, log=print):
    """Losses and gradient norms of `steps` steps."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    model = Network(layers, width, hidden, seed)
    teacher = torch.randn(width, width, device="cuda", generator=g) / width ** 0.5
    updater = muon.MuonUpdater([w.master for w in model.weights], beta=0.95, lr=lr, steps=5)
    first, second = ([torch.zeros_like(v) for v in model.vectors] for _ in range(2))
    losses, norms = [], []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
        target = x.float() @ teacher
        y, saved = model.forward(x)
        diff = y.float() - target
        losses.append(diff.square().mean())
        matrices, vectors = model.backward((2 * diff / diff.numel()).bfloat16(), saved)
        norms.append(muon.clip_grads(matrices + vectors, max_norm))
        updater.step(matrices)
        muon.adamw_tail(model.vectors, vectors, first, second, lr=1e-3, weight_decay=0.0, step=step)
        for w in model.weights:
            w.refresh()
    losses, norms = torch.stack(losses).tolist(), torch.stack(norms).tolist()
    for step, (loss, norm) in enumerate(zip(losses, norms), 1):
        log(f"step {step:3d}  loss {loss:.4f}  gradient norm {norm:.3f}")
    log(f"kept for the backward pass: {kept_bytes(saved) / tokens:.0f} bytes a token")
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("steps", 20), ("tokens", 2048), ("layers", 2), ("width", 512), ("hidden", 1024)):
        ap.add_argument("--" + name, type=int, default=default)
    train(**vars(ap.parse_args()))
