"""A residual MLP trained with the package's operators: RMS norms that write 8-bit activations, 8-bit products forward
and backward, gradients clipped by their global norm, Muon for the matrices and AdamW for the norms' weights.

    python examples/fp8_training_step.py --steps 20

The model learns a fixed random linear map of normal inputs.  Of torch it takes memory, the activation, the loss and
the loss's gradient.
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


class Mlp:
    """stream -> stream + down(silu(up(norm(stream)))), `layers` times, and a final norm."""

    def __init__(self, layers, width, hidden, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.up = [Weight(hidden, width, g) for _ in range(layers)]
        self.down = [Weight(width, hidden, g) for _ in range(layers)]
        self.norms = [torch.ones(width, device="cuda") for _ in range(layers + 1)]

    @property
    def weights(self):
        return [w for pair in zip(self.up, self.down) for w in pair]

    def forward(self, x):
        kept, stream, branch = [], x, None
        for up, down, norm in zip(self.up, self.down, self.norms):
            r = muon.rms_norm(stream, norm, residual=branch, fp8="e4m3")
            u = muon.fp8_matmul(r.q, up.rows)
            a = torch.nn.functional.silu(u)
            stream, branch = r.h, muon.fp8_matmul(muon.fp8_quantize(a)[0], down.rows)
            kept.append((r, u, a))
        last = muon.rms_norm(stream, self.norms[-1], residual=branch)
        return last.y, (kept, last)

    def backward(self, dy, saved):
        """Gradients of the matrices (bf16, in the order of `weights`) and of the norms' weights (fp32)."""
        kept, last = saved
        matrices, norms = [], []
        dstream, dnorm = muon.rms_norm_backward(dy, last.h, self.norms[-1], last.rstd)
        norms.append(dnorm)
        for (r, u, a), up, down, norm in zip(reversed(kept), reversed(self.up), reversed(self.down), reversed(self.norms[:-1])):
            d, dt = muon.fp8_quantize(dstream, "e5m2", cols=True)      # the branch's gradient is the stream's
            da = muon.fp8_matmul(d, down.cols)
            ddown = muon.fp8_matmul(dt, muon.fp8_quantize(a, rows=False, cols=True)[1])
            s = torch.sigmoid(u.float())
            du = (da.float() * s * (1 + u.float() * (1 - s))).bfloat16()
            d, dt = muon.fp8_quantize(du, "e5m2", cols=True)
            dup = muon.fp8_matmul(dt, muon.fp8_quantize(r.y, rows=False, cols=True)[1])
            dstream, dnorm = muon.rms_norm_backward(muon.fp8_matmul(d, up.cols), r.h, norm, r.rstd, dresidual=dstream)
            matrices = [dup, ddown] + matrices
            norms.insert(0, dnorm)
        return matrices, norms


def train(steps=20, tokens=2048, layers=2, width=512, hidden=1024, lr=0.05, max_norm=0.1, seed=0, log=print):
    """Losses and gradient norms of `steps` steps."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    model = Mlp(layers, width, hidden, seed)
    teacher = torch.randn(width, width, device="cuda", generator=g) / width ** 0.5
    updater = muon.MuonUpdater([w.master for w in model.weights], beta=0.95, lr=lr, steps=5)
    first, second = ([torch.zeros_like(n) for n in model.norms] for _ in range(2))
    losses, norms = [], []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
        target = x.float() @ teacher
        y, saved = model.forward(x)
        diff = y.float() - target
        losses.append(diff.square().mean())
        matrices, tail = model.backward((2 * diff / diff.numel()).bfloat16(), saved)
        norms.append(muon.clip_grads(matrices + tail, max_norm))
        updater.step(matrices)
        muon.adamw_tail(model.norms, tail, first, second, lr=1e-3, weight_decay=0.0, step=step)
        for w in model.weights:
            w.refresh()
    losses, norms = torch.stack(losses).tolist(), torch.stack(norms).tolist()
    for step, (loss, norm) in enumerate(zip(losses, norms), 1):
        log(f"step {step:3d}  loss {loss:.4f}  gradient norm {norm:.3f}")
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("steps", 20), ("tokens", 2048), ("layers", 2), ("width", 512), ("hidden", 1024)):
        ap.add_argument("--" + name, type=int, default=default)
    train(**vars(ap.parse_args()))
