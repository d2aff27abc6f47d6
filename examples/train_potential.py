"""A training loop of a small invariant potential with the operators of this
package, forward and backward, on one GPU:

    species -> embed_fwd -> x [N][1][C]
    x, spherical harmonics, radial weights -> conv_fwd (per-path outputs)
    -> path_mix_fwd (the trained matrices Wmix [P][C][C_out]) -> z
    z's l = 0 rows -> norm_act_fwd per structure -> h
    energy of a structure = sum over its atoms of <h, w_out>

and back: norm_act_bwd, path_mix_bwd, conv_bwd, embed_bwd.  Wmix takes the
orthogonalised momentum as its step, the other parameters plain gradient steps.
The data are random clusters of a few species, several structures to a batch;
their energies come from a fixed pair potential between species.

    python examples/train_potential.py [--steps 200] [--channels 64]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import clebsch_gordan_tensor_cgtp_amd as cg

SPECIES, CUTOFF = 6, 3.0


def batch(structures, seed, device):
    """Random clusters of 6 to 30 atoms: species, edges within the cutoff sorted
    by receiver, structure offsets, energies (mean 0, deviation 1)."""
    rng = np.random.default_rng(seed)
    strength = np.random.default_rng(7).normal(size=(SPECIES, SPECIES))
    species, row_ptr, src, r, seg, energy = [], [0], [], [], [0], []
    for _ in range(structures):
        n = int(rng.integers(6, 31))
        pos = rng.uniform(0, (n / 0.08) ** (1 / 3), size=(n, 3))
        s = rng.integers(0, SPECIES, n)
        d = pos[None, :, :] - pos[:, None, :]            # receiver, sender
        dist = np.linalg.norm(d, axis=2) + 10 * CUTOFF * np.eye(n)
        near = dist < CUTOFF
        pair = np.where(near, np.exp(-dist ** 2 / 2) * (strength + strength.T)[s][:, s], 0.0)
        energy.append(pair.sum() / n ** 0.5)
        for i in range(n):
            j = np.nonzero(near[i])[0]
            src.append(j + seg[-1])
            r.append(d[i, j])
            row_ptr.append(row_ptr[-1] + j.size)
        species.append(s)
        seg.append(seg[-1] + n)
    energy = np.array(energy)
    t = lambda a, k: torch.from_numpy(np.ascontiguousarray(a, dtype=k)).to(device)  # noqa: E731
    return {"species": t(np.concatenate(species), np.int32), "row_ptr": t(row_ptr, np.int32),
            "src": t(np.concatenate(src), np.int32), "r": t(np.concatenate(r), np.float32),
            "seg": t(seg, np.int32), "energy": t((energy - energy.mean()) / energy.std(), np.float32)}


class Potential:
    """The model's plan and parameters, its energies and its gradients."""

    def __init__(self, channels, out_channels, groups, device, seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.plan = cg.Plan(0, 2, 2, channels, path_outputs=True)
        self.groups, self.channels = groups, channels
        P = self.plan.num_paths
        self.params = {"table": rnd(SPECIES, channels), "Wmix": rnd(P, channels, out_channels) / channels ** 0.5,
                       "gamma": torch.ones(out_channels, device=device),
                       "beta": torch.zeros(out_channels, device=device), "w_out": 0.01 * rnd(out_channels)}
        # fixed radial weights per path and channel: Gaussians of the distance
        self.centre, self.width = 0.5 + CUTOFF * torch.rand(P, channels, generator=g, device=device), 0.5

    def forward(self, b):
        p, plan = self.params, self.plan
        x = cg.embed_fwd(b["species"], p["table"], self.channels ** -0.5).view(-1, 1, self.channels)
        dist = b["r"].norm(dim=1)[:, None, None]
        W = torch.exp(-((dist - self.centre) / self.width) ** 2)
        Y = plan.sh(b["r"])
        ws = plan.graph_prepare(b["row_ptr"], b["src"])
        mid = plan.conv_fwd(b["row_ptr"], b["src"], x, Y, W, ws)
        z = plan.path_mix_fwd(mid, p["Wmix"])
        h, mean, rstd = cg.norm_act_fwd(z[:, 0, :], p["gamma"], p["beta"], self.groups, b["seg"])
        atom = h @ p["w_out"]
        total = torch.cumsum(torch.cat([atom.new_zeros(1), atom]), 0)
        energy = total[b["seg"][1:].long()] - total[b["seg"][:-1].long()]
        return energy, (x, W, Y, ws, mid, z, h, mean, rstd)

    def backward(self, b, grad_energy, kept):
        """Gradients of the parameters for dL/denergy of each structure."""
        p, plan = self.params, self.plan
        x, W, Y, ws, mid, z, h, mean, rstd = kept
        counts = (b["seg"][1:] - b["seg"][:-1]).long()
        grad_atom = torch.repeat_interleave(grad_energy, counts, output_size=h.shape[0])
        grad_h = grad_atom[:, None] * p["w_out"]
        grad_z = torch.zeros_like(z)
        _, grad_gamma, grad_beta = cg.norm_act_bwd(z[:, 0, :], mean, rstd, p["gamma"], p["beta"], grad_h, self.groups,
                                                   b["seg"], grad_x=grad_z[:, 0, :])
        grad_mid, grad_Wmix = plan.path_mix_bwd(mid, p["Wmix"], grad_z)
        grad_x = plan.conv_bwd(b["row_ptr"], b["src"], x, Y, W, grad_mid, ws, want=("dx",))[0]
        grad_table = cg.embed_bwd(b["species"], grad_x[:, 0, :], SPECIES, self.channels ** -0.5)
        return {"table": grad_table, "Wmix": grad_Wmix, "gamma": grad_gamma, "beta": grad_beta,
                "w_out": h.t().contiguous() @ grad_atom}


def train(steps=40, channels=64, out_channels=64, groups=8, structures=64, device=None, log=print):
    """The mean squared error of every step."""
    device = torch.device(device or "cuda:0")
    model = Potential(channels, out_channels, groups, device)
    momentum = torch.zeros_like(model.params["Wmix"])
    data = [batch(structures, seed, device) for seed in range(4)]
    losses = []
    for step in range(steps):
        b = data[step % len(data)]
        energy, kept = model.forward(b)
        error = energy - b["energy"]
        losses.append(float((error * error).mean()))
        grads = model.backward(b, 2 * error / error.numel(), kept)
        momentum.mul_(0.9).add_(grads["Wmix"])
        rate = 0.02 * (1 - step / steps)
        model.params["Wmix"].sub_(rate * cg.orthogonalize(momentum))
        for name in ("table", "gamma", "beta", "w_out"):
            g = grads[name]
            model.params[name].sub_(rate * g / (g.norm() + 1e-6))
        if log and (step % 5 == 0 or step + 1 == steps):
            log(f"step {step:3d}  mean squared error {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--channels", type=int, default=64)
    a = ap.parse_args()
    train(a.steps, a.channels)
