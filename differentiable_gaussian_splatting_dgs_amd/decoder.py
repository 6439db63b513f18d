"""A network that decodes the 59 parameters of each Gaussian from learned
features, trained through the rasteriser.

    h = features + w2 gelu(w1 norm(features) + b1) + b2
    attributes[i] = heads[e] h[i] + hb[e]     (Gaussian i in block e of the scene)
    params = base + attributes

Gaussians are stored block by block; ``offsets[e] .. offsets[e + 1]`` are
those of block e and take its head (ragged sizes, empty blocks allowed, the
bounds on the device).  Everything between the features and the attributes,
forward and backward, runs in the library's network operators; storage is
bfloat16 (or float16, float32), master weights and their gradients float32.

``RoutedDecoder`` shares a row of features among several Gaussians and picks
each Gaussian's heads by a learned gate instead of by block:

    f = features[anchors[i]]
    h = f + w2 gelu(w1 norm(f) + b1) + b2
    attributes[i] = sum over the gate's choices e of p_e (heads[e] h[i] + hb[e])

with p the softmax of the chosen logits, gate h[i].

    python -m differentiable_gaussian_splatting_dgs_amd.decoder [steps] [routed]

trains one on the small reference scene and prints the loss of each step.
"""
from __future__ import annotations

import torch

from . import (GS_ACT_GELU, AdamW, gs_combine_bwd, gs_combine_fwd, gs_dispatch_bwd, gs_dispatch_fwd, gs_embedding_bwd,
               gs_embedding_fwd, gs_gate_bwd, gs_gate_fwd, gs_group_sort, gs_grouped_linear_bwd,
               gs_grouped_linear_fwd, gs_layer_norm_bwd, gs_layer_norm_fwd, gs_linear_bwd, gs_linear_fwd)

PLANES = 59
HEAD = 64          # a head's columns: the 59 parameters in whole 16-byte chunks
EPS = 1e-5


class AttributeDecoder:
    """Features of n Gaussians, the network, and its gradients.

    ``masters``: name -> float32 tensor (features, norm, layers, heads), with
    ``.grad`` filled (not added to) by ``backward``: hand ``parameters()`` to
    any torch.optim optimiser, then call ``sync()`` so that the storage
    copies the kernels read follow."""

    def __init__(self, offsets, width=64, hidden=256, dtype=torch.bfloat16, device="cuda", seed=0):
        self.device, self.dtype = torch.device(device), dtype
        bounds = torch.as_tensor(offsets, dtype=torch.int64).cpu()
        if bounds.dim() != 1 or bounds.numel() < 2 or bounds[0] != 0 or (bounds[1:] < bounds[:-1]).any():
            raise ValueError(f"offsets {bounds.tolist()}: (blocks + 1,) bounds from 0 on, ascending, expected")
        self.offsets = bounds.to(self.device).contiguous()
        blocks, n = bounds.numel() - 1, int(bounds[-1])
        gen = torch.Generator(device="cpu")
        gen.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen) * scale).to(self.device)

        self.masters = {
            "features": normal(n, width, scale=1.0),
            "gamma": torch.ones(width, device=self.device), "beta": torch.zeros(width, device=self.device),
            "w1": normal(hidden, width, scale=width ** -0.5), "b1": torch.zeros(hidden, device=self.device),
            "w2": normal(width, hidden, scale=hidden ** -0.5), "b2": torch.zeros(width, device=self.device),
            # small heads: training starts at the base parameters
            "heads": normal(blocks, HEAD, width, scale=0.02 * width ** -0.5),
            "hb": torch.zeros(blocks, HEAD, device=self.device),
        }
        self.stored = {k: torch.empty_like(self.masters[k], dtype=dtype) for k in ("features", "w1", "w2", "heads")}
        for v in self.masters.values():
            v.grad = torch.zeros_like(v)
        self.sync()

    def parameters(self):
        return list(self.masters.values())

    def sync(self):
        """The storage copies after a change of the masters."""
        for k, v in self.stored.items():
            v.copy_(self.masters[k])

    def optimizer(self, **kw):
        """An AdamW (``kw``: its arguments) of the masters whose step writes the
        storage copies too, so that no ``sync()`` is needed after it."""
        return AdamW(self.parameters(), copies=[self.stored.get(k) for k in self.masters], **kw)

    def _gradients(self):
        for v in self.masters.values():
            if v.grad is None:      # as an optimiser's zero_grad() leaves it
                v.grad = torch.empty_like(v)
        return {k: v.grad for k, v in self.masters.items()}

    def forward(self):
        """[n][HEAD] attributes (the first 59 columns)."""
        m, s = self.masters, self.stored
        self._n, self._mean, self._rstd = gs_layer_norm_fwd(s["features"], m["gamma"], m["beta"], EPS)
        self._a, self._z = gs_linear_fwd(self._n, s["w1"], m["b1"], GS_ACT_GELU, save_z=True)
        self._h = gs_linear_fwd(self._a, s["w2"], m["b2"], residual=s["features"])
        return gs_grouped_linear_fwd(self._h, s["heads"], self.offsets, m["hb"])

    def backward(self, dattr):
        """Gradients of every master from those of forward()'s attributes
        ([n][HEAD], of the storage type; unused columns 0)."""
        m, s, g = self.masters, self.stored, self._gradients()
        dh, _, _ = gs_grouped_linear_bwd(self._h, s["heads"], self.offsets, dattr, dw=g["heads"], db=g["hb"])
        da, _, _ = gs_linear_bwd(self._a, s["w2"], dh, dw=g["w2"], db=g["b2"])
        dn, _, _ = gs_linear_bwd(self._n, s["w1"], da, self._z, GS_ACT_GELU, dw=g["w1"], db=g["b1"])
        # the features reach h through the norm and past it
        df, _, _ = gs_layer_norm_bwd(s["features"], dn, m["gamma"], self._mean, self._rstd, dres=dh,
                                     dgamma=g["gamma"], dbeta=g["beta"])
        g["features"].copy_(df)

    def train_views(self, step, base, views=None):
        """One training pass through the rasteriser of a ``TrainStep``: decode
        its parameters (``base`` [59][n], not the step's own, + attributes),
        render and back-propagate the views, and leave the gradients in the
        masters.  Returns the views' losses (device tensor).  In float16 a
        gradient under 6e-8 is 0: raise the step's loss weights for it."""
        if base.untyped_storage().data_ptr() == step.params.untyped_storage().data_ptr():
            raise ValueError("base is the step's own parameters, which this pass overwrites: pass a copy")
        attr = self.forward()
        step.drop_next_view()       # its parameters change here
        step.params.copy_(base)
        step.params[:, :attr.shape[0]] += attr[:, :PLANES].t()
        losses = []
        for k in range(len(step.views)) if views is None else views:
            step.forward_view(k)
            step.backward_view(k)
            losses.append(step.views[k].loss.reshape(1).clone())
        dattr = torch.zeros_like(attr)
        dattr[:, :PLANES] = step.grads[:, :attr.shape[0]].t()
        step.grads.zero_()
        step.union_flags.zero_()
        self.backward(dattr)
        return torch.cat(losses)


class RoutedDecoder(AttributeDecoder):
    """Features of ``rows`` anchors, looked up by ``anchors`` ([n]; -1: a
    Gaussian without features, for which a row of zeros is decoded), and
    ``heads`` heads, ``choices`` of them for each Gaussian by the gate.  The
    masters have "gate" beside AttributeDecoder's."""

    def __init__(self, anchors, rows, heads, choices=2, width=64, hidden=256, dtype=torch.bfloat16, device="cuda",
                 seed=0):
        self.device, self.dtype, self.choices = torch.device(device), dtype, choices
        anchors = torch.as_tensor(anchors, dtype=torch.int64)
        if anchors.dim() != 1 or (anchors.numel() and not -1 <= int(anchors.min()) <= int(anchors.max()) < rows):
            raise ValueError(f"anchors of shape {tuple(anchors.shape)}: (n,) rows from -1 to {rows - 1} expected")
        if not 1 <= choices <= heads:
            raise ValueError(f"{choices} choices of {heads} heads")
        self.anchors = anchors.to(self.device).contiguous()
        gen = torch.Generator(device="cpu")
        gen.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen) * scale).to(self.device)

        self.masters = {
            "features": normal(rows, width, scale=1.0),
            "gamma": torch.ones(width, device=self.device), "beta": torch.zeros(width, device=self.device),
            "w1": normal(hidden, width, scale=width ** -0.5), "b1": torch.zeros(hidden, device=self.device),
            "w2": normal(width, hidden, scale=hidden ** -0.5), "b2": torch.zeros(width, device=self.device),
            "gate": normal(heads, width, scale=0.5 * width ** -0.5),
            "heads": normal(heads, HEAD, width, scale=0.02 * width ** -0.5),
            "hb": torch.zeros(heads, HEAD, device=self.device),
        }
        self.stored = {k: torch.empty_like(self.masters[k], dtype=dtype)
                       for k in ("features", "w1", "w2", "gate", "heads")}
        for v in self.masters.values():
            v.grad = torch.zeros_like(v)
        # which Gaussians an anchor's gradient sums over: as long as the anchors stay
        self._shares = gs_group_sort(self.anchors, rows, want_place=False)[:2]
        self.sync()

    def forward(self):
        m, s = self.masters, self.stored
        self._f = gs_embedding_fwd(s["features"], self.anchors)
        self._n, self._mean, self._rstd = gs_layer_norm_fwd(self._f, m["gamma"], m["beta"], EPS)
        self._a, self._z = gs_linear_fwd(self._n, s["w1"], m["b1"], GS_ACT_GELU, save_z=True)
        self._h = gs_linear_fwd(self._a, s["w2"], m["b2"], residual=self._f)
        self._logits = gs_linear_fwd(self._h, s["gate"])
        self._ids, self._p = gs_gate_fwd(self._logits, self.choices)
        self._offsets, _, self._place = gs_group_sort(self._ids, m["gate"].shape[0], want_order=False)
        self._hs = gs_dispatch_fwd(self._h, self._place)
        self._ys = gs_grouped_linear_fwd(self._hs, s["heads"], self._offsets, m["hb"])
        return gs_combine_fwd(self._ys, self._place, self._p)

    def backward(self, dattr):
        m, s, g = self.masters, self.stored, self._gradients()
        dys, dp = gs_combine_bwd(dattr, self._ys, self._place, self._p)
        dhs, _, _ = gs_grouped_linear_bwd(self._hs, s["heads"], self._offsets, dys, dw=g["heads"], db=g["hb"])
        dlogits = gs_gate_bwd(self._logits, self._ids, self._p, dp)
        dh, _, _ = gs_linear_bwd(self._h, s["gate"], dlogits, dw=g["gate"])
        dh = gs_dispatch_bwd(dhs, self._place, dres=dh, dx=dh)
        da, _, _ = gs_linear_bwd(self._a, s["w2"], dh, dw=g["w2"], db=g["b2"])
        dn, _, _ = gs_linear_bwd(self._n, s["w1"], da, self._z, GS_ACT_GELU, dw=g["w1"], db=g["b1"])
        df, _, _ = gs_layer_norm_bwd(self._f, dn, m["gamma"], self._mean, self._rstd, dres=dh, dgamma=g["gamma"],
                                     dbeta=g["beta"])
        gs_embedding_bwd(df, self.anchors, *self._shares, dtable=g["features"])


def shared_rows(positions, rows):
    """Anchors: the Gaussians in their order along x, in ``rows`` shares of
    about equal size."""
    x = torch.as_tensor(positions[0])
    at = torch.empty(x.numel(), dtype=torch.int64)
    at[torch.argsort(x, stable=True)] = torch.arange(x.numel())
    return at * rows // max(x.numel(), 1)


def block_offsets(positions, blocks):
    """(order, offsets): the Gaussians sorted into ``blocks`` equal slabs along
    x, the way a large scene is cut, and the slabs' bounds."""
    x = torch.as_tensor(positions[0])
    lo, hi = float(x.min()), float(x.max())
    slab = ((x - lo) * (blocks / max(hi - lo, 1e-30))).long().clamp_(0, blocks - 1)
    order = torch.argsort(slab, stable=True)
    counts = torch.bincount(slab, minlength=blocks)
    return order, torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])


def main(steps=20, routed=False):
    import synth

    from . import TrainStep
    work = synth.workload(0)
    order, offsets = block_offsets(work.params[:3], 4)
    base = torch.as_tensor(work.params)[:, order].contiguous()
    step = TrainStep(base, work.cameras, work.targets, work.w_l1, work.w_ssim, work.lr, work.beta1, work.beta2,
                     work.eps)
    if routed:
        rows = base.shape[1] // 4
        dec = RoutedDecoder(shared_rows(base[:3], rows), rows, 4, width=64, hidden=128)
        opt = dec.optimizer(lr=2e-3, weight_decay=0.0, bits=8)
    else:
        dec = AttributeDecoder(offsets, width=64, hidden=128)
        opt = torch.optim.Adam(dec.parameters(), lr=2e-3)
    base = base.to(dec.device)
    history = []
    for i in range(steps):
        loss = dec.train_views(step, base)
        opt.step()
        if not routed:
            dec.sync()
        history.append(float(loss.mean()))
        print(f"step {i}: loss {history[-1]:.6f}", flush=True)
    return history


if __name__ == "__main__":
    import sys
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 20, "routed" in sys.argv[2:])
