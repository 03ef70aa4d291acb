"""Training splat features through a mixture-of-experts head.

A render of 3 colours and D feature channels per pixel goes through a head --
layer norm over the feature channels (read in place from the wider image), a
router, two products per chosen expert with a ReLU between them, and the
weighted sum of the experts' answers -- whose loss is differentiated back to
every splat's features.  Only pixels that some splat reaches enter the
experts.  Every call is one of tile_gaussian_splat_gb300.binding; plain torch
does the router's small product, its softmax and the updates.

With "8" the head is EightBitHead: the library's router with a balance loss,
and the experts' products of rows kept in 8 bits.

    python examples/feature_head.py [steps] [8]
"""

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tile_gaussian_splat_gb300 import binding as gs  # noqa: E402
from tile_gaussian_splat_gb300 import scenes  # noqa: E402


class FeatureHead:
    """y = sum over the topk experts e of softmax(router)[e] * (W2[e]
    relu(W1[e] n + b1[e]) + b2[e]), n = the layer norm of a pixel's features.
    forward and backward on one stream, parameters in `params`, their
    gradients in `grads`, what the kernels report in `status`."""

    def __init__(self, features, hidden, out, experts, topk=2, seed=0, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        mat = lambda *s: torch.randn(s, generator=g, device=device) / s[-1] ** 0.5
        zeros = lambda *s: torch.zeros(s, device=device)
        self.topk, self.experts = topk, experts
        self.status = gs.new_status(device)
        self.params = dict(
            norm_w=torch.ones(features, device=device), norm_b=zeros(features),
            router=mat(experts, features), w1=mat(experts, hidden, features),
            b1=zeros(experts, hidden), w2=mat(experts, out, hidden), b2=zeros(experts, out))

    def forward(self, x, reached):
        """x (..., features), a channel slice of an image; reached: the pixels
        that take part (the others answer 0)."""
        p = self.params
        norm, mean, rstd = gs.gs_layer_norm_fwd(x, p["norm_w"], p["norm_b"])
        rows = norm.reshape(-1, norm.shape[-1])
        top, ids = torch.topk(rows @ p["router"].t(), self.topk, dim=1)
        weights = torch.softmax(top, 1)
        chosen = torch.where(reached.reshape(-1, 1), ids, -1).to(torch.int32)
        offsets, _, slots = gs.gs_expert_sort(chosen, self.experts)
        st = self.status
        xs = gs.gs_expert_dispatch(rows, slots, offsets, d_status=st)
        h = gs.gs_expert_linear_fwd(xs, offsets, p["w1"], p["b1"], d_status=st).relu_()
        ys = gs.gs_expert_linear_fwd(h, offsets, p["w2"], p["b2"], d_status=st)
        y = gs.gs_expert_combine(ys, slots, weights, d_status=st)
        self.kept = (x, mean, rstd, rows, ids, weights, offsets, slots, xs, h, ys)
        return y.reshape(*x.shape[:-1], -1)

    def backward(self, grad_y, grad_x):
        """Fills `grads` and grad_x (x's shape, such as the channel slice of
        the render's gradient) from the gradient of forward's answer."""
        p = self.params
        x, mean, rstd, rows, ids, weights, offsets, slots, xs, h, ys = self.kept
        gy = grad_y.reshape(rows.shape[0], -1)
        st = self.status
        gys, gw = gs.gs_expert_combine_bwd(gy, ys, slots, weights, offsets, d_status=st)
        gh, g_w2, g_b2 = gs.gs_expert_linear_bwd(gys, h, offsets, p["w2"], d_status=st)
        gh *= h > 0
        gxs, g_w1, g_b1 = gs.gs_expert_linear_bwd(gh, xs, offsets, p["w1"], d_status=st)
        g_rows = gs.gs_expert_combine(gxs, slots, d_status=st)  # the dispatch's adjoint
        # softmax over the chosen, then the router's product
        g_top = weights * (gw - (weights * gw).sum(1, keepdim=True))
        g_logits = torch.zeros((rows.shape[0], self.experts), device=rows.device)
        g_logits.scatter_(1, ids, g_top)
        g_router = g_logits.t() @ rows
        g_rows += g_logits @ p["router"]
        _, g_nw, g_nb = gs.gs_layer_norm_bwd(g_rows.reshape(x.shape), x, p["norm_w"], mean, rstd,
                                             out=grad_x)
        self.grads = dict(norm_w=g_nw, norm_b=g_nb, router=g_router, w1=g_w1, b1=g_b1, w2=g_w2,
                          b2=g_b2)

    def step(self, rate):
        for k, g in self.grads.items():
            self.params[k] -= rate * g


class EightBitHead(FeatureHead):
    """The same head with rows and weights of the experts' products in 8 bits,
    forward and backward (what the backward needs of a product is kept in 8
    bits only), the choice of experts by the library's router, and `balance`
    times its balance loss added to the loss.  The updates go to the float32
    parameters, as if the rounding to 8 bits were not there."""

    def __init__(self, *args, balance=0.01, **kwargs):
        super().__init__(*args, **kwargs)
        self.balance = torch.full((1,), balance, device=self.status.device)

    def forward(self, x, reached):
        p, st = self.params, self.status
        norm, mean, rstd = gs.gs_layer_norm_fwd(x, p["norm_w"], p["norm_b"])
        rows = norm.reshape(-1, norm.shape[-1])
        logits = rows @ p["router"].t()
        ids, weights, counts, self.balance_loss = gs.gs_expert_route_fwd(
            logits, self.topk, keep=reached.reshape(-1))
        offsets, _, slots = gs.gs_expert_sort(ids, self.experts)
        w1, w2 = gs.gs_rows_pack8(p["w1"]), gs.gs_rows_pack8(p["w2"])
        # 8-bit rows are dispatched as rows of 16-bit elements
        xs = [gs.gs_expert_dispatch(t.view(torch.float16), slots, offsets, d_status=st).view(t.dtype)
              for t in gs.gs_rows_pack8(rows)]
        h = gs.gs_expert_linear8_fwd(*xs, offsets, *w1, rows.shape[1], p["b1"],
                                     dtype=torch.float32, d_status=st).relu_()
        h8 = gs.gs_rows_pack8(h)
        ys = gs.gs_expert_linear8_fwd(*h8, offsets, *w2, h.shape[1], p["b2"], dtype=torch.float32,
                                      d_status=st)
        y = gs.gs_expert_combine(ys, slots, weights, d_status=st)
        self.kept = (x, mean, rstd, rows, logits, ids, weights, counts, offsets, slots, xs, h8, w1,
                     w2, ys)
        return y.reshape(*x.shape[:-1], -1)

    def backward(self, grad_y, grad_x):
        p, st = self.params, self.status
        (x, mean, rstd, rows, logits, ids, weights, counts, offsets, slots, xs, h8, w1, w2,
         ys) = self.kept
        hidden = p["w1"].shape[1]
        gy = grad_y.reshape(rows.shape[0], -1)
        gys, gw = gs.gs_expert_combine_bwd(gy, ys, slots, weights, offsets, d_status=st)
        gh, g_w2, g_b2 = gs.gs_expert_linear8_bwd(gys, *h8, offsets, *w2, hidden, d_status=st)
        gh *= gs.gs_rows_unpack8(*h8, hidden, torch.float32) > 0
        gxs, g_w1, g_b1 = gs.gs_expert_linear8_bwd(gh, *xs, offsets, *w1, rows.shape[1],
                                                   d_status=st)
        g_rows = gs.gs_expert_combine(gxs, slots, d_status=st)
        g_logits = gs.gs_expert_route_bwd(logits, ids, counts, gw, self.balance, d_status=st)
        g_rows += g_logits @ p["router"]
        _, g_nw, g_nb = gs.gs_layer_norm_bwd(g_rows.reshape(x.shape), x, p["norm_w"], mean, rstd,
                                             out=grad_x)
        self.grads = dict(norm_w=g_nw, norm_b=g_nb, router=g_logits.t() @ rows, w1=g_w1, b1=g_b1,
                          w2=g_w2, b2=g_b2)


def render(d, scene, colors):
    """(image (C, H, W, channels), alphas, what the backward needs)."""
    status = gs.new_status(colors.device)
    _, keys, ids = gs.gs_isect_tiles(d["means2d"], d["radii"], d["depths"], scene.tile_size,
                                     scene.tile_width, scene.tile_height, d_status=status)
    offsets = gs.gs_tile_offsets(keys, scene.C, scene.tile_width, scene.tile_height,
                                 d_status=status)
    rgb, alphas, last = gs.gs_rasterize_fwd(
        d["means2d"], d["conics"], colors, d["opacities"], None, None, scene.width, scene.height,
        scene.tile_size, offsets, ids, scene.alpha_cutoff, scene.transmittance_threshold,
        d_status=status)
    gs.check_status(status, "render")
    return rgb, alphas, (offsets, ids, last)


def render_grad(d, scene, colors, alphas, kept, grad_image):
    """The gradient of the splats' channels."""
    offsets, ids, last = kept
    status = gs.new_status(colors.device)
    grads = gs.gs_rasterize_bwd(
        d["means2d"], d["conics"], colors, d["opacities"], None, None, scene.width, scene.height,
        scene.tile_size, offsets, ids, scene.alpha_cutoff, alphas, last, grad_image,
        torch.zeros_like(alphas), d_status=status)
    gs.check_status(status, "render_grad")
    return grads["grad_colors"]


def train(steps=30, features=32, hidden=96, out=8, experts=8, width=96, height=64, rate=0.5,
          seed=0, head_type=None):
    """Fits the head and the splats' features to a smooth target image; returns
    the loss of every step."""
    scene = scenes.random_small(seed, C=1, N=600, W=width, H=height, sigma=(1.0, 8.0),
                                channels=3 + features)
    d = {k: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()
         for k, v in scene.arrays().items()}
    colors = d["colors"].clone()
    yy, xx = torch.meshgrid(torch.linspace(0, 3, height), torch.linspace(0, 3, width),
                            indexing="ij")
    k = torch.arange(1, out + 1)
    target = torch.sin(xx[..., None] * k / 2 + yy[..., None]).cuda()[None]
    head = (head_type or FeatureHead)(features, hidden, out, experts, seed=seed)
    losses = []
    for _ in range(steps):
        image, alphas, kept = render(d, scene, colors)
        reached = alphas[..., 0] > 0
        y = head.forward(image[..., 3:], reached)
        diff = (y - target) * reached[..., None]
        n = reached.sum() * out
        losses.append(float((diff * diff).sum() / n))
        grad_image = torch.zeros_like(image)  # no loss on the three colours
        head.backward(2 * diff / n, grad_image[..., 3:])
        grad_colors = render_grad(d, scene, colors, alphas, kept, grad_image)
        gs.check_status(head.status, "feature head")  # before anything is updated
        colors -= 20 * rate * grad_colors
        head.step(rate)
    return losses


if __name__ == "__main__":
    count = int(sys.argv[1]) if len(sys.argv) > 1 else 30
    kind = EightBitHead if "8" in sys.argv[2:] else None
    for i, loss in enumerate(train(count, head_type=kind)):
        print(f"step {i:3d}  loss {loss:.4f}")
