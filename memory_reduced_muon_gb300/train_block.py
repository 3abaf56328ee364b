"""A whole training step on the library's kernels, at a small size.

``python -m memory_reduced_muon_gb300.train_block [steps] [--gated]`` trains a residual
MLP language model on synthetic tokens.  torch supplies the matrix products
and autograd; everything else is the library's:

* the RMS norms with the residual's addition, forward and backward, and, when
  the model is evaluated, the last one's MXFP8 output;
* one clipping plan over every gradient, applied in place;
* ``qmuon_step`` for the matrices;
* AdamW with fp32 states for the gains and the head, and with 8-bit states,
  rounded stochastically, for the embedding.

``--gated`` trains the model with gated MLPs instead, on more of the library's
kernels: the embedding's lookup and its gradient in a fixed order, and the
gated block with what it keeps for the backward pass in 8 bits: the norm's
output, which the norm writes as a carrier beside its 16-bit one, and the
block's two projections.  The block's output is made again from them.
"""

from __future__ import annotations

import math
import sys

import torch
import torch.nn.functional as F

import memory_reduced_muon_gb300 as q

COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-5


class RmsNorm(torch.autograd.Function):
    """(sum, y) of x + residual: the residual stream goes on as ``sum``."""

    @staticmethod
    def forward(ctx, x, residual, gain):
        rows, cols = x.shape
        total, y = torch.empty_like(x), torch.empty_like(x)
        q.qmuon_rmsnorm_forward(x, gain, rows, cols, "bf16", EPS, y=y, residual=residual, sum=total)
        ctx.save_for_backward(total, gain)
        return total, y

    @staticmethod
    def backward(ctx, dsum, dy):
        h, gain = ctx.saved_tensors
        rows, cols = h.shape
        dx, dgain = torch.empty_like(h), torch.empty_like(gain)
        ws = torch.empty(q.qmuon_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device=h.device)
        q.qmuon_rmsnorm_backward(dy.contiguous(), h, gain, rows, cols, "bf16", EPS, dx, dgain, ws,
                                 dsum=None if dsum is None else dsum.contiguous())
        return dx, dx if ctx.needs_input_grad[1] else None, dgain      # x and residual enter the sum alike


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens):
        (vocab, cols), n = table.shape, tokens.numel()
        out = torch.empty(n, cols, dtype=table.dtype, device=table.device)
        q.qmuon_embedding_forward(table, tokens, out, n, vocab, cols, "bf16")
        ctx.save_for_backward(tokens)
        ctx.vocab = vocab
        return out

    @staticmethod
    def backward(ctx, dout):
        tokens, = ctx.saved_tensors
        n, cols = dout.shape
        grad = torch.empty(ctx.vocab, cols, dtype=dout.dtype, device=dout.device)
        ws = torch.empty(q.qmuon_embedding_workspace_size(n, ctx.vocab, cols), dtype=torch.uint8, device=dout.device)
        q.qmuon_embedding_backward(dout.contiguous(), tokens, grad, n, ctx.vocab, cols, "bf16", ws)
        return grad, None


class NormedGatedMlp(torch.autograd.Function):
    """(sum, MLP of the norm) of x + residual.  Kept for the backward pass: the sum, and carriers of the norm's output and
    of both projections, a little over 2 bytes per element of the inner width."""

    @staticmethod
    def forward(ctx, x, residual, gain, w_gate, w_up, w_down):
        rows, width = x.shape
        inner = w_gate.shape[0]
        byte = lambda *s: torch.empty(*s, dtype=torch.uint8, device=x.device)   # noqa: E731
        total, y = torch.empty_like(x), torch.empty_like(x)
        y8, y_scale = byte(rows, width), byte(rows, width // 32)
        q.qmuon_rmsnorm_forward(x, gain, rows, width, "bf16", EPS, y=y, residual=residual, sum=total, payload=y8, scale_inv=y_scale)
        h = torch.empty(rows, inner, dtype=x.dtype, device=x.device)
        kept = dict(gate=byte(rows, inner), up=byte(rows, inner), gate_scale=byte(rows, inner // 32), up_scale=byte(rows, inner // 32))
        call = q.gated_ffn(y, w_gate, w_up, h, rows, width, inner, "bf16", saved="mxfp8", **kept)
        q.qmuon_gated_ffn_forward(call, byte(q.qmuon_gated_ffn_workspace_size(call)))
        ctx.save_for_backward(total, gain, w_gate, w_up, w_down, y8, y_scale, *kept.values())
        return total, h @ w_down.T

    @staticmethod
    def backward(ctx, dsum, dout):
        total, gain, w_gate, w_up, w_down, y8, y_scale, *kept = ctx.saved_tensors
        rows, width = total.shape
        inner = w_gate.shape[0]
        dout = dout.contiguous()
        dh = dout @ w_down
        dy, dw_gate, dw_up, h = torch.empty_like(total), torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(dh)
        call = q.gated_ffn_grad(dh, y8, w_gate, w_up, dy, dw_gate, dw_up, rows, width, inner, "bf16", saved="mxfp8", x_scale=y_scale, h=h,
                                **dict(zip(("gate", "up", "gate_scale", "up_scale"), kept)))
        ws = torch.empty(q.qmuon_gated_ffn_backward_workspace_size(call), dtype=torch.uint8, device=dh.device)
        q.qmuon_gated_ffn_backward(call, ws)
        dx, dgain = torch.empty_like(total), torch.empty_like(gain)
        ws = torch.empty(q.qmuon_rmsnorm_workspace_size(rows, width), dtype=torch.uint8, device=dh.device)
        q.qmuon_rmsnorm_backward(dy, total, gain, rows, width, "bf16", EPS, dx, dgain, ws, dsum=None if dsum is None else dsum.contiguous())
        return dx, dx if ctx.needs_input_grad[1] else None, dgain, dw_gate, dw_up, dout.T @ h


class Block:
    """The model, its gradients at fixed addresses, and the plans over them."""

    def __init__(self, vocab=512, width=256, layers=2, seed=0, device="cuda", gated=False):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device)   # noqa: E731
        self.vocab, self.width, self.gated = vocab, width, gated
        # fp32 masters, and the bf16 copies that the products read
        self.embed = rnd(vocab, width)
        self.head = rnd(vocab, width) * width ** -0.5
        self.gains = [torch.ones(width, device=device) for _ in range(layers + 1)]
        shapes = [(2 * width, width), (2 * width, width), (width, 2 * width)] if gated else [(4 * width, width), (width, 4 * width)]
        self.mats = [rnd(*s) * s[1] ** -0.5 for _ in range(layers) for s in shapes]
        self.embed16, self.head16 = self.embed.bfloat16(), self.head.bfloat16()
        self.mats16 = [w.bfloat16() for w in self.mats]
        self.leaves = [self.embed16, self.head16, *self.mats16, *self.gains]
        for p in self.leaves:
            p.requires_grad_(True)
            p.grad = torch.zeros_like(p)
        zeros = lambda p, dt: torch.zeros(p.numel(), dtype=dt, device=device)   # noqa: E731
        blocks = -(-self.embed.numel() // 256)
        dt = {torch.bfloat16: "bf16", torch.float32: "f32"}
        self.clip = q.qmuon_clip_plan_create([(p.grad, dt[p.dtype]) for p in self.leaves])
        self.clip_ws = torch.empty(q.qmuon_clip_workspace_size(self.clip), dtype=torch.uint8, device=device)
        self.norm = torch.zeros(2, device=device)
        self.adam = q.qmuon_adamw_plan_create(
            [q.adamw_tensor(self.head, self.head16.grad, zeros(self.head, torch.float32), zeros(self.head, torch.float32),
                            self.head.numel(), "bf16", copy=self.head16, weight_decay=0.1)] +
            [q.adamw_tensor(w, w.grad, zeros(w, torch.float32), zeros(w, torch.float32), w.numel(), "f32") for w in self.gains])
        self.adam8 = q.qmuon_adamw_plan_create(
            [q.adamw_tensor(self.embed, self.embed16.grad, zeros(self.embed, torch.uint8), zeros(self.embed, torch.uint8),
                            self.embed.numel(), "bf16", torch.zeros(blocks, device=device), torch.zeros(blocks, device=device),
                            copy=self.embed16)], "e4m3")
        self.muon = q.qmuon_plan_create(
            [(torch.zeros(w.numel(), dtype=torch.int8, device=device), torch.zeros(-(-w.numel() // 256), device=device), p.grad,
              *w.shape) for w, p in zip(self.mats, self.mats16)])
        self.muon_ws = torch.empty(q.qmuon_workspace_size(self.muon, q.QMUON_WS_STEP), dtype=torch.uint8, device=device)
        self.t = 0

    def hidden(self, tokens):
        """The residual stream and the last MLP's output, before the final norm."""
        if self.gated:
            x, stream = Embedding.apply(self.embed16, tokens), None
            for i in range(len(self.mats) // 3):
                stream, x = NormedGatedMlp.apply(x, stream, self.gains[i], *self.mats16[3 * i:3 * i + 3])
            return stream, x
        x, stream = F.embedding(tokens, self.embed16), None
        for i in range(len(self.mats) // 2):
            stream, y = RmsNorm.apply(x, stream, self.gains[i])
            x = F.silu(y @ self.mats16[2 * i].T) @ self.mats16[2 * i + 1].T
        return stream, x

    def loss(self, tokens, targets):
        stream, x = self.hidden(tokens)
        _, y = RmsNorm.apply(x, stream, self.gains[-1])
        return F.cross_entropy((y @ self.head16.T).float(), targets)

    @torch.no_grad()
    def loss_mxfp8(self, tokens, targets):
        """The loss with the final norm's output in 8 bits."""
        stream, x = self.hidden(tokens)
        rows, cols = x.shape
        payload = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
        scale = torch.empty(rows, cols // 32, dtype=torch.uint8, device=x.device)
        q.qmuon_rmsnorm_forward(x, self.gains[-1], rows, cols, "bf16", EPS, residual=stream, payload=payload, scale_inv=scale)
        y = payload.view(torch.float8_e4m3fn).float().view(rows, -1, 32) * torch.exp2(scale.float() - 127)[..., None]
        return F.cross_entropy((y.view(rows, cols).bfloat16() @ self.head16.T).float(), targets)

    def step(self, tokens, targets, lr=3e-3, eta=0.02, max_norm=1.0):
        """One training step; the loss, on the device.  A step whose gradients are not finite changes nothing."""
        for p in self.leaves:
            p.grad.zero_()        # autograd adds into the plans' buffers
        loss = self.loss(tokens, targets)
        loss.backward()
        q.qmuon_grad_clip(self.clip, max_norm, True, self.norm, self.clip_ws)
        # AdamW alone could take the coefficient on the device, and changes nothing where that is not finite; the Muon
        # step takes none, so the host looks at the norm.  The gradients are scaled already.
        if not math.isfinite(self.norm[0].item()):
            return loss.detach()
        self.t += 1
        q.qmuon_adamw_step(self.adam, self.t, lr, 0.9, 0.95, 1e-8)
        q.qmuon_adamw_step_sr(self.adam8, self.t, lr, 0.9, 0.95, 1e-8, 17)
        q.qmuon_step(self.muon, self.t, 1, 0.95, eta, eta, self.mats, COEFFS, 5, None, self.muon_ws)
        with torch.no_grad():
            for p, w in zip(self.mats16, self.mats):
                p.copy_(w)
        return loss.detach()


def batches(vocab, rows, seed, device="cuda"):
    """Tokens and their successors under a fixed random permutation, one in ten replaced by noise."""
    g = torch.Generator(device=device).manual_seed(seed)
    follows = torch.randperm(vocab, generator=g, device=device)
    while True:
        x = torch.randint(0, vocab, (rows,), generator=g, device=device)
        noise = torch.randint(0, vocab, (rows,), generator=g, device=device)
        yield x, torch.where(torch.rand(rows, generator=g, device=device) < 0.1, noise, follows[x])


def train(steps=200, rows=2048, seed=0, every=0, gated=False):
    """Losses of the first and the last step, and the last model's with an 8-bit final norm."""
    model = Block(seed=seed, gated=gated)
    data = batches(model.vocab, rows, seed + 1)
    first = last = math.nan
    for i in range(steps):
        loss = model.step(*next(data))
        if i == 0:
            first = float(loss)
        if every and i % every == 0:
            print(f"step {i:4d}  loss {float(loss):.4f}  norm {float(model.norm[0]):.3f}")
    q.qmuon_sync_status(model.muon_ws)
    x, y = next(data)
    with torch.no_grad():
        last = float(model.loss(x, y))
    return first, last, float(model.loss_mxfp8(x, y))


if __name__ == "__main__":
    args = [a for a in sys.argv[1:] if a != "--gated"]
    n = int(args[0]) if args else 200
    first, last, last8 = train(n, every=max(1, n // 10), gated="--gated" in sys.argv)
    print(f"loss {first:.4f} -> {last:.4f} after {n} steps ({last8:.4f} with the final norm's output in MXFP8)")
