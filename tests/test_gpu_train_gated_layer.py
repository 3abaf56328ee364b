"""One layer of the training example's gated model backward, from the very
checkpoints that its forward pass kept: against fp64 of what their bytes stand
for, so that only roundings to bf16 are left.

Such a rounding is off by 2^-8 of a value at most, evenly: 2^-8 / sqrt 3 in the
mean square.  Roundings of different elements are independent, so that a
product's error has the norm of sqrt((a a) (b b)) times that; k of them one
behind another are allowed k 2^-8, 1.7 times their sum.  dh, then dgate and dup, then the
weights' gradients: 3.  dy and dx: 4.  h and the down projection's: 2."""

import pytest
import torch

from memory_reduced_muon_gb300 import train_block

pytestmark = pytest.mark.gpu


def _values(payload, scale):
    """A carrier's values in fp64."""
    codes = payload.view(torch.float8_e4m3fn).double().unflatten(1, (-1, 32))
    return (codes * torch.exp2(scale.double() - 127)[..., None]).flatten(1)


@pytest.mark.parametrize("rows", [1, 129, 2048])
@pytest.mark.parametrize("residual", [False, True])
def test_gradients_of_a_layer(rows, residual):
    gen = torch.Generator("cuda").manual_seed(rows)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    width, inner = 256, 512
    x, stream = (rnd(rows, width).bfloat16().requires_grad_(True) for _ in range(2))
    gain = (1 + 0.2 * rnd(width)).requires_grad_(True)
    w_gate, w_up, w_down = ((rnd(*s) * s[1] ** -0.5).bfloat16().requires_grad_(True) for s in ((inner, width), (inner, width), (width, inner)))
    total, out = train_block.NormedGatedMlp.apply(x, stream if residual else None, gain, w_gate, w_up, w_down)
    kept = out.grad_fn.saved_tensors
    dsum, dout = rnd(rows, width).bfloat16(), rnd(rows, width).bfloat16()
    leaves = [x, gain, w_gate, w_up, w_down] + ([stream] if residual else [])
    got = [g.double() for g in torch.autograd.grad((total, out), leaves, (dsum, dout))]

    sum_, g, wg, wu, wd, y8, ys, gate8, up8, gs, us = kept
    sum_, g, wg, wu, wd, d_out = (t.detach().double() for t in (sum_, g, wg, wu, wd, dout))
    y, gate, up = _values(y8, ys), _values(gate8, gs), _values(up8, us)
    s = torch.sigmoid(gate)
    a, slope = gate * s, s * (1 + gate * (1 - s))
    dh = d_out @ wd
    dgate, dup = dh * up * slope, dh * a
    dy = dgate @ wg + dup @ wu
    inv = torch.rsqrt(sum_.square().mean(1, keepdim=True) + train_block.EPS)
    n = sum_ * inv
    t = dy * g
    dx = inv * (t - n * (t * n).mean(1, keepdim=True)) + dsum.double()
    sq = torch.square
    r_dy = torch.sqrt(sq(dgate) @ sq(wg) + sq(dup) @ sq(wu))
    want = [dx, (dy * n).sum(0), dgate.T @ y, dup.T @ y, d_out.T @ (a * up)] + ([dx] if residual else [])
    rms = [torch.sqrt(sq(inv * g * r_dy) + sq(dx)), torch.sqrt((sq(r_dy) * sq(n)).sum(0)), torch.sqrt(sq(dgate).T @ sq(y)),
           torch.sqrt(sq(dup).T @ sq(y)), torch.sqrt(sq(d_out).T @ sq(a * up))]
    rms += rms[:1] if residual else []
    for what, (p, w, r, k) in zip(("dx", "dgain", "dw_gate", "dw_up", "dw_down", "dstream"), zip(got, want, rms, (4, 3, 3, 3, 2, 4))):
        assert float((p - w).norm()) <= k * 2.0 ** -8 * float(r.norm()), what
