"""What the binding refuses of a model's tensors in the clipping, AdamW and RMS
norm entries: types, strides, sizes and places that do not hold what the call
reads and writes.  Nothing is launched by any of them."""

import pytest
import torch

import memory_reduced_muon_gb300 as q

ROWS, COLS = 6, 64
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8


def _refused(call, *words):
    with pytest.raises(q.QmuonError) as e:
        call()
    assert e.value.status == q.QMUON_ERR_INVALID_ARGUMENT
    for w in words:
        assert w in str(e.value), (w, str(e.value))


def test_tensors_that_are_not_on_the_gpu_are_refused():
    x, gain = torch.zeros(ROWS, COLS, dtype=BF16), torch.ones(COLS)
    _refused(lambda: q.qmuon_rmsnorm_forward(x, gain, ROWS, COLS, "bf16", 1e-5, y=x, stream=0), "x has to be", "cpu")
    _refused(lambda: q.qmuon_rmsnorm_backward(x, x, gain, ROWS, COLS, "bf16", 1e-5, x, gain, x, stream=0), "dy has to be", "cpu")
    _refused(lambda: q.qmuon_clip_plan_create([(x, "bf16")]), "gradient", "cpu")
    _refused(lambda: q.adamw_tensor(gain, x, gain, gain, COLS), "param", "cpu")


def test_numbers_that_do_not_fit_are_refused():
    p = 0x7F0000000000      # never dereferenced
    for rows, eps in ((1 << 70, 1e-5), (1.5, 1e-5), (1, 1e300)):
        _refused(lambda: q.qmuon_rmsnorm_forward(p, p, rows, COLS, "bf16", eps, y=p, stream=0))
        _refused(lambda: q.qmuon_rmsnorm_backward(p, p, p, rows, COLS, "bf16", eps, p, p, p, ws_bytes=1 << 20, stream=0))
    _refused(lambda: q.qmuon_rmsnorm_forward(p, p, 1, COLS, "e4m3", 1e-5, y=p, stream=0))
    _refused(lambda: q.qmuon_rmsnorm_forward(p, p, 1, COLS, 7, 1e-5, y=p, stream=0))


@pytest.mark.gpu
def test_forward_refuses_and_takes():
    x = torch.randn(ROWS, COLS, device="cuda").to(BF16)
    gain = torch.ones(COLS, device="cuda")
    wide = torch.zeros(ROWS, 2 * COLS, dtype=BF16, device="cuda")
    pay, sc = torch.zeros(ROWS, COLS, dtype=U8, device="cuda"), torch.zeros(ROWS, COLS // 32, dtype=U8, device="cuda")

    def call(**kw):
        a = dict(x=x, gain=gain, y=torch.zeros_like(x))
        a.update(kw)
        q.qmuon_rmsnorm_forward(a.pop("x"), a.pop("gain"), ROWS, COLS, "bf16", 1e-5, **a)
        torch.cuda.synchronize()
        return a.get("y")
    _refused(lambda: call(gain=gain.to(BF16)), "gain has to be", "bfloat16")        # would be read past its end
    _refused(lambda: call(gain=gain[:-1]), "gain")
    _refused(lambda: call(gain=torch.ones(2 * COLS, device="cuda")[::2]), "gain")
    for name in ("x", "residual", "sum", "y"):
        _refused(lambda: call(**{name: torch.zeros(ROWS, COLS, device="cuda")}), f"{name} has to be", "float32")
        _refused(lambda: call(**{name: wide[:, :COLS]}), f"{name} has to be", "strides (128, 1)")       # no ld
        _refused(lambda: call(**{name: wide[:, :COLS], "ld_" + name: 2 * COLS + 8}), name)
        _refused(lambda: call(**{name: wide[:, ::2], "ld_" + name: 2 * COLS}), name)
        _refused(lambda: call(**{name: x[:-1]}), name)
        _refused(lambda: call(**{name: x.t()}), name)
        _refused(lambda: call(**{name: x.cpu()}), name, "cpu")
    for kw in (dict(payload=pay[:, :-1], scale_inv=sc), dict(payload=pay[:-1], scale_inv=sc), dict(payload=pay, scale_inv=sc[:-1]),
               dict(payload=pay.float(), scale_inv=sc)):
        _refused(lambda: call(**kw))
    # what is laid out as the arguments say is taken, however it came about
    want = call()
    wide[:, :COLS] = x
    assert torch.equal(call(x=wide[:, :COLS], ld_x=2 * COLS), want)
    assert torch.equal(call(x=x.view(2, 3, COLS)), want)
    out = torch.zeros_like(wide)
    call(y=out[:, :COLS], ld_y=2 * COLS)
    assert torch.equal(out[:, :COLS], want) and not bool(out[:, COLS:].any())
    call(y=out.view(-1)[1:1 + 5 * 2 * COLS + COLS], ld_y=2 * COLS)       # rows of a flat buffer that ends with the last one
    assert torch.equal(call(x=x.data_ptr(), gain=gain.data_ptr()), want)
    q.qmuon_rmsnorm_forward(x, gain, ROWS, COLS, "bf16", 1e-5, payload=pay.view(torch.float8_e4m3fn), scale_inv=sc)
    one = wide[:1, :COLS]
    q.qmuon_rmsnorm_forward(one, gain, 1, COLS, "bf16", 1e-5, y=torch.zeros(COLS, dtype=BF16, device="cuda"))
    col = wide[:, :1]
    q.qmuon_rmsnorm_forward(col, gain, ROWS, 1, "bf16", 1e-5, y=torch.zeros(ROWS, dtype=BF16, device="cuda"), ld_x=2 * COLS)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_backward_refuses():
    x = torch.randn(ROWS, COLS, device="cuda").to(BF16)
    gain = torch.ones(COLS, device="cuda")
    ws = torch.empty(q.qmuon_rmsnorm_workspace_size(ROWS, COLS), dtype=U8, device="cuda")

    def call(**kw):
        a = dict(dy=x, h=x, gain=gain, dx=torch.zeros_like(x), dgain=torch.zeros_like(gain), ws=ws)
        a.update(kw)
        q.qmuon_rmsnorm_backward(a.pop("dy"), a.pop("h"), a.pop("gain"), ROWS, COLS, "bf16", 1e-5, a.pop("dx"), a.pop("dgain"),
                                 a.pop("ws"), **a)
    call()
    for name in ("dy", "h", "dx", "dsum"):
        for bad in (x.float(), x[:-1], x.t(), x.cpu(), x[:, :-1]):
            _refused(lambda: call(**{name: bad}), f"{name} has to be")
    for name in ("gain", "dgain"):
        for bad in (gain.to(BF16), gain[:-1], gain.cpu()):
            _refused(lambda: call(**{name: bad}), f"{name} has to be")
    _refused(lambda: call(ws=ws.cpu()), "ws")
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_plans_and_scalars_refuse():
    g = torch.zeros(64, 64, device="cuda")
    _refused(lambda: q.qmuon_clip_plan_create([(g, "bf16")]), "gradient")
    _refused(lambda: q.qmuon_clip_plan_create([(g[:, 1:], "f32")]), "gradient")
    clip = q.qmuon_clip_plan_create([(g.t().t(), "f32"), (g[3], "f32")])
    ws = torch.empty(q.qmuon_clip_workspace_size(clip), dtype=U8, device="cuda")
    for norm in (torch.zeros(2, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(2)):
        _refused(lambda: q.qmuon_grad_clip(clip, 1.0, False, norm, ws), "norm")
    _refused(lambda: q.qmuon_grad_clip(clip, 1.0, False, torch.zeros(2, device="cuda"), ws.cpu()), "ws")
    n = 300
    z = lambda k, dt=F32: torch.zeros(k, dtype=dt, device="cuda")   # noqa: E731
    good = dict(param=z(n), grad=z(n, BF16), m=z(n), v=z(n), numel=n, grad_dtype="bf16", copy=z(n, BF16))
    for name, bad in (("param", z(n, BF16)), ("param", z(n - 1)), ("grad", z(n)), ("grad", z(2 * n, BF16)[::2]), ("copy", z(n)),
                      ("copy", z(n, torch.float16))):
        _refused(lambda: q.adamw_tensor(**{**good, name: bad}), f"{name} has to be")
    for bad in (z(n, BF16), z(n - 1), z(n, U8)):
        _refused(lambda: q.qmuon_adamw_plan_create([q.adamw_tensor(**{**good, "v": bad})]), "v has to be")
    eight = {**good, "m": z(n, U8), "v": z(n, torch.float8_e4m3fn), "m_absmax": z(2), "v_absmax": z(2)}
    q.qmuon_adamw_plan_create([q.adamw_tensor(**eight)], "e4m3")
    _refused(lambda: q.adamw_tensor(**{**eight, "m_absmax": z(1)}), "m_absmax")
    _refused(lambda: q.adamw_tensor(**{**eight, "v_absmax": z(2, BF16)}), "v_absmax")
    for bad in (z(n), z(n - 1, U8)):
        _refused(lambda: q.qmuon_adamw_plan_create([q.adamw_tensor(**{**eight, "m": bad})], "e4m3"), "m has to be")
    plan = q.qmuon_adamw_plan_create([q.adamw_tensor(**good)])
    for bad in (z(1, BF16), torch.ones(1), z(1, torch.float64)):
        _refused(lambda: q.qmuon_adamw_step(plan, 1, 1e-3, 0.9, 0.99, 1e-8, bad), "grad_scale")
    q.qmuon_adamw_step(plan, 1, 1e-3, 0.9, 0.99, 1e-8, z(2)[1:])
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_orders_and_slices_that_are_right_are_taken():
    # rows of a slice of (batch, time, width): uniformly apart; of a slice of (time, batch): not
    wide = torch.randn(3, 5, 2 * COLS, device="cuda")
    gain = torch.ones(COLS, device="cuda")
    y = torch.zeros(15, COLS, device="cuda")
    want = torch.zeros(15, COLS, device="cuda")
    part = wide[:, :, :COLS]
    q.qmuon_rmsnorm_forward(part.contiguous(), gain, 15, COLS, "f32", 1e-5, y=want)
    q.qmuon_rmsnorm_forward(part, gain, 15, COLS, "f32", 1e-5, y=y, ld_x=2 * COLS)
    assert torch.equal(y, want)
    q.qmuon_rmsnorm_forward(part[1], gain, 5, COLS, "f32", 1e-5, y=y, ld_x=2 * COLS)
    assert torch.equal(y[:5], want[5:10])
    q.qmuon_rmsnorm_forward(part[1:2, 2:3], gain, 1, COLS, "f32", 1e-5, y=y, ld_x=2 * COLS)
    assert torch.equal(y[:1], want[7:8])
    for bad in (part[:, :4], part.transpose(0, 1), part[:, ::2], part[..., 0], wide[0, 0, ::2]):
        _refused(lambda: q.qmuon_rmsnorm_forward(bad, gain, bad.numel() // COLS or 2, COLS, "f32", 1e-5, y=y, ld_x=2 * COLS), "x has")
    # transposed weights: the elements' order in memory is one and the same in what the step goes through together
    z = lambda *s: torch.zeros(*s, device="cuda")   # noqa: E731
    p, g, c = z(8, 40).t(), z(8, 40).t(), torch.zeros(8, 40, dtype=BF16, device="cuda").t()
    g.copy_(torch.arange(320.0, device="cuda").view(40, 8) + 1)
    plan = q.qmuon_adamw_plan_create([q.adamw_tensor(p, g, z(320), z(320), 320, "f32", copy=c)])
    q.qmuon_adamw_step(plan, 1, 0.5, 0.9, 0.99, 1e-8)
    assert bool(((p + 0.5).abs() < 1e-5).all()) and torch.equal(c, p.to(BF16))
    clip = q.qmuon_clip_plan_create([(g, "f32")])
    norm = torch.zeros(2, device="cuda")
    q.qmuon_grad_clip(clip, 1.0, False, norm, torch.empty(q.qmuon_clip_workspace_size(clip), dtype=U8, device="cuda"))
    assert abs(norm[0].item() - g.norm().item()) <= 1e-6 * norm[0].item()
    _refused(lambda: q.adamw_tensor(p, g.contiguous(), z(320), z(320), 320, "f32"), "param")
    _refused(lambda: q.adamw_tensor(p.contiguous(), g, z(320), z(320), 320, "f32"), "grad")
    _refused(lambda: q.adamw_tensor(p, g, z(40, 8), z(320), 320, "f32"), "param")
    _refused(lambda: q.adamw_tensor(p, g, z(320), z(320), 320, "f32", copy=c.contiguous()), "param")
    _refused(lambda: q.adamw_tensor(z(80, 8)[::2], z(320), z(320), z(320), 320, "f32"), "param")
    torch.cuda.synchronize()
