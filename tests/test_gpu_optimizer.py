"""AdamW over many tensors, the gradient norm and the 8-bit state on the GPU against the oracle.

Moments, codes and block steps must match bit for bit (every rounding up to the code is
fixed).  A parameter p' = p - lr (decay p + u) must lie within the roundings of its last
operations: u = m / (w ds + de) takes 2 of 2^-24 for the approximate root w, 1 each for ds, de and
the fused add, 2 for the approximate reciprocal, 1 for the product, the inner fused add 1,
lr * lr_scale 2: at most 11, bounded here by 16 of 2^-24 relative to lr (|decay p| + |u|);
the outer fused add and, for bf16, the last rounding take half a step of p' each."""
import numpy as np
import pytest
import torch

import bit_quantized_base_nf4_b200 as q
from oracle import training_oracle as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
B1, B2, EPS = 0.9, 0.999, 1e-8
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64).reshape(-1)


def _bits(x):
    return np.asarray(x, np.float32).view(np.uint32)


def _rand(g, n, spread=1.5):
    """Values whose magnitudes differ by orders from block to block, and within one."""
    x = torch.randn(n, generator=g) * torch.exp(spread * torch.randn(n, generator=g))
    return x * torch.exp(2 * torch.randn((n + 255) // 256, generator=g)).repeat_interleave(256)[:n] * 1e-3


def _make(g, n, param, grad, bits, copy, **kw):
    p = (torch.randn(n, generator=g) * 0.02).to(param).to(DEV)
    t = q.AdamWTensor.zeros(p, _rand(g, n).to(grad).to(DEV), bits=bits, **kw)
    if copy:
        t.param_bf16 = torch.full((n,), float("nan"), dtype=torch.bfloat16, device=DEV)
    return t


class Model:
    """The oracle's copy of one tensor."""

    def __init__(self, t):
        self.t, self.eight = t, t.exp_avg.dtype == torch.int8
        self.p = _np(t.param)
        n = self.p.size
        self.m, self.v = np.zeros(n), np.zeros(n)

    def step(self, k, lr, coef):
        t = self.t
        m, v, w = T.adamw_moments(_np(t.grad), coef, self.m, self.v, B1, B2)
        self.want, self.u = T.adamw_param(self.p, m, v, k, lr * t.lr_scale, t.weight_decay, B1, B2, EPS)
        self.tol = 16 * 2.0 ** -24 * lr * t.lr_scale * (np.abs(t.weight_decay * self.p) + np.abs(self.u))
        if self.eight:
            self.km, self.dm = T.adam8_encode(m, 127)
            self.kv, self.dv = T.adam8_encode(w, 255)
            m, w = T.adam8_decode(self.km, self.dm), T.adam8_decode(self.kv, self.dv)
            v = T.rn32(w * w)
        self.m, self.v = m, v

    def check(self, what):
        t, got = self.t, _np(self.t.param)
        half = HALF[t.param.dtype]
        tol = self.tol * (1 + half) + half * np.abs(self.want) + (0 if half == 2.0 ** -24 else 2.0 ** -24 * np.abs(self.want))
        bad = ~(np.abs(got - self.want) <= tol)
        assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} parameters off, first {np.argmax(bad)}"
        if t.param_bf16 is not None:
            assert torch.equal(t.param_bf16, t.param.to(torch.bfloat16)), f"{what}: bf16 copy"
        if self.eight:
            assert np.array_equal(t.exp_avg.cpu().numpy().astype(np.int64), self.km), f"{what}: m codes"
            assert np.array_equal(t.exp_avg_sq.cpu().numpy().astype(np.int64), self.kv), f"{what}: sqrt(v) codes"
            assert np.array_equal(_bits(t.exp_avg_step.cpu()), _bits(self.dm)), f"{what}: m steps"
            assert np.array_equal(_bits(t.exp_avg_sq_step.cpu()), _bits(self.dv)), f"{what}: sqrt(v) steps"
        else:
            assert np.array_equal(_bits(t.exp_avg.cpu()), _bits(self.m)), f"{what}: m"
            assert np.array_equal(_bits(t.exp_avg_sq.cpu()), _bits(self.v)), f"{what}: v"
        self.p = got          # the next step starts from the device's parameter


# ----------------------------------------------------------------- 8-bit code

@pytest.mark.parametrize("top,dtype", [(127, torch.int8), (255, torch.uint8)])
def test_adam8_codes_at_every_border(top, dtype):
    # d = 1: y = |x| exactly; every border, its neighbours in float32, and the squares themselves
    j = np.arange(top, dtype=np.float64)
    mid = (j * j + j + 0.5).astype(np.float32)
    vals = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)),
                           ((j + 1) ** 2).astype(np.float32)])
    x = np.zeros((-(-vals.size // 255), 256), np.float32)
    x[:, 0] = top * top
    x[:, 1:].reshape(-1)[:] = np.resize(vals, x.shape[0] * 255)
    if top == 127:
        x[1::2, 1:] *= -1
    src = x if top == 127 else (x.astype(np.float64) ** 2).astype(np.float32)     # v: its root is what is coded
    ref_in = x.reshape(-1) if top == 127 else T.rn32(np.sqrt(src.astype(np.float64))).reshape(-1)
    k, d = T.adam8_encode(ref_in, top)
    codes = torch.empty(x.size, dtype=dtype, device=DEV)
    steps = torch.empty(x.shape[0], device=DEV)
    q.qlora_adam8_encode(torch.from_numpy(src).to(DEV).reshape(-1), codes, steps)
    q.qlora_sync_status()
    assert np.array_equal(codes.cpu().numpy().astype(np.int64), k)
    assert np.array_equal(_bits(steps.cpu()), _bits(d))


@pytest.mark.parametrize("n", [1, 7, 255, 256, 257, 511, 4097, 300_001])
def test_adam8_round_trip_matches_oracle(n):
    g = torch.Generator().manual_seed(n)
    x = _rand(g, n, 3.0)
    x[n // 2] = -0.0
    for dtype, top in ((torch.int8, 127), (torch.uint8, 255)):
        src = x if top == 127 else x * x
        codes = torch.empty(n + 9, dtype=dtype, device=DEV).fill_(77)
        steps = torch.full(((n + 255) // 256 + 1,), 5.0, device=DEV)
        q.qlora_adam8_encode(src.to(DEV), codes[:n], steps[:-1])
        back = torch.full((n + 9,), 5.0, device=DEV)
        q.qlora_adam8_decode(codes[:n], steps[:-1], back[:n])
        q.qlora_sync_status()
        ref = _np(src) if top == 127 else T.rn32(np.sqrt(_np(src)))
        k, d = T.adam8_encode(ref, top)
        assert np.array_equal(codes[:n].cpu().numpy().astype(np.int64), k)
        assert np.array_equal(_bits(steps[:-1].cpu()), _bits(d))
        val = T.adam8_decode(k, d)
        assert np.array_equal(_bits(back[:n].cpu()), _bits(val if top == 127 else T.rn32(val * val)))
        assert (codes[n:] == 77).all() and steps[-1] == 5.0 and (back[n:] == 5.0).all()     # nothing behind the end


def test_adam8_special_blocks():
    x = torch.zeros(256 * 5)
    x[256 + 7], x[512 + 9], x[768:1024], x[1024:] = float("nan"), float("-inf"), 1e-40, 3e38
    codes, steps = torch.empty(1280, dtype=torch.int8, device=DEV), torch.empty(5, device=DEV)
    q.qlora_adam8_encode(x.to(DEV), codes, steps)
    k, d = T.adam8_encode(_np(x), 127)
    assert np.array_equal(codes.cpu().numpy().astype(np.int64), k)
    assert np.array_equal(np.isnan(steps.cpu().numpy()), np.isnan(d)) and steps[0] == 0 and steps[3] == 0
    assert _bits(steps[4].cpu()) == _bits(d[4])


# ----------------------------------------------------------------- the step

SIZES = [1, 3, 255, 256, 257, 1000, 2048, 2049, 40_003]
KINDS = [(torch.float32, torch.float32, True), (torch.float32, torch.bfloat16, False), (torch.bfloat16, torch.float32, False),
         (torch.bfloat16, torch.bfloat16, False)]


@pytest.mark.parametrize("bits", [32, 8, "mixed"])
@pytest.mark.parametrize("clip", [False, True])
def test_steps_match_oracle(bits, clip):
    g = torch.Generator().manual_seed(11)
    ts = []
    for i, n in enumerate(SIZES * 2):
        p, gr, copy = KINDS[i % 4]
        b = bits if bits != "mixed" else (8 if i % 2 else 32)
        ts.append(_make(g, n, p, gr, b, copy, lr_scale=[1.0, 4.0, 0.0][i % 3], weight_decay=[0.0, 0.01][i % 2]))
    ts.insert(5, _make(g, 0, torch.float32, torch.float32, 32, False))           # an empty tensor
    plan = q.qlora_adamw_plan_init(ts)
    models = [Model(t) for t in ts if t.grad.numel()]
    coef = torch.tensor([0.37], device=DEV) if clip else None
    for k in range(1, 5):
        for t in ts:
            t.grad.copy_(_rand(g, t.grad.numel()))                              # in place: the plan keeps its address
        lr = 2e-3 / k
        q.qlora_adamw_step(plan, lr, k, B1, B2, EPS, grad_scale=coef)
        q.qlora_sync_status()
        for i, mo in enumerate(models):
            mo.step(k, lr, 0.37 if clip else None)
            mo.check(f"step {k}, tensor {i} of {mo.p.size}")


def test_what_lies_behind_a_tensor_stays(n=1001):
    g = torch.Generator().manual_seed(12)
    for bits in (32, 8):
        for dt in (torch.float32, torch.bfloat16):
            t = _make(g, n + 64, dt, dt, bits, dt == torch.float32)
            cut = lambda x: None if x is None else x[:n]  # noqa: E731
            before = [x.clone() for x in (t.param, t.exp_avg, t.exp_avg_sq) + ((t.param_bf16,) if t.param_bf16 is not None else ())]
            steps = [None, None] if bits == 32 else [t.exp_avg_step[:4], t.exp_avg_sq_step[:4]]
            view = q.AdamWTensor(cut(t.param), cut(t.grad), cut(t.exp_avg), cut(t.exp_avg_sq), *steps, param_bf16=cut(t.param_bf16))
            q.qlora_adamw_step(q.qlora_adamw_plan_init([view]), 1e-3, 1)
            q.qlora_sync_status()
            after = (t.param, t.exp_avg, t.exp_avg_sq) + ((t.param_bf16,) if t.param_bf16 is not None else ())
            for a, b in zip(after, before):
                assert torch.equal(a[n:].float().nan_to_num(9), b[n:].float().nan_to_num(9))
                assert not torch.equal(a[:n].float().nan_to_num(9), b[:n].float().nan_to_num(9))


def test_chunked_plan_of_a_large_tensor():
    # more than 64 * 148 * 2048 elements: chunks of 2048, several a warp
    n = 64 * 148 * 2048 + 4097
    g = torch.Generator(device=DEV).manual_seed(13)
    grad = torch.randn(n, generator=g, device=DEV)
    t = q.AdamWTensor.zeros(torch.zeros(n, device=DEV), grad, bits=8)
    q.qlora_adamw_step(q.qlora_adamw_plan_init([t]), 1e-3, 1)
    q.qlora_sync_status()
    # from zero states the update is -lr g / (|g| + eps) at every element
    assert torch.allclose(t.param, -1e-3 * grad / (grad.abs() + EPS), rtol=2e-3)
    for lo in (0, 12345 * 256, n - 4097 // 256 * 256 - 4097 % 256):
        s = slice(lo, min(lo + 512, n))
        k, d = T.adam8_encode(T.adamw_moments(_np(grad[s]), None, 0, 0, B1, B2)[0], 127)
        assert np.array_equal(t.exp_avg[s].cpu().numpy().astype(np.int64), k)


def test_device_counter_and_rate_replay_as_steps():
    g = torch.Generator().manual_seed(14)
    a, b = (_make(torch.Generator().manual_seed(15), 5000, torch.float32, torch.float32, 8, True, weight_decay=0.01)
            for _ in range(2))
    plan_a, plan_b = q.qlora_adamw_plan_init([a]), q.qlora_adamw_plan_init([b])
    count, lr, coef = torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, device=DEV), torch.ones(1, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q.qlora_adamw_step(plan_b, 0.0, 0, grad_scale=coef, lr_dev=lr, step_dev=count)
    for k in range(1, 6):
        grad, rate, c = _rand(g, 5000).to(DEV), 1e-3 / k, [1.0, 0.5, 1.0, 0.25, 1.0][k - 1]
        a.grad.copy_(grad), b.grad.copy_(grad), lr.fill_(rate), coef.fill_(c)
        q.qlora_adamw_step(plan_a, float(lr.item()), k, grad_scale=coef)
        graph.replay()
        torch.cuda.synchronize()
        assert count.item() == k
        for x, y in ((a.exp_avg, b.exp_avg), (a.exp_avg_sq, b.exp_avg_sq), (a.param, b.param), (a.param_bf16, b.param_bf16)):
            assert torch.equal(x, y), k
    coef.fill_(float("nan"))
    before = [x.clone() for x in (b.param, b.exp_avg, b.exp_avg_sq, b.exp_avg_step)]
    graph.replay()
    torch.cuda.synchronize()
    assert count.item() == 5
    assert all(torch.equal(x, y) for x, y in zip((b.param, b.exp_avg, b.exp_avg_sq, b.exp_avg_step), before))


def test_non_finite_gradients():
    for bits in (32, 8):
        t = q.AdamWTensor.zeros(torch.ones(700, device=DEV), torch.ones(700, device=DEV), bits=bits)
        t.grad[300], t.grad[600] = float("nan"), float("inf")
        plan = q.qlora_adamw_plan_init([t])
        out = torch.empty(2, device=DEV)
        q.qlora_grad_norm(plan, 1.0, out)
        q.qlora_adamw_step(plan, 1e-3, 1, grad_scale=out[1:])
        assert torch.isnan(out[1]) and (t.param == 1).all() and not t.exp_avg.any()       # clipped: nothing changes
        q.qlora_adamw_step(plan, 1e-3, 1)
        assert torch.isnan(t.param[300]) and torch.isfinite(t.param[:300]).all() and torch.isfinite(t.param[301:600]).all()
        if bits == 8:
            assert torch.isnan(t.exp_avg_step).tolist() == [False, True, True]
            assert not t.exp_avg[256:].any() and not t.exp_avg_sq[256:].any()
        q.qlora_sync_status()


@pytest.mark.parametrize("size", [1e-16, 3e-19, 1e-21])
def test_tiny_gradients(size):
    # second moments below 2^-126 and steps at the edge of the code's range; eps = 0 keeps the ratio m / sqrt(v)
    g = torch.Generator().manual_seed(18)
    n = 1500
    for bits in (32, 8):
        t = q.AdamWTensor.zeros(torch.zeros(n, device=DEV), (_rand(g, n) / 1e-3 * size).to(DEV), bits=bits)
        plan, mo = q.qlora_adamw_plan_init([t]), Model(t)
        for k in (1, 2):
            q.qlora_adamw_step(plan, 1e-3, k, eps=0.0)
            q.qlora_sync_status()
            m, v, w = T.adamw_moments(_np(t.grad), None, mo.m, mo.v, B1, B2)
            live = v > 0                                   # below that the square is zero and the formula has no value
            want, u = T.adamw_param(mo.p[live], m[live], v[live], k, 1e-3, 0.0, B1, B2, 0.0)
            got = _np(t.param)
            assert (np.abs(got[live] - want) <= 16 * 2.0 ** -24 * 1e-3 * np.abs(u) + 2.0 ** -24 * np.abs(want)).all(), (bits, k)
            if bits == 8:
                for codes, steps, x, top in ((t.exp_avg, t.exp_avg_step, m, 127), (t.exp_avg_sq, t.exp_avg_sq_step, w, 255)):
                    ck, d = T.adam8_encode(x, top)
                    assert np.array_equal(codes.cpu().numpy().astype(np.int64), ck) and np.array_equal(_bits(steps.cpu()), _bits(d))
                mo.m, w = T.adam8_decode(*T.adam8_encode(m, 127)), T.adam8_decode(*T.adam8_encode(w, 255))
                mo.v = T.rn32(w * w)
            else:
                assert np.array_equal(_bits(t.exp_avg.cpu()), _bits(m)) and np.array_equal(_bits(t.exp_avg_sq.cpu()), _bits(v))
                mo.m, mo.v = m, v
            t.param.nan_to_num_(0.0, 0.0, 0.0)
            mo.p = _np(t.param)


def test_step_on_another_stream():
    g = torch.Generator().manual_seed(16)
    t = _make(g, 3000, torch.float32, torch.float32, 8, False)
    plan, mo, side = q.qlora_adamw_plan_init([t]), Model(t), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q.qlora_adamw_step(plan, 1e-3, 1, stream=side)
    q.qlora_sync_status(side)
    mo.step(1, 1e-3, None)
    mo.check("side stream")


def test_plan_made_on_another_stream_while_the_current_one_writes_freed_memory():
    # a freed block of the current stream's pool goes to the next request there, with its writes still queued
    g = torch.Generator().manual_seed(17)
    t = _make(g, 3000, torch.float32, torch.float32, 32, False)
    plain, side = q.qlora_adamw_plan_init([t]), torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        busy @ busy
    old = [torch.empty_like(plain.buffer).fill_(0xAB) for _ in range(8)]
    del old
    plan = q.qlora_adamw_plan_init([t], stream=side)
    torch.cuda.synchronize()
    # behind the head (scratch): chunks and tensors; nothing is launched on a list that differs
    used = plan.c_plan.chunks * 80
    head = 256 + 8 * 4096
    assert torch.equal(plan.buffer[head:head + used], plain.buffer[head:head + used])
    mo = Model(t)
    q.qlora_adamw_step(plan, 1e-3, 1, stream=side)
    q.qlora_sync_status(side)
    mo.step(1, 1e-3, None)
    mo.check("plan of a side stream")


# ----------------------------------------------------------------- the norm

@pytest.mark.parametrize("sizes", [[1], [255, 0, 257], [4097, 100_003, 1, 64], [64 * 148 * 2048 + 77]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grad_norm(sizes, dtype):
    g = torch.Generator().manual_seed(17)
    grads = [_rand(g, n).to(dtype).to(DEV) for n in sizes]
    plan = q.qlora_adamw_plan_init([q.AdamWTensor(None, x) for x in grads])
    for limit in (1e-3, 1e6, float("inf")):
        out = torch.empty(2, device=DEV)
        q.qlora_grad_norm(plan, limit, out)
        q.qlora_sync_status()
        n, c = T.grad_norm([_np(x) for x in grads], limit)
        # float64 sums of exact squares: only the last rounding to float32 shows
        assert abs(out[0].item() - n) <= 2.0 ** -23 * n and abs(out[1].item() - c) <= 2.0 ** -23 * c
        again = torch.empty(2, device=DEV)
        q.qlora_grad_norm(plan, limit, again)
        assert torch.equal(out, again)
    with pytest.raises(q.QloraError):
        q.qlora_adamw_step(plan, 1e-3, 1)          # gradients alone cannot be stepped


@pytest.mark.parametrize("value", [1e25, 1e-30])
def test_grad_norm_beyond_the_range_of_float32_squares(value):
    x = torch.full((1000,), value, device=DEV)
    out = torch.empty(2, device=DEV)
    q.qlora_grad_norm(q.qlora_adamw_plan_init([q.AdamWTensor(None, x)]), 1.0, out)
    want = float(np.sqrt(1000.0)) * np.float64(np.float32(value))
    assert abs(out[0].item() - want) <= 2.0 ** -23 * want and out[1].item() == pytest.approx(min(1, 1 / (want + 1e-6)), rel=1e-6)


def test_python_refusals():
    x = torch.zeros(512, device=DEV)
    with pytest.raises(ValueError, match="plan needs"):
        q.qlora_adamw_plan_init([])
    with pytest.raises(ValueError, match="exp_avg"):
        q.qlora_adamw_plan_init([q.AdamWTensor(x, x)])
    with pytest.raises(ValueError, match="grad alone"):
        q.qlora_adamw_plan_init([q.AdamWTensor(None, x, exp_avg=x)])
    with pytest.raises(ValueError, match="param"):
        q.qlora_adamw_plan_init([q.AdamWTensor.zeros(x.half(), x)])
    with pytest.raises(ValueError, match="contiguous"):
        q.qlora_adamw_plan_init([q.AdamWTensor.zeros(torch.zeros(512, 2, device=DEV)[:, 0], x)])
    with pytest.raises(q.QloraError, match="16-byte"):
        q.qlora_adamw_plan_init([q.AdamWTensor.zeros(x[1:], x[1:])])
    with pytest.raises(ValueError, match="codes"):
        q.qlora_adam8_encode(x, x, x)
    with pytest.raises(ValueError, match="grad_scale"):
        q.qlora_adamw_step(q.qlora_adamw_plan_init([q.AdamWTensor.zeros(x, x.clone())]), 1e-3, 1, grad_scale=x)
    plan = q.qlora_adamw_plan_init([q.AdamWTensor.zeros(x, x.clone())])
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(q.QloraError, match="capture"):
            q.qlora_adamw_plan_init(plan.tensors)
        x.add_(0)
