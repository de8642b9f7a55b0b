"""Branches of the AdamW step and the gradient norm that lists of production size take, against the definition
in 64 bits.  Moments, codes and block steps are compared bit for bit; a parameter within 16 * 2^-24 of
lr (|decay p| + |u|) for the approximate root and reciprocal, plus half a step of its type for each rounding of p'
(the count of roundings stands in test_gpu_optimizer.py)."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_base_nf4_b200 as q
from oracle import training_oracle as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
B1, B2 = 0.9, 0.999
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _rn(x):
    return x.float().double()


def _f32(x):
    return float(np.float32(x))


def _blocks(x):
    out = torch.zeros(-(-x.numel() // 256) * 256, dtype=torch.float64, device=DEV)
    out[:x.numel()] = x
    return out.view(-1, 256)


def _encode(x, top):
    """(codes, steps) of float64 values that are float32 ones: the definition, over all blocks at once."""
    b = _blocks(x)
    d = _rn(b.abs().amax(dim=1, keepdim=True) / (top * top))
    d = torch.where(d < 2.0 ** -126, torch.zeros_like(d), d)
    y = _rn(b.abs() * torch.where(d > 0, _rn(1.0 / d), torch.zeros_like(d)))
    j = torch.arange(top, dtype=torch.float64, device=DEV)
    k = torch.bucketize(y, j * j + j + 0.5).double()             # how many borders lie below y
    return (torch.where(b < 0, -k, k)).view(-1)[:x.numel()], d.view(-1)


def _decode(k, d):
    return _rn(_rn(k * k.abs()) * d.repeat_interleave(256)[:k.numel()])


def test_the_reference_encodes_as_the_oracle():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(3000, generator=g) * torch.exp(2 * torch.randn(3000, generator=g))).double()
    for top in (127, 255):
        v = x if top == 127 else x.abs()
        v = v.float().double()
        k, d = _encode(v.to(DEV), top)
        ko, do = T.adam8_encode(v.numpy(), top)
        assert np.array_equal(k.cpu().numpy(), ko) and np.array_equal(d.cpu().numpy(), do.astype(np.float64))


class Ref:
    def __init__(self, t):
        self.t, self.eight = t, t.exp_avg.dtype == torch.int8
        self.m = torch.zeros(t.grad.numel(), dtype=torch.float64, device=DEV)
        self.v = torch.zeros_like(self.m)
        self.p = t.param.double().clone()

    def step(self, k, lr, coef, eps, what):
        t = self.t
        g = t.grad.double()
        if coef is not None:
            g = _rn(g * _f32(coef))
        m = _rn(_rn(_f32(B1) * self.m) + _rn(_f32(1 - B1) * g))
        v = _rn(_rn(_f32(B2) * self.v) + _rn(_f32(1 - B2) * _rn(g * g)))
        w = _rn(v.sqrt())
        u = (m / (1 - B1 ** k)) / (v.sqrt() / math.sqrt(1 - B2 ** k) + eps)
        lr = lr * t.lr_scale
        want = self.p - lr * (t.weight_decay * self.p + u)
        half, got = HALF[t.param.dtype], t.param.double()
        tol = 16 * 2.0 ** -24 * lr * ((t.weight_decay * self.p).abs() + u.abs()) * (1 + half) + half * want.abs()
        if half > 2.0 ** -24:
            tol += 2.0 ** -24 * want.abs()
        bad = ~((got - want).abs() <= tol)
        assert not bad.any(), f"{what}: {int(bad.sum())} parameters off, first {int(bad.nonzero()[0])} of {bad.numel()}"
        if t.param_bf16 is not None:
            assert torch.equal(t.param_bf16, t.param.to(BF16)), f"{what}: copy"
        if self.eight:
            km, dm = _encode(m, 127)
            kv, dv = _encode(w, 255)
            for name, have, ref in (("m codes", t.exp_avg, km), ("sqrt(v) codes", t.exp_avg_sq, kv), ("m steps", t.exp_avg_step, dm),
                                    ("sqrt(v) steps", t.exp_avg_sq_step, dv)):
                bad = have.double() != ref
                assert not bad.any(), f"{what}: {int(bad.sum())} {name} differ, first {int(bad.nonzero()[0])} of {bad.numel()}"
            m, w = _decode(km, dm), _decode(kv, dv)
            v = _rn(w * w)
        else:
            for name, have, ref in (("m", t.exp_avg, m), ("v", t.exp_avg_sq, v)):
                bad = have.double() != ref
                assert not bad.any(), f"{what}: {int(bad.sum())} {name} differ, first {int(bad.nonzero()[0])} of {bad.numel()}"
        self.m, self.v, self.p = m, v, got.clone()


def _rand(g, n, size=1e-3):
    x = torch.randn(n, generator=g, device=DEV) * torch.exp(1.5 * torch.randn(n, generator=g, device=DEV))
    return x * torch.exp(2 * torch.randn((n + 255) // 256, generator=g, device=DEV)).repeat_interleave(256)[:n] * size


def _make(g, n, kind, bits, **kw):
    param, grad, copy = kind
    p = (torch.randn(n, generator=g, device=DEV) * 0.02).to(param)
    t = q.AdamWTensor.zeros(p, _rand(g, n).to(grad), bits=bits, **kw)
    if copy:
        t.param_bf16 = torch.full((n,), float("nan"), dtype=BF16, device=DEV)
    return t


KINDS = [(F32, F32, True), (F32, BF16, False), (BF16, F32, False), (BF16, BF16, False)]
# Elements of a chunk: 256 below 64 * 148 * 512 elements in all, 512 below 64 * 148 * 1024, 1024 from there on; tensors that
# end in every place of a chunk, of an 8-bit stage (512) and of a block.
LISTS = {
    512: [1_300_003, 1_200_257, 1_400_512, 1_250_000, 513, 511, 255, 1, 768, 1023],
    1024: [2_600_001, 2_500_255, 2_700_513, 2_400_769, 1025, 1023, 1280, 1, 512, 257, 2049],
}


def _run(ts, steps=3, eps=1e-8, clip=True, what=""):
    plan, refs = q.qlora_adamw_plan_init(ts), [Ref(t) for t in ts]
    g, out = torch.Generator(device=DEV).manual_seed(99), torch.empty(2, device=DEV)
    for k in range(1, steps + 1):
        for t in ts:
            t.grad.copy_(_rand(g, t.grad.numel()))
        coef = None
        if clip:
            q.qlora_grad_norm(plan, 0.5, out)
        q.qlora_adamw_step(plan, 2e-3 / k, k, B1, B2, eps, grad_scale=out[1:] if clip else None)
        q.qlora_sync_status()
        if clip:
            n = math.sqrt(sum(float(t.grad.double().square().sum()) for t in ts))
            assert abs(out[0].item() - n) <= 2.0 ** -23 * n
            coef = out[1].item()
        for i, r in enumerate(refs):
            r.step(k, 2e-3 / k, coef, eps, f"{what} step {k}, tensor {i} of {r.p.numel()}")


@pytest.mark.parametrize("chunk", [512, 1024])
@pytest.mark.parametrize("bits", [32, 8, "mixed"])
def test_lists_of_longer_chunks(chunk, bits):
    g = torch.Generator(device=DEV).manual_seed(chunk)
    ts = [_make(g, n, KINDS[i % 4], bits if bits != "mixed" else (8, 32)[(i + i // 4) % 2], lr_scale=[1.0, 4.0][i % 2],
                weight_decay=[0.0, 0.01][i // 2 % 2]) for i, n in enumerate(LISTS[chunk])]
    total = sum(t.grad.numel() for t in ts)
    assert 64 * 148 * 512 <= total < 64 * 148 * 1024 if chunk == 512 else total >= 64 * 148 * 1024
    _run(ts, what=f"{bits} bits")


@pytest.mark.parametrize("kind", range(4))
@pytest.mark.parametrize("bits", [32, 8])
def test_one_large_tensor_of_each_type(kind, bits):
    # 8-bit states: the stages hold 6, 8 or 10 bytes an element, and a warp goes through three chunks or more
    g = torch.Generator(device=DEV).manual_seed(kind)
    _run([_make(g, 64 * 148 * 1024 + 4097 + 256 * kind + kind, KINDS[kind], bits, weight_decay=0.01)], clip=kind % 2 == 0)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_of_a_few_elements_with_large_ones_between(bits):
    # chunks of 1024 that are mostly short: the ring of an 8-bit warp opens a new chunk at every copy
    g = torch.Generator(device=DEV).manual_seed(5)
    sizes = [4_000_001] + [1 + 13 * i for i in range(150)] + [3_000_300] + [1 + 7 * i for i in range(150)] + [3_000_000]
    _run([_make(g, n, KINDS[i % 4], bits) for i, n in enumerate(sizes)], steps=2)


@pytest.mark.parametrize("size", [1e-9, 1e-13, 1e-16, 3e-19, 1e-21])
@pytest.mark.parametrize("bits", [32, 8])
def test_tiny_gradients_with_an_eps(size, bits):
    # with eps the approximate root takes second moments below 2^-126 as zero; below 2^-92 codes are then worked out exactly
    g = torch.Generator(device=DEV).manual_seed(18)
    ts = [_make(g, n, kind, bits) for n, kind in ((1500, (F32, F32, False)), (5001, (BF16, F32, False)))]
    plan, refs = q.qlora_adamw_plan_init(ts), [Ref(t) for t in ts]
    for k in (1, 2, 3):
        for t in ts:
            t.grad.copy_(_rand(g, t.grad.numel(), size))
        q.qlora_adamw_step(plan, 1e-3, k, B1, B2, 1e-8)
        q.qlora_sync_status()
        for r in refs:
            r.step(k, 1e-3, None, 1e-8, f"gradients near {size}, step {k}")


# ----------------------------------------------------------------- the norm

@pytest.mark.parametrize("sizes", [[33_554_433], [20_000_001, 300, 20_000_000, 0, 7_000_003], [70_000_005, 1, 255], [130_000_001]])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_of_several_chunks_a_warp(sizes, dtype):
    # more than 8 * 4096 chunks of 1024
    g = torch.Generator(device=DEV).manual_seed(len(sizes))
    grads = [_rand(g, n).to(dtype) for n in sizes]
    plan = q.qlora_adamw_plan_init([q.AdamWTensor(None, x) for x in grads])
    out, again = torch.empty(2, device=DEV), torch.empty(2, device=DEV)
    q.qlora_grad_norm(plan, 0.3, out)
    q.qlora_grad_norm(plan, 0.3, again)
    q.qlora_sync_status()
    n = math.sqrt(math.fsum(float(x[lo:lo + (1 << 24)].double().square().sum()) for x in grads for lo in range(0, x.numel(), 1 << 24)))
    c = min(1.0, 0.3 / (n + 1e-6))
    assert abs(out[0].item() - n) <= 2.0 ** -23 * n and abs(out[1].item() - c) <= 2.0 ** -23 * c and torch.equal(out, again)


def test_norm_misses_no_chunk():
    # one gradient that is not zero, at every border of chunks, warps and CTAs in turn
    n = 70_000_005
    x = torch.zeros(n, device=DEV)
    plan, out = q.qlora_adamw_plan_init([q.AdamWTensor(None, x)]), torch.empty(64, 2, device=DEV)
    places = sorted({min(n - 1, max(0, b * s + o)) for s in (256, 1024, 8 * 1024, 3 * 8 * 1024) for b in (1, 5, 2000) for o in (-1, 0)} | {0, n - 1, n - 6})
    for i, at in enumerate(places):
        x[at] = 3.0
        q.qlora_grad_norm(plan, 1.0, out[i])
        x[at] = 0.0
    q.qlora_sync_status()
    assert out[:len(places), 0].tolist() == [3.0] * len(places)


def test_norm_of_nothing():
    for sizes in ([0], [0, 0, 0]):
        plan = q.qlora_adamw_plan_init([q.AdamWTensor(None, torch.empty(n, device=DEV)) for n in sizes])
        out = torch.full((2,), float("nan"), device=DEV)
        q.qlora_grad_norm(plan, 1e-7, out)
        q.qlora_sync_status()
        assert out[0] == 0 and abs(out[1].item() - 0.1) <= 2.0 ** -23


# ----------------------------------------------------------------- beyond 32 bits of elements

WINDOWS = [0, (1 << 31) - 512, (1 << 32) - 1024, (1 << 32)]       # each starts at a block of 256 and holds 1024 elements


@pytest.mark.parametrize("bits", [8, 32])
def test_a_tensor_beyond_32_bits_of_elements(bits):
    n = (1 << 32) + 4097
    g = torch.Generator(device=DEV).manual_seed(7)
    grad, param = torch.zeros(n, dtype=BF16, device=DEV), torch.zeros(n, dtype=BF16, device=DEV)
    for w in WINDOWS + [n // 256 * 256 - 1024]:                     # the last one, and what lies behind the last whole block
        grad[w:w + 1024] = _rand(g, 1024).to(BF16)
    grad[n - 1] = 0.5
    t = q.AdamWTensor.zeros(param, grad, bits=bits)
    plan, out = q.qlora_adamw_plan_init([t]), torch.empty(2, device=DEV)
    q.qlora_grad_norm(plan, float("inf"), out)
    q.qlora_adamw_step(plan, 1e-3, 1)
    q.qlora_sync_status()
    total = math.fsum(float(grad[lo:lo + (1 << 26)].double().square().sum()) for lo in range(0, n, 1 << 26))
    assert abs(out[0].item() - math.sqrt(total)) <= 2.0 ** -23 * math.sqrt(total)
    for w in WINDOWS + [n // 256 * 256 - 1024]:
        s = slice(w, min(w + 1024 + (n % 256 if w + 1024 == n // 256 * 256 else 0), n))
        b = slice(s.start // 256, -(-s.stop // 256))
        part = q.AdamWTensor(param[s], grad[s], t.exp_avg[s], t.exp_avg_sq[s], t.exp_avg_step[b] if bits == 8 else None,
                             t.exp_avg_sq_step[b] if bits == 8 else None)
        ref = Ref(part)
        ref.p.zero_()
        ref.step(1, 1e-3, None, 1e-8, f"window at {w}")
    live = sum(int((x != 0).sum()) for x in param.split(1 << 28))
    assert live == sum(int((x != 0).sum()) for x in grad.split(1 << 28))


def test_adam8_beyond_32_bits_of_elements():
    n = (1 << 32) + 300
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.zeros(n, device=DEV)
    at = WINDOWS[:3] + [n // 256 * 256 - 768]
    for w in at:
        x[w:w + 1024] = _rand(g, min(1024, n - w))
    codes, steps = torch.empty(n, dtype=torch.int8, device=DEV), torch.empty(-(-n // 256), device=DEV)
    q.qlora_adam8_encode(x, codes, steps)
    kept = []
    for w in at:
        e = min(w + 1024, n)
        k, d = _encode(x[w:e].double(), 127)
        assert torch.equal(codes[w:e].double(), k) and torch.equal(steps[w // 256:-(-e // 256)].double(), d)
        kept.append((w, e, _decode(k, d)))
    q.qlora_adam8_decode(codes, steps, x)
    q.qlora_sync_status()
    for w, e, v in kept:
        assert torch.equal(x[w:e].double(), v)
    assert sum(int((c != 0).sum()) for c in codes.split(1 << 28)) == sum(int((c != 0).sum()) for c in x.split(1 << 28))
