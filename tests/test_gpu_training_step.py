"""The training-step operators together, as a program uses them: tokens are looked up in a packed and
in a trained table, go through the frozen-base layer forward and backward, and the adapters and the
trained table take a clipped AdamW step; the next forward reads the updated bf16 adapters.  Every
stage is compared with the oracle's own stage on the same inputs, and the whole step runs again from
a captured graph."""
import numpy as np
import pytest
import torch

import bit_quantized_base_nf4_b200 as q
from bit_quantized_base_nf4_b200 import synthetic as syn
from oracle import nf4_oracle as O
from oracle import training_oracle as T

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Program:
    """One frozen matrix with an adapter behind a frozen NF4 table plus a trained bf16-read table."""

    def __init__(self, M=200, V=517, K=512, N=256, r=8, bits=8):
        self.M, self.V, self.K, self.N, self.r, self.s = M, V, K, N, r, 2.0
        z = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
        self.W0 = syn.normal_f32((N, K), 0.02, 801)
        self.w = q.NF4Weight.empty(N, K)
        q.qlora_quantize_nf4_dq(self.W0.to(DEV), self.w)
        self.E0 = syn.normal_f32((V, K), 0.5, 802)
        self.table = q.NF4Weight.empty(V, K)
        q.qlora_quantize_nf4_dq(self.E0.to(DEV), self.table)
        self.A32, self.B32 = syn.normal_f32((r, K), 0.05, 803).to(DEV), syn.normal_f32((N, r), 0.05, 804).to(DEV)
        self.A, self.B = self.A32.bfloat16(), self.B32.bfloat16()
        self.E = (syn.normal_f32((V, K), 0.5, 805)).to(DEV)
        g = torch.Generator().manual_seed(806)
        self.ids = torch.randint(0, V, (M,), generator=g).to(DEV)
        self.dY = torch.randn(M, N, generator=g).bfloat16().to(DEV)
        self.X, self.Xf, self.dX = (z(M, K, dtype=torch.bfloat16) for _ in range(3))
        self.Y, self.U, self.G = z(M, N, dtype=torch.bfloat16), z(M, r, dtype=torch.bfloat16), z(M, r, dtype=torch.bfloat16)
        self.dA, self.dB, self.dE = z(r, K), z(N, r), z(V, K)
        self.ws = torch.empty(q.qlora_workspace_bytes(M, N, K, r), dtype=torch.uint8, device=DEV)
        self.ews = torch.empty(q.qlora_embed_grad_workspace_bytes(M, V, K), dtype=torch.uint8, device=DEV)
        self.opt = [q.AdamWTensor.zeros(self.A32.view(-1), self.dA.view(-1), bits=bits, param_bf16=self.A.view(-1)),
                    q.AdamWTensor.zeros(self.B32.view(-1), self.dB.view(-1), bits=bits, param_bf16=self.B.view(-1), lr_scale=4.0),
                    q.AdamWTensor.zeros(self.E.view(-1), self.dE.view(-1), bits=32, weight_decay=0.01)]
        self.plan = q.qlora_adamw_plan_init(self.opt)
        self.norm = z(2)
        self.count, self.lr = torch.zeros(1, dtype=torch.int64, device=DEV), torch.full((1,), 1e-2, device=DEV)

    def forward(self):
        q.qlora_embed_fwd(self.E, self.ids, 1.0, self.X)
        q.qlora_embed_nf4_fwd(self.table, self.ids, 0.5, self.Xf)
        self.X.add_(self.Xf)
        q.qlora_lora_linear_fwd(self.w, self.X, self.A, self.B, self.r, self.s, self.Y, self.U, self.ws)

    def backward(self):
        q.qlora_lora_linear_bwd_dx(self.w, self.dY, self.A, self.B, self.r, self.s, self.dX, self.G, self.ws)
        q.qlora_lora_grad_AB(self.X, self.dY, self.U, self.G, self.r, self.s, self.dA, self.dB)
        q.qlora_embed_grad(self.ids, self.dX, 1.0, self.dE, ws=self.ews)

    def update(self):
        q.qlora_grad_norm(self.plan, 1.0, self.norm)
        q.qlora_adamw_step(self.plan, 0.0, 0, grad_scale=self.norm[1:], lr_dev=self.lr, step_dev=self.count)

    def step(self):
        self.forward()
        self.backward()
        self.update()


def test_stages_match_the_oracle():
    p = Program()
    ref = O.quantize_nf4_dq(p.W0.numpy())
    W = O.dequant(ref["codes"], ref["scales"], ref["scales2"]).reshape(p.N, p.K)
    ref = O.quantize_nf4_dq(p.E0.numpy())
    E4 = O.dequant(ref["codes"], ref["scales"], ref["scales2"]).reshape(p.V, p.K)
    states = [(np.zeros(t.grad.numel()), np.zeros(t.grad.numel())) for t in p.opt]
    ids = p.ids.cpu().numpy()
    for k in (1, 2):
        before = [_np(t.param).reshape(-1) for t in p.opt]
        A, B = _np(p.A), _np(p.B)
        p.forward()
        want = O.bf16_round(T.embed_rows(_np(p.E), ids, 1.0)).astype(np.float64) + \
            O.bf16_round(T.embed_rows(E4, ids, 0.5)).astype(np.float64)
        assert np.array_equal(_np(p.X), O.bf16_round(want.astype(np.float32)).astype(np.float64)), "tokens' rows"
        Y, u = O.lora_linear_fwd(W, p.X.cpu(), A, B, p.s)
        assert O.within_tolerance(p.Y.float().cpu(), Y), O.rel_errors(p.Y.float().cpu(), Y)
        p.backward()
        dX, gr = O.lora_linear_bwd_dx(W, p.dY.cpu(), A, B, p.s)
        dA, dB = O.lora_grad_ab(p.X.cpu(), p.dY.cpu(), u, gr, p.s)
        for got, want in ((p.dX, dX), (p.dA, dA), (p.dB, dB)):
            assert O.within_tolerance(got.float().cpu(), want), O.rel_errors(got.float().cpu(), want)
        dE, mag, cnt = T.embed_grad(ids, _np(p.dX), p.V, 1.0)
        assert (np.abs(_np(p.dE) - dE) <= (cnt[:, None] + 1) * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(dE)).all()
        p.update()
        q.qlora_sync_status()
        n, c = T.grad_norm([_np(t.grad) for t in p.opt], 1.0)
        assert abs(p.norm[0].item() - n) <= 2.0 ** -23 * n and abs(p.norm[1].item() - c) <= 2.0 ** -23 * c and c < 1
        coef, lr = p.norm[1].item(), p.lr.item()
        for i, t in enumerate(p.opt):
            m, v, w = T.adamw_moments(_np(t.grad).reshape(-1), coef, *states[i], 0.9, 0.999)
            want, upd = T.adamw_param(before[i], m, v, k, lr * t.lr_scale, t.weight_decay, 0.9, 0.999, 1e-8)
            tol = 16 * 2.0 ** -24 * lr * t.lr_scale * (np.abs(t.weight_decay * before[i]) + np.abs(upd)) + 2.0 ** -24 * np.abs(want)
            assert (np.abs(_np(t.param).reshape(-1) - want) <= tol * (1 + 2.0 ** -20)).all(), f"tensor {i}"
            if t.exp_avg.dtype == torch.int8:
                km, kv = T.adam8_encode(m, 127), T.adam8_encode(w, 255)
                assert np.array_equal(t.exp_avg.cpu().numpy().astype(np.int64), km[0])
                assert np.array_equal(t.exp_avg_sq.cpu().numpy().astype(np.int64), kv[0])
                w = T.adam8_decode(*kv)
                states[i] = (T.adam8_decode(*km), T.rn32(w * w))
            else:
                states[i] = (m, v)
        assert torch.equal(p.A, p.A32.bfloat16()) and torch.equal(p.B, p.B32.bfloat16())
        assert p.count.item() == k


def test_a_captured_step_replays_as_the_eager_ones():
    a, b = Program(), Program()
    # dA and dB add up in an order that a run does not fix, so the two programs are compared on the
    # same gradients: the layer's part runs eagerly in one program, and its gradients go to the other
    a.step()
    for x, y in ((b.dA, a.dA), (b.dB, a.dB)):
        x.copy_(y)

    def rest(p):
        q.qlora_embed_grad(p.ids, p.dX, 1.0, p.dE, ws=p.ews)
        p.update()
        q.qlora_embed_fwd(p.E, p.ids, 1.0, p.X)

    b.dX.copy_(a.dX)
    rest(b)                                             # first launches, outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rest(b)
    for k in range(2, 5):
        a.step()
        for x, y in ((b.dA, a.dA), (b.dB, a.dB), (b.dX, a.dX)):
            x.copy_(y)
        graph.replay()
        q.qlora_sync_status()
        assert b.count.item() == k == a.count.item()
        for x, y in ((a.A32, b.A32), (a.B, b.B), (a.E, b.E), (a.norm, b.norm), (a.dE, b.dE)):
            assert torch.equal(x, y), k


def test_the_step_leaves_an_eager_forward_its_memory():
    p = Program(bits=32)
    for _ in range(3):
        p.step()
    q.qlora_sync_status()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        p.step()
    q.qlora_sync_status()
    assert torch.cuda.mem_get_info()[0] == free
