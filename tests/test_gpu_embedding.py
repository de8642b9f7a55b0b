"""Embedding lookup and gradient on the GPU against the oracle.

Lookups are compared bit for bit.  A gradient element is a float32 sum of n terms, scaled and
added to the old value in one rounding: it must lie within n * 2^-24 of the sum of the
terms' magnitudes (n - 1 additions in any order, one more for the scale's product inside the
sum's bound) plus half a step of the result in its type."""
import numpy as np
import pytest
import torch

import bit_quantized_base_nf4_b200 as q
from bit_quantized_base_nf4_b200 import synthetic as syn
from oracle import nf4_oracle as O
from oracle import training_oracle as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _bits(x):
    return np.ascontiguousarray(np.asarray(x, np.float32)).view(np.uint32)


def _table(kind, fmt, V, H, seed):
    """(what the call takes, the table's float32 values)."""
    W = syn.normal_f32((V, H), 0.02, seed)
    if kind in ("nf4", "fp4"):
        w = q.NF4Weight.empty(V, H, quant_type=q.QLORA_QT_FP4 if kind == "fp4" else q.QLORA_QT_NF4, format=fmt)
        q.qlora_quantize_nf4_dq(W.to(DEV), w)
        book = O.fp4_codebook() if kind == "fp4" else O.nf4_codebook()
        ref = O.quantize_variant(W.numpy(), 128 if fmt & 1 else 64, not fmt & 2, bool(fmt & 4), book)
        return w, O.dequant_variant(ref["codes"], ref["scales"], ref.get("scales2"), 128 if fmt & 1 else 64, book).reshape(V, H)
    if kind == "q8_0":
        w = q.Q80Weight.empty(V, H)
        q.qlora_quantize_q8_0(W.to(DEV), w)
        ref = O.quantize_q8_0(W.numpy())
        return w, O.dequant_q8_0(ref["q"], ref["d"]).reshape(V, H)
    W = W.to(torch.bfloat16 if kind == "bf16" else torch.float32)
    return W.to(DEV), W.float().numpy()


CALL = {"nf4": "qlora_embed_nf4_fwd", "fp4": "qlora_embed_nf4_fwd", "q8_0": "qlora_embed_q8_0_fwd", "bf16": "qlora_embed_fwd",
        "fp32": "qlora_embed_fwd"}


def _lookup(kind, table, ids, scale, Y, **kw):
    getattr(q, CALL[kind])(table, ids, scale, Y, **kw)


FWD = [("nf4", 0, 64), ("nf4", 0, 1088), ("nf4", 1, 1152), ("nf4", 2, 2112), ("nf4", 3, 256), ("nf4", 4, 192), ("nf4", 5, 384),
       ("fp4", 0, 4096), ("fp4", 3, 128), ("q8_0", 0, 64), ("q8_0", 0, 1216), ("bf16", 0, 8), ("bf16", 0, 1032),
       ("fp32", 0, 8), ("fp32", 0, 2056), ("nf4", 0, 8192), ("q8_0", 0, 5120)]


@pytest.mark.parametrize("kind,fmt,H", FWD)
def test_lookup_bit_exact(kind, fmt, H):
    V = 300 if H < 3000 else 37
    table, ref = _table(kind, fmt, V, H, 701)
    g = torch.Generator().manual_seed(702)
    for n, (ids_t, out_t, scale) in zip((1, 2, 77, 260), [(torch.int64, torch.bfloat16, 1.0), (torch.int32, torch.float32, 64.0),
                                                           (torch.int32, torch.bfloat16, 0.3), (torch.int64, torch.float32, -1.7)]):
        ids = torch.randint(0, V, (n,), generator=g)
        ids[0] = V - 1
        if n > 2:
            ids[1:3] = ids[0]
            ids[-1] = 0
        Y = torch.full((n + 1, H), float("nan"), dtype=out_t, device=DEV)
        _lookup(kind, table, ids.to(ids_t).to(DEV), scale, Y[:n])
        q.qlora_sync_status()
        want = T.embed_rows(ref, ids, scale)
        if out_t == torch.bfloat16:
            want = O.bf16_round(want)
        assert np.array_equal(_bits(Y[:n].float().cpu()), _bits(want)), (n, ids_t, out_t)
        assert torch.isnan(Y[n]).all()


def test_lookup_matches_the_one_shot_dequant():
    table, _ = _table("nf4", 0, 64, 512, 703)
    full, Y = (torch.empty(64, 512, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q.qlora_dequant(table, full)
    q.qlora_embed_nf4_fwd(table, torch.arange(64, device=DEV), 1.0, Y)
    assert torch.equal(full, Y)


@pytest.mark.parametrize("kind", ["nf4", "q8_0", "bf16", "fp32"])
def test_lookup_of_ids_outside_the_table(kind):
    V, H = 50, 192
    table, ref = _table(kind, 0, V, H, 704)
    ids = torch.tensor([3, -1, V, 49, 2 ** 40, -2 ** 40, 0], device=DEV)
    Y = torch.full((7, H), float("nan"), device=DEV)
    _lookup(kind, table, ids, 2.0, Y)
    with pytest.raises(q.QloraError) as e:
        q.qlora_sync_status()
    assert e.value.status == 1 and "token id" in str(e.value)
    q.qlora_sync_status()                                  # reported once
    assert np.array_equal(_bits(Y.cpu()), _bits(T.embed_rows(ref, ids.cpu(), 2.0)))


def test_lookup_of_nothing_and_on_another_stream():
    table, ref = _table("nf4", 0, 50, 192, 705)
    q.qlora_embed_nf4_fwd(table, torch.empty(0, dtype=torch.int64, device=DEV), 1.0, torch.empty(0, 192, device=DEV))
    side = torch.cuda.Stream()
    ids, Y = torch.arange(50, device=DEV), torch.empty(50, 192, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    q.qlora_embed_nf4_fwd(table, ids, 1.0, Y, stream=side)
    q.qlora_sync_status(side)
    assert np.array_equal(_bits(Y.cpu()), _bits(ref))


def test_lookup_beyond_32_bits_of_elements():
    # a bf16 table of 2^32 + elements: rows behind the 2^31st and 2^32nd element
    V, H = 530_000, 8192
    table = torch.zeros(V, H, dtype=torch.bfloat16, device=DEV)
    rows = [0, 262_143, 262_144, 262_145, 524_287, 524_288, V - 1]
    for i, r in enumerate(rows):
        table[r] = i + 1
    Y = torch.empty(len(rows), H, dtype=torch.bfloat16, device=DEV)
    q.qlora_embed_fwd(table, torch.tensor(rows, device=DEV), 1.0, Y)
    q.qlora_sync_status()
    assert (Y == torch.arange(1, len(rows) + 1, device=DEV)[:, None]).all()


# ----------------------------------------------------------------- gradient

def _ids(g, T_, V, how):
    if how == "one":
        return torch.full((T_,), V // 2)
    if how == "zipf":
        return torch.exp(torch.rand(T_, generator=g, dtype=torch.float64) * np.log(V)).long().clamp(1, V) - 1
    if how == "runs":                                       # few ids, long runs
        return torch.randint(0, min(V, 3), (T_,), generator=g)
    return torch.randint(0, V, (T_,), generator=g)


def _check_grad(ids, dY, V, scale, pad, dE, old, what):
    want, mag, cnt = T.embed_grad(ids.cpu(), dY.float().cpu().numpy(), V, scale, pad)
    got = dE.float().cpu().numpy().astype(np.float64)
    base = 0.0 if old is None else old.float().cpu().numpy().astype(np.float64)
    full = want + base
    half = HALF[dE.dtype]
    tol = (cnt[:, None] + 1) * 2.0 ** -24 * (1 + 2.0 ** -10) * mag + 2.0 ** -24 * np.abs(full) + (half if half > 2.0 ** -24 else 0) * np.abs(full) * 1.01
    bad = ~(np.abs(got - full) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off in rows {np.unique(np.nonzero(bad)[0])[:5]}"
    untouched = cnt == 0
    want_bits = _bits(got[untouched] * 0 + (0 if old is None else base[untouched]))
    assert np.array_equal(_bits(got[untouched]), want_bits), f"{what}: rows without a token"


GRAD = [
    # T, V, H, ids, dY, dE, accumulate, padding, scale, id type
    (1, 1, 8, "any", torch.float32, torch.float32, False, -1, 1.0, torch.int64),
    (1, 5, 72, "any", torch.bfloat16, torch.bfloat16, True, -1, 2.0, torch.int32),
    (7, 3, 1024, "any", torch.bfloat16, torch.float32, False, 1, 0.5, torch.int64),
    (8, 40, 1032, "any", torch.float32, torch.bfloat16, False, -1, 1.0, torch.int64),
    (9, 511, 64, "one", torch.bfloat16, torch.float32, True, -1, -3.0, torch.int32),
    (33, 512, 136, "zipf", torch.float32, torch.float32, True, 0, 1.0, torch.int64),
    (128, 40, 1160, "zipf", torch.bfloat16, torch.float32, False, 2, 1.0, torch.int64),
    (128, 4096, 24, "one", torch.float32, torch.bfloat16, True, -1, 0.5, torch.int32),
    (129, 40, 1160, "zipf", torch.bfloat16, torch.float32, False, 2, 1.0, torch.int64),
    (192, 700, 1160, "zipf", torch.bfloat16, torch.float32, True, 2, 1.0, torch.int64),
    (192, 9, 64, "runs", torch.float32, torch.float32, False, -1, 1.0, torch.int32),
    (193, 700, 1160, "zipf", torch.bfloat16, torch.float32, False, 2, 1.0, torch.int64),
    (101, 30_000, 4096, "any", torch.bfloat16, torch.float32, False, 0, 1.0, torch.int64),
    (77, 3, 520, "runs", torch.bfloat16, torch.bfloat16, False, -1, 1.0, torch.int32),
    (1000, 513, 264, "zipf", torch.bfloat16, torch.float32, False, 0, 1.0, torch.int32),
    (1025, 40_000, 2056, "zipf", torch.bfloat16, torch.float32, False, -1, 1.0, torch.int64),
    (4097, 700, 128, "one", torch.bfloat16, torch.float32, False, -1, 1.0, torch.int64),
    (4097, 700, 4104, "runs", torch.float32, torch.float32, True, -1, 0.25, torch.int32),
    (9001, 300_000, 40, "any", torch.bfloat16, torch.bfloat16, False, 7, 1.0, torch.int64),
    (30_000, 100, 3000 // 8 * 8, "zipf", torch.bfloat16, torch.float32, True, 3, 1.0, torch.int64),
    (70_001, 262_144, 16, "zipf", torch.float32, torch.float32, False, -1, 1.0, torch.int32),
    (131_072, 50_000, 8, "zipf", torch.float32, torch.float32, False, -1, 1.0, torch.int64),
    (131_073, 50_000, 8, "zipf", torch.float32, torch.float32, False, -1, 1.0, torch.int64),
    (152_000, 50, 8, "zipf", torch.bfloat16, torch.float32, False, -1, 1.0, torch.int64),       # chunks of 128, swept sort
    (76_000, 900, 1032, "zipf", torch.bfloat16, torch.bfloat16, True, 4, 1.0, torch.int32),      # chunks of 128, held sort
    (200_003, 300_000, 24, "any", torch.bfloat16, torch.float32, True, 5, 1.0, torch.int32),
]


@pytest.mark.parametrize("case", GRAD, ids=[f"T{c[0]}-V{c[1]}-H{c[2]}-{c[3]}" for c in GRAD])
def test_grad_matches_oracle_and_repeats(case):
    n, V, H, how, dyt, det, acc, pad, scale, idt = case
    g = torch.Generator().manual_seed(n + V)
    ids = _ids(g, n, V, how).to(idt).to(DEV)
    dY = torch.randn(n, H, generator=g).to(dyt).to(DEV)
    old = torch.randn(V, H, generator=g).to(det).to(DEV) if acc else None
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(n, V, H), dtype=torch.uint8, device=DEV)
    got = []
    for fill in (0, 255):
        ws.fill_(fill)                                      # what the workspace held does not matter
        dE = old.clone() if acc else torch.full((V, H), float("nan"), dtype=det, device=DEV)
        q.qlora_embed_grad(ids, dY, scale, dE, padding_id=pad, accumulate=acc, ws=ws)
        q.qlora_sync_status()
        got.append(dE)
    assert torch.equal(got[0], got[1])
    _check_grad(ids, dY, V, scale, pad, got[0], old, "gradient")


def test_grad_long_runs_beside_short_ones():
    # ids whose runs end at, before and behind every chunk border, and one that spans hundreds of chunks
    g = torch.Generator().manual_seed(21)
    counts = [8, 8, 1, 7, 16, 15, 17, 3000, 1, 24, 23, 25, 260, 1, 1, 6, 300]
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    ids = ids[torch.randperm(ids.numel(), generator=g)].to(DEV)
    for H in (8, 256, 1160):
        dY = torch.randn(ids.numel(), H, generator=g).to(DEV)
        dE = torch.empty(30, H, device=DEV)
        ws = torch.empty(q.qlora_embed_grad_workspace_bytes(ids.numel(), 30, H), dtype=torch.uint8, device=DEV)
        q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws)
        _check_grad(ids, dY, 30, 1.0, -1, dE, None, f"H {H}")


def test_grad_of_ids_outside_the_table():
    g = torch.Generator().manual_seed(22)
    ids = torch.tensor([0, -5, 3, 10, 2 ** 33 + 3, 3, 9], device=DEV)
    dY = torch.randn(7, 64, generator=g).to(DEV)
    dE = torch.empty(10, 64, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(7, 10, 64), dtype=torch.uint8, device=DEV)
    q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws)
    with pytest.raises(q.QloraError, match="token id"):
        q.qlora_sync_status()
    _check_grad(ids, dY, 10, 1.0, -1, dE, None, "bad ids")


def test_grad_of_no_tokens():
    dE = torch.full((100, 64), 3.0, device=DEV)
    none, dY = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, 64, device=DEV)
    q.qlora_embed_grad(none, dY, 1.0, dE, accumulate=True)
    assert (dE == 3).all()
    q.qlora_embed_grad(none, dY, 1.0, dE)
    q.qlora_sync_status()
    assert not dE.any()


def test_grad_of_all_padding():
    ids, dY = torch.full((500,), 4, device=DEV), torch.ones(500, 64, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(500, 10, 64), dtype=torch.uint8, device=DEV)
    dE = torch.full((10, 64), 3.0, device=DEV)
    q.qlora_embed_grad(ids, dY, 1.0, dE, padding_id=4, accumulate=True, ws=ws)
    assert (dE == 3).all()
    q.qlora_embed_grad(ids, dY, 1.0, dE, padding_id=4, ws=ws)
    q.qlora_sync_status()
    assert not dE.any()


def test_grad_non_finite_rows_stay_in_their_row():
    ids = torch.tensor([1, 2, 1, 5], device=DEV)
    dY = torch.ones(4, 64, device=DEV)
    dY[1, 3], dY[3, 4] = float("nan"), float("inf")
    dE = torch.empty(8, 64, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(4, 8, 64), dtype=torch.uint8, device=DEV)
    q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws)
    assert torch.isnan(dE[2, 3]) and torch.isinf(dE[5, 4]) and torch.isfinite(dE).sum() == 8 * 64 - 2 and (dE[1] == 2).all()


def test_grad_is_the_adjoint_of_the_lookup():
    # <dE, D> = <dY, lookup(D)>, both inner products in float64; each side is off by its own roundings only
    g = torch.Generator().manual_seed(23)
    V, H, n = 600, 256, 3000
    ids = _ids(g, n, V, "zipf").to(DEV)
    dY, D = torch.randn(n, H, generator=g).to(DEV), torch.randn(V, H, generator=g).to(DEV)
    dE, Y = torch.empty(V, H, device=DEV), torch.empty(n, H, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(n, V, H), dtype=torch.uint8, device=DEV)
    q.qlora_embed_grad(ids, dY, 1.5, dE, ws=ws)
    q.qlora_embed_fwd(D, ids, 1.5, Y)
    _, mag, cnt = T.embed_grad(ids.cpu(), dY.cpu().numpy(), V, 1.5)
    lhs, rhs = (dE.double() * D.double()).sum().item(), (dY.double() * Y.double()).sum().item()
    slack = ((cnt[:, None] + 2) * 2.0 ** -24 * mag * np.abs(D.double().cpu().numpy())).sum() + \
        2.0 ** -24 * (dY.double() * Y.double()).abs().sum().item()
    assert abs(lhs - rhs) <= slack


def test_grad_captured_and_replayed_with_new_ids():
    g = torch.Generator().manual_seed(24)
    V, H, n = 900, 128, 700
    ids, dY, dE = torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros(n, H, device=DEV), torch.empty(V, H, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(n, V, H), dtype=torch.uint8, device=DEV)
    q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws)             # the shared-memory limit is set outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws)
    for how in ("zipf", "any", "one"):
        ids.copy_(_ids(g, n, V, how)), dY.copy_(torch.randn(n, H, generator=g))
        graph.replay()
        _check_grad(ids, dY, V, 1.0, -1, dE, None, how)


@pytest.mark.parametrize("n", [5000, 131_073])
def test_grad_of_larger_sorts_captured(n):
    g = torch.Generator().manual_seed(n)
    V, H = 3000, 16
    ids, dY = _ids(g, n, V, "zipf").to(DEV), torch.randn(n, H, generator=g).to(DEV)
    dE, ws = torch.empty(V, H, device=DEV), torch.empty(q.qlora_embed_grad_workspace_bytes(n, V, H), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws)
        q.qlora_embed_grad(ids, dY, 1.0, dE, accumulate=True, ws=ws)
    for _ in range(3):
        graph.replay()
    want, mag, cnt = T.embed_grad(ids.cpu(), dY.cpu().numpy(), V, 1.0)
    tol = 2 * (cnt[:, None] + 1) * 2.0 ** -24 * (1 + 2.0 ** -10) * mag + 2.0 ** -23 * np.abs(2 * want)
    assert (np.abs(dE.double().cpu().numpy() - 2 * want) <= tol).all()


def test_two_gradients_at_once_on_two_streams():
    g = torch.Generator().manual_seed(25)
    V, H, n = 5000, 1024, 6000
    streams, work = [torch.cuda.Stream() for _ in range(2)], []
    for _ in streams:
        work.append((_ids(g, n, V, "zipf").to(DEV), torch.randn(n, H, generator=g).to(DEV), torch.empty(V, H, device=DEV),
                     torch.empty(q.qlora_embed_grad_workspace_bytes(n, V, H), dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(3):
        for st, (ids, dY, dE, ws) in zip(streams, work):
            q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws, stream=st)
    torch.cuda.synchronize()
    for ids, dY, dE, ws in work:
        _check_grad(ids, dY, V, 1.0, -1, dE, None, "two streams")


def test_python_refusals():
    E, ids, Y = torch.zeros(10, 64, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, 64, device=DEV)
    with pytest.raises(ValueError, match="ids"):
        q.qlora_embed_fwd(E, ids.float(), 1.0, Y)
    with pytest.raises(ValueError, match="ids"):
        q.qlora_embed_fwd(E, ids[::2], 1.0, Y)
    with pytest.raises(ValueError, match="Y"):
        q.qlora_embed_fwd(E, ids, 1.0, Y[:3])
    with pytest.raises(ValueError, match="table"):
        q.qlora_embed_fwd(E.half(), ids, 1.0, Y)
    with pytest.raises(ValueError, match="table"):
        q.qlora_embed_fwd(E.t(), ids, 1.0, Y)
    with pytest.raises(ValueError, match="dY"):
        q.qlora_embed_grad(ids, Y[:2], 1.0, E)
    with pytest.raises(q.QloraError, match="workspace"):
        q.qlora_embed_grad(ids, Y, 1.0, E)
    with pytest.raises(q.QloraError, match="multiple of 8"):
        q.qlora_embed_fwd(torch.zeros(10, 12, device=DEV), ids, 1.0, torch.zeros(4, 12, device=DEV))
