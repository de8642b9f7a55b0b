"""Branches of the embedding calls that larger batches and longer rows take, compared without a tolerance.

Gradients: dY, the old dE and the scaled sums are small whole numbers (times a power of two), so that every
partial sum lies below 2^24 and float32 adds it exactly in any order.  A float32 gradient then equals
the sum in 64 bits; a bfloat16 one is that sum rounded once.  One token lost or counted twice shows."""
import numpy as np
import pytest
import torch

import bit_quantized_base_nf4_b200 as q
from bit_quantized_base_nf4_b200 import synthetic as syn
from oracle import nf4_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ----------------------------------------------------------------- lookup

def _table(kind, V, H):
    """(what the call takes, the table's float32 values on the device)."""
    W = syn.normal_f32((V, H), 0.02, 711)
    if kind == "nf4":
        w = q.NF4Weight.empty(V, H)
        q.qlora_quantize_nf4_dq(W.to(DEV), w)
        ref = O.quantize_variant(W.numpy(), 64, True, False, O.nf4_codebook())
        return w, torch.from_numpy(O.dequant_variant(ref["codes"], ref["scales"], ref["scales2"], 64, O.nf4_codebook()).reshape(V, H)).to(DEV)
    if kind == "q8_0":
        w = q.Q80Weight.empty(V, H)
        q.qlora_quantize_q8_0(W.to(DEV), w)
        ref = O.quantize_q8_0(W.numpy())
        return w, torch.from_numpy(O.dequant_q8_0(ref["q"], ref["d"]).reshape(V, H)).to(DEV)
    W = W.to(torch.bfloat16 if kind == "bf16" else torch.float32).to(DEV)
    return W, W.float()


CALL = {"nf4": "qlora_embed_nf4_fwd", "q8_0": "qlora_embed_q8_0_fwd", "bf16": "qlora_embed_fwd", "fp32": "qlora_embed_fwd"}


def _check_lookup(kind, V, H, T, out, bad):
    table, ref = _table(kind, V, H)
    g = torch.Generator(device=DEV).manual_seed(T + H)
    ids = torch.randint(0, V, (T,), generator=g, device=DEV)
    if bad:                                     # at the start, in the middle of a warp's tokens and at the end
        at = torch.cat([torch.arange(0, T, 37, device=DEV), torch.tensor([T - 1, T // 2, T // 2 + 1], device=DEV)])
        ids[at] = torch.where(at % 2 == 0, torch.full_like(at, -1), torch.full_like(at, V))
    Y = torch.full((T + 1, H), float("nan"), dtype=out, device=DEV)
    getattr(q, CALL[kind])(table, ids, 0.3, Y[:T])
    if bad:
        with pytest.raises(q.QloraError, match="token id"):
            q.qlora_sync_status()
    else:
        q.qlora_sync_status()
    assert torch.isnan(Y[T]).all()
    scale = float(np.float32(0.3))
    for lo in range(0, T, 4096):
        i, got = ids[lo:lo + 4096], Y[:T][lo:lo + 4096]
        ok = (i >= 0) & (i < V)
        want = (ref[i.clamp(0, V - 1)].double() * scale).float() * ok[:, None]        # exact product, rounded once
        assert torch.equal(got, want.to(out)), (kind, T, H, lo)


# Tokens of a CTA in one pass: 8 up to rows of 1024, 4 up to 2048, 2 up to 4096, 1 above.  From 2368 such CTAs on a
# warp takes two tokens, from 9472 on four (148 SMs).
@pytest.mark.parametrize("kind,H,T,out", [
    ("nf4", 64, 8 * 2368 + 3, torch.bfloat16), ("nf4", 64, 8 * 9472 + 5, torch.float32), ("nf4", 2112, 2 * 9472 + 1, torch.bfloat16),
    ("q8_0", 128, 8 * 9472 + 9, torch.bfloat16), ("q8_0", 1216, 4 * 2368 + 2, torch.float32), ("bf16", 1032, 4 * 9472 + 7, torch.bfloat16),
    ("bf16", 24, 8 * 2368, torch.float32), ("fp32", 8, 8 * 9472 + 31, torch.bfloat16), ("fp32", 4104, 2371, torch.float32),
])
@pytest.mark.parametrize("bad", [False, True])
def test_lookup_of_several_tokens_a_warp(kind, H, T, out, bad):
    _check_lookup(kind, 500, H, T, out, bad)


@pytest.mark.parametrize("kind,H", [("nf4", 8256), ("nf4", 17 * 1024 + 64), ("q8_0", 8256), ("q8_0", 16384), ("bf16", 8200),
                                    ("bf16", 24 * 1024 + 8), ("fp32", 8200), ("fp32", 9216)])
@pytest.mark.parametrize("T", [1, 77, 1185])
def test_lookup_of_rows_longer_than_a_ctas_segments(kind, H, T):
    _check_lookup(kind, 70, H, T, torch.bfloat16 if T != 77 else torch.float32, T == 77)


# ----------------------------------------------------------------- gradient

def _ids(g, T, V, how):
    if how == "one":
        return torch.full((T,), V - 1, device=DEV)
    if how == "zipf":
        return torch.exp(torch.rand(T, generator=g, device=DEV, dtype=torch.float64) * np.log(V)).long().clamp(1, V) - 1
    if how == "runs":
        return torch.randint(0, min(V, 3), (T,), generator=g, device=DEV)
    return torch.randint(0, V, (T,), generator=g, device=DEV)


def _check_grad(T, V, H, how, acc, dyt, det, idt=torch.int64, pad=-1, bad=False):
    g = torch.Generator(device=DEV).manual_seed(T * 7 + V)
    ids = _ids(g, T, V, how)
    if bad:
        ids[torch.arange(0, T, 11, device=DEV)] = V
        ids[torch.arange(5, T, 13, device=DEV)] = -7
    dY = torch.randint(-3, 4, (T, H), generator=g, device=DEV).to(dyt)
    old = torch.randint(-64, 65, (V, H), generator=g, device=DEV).to(det)            # exact in bfloat16 too
    dE = old.clone() if acc else torch.full((V, H), float("nan"), dtype=det, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(T, V, H), dtype=torch.uint8, device=DEV).fill_(0xA5)
    q.qlora_embed_grad(ids.to(idt), dY, 0.5, dE, padding_id=pad, accumulate=acc, ws=ws)
    if bad:
        with pytest.raises(q.QloraError, match="token id"):
            q.qlora_sync_status()
    else:
        q.qlora_sync_status()
    live = (ids >= 0) & (ids < V) & (ids != pad)
    assert 3 * T + 128 < 2 ** 23
    full = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[live], 0.5 * dY[live].double())
    if acc:
        full += old.double()
    want = full.float().to(det)
    wrong = (dE != want).any(dim=1).nonzero().flatten()
    assert wrong.numel() == 0, f"{wrong.numel()} rows differ, first {wrong[:5].tolist()}"


F32, BF16 = torch.float32, torch.bfloat16
LENGTHS = [1, 2, 5, 64, 129, 191, 192, 193, 255, 1024, 1025, 2047, 2048, 2049, 4097, 8193, 16384, 16385, 32768, 32769, 70_001, 131_071,
           131_072, 131_073, 152_000, 262_145]


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("how", ["one", "zipf", "runs", "any"])
def test_grad_of_whole_numbers_is_exact(T, how):
    for i, (V, H) in enumerate([(700, 16), (40_003, 8)]):
        acc = bool((T + i) & 1)
        _check_grad(T, V, H, how, acc, (F32, BF16)[T // 2 & 1], F32)
        _check_grad(T, V, H, how, not acc, BF16, F32, torch.int32, pad=0)


@pytest.mark.parametrize("T,V,H", [(150, 9000, 1160), (1500, 33_000, 2056), (9001, 5000, 1032), (40_000, 3000, 520), (140_000, 900, 264)])
@pytest.mark.parametrize("acc", [False, True])
def test_grad_of_wide_rows_types_and_bad_ids(T, V, H, acc):
    _check_grad(T, V, H, "zipf", acc, BF16, F32, bad=True)
    _check_grad(T, V, H, "zipf", acc, F32, F32, torch.int32, pad=3)
    _check_grad(T, V, H, "any", acc, BF16, BF16, pad=1)
    _check_grad(T, V, H, "runs", acc, F32, BF16, torch.int32)


@pytest.mark.parametrize("V,H,det", [(1, 8, F32), (1, 4104, BF16), (31, 8, BF16), (32, 16, F32), (33, 8, F32), (2049, 8, BF16), (1025, 8200, F32),
                                     (100_001, 24, F32), (7, 20_008, BF16)])
@pytest.mark.parametrize("T", [0, 1, 3, 192, 193, 300, 5000])
def test_grad_writes_every_row_of_the_table(V, H, det, T):
    # rows without a token become zero for every split of the table over CTAs; nothing behind it is touched
    g = torch.Generator(device=DEV).manual_seed(V + T)
    ids = torch.randint(0, V, (T,), generator=g, device=DEV)
    ids = torch.where(ids % 3 == 1, ids, ids // 2)
    dY = torch.randint(-3, 4, (T, H), generator=g, device=DEV).to(BF16)
    buf = torch.full((V * H + 64,), float("nan"), dtype=det, device=DEV)
    dE = buf[:V * H].view(V, H)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(T, V, H), dtype=torch.uint8, device=DEV).fill_(0xFF)
    q.qlora_embed_grad(ids, dY, 2.0, dE, ws=ws)
    q.qlora_sync_status()
    want = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids, 2.0 * dY.double())
    assert torch.equal(dE, want.float().to(det)) and torch.isnan(buf[V * H:]).all()


@pytest.mark.parametrize("T", [100, 1500, 9000, 140_000])
def test_grad_right_behind_the_writers_of_its_inputs_and_before_a_reader(T):
    # ids, dY and dE are written by the kernels just before the call, and dE is read just after it, again and again
    g = torch.Generator(device=DEV).manual_seed(T)
    V, H = 20_000, 64
    ids, dY, dE = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, H, device=DEV), torch.empty(V, H, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(T, V, H), dtype=torch.uint8, device=DEV)
    new = [(_ids(g, T, V, how), torch.randint(-3, 4, (T, H), generator=g, device=DEV).float()) for how in ("zipf", "any", "runs", "one") * 4]
    got = []
    for i, d in new:
        dE.fill_(float("nan"))
        ids.copy_(i), dY.copy_(d)
        q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws)
        got.append(dE.clone())
    q.qlora_sync_status()
    for (i, d), x in zip(new, got):
        want = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, i, d.double()).float()
        assert torch.equal(x, want)


@pytest.mark.parametrize("T", [193, 2047, 2049, 3001, 4096, 4097, 9001, 40_000, 140_000])
@pytest.mark.parametrize("V,H,det", [(20_000, 520, F32), (20_001, 536, F32), (30_011, 520, F32), (9_001, 4104, BF16), (700_001, 24, F32), (3, 5_000_008, F32)])
def test_grad_written_into_large_tables(T, V, H, det):
    # tables around and above the sizes from which another sort is taken and rows are zeroed beside it
    if T * H > 400_000_000:
        T = 200 + T % 7                                    # (rows of 20 MB: a few tokens are enough)
    for how in ("zipf", "one"):
        _check_grad(T, V, H, how, False, BF16, det, pad=2 if how == "zipf" and V > 3 else -1)


# ----------------------------------------------------------------- ends of the ranges

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1.0, 0.01, -3e-39, 1e30, 0.0])
def test_lookup_of_subnormal_huge_and_infinite_values(dtype, scale):
    x = torch.tensor([0.0, -0.0, 1e-38, -3e-39, 1.4e-45, 2 ** -126, 1.17e-38, 3e38, -3e38, 1e9, 7e-9, 65504.0, float("inf"), 1.0, -1.0, 3.3e38])
    table = x.to(dtype).repeat(3, 1).to(DEV)
    for out in (F32, BF16):
        Y = torch.empty(4, 16, dtype=out, device=DEV)
        q.qlora_embed_fwd(table, torch.tensor([2, 0, 1, 1], device=DEV), scale, Y)
        want = (table[0].double() * float(np.float32(scale))).float().to(out)
        for row in Y:
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(row), nan)
            word = torch.int32 if out == F32 else torch.int16
            assert torch.equal(row.view(word)[~nan], want.view(word)[~nan])


@pytest.mark.parametrize("T", [1, 5, 192, 300, 3000, 9000, 140_000])
@pytest.mark.parametrize("acc", [False, True])
def test_grad_of_bad_ids_alone(T, acc):
    V, H = 50, 24
    ids = torch.full((T,), V, device=DEV)
    ids[::2] = -1
    dY, dE = torch.full((T, H), float("nan"), device=DEV), torch.full((V, H), 3.0, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(T, V, H), dtype=torch.uint8, device=DEV).fill_(0xFF)
    q.qlora_embed_grad(ids, dY, 1.0, dE, accumulate=acc, ws=ws)
    with pytest.raises(q.QloraError, match="token id"):
        q.qlora_sync_status()
    assert (dE == (3.0 if acc else 0.0)).all()


@pytest.mark.parametrize("T", [100, 2000, 9000])
@pytest.mark.parametrize("acc", [False, True])
def test_grad_of_a_table_beyond_32_bits_of_elements(T, acc):
    V, H = 530_000, 8192                                   # 2^32 + elements
    g = torch.Generator(device=DEV).manual_seed(T)
    rows = torch.tensor([0, 262_143, 262_144, 262_145, 524_287, 524_288, V - 1], device=DEV)
    ids = rows[torch.randint(0, 7, (T,), generator=g, device=DEV)]
    dY = torch.randint(-3, 4, (T, H), generator=g, device=DEV).to(BF16)
    dE = torch.empty(V, H, dtype=BF16, device=DEV).fill_(1.0 if acc else float("nan"))
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(T, V, H), dtype=torch.uint8, device=DEV)
    q.qlora_embed_grad(ids, dY, 0.5, dE, accumulate=acc, ws=ws)
    q.qlora_sync_status()
    for r in rows.tolist():
        want = 0.5 * dY[ids == r].double().sum(dim=0) + (1.0 if acc else 0.0)
        assert torch.equal(dE[r], want.float().to(BF16)), r
        dE[r] = 1.0 if acc else 0.0
    for lo in range(0, V, 50_000):
        assert (dE[lo:lo + 50_000] == (1.0 if acc else 0.0)).all()


def test_grad_of_tokens_beyond_32_bits_of_elements():
    T, V, H = 270_001, 900, 16_384                         # 2^32 + elements of dY
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.randint(0, V, (T,), generator=g, device=DEV)
    dY = torch.empty(T, H, dtype=BF16, device=DEV)
    for lo in range(0, T, 30_000):
        dY[lo:lo + 30_000] = torch.randint(-3, 4, dY[lo:lo + 30_000].shape, generator=g, device=DEV, dtype=torch.int8)
    dE = torch.empty(V, H, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(T, V, H), dtype=torch.uint8, device=DEV)
    q.qlora_embed_grad(ids, dY, 1.0, dE, ws=ws)
    q.qlora_sync_status()
    for c in (0, 8000, H - 64):
        want = torch.zeros(V, 64, dtype=torch.float64, device=DEV).index_add_(0, ids, dY[:, c:c + 64].double())
        assert torch.equal(dE[:, c:c + 64], want.float())


@pytest.mark.parametrize("T,V,H", [(100, 9000, 264), (1500, 9000, 264), (3001, 20_500, 520), (9001, 30_100, 520), (140_000, 30_100, 520)])
def test_written_grad_captured_and_replayed_on_two_streams_at_once(T, V, H):
    g = torch.Generator(device=DEV).manual_seed(T)
    work = []
    for _ in range(2):
        ids, dY = torch.zeros(T, dtype=torch.int64, device=DEV), torch.zeros(T, H, dtype=BF16, device=DEV)
        dE, ws = torch.empty(V, H, device=DEV), torch.empty(q.qlora_embed_grad_workspace_bytes(T, V, H), dtype=torch.uint8, device=DEV)
        graph, stream, copies = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.empty(2, V, H, device=DEV)
        with torch.cuda.graph(graph):
            for i in range(2):                             # twice, with the same scratch; dE is read in between
                dE.fill_(float("nan"))
                q.qlora_embed_grad(ids, dY, 1.0, dE, padding_id=1, ws=ws)
                copies[i].copy_(dE)
        work.append((ids, dY, graph, stream, copies, dE, ws))      # (kept: the graph writes to their addresses)
    for how in ("zipf", "any", "one", "runs", "zipf"):
        for ids, dY, *_ in work:
            ids.copy_(_ids(g, T, V, how)), dY.copy_(torch.randint(-3, 4, (T, H), generator=g, device=DEV))
        torch.cuda.synchronize()
        for _, _, graph, stream, *_ in work:
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        q.qlora_sync_status()
        for ids, dY, _, _, copies, *_ in work:
            live = ids != 1
            want = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[live], dY[live].double()).float()
            assert torch.equal(copies[0], want) and torch.equal(copies[1], want), how
