"""Host-side checks of the embedding and optimizer calls that need no GPU: sizes, struct
layouts, and refusals before anything is launched."""
import ctypes

import pytest

from bit_quantized_base_nf4_b200 import AdamWTensor, _capi
from bit_quantized_base_nf4_b200 import build as libbuild

P = ctypes.c_void_p
ARG, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
IDS, Y, E, WS = 0x10000, 0x20000, 0x30000, 0x40000


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _capi.load()


def _err(lib):
    return lib.qlora_last_error().decode()


def _fwd(lib, E=E, eb=0, V=100, H=64, ids=IDS, idb=8, T=4, scale=1.0, Y=Y, yb=1):
    return lib.qlora_embed_fwd(P(E), eb, V, H, P(ids), idb, T, scale, P(Y), yb, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(E=None), ARG, "E is NULL"), (dict(E=E + 8), ALIGN, "E must"), (dict(eb=2), ARG, "e_is_bf16"),
    (dict(V=0), SHAPE, "V and H"), (dict(V=1 << 31), SHAPE, "V and H"), (dict(H=0), SHAPE, "V and H"),
    (dict(H=12), SHAPE, "multiple of 8"), (dict(T=-1), SHAPE, "T (-1)"), (dict(T=1 << 31), SHAPE, "T"),
    (dict(idb=2), ARG, "ids_bytes"), (dict(ids=None), ARG, "ids is NULL"), (dict(ids=IDS + 4), ALIGN, "ids must"),
    (dict(scale=float("nan")), ARG, "scale"), (dict(scale=float("inf")), ARG, "scale"), (dict(Y=None), ARG, "Y is NULL"),
    (dict(Y=Y + 4), ALIGN, "Y must"), (dict(yb=3), ARG, "y_is_bf16"),
    (dict(H=1 << 30), SHAPE, "too large"),
])
def test_embed_fwd_refusals(lib, kw, code, msg):
    assert _fwd(lib, **kw) == code and msg in _err(lib), _err(lib)


def test_embed_fwd_of_nothing_is_ok(lib):
    assert _fwd(lib, T=0, ids=None, Y=None) == 0
    w = _capi.Nf4WeightC(100, 64, 0x1000, 0x2000, 0x3000)
    assert lib.qlora_embed_nf4_fwd(ctypes.byref(w), None, 4, 0, 1.0, None, 0, None) == 0
    w8 = _capi.Q80WeightC(100, 64, 0x1000, 0x2000)
    assert lib.qlora_embed_q8_0_fwd(ctypes.byref(w8), None, 4, 0, 1.0, None, 0, None) == 0


def test_embed_packed_refusals(lib):
    assert lib.qlora_embed_nf4_fwd(None, P(IDS), 8, 4, 1.0, P(Y), 1, None) == ARG
    assert lib.qlora_embed_q8_0_fwd(None, P(IDS), 8, 4, 1.0, P(Y), 1, None) == ARG
    w = _capi.Nf4WeightC(100, 96, 0x1000, 0x2000, 0x3000)
    assert lib.qlora_embed_nf4_fwd(ctypes.byref(w), P(IDS), 8, 4, 1.0, P(Y), 1, None) == SHAPE
    w = _capi.Nf4WeightC(100, 64, 0x1000, 0x2000, 0x3000)
    assert lib.qlora_embed_nf4_fwd(ctypes.byref(w), P(IDS), 8, 4, 1.0, P(Y + 2), 1, None) == ALIGN
    assert lib.qlora_embed_nf4_fwd(ctypes.byref(w), P(IDS), 8, 4, float("nan"), P(Y), 1, None) == ARG
    w8 = _capi.Q80WeightC(100, 64, 0x1000, 0x2001)
    assert lib.qlora_embed_q8_0_fwd(ctypes.byref(w8), P(IDS), 8, 4, 1.0, P(Y), 1, None) == ALIGN


def _grad(lib, ids=IDS, idb=8, T=40, dY=Y, yb=1, V=100, H=64, scale=1.0, pad=-1, dE=E, eb=0, acc=0, ws=WS, wsb=1 << 30):
    return lib.qlora_embed_grad(P(ids), idb, T, P(dY), yb, V, H, scale, pad, P(dE), eb, acc, P(ws), wsb, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(ids=None), ARG, "ids is NULL"), (dict(ids=IDS + 1), ALIGN, "ids"), (dict(idb=3), ARG, "ids_bytes"),
    (dict(T=-2), SHAPE, "T"), (dict(H=60), SHAPE, "multiple of 8"), (dict(V=0), SHAPE, "V and H"),
    (dict(dY=None), ARG, "non-NULL"), (dict(dE=None), ARG, "non-NULL"), (dict(dY=Y + 8), ALIGN, "dY"),
    (dict(dE=E + 8), ALIGN, "dE"), (dict(yb=2), ARG, "dy_is_bf16"), (dict(eb=-1), ARG, "de_is_bf16"),
    (dict(acc=2), ARG, "accumulate"), (dict(scale=float("inf")), ARG, "scale"), (dict(pad=100), ARG, "padding_id"),
    (dict(pad=-2), ARG, "padding_id"), (dict(ws=None), WORKSPACE, "workspace"), (dict(wsb=100), WORKSPACE, "workspace"),
    (dict(ws=WS + 8), ALIGN, "workspace"), (dict(H=1 << 30, wsb=1 << 60), SHAPE, "at most"),
])
def test_embed_grad_refusals(lib, kw, code, msg):
    assert _grad(lib, **kw) == code and msg in _err(lib), _err(lib)


def test_embed_grad_of_nothing_added_is_ok(lib):
    assert _grad(lib, T=0, ids=None, dY=None, ws=None, wsb=0, acc=1) == 0


def test_embed_grad_workspace(lib):
    f = lib.qlora_embed_grad_workspace_bytes
    for T, V, H in [(1, 10, 8), (40, 100, 64), (32768, 32000, 8192), (1 << 20, 300000, 128)]:
        assert f(T, V, H) >= 16 * T                      # two lists of ids and positions at least
    assert f(0, 10, 8) > 0
    for bad in [(-1, 10, 8), (1, 0, 8), (1, 10, 0), (1, 10, 12), (1 << 31, 10, 8), (1, 1 << 31, 8)]:
        assert f(*bad) == 0
    n = f(40, 100, 64)
    assert _grad(lib, wsb=n - 1) == WORKSPACE


def _tensor(at=0, **kw):
    t = dict(param=0x10000, grad=0x20000, exp_avg=0x30000, exp_avg_sq=0x40000, numel=1000, lr_scale=1.0,
             weight_decay=0.0, flags=0)
    t = {k: v + at if k in ("param", "grad", "exp_avg", "exp_avg_sq") else v for k, v in t.items()}
    t.update(kw)
    return _capi.AdamWTensorC(**t)


def test_struct_layouts():
    assert ctypes.sizeof(_capi.AdamWTensorC) == 80 and _capi.AdamWTensorC.flags.offset == 72
    assert ctypes.sizeof(_capi.AdamWPlanC) == 48 and _capi.AdamWPlanC.magic.offset == 36


def test_plan_bytes_count_chunks(lib):
    f = lib.qlora_adamw_plan_bytes
    head = f((_capi.AdamWTensorC * 1)(_tensor(numel=0)), 1)
    assert f((_capi.AdamWTensorC * 1)(_tensor(numel=1)), 1) == head + 80
    assert f((_capi.AdamWTensorC * 1)(_tensor(numel=257)), 1) == head + 160
    # a large plan takes chunks of 1024; each tensor costs the same besides
    n, one = 64 * 148 * 1024, f((_capi.AdamWTensorC * 2)(_tensor(numel=0), _tensor(numel=0)), 2) - head
    assert f((_capi.AdamWTensorC * 2)(_tensor(numel=n), _tensor(numel=1025)), 2) == head + one + (n // 1024 + 2) * 80
    assert f(None, 1) == 0 and f((_capi.AdamWTensorC * 1)(_tensor()), 0) == 0


@pytest.mark.parametrize("kw,code,msg", [
    (dict(numel=-1), SHAPE, "numel"), (dict(flags=16), ARG, "flags"), (dict(grad=None), ARG, "grad is NULL"),
    (dict(grad=0x2004), ALIGN, "grad"), (dict(param=None), ARG, "non-NULL"), (dict(exp_avg=None), ARG, "non-NULL"),
    (dict(exp_avg_sq=None), ARG, "non-NULL"), (dict(param=0x1008), ALIGN, "aligned"), (dict(exp_avg=0x3001), ALIGN, "aligned"),
    (dict(param_bf16=0x5002), ALIGN, "aligned"), (dict(param_bf16=0x5000, flags=1), ARG, "copy"),
    (dict(flags=4), ARG, "block steps"), (dict(flags=4, exp_avg_step=0x6000, exp_avg_sq_step=0x7002), ALIGN, "block steps"),
    (dict(lr_scale=float("nan")), ARG, "lr_scale"), (dict(lr_scale=-1.0), ARG, "lr_scale"),
    (dict(weight_decay=float("inf")), ARG, "weight_decay"),
])
def test_plan_refusals_name_the_tensor(lib, kw, code, msg):
    arr = (_capi.AdamWTensorC * 2)(_tensor(), _tensor(0x100000, **kw))
    plan = _capi.AdamWPlanC()
    st = lib.qlora_adamw_plan_init(arr, 2, P(0x1000000), 1 << 30, ctypes.byref(plan), None)
    assert st == code and msg in _err(lib) and "tensor 1" in _err(lib), _err(lib)
    assert plan.magic == 0 and lib.qlora_adamw_plan_bytes(arr, 2) == 0


STEPS = dict(flags=4, exp_avg_step=0x60000, exp_avg_sq_step=0x70000)


@pytest.mark.parametrize("tensors,which", [
    ([_tensor(), _tensor()], 1),                                             # the same tensor twice
    ([_tensor(), _tensor(0x100000, param=0x10000 + 3984)], 1),               # one 16-byte word shared
    ([_tensor(), _tensor(0x100000, grad=0x30000)], 1),                       # a gradient in another's state
    ([_tensor(exp_avg_sq=0x30000)], 0),                                      # one state for both moments
    ([_tensor(param_bf16=0x20010)], 0),                                      # the copy in the gradient
    ([_tensor(exp_avg_step=0x60000, exp_avg_sq_step=0x6000c, flags=4)], 0),  # overlapping block steps
    ([_tensor(**STEPS), _tensor(0x100000, **STEPS)], 1),
])
def test_overlapping_buffers_are_refused(lib, tensors, which):
    arr = (_capi.AdamWTensorC * len(tensors))(*tensors)
    plan = _capi.AdamWPlanC()
    st = lib.qlora_adamw_plan_init(arr, len(tensors), P(0x1000000), 1 << 30, ctypes.byref(plan), None)
    assert st == ARG and "overlaps" in _err(lib) and f"tensor {which}" in _err(lib), _err(lib)


def test_neighbouring_buffers_and_shared_gradients_are_not_refused(lib):
    arr = (_capi.AdamWTensorC * 3)(_tensor(), _tensor(0x100000, param=0x10000 + 4000), _tensor(0x200000, grad=0x20000))
    plan = _capi.AdamWPlanC()
    st = lib.qlora_adamw_plan_init(arr, 3, P(0x1000000), 1 << 30, ctypes.byref(plan), None)
    assert st not in (ARG, SHAPE, ALIGN, WORKSPACE), _err(lib)      # fails later, for want of a GPU


def test_plan_buffer_refusals(lib):
    arr = (_capi.AdamWTensorC * 1)(_tensor())
    plan = _capi.AdamWPlanC()
    need = lib.qlora_adamw_plan_bytes(arr, 1)
    assert lib.qlora_adamw_plan_init(arr, 1, None, need, ctypes.byref(plan), None) == WORKSPACE
    assert lib.qlora_adamw_plan_init(arr, 1, P(0x100000), need - 1, ctypes.byref(plan), None) == WORKSPACE
    assert lib.qlora_adamw_plan_init(arr, 1, P(0x100010), need, ctypes.byref(plan), None) == ALIGN
    assert lib.qlora_adamw_plan_init(arr, 1, P(0x100000), need, None, None) == ARG
    assert lib.qlora_adamw_plan_init(arr, 0, P(0x100000), need, ctypes.byref(plan), None) == SHAPE


def _plan(**kw):
    p = dict(buffer=0x100000, chunks=4, chunks32=4, numel=1000, grad_only=0, magic=0x51504c4e)
    p.update(kw)
    return _capi.AdamWPlanC(**p)


def _step(lib, plan=None, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, gs=None, lr_dev=None, sd=None):
    p = plan if plan is not None else _plan()
    return lib.qlora_adamw_step(ctypes.byref(p), lr, b1, b2, eps, step, P(gs), P(lr_dev), P(sd), None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(plan=_plan(magic=0)), ARG, "qlora_adamw_plan_init"), (dict(plan=_plan(buffer=None)), ARG, "plan"),
    (dict(plan=_plan(grad_only=1)), ARG, "GRAD_ONLY"), (dict(b1=1.0), ARG, "betas"), (dict(b2=-0.1), ARG, "betas"),
    (dict(b2=float("nan")), ARG, "betas"), (dict(eps=-1e-8), ARG, "eps"), (dict(eps=float("inf")), ARG, "eps"),
    (dict(lr=-1.0), ARG, "lr"), (dict(lr=float("nan")), ARG, "lr"), (dict(step=0), ARG, "step"), (dict(step=-3), ARG, "step"),
    (dict(step=2, sd=0x8000), ARG, "step"), (dict(gs=0x8002), ALIGN, "aligned"), (dict(lr_dev=0x8001), ALIGN, "aligned"),
    (dict(step=0, sd=0x8004), ALIGN, "aligned"),
])
def test_step_refusals(lib, kw, code, msg):
    assert _step(lib, **kw) == code and msg in _err(lib), _err(lib)


def test_norm_and_adam8_refusals(lib):
    p = _plan()
    norm = lambda mx, out: lib.qlora_grad_norm(ctypes.byref(p), mx, P(out), None)  # noqa: E731
    assert norm(0.0, 0x8000) == ARG and norm(-1.0, 0x8000) == ARG and norm(float("nan"), 0x8000) == ARG
    assert norm(1.0, None) == ARG and norm(1.0, 0x8002) == ALIGN
    assert lib.qlora_grad_norm(None, 1.0, P(0x8000), None) == ARG
    for f, args in ((lib.qlora_adam8_encode, lambda k, c, s, x, n: (P(x), k, P(c), P(s), n, None)),
                    (lib.qlora_adam8_decode, lambda k, c, s, x, n: (P(c), k, P(s), P(x), n, None))):
        assert f(*args(2, 0x1000, 0x2000, 0x3000, 10)) == ARG
        assert f(*args(0, 0x1000, 0x2000, 0x3000, -1)) == SHAPE
        assert f(*args(0, None, 0x2000, 0x3000, 10)) == ARG
        assert f(*args(0, 0x1008, 0x2000, 0x3000, 10)) == ALIGN
        assert f(*args(1, 0x1000, 0x2002, 0x3000, 10)) == ALIGN
        assert f(*args(1, None, None, None, 0)) == 0


@pytest.mark.parametrize("b1,eps", [(0.9, 1e-39), (0.9, 1e-45), (0.9, 1e-300), (0.9, 1.1e-37), (1 - 1e-10, 1e-30)])
def test_step_refuses_an_eps_that_would_count_as_zero(lib, b1, eps):
    assert _step(lib, b1=b1, eps=eps) == ARG and "2^-126" in _err(lib)
    assert _step(lib, b1=b1, eps=eps, step=0, sd=0x9000) == ARG and "2^-126" in _err(lib)


@pytest.mark.parametrize("b1,eps", [(0.9, 0.0), (0.9, 1.2e-37), (0.0, 1.2e-38)])
def test_step_takes_the_smallest_eps(lib, b1, eps):
    # refused for its step number only, which is looked at after eps
    assert _step(lib, b1=b1, eps=eps, step=-1) == ARG and "step (-1)" in _err(lib)


def test_a_tensor_without_a_gradient_is_named():
    with pytest.raises(ValueError, match="grad is required"):
        AdamWTensor(None, None).c_struct()
