"""What the training-step calls leave to their caller: which error is reported, what a plan keeps and lists."""
import gc
import weakref

import pytest
import torch

import bit_quantized_base_nf4_b200 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("order", ["timeout first", "id first"])
@pytest.mark.parametrize("call", ["lookup", "gradient"])
def test_a_bad_id_does_not_hide_a_timeout(order, call):
    ids = torch.tensor([0, 99, -1], device=DEV)
    E, Y = torch.ones(10, 64, device=DEV), torch.ones(3, 64, device=DEV)
    ws = torch.empty(q.qlora_embed_grad_workspace_bytes(3, 10, 64), dtype=torch.uint8, device=DEV)

    def bad_ids():
        if call == "lookup":
            q.qlora_embed_fwd(E, ids, 1.0, Y)
        else:
            q.qlora_embed_grad(ids, Y, 1.0, E, ws=ws)

    q.qlora_sync_status()
    q.qlora_set_wait_limit_ns(20_000_000)
    try:
        for f in ((q.qlora_probe_wait_timeout, bad_ids) if order == "timeout first" else (bad_ids, q.qlora_probe_wait_timeout)):
            f()
        with pytest.raises(q.QloraError) as e:
            q.qlora_sync_status()
        assert e.value.status == 6 and "timed out" in str(e.value)
    finally:
        q.qlora_set_wait_limit_ns(2_000_000_000)
    q.qlora_sync_status()                                  # reported once
    bad_ids()
    with pytest.raises(q.QloraError, match="token id"):
        q.qlora_sync_status()


def test_a_plan_keeps_its_buffers_when_a_field_is_assigned_anew():
    t = q.AdamWTensor.zeros(torch.zeros(5000, device=DEV), torch.ones(5000, device=DEV), bits=8,
                            param_bf16=torch.zeros(5000, dtype=torch.bfloat16, device=DEV))
    plan = q.qlora_adamw_plan_init([t])
    fields = ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_step", "exp_avg_sq_step", "param_bf16")
    kept = {f: weakref.ref(getattr(t, f)) for f in fields}
    for f in fields:
        setattr(t, f, None)
    gc.collect()
    assert [f for f in fields if kept[f]() is None] == []
    # and the plan still works on them
    q.qlora_adamw_step(plan, 1e-3, 1)
    q.qlora_sync_status()
    assert torch.allclose(kept["param"](), torch.full((5000,), -1e-3, device=DEV), rtol=1e-5)
    del plan
    gc.collect()
    assert [f for f in fields if kept[f]() is not None] == []


def test_plans_made_on_two_streams_hold_the_same_list():
    ts = [q.AdamWTensor.zeros(torch.zeros(n, device=DEV), torch.ones(n, device=DEV), bits=b) for n, b in ((3000, 32), (70_001, 8), (1, 8))]
    side = torch.cuda.Stream()
    one, two = q.qlora_adamw_plan_init(ts), q.qlora_adamw_plan_init(ts, stream=side)
    torch.cuda.synchronize()
    head, used = 256 + 8 * 4096, one.c_plan.chunks * 80
    assert used == 80 * (12 + 274 + 1) and two.c_plan.chunks == one.c_plan.chunks
    assert one.buffer.data_ptr() != two.buffer.data_ptr()
    assert torch.equal(one.buffer[head:head + used], two.buffer[head:head + used])


def test_norm_beyond_float32_keeps_its_coefficient():
    # the norm is worked out in float64: out[0] reads infinity where float32 ends, out[1] is still max_norm / norm
    x = torch.full((1000,), 3e38, device=DEV)
    out = torch.empty(2, device=DEV)
    q.qlora_grad_norm(q.qlora_adamw_plan_init([q.AdamWTensor(None, x)]), 1e6, out)
    want = 1e6 / (1000 ** 0.5 * float(x[0]))
    assert torch.isinf(out[0]) and abs(out[1].item() - want) <= 2.0 ** -23 * want
