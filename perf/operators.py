"""The training-step operators around the frozen-base layer, as measured cases.

Each case is one pass through one operator: an AdamW step over many tensors (32-bit or
8-bit states), the gradient norm with its clip coefficient, an embedding lookup from a
packed or a plain table, or the gradient of an embedding table.  `run` computes the plain
form with elementary torch operations, or makes the library's calls when `own` is true.
Everything an operator updates is returned whole; 8-bit states are returned as the values
they stand for.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 256                    # values per 8-bit state block
BETA1, BETA2, EPS, LR = 0.9, 0.999, 1e-8, 2e-4
MAX_NORM = 0.3

# (n_out, n_in) of the adapted matrices: the 7B attention projections, a 7B layer
# (Q, K, V, O, up, down) and the 70B layer's three matrices
ATTN_7B = [(4096, 4096)] * 4
LAYER_7B = ATTN_7B + [(11008, 4096), (4096, 11008)]
LAYER_70B = [(8192, 8192), (28672, 8192), (8192, 28672)]


def listed():
    return [
        # the adapters of one 7B attention layer at rank 8: the smallest step, bound by latency
        dict(name="adamw32-7b-attn-r8", op="adamw", set="7b-attn", layers=1, r=8, bits=32, param="fp32", grad="fp32",
             copy=True, clip=False),
        # the adapters of a whole 32-layer 7B model at rank 64 (384 tensors, 1.3e8 parameters)
        dict(name="adamw32-7b-32layers-r64", op="adamw", set="7b", layers=32, r=64, bits=32, param="fp32", grad="fp32",
             copy=True, clip=True),
        # the adapters of one 70B-shape layer at rank 64, 8-bit states, clipped
        dict(name="adamw8-70b-layer-r64", op="adamw", set="70b", layers=1, r=64, bits=8, param="fp32", grad="fp32",
             copy=True, clip=True),
        # a bf16 embedding table trained as a whole: one tensor of 1.3e8 parameters
        dict(name="adamw8-table-32000x4096", op="adamw", set="table", V=32000, H=4096, bits=8, param="bf16",
             grad="bf16", copy=False, clip=True),
        # many tensors of odd sizes (norm weights, biases, small heads beside adapters)
        dict(name="adamw8-odd-61", op="adamw", set="odd", count=61, largest=200_003, shape_seed=7, bits=8,
             param="fp32", grad="bf16", copy=False, clip=False),
        # gradient norm before the smallest and the largest of these steps
        dict(name="norm-7b-attn-r8", op="norm", set="7b-attn", layers=1, r=8, grad="fp32"),
        dict(name="norm-7b-32layers-r64", op="norm", set="7b", layers=32, r=64, grad="fp32"),
        # one generated token: its row of a 4-bit table
        dict(name="embed-nf4-1", op="embed", table="nf4", V=32000, H=4096, T=1, fmt=0, out="bf16", ids=64, scale=1.0),
        # a large training batch from a 4-bit table of the 70B width
        dict(name="embed-nf4-16384", op="embed", table="nf4", V=32000, H=8192, T=16384, fmt=0, out="bf16", ids=64,
             scale=1.0),
        # a ragged batch from an 8-bit table, scaled by the root of the width
        dict(name="embed-q8_0-2047", op="embed", table="q8_0", V=32003, H=4096, T=2047, fmt=0, out="bf16", ids=32,
             scale=64.0),
        # one sequence into the gradient of a 7B-width table, written whole
        dict(name="embed-grad-2047", op="embed_grad", V=32000, H=4096, T=2047, dy="bf16", de="fp32", acc=False, pad=0,
             ids=64, scale=1.0),
        # a large batch added into the gradient of a 70B-width table
        dict(name="embed-grad-32768-acc", op="embed_grad", V=32000, H=8192, T=32768, dy="bf16", de="fp32", acc=True,
             pad=-1, ids=64, scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "norm", "embed", "embed_grad"])
    if op in ("adamw", "norm"):
        kind = rng.choice(["7b", "70b", "table", "odd", "odd"])
        c = dict(op=op, set=kind, grad=rng.choice(["fp32", "bf16"]))
        if kind == "7b":
            c.update(layers=_log(rng, 1, 32), r=8 * rng.randint(1, 8))
        elif kind == "70b":
            c.update(layers=rng.randint(1, 4), r=8 * rng.randint(1, 8))
        elif kind == "table":
            c.update(V=_log(rng, 1000, 31000), H=64 * rng.randint(1, 64))
        else:
            c.update(count=_log(rng, 1, 400), largest=_log(rng, 1, 300_000), shape_seed=rng.randrange(1 << 30))
        if op == "adamw":
            param = rng.choice(["fp32", "bf16"])
            c.update(bits=rng.choice([8, 32]), param=param, copy=param == "fp32" and rng.random() < 0.5,
                     clip=rng.random() < 0.5)
        return c
    c = dict(op=op, V=_log(rng, 500, 32100), T=_log(rng, 1, 16384), ids=rng.choice([32, 64]),
             scale=rng.choice([1.0, 0.5, 45.25, 64.0]))
    if op == "embed":
        table = rng.choice(["nf4", "nf4", "fp4", "q8_0", "bf16", "fp32"])
        fmt = rng.choice([0, 0, 1, 2, 3]) if table in ("nf4", "fp4") else 0
        step = 128 if fmt & 1 else 64 if table in ("nf4", "fp4", "q8_0") else 8
        c.update(table=table, fmt=fmt, H=step * rng.randint(1, 8192 // step), out=rng.choice(["bf16", "bf16", "fp32"]))
    else:
        c.update(H=8 * rng.randint(1, 1024), dy=rng.choice(["bf16", "bf16", "fp32"]),
                 de=rng.choice(["fp32", "fp32", "bf16"]), acc=rng.random() < 0.5,
                 pad=rng.choice([-1, 0, 3]))
    return c


# ------------------------------------------------------------------ inputs

def _sizes(c):
    """Numbers of elements of a case's tensors."""
    if c["set"] == "table":
        return [c["V"] * c["H"]]
    if c["set"] == "odd":
        rng = random.Random(c["shape_seed"])
        return [_log(rng, 1, c["largest"]) for _ in range(c["count"])]
    mats = {"7b-attn": ATTN_7B, "7b": LAYER_7B, "70b": LAYER_70B}[c["set"]] * c["layers"]
    return [n for n_out, n_in in mats for n in (c["r"] * n_in, c["r"] * n_out)]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _dtype(name):
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[name]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV, dtype=torch.float32)


def _optimizer_inputs(c, seed):
    """Parameters, gradients and states of the tensors, each tensor a slice of one flat
    buffer a kind that starts at a block of 256; what lies between tensors is zero."""
    g, sizes = _gen(seed), _sizes(c)
    blocks = [-(-n // BLOCK) for n in sizes]
    nb = sum(blocks)
    live = torch.ones(nb, BLOCK, dtype=torch.bool, device=DEV)
    starts, b = [], 0
    for n, k in zip(sizes, blocks):
        starts.append(b * BLOCK)
        if n % BLOCK:
            live[b + k - 1, n % BLOCK:] = False
        b += k
    s = dict(sizes=sizes, starts=starts, nb=nb)
    # gradient magnitudes differ from row to row by orders of magnitude, as real ones do
    mag = torch.exp(1.5 * _randn(g, nb, 1)) * 1e-3
    s["grad"] = (_randn(g, nb, BLOCK) * mag * live).to(_dtype(c["grad"]))
    if c["op"] == "norm":
        return s
    s["param"] = (_randn(g, nb, BLOCK) * 0.02 * live).to(_dtype(c["param"]))
    s["copy"] = s["param"].to(torch.bfloat16) if c["copy"] else None
    if c["bits"] == 32:
        s["m"] = _randn(g, nb, BLOCK) * mag * 0.3 * live
        s["v"] = (_randn(g, nb, BLOCK) * mag).square() * live
    else:
        # what some earlier step left: codes of blocks whose largest value is about 3 sigma
        s["m"] = ((_randn(g, nb, BLOCK) / 3).clamp(-1, 1) * live).to(torch.float32)
        s["m"] = (s["m"].sign() * s["m"].abs().sqrt() * 127).round().to(torch.int8)
        s["m_step"] = (mag * 0.9 / 127 ** 2).reshape(-1).contiguous()
        s["v"] = ((_rand(g, nb, BLOCK).sqrt() * 255).round() * live).to(torch.uint8)
        s["v_step"] = (mag * 3 / 255 ** 2).reshape(-1).contiguous()
    per = torch.tensor(blocks, device=DEV)
    # B learns at four times A's rate (every second tensor); single vectors do not decay
    lr = torch.tensor([4.0 if i % 2 else 1.0 for i in range(len(sizes))], device=DEV)
    wd = torch.tensor([0.0 if n < 20000 else 0.01 for n in sizes], device=DEV)
    s["lr_scales"], s["decays"] = lr.tolist(), wd.tolist()
    s["lr"] = (lr * LR).repeat_interleave(per)[:, None]
    s["wd"] = wd.repeat_interleave(per)[:, None]
    s["coef"] = (_rand(g, 1) * 0.8 + 0.1) if c["clip"] else None
    s["step"] = 100
    return s


def _ids(g, c):
    """Token ids: Zipf-like counts, the frequent tokens anywhere in the vocabulary."""
    V, T = c["V"], c["T"]
    rank = torch.exp(_rand(g, T).double() * math.log(V)).long().clamp(1, V) - 1
    perm = torch.randperm(V, generator=g, device=DEV)
    return perm[rank].to(torch.int64 if c["ids"] == 64 else torch.int32)


def _levels(table):
    if table == "fp4":
        mags = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
        return torch.tensor([-m / 6 for m in reversed(mags)] + [m / 6 for m in mags], dtype=torch.float64).float()
    delta = 0.5 * ((1 - 1 / 30) + (1 - 1 / 32))
    q = lambda n: torch.special.ndtri(0.5 + torch.arange(1, n + 1, dtype=torch.float64) * (delta - 0.5) / n)  # noqa: E731
    top = torch.special.ndtri(torch.tensor(delta, dtype=torch.float64))
    lv = torch.cat([-q(7).flip(0) / top, torch.zeros(1, dtype=torch.float64), q(8) / top])
    lv[0], lv[-1] = -1, 1
    return lv.float()


def _table(g, c):
    """The packed or plain table a program holds, as its buffers."""
    V, H, t = c["V"], c["H"], {}
    if c["table"] in ("nf4", "fp4"):
        B = 128 if c["fmt"] & 1 else 64
        nblk = V * H // B
        t["codes"] = torch.randint(0, 256, (V * H // 2,), generator=g, device=DEV, dtype=torch.uint8)
        if c["fmt"] & 2:
            t["scales"], t["scales2"] = _rand(g, nblk) * 0.05 + 0.01, torch.empty(0, device=DEV)
        else:
            t["scales"] = torch.randint(60, 256, (nblk,), generator=g, device=DEV, dtype=torch.uint8)
            t["scales2"] = _rand(g, -(-nblk // 256)) * 1e-4 + 2e-4
        t["levels"] = _levels(c["table"]).to(DEV)
    elif c["table"] == "q8_0":
        t["q"] = torch.randint(-127, 128, (V * H,), generator=g, device=DEV, dtype=torch.int8)
        t["d"] = (_rand(g, V * H // 32) * 4e-4 + 1e-4).half()
    else:
        t["table"] = (_randn(g, V, H) * 0.02).to(_dtype(c["table"]))
    return t


def prepare(case, seed):
    c = case
    if c["op"] in ("adamw", "norm"):
        s = dict(case=c, **_optimizer_inputs(c, seed))
        if own:
            import bit_quantized_base_nf4_b200 as q

            def part(name, i):
                t = s.get(name)
                return None if t is None else t.view(-1)[s["starts"][i]:s["starts"][i] + s["sizes"][i]]

            def steps(name, i):
                t = s.get(name)
                return None if t is None else t[s["starts"][i] // BLOCK:][:-(-s["sizes"][i] // BLOCK)]

            n = range(len(s["sizes"]))
            if c["op"] == "norm":
                s["plan"] = q.qlora_adamw_plan_init([q.AdamWTensor(param=None, grad=part("grad", i)) for i in n])
                s["out"] = torch.empty(2, dtype=torch.float32, device=DEV)
            else:
                s["plan"] = q.qlora_adamw_plan_init([q.AdamWTensor(
                    param=part("param", i), grad=part("grad", i), exp_avg=part("m", i), exp_avg_sq=part("v", i),
                    exp_avg_step=steps("m_step", i), exp_avg_sq_step=steps("v_step", i),
                    param_bf16=part("copy", i), lr_scale=s["lr_scales"][i], weight_decay=s["decays"][i]) for i in n])
                if c["bits"] == 8:
                    s["m_value"], s["v_value"] = (torch.empty(s["nb"], BLOCK, device=DEV) for _ in range(2))
        return s
    g = _gen(seed)
    s = dict(case=c, ids=_ids(g, c))
    if c["op"] == "embed":
        s.update(_table(g, c))
        if own:
            import bit_quantized_base_nf4_b200 as q

            s["Y"] = torch.empty(c["T"], c["H"], dtype=_dtype(c["out"]), device=DEV)
            if c["table"] in ("nf4", "fp4"):
                s["weight"] = q.NF4Weight(c["V"], c["H"], s["codes"], s["scales"], s["scales2"],
                                          q.QLORA_QT_FP4 if c["table"] == "fp4" else q.QLORA_QT_NF4, c["fmt"])
            elif c["table"] == "q8_0":
                s["weight"] = q.Q80Weight(c["V"], c["H"], s["q"], s["d"])
        return s
    s["dY"] = _randn(g, c["T"], c["H"]).to(_dtype(c["dy"]))
    s["dE"] = (_randn(g, c["V"], c["H"]) if c["acc"] else torch.zeros(c["V"], c["H"], device=DEV)).to(_dtype(c["de"]))
    if own:
        import bit_quantized_base_nf4_b200 as q

        s["ws"] = torch.empty(q.qlora_embed_grad_workspace_bytes(c["T"], c["V"], c["H"]), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return {"adamw": _adamw, "norm": _norm, "embed": _embed, "embed_grad": _embed_grad}[state["case"]["op"]](state)


def _f32(x):
    """x as the float32 value that a float32 operation sees."""
    return float(torch.tensor(x, dtype=torch.float64).float())


def _encode8(x, top):
    """x [blocks, 256] >= 0 as k^2 d: the step d of each block and the nearest k (ties down)."""
    a = x.amax(dim=1, keepdim=True)
    d = a / torch.full_like(a, top * top)      # a divisor on the device: a host scalar would multiply by its reciprocal
    d = torch.where(d < 2.0 ** -126, torch.zeros_like(d), d)
    y = x * torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    j = torch.arange(top, device=x.device, dtype=torch.float32)
    return torch.bucketize(y, j * j + j + 0.5, out_int32=True), d


def _adamw(s):
    c = s["case"]
    s["step"] += 1
    if own:
        import bit_quantized_base_nf4_b200 as q

        q.qlora_adamw_step(s["plan"], LR, s["step"], BETA1, BETA2, EPS, grad_scale=s["coef"])
        if c["bits"] == 8:
            q.qlora_adam8_decode(s["m"], s["m_step"], s["m_value"])
            q.qlora_adam8_decode(s["v"], s["v_step"], s["v_value"])
    else:
        g = s["grad"].float()
        if s["coef"] is not None:
            g = g * s["coef"]
        if c["bits"] == 8:
            km = s["m"].float()
            m = km * km.abs() * s["m_step"][:, None]
            w = s["v"].float().square() * s["v_step"][:, None]
            v = w * w
        else:
            m, v = s["m"], s["v"]
        m = m * _f32(BETA1) + g * _f32(1 - BETA1)
        v = v * _f32(BETA2) + (g * g) * _f32(1 - BETA2)
        w = v.sqrt()
        bc1, bc2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
        p = s["param"].float()
        p = p - s["lr"] * (s["wd"] * p + (m / bc1) / (w / math.sqrt(bc2) + EPS))
        s["param"].copy_(p)
        if s["copy"] is not None:
            s["copy"].copy_(p)
        if c["bits"] == 8:
            k, d = _encode8(m.abs(), 127)
            km = torch.where(m < 0, -k, k).float()
            s["m"].copy_(km)
            s["m_step"].copy_(d[:, 0])
            s["m_value"] = km * km.abs() * d
            k, d = _encode8(w, 255)
            s["v"].copy_(k)
            s["v_step"].copy_(d[:, 0])
            s["v_value"] = (k.float().square() * d).square()
        else:
            s["m"].copy_(m)
            s["v"].copy_(v)
    value = "_value" if c["bits"] == 8 else ""
    out = dict(param=s["param"], m=s["m" + value], v=s["v" + value])
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


def _norm(s):
    if own:
        import bit_quantized_base_nf4_b200 as q

        q.qlora_grad_norm(s["plan"], MAX_NORM, s["out"])
        return s["out"]
    n = s["grad"].double().square().sum().sqrt()
    return torch.stack([n, (MAX_NORM / (n + 1e-6)).clamp(max=1.0)]).float()


def _embed(s):
    c = s["case"]
    if own:
        import bit_quantized_base_nf4_b200 as q

        if c["table"] in ("nf4", "fp4"):
            q.qlora_embed_nf4_fwd(s["weight"], s["ids"], c["scale"], s["Y"])
        elif c["table"] == "q8_0":
            q.qlora_embed_q8_0_fwd(s["weight"], s["ids"], c["scale"], s["Y"])
        else:
            q.qlora_embed_fwd(s["table"], s["ids"], c["scale"], s["Y"])
        return s["Y"]
    ids, H, V = s["ids"].long(), c["H"], c["V"]
    if c["table"] in ("nf4", "fp4"):
        B = 128 if c["fmt"] & 1 else 64
        b = s["codes"].view(V, H // 2)[ids]
        code = torch.stack([b & 15, b >> 4], dim=2).view(-1, H).int()
        blk = ids[:, None] * (H // B) + torch.arange(H // B, device=DEV)
        a = s["scales"][blk].float()
        if not c["fmt"] & 2:
            a = a * s["scales2"][blk // 256]
        w = s["levels"][code].view(-1, H // B, B) * a[:, :, None]
    elif c["table"] == "q8_0":
        w = s["q"].view(V, H // 32, 32)[ids].float() * s["d"].view(V, H // 32, 1)[ids].float()
    else:
        w = s["table"][ids].float()
    return (w * c["scale"]).view(-1, H).to(_dtype(c["out"]))


def _embed_grad(s):
    c = s["case"]
    if own:
        import bit_quantized_base_nf4_b200 as q

        q.qlora_embed_grad(s["ids"], s["dY"], c["scale"], s["dE"], padding_id=c["pad"], accumulate=c["acc"], ws=s["ws"])
        return s["dE"]
    rows = s["dY"].float() * c["scale"]
    rows = torch.where((s["ids"] == c["pad"])[:, None], torch.zeros_like(rows), rows)
    dE = s["dE"].float() if c["acc"] else torch.zeros(c["V"], c["H"], device=DEV)
    s["dE"].copy_(dE.index_add_(0, s["ids"].long(), rows))
    return s["dE"]


# ------------------------------------------------------------------ what a pass cannot do without

def _distinct(c):
    """Expected number of distinct tokens under _ids (each rank r is drawn with probability log(1 + 1/r) / log V)."""
    V, T = c["V"], c["T"]
    r = torch.arange(1, V, dtype=torch.float64)
    return float((1 - (1 - torch.log1p(1 / r) / math.log(V)) ** T).sum())


def work(case):
    c = case
    if c["op"] in ("adamw", "norm"):
        n, g = sum(_sizes(c)), 2 if c["grad"] == "bf16" else 4
        if c["op"] == "norm":
            return dict(bytes=n * g + 8, flops=2 * n)
        p = 4 if c["param"] == "bf16" else 8                      # read and written
        state = 16 if c["bits"] == 32 else 4 + 16 / BLOCK + 8      # 8-bit: codes and steps, and the values returned
        return dict(bytes=n * (g + p + state + (2 if c["copy"] else 0)), flops=20 * n)
    T, H = c["T"], c["H"]
    idb = T * c["ids"] // 8
    u = _distinct(c)
    if c["op"] == "embed":
        per = {"nf4": 0.5, "fp4": 0.5, "q8_0": 1 + 2 / 32, "bf16": 2, "fp32": 4}[c["table"]]
        if c["table"] in ("nf4", "fp4"):
            per += (4 if c["fmt"] & 2 else 1 + 4 / 256) / (128 if c["fmt"] & 1 else 64)
        return dict(bytes=idb + u * H * per + T * H * (2 if c["out"] == "bf16" else 4), flops=2 * T * H)
    e = 2 if c["de"] == "bf16" else 4
    rows = 2 * u if c["acc"] else c["V"]
    return dict(bytes=idb + T * H * (2 if c["dy"] == "bf16" else 4) + rows * H * e, flops=2 * T * H)


# ------------------------------------------------------------------ the definitions in 64 bits

def _rn32(x):
    """The float32 rounding that the definition of the 8-bit state names, of a float64 value."""
    return x.float().double()


def _exact8(x, top):
    """Definition of the 8-bit code of x >= 0 (float64 holding float32 values), k by its closed form."""
    d = _rn32(x.max(dim=1).values / (top * top))[:, None]
    d[d < 2.0 ** -126] = 0
    inv = torch.where(d > 0, _rn32(1 / d), d)
    y = _rn32(x * inv)
    k = torch.ceil(torch.sqrt((y - 0.25).clamp(min=0)) - 0.5).clamp(0, top)
    return k, d


def exact(case, seed):
    global own
    c, was = case, own
    own = False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["op"] == "norm":
        n = torch.linalg.vector_norm(s["grad"].double())
        return torch.stack([n, torch.minimum(torch.ones_like(n), MAX_NORM / (n + 1e-6))])
    if c["op"] == "adamw":
        t, eight = 101, c["bits"] == 8
        rn = _rn32 if eight else (lambda x: x)                    # the 8-bit definition fixes every rounding up to the code
        b1, w1, b2, w2 = (_f32(x) for x in (BETA1, 1 - BETA1, BETA2, 1 - BETA2)) if eight else (
            BETA1, 1 - BETA1, BETA2, 1 - BETA2)
        g = s["grad"].double()
        if s["coef"] is not None:
            g = rn(g * s["coef"].double())
        m, v = s["m"].double(), s["v"].double()
        if eight:
            m = rn(m * m.abs() * s["m_step"].double()[:, None])
            v = rn(v * v * s["v_step"].double()[:, None])
            v = rn(v * v)
        m = rn(rn(b1 * m) + rn(w1 * g))
        v = rn(rn(b2 * v) + rn(w2 * rn(g * g)))
        del g
        w = rn(v.sqrt())
        p = s["param"].double()
        p = p - s["lr"].double() * (s["wd"].double() * p + m / (1 - BETA1 ** t) / (w / math.sqrt(1 - BETA2 ** t) + EPS))
        out = dict(param=p)
        if c["copy"]:
            out["copy"] = p
        if eight:
            k, d = _exact8(m.abs(), 127)
            out["m"] = m.sign() * k * k * d
            k, d = _exact8(w, 255)
            out["v"] = (k * k * d).square()
        else:
            out["m"], out["v"] = m, v
        return out
    if c["op"] == "embed":
        # row by row of the table: dequantize every row that occurs once, then copy it to its tokens
        rows, back = torch.unique(s["ids"].long(), return_inverse=True)
        H, V = c["H"], c["V"]
        if c["table"] in ("nf4", "fp4"):
            B = 128 if c["fmt"] & 1 else 64
            b = s["codes"].view(V, H // 2)[rows]
            lv = s["levels"].double()
            w = torch.empty(len(rows), H, dtype=torch.float64, device=DEV)
            w[:, 0::2], w[:, 1::2] = lv[(b % 16).long()], lv[(b // 16).long()]
            a = s["scales"].double()
            if not c["fmt"] & 2:
                a = a * s["scales2"].double().repeat_interleave(256)[:a.numel()]
            w = w * a.view(V, H // B)[rows].repeat_interleave(B, dim=1)
        elif c["table"] == "q8_0":
            w = s["q"].view(V, H)[rows].double() * s["d"].view(V, H // 32)[rows].double().repeat_interleave(32, dim=1)
        else:
            w = s["table"][rows].double()
        return (w * c["scale"])[back]
    # gradient: tokens in order of their id, running sums, and the difference at each id's last token
    ids, order = torch.sort(s["ids"].long(), stable=True)
    dE = s["dE"].double() if c["acc"] else torch.zeros(c["V"], c["H"], dtype=torch.float64, device=DEV)
    rows, counts = torch.unique_consecutive(ids, return_counts=True)
    ends = counts.cumsum(0) - 1
    for h in range(0, c["H"], 1024):
        run_sum = s["dY"][:, h:h + 1024].double()[order].cumsum(0)[ends]
        seg = torch.diff(run_sum, dim=0, prepend=torch.zeros(1, run_sum.shape[1], dtype=torch.float64, device=DEV))
        seg[rows == c["pad"]] = 0
        dE[rows, h:h + 1024] += seg * c["scale"]
    return dE
