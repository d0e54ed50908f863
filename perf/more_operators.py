"""Measured passes through the library's operators for adapted and sparse layers.

Each case is one call that a user's program makes: a whole mixture-of-experts
layer for the few tokens of a decode step, a shared projection with the
low-rank adapters of many requests beside it, and the 8-bit checkpoint of an
activation (taken, read back, and used in the backward pass).  ``listed()``
names fixed cases, ``draw(rng)`` gives further ones of the same ranges,
``prepare`` makes the inputs, ``run`` makes one pass, ``work`` states the bytes
and operations a pass cannot do without and ``exact`` computes the same outputs
in 64 bits.

``own`` selects the library's kernels; without it ``run`` computes the plain
form, elementary torch operations in 32 bits.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
ACTS = ("none", "silu", "gelu", "relu")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # Decode, one request: one token through a layer of 64 experts, 8 of
        # them active; bound by their weights, so latency counts.
        dict(name="mlp_one_token", kind="mlp", types="bf16", tokens=1, topk=8, groups=64, width=2048, hidden=1024,
             layout="bt_preshuffled", gated=True, act="silu", bias=False, weighted=True, residual=True, skew=0.0,
             drop=0.0),
        # Decode, a batch of 16 requests that share some of the active experts.
        dict(name="mlp_decode", kind="mlp", types="bf16", tokens=16, topk=4, groups=64, width=2048, hidden=1024,
             layout="bt_preshuffled", gated=True, act="silu", bias=False, weighted=True, residual=True, skew=0.0,
             drop=0.0),
        # Decode of a larger batch with the weights kept in 8 bits, uneven
        # experts, biases, and slots that belong to other ranks.
        dict(name="mlp_e4m3_batch", kind="mlp", types="e4m3", tokens=61, topk=4, groups=24, width=4096, hidden=2112,
             layout="bt", gated=True, act="gelu", bias=True, weighted=True, residual=False, skew=1.0, drop=0.1),
        # The smallest call of a decode loop that serves adapters: one token.
        dict(name="lora_one_token", kind="lora", out="bf16", m=1, n=2048, k=2048, layout="bt_preshuffled", rank=16,
             adapters=8, mix="rows", requests=1, plain=0.0, bias=False, act="none", residual=True, preact=False),
        # Decode of 32 requests, most with an adapter of their own.
        dict(name="lora_decode", kind="lora", out="bf16", m=32, n=8192, k=8192, layout="bt", rank=16, adapters=24,
             mix="rows", requests=32, plain=0.1, bias=False, act="none", residual=True, preact=False),
        # Prompts of six requests packed into one batch of odd length behind a
        # few decode rows.
        dict(name="lora_prompts", kind="lora", out="bf16", m=4001, n=4096, k=4160, layout="bt", rank=64, adapters=16,
             mix="packed", requests=6, plain=0.1, bias=True, act="silu", residual=False, preact=False),
        # Fine-tuning: a whole batch on one adapter, the pre-activation kept.
        dict(name="lora_train", kind="lora", out="bf16", m=8192, n=8192, k=2048, layout="bt_preshuffled", rank=32,
             adapters=1, mix="packed", requests=1, plain=0.0, bias=True, act="silu", residual=True, preact=True),
        # A short prompt's activation into 8 bits: latency.
        dict(name="pack_short", kind="pack", type="f32", m=77, n=2064),
        # A training step's pre-activation into 8 bits.
        dict(name="pack_train", kind="pack", type="bf16", m=8192, n=8192),
        # Backward pass: the activation made again from its 8-bit form, the
        # operand of the next layer's weight gradient.
        dict(name="unpack_train", kind="unpack", type="bf16", m=8192, n=4096, act="silu"),
        # Backward pass: the epilogue's gradient for uneven experts.
        dict(name="grad_experts", kind="grad", type="bf16", m=1013, n=2112, rows=1000, groups=16, act="gelu"),
        # Backward pass: the epilogue's gradient of a training step.
        dict(name="grad_train", kind="grad", type="bf16", m=8192, n=8192, rows=8192, groups=1, act="silu"),
    ]


_FLOP_CAP = 2.0 * 8192 * 8192 * 2048
_WEIGHT_CAP = 5.0e8                     # bytes of the active experts' weights
_ALL_WEIGHTS = 4.2e8                    # elements of all experts' weights


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _mult(rng, lo, hi, step):
    return max(lo, min(hi, _log(rng, lo, hi) // step * step))


def draw(rng):
    kind = rng.choice(["mlp", "mlp", "mlp", "lora", "lora", "lora", "pack", "unpack", "grad"])
    if kind == "mlp":
        width, hidden = _mult(rng, 256, 4096, 64), _mult(rng, 128, 2048, 64)
        gated = rng.random() < 0.7
        per = width * hidden * (3 if gated else 2)
        groups = max(2, min(_log(rng, 4, 128), int(_ALL_WEIGHTS / per)))
        topk = rng.randint(1, min(8, groups))
        types = rng.choice(["bf16", "bf16", "e4m3"])
        tokens = _log(rng, 1, 64)
        while tokens > 1 and _active(tokens, topk, groups) * per * (1 if types == "e4m3" else 2) > _WEIGHT_CAP:
            tokens //= 2
        return dict(kind=kind, types=types, tokens=tokens, topk=topk, groups=groups, width=width, hidden=hidden,
                    layout=rng.choice(["bt", "bt_preshuffled"]), gated=gated, act=rng.choice(ACTS),
                    bias=rng.random() < 0.4, weighted=rng.random() < 0.8, residual=rng.random() < 0.6,
                    skew=rng.choice([0.0, 0.5, 1.0, 2.0]), drop=rng.choice([0.0, 0.0, 0.1, 0.6]))
    if kind == "lora":
        n, k = _mult(rng, 256, 8192, 16), _mult(rng, 256, 8192, 32)
        rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
        out = rng.choice(["bf16", "bf16", "f32"])
        m = _log(rng, 1, min(4096 if out == "f32" else 8192, _FLOP_CAP / (2.0 * (n * k + rank * (n + k)))))
        return dict(kind=kind, out=out, m=m, n=n, k=k, layout=rng.choice(["bt", "bt_preshuffled"]), rank=rank,
                    adapters=_log(rng, 1, 64), mix="rows" if m <= 128 else "packed", requests=_log(rng, 1, 16),
                    plain=rng.choice([0.0, 0.1, 0.5]), bias=rng.random() < 0.5, act=rng.choice(ACTS),
                    residual=rng.random() < 0.6, preact=rng.random() < 0.3)
    m, n, kept = _log(rng, 1, 8192), _mult(rng, 128, 8192, 16), rng.choice(["bf16", "bf16", "f32"])
    if kept == "f32":
        m = min(m, 4096)
    if kind == "pack":
        return dict(kind=kind, type=kept, m=m, n=n)
    if kind == "unpack":
        return dict(kind=kind, type=kept, m=m, n=n, act=rng.choice(ACTS))
    return dict(kind=kind, type=kept, m=m, n=n, rows=m if rng.random() < 0.5 else rng.randint(0, m),
                groups=rng.choice([1, _log(rng, 2, 64)]), act=rng.choice(ACTS))


# ------------------------------------------------------------------ the inputs

def _randn(g, *shape, std=1.0, dtype=BF16):
    x = torch.empty(shape, dtype=F32, device="cuda")
    return x.normal_(0.0, std, generator=g).to(dtype)


def _quantise(x):
    """fp32 -> (e4m3 values, fp32 scales), one scale per row."""
    s = x.abs().amax(dim=-1, keepdim=True).clamp_(min=1e-12) / 448.0
    return (x / s).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), s.squeeze(-1).contiguous()


def _route(g, tokens, topk, groups, skew):
    """Distinct experts per token, some experts more popular than others."""
    pull = torch.empty(groups, device="cuda").normal_(0.0, 1.0, generator=g) * skew
    u = torch.empty((tokens, groups), device="cuda").uniform_(1e-6, 1.0 - 1e-6, generator=g)
    return (pull - torch.log(-torch.log(u))).topk(topk, dim=1).indices


def _ids(g, shape, top):
    return torch.randint(0, top, shape, generator=g, device="cuda")


def _adapters(g, case):
    """The adapter of every row, -1 for none: one per row (decode), or up to 16
    decode rows and then one adapter per packed prompt."""
    m, top = case["m"], case["adapters"]
    if case["mix"] == "rows":
        ids = _ids(g, (m,), top)
        none = torch.empty(m, device="cuda").uniform_(0.0, 1.0, generator=g) < case["plain"]
    else:
        head = min(16, m // 8) if top > 1 else 0
        cuts = (head + _ids(g, (case["requests"] - 1,), m - head)).sort().values
        of = head + (torch.arange(m, device="cuda")[:, None] >= cuts[None, :]).sum(dim=1)
        of = torch.where(torch.arange(m, device="cuda") < head, torch.arange(m, device="cuda"), of)
        ids = _ids(g, (head + case["requests"],), top)[of]
        none = (torch.empty(head + case["requests"], device="cuda").uniform_(0.0, 1.0, generator=g) < case["plain"])[of]
    return torch.where(none, -1, ids).to(torch.int32)


def _mx(x):
    """fp32 -> e4m3 values and the exponent byte of each block of 32 columns."""
    m, n = x.shape
    blocks = (n + 31) // 32
    full = torch.zeros((m, blocks * 32), dtype=F32, device=x.device)
    full[:, :n] = x
    full = full.view(m, blocks, 32)
    top = torch.where(torch.isfinite(full), full.abs(), 0.0).amax(dim=2)
    part, power = torch.frexp(top)
    power = torch.where(part <= 0.875, power - 9, power - 8)
    power = torch.where(top > 0, power, -127).clamp(-127, 127)
    q = (full * torch.exp2(-power.to(F32))[:, :, None]).view(m, blocks * 32)[:, :n]
    return q.to(torch.float8_e4m3fn).contiguous(), (power + 127).to(torch.uint8)


def _offsets(g, groups, rows):
    cuts = torch.randint(0, rows + 1, (groups - 1,), generator=g, device="cuda").sort().values
    return torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows)]).to(torch.int32)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, s = case["kind"], {}
    if kind == "mlp":
        tokens, topk, groups, width, hidden = (case[f] for f in ("tokens", "topk", "groups", "width", "hidden"))
        inner = hidden * (2 if case["gated"] else 1)
        s["x"] = _randn(g, tokens, width)
        ids = _route(g, tokens, topk, groups, case["skew"])
        lost = torch.empty((tokens, topk), device="cuda").uniform_(0.0, 1.0, generator=g) < case["drop"]
        s["ids"] = torch.where(lost, -1, ids).to(torch.int32)
        s["weights"] = torch.softmax(_randn(g, tokens, topk, dtype=F32), dim=1) if case["weighted"] else None
        up, down = (groups, inner, width), (groups, width, hidden)
        if case["types"] == "e4m3":
            s["up"], s["up_scale"] = _quantise(_randn(g, *up, std=width ** -0.5, dtype=F32))
            s["down"], s["down_scale"] = _quantise(_randn(g, *down, std=hidden ** -0.5, dtype=F32))
        else:
            s["up"], s["down"] = _randn(g, *up, std=width ** -0.5), _randn(g, *down, std=hidden ** -0.5)
            s["up_scale"] = s["down_scale"] = None
        s["up_bias"] = _randn(g, groups, inner, std=0.5, dtype=F32) if case["bias"] else None
        s["down_bias"] = _randn(g, groups, width, std=0.5, dtype=F32) if case["bias"] else None
        s["residual"] = _randn(g, tokens, width) if case["residual"] else None
        s["out"] = torch.zeros((tokens, width), dtype=BF16, device="cuda")
    elif kind == "lora":
        m, n, k, rank, top = (case[f] for f in ("m", "n", "k", "rank", "adapters"))
        kept = TYPES[case["out"]]
        s["a"], s["b"] = _randn(g, m, k), _randn(g, n, k, std=k ** -0.5)
        s["adapter"] = _adapters(g, case)
        s["down"] = _randn(g, top, rank, k, std=k ** -0.5)
        s["up"] = _randn(g, top, n, rank, std=0.5 * rank ** -0.5)
        s["scale"] = torch.empty(top, dtype=F32, device="cuda").uniform_(0.5, 2.0, generator=g)
        s["bias"] = _randn(g, n, std=0.5, dtype=F32) if case["bias"] or case["act"] != "none" else None
        s["residual"] = _randn(g, m, n, dtype=kept) if case["residual"] else None
        s["c"] = torch.zeros((m, n), dtype=kept, device="cuda")
        s["preact"] = torch.zeros((m, n), dtype=kept, device="cuda") if case["preact"] else None
    else:
        m, n, kept = case["m"], case["n"], TYPES[case["type"]]
        # rows of different size, as activations have
        z = _randn(g, m, n, std=1.5, dtype=F32) * torch.exp(_randn(g, m, 1, std=0.5, dtype=F32))
        if kind == "pack":
            s["src"] = z.to(kept)
            s["q"] = torch.zeros((m, n), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.zeros((m, (n + 31) // 32), dtype=torch.uint8, device="cuda")
            return s
        q, s["scales"] = _mx(z)
        s["q"] = q.view(torch.uint8)
        s["out"] = torch.zeros((m, n), dtype=kept, device="cuda")
        if kind == "grad":
            s["dc"] = _randn(g, m, n, dtype=kept)
            s["offsets"] = _offsets(g, case["groups"], case["rows"])
            s["dbias"] = torch.zeros((case["groups"], n), dtype=F32, device="cuda")
    return s


def _ptr(t):
    return None if t is None else t.data_ptr()


def _scratch(need):
    return torch.empty(max(16, need), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    kind = case["kind"]
    if not own:
        if kind == "mlp":
            ids = s["ids"].reshape(-1)
            s["slots_of"] = [(e, torch.nonzero(ids == e).flatten()) for e in sorted(set(ids.tolist())) if e >= 0]
        elif kind == "lora":
            s["rows_of"] = [(e, torch.nonzero(s["adapter"] == e).flatten())
                            for e in sorted(set(s["adapter"].tolist())) if e >= 0]
        elif kind == "grad":
            s["bounds"] = s["offsets"].tolist()
        return s
    import tiled_gemm_amd as tg
    stream = torch.cuda.current_stream().cuda_stream
    if kind == "mlp":
        plan = tg.GroupMlpPlan(case["groups"], case["tokens"], case["topk"], case["width"], case["hidden"],
                               tg.GEMM_TYPE_E4M3 if case["types"] == "e4m3" else tg.GEMM_TYPE_BF16,
                               tg.LAYOUTS[case["layout"]], case["gated"], _epilogue_code(tg, case["act"]))
        if case["layout"] == "bt_preshuffled":
            s["up_image"] = _scratch(s["up"].numel() * s["up"].element_size())
            s["down_image"] = _scratch(s["down"].numel() * s["down"].element_size())
            plan.preshuffle(s["up"].data_ptr(), s["up_image"].data_ptr(), s["down"].data_ptr(),
                            s["down_image"].data_ptr(), stream)
        s["ws"] = _scratch(plan.workspace_bytes())
        s["plan"] = plan
    elif kind == "lora":
        plan = tg.Plan(case["m"], case["n"], case["k"],
                       tg.GEMM_BF16_OUT_BF16 if case["out"] == "bf16" else tg.GEMM_BF16_OUT_F32,
                       tg.LAYOUTS[case["layout"]])
        if case["layout"] == "bt_preshuffled":
            s["image"] = _scratch(tg.gemm_preshuffled_b_bytes(plan.handle))
            plan.preshuffle_b(s["b"].data_ptr(), s["image"].data_ptr(), stream)
        s["ws"] = _scratch(plan.lora_workspace_bytes(case["rank"]))
        s["plan"] = plan
    elif kind == "grad":
        s["ws"] = _scratch(tg.gemm_act_grad_workspace_bytes(case["m"], case["n"], case["groups"]))
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    kind = state["case"]["kind"]
    return (_OWN if own else _PLAIN)[kind](state["case"], state)


def _epilogue_code(tg, act):
    return tg.EPILOGUES["bias" if act == "none" else "bias_" + act]


def _own_mlp(case, s):
    s["plan"].run(s["x"].data_ptr(), s["ids"].data_ptr(), s.get("up_image", s["up"]).data_ptr(),
                  s.get("down_image", s["down"]).data_ptr(), s["out"].data_ptr(), weights=_ptr(s["weights"]),
                  up_scale=_ptr(s["up_scale"]), down_scale=_ptr(s["down_scale"]), up_bias=_ptr(s["up_bias"]),
                  down_bias=_ptr(s["down_bias"]), residual=_ptr(s["residual"]), workspace=s["ws"].data_ptr(),
                  workspace_bytes=s["ws"].numel(), stream=torch.cuda.current_stream().cuda_stream)
    return [s["out"]]


def _own_lora(case, s):
    import tiled_gemm_amd as tg
    code = tg.EPILOGUES["none"] if s["bias"] is None else _epilogue_code(tg, case["act"])
    s["plan"].run_lora(s["a"].data_ptr(), s.get("image", s["b"]).data_ptr(), s["c"].data_ptr(),
                       s["adapter"].data_ptr(), case["adapters"], case["rank"], s["down"].data_ptr(),
                       s["up"].data_ptr(), scale=s["scale"].data_ptr(), residual=_ptr(s["residual"]),
                       preact=_ptr(s["preact"]), workspace=s["ws"].data_ptr(), workspace_bytes=s["ws"].numel(),
                       stream=torch.cuda.current_stream().cuda_stream, bias=_ptr(s["bias"]), epilogue=code)
    return [s["c"]] + ([s["preact"]] if case["preact"] else [])


def _own_pack(case, s):
    import tiled_gemm_amd as tg
    tg.gemm_ckpt_pack(case["m"], case["n"], _type_code(tg, case), s["src"].data_ptr(), s["q"].data_ptr(),
                      s["scales"].data_ptr(), stream=torch.cuda.current_stream().cuda_stream)
    return [s["q"].view(torch.float8_e4m3fn), s["scales"]]


def _own_unpack(case, s):
    import tiled_gemm_amd as tg
    tg.gemm_ckpt_unpack(case["m"], case["n"], _type_code(tg, case), _epilogue_code(tg, case["act"]),
                        s["q"].data_ptr(), s["scales"].data_ptr(), s["out"].data_ptr(),
                        stream=torch.cuda.current_stream().cuda_stream)
    return [s["out"]]


def _own_grad(case, s):
    import tiled_gemm_amd as tg
    tg.gemm_act_grad_ckpt(case["m"], case["n"], _type_code(tg, case), _epilogue_code(tg, case["act"]),
                          s["dc"].data_ptr(), s["q"].data_ptr(), s["scales"].data_ptr(), s["out"].data_ptr(),
                          d_bias=s["dbias"].data_ptr(), groups=case["groups"], offsets=s["offsets"].data_ptr(),
                          workspace=s["ws"].data_ptr(), workspace_bytes=s["ws"].numel(),
                          stream=torch.cuda.current_stream().cuda_stream)
    return [s["out"], s["dbias"]]


def _type_code(tg, case):
    return tg.GEMM_TYPE_F32 if case["type"] == "f32" else tg.GEMM_TYPE_BF16


_OWN = dict(mlp=_own_mlp, lora=_own_lora, pack=_own_pack, unpack=_own_unpack, grad=_own_grad)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return torch.ones_like(z)


def _plain_mlp(case, s):
    tokens, topk, hidden = case["tokens"], case["topk"], case["hidden"]
    x = s["x"].float()
    y = torch.zeros((tokens * topk, case["width"]), dtype=F32, device="cuda")
    for e, slots in s["slots_of"]:
        z = torch.mm(x[slots // topk], s["up"][e].float().t())
        if s["up_scale"] is not None:
            z = z * s["up_scale"][e]
        if s["up_bias"] is not None:
            z = z + s["up_bias"][e]
        h = _act(z[:, :hidden], case["act"]) * z[:, hidden:] if case["gated"] else _act(z, case["act"])
        d = torch.mm(h, s["down"][e].float().t())
        if s["down_scale"] is not None:
            d = d * s["down_scale"][e]
        if s["down_bias"] is not None:
            d = d + s["down_bias"][e]
        y[slots] = d
    y = y.view(tokens, topk, -1)
    if s["weights"] is not None:
        y = y * s["weights"][:, :, None]
    y = y.sum(dim=1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(BF16)]


def _plain_lora(case, s):
    a = s["a"].float()
    z = torch.mm(a, s["b"].float().t())
    for e, rows in s["rows_of"]:
        v = torch.mm(a[rows], s["down"][e].float().t()) * s["scale"][e]
        z[rows] += torch.mm(v, s["up"][e].float().t())
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(s["c"].dtype)] + ([z.to(s["c"].dtype)] if case["preact"] else [])


def _plain_pack(case, s):
    q, scales = _mx(s["src"].float())
    return [q, scales]


def _value(case, s):
    """The checkpoint's values in 32 bits."""
    q = s["q"].view(torch.float8_e4m3fn).float()
    step = torch.exp2(s["scales"].to(F32) - 127.0)
    return q * step.repeat_interleave(32, dim=1)[:, :case["n"]]


def _plain_unpack(case, s):
    return [_act(_value(case, s), case["act"]).to(s["out"].dtype)]


def _plain_grad(case, s):
    dz = s["dc"].float() * _act_slope(_value(case, s), case["act"])
    out, dbias = torch.zeros_like(s["out"]), torch.zeros_like(s["dbias"])
    out[:case["rows"]] = dz[:case["rows"]].to(out.dtype)
    for e in range(case["groups"]):
        dbias[e] = dz[s["bounds"][e]:s["bounds"][e + 1]].sum(dim=0)
    return [out, dbias]


_PLAIN = dict(mlp=_plain_mlp, lora=_plain_lora, pack=_plain_pack, unpack=_plain_unpack, grad=_plain_grad)


# ------------------------------------------------------------------ the work

def _active(tokens, topk, groups, drop=0.0):
    """Experts that get at least one token (even popularity)."""
    return groups * (1.0 - (1.0 - topk * (1.0 - drop) / groups) ** tokens)


def work(case):
    kind = case["kind"]
    if kind == "mlp":
        tokens, topk, width, hidden = (case[f] for f in ("tokens", "topk", "width", "hidden"))
        inner = hidden * (2 if case["gated"] else 1)
        e4m3 = case["types"] == "e4m3"
        vectors = (4 if e4m3 else 0) + (4 if case["bias"] else 0)          # bytes per output column of an expert
        each = (inner + hidden) * width * (1 if e4m3 else 2) + vectors * (inner + width)
        slots = tokens * topk
        return dict(bytes=_active(tokens, topk, case["groups"], case["drop"]) * each +
                    2 * tokens * width * (3 if case["residual"] else 2) + slots * (8 if case["weighted"] else 4),
                    flops=2.0 * slots * (1.0 - case["drop"]) * width * (inner + hidden))
    if kind == "lora":
        m, n, k, rank, top = (case[f] for f in ("m", "n", "k", "rank", "adapters"))
        with_one = m * (1.0 - case["plain"])
        # different adapters among the rows (one choice per row, or per request)
        used = top * (1.0 - (1.0 - 1.0 / top) ** ((m if case["mix"] == "rows" else case["requests"]) *
                                                  (1.0 - case["plain"])))
        ob = 2 if case["out"] == "bf16" else 4
        outs = 1 + bool(case["residual"]) + bool(case["preact"])
        bias = 4 * n if case["bias"] or case["act"] != "none" else 0
        return dict(bytes=2 * m * k + 2 * n * k + m * n * ob * outs + bias + 4 * m + used * (2 * rank * (n + k) + 4),
                    flops=2.0 * m * n * k + 2.0 * with_one * rank * (n + k))
    m, n = case["m"], case["n"]
    eb = 4 if case["type"] == "f32" else 2
    kept = 1.0 + 1.0 / 32.0
    if kind == "grad":
        return dict(bytes=(2 * eb + (kept if case["act"] != "none" else 0.0)) * case["rows"] * n +
                    4 * case["groups"] * n + 4 * (case["groups"] + 1), flops=8.0 * case["rows"] * n)
    return dict(bytes=(eb + kept) * m * n, flops=4.0 * m * n)


# ------------------------------------------------------------------ in 64 bits

def _slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    return 0.5 * torch.erfc(-z / 2.0 ** 0.5) + z * torch.exp(-z.square() / 2.0) * (2.0 * math.pi) ** -0.5


def _act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0.0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: 0.5 * z * torch.erfc(-z / 2.0 ** 0.5)}[act]()


def exact(case, seed):
    s, kind = _inputs(case, seed), case["kind"]
    d = torch.float64
    if kind == "mlp":
        y = s["residual"].to(d).clone() if case["residual"] else torch.zeros(s["out"].shape, dtype=d, device="cuda")
        for e in range(case["groups"]):
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            if t.numel() == 0:
                continue
            up, down = s["up"][e].to(d), s["down"][e].to(d)
            if case["types"] == "e4m3":
                up, down = up * s["up_scale"][e].to(d)[:, None], down * s["down_scale"][e].to(d)[:, None]
            z = s["x"].to(d).index_select(0, t) @ up.t().contiguous()
            if case["bias"]:
                z = z + s["up_bias"][e].to(d)
            if case["gated"]:
                gate, lin = z.chunk(2, dim=1)
                h = _act64(gate, case["act"]) * lin
            else:
                h = _act64(z, case["act"])
            o = h @ down.t().contiguous()
            if case["bias"]:
                o = o + s["down_bias"][e].to(d)
            if case["weighted"]:
                o = o * s["weights"][t, j].to(d)[:, None]
            y.index_add_(0, t, o)
        return [y]
    if kind == "lora":
        a = s["a"].to(d)
        z = a @ s["b"].to(d).t().contiguous()
        for e in range(case["adapters"]):
            mask = (s["adapter"] == e).nonzero().flatten()
            if mask.numel():
                both = (s["up"][e].to(d) @ s["down"][e].to(d)) * float(s["scale"][e])
                z.index_add_(0, mask, a.index_select(0, mask) @ both.t().contiguous())
        if s["bias"] is not None:
            z = z + s["bias"].to(d)
        y = _act64(z, case["act"])
        if case["residual"]:
            y = y + s["residual"].to(d)
        return [y, z] if case["preact"] else [y]
    if kind == "pack":
        x = s["src"].to(d)
        ends = list(range(0, case["n"], 32))
        tops = torch.stack([x[:, c:c + 32].abs().amax(dim=1) for c in ends], dim=1)
        power = torch.ceil(torch.log2(tops / 448.0)).clamp(-127, 127)
        power = torch.where(tops > 0, power, -127.0)
        cols = torch.arange(case["n"], device="cuda") // 32
        return [x / torch.pow(2.0, power.to(d)).index_select(1, cols), (power + 127).to(torch.uint8)]
    cols = torch.arange(case["n"], device="cuda") // 32
    z = s["q"].view(torch.float8_e4m3fn).to(d) * torch.pow(2.0, s["scales"].to(d) - 127.0).index_select(1, cols)
    if kind == "unpack":
        return [_act64(z, case["act"])]
    inside = torch.arange(case["m"], device="cuda") < case["rows"]
    dz = torch.where(inside[:, None], s["dc"].to(d) * _slope64(z, case["act"]), 0.0)
    running = torch.cat([dz.new_zeros(1, case["n"]), dz.cumsum(0)])
    at = s["offsets"].long()
    return [dz, running[at[1:]] - running[at[:-1]]]
