"""Measured passes through the library's large-language-model operators.

Each case is one call that a user's program makes: a product with bias,
activation and residual in its epilogue, the gradient of that epilogue, the
tables that sort tokens by expert, the experts' ragged products (forward,
input gradient, weight gradient) and the weighted sum that brings the experts'
rows back to their tokens.  ``listed()`` names fixed cases, ``draw(rng)`` gives
further ones of the same ranges, ``prepare`` makes the inputs, ``run`` makes
one pass, ``work`` states the bytes and operations a pass cannot do without
and ``exact`` computes the same outputs in 64 bits.

``own`` selects the library's kernels; without it ``run`` computes the plain
form, elementary torch operations in 32 bits.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("none", "silu", "gelu", "relu")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # The smallest call of a decode loop: one token through a projection
        # whose output joins the residual stream; latency counts.
        dict(name="residual_one_token", kind="residual", types="bf16", m=1, n=2048, k=2048, layout="bt_preshuffled",
             bias=False, act="none", residual=True, preact=False),
        # A prompt of odd length through a quantised layer, scales per token
        # and per output channel.
        dict(name="residual_e4m3_odd_prompt", kind="residual", types="e4m3", m=333, n=4096, k=4160, layout="bt",
             bias=True, act="gelu", residual=True, preact=False),
        # A training step's forward pass: the pre-activation is kept for the
        # backward pass.
        dict(name="residual_train", kind="residual", types="bf16", m=8192, n=8192, k=2048, layout="bt",
             bias=True, act="silu", residual=True, preact=True),
        # The backward pass of that epilogue: the gradient of the
        # pre-activation and of the bias.
        dict(name="act_grad_train", kind="act_grad", m=8192, n=8192, act="silu", groups=1, rows=8192),
        # Routing tables of one decode step.
        dict(name="sort_decode", kind="sort", tokens=32, topk=8, groups=64, local=1.0),
        # Routing tables of a long prefill on one of four expert-parallel
        # ranks: three quarters of the slots belong to other ranks.
        dict(name="sort_prefill", kind="sort", tokens=32768, topk=8, groups=64, local=0.25),
        # Decode: 16 tokens, 4 experts each; bound by the active experts'
        # weights.
        dict(name="experts_decode", kind="experts", types="bf16", tokens=16, topk=4, groups=64, n=2048, k=1024,
             layout="bt_preshuffled", bias=True, act="silu", gather=True, skew=0.0, spare=0),
        # Prefill in fp8: uneven experts, some short or empty, a capacity
        # larger than the routed rows.
        dict(name="experts_e4m3_prefill", kind="experts", types="e4m3", tokens=4001, topk=4, groups=24, n=4096, k=2112,
             layout="bt", bias=False, act="none", gather=True, skew=1.0, spare=77),
        # Training: the gradient of the experts' inputs (weights read K x N).
        dict(name="experts_input_grad", kind="experts", types="bf16", tokens=8192, topk=2, groups=16, n=2048, k=4096,
             layout="bn", bias=False, act="none", gather=False, skew=0.5, spare=0),
        # Training: the gradient of the experts' weights (ragged inner size).
        dict(name="experts_weight_grad", kind="weight_grad", out="bf16", tokens=8192, topk=2, groups=16, m=4096,
             n=2048, skew=0.5),
        # Decode: the experts' rows back to their tokens, onto the residual.
        dict(name="combine_decode", kind="combine", tokens=16, topk=4, n=2048, residual=True, weights=True, drop=0.0),
        # Training: the gradient of that sum, to the rows and to the weights.
        dict(name="combine_grad_train", kind="combine_grad", tokens=8192, topk=4, n=4096, drop=0.05),
    ]


_FLOP_CAP = 2.0 * 8192 * 8192 * 2048


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    return max(lo, min(hi, _log(rng, lo, hi) // step * step))


def draw(rng):
    kind = rng.choice(["residual", "residual", "act_grad", "sort", "experts", "experts", "experts", "weight_grad",
                       "combine", "combine_grad"])
    if kind == "residual":
        n, k = _mult(rng, 256, 8192, 16), _mult(rng, 256, 8192, 64)
        types = rng.choice(["bf16", "bf16", "bf16_f32", "e4m3"])
        m = _log(rng, 1, min(4096 if types == "bf16_f32" else 8192, _FLOP_CAP / (2.0 * n * k)))
        return dict(kind=kind, types=types, m=m, n=n, k=k,
                    layout=rng.choice(["bt", "bt_preshuffled"]), bias=rng.random() < 0.6, act=rng.choice(ACTS),
                    residual=rng.random() < 0.8, preact=rng.random() < 0.4)
    if kind == "act_grad":
        n = _mult(rng, 256, 8192, 16)
        rows = _log(rng, 1, 8192)
        return dict(kind=kind, m=rows + rng.choice([0, rng.randint(1, 40)]), n=n, act=rng.choice(ACTS),
                    groups=rng.choice([1, _log(rng, 2, 64)]), rows=rows)
    if kind == "sort":
        return dict(kind=kind, tokens=_log(rng, 1, 32768), topk=rng.randint(1, 8), groups=_log(rng, 8, 256),
                    local=rng.choice([1.0, rng.uniform(0.1, 1.0)]))
    groups = _log(rng, 2, 64)
    topk = rng.randint(1, min(8, groups))
    if kind == "experts":
        n, k = _mult(rng, 256, 4096, 16), _mult(rng, 256, 4096, 64)
        groups = max(topk, min(groups, int(2.0e8 / (n * k))))
        tokens = _log(rng, 1, min(8192, _FLOP_CAP / (2.0 * n * k * topk)))
        layout = rng.choice(["bt", "bt_preshuffled", "bn"])
        types = "bf16" if layout == "bn" else rng.choice(["bf16", "bf16", "bf16_f32", "e4m3"])
        bias = rng.random() < 0.5
        return dict(kind=kind, types=types, tokens=tokens, topk=topk, groups=groups, n=n, k=k, layout=layout,
                    bias=bias, act=rng.choice(ACTS), gather=rng.random() < 0.6, skew=rng.choice([0.0, 0.5, 1.0, 2.0]),
                    spare=rng.choice([0, rng.randint(1, 100)]))
    if kind == "weight_grad":
        m, n = _mult(rng, 256, 4096, 16), _mult(rng, 256, 2048, 16)
        tokens = _log(rng, 16, min(8192, _FLOP_CAP / (2.0 * m * n * topk)))
        return dict(kind=kind, out=rng.choice(["bf16", "f32"]), tokens=tokens, topk=topk, groups=min(groups, 16),
                    m=m, n=n, skew=rng.choice([0.0, 0.5, 1.0, 2.0]))
    n = _mult(rng, 256, 8192, 16)
    tokens = _log(rng, 1, min(16384, 8192 * 4 * 4096 / (n * topk)))
    out = dict(kind=kind, tokens=tokens, topk=topk, n=n, drop=rng.choice([0.0, 0.05, 0.5]))
    if kind == "combine":
        out.update(residual=rng.random() < 0.5, weights=rng.random() < 0.8)
    return out


# ------------------------------------------------------------------ the inputs

def _randn(g, *shape, std=1.0, dtype=BF16):
    x = torch.empty(shape, dtype=F32, device="cuda")
    return x.normal_(0.0, std, generator=g).to(dtype)


def _quantise(x, dim):
    """fp32 -> (e4m3 values, fp32 scales) with one scale per slice of `dim`."""
    s = x.abs().amax(dim=dim, keepdim=True).clamp_(min=1e-12) / 448.0
    return (x / s).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), s.squeeze(dim).contiguous()


def _route(g, tokens, topk, groups, skew):
    """Distinct experts per token, some experts more popular than others."""
    pull = torch.empty(groups, device="cuda").normal_(0.0, 1.0, generator=g) * skew
    u = torch.empty((tokens, groups), device="cuda").uniform_(1e-6, 1.0 - 1e-6, generator=g)
    return (pull - torch.log(-torch.log(u))).topk(topk, dim=1).indices


def _tables(ids, groups):
    """offsets, the token of each sorted row, the sorted row of each slot."""
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = (flat[:, None] == torch.arange(groups, device="cuda")).sum(dim=0)
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.arange(order.numel(), device="cuda")
    return offsets.to(torch.int32), (order // ids.shape[1]).to(torch.int32), slot_row.to(torch.int32)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, s = case["kind"], {}
    if kind == "residual":
        m, n, k = case["m"], case["n"], case["k"]
        if case["types"] == "e4m3":
            s["a"], s["sa"] = _quantise(_randn(g, m, k, dtype=F32), 1)
            s["b"], s["sb"] = _quantise(_randn(g, n, k, std=k ** -0.5, dtype=F32), 1)
        else:
            s["a"], s["b"] = _randn(g, m, k), _randn(g, n, k, std=k ** -0.5)
            s["sa"] = s["sb"] = None
        ctype = F32 if case["types"] == "bf16_f32" else BF16
        s["bias"] = _randn(g, n, std=0.5, dtype=F32) if case["bias"] or case["act"] != "none" else None
        s["residual"] = _randn(g, m, n, dtype=ctype) if case["residual"] else None
        s["c"] = torch.zeros((m, n), dtype=ctype, device="cuda")
        s["preact"] = torch.zeros((m, n), dtype=ctype, device="cuda") if case["preact"] else None
    elif kind == "act_grad":
        m, n, groups, rows = case["m"], case["n"], case["groups"], case["rows"]
        s["dc"], s["z"] = _randn(g, m, n), _randn(g, m, n, std=1.5)
        cuts = torch.randint(0, rows + 1, (groups - 1,), generator=g, device="cuda").sort().values
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows)]).to(torch.int32)
        s["dz"] = torch.zeros((m, n), dtype=BF16, device="cuda")
        s["dbias"] = torch.zeros((groups, n), dtype=F32, device="cuda")
    elif kind == "sort":
        slots = case["tokens"] * case["topk"]
        ids = torch.randint(0, max(case["groups"], int(case["groups"] / case["local"])),
                            (case["tokens"], case["topk"]), generator=g, device="cuda")
        s["ids"] = torch.where(ids < case["groups"], ids, -1).to(torch.int32)
        s["offsets"] = torch.zeros(case["groups"] + 1, dtype=torch.int32, device="cuda")
        s["row_token"] = torch.full((slots,), -1, dtype=torch.int32, device="cuda")
        s["slot_row"] = torch.zeros((case["tokens"], case["topk"]), dtype=torch.int32, device="cuda")
    elif kind == "experts":
        groups, n, k, tokens = case["groups"], case["n"], case["k"], case["tokens"]
        ids = _route(g, tokens, case["topk"], groups, case["skew"])
        s["offsets"], row_token, _ = _tables(ids, groups)
        rows = ids.numel() + case["spare"]
        s["row_index"] = None
        if case["gather"]:
            s["row_index"] = torch.cat([row_token, row_token.new_full((case["spare"],), -1)])
        a_rows = tokens if case["gather"] else rows
        shape = (groups, k, n) if case["layout"] == "bn" else (groups, n, k)
        if case["types"] == "e4m3":
            s["a"], s["sa"] = _quantise(_randn(g, a_rows, k, dtype=F32), 1)
            s["b"], s["sb"] = _quantise(_randn(g, *shape, std=k ** -0.5, dtype=F32), 2)
        else:
            s["a"], s["b"] = _randn(g, a_rows, k), _randn(g, *shape, std=k ** -0.5)
            s["sa"] = s["sb"] = None
        ctype = F32 if case["types"] == "bf16_f32" else BF16
        s["bias"] = _randn(g, groups, n, std=0.5, dtype=F32) if case["bias"] or case["act"] != "none" else None
        s["c"] = torch.zeros((rows, n), dtype=ctype, device="cuda")
    elif kind == "weight_grad":
        ids = _route(g, case["tokens"], case["topk"], case["groups"], case["skew"])
        s["offsets"], _, _ = _tables(ids, case["groups"])
        rows = ids.numel()
        s["a"], s["b"] = _randn(g, rows, case["m"]), _randn(g, rows, case["n"])
        s["c"] = torch.zeros((case["groups"], case["m"], case["n"]), dtype=BF16 if case["out"] == "bf16" else F32,
                             device="cuda")
    else:
        tokens, topk, n = case["tokens"], case["topk"], case["n"]
        ids = _route(g, tokens, topk, max(8, topk), 0.5)
        ids[torch.empty(ids.shape, device="cuda").uniform_(0.0, 1.0, generator=g) < case["drop"]] = 1 << 20
        keep = ids < (1 << 20)
        _, _, slot_row = _tables(ids, max(8, topk))
        s["slot_row"] = torch.where(keep, slot_row.view(tokens, topk), -1)
        s["rows"] = tokens * topk
        s["src"] = _randn(g, tokens * topk, n)
        s["weights"] = torch.softmax(_randn(g, tokens, topk, dtype=F32), dim=1)
        if kind == "combine":
            s["weights"] = s["weights"] if case["weights"] else None
            s["residual"] = _randn(g, tokens, n) if case["residual"] else None
            s["out"] = torch.zeros((tokens, n), dtype=BF16, device="cuda")
        else:
            s["dout"] = _randn(g, tokens, n)
            s["dsrc"] = torch.zeros((tokens * topk, n), dtype=BF16, device="cuda")
            s["dweights"] = torch.zeros((tokens, topk), dtype=F32, device="cuda")
    return s


def _ptr(t):
    return None if t is None else t.data_ptr()


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    kind = case["kind"]
    if not own:
        if "offsets" in s and kind != "sort":
            s["bounds"] = s["offsets"].tolist()
        return s
    import tiled_gemm_amd as tg
    stream = torch.cuda.current_stream().cuda_stream
    if kind == "residual":
        code = {"bf16": tg.GEMM_BF16_OUT_BF16, "bf16_f32": tg.GEMM_BF16_OUT_F32, "e4m3": tg.GEMM_E4M3_OUT_BF16}
        plan = tg.Plan(case["m"], case["n"], case["k"], code[case["types"]], tg.LAYOUTS[case["layout"]])
        if case["layout"] == "bt_preshuffled":
            image = torch.empty(tg.gemm_preshuffled_b_bytes(plan.handle), dtype=torch.uint8, device="cuda")
            plan.preshuffle_b(s["b"].data_ptr(), image.data_ptr(), stream)
            s["weights_image"] = image
        s["ws"] = torch.empty(max(16, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
        s["plan"] = plan
    elif kind == "act_grad":
        need = tg.gemm_act_grad_workspace_bytes(case["m"], case["n"], case["groups"])
        s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    elif kind == "sort":
        need = tg.gemm_group_sort_workspace_bytes(s["ids"].numel(), case["groups"])
        s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    elif kind == "experts":
        code = {"bf16": tg.GEMM_BF16_OUT_BF16, "bf16_f32": tg.GEMM_BF16_OUT_F32, "e4m3": tg.GEMM_E4M3_OUT_BF16}
        plan = tg.GroupPlan(case["groups"], s["c"].shape[0], case["n"], case["k"], code[case["types"]],
                            tg.LAYOUTS[case["layout"]])
        if case["layout"] == "bt_preshuffled":
            image = torch.empty(plan.preshuffled_b_bytes(), dtype=torch.uint8, device="cuda")
            plan.preshuffle_b(s["b"].data_ptr(), image.data_ptr(), stream)
            s["weights_image"] = image
        s["plan"] = plan
    elif kind == "weight_grad":
        code = tg.GEMM_BF16_OUT_BF16 if case["out"] == "bf16" else tg.GEMM_BF16_OUT_F32
        s["plan"] = tg.GroupPlan(case["groups"], case["m"], case["n"], s["a"].shape[0], code, tg.LAYOUTS["at_bn"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    kind = state["case"]["kind"]
    return (_OWN if own else _PLAIN)[kind](state["case"], state)


def _epilogue(tg, case, s):
    name = "none" if s["bias"] is None else _act_name(case)
    return dict(scale_a=_ptr(s["sa"]), scale_a_per_row=s["sa"] is not None, scale_b=_ptr(s["sb"]),
                scale_b_per_col=s["sb"] is not None, bias=_ptr(s["bias"]), epilogue=tg.EPILOGUES[name])


def _own_residual(case, s):
    import tiled_gemm_amd as tg
    b = s.get("weights_image", s["b"])
    s["plan"].run_res(s["a"].data_ptr(), b.data_ptr(), s["c"].data_ptr(), residual=_ptr(s["residual"]),
                      preact=_ptr(s["preact"]), workspace=s["ws"].data_ptr(), workspace_bytes=s["ws"].numel(),
                      stream=torch.cuda.current_stream().cuda_stream, **_epilogue(tg, case, s))
    return [s["c"]] + ([s["preact"]] if case["preact"] else [])


def _own_act_grad(case, s):
    import tiled_gemm_amd as tg
    tg.gemm_act_grad(case["m"], case["n"], tg.GEMM_TYPE_BF16, tg.EPILOGUES[_act_name(case)], s["dc"].data_ptr(),
                     s["z"].data_ptr(), s["dz"].data_ptr(), d_bias=s["dbias"].data_ptr(), groups=case["groups"],
                     offsets=s["offsets"].data_ptr(), workspace=s["ws"].data_ptr(), workspace_bytes=s["ws"].numel(),
                     stream=torch.cuda.current_stream().cuda_stream)
    return [s["dz"], s["dbias"]]


def _act_name(case):
    return "bias" if case["act"] == "none" else "bias_" + case["act"]


def _own_sort(case, s):
    import tiled_gemm_amd as tg
    tg.gemm_group_sort(s["ids"].data_ptr(), s["ids"].numel(), case["topk"], case["groups"], s["offsets"].data_ptr(),
                       s["row_token"].data_ptr(), s["slot_row"].data_ptr(), workspace=s["ws"].data_ptr(),
                       workspace_bytes=s["ws"].numel(), stream=torch.cuda.current_stream().cuda_stream)
    return [s["offsets"], s["row_token"], s["slot_row"]]


def _own_experts(case, s):
    import tiled_gemm_amd as tg
    b = s.get("weights_image", s["b"])
    s["plan"].run(s["a"].data_ptr(), b.data_ptr(), s["c"].data_ptr(), s["offsets"].data_ptr(),
                  row_index=_ptr(s["row_index"]), a_rows=s["a"].shape[0],
                  stream=torch.cuda.current_stream().cuda_stream, **_epilogue(tg, case, s))
    return [s["c"]]


def _own_weight_grad(case, s):
    s["plan"].run(s["a"].data_ptr(), s["b"].data_ptr(), s["c"].data_ptr(), s["offsets"].data_ptr(),
                  stream=torch.cuda.current_stream().cuda_stream)
    return [s["c"]]


def _own_combine(case, s):
    import tiled_gemm_amd as tg
    tg.gemm_group_combine(case["tokens"], case["topk"], case["n"], tg.GEMM_TYPE_BF16, s["src"].data_ptr(), s["rows"],
                          s["slot_row"].data_ptr(), s["out"].data_ptr(), weights=_ptr(s["weights"]),
                          residual=_ptr(s["residual"]), stream=torch.cuda.current_stream().cuda_stream)
    return [s["out"]]


def _own_combine_grad(case, s):
    import tiled_gemm_amd as tg
    tg.gemm_group_combine_grad(case["tokens"], case["topk"], case["n"], tg.GEMM_TYPE_BF16, s["dout"].data_ptr(),
                               s["src"].data_ptr(), s["rows"], s["slot_row"].data_ptr(), s["weights"].data_ptr(),
                               s["dsrc"].data_ptr(), s["dweights"].data_ptr(),
                               stream=torch.cuda.current_stream().cuda_stream)
    return [s["dsrc"], s["dweights"]]


_OWN = dict(residual=_own_residual, act_grad=_own_act_grad, sort=_own_sort, experts=_own_experts,
            weight_grad=_own_weight_grad, combine=_own_combine, combine_grad=_own_combine_grad)


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


def _plain_residual(case, s):
    z = torch.mm(s["a"].float(), s["b"].float().t())
    if s["sa"] is not None:
        z = z * s["sa"][:, None] * s["sb"][None, :]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(s["c"].dtype)] + ([z.to(s["c"].dtype)] if case["preact"] else [])


def _plain_act_grad(case, s):
    dz = s["dc"].float() * _act_slope(s["z"].float(), case["act"])
    out, dbias = torch.zeros_like(s["dz"]), torch.zeros_like(s["dbias"])
    out[:case["rows"]] = dz[:case["rows"]].to(BF16)
    for e in range(case["groups"]):
        dbias[e] = dz[s["bounds"][e]:s["bounds"][e + 1]].sum(dim=0)
    return [out, dbias]


def _plain_sort(case, s):
    ids, groups = s["ids"].reshape(-1), case["groups"]
    key = torch.where(ids >= 0, ids, groups)
    order = torch.argsort(key, stable=True)
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = (key[:, None] == torch.arange(groups, device="cuda")).sum(dim=0).cumsum(0)
    place = torch.arange(ids.numel(), device="cuda")
    routed = place < offsets[groups]
    row_token = torch.where(routed, order // case["topk"], -1)
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.where(routed, place, -1)
    return [offsets.to(torch.int32), row_token.to(torch.int32), slot_row.to(torch.int32).view(s["ids"].shape)]


def _plain_experts(case, s):
    c = torch.zeros_like(s["c"])
    for e in range(case["groups"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if lo == hi:
            continue
        rows = s["row_index"][lo:hi].long() if case["gather"] else slice(lo, hi)
        b = s["b"][e].float()
        z = torch.mm(s["a"][rows].float(), b if case["layout"] == "bn" else b.t())
        if s["sa"] is not None:
            z = z * s["sa"][rows][:, None] * s["sb"][e]
        if s["bias"] is not None:
            z = z + s["bias"][e]
        c[lo:hi] = _act(z, case["act"]).to(c.dtype)
    return [c]


def _plain_weight_grad(case, s):
    c = torch.zeros_like(s["c"])
    for e in range(case["groups"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        c[e] = torch.mm(s["a"][lo:hi].float().t(), s["b"][lo:hi].float()).to(c.dtype)
    return [c]


def _plain_combine(case, s):
    kept = s["slot_row"] >= 0
    rows = s["src"][s["slot_row"].clamp(min=0).long()].float()
    w = kept.float() if s["weights"] is None else s["weights"] * kept
    y = (rows * w[:, :, None]).sum(dim=1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(BF16)]


def _plain_combine_grad(case, s):
    kept = s["slot_row"] >= 0
    at = s["slot_row"].clamp(min=0).long()
    dout = s["dout"].float()
    dweights = (s["src"][at].float() * dout[:, None, :]).sum(dim=2) * kept
    dsrc = torch.zeros_like(s["dsrc"])
    dsrc[at[kept]] = (dout[:, None, :] * s["weights"][:, :, None])[kept].to(BF16)
    return [dsrc, dweights]


_PLAIN = dict(residual=_plain_residual, act_grad=_plain_act_grad, sort=_plain_sort, experts=_plain_experts,
              weight_grad=_plain_weight_grad, combine=_plain_combine, combine_grad=_plain_combine_grad)


# ------------------------------------------------------------------ the work

def _active(case):
    """Experts that get at least one token (even popularity)."""
    return case["groups"] * (1.0 - (1.0 - case["topk"] / case["groups"]) ** case["tokens"])


def work(case):
    kind = case["kind"]
    if kind in ("residual", "experts"):
        n, k = case["n"], case["k"]
        eb, ob = (1 if case["types"] == "e4m3" else 2), (4 if case["types"] == "bf16_f32" else 2)
        scales = 4 if case["types"] == "e4m3" else 0
        bias = 4 * n if case["bias"] or case["act"] != "none" else 0
        if kind == "residual":
            m = case["m"]
            outs = 1 + bool(case["residual"]) + bool(case["preact"])
            return dict(bytes=m * k * eb + n * k * eb + m * n * ob * outs + bias + scales * (m + n),
                        flops=2.0 * m * n * k)
        rows = case["tokens"] * case["topk"]
        a_rows = case["tokens"] if case["gather"] else rows
        return dict(bytes=a_rows * k * eb + _active(case) * (n * k * eb + bias + scales * n) + rows * n * ob +
                    scales * a_rows + (4 * rows if case["gather"] else 0) + 4 * (case["groups"] + 1),
                    flops=2.0 * rows * n * k)
    if kind == "act_grad":
        return dict(bytes=6 * case["rows"] * case["n"] + 4 * case["groups"] * case["n"],
                    flops=8.0 * case["rows"] * case["n"])
    if kind == "sort":
        slots = case["tokens"] * case["topk"]
        return dict(bytes=4 * (slots + slots + slots * case["local"] + case["groups"] + 1), flops=0.0)
    if kind == "weight_grad":
        rows = case["tokens"] * case["topk"]
        return dict(bytes=2 * rows * (case["m"] + case["n"]) +
                    case["groups"] * case["m"] * case["n"] * (2 if case["out"] == "bf16" else 4),
                    flops=2.0 * rows * case["m"] * case["n"])
    tokens, topk, n = case["tokens"], case["topk"], case["n"]
    live = tokens * topk * (1.0 - case["drop"])
    if kind == "combine":
        return dict(bytes=2 * live * n + 2 * tokens * n * (2 if case["residual"] else 1) +
                    4 * tokens * topk * (2 if case["weights"] else 1), flops=2.0 * live * n)
    return dict(bytes=4 * live * n + 2 * tokens * n + 12 * tokens * topk, flops=3.0 * live * n)


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
    if kind == "residual":
        acc = s["a"].to(d) @ s["b"].to(d).t().contiguous()
        if s["sa"] is not None:
            acc *= torch.outer(s["sa"].to(d), s["sb"].to(d))
        z = acc if s["bias"] is None else acc + s["bias"].to(d)
        y = _act64(z, case["act"])
        if case["residual"]:
            y = y + s["residual"].to(d)
        return [y, z] if case["preact"] else [y]
    if kind == "act_grad":
        inside = torch.arange(case["m"], device="cuda") < case["rows"]
        dz = torch.where(inside[:, None], s["dc"].to(d) * _slope64(s["z"].to(d), case["act"]), 0.0)
        running = torch.cat([dz.new_zeros(1, case["n"]), dz.cumsum(0)])
        at = s["offsets"].long()
        return [dz, running[at[1:]] - running[at[:-1]]]
    if kind == "sort":
        ids, groups = s["ids"].reshape(-1).tolist(), case["groups"]
        rows = [[] for _ in range(groups)]
        for slot, e in enumerate(ids):
            if 0 <= e < groups:
                rows[e].append(slot)
        offsets, row_token, slot_row = [0], [-1] * len(ids), [-1] * len(ids)
        for e in range(groups):
            for i, slot in enumerate(rows[e]):
                row_token[offsets[e] + i] = slot // case["topk"]
                slot_row[slot] = offsets[e] + i
            offsets.append(offsets[e] + len(rows[e]))
        as_ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        return [as_ints(offsets), as_ints(row_token), as_ints(slot_row).view(case["tokens"], case["topk"])]
    if kind == "experts":
        c = torch.zeros(s["c"].shape, dtype=d, device="cuda")
        cut = s["offsets"].tolist()
        for e, (lo, hi) in enumerate(zip(cut[:-1], cut[1:])):
            a = s["a"].to(d) if not case["gather"] else None
            a = a[lo:hi] if a is not None else s["a"].to(d).index_select(0, s["row_index"][lo:hi])
            z = a @ (s["b"][e].to(d) if case["layout"] == "bn" else s["b"][e].to(d).t().contiguous())
            if s["sa"] is not None:
                sa = s["sa"].to(d)
                sa = sa.index_select(0, s["row_index"][lo:hi]) if case["gather"] else sa[lo:hi]
                z = z * torch.outer(sa, s["sb"][e].to(d))
            if s["bias"] is not None:
                z = z + s["bias"][e].to(d)
            c[lo:hi] = _act64(z, case["act"])
        return [c]
    if kind == "weight_grad":
        cut = s["offsets"].tolist()
        return [torch.stack([s["a"][lo:hi].to(d).t().contiguous() @ s["b"][lo:hi].to(d)
                             for lo, hi in zip(cut[:-1], cut[1:])])]
    live = (s["slot_row"] >= 0).to(d)
    if kind == "combine":
        y = torch.zeros((case["tokens"], case["n"]), dtype=d, device="cuda")
        for j in range(case["topk"]):
            w = live[:, j] if s["weights"] is None else live[:, j] * s["weights"][:, j].to(d)
            y += w[:, None] * s["src"].to(d).index_select(0, s["slot_row"][:, j].clamp(min=0))
        return [y + s["residual"].to(d) if case["residual"] else y]
    dsrc = torch.zeros(s["dsrc"].shape, dtype=d, device="cuda")
    dweights = torch.zeros(s["dweights"].shape, dtype=d, device="cuda")
    for j in range(case["topk"]):
        t = torch.nonzero(live[:, j]).flatten()
        at = s["slot_row"][:, j].index_select(0, t).long()
        up = s["dout"].to(d).index_select(0, t)
        dsrc[at] = up * s["weights"][:, j].to(d).index_select(0, t)[:, None]
        dweights[t, j] = (up * s["src"].to(d).index_select(0, at)).sum(dim=1)
    return [dsrc, dweights]
