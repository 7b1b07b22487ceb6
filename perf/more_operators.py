"""Cases and plain forms of the router, the grouped products and 4-bit operands that run a layer's experts.

Operators (op of a case):
  route     selection, weights and the expert-sorted worklist from router logits (ops.route)
  group     bf16 or f32 products grouped by expert over a worklist, its rows gathered, SwiGLU (ops.grouped_matmul)
  quant     quantisation to e2m1 with a scale for each 16 (nvfp4) or 32 (mxfp4) columns and the values that it stands
            for (ops.fp4_quantize, ops.fp4_dequantize)
  fp4       product of such operands, dense or grouped by expert (ops.fp4_matmul)
  combine   the weighted sum of each position's edges, shared experts and residual added (ops.combine)
With `own` false every operator runs in its plain form: elementary torch operations in 32 bits, and in 64 where a
selection's border is decided.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DTYPES = {"bf16": BF16, "f32": F32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}  # columns that share a scale
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # magnitudes of the codes 0 .. 7; bit 3 is the sign


# ------------------------------------------------------------------------------------------ cases
def listed():
    route = dict(op="route", E=256, k=8, router="softmax", groups=1, topk_group=1, raw=False, dtype="f32", live=1.0, eligible=1.0)
    combine = dict(op="combine", k=8, dtype="bf16", shared=False, residual="none", out="bf16", live=1.0)
    group = dict(op="group", dtype="bf16", out="bf16", gather=False, swiglu=False, skew=0.6)
    fp4 = dict(op="fp4", E=1, skew=0.0, out="bf16", swiglu=False)
    return [
        # one token of one sequence: all latency
        dict(route, name="route_token", T=1),
        # a long prompt's positions, a sixteenth of them padding, with the group-limited router
        dict(route, name="route_prompt", T=16384, router="sigmoid_group", groups=8, topk_group=4, live=0.9375),
        # one diffusion block of 32 positions, shared expert and residual stream added
        dict(combine, name="combine_block", T=32, H=2048, shared=True, residual="f32", out="f32"),
        # a long prompt's edges
        dict(combine, name="combine_prompt", T=8192, H=4096),
        # gate and up products of one diffusion block's 256 edges over 256 experts, gathered, SwiGLU
        dict(group, name="group_block", m=256, src=32, E=256, N=1024, K=2048, gather=True, swiglu=True),
        # the same of a long prompt over 64 wider experts
        dict(group, name="group_prompt", m=65536, src=8192, E=64, N=2048, K=2048, gather=True, swiglu=True),
        # a down product with an odd number of edges, very uneven, kept in 32 bits for the combine
        dict(group, name="group_down_5003", m=5003, src=5003, E=48, N=2000, K=1024, out="f32", skew=1.1),
        # the worklist's rows of a full batch (8 experts a position), gathered
        dict(op="quant", name="quant_worklist", way="gather", form="nvfp4", n=8192, src=1024, K=2048, dtype="bf16", tscale=0.125),
        # the activations between an expert's two products, an odd number of rows
        dict(op="quant", name="quant_swiglu_333", way="swiglu", form="mxfp4", n=333, src=333, K=512, dtype="bf16", tscale=1.0),
        # a projection of one token
        dict(fp4, name="fp4_token", form="nvfp4", m=1, N=4096, K=2048),
        # a projection of a long prompt
        dict(fp4, name="fp4_prompt", form="nvfp4", m=8192, N=4096, K=4096),
        # gate and up products of 256 experts over a full batch's worklist, ragged, some empty, SwiGLU
        dict(fp4, name="fp4_experts", form="mxfp4", m=8192, N=1024, K=2048, E=256, skew=1.1, swiglu=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "group", "group", "quant", "fp4", "fp4", "combine"])
    if op == "route":
        router = rng.choice(["softmax", "softmax", "sigmoid_group"])
        groups = rng.choice([1, 2, 4, 8]) if router == "sigmoid_group" else 1
        E = max(1, _log(rng, 2, 512) // groups) * groups
        T = _log(rng, 1, 16384 if E <= 256 else 8192)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(16, E)), router=router, groups=groups,
                    topk_group=rng.randint(1, groups), raw=rng.random() < 0.3, dtype=rng.choice(["f32", "f32", "bf16"]),
                    live=rng.choice([1.0, 1.0, 0.7]), eligible=rng.choice([1.0, 1.0, 0.5]))
    if op == "combine":
        H = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            H = (H + 7) // 8 * 8
        k = rng.randint(1, 12)
        return dict(op=op, T=_log(rng, 1, max(1, min(16384, 200000000 // (H * k)))), k=k, H=H, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    shared=rng.random() < 0.4, residual=rng.choice(["none", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                    live=rng.choice([1.0, 0.8]))
    if op == "quant":
        form, K = rng.choice(["nvfp4", "mxfp4"]), 32 * _log(rng, 2, 128)
        n, way = _log(rng, 1, 8192), rng.choice(["rows", "gather", "swiglu"])
        return dict(op=op, way=way, form=form, n=n, src=n if way != "gather" else max(1, n // rng.randint(1, 8)), K=K,
                    dtype=rng.choice(["bf16", "f32"]), tscale=2.0 ** rng.randint(-6, 1) if form == "nvfp4" else 1.0)
    E = _log(rng, 2, 128) if op == "group" else rng.choice([1, 1, _log(rng, 2, 128)])
    swiglu = rng.random() < 0.4
    N = rng.choice([1, 8, 64]) * _log(rng, 16, 64)
    N += N % 2 if swiglu else 0
    if op == "fp4":
        return dict(op=op, form=rng.choice(["nvfp4", "mxfp4"]), m=_log(rng, 1, 8192), N=N, K=32 * _log(rng, 2, 128), E=E,
                    skew=rng.choice([0.0, 1.1]), out=rng.choice(["bf16", "bf16", "f32"]), swiglu=swiglu)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    m = _log(rng, 1, 32768 if dtype == "bf16" else 2048)
    gather = rng.random() < 0.5
    if dtype == "f32":
        N = min(N, 512)
    return dict(op=op, dtype=dtype, out=rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32", m=m,
                src=max(1, m // rng.randint(1, 8)) if gather else m, E=E, N=N, K=8 * _log(rng, 8, 256 if dtype == "bf16" else 64),
                gather=gather, swiglu=swiglu, skew=rng.choice([0.0, 0.6, 1.1]))


def work(case):
    c = case
    if c["op"] == "route":
        edges = c["T"] * c["k"]
        return {"bytes": c["T"] * c["E"] * (4 if c["dtype"] == "f32" else 2) + 4 * (4 * edges + c["E"] + 1),
                "flops": (2.0 if c["router"] == "softmax" else 8.0) * c["T"] * c["E"]}
    size = {"bf16": 2, "f32": 4, "none": 0}
    if c["op"] == "combine":
        n = c["T"] * c["H"]
        return {"bytes": n * (size[c["dtype"]] * (c["k"] + c["shared"]) + size[c["residual"]] + size[c["out"]]) + 8 * c["T"] * c["k"],
                "flops": 2.0 * n * c["k"]}
    if c["op"] == "quant":
        wide = 2 if c["way"] == "swiglu" else 1
        return {"bytes": size[c["dtype"]] * wide * c["src"] * c["K"] + c["n"] * (2 * c["K"] + c["K"] // BLOCK[c["form"]]) + (4 * c["n"] if c["way"] == "gather" else 0),
                "flops": 4.0 * c["n"] * c["K"]}
    used = sum(1 for s in _sizes(c, np.random.RandomState(1)) if s)
    out = c["m"] * (c["N"] // 2 if c["swiglu"] else c["N"]) * size[c["out"]]
    if c["op"] == "group":
        each = size[c["dtype"]]
        return {"bytes": each * c["K"] * (c["src"] + used * c["N"]) + out + (4 * c["m"] if c["gather"] else 0), "flops": 2.0 * c["m"] * c["N"] * c["K"]}
    return {"bytes": (c["m"] + used * c["N"]) * (c["K"] // 2 + c["K"] // BLOCK[c["form"]]) + out, "flops": 2.0 * c["m"] * c["N"] * c["K"]}


# ----------------------------------------------------------------------------------------- inputs
def _sizes(c, r):
    """Rows of each expert: every row picks one, by a Zipf mass where the routing is skewed."""
    p = (1.0 + r.permutation(c["E"])) ** -c["skew"]
    return np.bincount(r.choice(c["E"], c["m"], p=p / p.sum()), minlength=c["E"])


def _codes(v, s):
    """e2m1 codes of v / s (to nearest, ties to the even code), out of range to the largest. v, s: f32 whose quotient with a
    border needs no rounding (s has four bits at most)."""
    a, code = v.abs(), torch.zeros_like(v, dtype=torch.uint8)
    for i in range(7):  # borders between neighbouring magnitudes, taken up where the upper code is even
        border = s * ((E2M1[i] + E2M1[i + 1]) / 2)
        code += (a >= border) if i % 2 else (a > border)
    return code | (torch.signbit(v).to(torch.uint8) << 3)


def _scales(m, form):
    """The scale of blocks whose largest magnitudes are m, in the form's type."""
    if form == "nvfp4":
        s = (m.double() / 6.0).clamp(max=448.0).float()
        return s.clamp(min=2.0 ** -9).to(E4M3)
    e = torch.frexp(m).exponent - 3  # floor(log2(m)) - 2
    return torch.where(m > 0, e.clamp(-127, 127) + 127, 0).to(torch.uint8).view(E8M0)


def _fp4(x, form):
    """(codes, scales) of x [.., K] f32: a scale for each block of columns."""
    b = x.unflatten(-1, (-1, BLOCK[form]))
    s = _scales(b.abs().amax(-1), form)
    return _codes(b, s.float().unsqueeze(-1)).flatten(-2), s


def _packed(code):
    """Two codes a byte, the even column in the low half."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _laid(s, form):
    """[.., n, K / block] -> [.., ceil(K / 256), n, scales of 256 columns]: what the products read of a tile's rows is contiguous."""
    per = 256 // BLOCK[form]
    kb = -(-s.shape[-1] // per)
    p = torch.nn.functional.pad(s.view(torch.uint8), (0, kb * per - s.shape[-1]))
    return p.unflatten(-1, (kb, per)).transpose(-2, -3).contiguous().view(s.dtype)


def _routing(sel, E):
    """(positions, offsets, slots) of a selection [T, k] (-1: none): the expert-sorted worklist, positions ascending."""
    T, k = sel.shape
    flat = torch.where(sel < 0, E, sel).reshape(-1)
    key, order = torch.sort(flat, stable=True)
    place = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=sel.device))
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=sel.device))
    return torch.where(key < E, order // k, -1).to(I32), offsets.to(I32), torch.where(flat < E, place, -1).view(T, k).to(I32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *shape, std=1.0: torch.randn(*shape, generator=g, device=DEV) * std  # noqa: E731
    chance = lambda n, p: torch.rand(n, generator=g, device=DEV) < p  # noqa: E731
    s = {"c": c}
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        p = (1.0 + np.random.RandomState(7).permutation(E)) ** -1.1  # some experts are liked more
        b = np.log(p / p.sum())
        b = torch.from_numpy((0.05 * (b - b.mean()) if c["router"] == "sigmoid_group" else b).astype(np.float32)).to(DEV)
        s |= {"logits": (rnd(T, E) if c["router"] == "sigmoid_group" else rnd(T, E) + b).to(DTYPES[c["dtype"]]),
              "bias": b if c["router"] == "sigmoid_group" else None,
              "live": None if c["live"] == 1.0 else chance(T, c["live"]).to(torch.uint8),
              "eligible": None if c["eligible"] == 1.0 else chance(E, c["eligible"]).to(torch.uint8)}
    elif c["op"] == "combine":
        T, k, H = c["T"], c["k"], c["H"]
        sel = torch.rand(T, 64, generator=g, device=DEV).argsort(1)[:, :k]
        sel = torch.where(chance(T, c["live"]).unsqueeze(1), sel, -1)
        w = torch.rand(T, k, generator=g, device=DEV) + 0.1
        s |= {"edges": rnd(T * k, H).to(DTYPES[c["dtype"]]), "slots": _routing(sel, 64)[2], "w": w / w.sum(1, keepdim=True),
              "shared": rnd(T, H).to(DTYPES[c["dtype"]]) if c["shared"] else None,
              "residual": rnd(T, H, std=2.0).to(DTYPES[c["residual"]]) if c["residual"] != "none" else None,
              "out": torch.empty(T, H, device=DEV, dtype=DTYPES[c["out"]])}
    elif c["op"] == "quant":
        x = rnd(c["src"], c["K"] * (2 if c["way"] == "swiglu" else 1)) * (1.0 + 9.0 * chance(c["K"] * (2 if c["way"] == "swiglu" else 1), 0.01))
        x[1:2] = 0  # a position that is padding
        s |= {"x": x.to(DTYPES[c["dtype"]]), "rows": torch.randint(0, c["src"], (c["n"],), generator=g, device=DEV, dtype=I32) if c["way"] == "gather" else None}
    else:
        m, N, K, E = c["m"], c["N"], c["K"], c["E"]
        sizes = _sizes(c, np.random.RandomState(seed % (1 << 31)))
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEV)
        s["most"] = int(sizes.max())
        s["out"] = torch.empty(m, N // 2 if c["swiglu"] else N, device=DEV, dtype=DTYPES[c["out"]])
        if c["op"] == "group":
            d = DTYPES[c["dtype"]]
            s |= {"x": rnd(c["src"], K).to(d), "w": (rnd(E, N, K, std=K ** -0.5)).to(d),
                  "rows": torch.randint(0, c["src"], (m,), generator=g, device=DEV, dtype=I32) if c["gather"] else None}
        else:
            a, sa = _fp4(rnd(m, K), c["form"])
            w = rnd(E, N, K, std=K ** -0.5)
            # a power of two for each matrix, so that e4m3 holds the scales of its blocks (mxfp4's hold any)
            t = torch.exp2(torch.ceil(torch.log2(w.abs().amax((1, 2)) / (6 * 448)))) if c["form"] == "nvfp4" else torch.ones(E, device=DEV)
            w /= t.view(-1, 1, 1)
            b, sb = _fp4(w, c["form"])
            s |= {"a": _packed(a), "sa": _laid(sa, c["form"]), "b": _packed(b), "sb": _laid(sb, c["form"]), "scale": t}
    return s


# -------------------------------------------------------------------------------------- plain forms
def _route_plain(s):
    c = s["c"]
    T, E, k, groups = c["T"], c["E"], c["k"], c["groups"]
    logits = s["logits"].float()
    open_ = torch.ones(T, E, device=DEV, dtype=torch.bool) if s["eligible"] is None else (s["eligible"] != 0).expand(T, E)
    if s["live"] is not None:
        open_ = open_ & (s["live"] != 0).unsqueeze(1)
    if c["router"] == "softmax":
        pick = logits.double()
    else:
        score = 1.0 / (1.0 + torch.exp(-logits.double()))  # 64 bits: borders between sums of a score and its bias
        pick = score + s["bias"].double()
        if c["topk_group"] < groups:
            shut = torch.where(open_, pick, -math.inf).view(T, groups, -1)
            two = torch.sort(shut, dim=2, descending=True).values[..., :2]
            rank = torch.where(torch.isinf(two), 0.0, two).sum(2)
            count = open_.reshape(T, groups, -1).sum(2)
            order = torch.sort(torch.where(count > 0, rank, -math.inf), dim=1, descending=True, stable=True).indices
            held = count.gather(1, order)
            use = (torch.arange(groups, device=DEV) < c["topk_group"]) | (held.cumsum(1) - held < k)
            use = torch.zeros_like(use).scatter_(1, order, use) & (count > 0)
            open_ = open_ & use.repeat_interleave(E // groups, 1)
    place = torch.sort(torch.where(open_, pick, -math.inf), dim=1, descending=True, stable=True).indices[:, :k]
    none = ~open_.gather(1, place)
    if c["router"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True)) if c["raw"] else torch.exp(logits - logits.gather(1, place[:, :1]))
        w = torch.where(none, 0.0, e.gather(1, place))
        total = e if c["raw"] else w
    else:
        w = torch.where(none, 0.0, score.float().gather(1, place))
        total = w
    if not (c["raw"] and c["router"] != "softmax"):
        w = torch.where(none, 0.0, w / total.sum(1, keepdim=True))
    sel = torch.where(none, -1, place)
    return (sel.to(I32), w) + _routing(sel, E)


def _combine_plain(s):
    slots = s["slots"].long()
    w = torch.where(slots < 0, 0.0, s["w"])
    y = (s["edges"][slots.clamp(min=0)].float() * w.unsqueeze(2)).sum(1)
    for more in (s["shared"], s["residual"]):
        if more is not None:
            y = y + more.float()
    return y.to(s["out"].dtype)


def _swiglu(x):
    gate, up = x.chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _quant_plain(s):
    c = s["c"]
    x = s["x"].float()
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    if c["way"] == "swiglu":
        x = _swiglu(x)
    code, scale = _fp4(x / c["tscale"], c["form"])
    return _values(code, scale, c["tscale"]).to(BF16), _laid(scale, c["form"])


def _values(code, scale, tscale):
    """What codes [.., K] with scales [.., K / block] stand for, in 32 bits."""
    v = torch.tensor(E2M1 + [-x for x in E2M1], device=code.device)[code.int()]
    return (v.unflatten(-1, (scale.shape[-1], -1)) * (scale.float() * tscale).unsqueeze(-1)).flatten(-2)


def _opened(q, scale, K):
    """Values of packed codes [.., n, K / 2]."""
    rows = scale.view(torch.uint8).transpose(-2, -3).flatten(-2)
    block = 16 if scale.dtype == E4M3 else 32
    return _values(torch.stack([q & 15, q >> 4], -1).flatten(-2), rows[..., :K // block].contiguous().view(scale.dtype), 1.0)


def _grouped_plain(a, b, s, scale=None):
    """Rows of a [m, K] times their expert's b[e] [N, K]: every expert's rows padded to the most."""
    c, m = s["c"], a.shape[0]
    first = s["offsets"][:-1].long()
    if c["E"] == 1:
        y = a @ b[0].T
        y = y if scale is None else y * scale
    else:
        expert = torch.bucketize(torch.arange(m, device=DEV, dtype=I32), s["offsets"][1:], right=True)
        at = (first.unsqueeze(1) + torch.arange(s["most"], device=DEV)).clamp(max=m - 1)
        y = torch.bmm(a[at], b.mT)[expert, torch.arange(m, device=DEV) - first[expert]]
        y = y if scale is None else y * scale[expert].unsqueeze(1)
    return (_swiglu(y) if c["swiglu"] else y).to(s["out"].dtype)


# --------------------------------------------------------------------------------------------- run
def run(state):
    s, c = state, state["c"]
    if not own:
        if c["op"] == "group":
            x = s["x"] if s["rows"] is None else s["x"][s["rows"].long()]
            return _grouped_plain(x.float(), s["w"].float(), s)
        if c["op"] == "fp4":
            return _grouped_plain(_opened(s["a"], s["sa"], c["K"]), _opened(s["b"], s["sb"], c["K"]), s, s["scale"])
        return {"route": _route_plain, "combine": _combine_plain, "quant": _quant_plain}[c["op"]](s)
    from sparse_moe_layer_gate_gb300 import ops
    if c["op"] == "route":
        r = ops.route(s["logits"], c["k"], router=c["router"], bias=s["bias"], n_group=c["groups"], topk_group=c["topk_group"],
                      raw_weights=c["raw"], live=s["live"], eligible=s["eligible"])
        return r.sel, r.weights, r.positions, r.offsets, r.slots
    if c["op"] == "combine":
        return ops.combine(s["edges"], s["slots"], s["w"], shared=s["shared"], residual=s["residual"], out=s["out"])
    if c["op"] == "group":
        return ops.grouped_matmul(s["x"], s["w"], s["offsets"], rows=s["rows"], swiglu=c["swiglu"], out=s["out"])
    if c["op"] == "quant":
        q, scales = ops.fp4_quantize(s["x"], form=c["form"], rows=s["rows"], swiglu=c["way"] == "swiglu", tensor_scale=c["tscale"])
        return ops.fp4_dequantize(q, scales, tensor_scale=c["tscale"], out_dtype=BF16), scales
    if c["E"] == 1:
        return ops.fp4_matmul(s["a"], s["sa"], s["b"][0], s["sb"][0], scale=s["scale"], swiglu=c["swiglu"], out=s["out"])
    return ops.fp4_matmul(s["a"], s["sa"], s["b"], s["sb"], offsets=s["offsets"], scale=s["scale"], swiglu=c["swiglu"], out=s["out"])


# ------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "route":
        return _route_exact(s, c)
    if c["op"] == "combine":
        y = torch.zeros(c["T"], c["H"], device=DEV, dtype=F64)
        for j in range(c["k"]):
            at = s["slots"][:, j].long()
            on = at >= 0
            y[on] += s["w"][on, j].double().unsqueeze(1) * s["edges"].index_select(0, at[on]).double()
        for more in ("shared", "residual"):
            if s[more] is not None:
                y += s[more].double()
        return y
    silu = lambda v: torch.nn.functional.silu(v[:, :v.shape[1] // 2]) * v[:, v.shape[1] // 2:]  # noqa: E731
    if c["op"] == "quant":
        x = s["x"].double() if s["rows"] is None else s["x"].double().index_select(0, s["rows"].long())
        x = (silu(x) if c["way"] == "swiglu" else x) / c["tscale"]
        grid = torch.tensor(E2M1, device=DEV, dtype=F64)
        v, scales = torch.empty_like(x), []
        for k in range(0, c["K"], BLOCK[c["form"]]):
            b = x[:, k:k + BLOCK[c["form"]]]
            most = b.abs().max(1, keepdim=True).values
            if c["form"] == "nvfp4":
                scale = (most / 6).clamp(2.0 ** -9, 448.0).float().to(E4M3).double()
                scales.append(scale)
            else:
                low = torch.floor(torch.log2(most)) - 2
                low = torch.where(most > 0, low, -127.0).clamp(min=-127.0)
                scale = torch.exp2(low)
                scales.append(scale)
            far = (b.abs() / scale).unsqueeze(-1) - grid
            near = far.abs()
            best = near.min(-1, keepdim=True).values
            # among equally near ones the even code
            code = torch.where(near == best, torch.arange(8, device=DEV) % 2, 2).argmin(-1)
            v[:, k:k + BLOCK[c["form"]]] = torch.copysign(grid[code], b) * scale * c["tscale"]
        per = 256 // BLOCK[c["form"]]
        flat = torch.cat(scales, 1)
        pad = -flat.shape[1] % per
        flat = torch.cat([flat, torch.full((c["n"], pad), 0.0 if c["form"] == "nvfp4" else 2.0 ** -127, device=DEV, dtype=F64)], 1)
        return v, torch.stack(flat.split(per, 1))
    off = s["offsets"].tolist()
    y = torch.zeros(c["m"], c["N"], device=DEV, dtype=F64)
    x = None
    if c["op"] == "group":
        x = s["x"].double() if s["rows"] is None else s["x"].double().index_select(0, s["rows"].long())
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if hi <= lo:
            continue
        if c["op"] == "group":
            y[lo:hi] = x[lo:hi] @ s["w"][e].double().T
        else:
            y[lo:hi] = _fp4_exact(s["a"][lo:hi], s["sa"][:, lo:hi], c["K"]) @ _fp4_exact(s["b"][e], s["sb"][e], c["K"]).T
            y[lo:hi] *= s["scale"][e].double()
    return silu(y) if c["swiglu"] else y


def _fp4_exact(q, scales, K):
    """The values of packed rows in 64 bits, column by column of the codes' bits."""
    n = q.shape[0]
    v = torch.empty(n, K, device=DEV, dtype=F64)
    for half, code in ((0, q & 15), (1, q >> 4)):
        code = code.int()
        exponent, fraction = (code >> 1) & 3, (code & 1).double()
        size = torch.where(exponent == 0, 0.5 * fraction, (1 + 0.5 * fraction) * torch.exp2((exponent - 1).double()))
        v[:, half::2] = torch.where(code >= 8, -size, size)
    raw = scales.contiguous()
    wide = raw.float().double() if scales.dtype == E4M3 else torch.exp2(raw.view(torch.uint8).double() - 127)
    block = 16 if scales.dtype == E4M3 else 32
    column = torch.arange(K, device=DEV)
    return v * wide[column // 256, :, (column % 256) // block].T


def _route_exact(s, c):
    T, E, k = c["T"], c["E"], c["k"]
    g = s["logits"].double().cpu().numpy()
    can = np.ones(E, bool) if s["eligible"] is None else s["eligible"].cpu().numpy() != 0
    live = np.ones(T, bool) if s["live"] is None else s["live"].cpu().numpy() != 0
    sigmoid = c["router"] != "softmax"
    score = 1.0 / (1.0 + np.exp(-g)) if sigmoid else g
    pick = np.where(can, score + s["bias"].double().cpu().numpy() if sigmoid else g, -np.inf)
    if sigmoid and c["topk_group"] < c["groups"]:
        size = E // c["groups"]
        counts = can.reshape(c["groups"], size).sum(1)
        for t in range(T):
            best = [(-sum(sorted((v for v in pick[t, i * size:(i + 1) * size] if v > -np.inf), reverse=True)[:2]), i) for i in range(c["groups"]) if counts[i]]
            held = 0
            for rank, (_, i) in enumerate(sorted(best)):
                if rank >= c["topk_group"] and held >= k:
                    pick[t, i * size:(i + 1) * size] = -np.inf
                held += counts[i]
    sel = np.argsort(-pick, axis=1, kind="stable")[:, :k]
    sel = np.where(np.isinf(np.take_along_axis(pick, sel, 1)) | ~live[:, None], -1, sel)
    on = sel >= 0
    w = np.where(on, np.take_along_axis(score, np.maximum(sel, 0), 1), 0.0 if sigmoid else -np.inf)
    if not sigmoid:
        top = (g if c["raw"] else np.where(on[:, :1], w, 0.0)).max(1, keepdims=True)
        w = np.exp(w - top)
        total = np.exp(g - top).sum(1, keepdims=True) if c["raw"] else w.sum(1, keepdims=True)
    else:
        total = 1.0 if c["raw"] else w.sum(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        w = np.where(on, w / total, 0.0)
    edges = [[] for _ in range(E)]
    for t, j in zip(*np.nonzero(on)):
        edges[sel[t, j]].append((t, j))
    slots, positions = np.full((T, k), -1), np.full(T * k, -1)
    offsets, at = [0], 0
    for e in range(E):
        for t, j in edges[e]:
            slots[t, j], positions[at] = at, t
            at += 1
        offsets.append(at)
    i = lambda v: torch.from_numpy(np.asarray(v, np.int32))  # noqa: E731
    return i(sel), torch.from_numpy(w), i(positions), i(offsets), i(slots)
