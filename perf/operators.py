"""What is measured of the mixture-of-experts operators, and their plain forms.

Four operators make a feed-forward block of experts out of MXFP4 weights: the
router's choice (``route``), the product grouped by expert (``grouped``), the
gated activation with its quantizer (``glu``) and the norms around the block
with gate, residual and quantizer (``norm``).  Each case is one call of one of
them.

Quantized outputs are returned as the values they stand for: the elements in
float8_e4m3fn (which holds every E2M1 value too) and the block scales in
float8_e8m0fnu.
"""
import math

import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases --------------------------------------------------------------------

def _route(tokens, experts, top_k, bf16, renorm, masked):
    return {"op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "bf16": bf16, "renorm": renorm,
            "masked": masked}


def _grouped(tokens, experts, top_k, N, K, fp8, gather):
    return {"op": "grouped", "tokens": tokens, "experts": experts, "top_k": top_k, "N": N, "K": K, "fp8": fp8,
            "gather": gather}


def _glu(rows, K, fp8):
    return {"op": "glu", "rows": rows, "K": K, "fp8": fp8}


def _norm(tokens, K, top_k, post, gate, fp8):
    return {"op": "norm", "tokens": tokens, "K": K, "top_k": top_k, "post": post, "gate": gate, "fp8": fp8}


def listed():
    return [
        # one token of a decode: the latency of the choice
        dict(_route(1, 32, 4, False, True, False), name="route_1x32"),
        # a short prompt of odd length
        dict(_route(509, 64, 6, True, True, True), name="route_509x64"),
        # a long prefill over many experts, weights from the softmax over all
        dict(_route(16384, 128, 8, False, False, False), name="route_16384x128"),
        # one token's gate and up products: four experts' weights are streamed
        dict(_grouped(1, 32, 4, 4096, 2048, False, True), name="grouped_1_fp4"),
        # a decode batch: every expert has a few rows, all weights are streamed
        dict(_grouped(32, 32, 4, 4096, 2048, True, True), name="grouped_32_fp8"),
        # a short prompt on sizes that fill neither a tile nor a 128-element step
        dict(_grouped(509, 64, 4, 1440, 2880, True, True), name="grouped_509_fp8_ragged"),
        # a long prefill's gate and up products: bound by the matrix units
        dict(_grouped(8192, 32, 4, 4096, 2048, False, True), name="grouped_8192_fp4"),
        # one token's activations (four experts' rows)
        dict(_glu(4, 2048, True), name="glu_4x2048_fp8"),
        # a long prefill's activations
        dict(_glu(32768, 2048, False), name="glu_32768x2048_fp4"),
        # one token behind the experts, in front of the next block
        dict(_norm(1, 4096, 4, True, False, True), name="norm_1x4096_fp8"),
        # a dense block between two norms, with a gate per token, odd length
        dict(_norm(509, 2880, 0, True, True, False), name="norm_509x2880_fp4"),
        # a long prefill behind the experts
        dict(_norm(8192, 4096, 4, True, False, True), name="norm_8192x4096_fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "glu", "norm"])
    if op == "route":
        experts = rng.choice([rng.randint(4, 128), 8, 16, 32, 64, 128])
        return _route(_log(rng, 1, 16384), experts, rng.randint(1, min(8, experts)), rng.random() < 0.5,
                      rng.random() < 0.5, rng.random() < 0.3)
    if op == "grouped":
        experts = rng.choice([rng.randint(1, 64), 8, 16, 32, 64])
        K = 32 * rng.choice([rng.randint(8, 128), 32, 64, 128])
        N = rng.choice([rng.randint(200, 4096), 16 * rng.randint(16, 256), 1024, 2048, 4096])
        N = min(N, max(200, 32 * 4096 * 2048 // (experts * K)))
        top_k = rng.randint(1, min(8, experts))
        most = max(1, 4 * 8192 * 4096 * 2048 // (top_k * N * K))
        return _grouped(_log(rng, 1, min(8192, most)), experts, top_k, N, K, rng.random() < 0.5, rng.random() < 0.6)
    if op == "glu":
        K = 32 * rng.choice([rng.randint(8, 128), 32, 64, 128])
        return _glu(_log(rng, 1, min(32768, 32768 * 2048 // K)), K, rng.random() < 0.5)
    K = 32 * rng.choice([rng.randint(8, 256), 64, 128, 256])
    top_k = rng.choice([0, 1, 2, 4, 6, 8])
    most = 8192 * 4096 * 8 // (K * max(4 + 2 * top_k, 8))
    return _norm(_log(rng, 1, most), K, top_k, rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _fp4_bytes(g, *shape):
    """Two E2M1 codes a byte, each a normal value rounded to E2M1 under a block scale of about 4 / max."""
    q = (torch.arange(256, device="cuda") + 0.5) / 256
    v = torch.erfinv(2 * q - 1) * math.sqrt(2) * 2.0
    grid = torch.tensor(E2M1, device="cuda")
    code = (v.abs()[:, None] - grid).abs().argmin(1) + 8 * (v < 0)
    table = (code[:, None] * 16 + code[None, :]).reshape(-1).to(torch.uint8)
    return table[torch.randint(0, 65536, shape, device="cuda", dtype=torch.int32, generator=g)]


def _scales(g, middle, *shape):
    return (torch.randint(-1, 2, shape, device="cuda", generator=g) + middle).to(torch.uint8)


def _routing(g, tokens, experts, top_k):
    """A routing as a router makes it: some experts are asked for more than others."""
    logits = torch.randn(tokens, experts, device="cuda", generator=g)
    logits += torch.randn(experts, device="cuda", generator=g)
    ids = logits.topk(top_k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=experts)
    offsets = torch.zeros(experts + 1, device="cuda", dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    return offsets, torch.div(order, top_k, rounding_mode="floor").to(torch.int32), order, counts


def prepare(case, seed):
    g = _gen(seed)
    c, st = dict(case), dict(case)
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        x = 2 * torch.randn(T, E, device="cuda", generator=g)
        if c["masked"]:  # experts that are switched off for a token; now and then all of them
            x[torch.rand(T, E, device="cuda", generator=g) < 0.3] = -math.inf
            x[torch.rand(T, device="cuda", generator=g) < 0.05] = -math.inf
        st["logits"] = x.to(torch.bfloat16) if c["bf16"] else x
        i32 = dict(device="cuda", dtype=torch.int32)
        st["ids"], st["pos"] = torch.empty(T, k, **i32), torch.empty(T, k, **i32)
        st["weights"] = torch.empty(T, k, device="cuda")
        st["offsets"], st["rows"] = torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
        st["workspace"] = torch.empty(_route_workspace(T, E), device="cuda", dtype=torch.uint8)
    elif c["op"] == "grouped":
        T, E, k, N, K = c["tokens"], c["experts"], c["top_k"], c["N"], c["K"]
        st["offsets"], st["a_rows"], _, counts = _routing(g, T, E, k)
        a = T if c["gather"] else T * k
        if c["fp8"]:
            st["A"] = (torch.randn(a, K, device="cuda", generator=g) * 96).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            st["A"] = _fp4_bytes(g, a, K // 2)
        st["SA"] = _scales(g, 120 if c["fp8"] else 126, a, K // 32)
        st["B"], st["SB"] = _fp4_bytes(g, E, N, K // 2), _scales(g, 120, E, N, K // 32)
        st["D"] = torch.zeros(T * k, N, device="cuda", dtype=torch.bfloat16)
        # the plain form's plan: the experts that have rows, and how many the largest has
        st["active"] = torch.nonzero(counts).reshape(-1)
        st["most"] = int(counts.max())
    elif c["op"] == "glu":
        M, K = c["rows"], c["K"]
        st["X"] = torch.randn(M, 2 * K, device="cuda", generator=g).to(torch.bfloat16)
        st["A"] = torch.zeros(M, K if c["fp8"] else K // 2, device="cuda", dtype=torch.uint8)
        st["SA"] = torch.zeros(M, K // 32, device="cuda", dtype=torch.uint8)
        st["live"] = torch.tensor([M - M // 16], device="cuda", dtype=torch.int32)  # some tokens were not routed
    else:
        T, K, k = c["tokens"], c["K"], c["top_k"]
        bf = dict(device="cuda", dtype=torch.bfloat16)
        st["Y"] = torch.randn(T * max(k, 1), K, device="cuda", generator=g).to(torch.bfloat16)
        st["X"] = (2 * torch.randn(T, K, device="cuda", generator=g)).to(torch.bfloat16)
        if k:
            st["pos"] = torch.randperm(T * k, device="cuda", generator=g).to(torch.int32).reshape(T, k)
            st["pos"][torch.rand(T, k, device="cuda", generator=g) < 0.02] = -1
            st["weights"] = torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1)
        if c["post"]:
            st["w_post"] = (1 + 0.1 * torch.randn(K, device="cuda", generator=g)).to(torch.bfloat16)
        if c["gate"]:
            st["G"] = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
        st["w_pre"] = (1 + 0.1 * torch.randn(K, device="cuda", generator=g)).to(torch.bfloat16)
        st["scale"] = 0.75
        st["H"], st["Z"] = torch.empty(T, K, **bf), torch.empty(T, K, **bf)
        st["A"] = torch.empty(T, K if c["fp8"] else K // 2, device="cuda", dtype=torch.uint8)
        st["SA"] = torch.empty(T, K // 32, device="cuda", dtype=torch.uint8)
    # what a byte of two E2M1 codes stands for, as two float8_e4m3fn bytes
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    b = torch.arange(256, device="cuda")
    st["e2m1_pairs"] = torch.stack((v[b & 15], v[b >> 4]), 1).view(torch.int16).reshape(-1)
    return st


def _route_workspace(tokens, experts):
    """Bytes of the choice's workspace: a count for every expert and 64 tokens."""
    return 4 * experts * ((tokens + 63) // 64)


# ---- plain forms --------------------------------------------------------------

def _elements(bytes_, fp8):
    """The values of 8-bit or packed 4-bit elements, in 32 bits."""
    if fp8:
        return bytes_.view(torch.float8_e4m3fn).float()
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=bytes_.device)
    return torch.stack((v[(bytes_ & 15).int()], v[(bytes_ >> 4).int()]), -1).reshape(*bytes_.shape[:-1], -1)


def _power(x):
    """2^x in 32 bits, exactly, for -127 < x < 128."""
    return ((x.int() + 127) << 23).view(torch.float32)


def _times_scale(values, scales):
    s = _power(scales.int() - 127)
    return (values.reshape(*scales.shape, 32) * s[..., None]).reshape(values.shape)


def _quantize(v, fp8):
    """Elements and scales of bf16 rows: a power of two for each 32, elements to nearest even, saturating."""
    b = v.float().reshape(*v.shape[:-1], -1, 32)
    most = b.abs().amax(-1, keepdim=True)
    special = ~torch.isfinite(most)
    x = (torch.frexp(most).exponent - 1 - (8 if fp8 else 2)).clamp(-127, 127)
    x = torch.where(most == 0, -127, x)
    s = b * _power(-x)
    if fp8:
        q = s.clamp(-448, 448)
    else:
        m = s.abs().clamp(max=6)
        step = 0.5 + 0.5 * (m >= 2) + 1.0 * (m >= 4)
        q = torch.copysign(torch.round(m / step) * step, s)
    q = torch.where(special, 0.0, q).to(torch.float8_e4m3fn)
    scale = torch.where(special, 255, x + 127).to(torch.uint8)[..., 0]
    return q.reshape(v.shape), scale.view(torch.float8_e8m0fnu)


def _plain_route(s):
    x, k, E = s["logits"].float(), s["top_k"], s["experts"]
    x = torch.where(torch.isnan(x), -math.inf, x)
    ranked = torch.sort(x, dim=1, descending=True, stable=True)
    some = ranked.values[:, :k] > -math.inf
    ids = torch.where(some, ranked.indices[:, :k], -1)
    top = ranked.values[:, :1]
    p = torch.where(ranked.values == top, 1.0, torch.exp(ranked.values - top))
    total = p[:, :k].sum(1, keepdim=True) if s["renorm"] else p.sum(1, keepdim=True)
    weights = torch.where(some, p[:, :k] / total, 0.0)
    flat = ids.reshape(-1)
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    counts = torch.bincount(torch.where(flat < 0, E, flat), minlength=E + 1)[:E]
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    place = torch.arange(flat.numel(), device=x.device)
    rows = torch.where(place < offsets[-1], torch.div(order, k, rounding_mode="floor"), -1)
    pos = torch.empty_like(flat)
    pos[order] = place
    pos = torch.where(flat < 0, -1, pos).reshape(ids.shape)
    return {"ids": ids.int(), "weights": weights, "pos": pos.int(), "offsets": offsets.int(), "rows": rows.int()}


def _plain_grouped(s):
    a = _times_scale(_elements(s["A"], s["fp8"]), s["SA"])
    b = _times_scale(_elements(s["B"][s["active"]], False), s["SB"][s["active"]])
    if s["gather"]:
        a = a[s["a_rows"].long()]
    i = torch.arange(a.shape[0], device=a.device)
    e = torch.searchsorted(s["offsets"][1:].long(), i, right=True)
    slot, mine = i - s["offsets"][e].long(), torch.searchsorted(s["active"], e)
    padded = a.new_zeros(b.shape[0], s["most"], a.shape[1])
    padded[mine, slot] = a
    d = torch.bmm(padded, b.transpose(1, 2).contiguous())
    return d[mine, slot].to(torch.bfloat16)


def _plain_glu(s):
    K = s["K"]
    gate, up = s["X"][:, :K].float(), s["X"][:, K:].float()
    q, scale = _quantize((gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16), s["fp8"])
    live = torch.arange(s["rows"], device=gate.device)[:, None] < s["live"]
    zero = torch.zeros((), device=gate.device, dtype=torch.uint8)
    return {"elements": torch.where(live, q.view(torch.uint8), zero).view(q.dtype),
            "scales": torch.where(live, scale.view(torch.uint8), zero).view(scale.dtype)}


def _plain_rms(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _plain_norm(s):
    if s["top_k"]:
        y = s["Y"].float()[s["pos"].clamp(min=0).long()]
        y = (y * torch.where(s["pos"] < 0, 0.0, s["weights"])[..., None]).sum(1)
    else:
        y = s["Y"].float()
    if s["post"]:
        y = _plain_rms(y, s["w_post"])
    if s["gate"]:
        y = y * s["G"].float()
    h = (s["X"].float() + s["scale"] * y).to(torch.bfloat16)
    z = _plain_rms(h.float(), s["w_pre"]).to(torch.bfloat16)
    q, scale = _quantize(z, s["fp8"])
    return {"H": h, "Z": z, "elements": q, "scales": scale}


# ---- the framework's calls ------------------------------------------------------

def _values(s):
    """The quantized outputs as the values they stand for."""
    if s["fp8"]:
        q = s["A"].view(torch.float8_e4m3fn)
    else:
        q = s["e2m1_pairs"][s["A"].int()].view(torch.float8_e4m3fn)
    return {"elements": q, "scales": s["SA"].view(torch.float8_e8m0fnu)}


def _own(s):
    import block_scaled_precision_mxfp4_amd as mx
    fmt = mx.FMT_FP8_E4M3 if s.get("fp8") else mx.FMT_FP4
    if s["op"] == "route":
        mx.mxgemm_route(s["ids"], s["weights"], s["pos"], s["offsets"], s["rows"], s["logits"], s["tokens"], s["experts"],
                        s["top_k"], bf16=s["bf16"], renorm=s["renorm"], workspace=s["workspace"],
                        workspace_bytes=s["workspace"].numel())
        return {n: s[n] for n in ("ids", "weights", "pos", "offsets", "rows")}
    if s["op"] == "grouped":
        rows = s["tokens"] * s["top_k"]
        mx.mxgemm_grouped_run(s["D"], s["A"], s["B"], s["SA"], s["SB"], s["offsets"], rows, s["N"], s["K"], s["experts"],
                              a_rows=s["a_rows"] if s["gather"] else None, a_count=s["tokens"] if s["gather"] else rows,
                              a_format=fmt)
        return s["D"]
    if s["op"] == "glu":
        mx.mxgemm_glu_quantize(s["A"], s["SA"], s["X"], s["rows"], s["K"], live=s["live"], a_format=fmt)
        return _values(s)
    mx.mxgemm_norm_quantize(s["tokens"], s["K"], Y=s["Y"], pos=s.get("pos"), weights=s.get("weights"), top_k=s["top_k"],
                            y_rows=s["Y"].shape[0], w_post=s.get("w_post"), gate=s.get("G"), res_scale=s["scale"], X=s["X"],
                            H=s["H"], w_pre=s["w_pre"], Z=s["Z"], A=s["A"], scaleA=s["SA"], a_format=fmt, eps=EPS)
    return {"H": s["H"], "Z": s["Z"], **_values(s)}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "grouped": _plain_grouped, "glu": _plain_glu, "norm": _plain_norm}[state["op"]](state)


# ---- work -----------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        return {"bytes": T * E * (2 if c["bf16"] else 4) + T * k * 16 + 4 * (E + 1), "flops": 4 * T * E}
    width = 1.0 if c["fp8"] else 0.5
    if c["op"] == "grouped":
        T, E, k, N, K = c["tokens"], c["experts"], c["top_k"], c["N"], c["K"]
        active = E * (1 - (1 - k / E) ** T)  # expected number of experts that have rows
        a = T if c["gather"] else T * k
        return {"bytes": active * N * K * 17 / 32 + a * K * (width + 1 / 32) + 2 * T * k * N, "flops": 2 * T * k * N * K}
    if c["op"] == "glu":
        n = c["rows"] * c["K"]
        return {"bytes": n * (4 + width + 1 / 32), "flops": 8 * n}
    n, k = c["tokens"] * c["K"], c["top_k"]
    return {"bytes": n * (2 * max(k, 1) + 2 + 2 * c["gate"] + 4 + width + 1 / 32), "flops": n * (12 + 2 * k)}


# ---- 64 bits --------------------------------------------------------------------

def _exact_elements(bytes_, fp8):
    """Elements by the formats' fields: sign, exponent, fraction."""
    if fp8:
        b = bytes_.long()
        sign, e, f = 1 - 2 * (b >> 7), (b >> 3) & 15, (b & 7).double()
        m = torch.where(e == 0, f / 512, (8 + f) * _exact_power(e - 10))
    else:
        b = torch.stack((bytes_ & 15, bytes_ >> 4), -1).reshape(*bytes_.shape[:-1], -1).long()
        sign, e, f = 1 - 2 * (b >> 3), (b >> 1) & 3, (b & 1).double()
        m = torch.where(e == 0, f / 2, (2 + f) * _exact_power(e - 2))
    return sign * m


def _exact_operand(bytes_, scales, fp8):
    s = _exact_power(scales.long() - 127)
    return _exact_elements(bytes_, fp8) * s.repeat_interleave(32, dim=-1)


def _exact_power(x):
    """2^x in 64 bits, by its exponent field."""
    return ((x.long() + 1023) << 52).view(torch.float64)


def _to_bf16(x):
    """64 bits to bf16's values in one rounding: 8 bits of fraction with its leading one, ties to even."""
    m, e = torch.frexp(x)
    return torch.round(m * 256) * _exact_power(e - 8)


def _exact_quantized(v, fp8):
    """v: bf16 values in 64 bits."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    most = b.abs().amax(-1)
    x = (torch.frexp(most).exponent - 1 - (8 if fp8 else 2)).clamp(-127, 127)
    x = torch.where(most > 0, x, -127)
    s = b * _exact_power(-x)[..., None]
    limit, bits, least = (448.0, 3, -6) if fp8 else (6.0, 1, 0)
    m = s.abs().clamp(max=limit)
    step = _exact_power(torch.frexp(m.clamp(min=2.0 ** least)).exponent - 1 - bits)
    return (torch.copysign(torch.round(m / step) * step, s)).reshape(v.shape), _exact_power(x)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        x, k = s["logits"].double(), s["top_k"]
        w, ids = torch.topk(x, k, dim=1)
        e = torch.exp(x - x.max(1, keepdim=True).values)
        total = (torch.exp(w - w[:, :1]) if s["renorm"] else e).sum(1, keepdim=True)
        w = torch.exp(w - w[:, :1]) / total
        return {"ids": None, "weights": torch.where(torch.isnan(w), 0.0, w), "pos": None, "offsets": None, "rows": None}
    if case["op"] == "grouped":
        a = _exact_operand(s["A"], s["SA"], s["fp8"])
        if s["gather"]:
            a = a[s["a_rows"].long()]
        out, off = torch.empty(a.shape[0], s["N"], device="cuda", dtype=torch.float64), s["offsets"].tolist()
        for e in range(s["experts"]):
            if off[e + 1] > off[e]:
                out[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ _exact_operand(s["B"][e], s["SB"][e], False).T
        return out
    if case["op"] == "glu":
        live = int(s["live"])
        x = s["X"].double()
        v = x[:, :s["K"]] * torch.sigmoid(x[:, :s["K"]]) * x[:, s["K"]:]
        q, scale = _exact_quantized(_to_bf16(v), s["fp8"])
        q[live:], scale[live:] = 0, 2.0 ** -127
        return {"elements": q, "scales": scale}
    if s["top_k"]:
        y = torch.zeros(s["tokens"], s["K"], device="cuda", dtype=torch.float64)
        for j in range(s["top_k"]):
            p = s["pos"][:, j].long()
            y += torch.where((p >= 0)[:, None], s["weights"][:, j:j + 1].double() * s["Y"][p.clamp(min=0)].double(), 0)
    else:
        y = s["Y"].double()
    norm = lambda t, w: t / torch.sqrt((t * t).sum(-1, keepdim=True) / s["K"] + EPS) * w.double()  # noqa: E731
    y = norm(y, s["w_post"]) if s["post"] else y
    y = y * s["G"].double() if s["gate"] else y
    h = s["X"].double() + s["scale"] * y
    z = norm(_to_bf16(h), s["w_pre"])
    q, scale = _exact_quantized(_to_bf16(z), s["fp8"])
    return {"H": h, "Z": z, "elements": q, "scales": scale}
