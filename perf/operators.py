"""The operators around the grouped expert product, as cases to measure: tokens sorted by expert and
back (with gates and gradients), rows quantised to e4m3 with a scale for each 128 columns, and the
grouped e4m3 product with block scales.

A case names one operator (``op``) and its sizes: T tokens, k experts per token out of E, rows of
H (or K) columns, N output columns.  ``router`` is "even" (normal logits) or "zipf" (a few experts
take most tokens); ``drop`` is the share of (token, slot) assignments that name no expert (padded
tokens of a batch, assignments over an expert's capacity).

With ``own`` false ``run`` computes the plain form in 32 bits from elementary torch operations; with
``own`` true it makes the library's calls.
"""
import math

import torch

own = False

_SIZE = {"float16": 2, "bfloat16": 2, "float32": 4}
_BLOCK = 128
_E4M3_MAX = 448.0
_TINY = 2.0 ** -100   # the smallest block maximum a scale is taken from


def listed():
    return [
        # one decode step of 16 sequences through the 60-expert layer: latency
        dict(name="permute_decode", op="permute", T=16, H=2048, E=60, k=4, dtype="float16", router="even", drop=0.0),
        # a prefill chunk through the 64-expert layer
        dict(name="permute_prefill", op="permute", T=2048, H=3584, E=64, k=8, dtype="bfloat16", router="even", drop=0.0),
        # training in 32 bits with 512 experts, an odd number of tokens and skewed routing
        dict(name="permute_grad_512", op="permute_grad", T=4099, H=2048, E=512, k=10, dtype="float32", router="zipf", drop=0.0),
        # a single new token, top-2 of 8
        dict(name="unpermute_decode", op="unpermute", T=1, H=4096, E=8, k=2, dtype="float16", router="even", drop=0.0, add=False),
        # several prefill chunks at once, the shared expert's output added, padded tokens among them
        dict(name="unpermute_prefill", op="unpermute", T=8192, H=3584, E=64, k=8, dtype="bfloat16", router="even", drop=0.04, add=True),
        # the backward pass of a training batch
        dict(name="unpermute_grad", op="unpermute_grad", T=4096, H=3584, E=64, k=8, dtype="bfloat16", router="even", drop=0.0),
        # activations of one decode step
        dict(name="quantize_decode", op="quantize", T=16, K=2048, dtype="float16"),
        # gate_up's output of a prefill chunk on its way into the down product; rows behind the placed pairs are left alone
        dict(name="silu_quantize_prefill", op="silu_quantize", T=16384, K=2560, dtype="bfloat16", drop=0.05),
        # gate_up of a single token, top-2 of 8: two experts' weights are read
        dict(name="gemm_decode_1", op="gemm", T=1, N=28672, K=4096, E=8, k=2, gather=True, dtype="float16", router="even", drop=0.0),
        # gate_up of 128 decoding sequences, top-8 of 64: every expert is read for a few rows
        dict(name="gemm_decode_128", op="gemm", T=128, N=5120, K=3584, E=64, k=8, gather=True, dtype="bfloat16", router="even", drop=0.0),
        # gate_up of a prefill chunk: about 256 rows for each expert
        dict(name="gemm_prefill_2048", op="gemm", T=2048, N=5120, K=3584, E=64, k=8, gather=True, dtype="bfloat16", router="even", drop=0.0),
        # the always-on shared expert's gate_up for a ragged batch, plain (not grouped), kept in 32 bits
        dict(name="gemm_shared_777", op="gemm", T=777, N=11264, K=2048, E=1, k=1, gather=False, dtype="float32", router="even", drop=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "permute_grad", "unpermute", "unpermute_grad", "quantize", "silu_quantize", "gemm", "gemm"])
    dtype = rng.choice(["float16", "bfloat16", "float32"])
    drop = rng.choice([0.0, 0.0, 0.03, 0.3])
    if op in ("quantize", "silu_quantize"):
        while True:
            case = dict(op=op, T=_log_int(rng, 1, 16384), K=_log_int(rng, 1, 8192), dtype=dtype)
            if op == "silu_quantize":
                case["drop"] = drop
            if case["T"] * case["K"] <= 40_000_000:
                return case
    while True:
        E = _log_int(rng, 1, 512)
        case = dict(op=op, E=E, k=rng.randint(1, min(E, 10)), dtype=dtype, router=rng.choice(["even", "zipf"]), drop=drop)
        if op == "gemm":
            case.update(T=_log_int(rng, 1, 4096), N=_log_int(rng, 64, 12000), K=16 * _log_int(rng, 4, 512), gather=rng.random() < 0.5)
            if E == 1:
                case.update(gather=False, drop=0.0)
            if E * case["N"] * case["K"] > 1_150_000_000 or case["T"] * case["k"] * case["N"] * case["K"] > 3.0e11:
                continue
            if case["T"] * max(case["k"] * max(case["N"], case["K"]) * 16, E * max(case["N"], case["K"])) > 2_560_000_000:
                continue
            return case
        case.update(T=_log_int(rng, 1, 8192), H=_log_int(rng, 8, 8192))
        if op == "unpermute":
            case["add"] = rng.random() < 0.5
        if case["T"] * case["k"] * case["H"] * _SIZE[dtype] <= 460_000_000:
            return case


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _dtype(case):
    return getattr(torch, case["dtype"])


def _routing(case, g):
    """One batch's routing and grouping, as moe_route_topk and moe_group_by_expert leave it."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, device="cuda", generator=g)
    if case["router"] == "zipf":
        logits -= 1.1 * torch.log(torch.randperm(E, device="cuda", generator=g).float() + 1)
    top, ids = torch.topk(logits, k, dim=1)
    gates = torch.softmax(top, dim=1)
    if case["drop"]:
        ids = ids.masked_fill(torch.rand(T, k, device="cuda", generator=g) < case["drop"], -1)
    key = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    n = int(offsets[E])
    pairs = torch.zeros(T * k, dtype=torch.int32, device="cuda")
    pairs[:n] = order[:n]
    rows = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    rows[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    return dict(ids=ids.int().contiguous(), gates=gates.contiguous(), offsets=offsets, pairs=pairs, rows=rows.view(T, k),
                n=n, counts=counts)


def _padding(s):
    """The plan of the grouped product's plain form: its active experts and the place of every sorted
    row in a stack of equally high groups."""
    active = torch.nonzero(s["counts"]).reshape(-1)
    counts = s["counts"][active]
    high = int(counts.max()) if active.numel() else 0
    group = torch.repeat_interleave(torch.arange(active.numel(), device="cuda"), counts)
    first = s["offsets"][active].long()
    place = group * high + torch.arange(s["n"], device="cuda") - first[group]
    return active, high, place


def _e4m3(g, *shape):
    """Values as a quantiser leaves them: most of the range used, in fractions of 448."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in out.view(-1, shape[-1]).split(1 << 14):
        part.copy_((torch.randn(part.shape, device="cuda", generator=g) * 120).clamp_(-_E4M3_MAX, _E4M3_MAX))
    return out


def prepare(case, seed):
    g, op, dt = _generator(seed), case["op"], _dtype(case)
    s = dict(case=case)
    if op in ("quantize", "silu_quantize"):
        T, K = case["T"], case["K"]
        wide = 2 * K if op == "silu_quantize" else K
        s["x"] = (torch.randn(T, wide, device="cuda", generator=g) * torch.exp(torch.randn(T, 1, device="cuda", generator=g))).to(dt)
        s["n"] = T - int(T * case.get("drop", 0.0))
        s["n_rows"] = torch.tensor([s["n"]], dtype=torch.int32, device="cuda") if op == "silu_quantize" else None
        s["q"] = torch.zeros(T, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.zeros(T, -(-K // _BLOCK), device="cuda")
        return s
    s.update(_routing(case, g))
    T, k, E, pairs = case["T"], case["k"], case["E"], case["T"] * case["k"]
    if op == "gemm":
        N, K = case["N"], case["K"]
        nb, kb = -(-N // _BLOCK), -(-K // _BLOCK)
        rows = T if case["gather"] else pairs
        s["a"] = _e4m3(g, rows, K)
        s["a_scales"] = torch.exp(0.5 * torch.randn(rows, kb, device="cuda", generator=g)) / 120
        s["w"] = _e4m3(g, E, N, K)
        s["w_scales"] = torch.exp(0.25 * torch.randn(E, nb, kb, device="cuda", generator=g)) * (0.02 / 120)
        s["c"] = torch.zeros(pairs, N, dtype=dt, device="cuda")
        s["active"], s["high"], s["place"] = _padding(s)
        return s
    H = case["H"]
    if op == "permute":
        s["x"] = torch.randn(T, H, device="cuda", generator=g).to(dt)
        s["xs"] = torch.zeros(pairs, H, dtype=dt, device="cuda")
        s["rows_out"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    elif op == "permute_grad":
        s["dxs"] = torch.randn(pairs, H, device="cuda", generator=g).to(dt)
        s["dx"] = torch.zeros(T, H, dtype=dt, device="cuda")
    elif op == "unpermute":
        s["ys"] = torch.randn(pairs, H, device="cuda", generator=g).to(dt)
        s["add"] = torch.randn(T, H, device="cuda", generator=g).to(dt) if case["add"] else None
        s["y"] = torch.zeros(T, H, dtype=dt, device="cuda")
    else:
        s["dy"] = torch.randn(T, H, device="cuda", generator=g).to(dt)
        s["ys"] = torch.randn(pairs, H, device="cuda", generator=g).to(dt)
        s["dys"] = torch.zeros(pairs, H, dtype=dt, device="cuda")
        s["dgates"] = torch.zeros(T, k, device="cuda")
    return s


def _own(s, op):
    import any_precision_expert_router_amd as apq
    if op == "permute":
        apq.moe_permute_tokens(s["x"], s["ids"], s["offsets"], s["pairs"], s["xs"], s["rows_out"])
        return s["xs"], s["rows_out"]
    if op == "permute_grad":
        apq.moe_permute_tokens_backward(s["dxs"], s["rows"], s["dx"])
        return s["dx"]
    if op == "unpermute":
        apq.moe_unpermute_tokens(s["ys"], s["rows"], s["gates"], s["y"], add=s["add"])
        return s["y"]
    if op == "unpermute_grad":
        apq.moe_unpermute_tokens_backward(s["dy"], s["ys"], s["rows"], s["gates"], s["dys"], s["dgates"])
        return s["dys"], s["dgates"]
    if op == "quantize":
        apq.moe_fp8_quantize(s["x"], s["q"], s["scales"])
        return s["q"], s["scales"]
    if op == "silu_quantize":
        apq.moe_fp8_quantize_silu(s["x"], s["q"], s["scales"], n_rows=s["n_rows"])
        return s["q"], s["scales"]
    grouped = s["case"]["E"] > 1
    apq.moe_fp8_gemm(s["a"], s["a_scales"], s["w"], s["w_scales"], s["c"], expert_offsets=s["offsets"] if grouped else None,
                     sorted_pairs=s["pairs"] if s["case"]["gather"] else None, k=s["case"]["k"])
    return s["c"]


def _gathered(ys, rows, weights):
    """sum over a token's slots of weight * row, slots without a row left out."""
    taken = ys.float()[rows.clamp(min=0).long()]
    if weights is not None:
        taken = taken * weights[..., None]
    return torch.where(rows[..., None] >= 0, taken, 0.0).sum(1)


def _wide(scales, dim, size):
    return scales.repeat_interleave(_BLOCK, dim).narrow(dim, 0, size)


def _quantized(x, s):
    T, K = x.shape
    kb = -(-K // _BLOCK)
    m = torch.nn.functional.pad(x.abs(), (0, kb * _BLOCK - K)).view(T, kb, _BLOCK).amax(2).clamp(min=_TINY)
    s["q"][:T] = (x * _wide(_E4M3_MAX / m, 1, K)).to(torch.float8_e4m3fn)
    s["scales"][:T] = m / _E4M3_MAX
    return s["q"], s["scales"]


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "quantize":
        return _quantized(s["x"].float(), s)
    if op == "silu_quantize":
        gate, up = s["x"][:s["n"]].float().chunk(2, 1)
        return _quantized(gate / (1 + torch.exp(-gate)) * up, s)
    n, k = s["n"], s["case"]["k"]
    pairs = s["pairs"][:n].long()
    if op == "permute":
        s["xs"][:n] = s["x"][pairs // k]
        s["rows_out"].fill_(-1)
        s["rows_out"].view(-1)[pairs] = torch.arange(n, dtype=torch.int32, device="cuda")
        return s["xs"], s["rows_out"]
    if op == "permute_grad":
        s["dx"].copy_(_gathered(s["dxs"], s["rows"], None))
        return s["dx"]
    if op == "unpermute":
        y = _gathered(s["ys"], s["rows"], s["gates"])
        s["y"].copy_(y if s["add"] is None else y + s["add"].float())
        return s["y"]
    if op == "unpermute_grad":
        dy = s["dy"].float()[pairs // k]
        s["dys"][:n] = (dy * s["gates"].view(-1)[pairs][:, None]).to(s["dys"].dtype)
        s["dgates"].zero_()
        s["dgates"].view(-1)[pairs] = (dy * s["ys"][:n].float()).sum(1)
        return s["dys"], s["dgates"]
    N, K = s["case"]["N"], s["case"]["K"]
    a = s["a"].float() * _wide(s["a_scales"], 1, K)
    a = a[pairs // k] if s["case"]["gather"] else a[:n]
    w = s["w"][s["active"]].float()
    w *= _wide(_wide(s["w_scales"][s["active"]], 1, N), 2, K)
    stacked = torch.zeros(s["active"].numel() * s["high"], K, device="cuda")
    stacked[s["place"]] = a
    c = torch.bmm(stacked.view(s["active"].numel(), s["high"], K), w.transpose(1, 2)).view(-1, N)
    s["c"][:n] = c[s["place"]].to(s["c"].dtype)
    return s["c"]


def _pairs_of(case):
    return case["T"] * case["k"] * (1 - case["drop"])


def work(case):
    op, T, size = case["op"], case["T"], _SIZE[case["dtype"]]
    if op in ("quantize", "silu_quantize"):
        K, wide = case["K"], 2 if op == "silu_quantize" else 1
        T = T - int(T * case.get("drop", 0.0))
        return dict(bytes=T * K * (wide * size + 1) + 4 * T * -(-K // _BLOCK), flops=T * K * (2 if wide == 1 else 6))
    P, E, k = _pairs_of(case), case["E"], case["k"]
    index = 4 * T * k
    if op == "gemm":
        N, K = case["N"], case["K"]
        active = E * (1 - (1 - k / E) ** (T * (1 - case["drop"]))) if E > 1 else 1
        a_rows = T if case["gather"] else P
        return dict(bytes=active * (N * K + 4 * (N // _BLOCK) * (K // _BLOCK)) + a_rows * (K + 4 * (K // _BLOCK)) + P * N * size,
                    flops=2 * P * N * K)
    row = case["H"] * size
    if op == "permute":
        return dict(bytes=T * row + P * row + 3 * index, flops=0)
    if op == "permute_grad":
        return dict(bytes=P * row + T * row + index, flops=P * case["H"])
    if op == "unpermute":
        return dict(bytes=P * row + T * row * (2 if case["add"] else 1) + 2 * index, flops=2 * P * case["H"])
    return dict(bytes=2 * P * row + T * row + 3 * index, flops=3 * P * case["H"])


def _nearest_e4m3(v):
    """The e4m3 value nearest to each double, ties to an even last bit (4 significant bits, exponents from -6)."""
    exponent = torch.frexp(v.abs())[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    """The definitions in 64 bits, one token's slot, one block column or one expert at a time."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("quantize", "silu_quantize"):
        n, K = s["n"], case["K"]
        x = s["x"][:n].double()
        if op == "silu_quantize":
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        q = torch.zeros(case["T"], K, dtype=torch.float64, device="cuda")
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
        for b, first in enumerate(range(0, K, _BLOCK)):
            block = x[:, first:first + _BLOCK]
            top = block.abs().max(1, keepdim=True).values.clamp(min=_TINY)
            q[:n, first:first + _BLOCK] = _nearest_e4m3(block * (_E4M3_MAX / top))
            scales[:n, b] = top[:, 0] / _E4M3_MAX
        return q, scales
    T, k = case["T"], case["k"]
    if op == "permute":
        xs = torch.zeros(s["xs"].shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            there = s["rows"][:, j] >= 0
            xs[s["rows"][there, j].long()] = s["x"][there].double()
        return xs, s["rows"]
    if op in ("permute_grad", "unpermute"):
        src = s["dxs"] if op == "permute_grad" else s["ys"]
        y = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
        if op == "unpermute" and s["add"] is not None:
            y += s["add"].double()
        for j in range(k):
            there = s["rows"][:, j] >= 0
            term = src[s["rows"][there, j].long()].double()
            y[there] += term if op == "permute_grad" else s["gates"][there, j].double()[:, None] * term
        return y
    if op == "unpermute_grad":
        dys = torch.zeros(s["dys"].shape, dtype=torch.float64, device="cuda")
        dgates = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            there = s["rows"][:, j] >= 0
            row, dy = s["rows"][there, j].long(), s["dy"][there].double()
            dys[row] = s["gates"][there, j].double()[:, None] * dy
            dgates[there, j] = torch.linalg.vecdot(dy, s["ys"][row].double())
        return dys, dgates
    N, K = case["N"], case["K"]
    column = torch.arange(K, device="cuda") // _BLOCK
    block = torch.arange(N, device="cuda") // _BLOCK
    c = torch.zeros(s["c"].shape, dtype=torch.float64, device="cuda")
    edges = s["offsets"].tolist()
    for e in range(case["E"]):
        first, last = edges[e], edges[e + 1]
        if first == last:
            continue
        source = s["pairs"][first:last].long() // k if case["gather"] else torch.arange(first, last, device="cuda")
        a = s["a"][source].double() * s["a_scales"][source].double()[:, column]
        w = s["w"][e].double() * s["w_scales"][e].double()[block][:, column]
        c[first:last] = a @ w.t()
    return c
