"""Cases of the operators that run a calibrated layer: NVFP4 quantisation of tokens, the product of NVFP4 tokens and
weights (one matrix, or one matrix per expert), tokens sorted by expert, and the experts' rows brought back.

Every case can be computed in two ways on the same inputs: in the plain form (elementary torch operations in 32 bits)
and by the library's calls (`own`).

The NVFP4 definition used throughout, for a row x of c_in values in blocks of 16:
    g     = fp32(amax / 2688), amax the largest |x| of the row, or a given amax of the whole tensor
    v_b   = E4M3_RNE_sat(fp32(fp32(amax_b / 6) / g)), at least 2^-9 (2^-9 where g == 0)
    s_b   = fp32(v_b * g)
    q_i   = E2M1_RNE_sat(fp32(x_i / s_b))   (0 where s_b == 0)
    value = fp32(q_i * s_b)
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one token of a serving step, one scale per token; what the token's values become is kept beside the codes
        {"name": "tokens_one", "op": "tokens", "n": 1, "c": 4096, "type": BF16, "scale": "token"},
        # a prompt's activations before a 4096-wide layer
        {"name": "tokens_prompt", "op": "tokens", "n": 8192, "c": 4096, "type": BF16, "scale": "token"},
        # an odd number of unrounded tokens before a down projection, with the calibrated amax of the tensor
        {"name": "tokens_wide_f32", "op": "tokens", "n": 1777, "c": 17408, "type": F32, "scale": "tensor"},
        # single-token decoding through an attention projection
        {"name": "linear_one", "op": "linear", "n": 1, "c": 4096, "m": 4096, "type": BF16, "scale": "token"},
        # a ragged batch through a down projection, results kept in 32 bits
        {"name": "linear_ragged", "op": "linear", "n": 333, "c": 17408, "m": 5120, "type": F32, "scale": "tensor"},
        # a prompt through an up projection
        {"name": "linear_prompt", "op": "linear", "n": 8192, "c": 4096, "m": 12288, "type": BF16, "scale": "token"},
        # one decoding step of 48 sequences through an expert bank
        {"name": "experts_decode", "op": "experts", "n": 48, "k": 4, "e": 64, "c": 2048, "m": 1536, "type": BF16},
        # a prompt through the same bank
        {"name": "experts_prompt", "op": "experts", "n": 8192, "k": 4, "e": 64, "c": 2048, "m": 1536, "type": BF16},
        # the sorting of a decoding step's tokens and of a calibration batch's
        {"name": "dispatch_decode", "op": "dispatch", "n": 48, "k": 4, "e": 64, "c": 2048, "type": BF16},
        {"name": "dispatch_prompt", "op": "dispatch", "n": 8192, "k": 4, "e": 64, "c": 2048, "type": BF16},
        # the experts' rows back to a decoding step's tokens
        {"name": "combine_decode", "op": "combine", "n": 48, "k": 4, "e": 64, "c": 1536, "type": F32, "grad": False},
        # the same for a training batch, forward and backward
        {"name": "combine_train", "op": "combine", "n": 8192, "k": 4, "e": 64, "c": 1536, "type": BF16, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tokens", "linear", "linear", "experts", "experts", "dispatch", "combine"])
    t = rng.choice([BF16, BF16, F32])
    if op == "tokens":
        c = 16 * _log(rng, 1, 1088)
        return {"op": op, "n": min(_log(rng, 1, 8192), 33_000_000 // c), "c": c, "type": t,
                "scale": rng.choice(["token", "tensor"])}
    if op == "linear":
        c, m = 32 * _log(rng, 1, 544), _log(rng, 1, 12288)
        n = min(_log(rng, 1, 8192), max(1, 400_000_000_000 // (c * m)))
        return {"op": op, "n": n, "c": c, "m": m, "type": t, "scale": rng.choice(["token", "tensor"])}
    k = rng.choice([1, 2, 3, 4, 6, 8])
    e = max(k, _log(rng, 4, 96))
    n = min(_log(rng, 1, 16384), 32768 // k)
    if op == "experts":
        c, m = 32 * _log(rng, 2, 96), _log(rng, 16, 2048)
        return {"op": op, "n": n, "k": k, "e": e, "c": c, "m": m, "type": t}
    c = _log(rng, 8, 2048) if op == "dispatch" else _log(rng, 8, 1536)
    case = {"op": op, "n": n, "k": k, "e": e, "c": c, "type": t}
    if op == "combine":
        case["grad"] = rng.choice([True, False])
    return case


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _pitch(c, t):
    """Columns of a buffer whose rows are 16-byte aligned."""
    per = 8 if t == BF16 else 4
    return -(-c // per) * per


def _buffer(rows, c, t):
    return torch.empty(rows, _pitch(c, t), dtype=TYPES[t], device=DEV)


def _activations(n, c, t, gen):
    """N(0,1) times one lognormal factor per channel: the spread that calibration meets."""
    x = torch.randn(n, c, generator=gen, device=DEV)
    x *= torch.randn(c, generator=gen, device=DEV).mul_(0.7).exp_()
    b = _buffer(n, c, t)
    b.zero_()
    b[:, :c] = x
    return b


def _weights(mats, m, c, gen):
    """Gaussian weights in packed NVFP4 by max scaling: codes two to a byte (even column in the low nibble), E4M3
    bytes [mats, m, c/16], the same bytes in the products' tile order, and one global scale per matrix."""
    w = torch.randn(mats, m, c, generator=gen, device=DEV).mul_(0.02)
    v, g = _block_scales(w, w.abs().amax((1, 2)).view(mats, 1))
    q = _e2m1(w, v, g)
    del w
    mag = q.abs()
    code = torch.where(mag <= 2, mag * 2, mag + 2 - (mag == 6).float()).to(torch.uint8)
    code |= torch.signbit(q).to(torch.uint8) << 3
    packed = (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous()
    scales = v.to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
    return {"packed": packed, "scales": scales, "tiled": _tiled(scales), "g": g.view(mats).contiguous()}


def _tiled(scales):
    """Scale bytes [mats, m, J] in tiles of 128 rows x 4 blocks: byte (r, j) of a matrix at tile (r/128, j/4), offset
    16 (r%32) + 4 (r%128/32) + j%4; rows and blocks past the matrix are 0."""
    mats, m, J = scales.shape
    R, K = -(-m // 128), -(-J // 4)
    p = torch.zeros(mats, R * 128, K * 4, dtype=torch.uint8, device=scales.device)
    p[:, :m, :J] = scales
    return p.view(mats, R, 4, 32, K, 4).permute(0, 1, 4, 3, 2, 5).contiguous()


def _routing(n, k, e, gen):
    """k distinct experts per token, expert i drawn in proportion to 1 / (i + 1)^1.1, and weights that sum to 1."""
    logp = torch.arange(1, e + 1, device=DEV, dtype=torch.float32).log_().mul_(-1.1)
    noise = -(-torch.rand(n, e, generator=gen, device=DEV).clamp_(1e-20, 1 - 1e-7).log_()).log_()
    top = (logp + noise).topk(k, dim=1).indices
    w = torch.randn(n, k, generator=gen, device=DEV).softmax(1)
    return top.to(torch.int32).contiguous(), w.contiguous()


def _sorted(ids, e):
    """Stable order of the flat ids by expert: order (flat index of each sorted row), its inverse, the offsets."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(flat.numel(), device=flat.device)
    off = torch.zeros(e + 1, dtype=torch.int64, device=flat.device)
    off[1:] = torch.bincount(flat, minlength=e).cumsum(0)
    return order.to(torch.int32), pos.to(torch.int32), off


def _token_workspace(rows, c, groups):
    """Codes, scale tiles and scales of the quantised tokens, each part rounded up to 256 bytes."""
    up = lambda b: -(-b // 256) * 256  # noqa: E731
    need = up(rows * c // 2) + up((rows // 128 + groups) * -(-c // 64) * 512) + up(rows * 4)
    return torch.empty(need, dtype=torch.uint8, device=DEV)


def prepare(case, seed):
    gen = _generator(seed)
    op, n, c, t = case["op"], case["n"], case["c"], case["type"]
    s = {"case": case}
    if op == "tokens":
        s["x"] = _activations(n, c, t, gen)
        s["amax"] = s["x"].float().abs().amax().view(1) if case["scale"] == "tensor" else None
        s["packed"] = torch.empty(n, c // 2, dtype=torch.uint8, device=DEV)
        s["tiles"] = torch.empty((n // 128 + 1) * -(-c // 64) * 512, dtype=torch.uint8, device=DEV)
        s["g"] = torch.empty(n, dtype=torch.float32, device=DEV)
        s["values"] = torch.empty(n, c, dtype=TYPES[t], device=DEV)
    elif op == "linear":
        s["x"] = _activations(n, c, t, gen)
        s["amax"] = s["x"].float().abs().amax().view(1) if case["scale"] == "tensor" else None
        s["w"] = _weights(1, case["m"], c, gen)
        s["y"] = _buffer(n, case["m"], t)
        s["ws"] = _token_workspace(n, c, 1)
    elif op == "experts":
        s["x"] = _activations(n, c, t, gen)
        ids, _ = _routing(n, case["k"], case["e"], gen)
        s["order"], _, s["offsets"] = _sorted(ids, case["e"])
        s["w"] = _weights(case["e"], case["m"], c, gen)
        s["y"] = _buffer(n * case["k"], case["m"], t)
        s["ws"] = _token_workspace(n * case["k"], c, case["e"])
    elif op == "dispatch":
        rows = n * case["k"]
        s["x"] = _activations(n, c, t, gen)
        s["ids"], _ = _routing(n, case["k"], case["e"], gen)
        s["offsets"] = torch.empty(case["e"] + 1, dtype=torch.int64, device=DEV)
        s["order"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        s["pos"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        s["rows"] = _buffer(rows, c, t)
    else:
        rows = n * case["k"]
        ids, s["weights"] = _routing(n, case["k"], case["e"], gen)
        _, s["pos"], _ = _sorted(ids, case["e"])
        s["rows"] = _activations(rows, c, t, gen)
        s["y"] = _buffer(n, c, t)
        if case["grad"]:
            s["dy"] = _activations(n, c, t, gen)
            s["drows"] = _buffer(rows, c, t)
            s["dweights"] = torch.empty(n, case["k"], dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- the plain form


def _over(a, d):
    """a / d with the IEEE quotient (a Python number as the divisor would be turned into a factor)."""
    return a / torch.full((), d, dtype=a.dtype, device=a.device)


def _block_scales(x, amax):
    """(v [..., J], g [..., 1]): the E4M3 values of the blocks' scales and the global scale, from amax [..., 1]."""
    g = _over(amax, 2688.0)
    a = x.unflatten(-1, (-1, 16)).abs().amax(-1)
    ge = g.unsqueeze(-1) if g.dim() < a.dim() else g
    v = (_over(a, 6.0) / ge).clamp_(max=448.0).to(torch.float8_e4m3fn).float()
    return torch.where(v >= 2.0 ** -9, v, torch.full_like(v, 2.0 ** -9)), g


def _e2m1(x, v, g):
    """q [..., c]: x over its block's scale, rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even
    code."""
    ge = g.unsqueeze(-1) if g.dim() < v.dim() else g
    s = (v * ge).unsqueeze(-1)
    u = x.unflatten(-1, (-1, 16)) / s
    u = torch.where(s == 0, torch.zeros_like(u), u)
    a = u.abs()
    q = ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) * 0.5
    q += (a > 2.5).float() + (a >= 3.5) + (a > 5.0).float() * 2
    return torch.copysign(q, u).flatten(-2)


def _token_values(x, amax):
    """(values [n, c], g [n]) of tokens x [n, c] in 32 bits."""
    x = x.float()
    a = amax.expand(x.shape[0], 1) if amax is not None else x.abs().amax(-1, keepdim=True)
    v, g = _block_scales(x, a)
    q = _e2m1(x, v, g)
    return (q.unflatten(-1, (-1, 16)) * (v * g).unsqueeze(-1)).flatten(-2), g.reshape(-1)


def _weight_values(w, m):
    """Matrix m's weights [rows, c] in 32 bits from their codes."""
    b = w["packed"][m]
    code = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    mag = (code & 7).float()
    mag = torch.where(mag <= 4, mag * 0.5, mag - 2 + (mag == 7).float())
    q = torch.where(code >= 8, -mag, mag)
    s = w["scales"][m].view(torch.float8_e4m3fn).float() * w["g"][m]
    return (q.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _run_plain(s):
    case = s["case"]
    op, n, c, t = case["op"], case["n"], case["c"], TYPES[case["type"]]
    if op == "tokens":
        values, g = _token_values(s["x"][:, :c], s["amax"])
        return {"values": values.to(t), "g": g}
    if op == "linear":
        values, _ = _token_values(s["x"][:, :c], s["amax"])
        return {"y": (values @ _weight_values(s["w"], 0).t()).to(t)}
    if op == "experts":
        values, _ = _token_values(s["x"][:, :c], None)
        values = values[s["order"].long() // case["k"]]
        edges = s["offsets"].tolist()
        # one product per expert: the rows of an expert are its own, and padding all to the longest would multiply
        # mostly zeros
        parts = [values[a:b] @ _weight_values(s["w"], i).t() for i, (a, b) in enumerate(zip(edges, edges[1:])) if b > a]
        return {"y": torch.cat(parts).to(t)}
    if op == "dispatch":
        order, pos, off = _sorted(s["ids"], case["e"])
        return {"order": order, "pos": pos, "offsets": off, "rows": s["x"][order.long() // case["k"], :c]}
    rows = s["rows"][:, :c].float()[s["pos"].long()].view(n, case["k"], c)
    out = {"y": (rows * s["weights"].unsqueeze(-1)).sum(1).to(t)}
    if case["grad"]:
        dy = s["dy"][:, :c].float()
        d = torch.empty(n * case["k"], c, device=DEV)
        d[s["pos"].long()] = (dy.unsqueeze(1) * s["weights"].unsqueeze(-1)).view(-1, c)
        out["drows"] = d.to(t)
        out["dweights"] = (rows * dy.unsqueeze(1)).sum(-1)
    return out


# ---------------------------------------------------------------- the library's calls


def _run_own(s):
    import scale_calibration_b200 as lh
    case = s["case"]
    op, n, c = case["op"], case["n"], case["c"]
    if op == "tokens":
        x = s["x"]
        lh.lh_quantize_tokens(x, x, n, c, x.stride(0), None, 1, n, None, 1, s["amax"], s["packed"], s["tiles"], s["g"],
                              s["values"], s["values"])
        return {"values": s["values"], "g": s["g"]}
    if op == "linear":
        x, w, y = s["x"], s["w"], s["y"]
        lh.lh_nvfp4_linear(x, x, n, c, x.stride(0), None, 1, n, None, 1, s["amax"], w["packed"], w["tiled"], w["g"],
                           case["m"], y, y, y.stride(0), s["ws"], s["ws"].numel())
        return {"y": y[:, :case["m"]]}
    if op == "experts":
        x, w, y = s["x"], s["w"], s["y"]
        lh.lh_nvfp4_linear(x, x, n, c, x.stride(0), s["order"], case["k"], n * case["k"], s["offsets"], case["e"], None,
                           w["packed"], w["tiled"], w["g"], case["m"], y, y, y.stride(0), s["ws"], s["ws"].numel())
        return {"y": y[:, :case["m"]]}
    if op == "dispatch":
        x, rows, k = s["x"], s["rows"], case["k"]
        lh.lh_route_tokens(s["ids"], n, k, case["e"], s["offsets"], s["order"], s["pos"])
        lh.lh_gather_tokens(x, x, n, c, x.stride(0), s["order"], k, n * k, rows, rows.stride(0))
        return {"order": s["order"], "pos": s["pos"], "offsets": s["offsets"], "rows": rows[:, :c]}
    rows, y, k = s["rows"], s["y"], case["k"]
    lh.lh_combine_tokens(rows, rows, n * k, c, rows.stride(0), s["pos"], s["weights"], n, k, y, y.stride(0))
    out = {"y": y[:, :c]}
    if case["grad"]:
        dy, d = s["dy"], s["drows"]
        lh.lh_combine_tokens_grad(dy, dy, n, k, c, dy.stride(0), rows, rows.stride(0), n * k, s["pos"], s["weights"], d,
                                  d.stride(0), s["dweights"])
        out["drows"], out["dweights"] = d[:, :c], s["dweights"]
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without


def _active(case):
    """Experts that get a row: rows are drawn in proportion to 1 / (i + 1)^1.1."""
    p = [(i + 1) ** -1.1 for i in range(case["e"])]
    total, rows = sum(p), case["n"] * case["k"]
    return sum(1 - (1 - x / total) ** rows for x in p)


def work(case):
    op, n, c = case["op"], case["n"], case["c"]
    eb = 2 if case["type"] == BF16 else 4
    if op == "tokens":
        return {"bytes": n * c * (2 * eb + 0.5 + 1 / 16) + 4 * n, "flops": 0}
    if op in ("linear", "experts"):
        rows = n * case.get("k", 1)
        mats = _active(case) if op == "experts" else 1
        m = case["m"]
        b = n * c * eb + mats * m * c * (0.5 + 1 / 16) + rows * m * eb + (4 * rows + 8 * case["e"] if op == "experts" else 0)
        return {"bytes": b, "flops": 2 * rows * m * c}
    k = case["k"]
    if op == "dispatch":
        return {"bytes": 12 * n * k + 8 * case["e"] + n * c * eb + n * k * c * eb, "flops": 0}
    b = n * k * c * eb + 8 * n * k + n * c * eb
    f = 2 * n * k * c
    if case["grad"]:
        b += n * c * eb + n * k * c * eb + 4 * n * k  # the rows are read once for both directions
        f += 3 * n * k * c
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the definition in 64 bits


def _rounded(x):
    """x (64 bits) rounded once to 32 bits, as 64 bits."""
    return x.to(torch.float32).double()


def _exact_tokens(x, amax):
    """The definition with each of its 32-bit roundings made from a 64-bit result (a quotient or product of two 32-bit
    numbers in 64 bits rounds to 32 as the exact one does)."""
    n, c = x.shape
    b = x.double().reshape(n, c // 16, 16)
    peak = b.abs().max(-1).values
    top = peak.max(-1).values if amax is None else amax.double().expand(n)
    g = _rounded(top / 2688.0)
    r = _rounded(_rounded(peak / 6.0) / g[:, None])
    r = torch.nan_to_num(r, nan=0.0, posinf=448.0).clamp(0.0, 448.0)
    # E4M3: steps of 2^-9 below 2^-6, three mantissa bits above; torch.round takes ties to even
    step = torch.exp2(torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3)
    v = (torch.round(r / step) * step).clamp(2.0 ** -9, 448.0)
    s = _rounded(v * g[:, None])[..., None]
    u = torch.where(s > 0, _rounded(b / s), torch.zeros_like(b)).clamp(-6.0, 6.0)
    # E2M1: steps of .5 below 2, then one mantissa bit
    half = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=1.0))) - 1)
    q = torch.round(u / half) * half
    return _rounded(q * s).reshape(n, c), g


def _exact_weights(w, i):
    b = w["packed"][i].long()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=b.device)
    table = torch.cat([table, -table])
    q = torch.empty(b.shape[0], 2 * b.shape[1], dtype=torch.float64, device=b.device)
    q[:, 0::2], q[:, 1::2] = table[b & 15], table[b >> 4]
    v = w["scales"][i].long()
    e, f = v >> 3, (v & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).double()))
    return q * (v * w["g"][i].double()).repeat_interleave(16, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, n, c = case["op"], case["n"], case["c"]
    if op == "tokens":
        values, g = _exact_tokens(s["x"][:, :c], s["amax"])
        return {"values": values, "g": g}
    if op == "linear":
        values, _ = _exact_tokens(s["x"][:, :c], s["amax"])
        return {"y": values @ _exact_weights(s["w"], 0).t()}
    if op == "experts":
        values, _ = _exact_tokens(s["x"][:, :c], None)
        token = s["order"].long() // case["k"]
        off = s["offsets"].tolist()
        y = torch.zeros(n * case["k"], case["m"], dtype=torch.float64, device=DEV)
        for i in range(case["e"]):
            if off[i + 1] > off[i]:
                y[off[i]:off[i + 1]] = values[token[off[i]:off[i + 1]]] @ _exact_weights(s["w"], i).t()
        return {"y": y}
    if op == "dispatch":
        flat = s["ids"].reshape(-1).long()
        first = torch.sort(flat * flat.numel() + torch.arange(flat.numel(), device=DEV)).values % flat.numel()
        return {"order": None, "pos": None, "offsets": None, "rows": s["x"].double()[first // case["k"], :c]}
    w, rows, pos = s["weights"].double(), s["rows"][:, :c].double(), s["pos"].long().view(n, case["k"])
    y = torch.zeros(n, c, dtype=torch.float64, device=DEV)
    for j in range(case["k"]):
        y += w[:, j:j + 1] * rows[pos[:, j]]
    out = {"y": y}
    if case["grad"]:
        dy = s["dy"][:, :c].double()
        d, dw = torch.empty_like(rows), torch.empty_like(w)
        for j in range(case["k"]):
            d[pos[:, j]] = w[:, j:j + 1] * dy
            dw[:, j] = (dy * rows[pos[:, j]]).sum(1)
        out["drows"], out["dweights"] = d, dw
    return out
