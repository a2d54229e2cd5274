"""What the operators around the attention of a decoder layer are measured on.

Three operators, each in its plain form (elementary torch operations) and, with ``own`` set, as the
framework's call:

* ``norm``   residual addition + RMSNorm, with a bf16 and an 8-bit output: ``add_rmsnorm``
* ``linear`` few tokens times an int4 affine matrix, with an unmerged LoRA: ``Int4Linear``
* ``moe``    a whole mixture-of-experts layer for few tokens: ``MoeLayer.few``
"""
import torch

own = False

EPS = 1e-6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn
Q_MAX = {"int8": 127.0, "e4m3": 448.0}


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------
def _norm(T, d, fmt, group, delta="bf16", x=True):
    return {"op": "norm", "T": T, "d": d, "fmt": fmt, "group": group, "delta": delta, "x": x}


def _linear(T, N, K, g=64, act="bf16", act_group=0, r=0, out="bf16"):
    return {"op": "linear", "T": T, "N": N, "K": K, "g": g, "act": act, "act_group": act_group, "r": r, "out": out}


def _moe(T, d, E, I, k, r, route=False, delta=True):
    return {"op": "moe", "T": T, "d": d, "E": E, "I": I, "k": k, "r": r, "route": route, "delta": delta}


def listed():
    cases = {
        # one decoded token before an 8-bit projection: nothing but latency
        "norm_t1": _norm(1, 2048, "e4m3", 64),
        # a batch of streams, one scale a token
        "norm_t64_int8": _norm(64, 4096, "int8", 0, x=False),
        # a short prompt of an odd width: the last group of each row is ragged; the MoE's fp32 output as the delta
        "norm_t517_odd": _norm(517, 1000, "e4m3", 64, delta="f32"),
        # a long prompt's chunk
        "norm_t16384": _norm(16384, 2048, "e4m3", 128),
        # one token through an attention output projection with its recovery LoRA
        "linear_t1_lora": _linear(1, 2048, 2048, r=16),
        # a batch of streams through a projection of queries, keys and values on 8-bit activations
        "linear_t8_int8": _linear(8, 5120, 2048, act="int8", act_group=64),
        # one token's logits over a vocabulary of odd size, kept in 32 bits
        "linear_t1_logits": _linear(1, 65521, 2048, g=128, out="f32"),
        # drafted tokens of several streams through a wide matrix
        "linear_t32_wide": _linear(32, 8192, 4096, act="e4m3", act_group=0),
        # the small layer of the tests, a ragged batch, its own router
        "moe_t5_small": _moe(5, 256, 16, 128, 4, 8),
        # one decoded token, routed by the prerouter's prediction
        "moe_t1": _moe(1, 2048, 256, 512, 4, 16, route=True),
        # a small batch of streams
        "moe_t8": _moe(8, 2048, 256, 512, 4, 16),
        # the largest batch
        "moe_t64": _moe(64, 2048, 256, 512, 4, 16),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["norm", "linear", "moe"])
    if op == "norm":
        d = _log(rng, 64, 8192)
        T = _log(rng, 1, min(16384, (1 << 25) // d))
        if rng.random() < 0.5:
            d = max(64, d // 64 * 64)
        fmt = rng.choice(["int8", "e4m3"])
        group = rng.choice([0, 64, 128]) if fmt == "e4m3" else rng.choice([0, 64] if d % 64 == 0 else [0])
        return _norm(T, d, fmt, group, rng.choice(["bf16", "f32", "none"]), rng.random() < 0.7)
    if op == "linear":
        g = rng.choice([64, 64, 128])
        K = g * _log(rng, 2, 8192 // g)
        N = _log(rng, 64, min(65536, (1 << 27) // K))
        T = _log(rng, 1, 32)
        act = rng.choice(["bf16", "bf16", "int8", "e4m3"])
        return _linear(T, N, K, g, act, rng.choice([0, 64, 128] if K % 128 == 0 else [0, 64]) if act != "bf16" else 0,
                       rng.choice([0, 0, 5, 16, 32]), rng.choice(["bf16", "f32"]))
    d = 256 * _log(rng, 1, 8)
    I = 128 * _log(rng, 1, max(1, (2048 * 512) // (128 * d)))
    E = _log(rng, 8, 256)
    return _moe(_log(rng, 1, 64), d, E, I, rng.choice([1, 2, 3, 4]), rng.choice([0, 7, 16]), rng.random() < 0.3,
                rng.random() < 0.7)


def work(c):
    T = c["T"]
    if c["op"] == "norm":
        d = c["d"]
        n = T * d
        groups = T * (-(-d // c["group"]) if c["group"] else 1)
        moved = 2 * n + {"bf16": 2, "f32": 4, "none": 0}[c["delta"]] * n + 2 * d  # h, delta, gamma
        moved += (2 * n if c["delta"] != "none" else 0) + (2 * n if c["x"] else 0) + n + 4 * groups  # h', x, 8 bits, scales
        return {"bytes": moved, "flops": 8 * n}
    if c["op"] == "linear":
        N, K, r = c["N"], c["K"], c["r"]
        x = T * K * 2 if c["act"] == "bf16" else T * K + 4 * T * (K // c["act_group"] if c["act_group"] else 1)
        moved = N * K // 2 + 4 * N * (K // c["g"]) + x + T * N * (2 if c["out"] == "bf16" else 4) + 2 * r * (N + K)
        return {"bytes": moved, "flops": 2 * T * (N * K + r * (N + K))}
    d, E, I, k, r = c["d"], c["E"], c["I"], c["k"], c["r"]
    blob = 3 * (I * d // 2 + 4 * I * (d // 64))
    distinct = E * (1 - (1 - k / E) ** T)  # expected number of experts that T tokens choose
    moved = (distinct + 1) * blob + 2 * d * E + 2 * d + 2 * r * 3 * (d + I)
    moved += T * d * (2 + (4 if c["delta"] else 0) + 2) + T * k * (4 + 4 + (4 if c["route"] else 0))
    return {"bytes": moved, "flops": 2 * T * ((k + 1) * 3 * I * d + E * d + 3 * r * (d + I))}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _sections(d, I):
    """Byte ranges of one expert's blob: gate, up and down, each codes | scale | min."""
    at, out = 0, {}
    for name, rows, cols in (("gate", I, d), ("up", I, d), ("down", d, I)):
        for part, size in (("codes", rows * cols // 2), ("scale", rows * cols // 32), ("min", rows * cols // 32)):
            out[name, part] = (at, at + size)
            at += size
    return out, at


def _scales(shape, gen):
    return (torch.rand(shape, generator=gen, device="cuda") * 0.015 + 0.005).to(BF16)


def _mins(shape, gen):
    return (torch.rand(shape, generator=gen, device="cuda") * 0.2 - 0.1).to(BF16)


def _blobs(n, d, I, gen):
    sections, size = _sections(d, I)
    blobs = torch.randint(0, 256, (n, size), dtype=torch.uint8, generator=gen, device="cuda")
    for (_, part), (a, b) in sections.items():
        if part != "codes":
            make = _scales if part == "scale" else _mins
            blobs[:, a:b] = make((n, (b - a) // 2), gen).view(torch.uint8)
    return blobs


def _normal(shape, gen, scale=1.0, dtype=BF16):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    c, T = case, case["T"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm":
        d = c["d"]
        # a residual stream: most channels of ordinary size, a few that stand out, tokens of different sizes
        channel = torch.where(torch.rand(d, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
        token = torch.exp(torch.randn((T, 1), generator=gen, device="cuda"))
        s["h"] = (torch.randn((T, d), generator=gen, device="cuda") * channel * token).to(BF16)
        s["delta"] = None if c["delta"] == "none" else _normal((T, d), gen, 0.5, BF16 if c["delta"] == "bf16" else F32)
        s["gamma"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(BF16)
        # the buffers that a serving loop keeps
        s["h_out"] = torch.empty((T, d), dtype=BF16, device="cuda") if s["delta"] is not None else None
        s["x"] = torch.empty((T, d), dtype=BF16, device="cuda") if c["x"] else None
        s["q8"] = torch.empty((T, d), dtype=torch.int8 if c["fmt"] == "int8" else E4M3, device="cuda")
        s["q8_scale"] = torch.empty((T, -(-d // c["group"]) if c["group"] else 1), dtype=F32, device="cuda")
    elif c["op"] == "linear":
        N, K, g, r = c["N"], c["K"], c["g"], c["r"]
        s["codes"] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=gen, device="cuda")
        s["scale"], s["min"] = _scales((N, K // g), gen), _mins((N, K // g), gen)
        s["lora_A"] = _normal((r, K), gen, K ** -0.5) if r else None
        s["lora_B"] = _normal((N, r), gen, 0.01) if r else None
        x = torch.randn((T, K), generator=gen, device="cuda")
        s["x_scale"] = None
        if c["act"] == "bf16":
            s["x"] = x.to(BF16)
        else:
            xg = x.view(T, -1, c["act_group"] or K)
            scale = xg.abs().amax(-1, keepdim=True) / Q_MAX[c["act"]]
            q = (xg / scale).view(T, K)
            s["x"] = q.round().to(torch.int8) if c["act"] == "int8" else q.to(E4M3)
            s["x_scale"] = scale.view(T, -1).contiguous()
        s["y"] = torch.empty((T, N), dtype=BF16 if c["out"] == "bf16" else F32, device="cuda")
        if own:  # the handle that a program makes once for its weights
            import int4_expert_streaming_prerouter_b200 as e0
            s["handle"] = e0.Int4Linear(s["codes"], s["scale"], s["min"], s["lora_A"], s["lora_B"], 1.0)
    else:
        d, E, I, k, r = c["d"], c["E"], c["I"], c["k"], c["r"]
        s["h"] = _normal((T, d), gen)
        s["delta"] = _normal((T, d), gen, 0.5) if c["delta"] else None
        layer = {"experts": _blobs(E, d, I, gen), "shared": _blobs(1, d, I, gen)[0],
                 "router_w": _normal((E, d), gen, 0.02), "norm_w": (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(BF16)}
        if r:
            layer |= {"lora_Ag": _normal((r, d), gen, d ** -0.5), "lora_Bg": _normal((I, r), gen, 0.01),
                      "lora_Au": _normal((r, d), gen, d ** -0.5), "lora_Bu": _normal((I, r), gen, 0.01),
                      "lora_Ad": _normal((r, I), gen, I ** -0.5), "lora_Bd": _normal((d, r), gen, 0.01)}
        s["layer"] = layer
        # predicted routing: k different experts a token
        s["route"] = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous() if c["route"] else None
        s["h_out"] = torch.empty((T, d), dtype=BF16, device="cuda") if c["delta"] else None
        s["y"] = torch.empty((T, d), dtype=BF16, device="cuda")
        s["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["gates"] = torch.empty((T, k), dtype=F32, device="cuda")
        if own:  # the handle that a program makes once for its weights, and its workspace
            import int4_expert_streaming_prerouter_b200 as e0
            s["handle"] = e0.MoeLayer(e0.make_dims(d, E, I, k, r, eps=EPS), layer)
            s["workspace"] = s["handle"].few_workspace(T)
    return s


# ---------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------
def _round_bf16(v):
    """A double (in the normal range) rounded once to bf16, ties to even, on its bits."""
    b = v.view(torch.int64)
    return ((b + ((1 << 44) - 1) + ((b >> 45) & 1)) & -(1 << 45)).view(F64).to(BF16)


def _add(h, delta):
    return h if delta is None else _round_bf16(h.double() + delta.double())


def _rms(h, gamma):
    v = h.double()  # in 64 bits: x is taken to the nearest bf16, and its 8-bit value from that
    return _round_bf16(v * gamma.double() / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS))


def _plain_norm(s, c):
    T, d = c["T"], c["d"]
    h = _add(s["h"], s["delta"])
    x = _rms(h, s["gamma"])
    group = c["group"] or d
    xg = torch.nn.functional.pad(x.float(), (0, -d % group)).view(T, -1, group)
    most = xg.abs().amax(-1).double()
    scale = (most / Q_MAX[c["fmt"]]).float()
    # x / (most / M) is written x M / most: a product without rounding, so that ties stay ties
    q = torch.where(most[..., None] > 0, xg.double() * Q_MAX[c["fmt"]] / most[..., None], 0.0)
    if c["fmt"] == "int8":
        return h, x, (q.round() * scale[..., None]).float().view(T, -1)[:, :d], scale
    # the spacing of e4m3 at |q|: three bits below the leading one, which is at 2^-6 at least
    lead = ((q.abs().view(torch.int64) >> 52) - 1023).clamp(min=-6)
    step = ((lead - 3 + 1023) << 52).view(F64)
    q = ((q / step).round() * step).clamp(-448, 448)
    return h, x, q.float().view(T, -1)[:, :d].to(E4M3), scale


def _dequant(codes, scale, mins, g):
    """codes [..., n, k / 2] u8, scale and min [..., n, k / g] -> [..., n, k] in 32 bits."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    q = q.view(*scale.shape, g) * scale.float()[..., None] + mins.float()[..., None]
    return q.flatten(-2)


def _plain_linear(s, c):
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = (x.view(*s["x_scale"].shape, -1) * s["x_scale"][..., None]).view(c["T"], -1)
    y = x @ _dequant(s["codes"], s["scale"], s["min"], c["g"]).T
    if s["lora_A"] is not None:
        y = y + (x @ s["lora_A"].float().T) @ s["lora_B"].float().T
    return y.to(s["y"].dtype)


def _plain_moe(s, c):
    T, d, I, k = c["T"], c["d"], c["I"], c["k"]
    w = s["layer"]
    h = _add(s["h"], s["delta"])
    x = _rms(h, w["norm_w"])
    logits = x.double() @ w["router_w"].double().T  # in 64 bits: near ties decide which experts run
    idx = s["route"].long() if s["route"] is not None else logits.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    chosen = logits.gather(1, idx).float()
    e = torch.exp(chosen - chosen.amax(-1, keepdim=True))
    gates = e / e.sum(-1, keepdim=True)
    xf = x.float()
    sections, _ = _sections(d, I)

    def matrix(blobs, name, rows, cols):
        part = lambda p: blobs[:, slice(*sections[name, p])].contiguous()  # noqa: E731
        scale, mins = (part(p).view(BF16).view(-1, rows, cols // 64) for p in ("scale", "min"))
        return _dequant(part("codes").view(-1, rows, cols // 2), scale, mins, 64)

    def expert(blobs, x, lora):
        """blobs [n, bytes], x [n, m, d] -> [n, m, d]"""
        g = x @ matrix(blobs, "gate", I, d).transpose(1, 2)
        u = x @ matrix(blobs, "up", I, d).transpose(1, 2)
        if lora:
            g = g + (x @ w["lora_Ag"].float().T) @ w["lora_Bg"].float().T
            u = u + (x @ w["lora_Au"].float().T) @ w["lora_Bu"].float().T
        a = (g / (1 + torch.exp(-g)) * u).to(BF16).float()
        y = a @ matrix(blobs, "down", d, I).transpose(1, 2)
        return y + (a @ w["lora_Ad"].float().T) @ w["lora_Bd"].float().T if lora else y

    each = expert(w["experts"][idx.flatten()], xf.repeat_interleave(k, 0)[:, None], False).view(T, k, d)
    y = (each * gates[..., None]).sum(1) + expert(w["shared"][None], xf[None], c["r"] > 0)[0]
    return h, y.to(BF16), idx.to(torch.int32), gates


def run(state):
    s, c = state, state["case"]
    if c["op"] == "norm":
        if own:
            import int4_expert_streaming_prerouter_b200 as e0
            e0.add_rmsnorm(s["h"], s["gamma"], delta=s["delta"], eps=EPS, h_out=s["h_out"], x=s["x"], q8=s["q8"],
                           q8_scale=s["q8_scale"], q8_group=c["group"])
            h, x, q8, scale = s["h_out"], s["x"], s["q8"], s["q8_scale"]
            if c["fmt"] == "int8":  # the values that the codes stand for
                q8 = (q8.view(*scale.shape, -1) * scale[..., None]).view(c["T"], -1)
        else:
            h, x, q8, scale = _plain_norm(s, c)
        return {"h": h if s["delta"] is not None else None, "x": x if c["x"] else None, "q8": q8, "scale": scale}
    if c["op"] == "linear":
        return {"y": s["handle"](s["x"], x_scale=s["x_scale"], y=s["y"]) if own else _plain_linear(s, c)}
    if own:
        s["handle"].few(s["h"], delta=s["delta"], route_idx=s["route"], h_out=s["h_out"], y=s["y"], idx=s["idx"],
                        gates=s["gates"], workspace=s["workspace"])
        h, y, idx, gates = s["h_out"], s["y"], s["idx"], s["gates"]
    else:
        h, y, idx, gates = _plain_moe(s, c)
    return {"h": h if s["delta"] is not None else None, "y": y, "idx": idx, "gates": gates}


# ---------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _nearest(v, bits, least):
    """v in 64 bits, rounded to `bits` significant bits, ties to even; spacing at least 2^least."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - bits).clamp(min=least).double())
    return torch.round(v / step) * step


def _codes64(codes):
    """[n, k / 2] bytes -> [n, k] numbers, the low half of a byte first."""
    out = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=F64, device=codes.device)
    out[..., 0::2] = codes.remainder(16)
    out[..., 1::2] = codes.div(16, rounding_mode="floor")
    return out


def _matrix64(codes, scale, mins, g):
    wide = lambda v: v.double().repeat_interleave(g, -1)  # noqa: E731
    return wide(scale) * _codes64(codes) + wide(mins)


def _expert64(blob, x, d, I, lora):
    at, mats = 0, []
    for rows, cols in ((I, d), (I, d), (d, I)):
        n, m = rows * cols // 2, rows * cols // 32
        codes = blob[at:at + n].view(rows, cols // 2)
        scale, mins = (blob[o:o + m].clone().view(BF16).view(rows, -1) for o in (at + n, at + n + m))
        mats.append(_matrix64(codes, scale, mins, 64))
        at += n + 2 * m
    g, u = x @ mats[0].T, x @ mats[1].T
    if lora is not None:
        g, u = g + lora["Bg"] @ (lora["Ag"] @ x), u + lora["Bu"] @ (lora["Au"] @ x)
    a = _nearest(g * torch.sigmoid(g) * u, 8, -133)
    y = mats[2] @ a
    return y if lora is None else y + lora["Bd"] @ (lora["Ad"] @ a)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        x = s["x"].double()
        if s["x_scale"] is not None:
            x = x * s["x_scale"].double().repeat_interleave(c["K"] // s["x_scale"].shape[1], 1)
        y = torch.cat([x @ _matrix64(*(s[n][i:i + 4096] for n in ("codes", "scale", "min")), c["g"]).T
                       for i in range(0, c["N"], 4096)], 1)
        if c["r"]:
            y += x @ s["lora_A"].double().T @ s["lora_B"].double().T
        return {"y": y}
    gamma = s["gamma"] if c["op"] == "norm" else s["layer"]["norm_w"]
    total = s["h"].double() + (s["delta"].double() if s["delta"] is not None else 0)
    h = _nearest(total, 8, -133)
    x = h * gamma.double() / ((h ** 2).sum(1, keepdim=True) / c["d"] + EPS) ** 0.5
    xr = _nearest(x, 8, -133)
    if c["op"] == "norm":
        scales, values = [], []
        for i in range(0, c["d"], c["group"] or c["d"]):
            part = xr[:, i:i + (c["group"] or c["d"])]
            most, top = part.abs().amax(1, keepdim=True), Q_MAX[c["fmt"]]
            q = torch.where(most > 0, top * part / most, 0.0)
            values.append(torch.round(q) * (most / top) if c["fmt"] == "int8" else _nearest(q, 4, -9).clamp(-448, 448))
            scales.append(most / top)
        return {"h": total if s["delta"] is not None else None, "x": x if c["x"] else None, "q8": torch.cat(values, 1),
                "scale": torch.cat(scales, 1)}
    w, k = s["layer"], c["k"]
    logits = (w["router_w"].double() @ xr.T).T
    idx = s["route"].long() if s["route"] is not None else torch.argsort(-logits, dim=1, stable=True)[:, :k]
    gates = torch.softmax(logits.gather(1, idx), 1)
    lora = {n[5:]: v.double() for n, v in w.items() if n.startswith("lora_")} or None
    y = torch.stack([_expert64(w["shared"], v, c["d"], c["I"], lora) for v in xr])
    for t in range(c["T"]):
        for j, e in enumerate(idx[t].tolist()):
            y[t] += gates[t, j] * _expert64(w["experts"][e], xr[t], c["d"], c["I"], None)
    return {"h": total if s["delta"] is not None else None, "y": y, "idx": idx.to(torch.int32), "gates": gates}
