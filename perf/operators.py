"""Timed operators: microscaled 4-bit quantisation, the expert feed-forward on
microscaled 4-bit weights, and the whole block for a few tokens.

The microscaled 4-bit format ("mx4"): blocks of 32 consecutive values along a
row share one power-of-two scale 2^(b - 127) (one byte b), each value is a
4-bit code with one sign, two exponent and one mantissa bit (0, 0.5, 1, 1.5, 2,
3, 4, 6 and their negatives), two codes per byte, the lower-indexed value in the
low half.  The scale bytes of 128 rows x 128 columns are stored together: 512
bytes, byte (r % 32) * 16 + (r / 32) * 4 + (c / 32) for row r and column c of
that tile; tiles run along the columns, then down the rows.

`own` False computes the plain form in elementary torch operations; `own` True
calls the library.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # quantise a matrix and read it back: one token batch of hidden states
        {"name": "quantize_token_batch", "op": "quantize", "batch": 1, "rows": 16, "cols": 2048, "dtype": "bf16"},
        # rows and columns that fill no whole 128 x 128 scale tile
        {"name": "quantize_ragged_f32", "op": "quantize", "batch": 3, "rows": 515, "cols": 1376, "dtype": "f32"},
        # one expert's gate matrix of the large block
        {"name": "quantize_expert_matrix", "op": "quantize", "batch": 1, "rows": 2048, "cols": 8192, "dtype": "bf16"},
        # every expert's down matrix of a block, as when weights are converted at load
        {"name": "quantize_expert_stack", "op": "quantize", "batch": 256, "rows": 2048, "cols": 512, "dtype": "bf16"},
        # a decode batch: most experts see zero to two rows
        {"name": "experts_decode_batch", "op": "experts", "T": 16, "d": 2048, "E": 256, "k": 8, "I": 512, "I_s": 512,
         "load": "even"},
        # strongly skewed loads, empty experts, no shared expert, odd tile counts
        {"name": "experts_skewed_ragged", "op": "experts", "T": 777, "d": 1408, "E": 40, "k": 3, "I": 640, "I_s": 0,
         "load": "zipf"},
        # prefill of the small block: about 128 rows an expert
        {"name": "experts_prefill", "op": "experts", "T": 4096, "d": 2048, "E": 256, "k": 8, "I": 512, "I_s": 512,
         "load": "even"},
        # the large block with 2048 tokens: about 40 rows an expert, every weight read once
        {"name": "experts_wide", "op": "experts", "T": 2048, "d": 8192, "E": 512, "k": 10, "I": 2048, "I_s": 2048,
         "load": "even"},
        # one token through the small block: latency
        {"name": "few_one_token_bf16", "op": "few", "T": 1, "d": 2048, "E": 256, "k": 8, "I": 512, "I_s": 512,
         "w": "bf16", "bias": False, "norm": False},
        # the largest few-token batch at widths that are only multiples of 8, with the norm, gate and bias
        {"name": "few_odd_widths_bf16", "op": "few", "T": 16, "d": 1000, "E": 24, "k": 3, "I": 328, "I_s": 200,
         "w": "bf16", "bias": True, "norm": True},
        # a few speculated tokens on block-scaled 8-bit weights
        {"name": "few_four_tokens_fp8", "op": "few", "T": 4, "d": 4096, "E": 64, "k": 6, "I": 1536, "I_s": 1536,
         "w": "fp8", "bias": False, "norm": True},
        # eight sequences decoding on the large block with 4-bit weights
        {"name": "few_eight_tokens_mx4", "op": "few", "T": 8, "d": 8192, "E": 512, "k": 10, "I": 2048, "I_s": 2048,
         "w": "mx4", "bias": False, "norm": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["quantize", "experts", "few"])
    if op == "quantize":
        return {"op": op, "batch": _log(rng, 1, 64), "rows": _log(rng, 1, 4096), "cols": 32 * _log(rng, 1, 256),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "experts":
        E = _log(rng, 4, 256)
        I = 128 * _log(rng, 1, 16)
        return {"op": op, "T": _log(rng, 1, 4096), "d": 128 * _log(rng, 1, 64), "E": E,
                "k": rng.randint(1, min(E, 10)), "I": I, "I_s": rng.choice([0, I, 128 * _log(rng, 1, 16)]),
                "load": rng.choice(["even", "zipf"])}
    w = rng.choice(["bf16", "fp8", "mx4"])
    q = 8 if w == "bf16" else 128
    E = _log(rng, 4, 256)
    d, I = q * _log(rng, 128 // q, 8192 // q), q * _log(rng, 128 // q, 2048 // q)
    return {"op": op, "T": rng.randint(1, 16), "d": d, "E": E, "k": rng.randint(1, min(E, 10)), "I": I,
            "I_s": rng.choice([0, I, q * _log(rng, 128 // q, 2048 // q)]), "w": w, "bias": rng.random() < 0.5,
            "norm": rng.random() < 0.5}


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    while True:
        c = _draw(rng)
        if _cost(c) <= top[c["op"]] and _weight_bytes(c) <= 8e9:
            return c


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.5e12, w["flops"] / 1.6e15)


def _weight_bytes(case):
    if case["op"] == "quantize":
        return 0
    per = {"bf16": 2.0, "fp8": 1.0, "mx4": 17 / 32}[case.get("w", "mx4")]
    return 3 * case["d"] * (case["E"] * case["I"] + case["I_s"]) * per


def work(case):
    """Bytes and operations one pass cannot do without."""
    if case["op"] == "quantize":
        n = case["batch"] * case["rows"] * case["cols"]
        # read the values, write codes and scales; read those, write the values back in bf16
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 2 * (n // 2 + n // 32) + 2 * n, "flops": 4 * n}
    T, d, E, k, I, I_s = (case[n] for n in ("T", "d", "E", "k", "I", "I_s"))
    active = E * (1.0 - (1.0 - k / E) ** T)
    if case.get("load") == "zipf":
        active = sum(1.0 - (1.0 - p) ** (T * k) for p in _shares(E, "zipf"))
    per = {"bf16": 2.0, "fp8": 1.0 + 4.0 / 16384, "mx4": 17 / 32}[case.get("w", "mx4")]
    weights = 3 * d * (active * I + I_s) * per
    flops = 6 * d * T * (k * I + I_s)
    if case["op"] == "experts":
        rows = T * k + (T if I_s else 0)
        return {"bytes": int(weights + 4 * rows * d), "flops": flops}
    return {"bytes": int(weights + 2 * E * d + 4 * T * d + 8 * T * k), "flops": flops + 2 * T * d * E}


def _shares(E, load):
    p = [(e + 1.0) ** -1.1 if load == "zipf" else 1.0 for e in range(E)]
    return [v / sum(p) for v in p]


# ------------------------------------------------------------------ the format, plainly
def _tiles(s):
    """Scale bytes [..., R, C/32] -> tiles of 128 x 128 values, flattened per matrix."""
    *lead, R, C = s.shape
    Rp, Cp = -(-R // 128) * 128, -(-C // 4) * 4
    p = torch.full((*lead, Rp, Cp), 127, dtype=torch.uint8, device=s.device)
    p[..., :R, :C] = s
    p = p.reshape(*lead, Rp // 128, 4, 32, Cp // 4, 4)
    n = len(lead)
    return p.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4).reshape(*lead, -1)


def _rows_of_tiles(t, R, K, dtype=torch.float32):
    """Scale tiles [..., n] of matrices [R, K] (multiples of 128) -> the scales [..., R, K/32]."""
    lead = t.shape[:-1]
    n = len(lead)
    b = t.reshape(*lead, R // 128, K // 128, 32, 4, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return torch.exp2(b.reshape(*lead, R, K // 32).to(dtype) - 127)


def _values(codes, scales, dtype=torch.float32):
    """Packed codes [..., R, K/2] and scales [..., R, K/32] -> values [..., R, K]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    q = torch.stack([codes & 15, codes >> 4], -1).int()
    v = table[q].reshape(*codes.shape[:-1], -1, 32)
    return (v * scales[..., None]).flatten(-2)


def _quantize(x):
    """x [..., R, C] -> (packed codes [..., R, C/2], scale bytes [..., R, C/32]); ties to the even code."""
    v = x.float().unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 1 - 2).clamp(-127, 125)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    a = torch.ldexp(v.abs(), -e)
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5).int())
    c = (c + 8 * torch.signbit(v).int()).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), (e[..., 0] + 127).to(torch.uint8)


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _weight(gen, shape, w):
    """One weight tensor N(0, 0.02^2) -> (weights, scales or None), a few experts at a time."""
    if w == "bf16":
        out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        for i in range(shape[0]):
            out[i] = _normal(gen, shape[1:], 0.02, torch.bfloat16)
        return out, None
    qs, ss = [], []
    for _ in range(shape[0]):
        t = _normal(gen, shape[1:], 0.02, torch.float32)
        if w == "mx4":
            q, s = _quantize(t)
            ss.append(_tiles(s))
        else:
            R, K = t.shape
            b = t.reshape(R // 128, 128, K // 128, 128)
            s = b.abs().amax((1, 3)) / 448.0
            q = (b / s[:, None, :, None]).reshape(R, K).clamp(-448, 448).to(torch.float8_e4m3fn)
            ss.append(s.reshape(-1))
        qs.append(q)
    return torch.stack(qs), torch.stack(ss)


def _weights(gen, case, w):
    E, d, I, I_s = case["E"], case["d"], case["I"], case["I_s"]
    st, sc = {}, []
    shapes = {"wg": (E, I, d), "wu": (E, I, d), "wd": (E, d, I)}
    if I_s:
        shapes.update(s_wg=(1, I_s, d), s_wu=(1, I_s, d), s_wd=(1, d, I_s))
    for name, shape in shapes.items():
        t, s = _weight(gen, shape, w)
        st[name] = t if shape[0] == E and not name.startswith("s_") else t[0]
        if s is not None:
            sc.append(s.reshape(-1))
    for name in ("s_wg", "s_wu", "s_wd"):
        st.setdefault(name, None)
    st["scales"] = torch.cat(sc) if sc else None
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1009 * seed + 17)
    st = {"case": case}
    if case["op"] == "quantize":
        shape = (case["batch"], case["rows"], case["cols"])
        st["x"] = _normal(gen, shape, 0.02, DT[case["dtype"]])
    elif case["op"] == "experts":
        T, E, k = case["T"], case["E"], case["k"]
        st.update(_weights(gen, case, "mx4"))
        # k distinct experts a token, drawn by the load's shares
        keys = -torch.log(torch.rand((T, E), generator=gen, device="cuda")) / torch.tensor(
            _shares(E, case["load"]), device="cuda")
        ids = keys.argsort(1)[:, :k].reshape(-1)
        counts = torch.bincount(ids, minlength=E).tolist()
        order = torch.sort(ids, stable=True).indices // k
        sizes = counts + ([T] if case["I_s"] else [0])
        if case["I_s"]:
            order = torch.cat([order, torch.arange(T, device="cuda")])
        st["x_perm"] = _normal(gen, (T, case["d"]), 1.0, torch.bfloat16)[order]
        st["sizes"] = sizes
        st["offs"] = torch.tensor([sum(sizes[:i]) for i in range(E + 2)], dtype=torch.int32, device="cuda")
    else:
        T, d, E = case["T"], case["d"], case["E"]
        st["x"] = _normal(gen, (T, d), 1.0, torch.bfloat16)
        st["w_router"] = _normal(gen, (E, d), 0.02, torch.bfloat16)
        st["bias"] = _normal(gen, (E,), 0.5, torch.float32) if case["bias"] else None
        st["norm"] = _normal(gen, (d,), 0.1, torch.bfloat16) if case["norm"] else None
        st["gate"] = _normal(gen, (d,), 0.02, torch.bfloat16) if case["norm"] and case["I_s"] else None
        st.update(_weights(gen, case, case["w"]))
    if own:
        import sparse_moe_layer_top_b200 as moe
        if case["op"] != "quantize":
            p = st["prob"] = moe.Problem.make(case["T"], case["d"], case["E"], case["k"], case["I"], case["I_s"],
                                              "bf16", case.get("w", "mx4"))
            n = moe.stage_workspace_size(p) if case["op"] == "experts" else moe.decode_workspace_size(p)
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "quantize":
        q, s = _quantize(st["x"])
        s = torch.exp2(s.float() - 127)
        return {"values": _values(q, s).to(torch.bfloat16)}
    if case["op"] == "experts":
        return {"y_perm": _experts(st, case, torch.float32).to(torch.bfloat16)}
    y, ids, w = _few(st, case)
    return {"y": y.to(torch.bfloat16), "topk_ids": ids.int(), "topk_w": w.float()}


def _run_own(st, case):
    import sparse_moe_layer_top_b200 as moe
    if case["op"] == "quantize":
        codes, scales = moe.quantize_mx4(st["x"])
        return {"values": moe.dequantize_mx4(codes, scales)}
    W = [st[n] for n in ("wg", "wu", "wd", "s_wg", "s_wu", "s_wd")]
    if case["op"] == "experts":
        return {"y_perm": moe.expert_ffn(st["prob"], st["x_perm"], st["offs"], *W, scales=st["scales"], ws=st["ws"])}
    ids = torch.empty((case["T"], case["k"]), dtype=torch.int32, device="cuda")
    tw = torch.empty((case["T"], case["k"]), dtype=torch.float32, device="cuda")
    y = moe.decode_forward(st["prob"], st["x"], st["w_router"], st["bias"], *W, scales=st["scales"],
                           norm_weight=st["norm"], shared_gate=st["gate"], topk_ids=ids, topk_w=tw, ws=st["ws"])
    return {"y": y, "topk_ids": ids, "topk_w": tw}


def _scale_parts(st, case):
    """The packed scale buffer, cut per matrix: gate, up, down [E, ...], shared gate, up, down [1, ...]."""
    E, d, I, I_s = case["E"], case["d"], case["I"], case["I_s"]
    unit = 32 if case.get("w", "mx4") == "mx4" else 16384
    sizes = [(E, I * d)] * 3 + ([(1, I_s * d)] * 3 if I_s else [])
    parts = st["scales"].split([g * n // unit for g, n in sizes])
    return [p.reshape(g, -1) for p, (g, _) in zip(parts, sizes)]


def _dense(st, case, parts, i, pick, dtype):
    """Matrix i (gate, up, down, shared gate, up, down) as values; `pick` chooses experts."""
    name = ("wg", "wu", "wd", "s_wg", "s_wu", "s_wd")[i]
    w = st[name][pick] if i < 3 else st[name][None]
    kind = case.get("w", "mx4")
    if kind == "bf16":
        return w.to(dtype)
    if kind == "fp8":
        w = (st[name].view(torch.uint8)[pick] if i < 3 else st[name].view(torch.uint8)[None]).view(torch.float8_e4m3fn)
        s = parts[i][pick if i < 3 else slice(None)]
        G, R, K = w.shape
        b = w.to(dtype).reshape(G, R // 128, 128, K // 128, 128)
        return (b * s.to(dtype).reshape(G, R // 128, 1, K // 128, 1)).reshape(G, R, K)
    s = parts[i][pick if i < 3 else slice(None)]
    return _values(w, _rows_of_tiles(s, w.shape[1], 2 * w.shape[2], dtype), dtype)


def _experts(st, case, dtype):
    E, sizes = case["E"], st["sizes"]
    parts = _scale_parts(st, case)
    out, r = [], 0
    for g in range(E + 1):
        n = sizes[g]
        if n:
            o = 0 if g < E else 3
            pick = slice(g, g + 1)
            x = st["x_perm"][r:r + n].to(dtype)
            a = x @ _dense(st, case, parts, o, pick, dtype)[0].T
            b = x @ _dense(st, case, parts, o + 1, pick, dtype)[0].T
            h = a / (1 + torch.exp(-a)) * b
            out.append(h @ _dense(st, case, parts, o + 2, pick, dtype)[0].T)
        r += n
    return torch.cat(out)


def _few(st, case):
    T, k = case["T"], case["k"]
    x = st["x"].float()
    if st["norm"] is not None:
        x = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * (1 + st["norm"].float())
        x = x.to(torch.bfloat16).float()  # the normalised input is held in the activation type
    logits = x.double() @ st["w_router"].double().T
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    p, ids = torch.sort(torch.softmax(logits, 1), dim=1, descending=True, stable=True)
    p, ids = p[:, :k], ids[:, :k]
    w = (p / p.sum(1, keepdim=True)).float()
    parts = _scale_parts(st, case) if st["scales"] is not None else None
    ys = []
    for t in range(T):
        a = _dense(st, case, parts, 0, ids[t], torch.float32) @ x[t]
        b = _dense(st, case, parts, 1, ids[t], torch.float32) @ x[t]
        h = a / (1 + torch.exp(-a)) * b * w[t][:, None]
        ys.append((_dense(st, case, parts, 2, ids[t], torch.float32) @ h[:, :, None])[:, :, 0].sum(0))
    y = torch.stack(ys)
    if case["I_s"]:
        a = x @ _dense(st, case, parts, 3, None, torch.float32)[0].T
        b = x @ _dense(st, case, parts, 4, None, torch.float32)[0].T
        s = (a / (1 + torch.exp(-a)) * b) @ _dense(st, case, parts, 5, None, torch.float32)[0].T
        if st["gate"] is not None:
            s = s / (1 + torch.exp(-(x @ st["gate"].float())))[:, None]
        y = y + s
    return y, ids, w


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        v = st["x"].double().unflatten(-1, (-1, 32))
        amax = v.abs().amax(-1, keepdim=True)
        s = torch.exp2(torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)))) - 2)
        a = v.abs() / s
        # spacing of the 4-bit values around a: 0.5 below 2, 1 below 4, 2 above
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
        q = (torch.round(a / step) * step).clamp(max=6.0)
        return {"values": (torch.copysign(q, v) * s).flatten(-2)}
    kind = case.get("w", "mx4")
    E, d, I, I_s = case["E"], case["d"], case["I"], case["I_s"]
    at = {"o": 0}

    def matrices(name, R, K, G):
        """expert -> matrix [R, K] in 64 bits, consuming the scale buffer in its packed order"""
        t, o = st[name], at["o"]
        if kind == "bf16":
            return lambda e: (t[e] if G else t).double()
        n = (G or 1) * R * K // (32 if kind == "mx4" else 16384)
        sc = st["scales"][o:o + n].reshape(G or 1, -1)
        at["o"] = o + n
        if kind == "fp8":
            return lambda e: (t[e] if G else t).to(torch.float32).double() * sc[e].double().reshape(
                R // 128, K // 128).repeat_interleave(128, 0).repeat_interleave(128, 1)

        def dec(e):
            c = (t[e] if G else t).reshape(-1).long()
            c = torch.stack([c % 16, c // 16], 1).reshape(R, K)
            sign, ex, m = 1 - 2 * (c // 8), (c // 2) % 4, (c % 2).double()
            mag = torch.where(ex == 0, m * 0.5, (1 + 0.5 * m) * torch.exp2(ex.double() - 1))
            rr = torch.arange(R, device=c.device)[:, None]
            bb = torch.arange(K // 32, device=c.device)[None, :]
            pos = ((rr // 128) * (K // 128) + bb // 4) * 512 + (rr % 32) * 16 + (rr % 128) // 32 * 4 + bb % 4
            return sign * mag * torch.exp2(sc[e][pos].double() - 127).repeat_interleave(32, 1)
        return dec

    G_, U_, D_ = matrices("wg", I, d, E), matrices("wu", I, d, E), matrices("wd", d, I, E)
    sh = [matrices(n, *s, 0) for n, s in (("s_wg", (I_s, d)), ("s_wu", (I_s, d)), ("s_wd", (d, I_s)))] if I_s else None

    def ffn(x, f, e):
        g = x @ f[0](e).T
        return (g * torch.sigmoid(g) * (x @ f[1](e).T)) @ f[2](e).T

    if case["op"] == "experts":
        y = torch.empty((sum(st["sizes"]), d), dtype=torch.float64, device="cuda")
        r = 0
        for e, n in enumerate(st["sizes"]):
            if n:
                y[r:r + n] = ffn(st["x_perm"][r:r + n].double(), (G_, U_, D_) if e < E else sh, e if e < E else 0)
            r += n
        return {"y_perm": y}
    x = st["x"].double()
    if st["norm"] is not None:
        x = x * torch.rsqrt(x.pow(2).mean(1, keepdim=True) + 1e-6) * (1 + st["norm"].double())
        x = x.to(torch.bfloat16).double()
    l = x @ st["w_router"].double().T + (0 if st["bias"] is None else st["bias"].double())
    ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :case["k"]]
    w = torch.softmax(l.gather(1, ids), 1)
    y = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y[t] += w[t, j][:, None] * ffn(x[t], (G_, U_, D_), e)
    if I_s:
        g = torch.ones(case["T"], dtype=torch.float64, device="cuda")
        if st["gate"] is not None:
            g = torch.sigmoid(x @ st["gate"].double())
        y += g[:, None] * ffn(x, sh, 0)
    return {"y": y, "topk_ids": ids.int(), "topk_w": w}
