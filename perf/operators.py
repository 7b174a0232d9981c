"""Operators for a few tokens and for 4-bit weights: their cases, plain forms and floors.

Four operators of the package, each in two forms. The plain form is elementary torch; the
other (``own`` true) makes the calls that a user's program makes:

* ``few``     moe_layer_forward_few: the whole MoE layer for 1 to 8 tokens, bf16 experts
* ``few_w4``  moe_layer_forward_few_w4: the same layer on 4-bit routed experts
* ``matvec``  moe_matvec_w4: y = x W^T for 1 to 16 rows of x, W in 4-bit groups
* ``quant``   moe_quantize_w4 and moe_dequantize_w4: a matrix to 4-bit groups and back

The 4-bit format: group g of ``group`` consecutive elements of a row has a bf16 scale
s = bf16(amax_g / 7) and codes c = clamp(round_half_even(w / s), -8, 7) + 8, standing for
(c - 8) s. A row is stored in blocks of 128 elements = 64 bytes: element 32 j + 8 t + i of a
block (j, t < 4, i < 8) is nibble (i >> 1) + 4 (i & 1) of the little-endian 32-bit word
4 t + j; elements behind the row's end have code 8. Scales are padded to a multiple of 8 a row.
"""
import math

import torch

own = False

SIGMA_W = 0.02  # expert and router weights, as this repository's input generator draws them


# ------------------------------------------------------------------------------------ cases

def _layer(op, name, T, H, E, k, I, Is, bias=False, skew=0.0, group=0):
    c = dict(op=op, T=T, H=H, E=E, k=k, I=I, Is=Is, bias=bias, skew=skew)
    if group:
        c["group"] = group
    if name:
        c["name"] = name
    return c


def _matvec(name, T, N, K, group, x, y, pad=0):
    c = dict(op="matvec", T=T, N=N, K=K, group=group, x=x, y=y, pad=pad)
    if name:
        c["name"] = name
    return c


def _quant(name, rows, K, group, to):
    c = dict(op="quant", rows=rows, K=K, group=group, to=to)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the repository's tiny layer, one token: nothing but latency
        _layer("few", "few_tiny_t1", 1, 256, 16, 4, 128, 128),
        # one sequence decoding on the Flash-Next-shaped layer
        _layer("few", "few_flash_t1", 1, 2560, 512, 10, 640, 640),
        # eight sequences, or two with three drafted tokens each, on the same layer
        _layer("few", "few_flash_t8", 8, 2560, 512, 10, 640, 640, bias=True),
        # four tokens on the 2.4T-shaped layer with 64 experts, some of them popular
        _layer("few", "few_t24_e64_t4", 4, 8192, 64, 10, 2048, 2048, bias=True, skew=1.1),
        # one sequence decoding, 4-bit experts with a scale for each 32 weights
        _layer("few_w4", "few_w4_flash_t1", 1, 2560, 512, 10, 640, 640, group=32),
        # an odd batch with scales for 64 weights
        _layer("few_w4", "few_w4_flash_t5", 5, 2560, 512, 10, 640, 640, bias=True, group=64),
        # eight tokens on the 2.4T-shaped layer with 64 experts, scales for 128 weights
        _layer("few_w4", "few_w4_t24_e64_t8", 8, 8192, 64, 10, 2048, 2048, group=128),
        # one expert's down matrix and one token: the smallest product
        _matvec("matvec_t1_2560x640", 1, 2560, 640, 32, "bf16", "fp32"),
        # odd sizes, a ragged last group, rows with a stride
        _matvec("matvec_t5_4099x2501", 5, 4099, 2501, 64, "fp16", "fp16", pad=11),
        # an output head over a large vocabulary, sixteen rows
        _matvec("matvec_t16_65536x8192", 16, 65536, 8192, 128, "bf16", "bf16"),
        # load time: the gate|up matrices of 32 Flash-Next-shaped experts
        _quant("quant_flash_40960x2560", 40960, 2560, 32, "fp32"),
        # load time: the down matrices of 16 2.4T-shaped experts, read back as bf16
        _quant("quant_t24_131072x2048", 131072, 2048, 128, "bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["few", "few", "few_w4", "few_w4", "matvec", "matvec", "quant"])
    if op in ("few", "few_w4"):
        T = rng.randint(1, 8)
        H = _log_int(rng, 256, 8192, 64)
        E = _log_int(rng, 8, 512)
        k = rng.randint(1, min(10, E))
        I = _log_int(rng, 64, 2048, 64)
        Is = rng.choice([I, _log_int(rng, 64, 2048, 64)])
        while E > 8 and E * 3 * H * I * 2 > 3_200_000_000:  # what the largest listed case reads
            E = max(8, E // 2)
        k = min(k, E)
        return _layer(op, None, T, H, E, k, I, Is, bias=rng.random() < 0.5,
                      skew=rng.choice([0.0, 0.0, 1.1]),
                      group=rng.choice([32, 64, 128]) if op == "few_w4" else 0)
    if op == "matvec":
        x = rng.choice(["bf16", "fp16"])
        return _matvec(None, rng.randint(1, 16), _log_int(rng, 64, 32768), _log_int(rng, 64, 8192),
                       rng.choice([32, 64, 128]), x, rng.choice([x, "fp32"]),
                       pad=rng.choice([0, 0, 5, 8]))
    return _quant(None, _log_int(rng, 64, 60000), _log_int(rng, 64, 4096), rng.choice([32, 64, 128]),
                  rng.choice(["fp32", "bf16"]))


# ------------------------------------------------------------------------------------ inputs

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _normal(gen, shape, sigma, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=gen)


def _pack(codes):
    """Codes 0..15 [..., blocks * 128] -> bytes [..., blocks * 64]."""
    lead, n = codes.shape[:-1], codes.shape[-1] // 128
    # element = 32 j + 8 t + 4 b + 2 h + odd; byte = 16 t + 4 j + 2 odd + b, nibble h
    c = codes.reshape(*lead, n, 4, 4, 2, 2, 2)
    d = c.dim()
    c = c.permute(*range(d - 5), d - 4, d - 5, d - 1, d - 3, d - 2)
    return (c[..., 0] | (c[..., 1] << 4)).reshape(*lead, n * 64).contiguous()


def _quantized(w, group):
    """(bytes, scales) of a matrix [rows, K], by the format's definition."""
    rows, K = w.shape
    blocks, groups = -(-K // 128), -(-K // group)
    v = torch.zeros((rows, blocks * 128), dtype=torch.float32, device=w.device)
    v[:, :K] = w.float()
    v = v.reshape(rows, -1, group)
    s = (v.abs().amax(-1) / 7).to(torch.bfloat16)
    f = s.float()[..., None]
    codes = torch.where(f > 0, v / f, 0.0).round().clamp(-8, 7).to(torch.int8) + 8
    pad = torch.zeros((rows, -(-groups // 8) * 8), dtype=torch.bfloat16, device=w.device)
    pad[:, :groups] = s[:, :groups]
    return _pack(codes.to(torch.uint8).reshape(rows, -1)), pad


def _quantized_bank(gen, E, rows, K, group):
    """A bank of E random expert matrices, quantised expert by expert."""
    q = torch.empty((E, rows, -(-K // 128) * 64), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, rows, -(-(-(-K // group)) // 8) * 8), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        q[e], s[e] = _quantized(_normal(gen, (rows, K), SIGMA_W), group)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "quant":
        c["w"] = _normal(gen, (c["rows"], c["K"]), SIGMA_W)
        # rows whose weights are all zero, as pruned channels leave them
        c["w"][torch.rand(c["rows"], device="cuda", generator=gen) < 0.05] = 0
        c["q"] = torch.empty((c["rows"], -(-c["K"] // 128) * 64), dtype=torch.uint8, device="cuda")
        c["s"] = torch.empty((c["rows"], -(-(-(-c["K"] // c["group"])) // 8) * 8),
                             dtype=torch.bfloat16, device="cuda")
        c["back"] = torch.empty((c["rows"], c["K"]), dtype=DTYPES[c["to"]], device="cuda")
        return c
    if c["op"] == "matvec":
        c["q"], c["s"] = _quantized(_normal(gen, (c["N"], c["K"]), SIGMA_W), c["group"])
        c["x"] = _normal(gen, (c["T"], c["K"] + c["pad"]), 1.0, DTYPES[c["x"]])[:, :c["K"]]
        c["out"] = torch.empty((c["T"], c["N"] + c["pad"]), dtype=DTYPES[c["y"]],
                               device="cuda")[:, :c["N"]]
        return c
    T, H, E, k, I, Is = (c[n] for n in ("T", "H", "E", "k", "I", "Is"))
    w = {"w_router": _normal(gen, (E, H), SIGMA_W, torch.float32),
         "ws_gate_up": _normal(gen, (2 * Is, H), SIGMA_W), "ws_down": _normal(gen, (H, Is), SIGMA_W),
         "w_shared_gate": _normal(gen, (H,), SIGMA_W)}
    if c["bias"] or c["skew"]:
        b = 0.1 * torch.randn(E, device="cuda", generator=gen)
        if c["skew"]:  # a few experts that most tokens choose
            rank = torch.randperm(E, device="cuda", generator=gen).float() + 1
            b = b - c["skew"] * rank.log()
        w["router_bias"] = b
    if c["op"] == "few":
        w["w_gate_up"] = _normal(gen, (E, 2 * I, H), SIGMA_W)
        w["w_down"] = _normal(gen, (E, H, I), SIGMA_W)
    else:
        c["q_gate_up"], c["s_gate_up"] = _quantized_bank(gen, E, 2 * I, H, c["group"])
        c["q_down"], c["s_down"] = _quantized_bank(gen, E, H, I, c["group"])
    c["w"] = w
    c["x"] = _normal(gen, (T, H), 1.0)
    c["out"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
    c["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
    c["p"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    # the room that the package's layer calls work in, as a program keeps it
    c["ws"] = torch.zeros(_room(T, H, E, k, I, Is), dtype=torch.uint8, device="cuda")
    return c


def _room(T, H, E, k, I, Is):
    """Bytes that hold the layer's intermediates with space to spare (moe_workspace_bytes
    needs less)."""
    R, L = T * k, max(I, Is)
    return (64 << 20) + 6 * E * H + 64 * 511 * E + 4 * R * H + 12 * (R + T) * L + 4096 * E


# ------------------------------------------------------------------------------------ run

def run(state):
    return {"few": _run_layer, "few_w4": _run_layer, "matvec": _run_matvec,
            "quant": _run_quant}[state["op"]](state)


def _package():
    import sparse_moe_expert_fp32_b200 as moe

    return moe


def _run_layer(c):
    if own:
        moe = _package()
        s = moe.make_shape(c["T"], c["H"], c["E"], c["k"], c["I"], c["Is"])
        if c["op"] == "few":
            moe.moe_layer_forward_few(s, c["x"], c["w"], c["out"], c["ws"], topk_ids=c["ids"],
                                      topk_w=c["p"])
        else:
            q = {n: c[n] for n in ("q_gate_up", "s_gate_up", "q_down", "s_down", "group")}
            moe.moe_layer_forward_few_w4(s, c["x"], c["w"], q, c["out"], c["ws"],
                                         topk_ids=c["ids"], topk_w=c["p"])
        return {"out": c["out"], "ids": c["ids"], "p": c["p"]}
    w, x = c["w"], c["x"].float()
    # 64 bits: two logits that nearly tie decide which expert a token goes to
    logits = c["x"].double() @ w["w_router"].double().T
    if "router_bias" in w:
        logits = logits + w["router_bias"].double()
    top, ids = logits.sort(dim=-1, descending=True, stable=True)  # ties: the lowest index first
    top, ids = top[:, :c["k"]].float(), ids[:, :c["k"]]
    p = (top - top[:, :1]).exp()
    p = p / p.sum(-1, keepdim=True)
    if c["op"] == "few":
        gate_up, down = w["w_gate_up"][ids].float(), w["w_down"][ids].float()
    else:
        gate_up = _weights(c["q_gate_up"][ids], c["s_gate_up"][ids], c["H"], c["group"])
        down = _weights(c["q_down"][ids], c["s_down"][ids], c["I"], c["group"])
    routed = _swiglu(x[:, None], gate_up, down)  # [T, k, H]
    shared = _swiglu(x, w["ws_gate_up"].float(), w["ws_down"].float())
    open_ = 1 / (1 + (-(x @ w["w_shared_gate"].float())).exp())
    out = (p[..., None] * routed).sum(1) + open_[:, None] * shared
    return {"out": out, "ids": ids.to(torch.int32), "p": p}


def _swiglu(x, gate_up, down):
    gu = (gate_up @ x[..., None])[..., 0] if gate_up.dim() > 2 else x @ gate_up.T
    n = gu.shape[-1] // 2
    h = gu[..., :n] / (1 + (-gu[..., :n]).exp()) * gu[..., n:]
    return (down @ h[..., None])[..., 0] if down.dim() > 2 else h @ down.T


def _codes(q, K):
    """Bytes [..., blocks * 64] -> codes - 8 as fp32 [..., K]."""
    lead, n = q.shape[:-1], q.shape[-1] // 64
    b = q.reshape(*lead, n, 4, 4, 2, 2)  # t, j, odd, b
    c = torch.stack((b & 15, b >> 4), -1)  # t, j, odd, b, h
    d = c.dim()
    c = c.permute(*range(d - 5), d - 4, d - 5, d - 2, d - 1, d - 3)  # j, t, b, h, odd
    return c.reshape(*lead, n * 128)[..., :K].float() - 8


def _weights(q, s, K, group):
    """The fp32 matrix that bytes and scales stand for (exact: 4 by 8 significant bits)."""
    scale = s[..., : -(-K // group), None].float().expand(*s.shape[:-1], -(-K // group), group)
    return _codes(q, K) * scale.reshape(*s.shape[:-1], -1)[..., :K]


def _run_matvec(c):
    if own:
        _package().moe_matvec_w4(c["x"], c["q"], c["s"], c["out"], c["group"])
        return c["out"]
    y = c["x"].float() @ _weights(c["q"], c["s"], c["K"], c["group"]).T
    return y.to(DTYPES[c["y"]])


def _run_quant(c):
    if own:
        moe = _package()
        moe.moe_quantize_w4(c["w"], c["q"], c["s"], c["group"])
        moe.moe_dequantize_w4(c["q"], c["s"], c["back"], c["group"])
        return {"values": c["back"], "scales": c["s"]}
    q, s = _quantized(c["w"], c["group"])
    return {"values": _weights(q, s, c["K"], c["group"]).to(DTYPES[c["to"]]), "scales": s}


# ------------------------------------------------------------------------------------ floors

def work(case):
    c = case
    if c["op"] == "quant":
        # the matrix read, codes and scales written, both read again, the values written
        n = c["rows"] * c["K"]
        packed = n / 2 + 2 * c["rows"] * -(-c["K"] // c["group"])
        return {"bytes": 2 * n + 2 * packed + n * (4 if c["to"] == "fp32" else 2), "flops": 4 * n}
    if c["op"] == "matvec":
        n = c["N"] * c["K"]
        return {"bytes": n / 2 + 2 * c["N"] * -(-c["K"] // c["group"]) + 2 * c["T"] * c["K"]
                + (4 if c["y"] == "fp32" else 2) * c["T"] * c["N"], "flops": 2 * n * c["T"]}
    T, H, E, k, I, Is = (c[n] for n in ("T", "H", "E", "k", "I", "Is"))
    # experts that at least one token chooses: the mean over uniform choices
    active = E * (1 - (1 - k / E) ** T)
    byte = 2 if c["op"] == "few" else 0.5 + 2 / c["group"]
    return {"bytes": active * 3 * H * I * byte + 6 * Is * H + 4 * E * H + 2 * H + 6 * T * H + 8 * T * k,
            "flops": 2 * T * (H * E + 3 * H * (k * I + Is))}


# ------------------------------------------------------------------------------------ exact

def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "quant":
        w = c["w"].double()
        groups = -(-c["K"] // c["group"])
        s = torch.stack([w[:, g * c["group"]:(g + 1) * c["group"]].abs().amax(1) for g in range(groups)], 1)
        s = (s / 7).to(torch.bfloat16)
        scale = s.double().repeat_interleave(c["group"], 1)[:, :c["K"]]
        v = torch.where(scale > 0, w / scale, 0.0).round().clamp(-8, 7) * scale
        full = torch.zeros(c["s"].shape, dtype=torch.float64, device="cuda")
        full[:, :groups] = s.double()
        return {"values": v, "scales": full}
    if c["op"] == "matvec":
        x, rows = c["x"].double(), []
        for n in range(0, c["N"], 4096):  # a slice of the matrix at a time
            rows.append(x @ _exact_weights(c["q"][n:n + 4096], c["s"][n:n + 4096], c["K"], c["group"]).T)
        return torch.cat(rows, 1)
    w, x = c["w"], c["x"].double()
    out, chosen, probs = [], [], []
    for t in range(c["T"]):
        logits = (w["w_router"].double() * x[t]).sum(1)
        if "router_bias" in w:
            logits = logits + w["router_bias"].double()
        by = sorted(range(c["E"]), key=lambda e, v=logits.tolist(): (-v[e], e))[:c["k"]]
        p = torch.softmax(logits[by], 0)
        y = torch.sigmoid((w["w_shared_gate"].double() * x[t]).sum()) * _exact_expert(
            w["ws_gate_up"].double(), w["ws_down"].double(), x[t])
        for e, pe in zip(by, p):
            if c["op"] == "few":
                gate_up, down = w["w_gate_up"][e].double(), w["w_down"][e].double()
            else:
                gate_up = _exact_weights(c["q_gate_up"][e], c["s_gate_up"][e], c["H"], c["group"])
                down = _exact_weights(c["q_down"][e], c["s_down"][e], c["I"], c["group"])
            y = y + pe * _exact_expert(gate_up, down, x[t])
        out.append(y)
        chosen.append(by)
        probs.append(p)
    return {"out": torch.stack(out), "ids": torch.tensor(chosen, dtype=torch.int32, device="cuda"),
            "p": torch.stack(probs)}


def _exact_expert(gate_up, down, x):
    n = gate_up.shape[0] // 2
    g, u = gate_up[:n] @ x, gate_up[n:] @ x
    return down @ (torch.sigmoid(g) * g * u)


def _exact_weights(q, s, K, group):
    """Element by element from the format's definition, in 64 bits."""
    e = torch.arange(K, device=q.device)
    block, j, t, i = e // 128, e // 32 % 4, e // 8 % 4, e % 8
    nibble = i // 2 + 4 * (i % 2)
    byte = q[:, block * 64 + 16 * t + 4 * j + nibble // 2].to(torch.int16)
    code = torch.where(nibble % 2 == 1, byte >> 4, byte & 15) - 8
    return code.double() * s[:, e // group].double()
