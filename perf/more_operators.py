"""The gated feed-forward block in 8 bits and the products with 4-bit weights in
groups, as measured: what a pass is, its plain form in elementary torch
operations, and its definition in 64 bits.

Operators (Python names of the package):
  nf4_fp8_gated_fwd       A = act(X Wg^T) * (X Wu^T) from block-scaled e4m3
                          operands, written in 8 bits for the next product or
                          in 16 / 32; G = X Wg^T and U = X Wu^T on request
  nf4_fp8_gated_bwd       dG = dA U act'(G), dU = dA act(G), in 8 bits
  nf4_fp8_gated_bwd_dx    dX = dG Wg + dU Wu
  nf4_int4_quantize       W -> 4-bit codes with a scale (and a zero point) for
                          each group along a row, and
  nf4_int4_dequantize     the values that they stand for
  nf4_int4_matmul_fwd     Y = X w^T, w = (code - zero point) * scale
  nf4_int4_gated_fwd      Y = act(X wg^T) * (X wu^T)

With `own` false a pass runs the plain form, in 32 bits; with `own` true it
makes the calls that a user of the package makes.
"""
import math

import torch

own = False

BLOCK = 128                     # values of an 8-bit scale along a row
E4M3_MAX = 448.0
MIN_AMAX = 2.0 ** -117          # blocks whose largest magnitude is below it are stored as zeros
FP8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "fp8": FP8}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "fp8": 1}
# act(g) = g sigma(g (c0 + c1 g^2))
GELU = 2.0 * math.sqrt(2.0 / math.pi)
CURVE = {"silu": (1.0, 0.0), "gelu_tanh": (GELU, GELU * 0.044715)}


def listed():
    return [
        # one token through an MLP's gate and up projections, on to the down product in 8 bits
        dict(name="gated_decode_m1_18944x3584", op="gated", m=1, n=18944, k=3584, act="silu", out="fp8",
             save=False),
        # a batch of 64 decoding sequences: the two weights' bytes
        dict(name="gated_batch_m64_18944x3584", op="gated", m=64, n=18944, k=3584, act="silu", out="fp8",
             save=False),
        # a ragged prompt, widths that end inside a block, fp32 output
        dict(name="gated_ragged_m777_4112x3600", op="gated", m=777, n=4112, k=3600, act="gelu_tanh",
             out="f32", save=False),
        # a training step's forward: the tensor cores, and what the backward keeps
        dict(name="gated_train_m4096_11008x4096", op="gated", m=4096, n=11008, k=4096, act="silu",
             out="fp8", save=True),
        # the gradients of a short ragged batch through a narrow block
        dict(name="gated_bwd_short_m250_1040x3584", op="gated_bwd", m=250, n=1040, k=3584,
             act="gelu_tanh", da="bf16", out="bf16"),
        # a training step's gradients
        dict(name="gated_bwd_train_m2048_11008x4096", op="gated_bwd", m=2048, n=11008, k=4096, act="silu",
             da="bf16", out="bf16"),
        # one token's query projection in 4 bits: latency and the weight's bytes
        dict(name="int4_decode_m1_4096x4096", op="int4", m=1, n=4096, k=4096, group=128, zero=True,
             x="bf16", out="f32"),
        # a batch of 16 sequences through the long rows of a down projection, symmetric codes
        dict(name="int4_batch_m16_3584x18944", op="int4", m=16, n=3584, k=18944, group=64, zero=False,
             x="f16", out="f16"),
        # one token through a whole MLP's gate and up projections
        dict(name="int4_gated_m1_18944x3584", op="int4_gated", m=1, n=18944, k=3584, group=128, zero=True,
             x="bf16", out="bf16", act="silu"),
        # seven draft tokens through a smaller MLP with fine groups
        dict(name="int4_gated_m7_11008x4096", op="int4_gated", m=7, n=11008, k=4096, group=32, zero=True,
             x="bf16", out="bf16", act="gelu_tanh"),
        # a key projection of a 16-bit checkpoint taken to 4 bits and back, symmetric
        dict(name="int4_quant_512x3584", op="int4_quant", n=512, k=3584, group=64, zero=False, x="bf16",
             out="f32"),
        # an up projection of a 32-bit checkpoint, with zero points, the values for a library product
        dict(name="int4_quant_11008x4096", op="int4_quant", n=11008, k=4096, group=128, zero=True, x="f32",
             out="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, in whole steps."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "int4", "int4", "int4_gated", "int4_quant"])
    act = rng.choice(sorted(CURVE))
    if op in ("gated", "gated_bwd"):
        c = dict(op=op, m=_log(rng, 1, 4096), n=_log(rng, 256, 18944, 16), k=_log(rng, 256, 8192, 16),
                 act=act)
        while c["m"] * c["n"] * c["k"] > 4096 * 11008 * 4096:
            c["m"] = (c["m"] + 1) // 2
        if op == "gated":
            return dict(c, out=rng.choice(["fp8", "fp8", "bf16", "f32"]), save=rng.random() < 0.5)
        return dict(c, da=rng.choice(["bf16", "f32"]), out="bf16")
    group, zero = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "int4_quant":
        return dict(op=op, n=_log(rng, 1, 11008), k=_log(rng, 256, 8192, group), group=group, zero=zero,
                    x=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]))
    x = rng.choice(["bf16", "f16"])
    c = dict(op=op, m=_log(rng, 1, 32), n=_log(rng, 64, 18944), k=_log(rng, 256, 18944, group), group=group,
             zero=zero, x=x, out=rng.choice(["f32", x]))
    return dict(c, act=act) if op == "int4_gated" else c


# ------------------------------------------------------------- plain forms --

def _blocks(x):
    """x [m, k] as 1 x 128 blocks [m, ceil(k / 128), 128], filled up with zeros."""
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK))
    return x.reshape(x.shape[0], -1, BLOCK)


def _plain_quantize(x):
    """(codes, scale): scale = max|x| / 448 of each 1 x 128 block, codes = x / scale rounded to e4m3."""
    m, k = x.shape
    b = _blocks(x)
    amax = b.abs().amax(dim=2)
    live = amax >= MIN_AMAX
    scale = torch.where(live, amax / torch.full_like(amax, E4M3_MAX), 0.0)
    inverse = torch.where(live, 1.0 / scale, 0.0)
    q = (b * inverse[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.reshape(m, -1)[:, :k].to(FP8).contiguous(), scale


def _plain_values(codes, scale, rows):
    """The values that 8-bit codes and scales stand for, in 32 bits."""
    m, k = codes.shape
    s = scale.repeat_interleave(rows, 0)[:m] if rows > 1 else scale
    return codes.float() * s.repeat_interleave(BLOCK, 1)[:, :k]


def _plain_sigma(g, act):
    c0, c1 = CURVE[act]
    return torch.sigmoid(g * (c0 + c1 * g * g))


def _plain_int4_values(codes, scale, zero):
    """The values of 4-bit codes (the even one of a byte in its high half), in 32 bits."""
    n, half = codes.shape
    q = torch.stack([codes >> 4, codes & 15], dim=2).reshape(n, 2 * half).float()
    group = q.shape[1] // scale.shape[1]
    z = 8.0 if zero is None else zero.float().repeat_interleave(group, 1)
    return (q - z) * scale.float().repeat_interleave(group, 1)


def _plain_int4_quantize(w, group, zero, dtype):
    n, k = w.shape
    g = w.float().reshape(n, k // group, group)
    if zero:
        lo, hi = g.amin(dim=2).clamp(max=0.0), g.amax(dim=2).clamp(min=0.0)
        scale = ((hi - lo) / torch.full_like(hi, 15.0)).to(dtype)
        s = torch.where(scale == 0, 1.0, scale.float())
        z = torch.where(scale == 0, 0.0, torch.round(-lo / s).clamp(0, 15))
    else:
        a = g.abs().amax(dim=2)
        scale = (a / torch.full_like(a, 7.0)).to(dtype)
        s = torch.where(scale == 0, 1.0, scale.float())
        z = torch.full_like(s, 8.0)
    live = (scale != 0)[:, :, None]
    q = torch.where(live, (torch.round(g / s[:, :, None]) + z[:, :, None]).clamp(0, 15), z[:, :, None])
    q = q.reshape(n, k // 2, 2).to(torch.uint8)
    return q[:, :, 0] << 4 | q[:, :, 1], scale, z.to(torch.uint8) if zero else None


# ------------------------------------------------------------------ inputs --

def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _activations(gen, m, k, dtype):
    """Hidden states: unit normal, a few channels 20 times larger, the last of many rows
    padding (all zeros)."""
    x = torch.randn((m, k), generator=gen, device="cuda")
    x[:, torch.randint(0, k, (max(1, k // 500),), generator=gen, device="cuda")] *= 20.0
    if m > 8:
        x[-1] = 0.0
    return x.to(dtype)


def _weight8(gen, n, k):
    """A weight in 8 bits with a scale for each 128 x 128 block, as a program keeps it."""
    w = torch.nn.functional.pad(_normal(gen, (n, k), 0.02, torch.float32), (0, -k % BLOCK, 0, -n % BLOCK))
    b = w.reshape(w.shape[0] // BLOCK, BLOCK, w.shape[1] // BLOCK, BLOCK)
    scale = b.abs().amax(dim=(1, 3)) / E4M3_MAX
    q = (b / scale[:, None, :, None]).reshape(w.shape)[:n, :k]
    return q.to(FP8).contiguous(), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, n, k = case["op"], case["n"], case["k"]
    if op == "int4_quant":
        return dict(case=case, w=_normal(gen, (n, k), 0.02, TYPES[case["x"]]))
    m = case["m"]
    if op in ("gated", "gated_bwd"):
        state = dict(case=case, wg=_weight8(gen, n, k), wu=_weight8(gen, n, k))
        if op == "gated":      # the left operand as a norm has just left it
            return dict(state, a=_plain_quantize(_activations(gen, m, k, torch.float32)))
        # the projections as the forward kept them, the gradient as the down product left it
        return dict(state, g=_normal(gen, (m, n), 1.5, torch.bfloat16),
                    u=_normal(gen, (m, n), 1.5, torch.bfloat16), da=_normal(gen, (m, n), 0.01, TYPES[case["da"]]))
    # weights as a program keeps them, in the activations' type of scale
    t = TYPES[case["x"]]
    state = dict(case=case, x=_activations(gen, m, k, t))
    for name in ("w",) if op == "int4" else ("wg", "wu"):
        state[name] = _plain_int4_quantize(_normal(gen, (n, k), 0.02, torch.float32), case["group"],
                                           case["zero"], t)
    return state


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import dequant_gemm_gb300 as nf4
        if op in ("gated", "gated_bwd"):
            wg, wu = nf4.FP8Tensor(*state["wg"], block_rows=128), nf4.FP8Tensor(*state["wu"], block_rows=128)
        if op == "gated":
            y, g, u = nf4.nf4_fp8_gated_fwd(nf4.FP8Tensor(*state["a"]), wg, wu, activation=case["act"],
                                            out_dtype=TYPES[case["out"]], save=case["save"])
            got = {"codes": y.codes, "scale": y.scale} if case["out"] == "fp8" else {"y": y}
            return dict(got, g=g, u=u) if case["save"] else got
        if op == "gated_bwd":
            dg, du = nf4.nf4_fp8_gated_bwd(state["da"], state["g"], state["u"], activation=case["act"])
            dx = nf4.nf4_fp8_gated_bwd_dx(dg, du, wg, wu, out_dtype=TYPES[case["out"]])
            return {"dg": dg.codes, "dg_scale": dg.scale, "du": du.codes, "du_scale": du.scale, "dx": dx}
        if op == "int4":
            return nf4.nf4_int4_matmul_fwd(state["x"], nf4.Int4Weight(*state["w"]), out_dtype=TYPES[case["out"]])
        if op == "int4_gated":
            return nf4.nf4_int4_gated_fwd(state["x"], nf4.Int4Weight(*state["wg"]), nf4.Int4Weight(*state["wu"]),
                                          activation=case["act"], out_dtype=TYPES[case["out"]])
        q = nf4.nf4_int4_quantize(state["w"], group=case["group"], zero_point=case["zero"],
                                  scale_dtype=torch.bfloat16)
        return {"values": nf4.nf4_int4_dequantize(q, out_dtype=TYPES[case["out"]]), "scale": q.scale}
    if op == "gated":
        x = _plain_values(*state["a"], 1)
        g, u = x @ _plain_values(*state["wg"], 128).t(), x @ _plain_values(*state["wu"], 128).t()
        y = g * _plain_sigma(g, case["act"]) * u
        if case["out"] == "fp8":
            codes, scale = _plain_quantize(y)
            got = {"codes": codes, "scale": scale}
        else:
            got = {"y": y.to(TYPES[case["out"]])}
        return dict(got, g=g.bfloat16(), u=u.bfloat16()) if case["save"] else got
    if op == "gated_bwd":
        da, g, u = state["da"].float(), state["g"].float(), state["u"].float()
        c0, c1 = CURVE[case["act"]]
        s = _plain_sigma(g, case["act"])
        dg = _plain_quantize(da * u * (s + g * s * (1.0 - s) * (c0 + 3.0 * c1 * g * g)))
        du = _plain_quantize(da * g * s)
        dx = _plain_values(*dg, 1) @ _plain_values(*state["wg"], 128) \
            + _plain_values(*du, 1) @ _plain_values(*state["wu"], 128)
        return {"dg": dg[0], "dg_scale": dg[1], "du": du[0], "du_scale": du[1], "dx": dx.to(TYPES[case["out"]])}
    if op == "int4":
        return (state["x"].float() @ _plain_int4_values(*state["w"]).t()).to(TYPES[case["out"]])
    if op == "int4_gated":
        x = state["x"].float()
        g, u = x @ _plain_int4_values(*state["wg"]).t(), x @ _plain_int4_values(*state["wu"]).t()
        return (g * _plain_sigma(g, case["act"]) * u).to(TYPES[case["out"]])
    q = _plain_int4_quantize(state["w"], case["group"], case["zero"], torch.bfloat16)
    return {"values": _plain_int4_values(*q).to(TYPES[case["out"]]), "scale": q[1]}


def work(case):
    op, n, k = case["op"], case["n"], case["k"]
    if op in ("gated", "gated_bwd"):
        m, nb, kb = case["m"], -(-n // BLOCK), -(-k // BLOCK)
        b = 2 * (n * k + 4 * nb * kb)
        if op == "gated":
            b += m * (k + 4 * kb) + m * n * (BYTES[case["out"]] + (4 if case["save"] else 0))
            return {"bytes": b + (4 * m * nb if case["out"] == "fp8" else 0), "flops": 4 * m * n * k}
        b += m * n * (BYTES[case["da"]] + 4) + 2 * m * (n + 4 * nb) + m * k * BYTES[case["out"]]
        return {"bytes": b, "flops": 4 * m * n * k}
    w = n * k // 2 + n * (k // case["group"]) * (3 if case["zero"] else 2)
    if op == "int4_quant":
        return {"bytes": n * k * (BYTES[case["x"]] + BYTES[case["out"]]) + 2 * w, "flops": 7 * n * k}
    m, weights = case["m"], 2 if op == "int4_gated" else 1
    return {"bytes": weights * w + m * k * BYTES[case["x"]] + m * n * BYTES[case["out"]],
            "flops": 2 * weights * m * n * k}


# -------------------------------------------------- the definitions, 64 bits --

def _exact8(codes, scale, rows):
    i = torch.arange(codes.shape[0], device=scale.device) // rows
    j = torch.arange(codes.shape[1], device=scale.device) // BLOCK
    return codes.double() * scale.double()[i][:, j]


def _exact_quantize8(x):
    m, k = x.shape
    scale = torch.stack([c.abs().amax(dim=1) for c in x.split(BLOCK, dim=1)], dim=1) / E4M3_MAX
    scale[scale < MIN_AMAX / E4M3_MAX] = 0.0
    each = scale[:, torch.arange(k, device=x.device) // BLOCK]
    return torch.where(each > 0, x / torch.where(each > 0, each, 1.0), 0.0).to(FP8), scale


def _exact4(codes, scale, zero):
    n, k = codes.shape[0], 2 * codes.shape[1]
    at = torch.arange(k, device=codes.device)
    q = codes[:, at // 2].to(torch.int64) // torch.where(at % 2 == 0, 16, 1) % 16
    j = at // (k // scale.shape[1])
    return (q - (8 if zero is None else zero.to(torch.int64)[:, j])).double() * scale.double()[:, j]


def _exact_act(g, act):
    """(act(g), act'(g)) by the activation's own formula."""
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-g))
        return g * e, e * (1.0 + g * (1.0 - e))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g.pow(3)))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 0.134145 * g * g)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        x = _exact8(*state["a"], 1)
        g = torch.einsum("mk,nk->mn", x, _exact8(*state["wg"], BLOCK))
        u = torch.einsum("mk,nk->mn", x, _exact8(*state["wu"], BLOCK))
        y = _exact_act(g, case["act"])[0] * u
        got = dict(zip(("codes", "scale"), _exact_quantize8(y))) if case["out"] == "fp8" else {"y": y}
        return dict(got, g=g, u=u) if case["save"] else got
    if op == "gated_bwd":
        da, g, u = (state[t].double() for t in ("da", "g", "u"))
        f, slope = _exact_act(g, case["act"])
        dg, du = _exact_quantize8(da * u * slope), _exact_quantize8(da * f)
        dx = torch.einsum("mn,nk->mk", _exact8(*dg, 1), _exact8(*state["wg"], BLOCK))
        dx += torch.einsum("mn,nk->mk", _exact8(*du, 1), _exact8(*state["wu"], BLOCK))
        return {"dg": dg[0], "dg_scale": dg[1], "du": du[0], "du_scale": du[1], "dx": dx}
    if op == "int4":
        return torch.einsum("mk,nk->mn", state["x"].double(), _exact4(*state["w"]))
    if op == "int4_gated":
        x = state["x"].double()
        g = torch.einsum("mk,nk->mn", x, _exact4(*state["wg"]))
        return _exact_act(g, case["act"])[0] * torch.einsum("mk,nk->mn", x, _exact4(*state["wu"]))
    w = state["w"].double().unflatten(1, (-1, case["group"]))
    if case["zero"]:
        low = -w.amin(dim=2, keepdim=True).clamp(max=0)
        scale = ((w.amax(dim=2, keepdim=True).clamp(min=0) + low) / 15.0).bfloat16().double()
        z = torch.round(low / scale).clamp(0, 15)      # no group of normal values is all zeros
    else:
        scale = (w.abs().amax(dim=2, keepdim=True) / 7.0).bfloat16().double()
        z = 8.0
    values = ((w / scale + z).round().clamp(0, 15) - z) * scale
    return {"values": values.flatten(1), "scale": scale[:, :, 0]}
