"""The 8-bit floating point operators as measured: what a pass is, its plain
form in elementary torch operations, and its definition in 64 bits.

Operators (Python names of the package):
  nf4_fp8_quantize        x -> e4m3 codes with an fp32 scale for each 1 x 128
                          (activations) or 128 x 128 (weights) block
  nf4_fp8_matmul_fwd      Y = dq(X) dq(W)^T from such codes and scales
  nf4_fp8_matmul_bwd_dx   dX = dq(dY) dq(W), the input gradient of the frozen W
  nf4_rmsnorm_fwd         h = x + residual, y = h / rms(h) * weight, y in 8 bits
                          with scales (for the product above) or in 16 / 32 bits
  nf4_rmsnorm_bwd         the gradients of the norm's input and weight

With `own` false a pass runs the plain form, in 32 bits; with `own` true it
makes the calls that a user of the package makes.
"""
import math

import torch

own = False

BLOCK = 128                     # values of a scale along a row
E4M3_MAX = 448.0
MIN_AMAX = 2.0 ** -117          # blocks whose largest magnitude is below it are stored as zeros
EPS = 1e-6
FP8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "fp8": FP8}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "fp8": 1}


def listed():
    return [
        # one token's query projection in a decoding step: latency and the weight's bytes
        dict(name="fwd_decode_m1_4096x4096", op="fwd", m=1, n=4096, k=4096, out="bf16"),
        # a batch of 64 decoding sequences through an MLP gate: the weight's bytes
        dict(name="fwd_batch_m64_18944x3584", op="fwd", m=64, n=18944, k=3584, out="bf16"),
        # a ragged prompt, a width whose last block is short, rows that end inside a block, fp32 output
        dict(name="fwd_ragged_m777_4112x3600", op="fwd", m=777, n=4112, k=3600, out="f32"),
        # a prompt of 4096 tokens through an MLP up projection: the tensor cores
        dict(name="fwd_prefill_m4096_11008x4096", op="fwd", m=4096, n=11008, k=4096, out="bf16"),
        # a short ragged batch's gradient through a narrow key projection, fp32 output
        dict(name="dx_short_m250_512x3584", op="dx", m=250, n=512, k=3584, out="f32"),
        # a training step's gradient through an MLP down projection
        dict(name="dx_train_m2048_4096x11008", op="dx", m=2048, n=4096, k=11008, out="bf16"),
        # the norm before one token's projections: latency alone
        dict(name="norm_decode_m1_3584", op="norm", m=1, k=3584, x="bf16", residual="bf16",
             out="fp8", rstd=False),
        # the norm of a long prompt with the residual stream held in 32 bits: bandwidth
        dict(name="norm_prompt_m8192_4096", op="norm", m=8192, k=4096, x="bf16", residual="f32",
             out="fp8", rstd=False),
        # the norm's gradients in a training step
        dict(name="norm_bwd_m4096_3584", op="norm_bwd", m=4096, k=3584, x="bf16", w="f32", dh=True),
        # a ragged batch, an odd width, no gradient from the stream, all in 32 bits
        dict(name="norm_bwd_ragged_m333_5001", op="norm_bwd", m=333, k=5001, x="f32", w="f32",
             dh=False),
        # the activations of a prompt, rounded between two products
        dict(name="quant_act_m4096_18944", op="quant", m=4096, k=18944, x="bf16", rows=1),
        # a weight taken from a checkpoint in 32 bits
        dict(name="quant_weight_11008x4096", op="quant", m=11008, k=4096, x="f32", rows=128),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, in whole steps."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "dx", "norm", "norm_bwd", "quant"])
    if op in ("fwd", "dx"):
        c = dict(op=op, m=_log(rng, 1, 4096), n=_log(rng, 256, 18944, 16),
                 k=_log(rng, 256, 18944, 16), out=rng.choice(["bf16", "f32"]))
        while c["m"] * c["n"] * c["k"] > 4096 * 11008 * 4096:
            c["m"] = (c["m"] + 1) // 2
        return c
    if op == "norm":
        out = rng.choice(["fp8", "fp8", "bf16"])
        return dict(op=op, m=_log(rng, 1, 8192), k=_log(rng, 256, 4096, 16 if out == "fp8" else 1),
                    x="bf16", residual=rng.choice(["none", "bf16", "f32"]), out=out,
                    rstd=rng.random() < 0.5)
    if op == "norm_bwd":
        x = rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, m=_log(rng, 1, 4096), k=_log(rng, 256, 5120), x=x,
                    w=rng.choice(["f32", x]), dh=rng.random() < 0.5)
    rows = rng.choice([1, 128])
    x = rng.choice(["bf16", "f32"])
    return dict(op=op, m=_log(rng, 1, 4096), k=_log(rng, 256, 11008, 16), x=x, rows=rows)


# ------------------------------------------------------------- plain forms --

def _blocks(x, rows):
    """x [m, k] as blocks [ceil(m / rows), rows, ceil(k / 128), 128], filled up with zeros."""
    m, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % BLOCK, 0, -m % rows))
    return x.reshape(x.shape[0] // rows, rows, x.shape[1] // BLOCK, BLOCK)


def _plain_quantize(x, rows):
    """(codes, scale): scale = max|x| / 448 of the block, codes = x / scale rounded to e4m3."""
    m, k = x.shape
    b = _blocks(x.float(), rows)
    amax = b.abs().amax(dim=(1, 3))
    live = amax >= MIN_AMAX
    scale = torch.where(live, amax / E4M3_MAX, 0.0)
    inverse = torch.where(live, 1.0 / scale, 0.0)
    q = (b * inverse[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.reshape(b.shape[0] * rows, -1)[:m, :k]
    return q.to(FP8).contiguous(), scale


def _plain_values(codes, scale, rows):
    """The values that codes and scales stand for, in 32 bits."""
    m, k = codes.shape
    s = scale.repeat_interleave(rows, 0)[:m] if rows > 1 else scale
    return codes.float() * s.repeat_interleave(BLOCK, 1)[:, :k]


def _plain_norm(x, residual, weight, eps, out, keep_rstd):
    h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(dim=1, keepdim=True) + eps)
    y = hf * rstd * weight.float()
    got = {}
    if out == FP8:
        got["codes"], got["scale"] = _plain_quantize(y, 1)
    else:
        got["y"] = y.to(out)
    if residual is not None:
        got["h"] = h
    if keep_rstd:
        got["rstd"] = rstd[:, 0]
    return got


def _plain_norm_bwd(dy, h, weight, rstd, dh):
    g, hf, r = dy.float(), h.float(), rstd[:, None]
    xhat = hf * r
    gw = g * weight.float()
    dx = (gw - xhat * (gw * xhat).mean(dim=1, keepdim=True)) * r
    if dh is not None:
        dx = dx + dh.float()
    return {"dx": dx.to(h.dtype), "dweight": (g * xhat).sum(dim=0).to(weight.dtype)}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op in ("fwd", "dx"):
        # the weight as a program keeps it, and the left operand as a norm or a
        # quantize call has just left it
        w = _plain_quantize(_normal(gen, (case["n"], k), 0.02, torch.float32), 128)
        if op == "fwd":
            a = _plain_quantize(_activations(gen, m, k, torch.bfloat16), 1)
        else:
            a = _plain_quantize(_normal(gen, (m, case["n"]), 0.01, torch.bfloat16), 1)
        return dict(case=case, a=a, w=w)
    if op == "norm":
        x = _activations(gen, m, k, TYPES[case["x"]])
        res = None if case["residual"] == "none" else _activations(gen, m, k, TYPES[case["residual"]])
        return dict(case=case, x=x, residual=res,
                    weight=1.0 + _normal(gen, (k,), 0.1, torch.float32))
    if op == "norm_bwd":
        t = TYPES[case["x"]]
        h = _activations(gen, m, k, t)
        rstd = torch.rsqrt(h.float().square().mean(dim=1) + EPS)
        return dict(case=case, h=h, rstd=rstd, dy=_normal(gen, (m, k), 0.01, t),
                    dh=_normal(gen, (m, k), 0.01, t) if case["dh"] else None,
                    weight=(1.0 + _normal(gen, (k,), 0.1, torch.float32)).to(TYPES[case["w"]]))
    if case["rows"] == 1:
        return dict(case=case, x=_activations(gen, m, k, TYPES[case["x"]]))
    return dict(case=case, x=_normal(gen, (m, k), 0.02, TYPES[case["x"]]))


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import dequant_gemm_gb300 as nf4
        if op in ("fwd", "dx"):
            a, w = nf4.FP8Tensor(*state["a"]), nf4.FP8Tensor(*state["w"], block_rows=128)
            call = nf4.nf4_fp8_matmul_fwd if op == "fwd" else nf4.nf4_fp8_matmul_bwd_dx
            return call(a, w, out_dtype=TYPES[case["out"]])
        if op == "norm":
            y, h, rstd = nf4.nf4_rmsnorm_fwd(state["x"], state["weight"], state["residual"], eps=EPS,
                                             out_dtype=TYPES[case["out"]], save_rstd=case["rstd"])
            got = {"codes": y.codes, "scale": y.scale} if case["out"] == "fp8" else {"y": y}
            if state["residual"] is not None:
                got["h"] = h
            if case["rstd"]:
                got["rstd"] = rstd
            return got
        if op == "norm_bwd":
            dx, dweight = nf4.nf4_rmsnorm_bwd(state["dy"], state["h"], state["weight"],
                                              state["rstd"], dh=state["dh"])
            return {"dx": dx, "dweight": dweight}
        q = nf4.nf4_fp8_quantize(state["x"], block_rows=case["rows"])
        return {"codes": q.codes, "scale": q.scale}
    if op == "fwd":
        y = _plain_values(*state["a"], 1) @ _plain_values(*state["w"], 128).t()
        return y.to(TYPES[case["out"]])
    if op == "dx":
        return (_plain_values(*state["a"], 1) @ _plain_values(*state["w"], 128)).to(TYPES[case["out"]])
    if op == "norm":
        return _plain_norm(state["x"], state["residual"], state["weight"], EPS, TYPES[case["out"]],
                           case["rstd"])
    if op == "norm_bwd":
        return _plain_norm_bwd(state["dy"], state["h"], state["weight"], state["rstd"], state["dh"])
    codes, scale = _plain_quantize(state["x"], case["rows"])
    return {"codes": codes, "scale": scale}


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    kb = -(-k // BLOCK)
    if op in ("fwd", "dx"):
        n = case["n"]
        red, cols = (k, n) if op == "fwd" else (n, k)
        b = n * k + 4 * -(-n // BLOCK) * kb + m * red + 4 * m * -(-red // BLOCK)
        return {"bytes": b + m * cols * BYTES[case["out"]], "flops": 2 * m * n * k}
    if op == "norm":
        res = 0 if case["residual"] == "none" else 2 * BYTES[case["residual"]]
        b = m * k * (BYTES[case["x"]] + res + BYTES[case["out"]]) + 4 * k
        b += 4 * m * kb if case["out"] == "fp8" else 0
        return {"bytes": b + (4 * m if case["rstd"] else 0), "flops": 6 * m * k}
    if op == "norm_bwd":
        t = BYTES[case["x"]]
        return {"bytes": m * k * t * (4 if case["dh"] else 3) + 4 * m + 2 * k * BYTES[case["w"]],
                "flops": 10 * m * k}
    return {"bytes": m * k * (BYTES[case["x"]] + 1) + 4 * -(-m // case["rows"]) * kb,
            "flops": 3 * m * k}


# -------------------------------------------------- the definitions, 64 bits --

def _grid(scale, m, k, rows):
    """The scale of every element of an [m, k] matrix."""
    i = torch.arange(m, device=scale.device) // rows
    j = torch.arange(k, device=scale.device) // BLOCK
    return scale.double()[i][:, j]


def _exact_quantize(x, rows):
    m, k = x.shape
    mb, kb = -(-m // rows), -(-k // BLOCK)
    amax = torch.zeros(mb, kb, dtype=torch.float64, device=x.device)
    for j in range(kb):
        col = x[:, BLOCK * j:BLOCK * (j + 1)].abs().amax(dim=1)
        row = torch.arange(m, device=x.device) // rows
        amax[:, j] = amax[:, j].scatter_reduce(0, row, col, "amax")
    amax[amax < MIN_AMAX] = 0.0
    scale = amax / E4M3_MAX
    each = _grid(scale, m, k, rows)
    q = torch.where(each > 0, x / torch.where(each > 0, each, 1.0), 0.0)
    return q.to(FP8), scale


def exact(case, seed):
    state = prepare(case, seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op in ("fwd", "dx"):
        (qa, sa), (qw, sw) = state["a"], state["w"]
        w = qw.double() * _grid(sw, case["n"], k, BLOCK)
        a = qa.double() * _grid(sa, *qa.shape, 1)
        return torch.einsum("mk,nk->mn" if op == "fwd" else "mn,nk->mk", a, w)
    if op == "norm":
        h, got = state["x"].double(), {}
        if state["residual"] is not None:      # the stream is held in the residual's type
            got["h"] = (h + state["residual"].double()).to(state["residual"].dtype)
            h = got["h"] = got["h"].double()
        rms = torch.sqrt(h.pow(2).sum(dim=1) / k + EPS)
        y = h / rms[:, None] * state["weight"].double()
        if case["out"] == "fp8":
            got["codes"], got["scale"] = _exact_quantize(y, 1)
        else:
            got["y"] = y
        if case["rstd"]:
            got["rstd"] = 1.0 / rms
        return got
    if op == "norm_bwd":
        g, h = state["dy"].double(), state["h"].double()
        w, r = state["weight"].double(), state["rstd"].double()[:, None]
        along = (g * w * h).sum(dim=1, keepdim=True) / k
        dx = r * g * w - r.pow(3) * along * h
        if state["dh"] is not None:
            dx = dx + state["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("mk,mk->k", g, h * r)}
    codes, scale = _exact_quantize(state["x"].double(), case["rows"])
    return {"codes": codes, "scale": scale}
