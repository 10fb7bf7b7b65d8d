"""The operators around the hash-grid encoder's residual head, case by case: how each is called, its plain form in
elementary torch operations, and its definition in 64 bits.

  linear      y = act(x W^T + b) + r, forward and backward, 16-bit operands, or 8-bit ones with scales
  rms_norm    y = s / sqrt(mean(s^2) + eps) * w of s = x + r, forward (16-bit or 8-bit output) and backward
  adamw       one AdamW step over many tensors, moments in 32 bits or in 8 bits with block exponents
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "f8": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "f8": 1}
ACTS = ("none", "relu", "silu", "gelu_tanh")
EPS = 1e-6
F8_MAX = 448.0
BETA1, BETA2, ADAM_EPS = 0.9, 0.99, 1e-15  # the tables' usual Adam constants
BLOCK = 256                                # values that share one exponent in an 8-bit moment
TABLE = 1 << 20                            # values of one level's table at the standard grid (T = 2^19, F = 2)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One point asked of a trained head: the page's 96-wide input (32 encoded features + a 64-wide code); latency.
        dict(name="linear one point", op="linear", m=1, k=96, n=64, type="f16", out="f16", act="relu", residual=False, pre=False, pad=0),
        # The stem of a training step: 2^18 points' encodings into the head's width, with the pre-activation kept.
        dict(name="linear stem train", op="linear", m=1 << 18, k=32, n=256, type="f16", out="f16", act="silu", residual=False, pre=True, pad=0),
        # A block's product over the ray batch (4096 rays x 256 samples) with its residual: the largest call.
        dict(name="linear block rays", op="linear", m=1 << 20, k=256, n=256, type="bf16", out="bf16", act="silu", residual=True, pre=False, pad=0),
        # The head's 4 outputs in fp32, ragged number of points.
        dict(name="linear outputs ragged", op="linear", m=100003, k=256, n=4, type="bf16", out="f32", act="none", residual=False, pre=False, pad=0),
        # Rendering with a wide 8-bit head.
        dict(name="linear 8-bit wide", op="linear", m=1 << 18, k=512, n=512, type="f8", out="bf16", act="gelu_tanh", residual=True, pre=False, pad=0),
        # Backward of a block's product at the training batch.
        dict(name="linear grad block", op="linear_grad", m=1 << 18, k=256, n=256, type="bf16", act="silu", pad=0),
        # Backward of the coordinate + encoding input (3 + 32 columns): odd rows, odd row length.
        dict(name="linear grad 35 odd", op="linear_grad", m=65537, k=35, n=64, type="f16", act="relu", pad=0),
        # The norm of a training step: residual added, the sum and 1/rms kept for the backward.
        dict(name="norm train", op="norm", m=1 << 18, c=256, type="bf16", out="bf16", residual=True, keep=True, pad=0),
        # The norm in front of an 8-bit product, over the ray batch.
        dict(name="norm 8-bit rays", op="norm", m=1 << 20, c=256, type="bf16", out="f8", residual=True, keep=False, pad=0),
        # Backward of the norm, the residual stream's own gradient added; rows of the 96-wide input.
        dict(name="norm grad", op="norm_grad", m=200003, c=96, type="f16", residual=True, pad=0),
        # A training step's update: 16 tables, 30 head tensors; moments in 32 bits, binary16 copy for the kernels.
        dict(name="adamw tables f32", op="adamw", tables=16, size=TABLE, tensors=30, bits=32, grad="f32", copy="f16"),
        # The same in 8 bits, twice the levels.
        dict(name="adamw tables 8-bit", op="adamw", tables=32, size=TABLE, tensors=30, bits=8, grad="f32", copy="f16"),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def size_of(rng, lo, hi):
    """A size spread over its logarithm: as drawn (mostly odd or ragged), or rounded to a multiple of 32."""
    v = log_int(rng, lo, hi)
    return max(32, v // 32 * 32) if rng.random() < 0.5 and hi >= 32 else v


def draw(rng):
    top = work(listed()[2])
    while True:
        op = rng.choice(["linear", "linear", "linear_grad", "norm", "norm_grad", "adamw"])
        pad = rng.choice([0, 0, 8, 3])  # columns of a wider buffer that the rows are a part of
        if op == "linear":
            t = rng.choice(["f16", "bf16", "f8"])
            out = rng.choice(["f16", "bf16", "f32"]) if t == "f8" else rng.choice([t, t, "f32"])
            c = dict(op=op, m=log_int(rng, 1, 1 << 20), k=size_of(rng, 1, 1024), n=size_of(rng, 1, 1024), type=t, out=out,
                     act=rng.choice(ACTS), residual=rng.random() < 0.5, pre=t != "f8" and rng.random() < 0.3, pad=pad)
        elif op == "linear_grad":
            c = dict(op=op, m=log_int(rng, 1, 1 << 19), k=size_of(rng, 1, 1024), n=size_of(rng, 1, 1024),
                     type=rng.choice(["f16", "bf16"]), act=rng.choice(ACTS), pad=pad)
        elif op == "norm":
            t = rng.choice(["f16", "bf16", "f32"])
            c = dict(op=op, m=log_int(rng, 1, 1 << 20), c=size_of(rng, 1, 4096), type=t, out=rng.choice([t, "f8"]),
                     residual=rng.random() < 0.6, keep=rng.random() < 0.5, pad=pad)
        elif op == "norm_grad":
            c = dict(op=op, m=log_int(rng, 1, 1 << 20), c=size_of(rng, 1, 4096), type=rng.choice(["f16", "bf16", "f32"]),
                     residual=rng.random() < 0.6, pad=pad)
        else:
            c = dict(op=op, tables=rng.randint(0, 16), size=log_int(rng, 1 << 10, TABLE), tensors=rng.randint(1, 80),
                     bits=rng.choice([8, 32]), grad=rng.choice(["f32", "f16", "bf16"]), copy=rng.choice(["none", "f16", "bf16"]))
        w = work(c)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return c


def head_shapes(count):
    """Shapes of a head's parameters: weights, biases and norm weights of blocks of three widths, in turn."""
    kinds = [(256, 32), (256,), (256, 256), (256,), (64, 96), (4, 256), (4,), (64, 35), (33, 7), (1,)]
    return [kinds[i % len(kinds)] for i in range(count)]


def adamw_counts(c):
    return [c["size"]] * c["tables"] + [math.prod(s) for s in head_shapes(c["tensors"])]


def work(case):
    c = case
    if c["op"] == "linear":
        e, o = SIZE[c["type"]], SIZE[c["out"]]
        b = c["m"] * c["k"] * e + c["n"] * c["k"] * e + 4 * c["n"] + c["m"] * c["n"] * o * (2 if c["residual"] else 1)
        b += c["m"] * c["n"] * e if c["pre"] else 0
        b += 4 * (c["m"] + c["n"]) if c["type"] == "f8" else 0
        return {"bytes": b, "flops": 2 * c["m"] * c["k"] * c["n"]}
    if c["op"] == "linear_grad":
        b = 2 * c["m"] * c["n"] * (1 if c["act"] == "none" else 2) + 2 * c["m"] * c["k"] * 2 + 2 * 2 * c["n"] * c["k"] + 4 * c["n"]
        return {"bytes": b, "flops": 4 * c["m"] * c["k"] * c["n"]}
    if c["op"] == "norm":
        e, v = SIZE[c["type"]], c["m"] * c["c"]
        b = v * e * (2 if c["residual"] else 1) + v * SIZE[c["out"]] + 4 * c["c"]
        b += v * e if c["keep"] and c["residual"] else 0
        b += 4 * c["m"] if c["keep"] else 0
        b += 4 * c["m"] if c["out"] == "f8" else 0
        return {"bytes": b, "flops": 6 * v}
    if c["op"] == "norm_grad":
        e, v = SIZE[c["type"]], c["m"] * c["c"]
        return {"bytes": v * e * (4 if c["residual"] else 3) + 8 * c["c"] + 4 * c["m"], "flops": 10 * v}
    total = sum(adamw_counts(c))  # parameter read and written, gradient read, moments read and written, copy written
    per = 8 + SIZE[c["grad"]] + (0 if c["copy"] == "none" else 2) + (16 if c["bits"] == 32 else 4 + 4 / BLOCK)
    return {"bytes": total * per, "flops": 15 * total}


# ------------------------------------------------------------------ inputs

def rows(g, m, n, kind, pad, scale=1.0):
    """[m, n] normal values as columns of a buffer that is `pad` columns wider."""
    t = (torch.randn(m, n + pad, generator=g, device=DEV) * scale).to(TYPES[kind])
    return t[:, :n]


def f8_rows(g, m, k, pad):
    """8-bit rows and their scales, as the norm leaves them (largest value of a row at 448)."""
    v = torch.randn(m, k + pad, generator=g, device=DEV)
    amax = v[:, :k].abs().amax(1).clamp_min(1e-6)
    q = (v * (F8_MAX / amax)[:, None]).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
    return q[:, :k], amax / F8_MAX


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": c}
    if c["op"] in ("linear", "linear_grad"):
        m, k, n, pad = c["m"], c["k"], c["n"], c["pad"]
        bound = 1.0 / math.sqrt(k)
        w = (torch.rand(n, k, generator=g, device=DEV) * 2 - 1) * bound
        s["b"] = (torch.rand(n, generator=g, device=DEV) * 2 - 1) * bound
        if c["type"] == "f8":
            amax = w.abs().amax(1).clamp_min(1e-12)
            s["w"], s["ws"] = (w * (F8_MAX / amax)[:, None]).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn), amax / F8_MAX
            s["x"], s["xs"] = f8_rows(g, m, k, pad)
        else:
            s["w"], s["x"] = w.to(TYPES[c["type"]]), rows(g, m, k, c["type"], pad)
        if c["op"] == "linear":
            s["r"] = rows(g, m, n, c["out"], pad) if c["residual"] else None
        else:
            s["dy"] = rows(g, m, n, c["type"], pad)
            s["z"] = rows(g, m, n, c["type"], pad) if c["act"] != "none" else None
    elif c["op"] == "norm":
        s["x"] = rows(g, c["m"], c["c"], c["type"], c["pad"])
        s["r"] = rows(g, c["m"], c["c"], c["type"], c["pad"]) if c["residual"] else None
        s["w"] = 1 + 0.1 * torch.randn(c["c"], generator=g, device=DEV)
    elif c["op"] == "norm_grad":
        s["s"] = rows(g, c["m"], c["c"], c["type"], c["pad"], 1.4)
        s["rstd"] = 1.0 / torch.sqrt(s["s"].float().square().mean(1) + EPS)
        s["dy"] = rows(g, c["m"], c["c"], c["type"], c["pad"])
        s["ds"] = rows(g, c["m"], c["c"], c["type"], c["pad"]) if c["residual"] else None
        s["w"] = 1 + 0.1 * torch.randn(c["c"], generator=g, device=DEV)
    else:
        s.update(prepare_adamw(c, g))
        s["seed"] = int(seed) & 0x7FFFFFFF
    if own:
        own_plan(s)
    return s


def arena(counts, dtype, per=1):
    """One buffer for the values of every tensor (one value for `per` of them) and each tensor's part of it, 64 values apart at least."""
    sizes = [-(-n // per) for n in counts]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + -(-n // 64) * 64)
    flat = torch.zeros(starts[-1], dtype=dtype, device=DEV)
    return flat, [flat[a:a + n] for a, n in zip(starts, sizes)]


def prepare_adamw(c, g):
    """Tables and head tensors some steps into a training: gradients that are zero where no point came, moments that have seen
    earlier ones. The tensors of a kind lie in one buffer, as a program that saves them together keeps them."""
    counts, eight = adamw_counts(c), c["bits"] == 8
    kinds = {"p": (torch.float32, 1), "g": (TYPES[c["grad"]], 1), "m": (torch.float8_e4m3fn if eight else torch.float32, 1),
             "v": (torch.uint8 if eight else torch.float32, 1)}
    if eight:
        kinds.update(me=(torch.uint8, BLOCK), ve=(torch.uint8, BLOCK))
    if c["copy"] != "none":
        kinds["copy"] = (TYPES[c["copy"]], 1)
    lists = {"flat": {}, "t": 50, "lr": [], "wd": []}
    for k, (dtype, per) in kinds.items():
        lists["flat"][k], lists[k] = arena(counts, dtype, per)
    for i, n in enumerate(counts):
        table = i < c["tables"]
        scale = 1e-4 if table else 1e-2
        touched = (torch.rand(n, generator=g, device=DEV) < 0.7).float() if table else 1.0
        seen = (torch.rand(n, generator=g, device=DEV) < 0.9).float() if table else 1.0
        lists["p"][i].normal_(generator=g).mul_(0.1)
        lists["g"][i].copy_(torch.randn(n, generator=g, device=DEV) * scale * touched)
        m = torch.randn(n, generator=g, device=DEV) * (0.3 * scale) * seen
        v = (torch.randn(n, generator=g, device=DEV).square() * scale ** 2 + m.square()) * seen
        if eight:
            zero = torch.zeros(n, dtype=torch.int64, device=DEV)
            code, e = to_codes(m, *M8, zero)
            lists["m"][i].copy_(code.view(torch.float8_e4m3fn))
            lists["me"][i].copy_(e)
            code, e = to_codes(v, *V8, zero)
            lists["v"][i].copy_(code)
            lists["ve"][i].copy_(e)
        else:
            lists["m"][i].copy_(m)
            lists["v"][i].copy_(v)
        if "copy" in lists:
            lists["copy"][i].copy_(lists["p"][i])
        lists["lr"].append(1e-2 if table else 1e-3)   # the tables' rate is 10 times the head's
        lists["wd"].append(0.0 if table else 1e-2)    # no decay on the tables
    return lists


def part(s, kind, i):
    return s[kind][i] if kind in s else None


# ------------------------------------------------------------------ calls of the framework

def own_plan(s):
    """What a program keeps between steps: the list of tensors an optimizer updates."""
    if s["case"]["op"] == "adamw":
        import multiresolution_hash_grid_amd as hg
        s["plan"] = hg.HashGridAdamWPlan([
            hg.AdamWTensor(param=s["p"][i], grad=s["g"][i], m=s["m"][i], v=s["v"][i], m_exp=part(s, "me", i), v_exp=part(s, "ve", i),
                           copy=part(s, "copy", i), lr=s["lr"][i], weight_decay=s["wd"][i]) for i in range(len(s["p"]))])


def run_own(s):
    import multiresolution_hash_grid_amd as hg
    c = s["case"]
    if c["op"] == "linear":
        return hg.hashgrid_linear_forward(s["x"], s["w"], s["b"], act=c["act"], residual=s["r"], x_scale=s.get("xs"),
                                          weight_scale=s.get("ws"), out_dtype=TYPES[c["out"]], save_pre=c["pre"])
    if c["op"] == "linear_grad":
        return hg.hashgrid_linear_backward(s["dy"], s["x"], s["w"], act=c["act"], pre=s["z"], weight_dtype=TYPES[c["type"]])
    if c["op"] == "norm":
        return hg.hashgrid_rms_norm_forward(s["x"], s["w"], residual=s["r"], eps=EPS, out_dtype=TYPES[c["out"]],
                                            save_sum=c["keep"] and c["residual"], save_rstd=c["keep"])
    if c["op"] == "norm_grad":
        return hg.hashgrid_rms_norm_backward(s["dy"], s["s"], s["w"], s["rstd"], ds=s["ds"])
    s["t"] += 1
    s["plan"].step(step=s["t"], beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, seed=s["seed"] + s["t"])
    return adamw_outputs(s)


def adamw_outputs(s):
    """The updated state, whole. The 8-bit second moments are their codes: equal where their values are."""
    return {k: v for k, v in s["flat"].items() if k != "g"}


# ------------------------------------------------------------------ plain forms

def activate(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
        return z / (1 + torch.exp(-2 * u))
    return z


def slope(z, act):
    """d activate / dz."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    a = math.sqrt(2 / math.pi)
    p = 1 / (1 + torch.exp(-2 * a * (z + 0.044715 * z * z * z)))
    return p + z * p * (1 - p) * 2 * a * (1 + 3 * 0.044715 * z * z)


def run_plain(s):
    c = s["case"]
    if c["op"] == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if c["type"] == "f8":
            z = z * s["xs"][:, None] * s["ws"]
        z = z + s["b"]
        y = activate(z, c["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        y = y.to(TYPES[c["out"]])
        return (y, z.to(TYPES[c["type"]])) if c["pre"] else y
    if c["op"] == "linear_grad":
        dz = s["dy"].float()
        if c["act"] != "none":
            dz = dz * slope(s["z"].float(), c["act"])
        t = TYPES[c["type"]]
        return (dz @ s["w"].float()).to(t), (dz.t() @ s["x"].float()).to(t), dz.sum(0)
    if c["op"] == "norm":
        v = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        rstd = 1 / torch.sqrt((v * v).mean(1) + EPS)
        y = v * rstd[:, None] * s["w"]
        scale = None
        if c["out"] == "f8":
            amax = y.abs().amax(1)
            scale = amax / F8_MAX
            y = torch.where(amax > 0, F8_MAX / amax, torch.zeros_like(amax))[:, None] * y
            y = y.clamp(-F8_MAX, F8_MAX)
        kept = v.to(TYPES[c["type"]]) if c["keep"] and c["residual"] else None
        return y.to(TYPES[c["out"]]), scale, kept, rstd if c["keep"] else None
    if c["op"] == "norm_grad":
        v, dy, r = s["s"].float(), s["dy"].float(), s["rstd"][:, None]
        h = v * r
        dh = dy * s["w"]
        dx = r * (dh - h * (dh * h).mean(1, keepdim=True))
        if s["ds"] is not None:
            dx = dx + s["ds"].float()
        return dx.to(TYPES[c["type"]]), (dy * h).sum(0)
    s["t"] += 1
    for i in range(len(s["p"])):
        adamw_one(s, i)
    return adamw_outputs(s)


# An 8-bit moment: blocks of 256 values share a power of two 2^(e - 127), held as the byte e; a value over it is a small float
# of 8 bits. The first moment: sign, 4 exponent bits (bias 7), 3 mantissa bits (the values of float8_e4m3fn). The second: no
# sign, 5 exponent bits (bias 15), 3 mantissa bits. The block's largest value lies in [2^top, 2^(top + 1)).
M8 = (7, 7)    # bias, top
V8 = (15, 15)


def block_max(a):
    n = a.numel()
    f = torch.zeros(-(-n // BLOCK) * BLOCK, device=a.device, dtype=a.dtype)
    f[:n] = a.reshape(-1)
    return f.view(-1, BLOCK).amax(1)


def per_value(e, like):
    return e.repeat_interleave(BLOCK)[: like.numel()].view(like.shape)


def pow2(k):
    """2^k of whole k in [-126, 127], exactly: the exponent field of a float."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def to_codes(x, bias, top, noise):
    """(codes, block exponents) of x >= 0 or signed; `noise` (20 bits) is added below the last bit kept: stochastic rounding.
    Nonzero values keep a code of at least 1, so that no second moment turns into zero under a first one that is not."""
    a = x.abs()
    bits = block_max(a).view(torch.int32)
    e = torch.where(bits > 0, ((bits >> 23) - top).clamp(1, 254), torch.ones_like(bits))
    k = per_value(e, x).to(torch.int64)
    t = (a * pow2(127 - k)) * 2.0 ** (bias - 127)
    code = (t.view(torch.int32).to(torch.int64) + noise) >> 20
    if bias == 15:
        code = torch.where((code == 0) & (x > 0), torch.ones_like(code), code)
    else:
        code = code | torch.where((x < 0) & (code > 0), 128, 0)
    return code.to(torch.uint8), e.to(torch.uint8)


def from_codes(code, e, bias):
    code = code.view(torch.uint8).to(torch.int32)
    mag = ((code if bias == 15 else code & 127) << 20).view(torch.float32)
    k = per_value(e, code).to(torch.int64)
    x = (mag * 2.0 ** (127 - bias)) * pow2(k - 127)
    return x if bias == 15 else torch.where(code >= 128, -x, x)


def mix(h):
    """A 32-bit finalizer of multiplications and shifts (MurmurHash3's fmix32, public domain), on whole numbers below 2^32."""
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def noise_of(seed, tensor, like):
    """32 random bits of each value: of the step's seed, the tensor's place in the list and the value's place in the tensor."""
    key = mix(torch.tensor([(seed + 0x9E3779B9 * (tensor + 1)) & 0xFFFFFFFF], device=DEV, dtype=torch.int64))
    at = torch.arange(like.numel(), device=DEV, dtype=torch.int64) & 0xFFFFFFFF
    return mix(at ^ key).view(like.shape)


def f32(v):
    return torch.tensor(v, dtype=torch.float32).item()


def adamw_one(s, i):
    t, b1, b2 = s["t"], f32(BETA1), f32(BETA2)
    step = f32(f32(s["lr"][i]) / (1 - b1 ** t))
    root = f32(1 / math.sqrt(1 - b2 ** t))
    keep = f32(1 - f32(s["lr"][i]) * f32(s["wd"][i]))
    p, g = s["p"][i], s["g"][i].float()
    eight = s["case"]["bits"] == 8
    m, v = (from_codes(s["m"][i], s["me"][i], 7), from_codes(s["v"][i], s["ve"][i], 15)) if eight else (s["m"][i], s["v"][i])
    m = m * b1 + g * f32(1 - b1)
    v = v * b2 + (g * g) * f32(1 - b2)
    p.copy_(p * keep - step * m / (torch.sqrt(v) * root + f32(ADAM_EPS)))
    if eight:
        h = noise_of(s["seed"] + t, i, p)
        code, e = to_codes(m, *M8, (h & 0xFFFF) << 4)
        s["m"][i].copy_(code.view(torch.float8_e4m3fn))
        s["me"][i].copy_(e)
        code, e = to_codes(v, *V8, (h >> 16) << 4)
        s["v"][i].copy_(code)
        s["ve"][i].copy_(e)
    else:
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)
    if "copy" in s:
        s["copy"][i].copy_(p)


def run(state):
    return run_own(state) if own else run_plain(state)


# ------------------------------------------------------------------ definitions in 64 bits

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    d = lambda t: t.double()  # noqa: E731
    if c["op"] == "linear":
        x, w = d(s["x"]), d(s["w"])
        if c["type"] == "f8":
            x, w = x * d(s["xs"]).unsqueeze(1), w * d(s["ws"]).unsqueeze(1)
        z = torch.addmm(d(s["b"]), x, w.t())
        if c["act"] == "none":
            y = z
        elif c["act"] == "relu":
            y = z.clamp_min(0)
        elif c["act"] == "silu":
            y = z * torch.sigmoid(z)
        else:
            y = 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
        if c["residual"]:
            y = y + d(s["r"])
        return (y, z) if c["pre"] else y
    if c["op"] == "linear_grad":
        dz = d(s["dy"])
        if c["act"] != "none":
            z = d(s["z"])
            if c["act"] == "relu":
                dz = torch.where(z > 0, dz, 0.0)
            elif c["act"] == "silu":
                p = torch.sigmoid(z)
                dz = dz * (p + z * p * (1 - p))
            else:
                a = (2 / math.pi) ** 0.5
                th = torch.tanh(a * (z + 0.044715 * z ** 3))
                dz = dz * (0.5 * (1 + th) + 0.5 * z * (1 - th * th) * a * (1 + 0.134145 * z * z))
        return dz @ d(s["w"]), d(s["x"]).t().matmul(dz).t(), dz.sum(0)
    if c["op"] == "norm":
        v = d(s["x"]) + (d(s["r"]) if c["residual"] else 0.0)
        rstd = (v.pow(2).sum(1) / c["c"] + EPS).rsqrt()
        y = v * rstd.unsqueeze(1) * d(s["w"])
        scale = None
        if c["out"] == "f8":
            scale = y.abs().max(1).values / F8_MAX
            y = y / scale.unsqueeze(1)
        return y, scale, v if c["keep"] and c["residual"] else None, rstd if c["keep"] else None
    if c["op"] == "norm_grad":
        v, dy, w, r = d(s["s"]), d(s["dy"]), d(s["w"]), d(s["rstd"]).unsqueeze(1)
        g = dy * w * r - v * r.pow(3) * ((dy * w * v).sum(1, keepdim=True) / c["c"])
        return g + (d(s["ds"]) if c["residual"] else 0.0), (dy * v * r).sum(0)
    return exact_adamw(c, s)


def exact_adamw(c, s):
    """Parameters, and moments before they are rounded: 32-bit ones whole, the 8-bit first moment over its block's power of two;
    what is held as whole numbers has no value here."""
    t, eight = s["t"] + 1, c["bits"] == 8
    b1, b2 = f32(BETA1), f32(BETA2)
    out = {k: (None if eight and k in ("v", "me", "ve") else v.double()) for k, v in adamw_outputs(s).items()}
    starts = [x.storage_offset() for x in s["p"]]
    for i, at in enumerate(starts):
        g, p = s["g"][i].double(), s["p"][i].double()
        if eight:
            m = s["m"][i].double() * torch.exp2(per_value(s["me"][i].double() - 127, p))
            code = s["v"][i].double()
            top, low = torch.floor(code / 8), torch.remainder(code, 8)
            small = torch.where(top > 0, (1 + low / 8) * torch.exp2(top - 15), low / 8 * 2.0 ** -14)
            v = small * torch.exp2(per_value(s["ve"][i].double() - 127, p))
        else:
            m, v = s["m"][i].double(), s["v"][i].double()
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        lr, wd = f32(s["lr"][i]), f32(s["wd"][i])
        p = p - lr * wd * p - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + f32(ADAM_EPS))
        span = slice(at, at + p.numel())
        out["p"][span] = p
        if "copy" in out:
            out["copy"][span] = p
        if eight:
            big = torch.frexp(block_max(m.abs())).exponent - 1
            m = m * torch.exp2(7.0 - per_value(big, p).double())
        else:
            out["v"][span] = v
        out["m"][span] = m
    return out
