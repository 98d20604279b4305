"""The optimizer-step operators that are measured, in their plain form and through the library.

Three operators, over lists of tensors as a model has them:

norm     the global 2-norm of the gradients and the clip factor min(1, max_norm / norm);
adamw    AdamW with 32-bit moments over every tensor of a list, whatever its types;
adamw8   the same with the moments in 8 bits: m and r = sqrt(v) as e4m3 codes with a scale for each block of 256.

``step`` cases run norm and then the update that takes its clip factor and step number, the matrices with 8-bit
states and the vectors with 32-bit ones, as a training loop does.

A case's ``tensors`` text lists the sizes: "65*4096,524288000" (repeats), or "ragged:COUNT:TOTAL:KEY" for COUNT odd
sizes that add up to about TOTAL.  All tensors of one type live in one flat buffer (a bucket), each starting on a
multiple of 256 elements, which is what a data-parallel trainer has in hand; the gaps hold zeros and stay zero.
"""

import math
import random

import torch

own = False

BLOCK = 256          # elements that share a scale
TOP = 448.0          # largest e4m3 value
LEAST = 2.0 ** -9    # smallest e4m3 value above zero
TINY = 2.0 ** -100   # a block whose largest value is below this holds zeros
LR, B1, B2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1
SEED = 20251
T0 = 1000            # updates done before the measured one
MAX_NORM = 1.0


def listed():
    return [
        # the norm weights of a 32-layer model alone: nothing but latency
        {"name": "norm: 65 norm weights", "op": "norm", "tensors": "65*4096", "param": "f32", "grad": "f32"},
        # a model of odd widths, bf16 matrices beside fp32 vectors
        {"name": "norm: ragged, mixed types", "op": "norm", "tensors": "ragged:301:20000003:5", "param": "mixed",
         "grad": "same"},
        # embedding, head and norm weights of an 8B-style model
        {"name": "norm: 8B non-matrix set", "op": "norm", "tensors": "2*524288000,65*4096", "param": "bf16",
         "grad": "bf16"},
        # norm weights again, updated
        {"name": "adamw: 65 norm weights", "op": "adamw", "tensors": "65*4096", "param": "bf16", "grad": "bf16"},
        # fp32 master parameters with the bf16 gradients of a model of odd widths
        {"name": "adamw: ragged, f32 p, bf16 g", "op": "adamw", "tensors": "ragged:173:30000001:7", "param": "f32",
         "grad": "bf16"},
        # the whole non-matrix set of the 8B-style model
        {"name": "adamw: 8B non-matrix set", "op": "adamw", "tensors": "2*524288000,65*4096", "param": "bf16",
         "grad": "bf16"},
        # biases of a small model: 24 vectors, 8-bit states
        {"name": "adamw8: 24 small vectors", "op": "adamw8", "tensors": "12*768,12*2048", "param": "bf16",
         "grad": "bf16"},
        # fp32 parameters and gradients, odd sizes
        {"name": "adamw8: ragged, f32", "op": "adamw8", "tensors": "ragged:211:25000001:9", "param": "f32",
         "grad": "f32"},
        # experts of one MoE layer under AdamW
        {"name": "adamw8: 48 experts' matrices", "op": "adamw8", "tensors": "48*1572864", "param": "bf16",
         "grad": "bf16"},
        # embedding, head and norm weights, 8-bit states: the case the 8 bits are for
        {"name": "adamw8: 8B non-matrix set", "op": "adamw8", "tensors": "2*524288000,65*4096", "param": "bf16",
         "grad": "bf16"},
        # a whole clipped step: bf16 matrices with 8-bit states, fp32 vectors with 32-bit ones
        {"name": "step: small mixed model", "op": "step", "tensors": "ragged:40:300001:11", "param": "mixed",
         "grad": "same"},
        {"name": "step: mixed model", "op": "step", "tensors": "ragged:387:150000001:13", "param": "mixed",
         "grad": "same"},
    ]


def draw(rng):
    op = rng.choice(["norm", "adamw", "adamw8", "step"])
    total = int(math.exp(rng.uniform(math.log(2e3), math.log(2.5e8))))
    count = max(1, min(int(math.exp(rng.uniform(0.0, math.log(400.0)))), total // 4))
    param = "mixed" if op == "step" else rng.choice(["bf16", "f32", "mixed"])
    return {"op": op, "tensors": "ragged:%d:%d:%d" % (count, total, rng.randrange(10 ** 6)), "param": param,
            "grad": rng.choice(["bf16", "f32", "same"])}


def _sizes(case):
    text = case["tensors"]
    if text.startswith("ragged:"):
        count, total, key = (int(x) for x in text.split(":")[1:])
        r = random.Random(key)
        w = [math.exp(r.uniform(-3.0, 3.0)) for _ in range(count)]
        return [max(1, int(total * x / sum(w))) for x in w]
    out = []
    for part in text.split(","):
        n, _, size = part.rpartition("*")
        out += [int(size)] * int(n or 1)
    return out


def _split(case):
    """Tensor sizes of the bf16 bucket and of the fp32 bucket."""
    sizes = _sizes(case)
    if case["param"] == "bf16":
        return sizes, []
    if case["param"] == "f32":
        return [], sizes
    return [n for i, n in enumerate(sizes) if i % 3], [n for i, n in enumerate(sizes) if i % 3 == 0]


def _bits(case, low):
    """State width of a bucket's tensors."""
    return 8 if case["op"] == "adamw8" or (case["op"] == "step" and low) else 32


def _grad_type(case, low):
    if case["grad"] == "same":
        return torch.bfloat16 if low else torch.float32
    return torch.bfloat16 if case["grad"] == "bf16" else torch.float32


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _bucket(case, sizes, low, gen, first):
    """One bucket's buffers: parameters, gradients, moments and the per-block tables the plain form uses."""
    if not sizes:
        return None
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _padded(n))
    total = starts[-1]
    dev = "cuda"
    inside = torch.zeros(total, dtype=torch.bool, device=dev)
    spread = torch.empty(total // BLOCK, 1, device=dev)
    decay = torch.empty(total // BLOCK, 1, device=dev)
    pick = torch.rand(len(sizes), generator=gen, device=dev).tolist()
    for i, (s, n) in enumerate(zip(starts, sizes)):
        inside[s:s + n] = True
        spread[s // BLOCK:starts[i + 1] // BLOCK] = 10.0 ** (-4.0 + 3.0 * pick[i])  # gradients of one tensor
        decay[s // BLOCK:starts[i + 1] // BLOCK] = DECAY if i % 2 == 0 else 0.0

    def normal():
        return torch.randn(total // BLOCK, BLOCK, generator=gen, device=dev)

    def flat(x):
        return x.view(-1).masked_fill_(~inside, 0.0)

    # runs of 16 blocks that saw no token this step (their gradient is zero), and some that never did
    rows = torch.rand(-(-total // (16 * BLOCK)), 1, generator=gen, device=dev).expand(-1, 16).reshape(-1, 1)
    rows = rows[:total // BLOCK]
    b = {"sizes": sizes, "starts": starts, "total": total, "first": first, "decay": decay,
         "p": flat(normal().mul_(0.02)).to(torch.bfloat16 if low else torch.float32)}
    each = torch.exp(normal()) * spread  # gradient size of each element
    b["g"] = flat(normal().mul_(each).mul_(rows > 0.3)).to(_grad_type(case, low))
    each.mul_(rows > 0.1)
    if case["op"] == "norm":
        return b
    m = flat(normal().mul_(each).mul_(0.3))
    v = flat(each.square_().mul_(normal().abs_().add_(0.3)))
    b["bits"] = _bits(case, low)
    if b["bits"] == 32:
        b["m"], b["v"] = m, v
    else:
        b["cm"], b["sm"] = _nearest(m)
        b["cr"], b["sr"] = _nearest(v.sqrt_())
    return b


def _nearest(x):
    """Codes and scales of a starting moment."""
    x = x.view(-1, BLOCK)
    s = x.abs().amax(1, keepdim=True) / TOP
    return torch.where(s > 0, x / s, 0.0).to(torch.float8_e4m3fn).view(-1), s


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    low, high = _split(case)
    buckets = [_bucket(case, low, True, gen, 0)]
    buckets.append(_bucket(case, high, False, gen, buckets[0]["total"] if low and _bits(case, True) == 8 else 0))
    st = {"op": case["op"], "t": T0, "low": buckets[0], "high": buckets[1]}
    if own:
        _library(st, case)
    return st


def _library(st, case):
    """The handles that a program keeps: the clip and the optimizer over the buckets' tensors."""
    import matrix_aware_optimizer_step_amd as mx
    params, grads, decays, bits = [], [], [], []
    for b in (st["low"], st["high"]):
        if b is None:
            continue
        for i, (s, n) in enumerate(zip(b["starts"], b["sizes"])):
            params.append(b["p"][s:s + n])
            grads.append(b["g"][s:s + n])
            decays.append(DECAY if i % 2 == 0 else 0.0)
            bits.append(b.get("bits", 32))
    control = None
    if case["op"] in ("norm", "step"):
        control = mx.StepControl("cuda", step=T0)
        st["clip"] = mx.GradClip(grads, max_norm=MAX_NORM, control=control)
    if case["op"] == "norm":
        return
    opt = mx.AdamWMulti(params, grads, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decays, state_bits=bits,
                        seed=SEED, control=control)
    opt.t = T0
    at8 = at32 = 0
    for b in (st["low"], st["high"]):
        if b is None:
            continue
        n = b["total"]
        if b["bits"] == 8:
            opt.codes_m[at8:at8 + n] = b.pop("cm")
            opt.codes_r[at8:at8 + n] = b.pop("cr")
            opt.scales[at8 // BLOCK:(at8 + n) // BLOCK] = torch.cat([b.pop("sm"), b.pop("sr")], 1)
            at8 += n
        else:
            opt.exp_avg[at32:at32 + n] = b.pop("m")
            opt.exp_avg_sq[at32:at32 + n] = b.pop("v")
            at32 += n
    st["opt"] = opt


def run(st):
    out = {}
    if own:
        if "clip" in st:
            st["clip"].step()
            c = st["clip"].control
            out = {"norm": c.norm, "scale": c.scale, "step": c.step}
        if "opt" in st:
            o = st["opt"]
            o.step()
            out |= {"p_low": st["low"] and st["low"]["p"], "p_high": st["high"] and st["high"]["p"], "m": o.exp_avg,
                    "v": o.exp_avg_sq, "codes_m": o.codes_m, "codes_r": o.codes_r, "scales": o.scales}
        return out
    st["t"] += 1
    low, high, scale = st["low"], st["high"], 1.0
    if st["op"] in ("norm", "step"):
        norm = (_sumsq(low) + _sumsq(high)).sqrt().float()
        scale = (MAX_NORM / norm).clamp(max=1.0)
        out = {"norm": norm, "scale": scale, "step": st["t"]}
    if st["op"] != "norm":
        a, b = _update(low, st["t"], scale), _update(high, st["t"], scale)
        out |= {"p_low": low and low["p"], "p_high": high and high["p"]}
        for key in ("m", "v", "codes_m", "codes_r", "scales"):
            out[key] = _join(a.get(key), b.get(key))
    return out


def _join(a, b):
    return b if a is None else a if b is None else torch.cat([a, b])


# ------------------------------------------------------------ plain forms

def _sumsq(b):
    """Sum of squares of a bucket's gradients; long sums in 64 bits."""
    return torch.zeros((), dtype=torch.float64, device="cuda") if b is None else b["g"].double().square().sum()


def _update(b, t, scale):
    """AdamW on one bucket, in 32 bits, its buffers updated in place."""
    if b is None:
        return {}
    g = b["g"].float() * scale
    if b["bits"] == 32:
        m, v = b["m"], b["v"]
    else:
        m = (b["cm"].float().view(-1, BLOCK) * b["sm"]).view(-1)
        v = (b["cr"].float().view(-1, BLOCK) * b["sr"]).square_().view(-1)
    m = m * B1 + g * (1 - B1)
    v = v * B2 + g * g * (1 - B2)
    r = v.sqrt()
    step = LR / (1 - B1 ** t) * m / (r / math.sqrt(1 - B2 ** t) + EPS)
    keep = b["p"].float().view(-1, BLOCK) * (1 - LR * b["decay"])
    b["p"].copy_((keep - step.view(-1, BLOCK)).view(-1))
    if b["bits"] == 32:
        b["m"].copy_(m)
        b["v"].copy_(v)
        return {"m": b["m"], "v": b["v"]}
    um, ur = _random(b["first"], b["total"], t, m.device)
    b["cm"], b["sm"] = _encode(m, um, 0.0)
    b["cr"], b["sr"] = _encode(r, ur, LEAST)
    return {"codes_m": b["cm"], "codes_r": b["cr"], "scales": torch.cat([b["sm"], b["sr"]], 1)}


def _mix(x):
    """A 32-bit mixing function on int32 (products wrap)."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * (0xBB67AE85 - (1 << 32))
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * (0x9E3779B9 - (1 << 32))
    return x ^ ((x >> 16) & 0xFFFF)


def _random(first, total, t, device):
    """20 random bits for each element's m and r, from its position, the step and the seed."""
    key = _mix(_mix(torch.tensor(t, dtype=torch.int32, device=device)) ^ SEED)
    a = _mix(torch.arange(first // 16, (first + total) // 16, dtype=torch.int32, device=device) ^ key)
    lane = torch.arange(16, dtype=torch.int32, device=device)
    s = (a[:, None] + _mix(a + 0x6A09E667)[:, None] * lane).view(-1)
    return (s >> 12) & 0xFFFFF, ((s & 0xFFFF) << 4) | ((s >> 28) & 0xF)


def _encode(x, u, least):
    """e4m3 codes and scales of x, rounded up or down by the random bits u."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    s = torch.where(top < TINY, 0.0, top / TOP)
    y = x * torch.where(top < TINY, 0.0, TOP / top)
    a = torch.where(y == 0, 0.0, y.abs().clamp(min=least, max=TOP)).view(-1)
    # a value of at least 2^-6 has 20 bits below its third mantissa bit; below it the step is 2^-9
    normal = ((a.view(torch.int32) + u) & -0x100000).view(torch.float32)
    small = torch.floor(a * 512.0 + u * 2.0 ** -20) * LEAST
    a = torch.where(a < 2.0 ** -6, small, normal)
    return torch.copysign(a, x.view(-1)).to(torch.float8_e4m3fn), s


# ------------------------------------------------------------ the work and the exact values

def work(case):
    nbytes = flops = 0
    for low, sizes in zip((True, False), _split(case)):
        n, p, g = sum(sizes), 2 if low else 4, _grad_type(case, low).itemsize
        flops += 2 * n
        nbytes += n * g
        if case["op"] != "norm":
            flops += 18 * n
            blocks = sum(-(-k // BLOCK) for k in sizes)
            nbytes += n * 2 * p + (n * 4 + blocks * 16 if _bits(case, low) == 8 else n * 16)
    return {"bytes": nbytes, "flops": flops}


def exact(case, seed):
    st = prepare(dict(case), seed)
    dev, f64 = "cuda", torch.float64
    t, out, scale = T0 + 1, {}, 1.0
    buckets = [b for b in (st["low"], st["high"]) if b is not None]
    if case["op"] in ("norm", "step"):
        total = 0.0
        for b in buckets:
            for part in b["g"].split(1 << 27):
                d = part.to(f64)
                total = total + torch.dot(d, d).item()
        norm = math.sqrt(total)
        scale = min(1.0, MAX_NORM / norm)
        out = {"norm": torch.tensor(norm, dtype=f64), "scale": torch.tensor(scale, dtype=f64), "step": None}
    if case["op"] == "norm":
        return out
    got = {k: [] for k in ("m", "v", "codes_m", "codes_r", "scales")}
    for name in ("low", "high"):
        b = st[name]
        out["p_" + name] = None
        if b is None:
            continue
        new_p = torch.empty(b["total"], dtype=f64, device=dev)
        kept = {k: torch.empty(b["total"], dtype=f64, device=dev)
                for k in (("m", "v") if b["bits"] == 32 else ("codes_m", "codes_r"))}
        scales = torch.empty(b["total"] // BLOCK, 2, dtype=f64, device=dev)
        for lo in range(0, b["total"], 1 << 26):
            hi = min(b["total"], lo + (1 << 26))
            rows = slice(lo // BLOCK, hi // BLOCK)
            wide = (hi - lo) // BLOCK, BLOCK
            g = b["g"][lo:hi].to(f64) * scale
            if b["bits"] == 32:
                m, v = b["m"][lo:hi].to(f64), b["v"][lo:hi].to(f64)
            else:
                m = (b["cm"][lo:hi].to(f64).view(wide) * b["sm"][rows].to(f64)).view(-1)
                v = (b["cr"][lo:hi].to(f64).view(wide) * b["sr"][rows].to(f64)).view(-1) ** 2
            m = m + (1 - B1) * (g - m)
            v = v + (1 - B2) * (g ** 2 - v)
            m_hat, v_hat = m / (1 - B1 ** t), v / (1 - B2 ** t)
            p = b["p"][lo:hi].to(f64)
            wd = b["decay"][rows].gt(0).to(f64).mul(DECAY).expand(wide).reshape(-1)
            new_p[lo:hi] = p - LR * wd * p - LR * m_hat / (v_hat.sqrt() + EPS)
            if b["bits"] == 32:
                kept["m"][lo:hi], kept["v"][lo:hi] = m, v
                continue
            at = torch.arange(b["first"] + lo, b["first"] + hi, device=dev)
            s = _exact_random(at, t)
            bits = (s // 4096, (s % 65536) * 16 + s // (1 << 28))
            for k, (key, x, least) in enumerate((("codes_m", m, 0.0), ("codes_r", v.sqrt(), LEAST))):
                top = x.abs().view(wide).amax(1, keepdim=True)
                scales[rows, k] = torch.where(top < TINY, 0.0, top / TOP).view(-1)
                y = (x.view(wide) / torch.where(top < TINY, math.inf, top / TOP)).view(-1)
                a = torch.where(y == 0, 0.0, y.abs().clamp(least, TOP))
                quantum = torch.ldexp(torch.ones_like(a), (torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
                kept[key][lo:hi] = torch.sign(x) * quantum * torch.floor(a / quantum + bits[k].to(f64) / (1 << 20))
        out["p_" + name] = new_p
        for k, x in kept.items():
            got[k].append(x)
        if b["bits"] == 8:
            got["scales"].append(scales)
    return out | {k: torch.cat(x) if x else None for k, x in got.items()}


def _exact_random(at, t):
    """The 32 random bits of the elements at these positions, in 64-bit integers."""
    word = (1 << 32) - 1

    def mix(x):
        x = x ^ (x >> 16)
        x = _times(x, 0xBB67AE85)
        x = x ^ (x >> 15)
        x = _times(x, 0x9E3779B9)
        return x ^ (x >> 16)

    a = mix((at // 16) ^ mix(mix(torch.tensor(t, device=at.device)) ^ SEED))
    return (a + (at % 16) * mix((a + 0x6A09E667) & word)) & word


def _times(x, k):
    """x * k modulo 2^32, x below 2^32, no product past 63 bits."""
    word = (1 << 32) - 1
    return ((x * (k & 0xFFFF)) + (((x * (k >> 16)) & 0xFFFF) << 16)) & word
