"""The optimizer step over a list of tensors: what is measured, and its plain forms.

Four operators, each over many tensors at once (the tensors of a model as they lie in
memory, each with its own learning-rate scale and weight decay):

  norm    loss-scale removal, overflow check, global gradient norm, clip coefficient and
          the step's scalars
  adamw   AdamW with 32-bit states, and the cast into the 16-bit parameters
  adamw8  AdamW with 8-bit block-scaled states, stochastically rounded, then the states
          read out as values (as a checkpoint or a monitor takes them)
  codec   32-bit states written into the 8-bit form and read back (a checkpoint moved from
          one form to the other)

With `own` false every operator is computed from elementary torch operations in 32 bits
over the arenas that the tensors are views of; with `own` true the framework's entry
points are called on the list of tensors.  exact() gives the same outputs in 64 bits from
the operators' definitions.

The 8-bit form: a tensor is cut into blocks of 256 elements.  A block keeps one exponent
byte b for m and one for v, with the block's largest magnitude <= 1.875 * 2^(b-127).  m is
a sign, 4 exponent and 3 mantissa bits below it, v 5 exponent and 3 mantissa bits; both
have a subnormal binade, and a v > 0 is never rounded to 0.
"""
import math

import numpy as np
import torch

own = False

BETA1, BETA2, EPS, LR, WEIGHT_DECAY, MAX_NORM = 0.9, 0.999, 1e-8, 1e-3, 0.01, 1.0
BLOCK = 256
MASK = 0xFFFFFFFF
GOLDEN = 0x9E3779B9
SEED = 0x1234567890ABCDEF
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def f32(x):
    return float(np.float32(x))


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    gpt2 = dict(kind="stack", layers=48, d=1600, ffn=6400, vocab=50257, positions=1024)
    mid = dict(kind="stack", layers=12, d=640, ffn=2560, vocab=32000, positions=512)
    odd = dict(kind="glu", layers=6, d=641, ffn=1733, vocab=10007, positions=0)
    low = dict(kind="adapter", layers=4, d=512, ffn=4, vocab=0, positions=0)
    vec = dict(kind="vectors", layers=48, d=1600, ffn=6400, vocab=0, positions=0)
    return [
        # fine-tuning of low-rank adapters with fp32 gradients: 16 tensors of 2,048 elements,
        # one call's latency
        dict(name="norm_adapter", op="norm", grad="f32", shift=0, **low),
        # a small model in fp16 with a loss scale, 80 million parameters
        dict(name="norm_small_f16", op="norm", grad="f16", shift=0, **mid),
        # GPT-2 1.5B's 580 tensors, bf16 gradients: one full training step's norm
        dict(name="norm_gpt2_1_5b", op="norm", grad="bf16", shift=0, **gpt2),
        # the adapters' update: fp32 gradients, bf16 parameters
        dict(name="adamw_adapter", op="adamw", grad="f32", shift=0, params="bf16", **low),
        # only the norms and biases of GPT-2 1.5B train: hundreds of short tensors
        dict(name="adamw_vectors", op="adamw", grad="bf16", shift=0, params="bf16", **vec),
        # odd sizes, every buffer off the 16-byte grid: pieces of a flat fp16 buffer
        dict(name="adamw_odd_f16", op="adamw", grad="f16", shift=3, params="f16", **odd),
        # one full training step of GPT-2 1.5B with 32-bit states
        dict(name="adamw_gpt2_1_5b", op="adamw", grad="bf16", shift=0, params="bf16", **gpt2),
        # three of these situations with 8-bit states
        dict(name="adamw8_adapter", op="adamw8", grad="f32", shift=0, params="bf16", **low),
        dict(name="adamw8_odd_f16", op="adamw8", grad="f16", shift=0, params="f16", **odd),
        dict(name="adamw8_gpt2_1_5b", op="adamw8", grad="bf16", shift=0, params="bf16", **gpt2),
        # a checkpoint's 32-bit states into the 8-bit form, and its values back: the adapters,
        # and the small model
        dict(name="codec_adapter", op="codec", grad="f32", shift=0, **low),
        dict(name="codec_small", op="codec", grad="bf16", shift=0, **mid),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        c = dict(op=rng.choice(["norm", "adamw", "adamw8", "codec"]),
                 kind=rng.choice(["stack", "glu", "adapter", "vectors"]),
                 layers=log(1, 48), d=log(17, 2048), vocab=log(50, 50257), positions=log(1, 1024),
                 grad=rng.choice(["bf16", "f16", "f32"]), shift=rng.choice([0, 0, 0, 1, 3, 4, 8]))
        c["ffn"] = log(1, 64) if c["kind"] == "adapter" else rng.choice([4 * c["d"], log(c["d"], 4 * c["d"])])
        if c["op"] in ("adamw", "adamw8"):
            c["params"] = rng.choice(["bf16", "f16"])
        if any(k * c["d"] == 3072 for k in (1, 3, 4)) or c["ffn"] == 3072:
            continue
        if sum(sizes(c)) <= 1_200_000_000:
            return c


def sizes(case):
    """Elements of each tensor, in the model's order."""
    d, ff, n = case["d"], case["ffn"], case["layers"]
    if case["kind"] == "adapter":    # two pairs of rank-ffn matrices a layer
        return [ff * d] * (4 * n)
    if case["kind"] == "vectors":    # the norms and biases of `stack`
        return [d, d, 3 * d, d, d, d, ff, d] * n + [d, d]
    if case["kind"] == "glu":        # no biases, a gated MLP, an untied head
        layer = [d * d] * 4 + [ff * d, ff * d, d * ff, d, d]
        return [case["vocab"] * d] + layer * n + [d, case["vocab"] * d]
    layer = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, d * ff, ff, ff * d, d]
    return [case["vocab"] * d, case["positions"] * d] + layer * n + [d, d]


def work(case):
    e = sum(sizes(case))
    blocks = sum(-(-n // BLOCK) for n in sizes(case))
    g = 4 if case["grad"] == "f32" else 2
    if case["op"] == "norm":         # the gradients, once
        return {"bytes": e * g, "flops": 3 * e}
    if case["op"] == "adamw":        # gradient, master, m, v in; master, m, v, parameter out
        return {"bytes": e * (g + 12 + 12 + 2), "flops": 14 * e}
    if case["op"] == "adamw8":       # 4-byte master, 1-byte m and v; the values in bf16
        return {"bytes": e * (g + 6 + 6 + 2 + 4) + 4 * blocks, "flops": 16 * e}
    return {"bytes": e * (8 + 2 + 4) + 2 * blocks, "flops": 4 * e}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def scalars(case):
    """The step's scalars as the norm leaves them, in fp32 values: step t = 1000."""
    t = 1000
    b1, b2 = f32(BETA1), f32(BETA2)
    return dict(t=t, c=f32(0.731), inv_scale=1.0 / loss_scale(case), b1=b1, b2=b2,
                omb1=float(np.float32(1) - np.float32(b1)), omb2=float(np.float32(1) - np.float32(b2)),
                step=f32(f32(LR) / (1.0 - b1 ** t)), rbc2=f32(math.sqrt(1.0 - b2 ** t)), eps=f32(EPS))


def loss_scale(case):
    return 1024.0 if case["grad"] == "f16" else 1.0


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    size, op, shift = sizes(case), case["op"], case["shift"]
    padded = [-(-n // BLOCK) * BLOCK for n in size]
    off = [0]
    for n in padded:
        off.append(off[-1] + n)
    total, elems = off[-1], sum(size)
    # every tensor is a view of an arena, on a block boundary past the arena's start; the
    # arena itself starts `shift` elements off the allocation
    spans = [(o, n) for o, n in zip(off, size)]
    s = dict(op=op, case=dict(case), spans=spans, blocks=total // BLOCK, sc=scalars(case))

    def arena(dtype, sigma=None, square=False):
        a = torch.empty(total + shift, dtype=dtype, device=dev)[shift:]
        a.zero_() if sigma is None else a.normal_(0.0, sigma, generator=gen)
        if square:
            a.square_()
        for (o, n), p in zip(spans, padded):
            if p > n:
                a[o + n:o + p].zero_()
        return a

    sigma = 2.0 / math.sqrt(elems)   # a gradient norm of 2: the clip bites
    if op != "codec":
        s["grad"] = arena(DTYPES[case["grad"]], sigma * loss_scale(case))
        if case["kind"] in ("stack", "glu"):   # half of the embedding's rows saw no token
            s["grad"][:size[0] // 2].zero_()
    if op in ("adamw", "adamw8"):
        s["master"] = arena(torch.float32, 0.02)
        s["params"] = arena(DTYPES[case["params"]])
    if op != "norm":
        s["m"] = arena(torch.float32, sigma)
        s["v"] = arena(torch.float32, sigma, square=True)
    if op in ("adamw8", "codec"):
        s["values_m"], s["values_v"] = arena(torch.bfloat16), arena(torch.bfloat16)
        s["codes_m"], s["codes_v"] = arena(torch.uint8), arena(torch.uint8)
        s["exps"] = torch.zeros(total // BLOCK, 2, dtype=torch.uint8, device=dev)
    if op == "adamw8":               # the states of a run under way, in their 8-bit form
        half = 1 << 19
        s["codes_m"].view(-1, BLOCK)[:], s["exps"][:, 0] = encode_m(s["m"].view(-1, BLOCK), half)
        s["codes_v"].view(-1, BLOCK)[:], s["exps"][:, 1] = encode_v(s["v"].view(-1, BLOCK), half)
        del s["m"], s["v"]
    # vectors have no weight decay, an embedding half the learning rate
    longest = 4 * max(case["d"], case["ffn"])
    decay = [WEIGHT_DECAY if n > longest else 0.0 for n in size]
    scale = [0.5 if k == 0 and case["kind"] in ("stack", "glu") else 1.0 for k in range(len(size))]
    if op in ("adamw", "adamw8"):
        per = torch.tensor([[p // BLOCK for p in padded]], device=dev)[0]
        fac = [f32(1.0 - f32(LR) * f32(r) * f32(w)) for r, w in zip(scale, decay)]
        s["block_step"] = torch.repeat_interleave(torch.tensor(
            [f32(s["sc"]["step"] * r) for r in scale], device=dev), per)[:, None]
        s["block_decay"] = torch.repeat_interleave(torch.tensor(fac, device=dev), per)[:, None]
        s["rbc2"] = torch.tensor(s["sc"]["rbc2"], device=dev)
    s["t"] = torch.tensor([s["sc"]["t"]], dtype=torch.int32, device=dev)
    s["b1"], s["b2"] = (torch.tensor(s["sc"][k], device=dev) for k in ("b1", "b2"))
    s["jump"] = [torch.tensor(x, device=dev) for x in zip(*jumps(16))]
    if own:
        prepare_own(s, dev, scale, decay)
    return s


def prepare_own(s, dev, scale, decay):
    """The handles a user's program keeps: the lists of tensors and the step state."""
    import zero_partitioned_optimizer_shard_gb300 as z
    names = [k for k in ("grad", "master", "params") if k in s]
    cut = lambda a: [a[o:o + n] for o, n in s["spans"]]  # noqa: E731
    lists = {k: cut(s[k]) for k in names}
    if s["op"] in ("adamw8", "codec"):
        exps = [s["exps"][o // BLOCK:o // BLOCK + -(-n // BLOCK)] for o, n in s["spans"]]
        s["list"] = z.TensorList(m=cut(s["codes_m"]), v=cut(s["codes_v"]), exps=exps, lr_scale=scale,
                                 weight_decay=decay, **lists)
        s["values"] = z.TensorList(m=cut(s["values_m"]), v=cut(s["values_v"]))
        if s["op"] == "codec":
            s["list32"] = z.TensorList(m=cut(s["m"]), v=cut(s["v"]))
    else:
        if s["op"] == "adamw":
            lists.update(m=cut(s["m"]), v=cut(s["v"]))
        s["list"] = z.TensorList(lr_scale=scale, weight_decay=decay, **lists)
    sc = s["sc"]
    s["hp"] = z.hparams(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=WEIGHT_DECAY, max_grad_norm=MAX_NORM)
    s["st"] = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device=dev)
    s["work"] = torch.empty(z.zero_tensors_workspace_bytes(len(s["spans"])), dtype=torch.uint8, device=dev)
    z.zero_tensors_state_init(1, 1.0 / sc["inv_scale"], False, 0, s["st"])
    st = z.zero_step_state_read(s["st"])
    st.t, st.clip_coef, st.inv_scale_used, st.step_size, st.rbc2 = sc["t"], sc["c"], sc["inv_scale"], sc["step"], sc["rbc2"]
    z.zero_step_state_write(s["st"], st)


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        return run_own(s)
    return {"norm": plain_norm, "adamw": plain_adamw, "adamw8": plain_adamw8, "codec": plain_codec}[s["op"]](s)


def run_own(s):
    import zero_partitioned_optimizer_shard_gb300 as z
    if s["op"] == "norm":
        z.zero_tensors_grad_norm(s["list"], s["hp"], s["work"], s["st"])
        f, i, at = s["st"].view(torch.float32), s["st"].view(torch.int32), lambda x: x.offset // 4
        one = lambda a, x: a[at(x):at(x) + 1]  # noqa: E731
        return {"norm": s["st"].view(torch.float64)[1:2].float(), "clip_coef": one(f, z.StepState.clip_coef),
                "step_size": one(f, z.StepState.step_size), "rbc2": one(f, z.StepState.rbc2),
                "skip": one(i, z.StepState.skip), "t": one(i, z.StepState.t)}
    if s["op"] == "adamw":
        z.zero_tensors_adamw(s["list"], s["hp"], s["st"])
        return {k: s[k] for k in ("master", "m", "v", "params")}
    if s["op"] == "adamw8":
        z.zero_tensors_adamw8(s["list"], s["hp"], SEED, s["st"])
        z.zero_tensors_state8_read(s["list"], s["values"])
        return {k: s[k] for k in ("master", "params", "values_m", "values_v")}
    z.zero_tensors_state8_write(s["list"], s["list32"])
    z.zero_tensors_state8_read(s["list"], s["values"])
    return {k: s[k] for k in ("values_m", "values_v")}


def plain_norm(s):
    sc = s["sc"]
    g = s["grad"].float() * sc["inv_scale"]
    skip = (~torch.isfinite(g)).any().reshape(1).int()
    norm = torch.sqrt((g * g).sum()).reshape(1)
    clip = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
    s["t"] += 1 - skip
    return {"norm": norm, "clip_coef": torch.where(skip > 0, torch.ones_like(clip), clip),
            "step_size": f32(LR) / (1.0 - s["b1"] ** s["t"]), "rbc2": torch.sqrt(1.0 - s["b2"] ** s["t"]),
            "skip": skip, "t": s["t"]}


def moments(s, m, v):
    """Both moments after this step, and the clipped gradient's part in them."""
    sc = s["sc"]
    gc = (s["grad"].view(-1, BLOCK).float() * sc["inv_scale"]) * sc["c"]
    return m * sc["b1"] + gc * sc["omb1"], v * sc["b2"] + (gc * gc) * sc["omb2"]


def plain_adamw(s):
    m, v, p = (s[k].view(-1, BLOCK) for k in ("m", "v", "master"))
    m1, v1 = moments(s, m, v)
    denom = torch.sqrt(v1) / s["rbc2"] + s["sc"]["eps"]
    m.copy_(m1)
    v.copy_(v1)
    p.copy_(p * s["block_decay"] - s["block_step"] * (m1 / denom))
    s["params"].copy_(s["master"])
    return {k: s[k] for k in ("master", "m", "v", "params")}


def plain_adamw8(s):
    p, exps = s["master"].view(-1, BLOCK), s["exps"]
    codes_m, codes_v = s["codes_m"].view(-1, BLOCK), s["codes_v"].view(-1, BLOCK)
    m1, v1 = moments(s, decode_m(codes_m, exps[:, :1]), decode_v(codes_v, exps[:, 1:]))
    denom = torch.sqrt(v1) * (1.0 / s["rbc2"]) + s["sc"]["eps"]
    p.copy_(p * s["block_decay"] - s["block_step"] * (m1 / denom))
    s["params"].copy_(s["master"])
    codes_m[:], exps[:, 0] = encode_m(m1, random20(s, 1))
    codes_v[:], exps[:, 1] = encode_v(v1, random20(s, 9))
    return read_values(s)


def plain_codec(s):
    half = 1 << 19                   # to the nearest code
    s["codes_m"].view(-1, BLOCK)[:], s["exps"][:, 0] = encode_m(s["m"].view(-1, BLOCK), half)
    s["codes_v"].view(-1, BLOCK)[:], s["exps"][:, 1] = encode_v(s["v"].view(-1, BLOCK), half)
    return {k: x for k, x in read_values(s).items() if k.startswith("values")}


def read_values(s):
    s["values_m"].view(-1, BLOCK).copy_(decode_m(s["codes_m"].view(-1, BLOCK), s["exps"][:, :1]))
    s["values_v"].view(-1, BLOCK).copy_(decode_v(s["codes_v"].view(-1, BLOCK), s["exps"][:, 1:]))
    return {k: s[k] for k in ("master", "params", "values_m", "values_v") if k in s}


def mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & MASK
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & MASK
    return x ^ (x >> 16)


def jumps(n):
    """(a, c) for k = 1 .. n: the generator's k-th output is a * seed + c."""
    a, c, steps = 1, 0, []
    for _ in range(n):
        a, c = (a * 1664525) & MASK, (c * 1664525 + 1013904223) & MASK
        steps.append((a, c))
    return steps


def random20(s, first):
    """20 random bits for each element: outputs first .. first+7 of the generator of each
    group of 8 elements."""
    dev = s["master"].device
    key = mix(mix(((SEED & MASK) + s["sc"]["t"] * GOLDEN) & MASK) ^ (SEED >> 32))
    seed = mix((torch.arange(s["blocks"] * 32, device=dev) * GOLDEN + key) & MASK)
    mul, add = (x[first - 1:first + 7] for x in s["jump"])
    r = seed[:, None] * mul
    r += add
    r &= MASK
    r >>= 12
    return r.to(torch.int32).view(-1, BLOCK)


def block_exponent(x):
    top = x.amax(1, keepdim=True)
    b = ((top.view(torch.int32) + 0xFFFFF) >> 23).clamp(27, 253)
    return torch.where(top > 0, b, torch.zeros_like(b))


def encode_m(x, r):
    a = x.abs()
    b = block_exponent(a)
    y = (a * ((254 - b) << 23).view(torch.float32)) * 2.0 ** -112
    c = ((y.view(torch.int32) + r) >> 20).clamp(max=127)
    return (c | ((x.view(torch.int32) >> 24) & 0x80)).to(torch.uint8), b[:, 0].to(torch.uint8)


def encode_v(x, r):
    b = block_exponent(x)
    y = (x * ((254 - b) << 23).view(torch.float32)) * 2.0 ** -96
    c = torch.maximum(((y.view(torch.int32) + r) >> 20).clamp(max=255), (x > 0).int())
    return c.to(torch.uint8), b[:, 0].to(torch.uint8)


def decode_m(c, b):
    c = c.to(torch.int32)
    y = ((c & 0x7F) << 20).view(torch.float32) * 2.0 ** 112 * (b.to(torch.int32) << 23).view(torch.float32)
    return torch.where(c >= 0x80, -y, y)


def decode_v(c, b):
    return (c.to(torch.int32) << 20).view(torch.float32) * 2.0 ** 96 * (b.to(torch.int32) << 23).view(torch.float32)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    sc, op = s["sc"], case["op"]
    if op == "norm":
        total = sum(float((part.double() * sc["inv_scale"]).square().sum()) for part in s["grad"].split(1 << 26))
        t, norm = sc["t"] + 1, math.sqrt(total)
        one = lambda x: torch.tensor([x], dtype=torch.float64)  # noqa: E731
        return {"norm": one(norm), "clip_coef": one(min(1.0, MAX_NORM / (norm + 1e-6))),
                "step_size": one(f32(LR) / (1.0 - sc["b1"] ** t)), "rbc2": one(math.sqrt(1.0 - sc["b2"] ** t)),
                "skip": None, "t": None}
    names = {"adamw": ("master", "m", "v", "params"), "adamw8": ("master", "params", "values_m", "values_v"),
             "codec": ("values_m", "values_v")}[op]
    n = s["blocks"] * BLOCK
    out = {k: torch.empty(n, dtype=torch.float64, device=s["t"].device) for k in names}
    for lo in range(0, n, 1 << 25):
        hi = min(n, lo + (1 << 25))
        for k, x in exact_part(s, op, lo, hi).items():
            out[k][lo:hi] = x
    return out


def exact_part(s, op, lo, hi):
    """Elements [lo, hi) of the outputs: whole blocks."""
    sc, rows = s["sc"], slice(lo // BLOCK, hi // BLOCK)
    if op == "codec":
        return {"values_m": nearest(s["m"][lo:hi].double(), 4, None), "values_v": nearest(s["v"][lo:hi].double(), 5, None)}
    if op == "adamw":
        m, v = s["m"][lo:hi].double(), s["v"][lo:hi].double()
    else:
        m = value_of(s["codes_m"][lo:hi], s["exps"][rows, 0], 4)
        v = value_of(s["codes_v"][lo:hi], s["exps"][rows, 1], 5)
    g = s["grad"][lo:hi].double() * (sc["inv_scale"] * sc["c"])
    m = sc["b1"] * m + sc["omb1"] * g
    v = sc["b2"] * v + sc["omb2"] * g ** 2
    rate = s["block_step"][rows].double().expand(-1, BLOCK).reshape(-1)
    keep = s["block_decay"][rows].double().expand(-1, BLOCK).reshape(-1)
    p = keep * s["master"][lo:hi].double() - rate * m / (v.sqrt() / sc["rbc2"] + sc["eps"])
    if op == "adamw":
        return {"master": p, "m": m, "v": v, "params": p}
    return {"master": p, "params": p, "values_m": nearest(m, 4, uniform(s, lo, hi, 0)),
            "values_v": nearest(v, 5, uniform(s, lo, hi, 8))}


def value_of(code, b, exponent_bits):
    """The value a code stands for: the block's power of two times a small float whose top
    exponent is 0."""
    code = code.long()
    sign = 1.0 - 2.0 * (code >> 7).double() if exponent_bits == 4 else torch.ones_like(code, dtype=torch.float64)
    e = (code >> 3) & ((1 << exponent_bits) - 1)
    top = (1 << exponent_bits) - 1
    small = (code & 7).double() / 8 + (e > 0)
    power = torch.pow(2.0, (e.clamp(min=1) - top).double())
    b = b.double()[:, None].expand(-1, BLOCK).reshape(-1)
    return torch.where(b > 0, sign * small * power * torch.pow(2.0, b - 127), torch.zeros_like(small))


def nearest(x, exponent_bits, u):
    """x in the block form: rounded up where the fraction past the lower neighbour and u
    make 1 (u uniform in [0, 1): unbiased; None: one half)."""
    mag = x.abs().view(-1, BLOCK)
    top = mag.amax(1, keepdim=True)
    frac, e = torch.frexp(top)       # top = frac * 2^e, frac in [0.5, 1)
    e = (e + (frac > 0.9375) - 1).clamp(27 - 127, 253 - 127)
    unit = torch.pow(2.0, e.double())
    span = (1 << exponent_bits) - 1
    y = mag / unit
    own_e = (torch.frexp(y)[1] - 1).clamp(1 - span, 0)
    step = torch.pow(2.0, own_e.double() - 3)
    q = torch.floor(y / step + (0.5 if u is None else u.view(-1, BLOCK))) * step
    q = q.clamp(max=1.875)
    if exponent_bits == 5:
        q = torch.where(mag > 0, q.clamp(min=2.0 ** (1 - span - 3)), q)
    return (torch.sign(x).view(-1, BLOCK) * q * unit).view(-1)


def uniform(s, lo, hi, skip):
    """The random fractions of elements [lo, hi): the generator of each group of 8, run
    element by element past its first `skip` outputs."""
    def scramble(h):
        h = torch.bitwise_xor(h, torch.div(h, 65536, rounding_mode="floor"))
        h = torch.remainder(h * 1779033703, 4294967296)
        h = torch.bitwise_xor(h, torch.div(h, 32768, rounding_mode="floor"))
        h = torch.remainder(h * 3144134277, 4294967296)
        return torch.bitwise_xor(h, torch.div(h, 65536, rounding_mode="floor"))

    key = torch.tensor(((SEED % 2 ** 32) + s["sc"]["t"] * 2654435769) % 2 ** 32)
    key = scramble(torch.bitwise_xor(scramble(key), torch.tensor(SEED // 2 ** 32)))
    groups = torch.arange(lo // 8, hi // 8, device=s["t"].device)
    h = scramble(torch.remainder(groups * 2654435769 + int(key), 4294967296))
    columns = []
    for k in range(skip + 8):
        h = torch.remainder(h * 1664525 + 1013904223, 4294967296)
        if k >= skip:
            columns.append(torch.div(h, 4096, rounding_mode="floor").double() / 1048576)
    return torch.stack(columns, 1).reshape(-1)
