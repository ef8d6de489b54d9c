"""The operators beside a model's matrix products in training: what is measured, and their plain forms.

Three operators, forward and backward, whose gradients the step over a list of tensors reads:

  layernorm   y = (x - mean) * rstd * weight + bias per row; its gradients, those of weight and
              bias summed over all rows
  embedding   out = scale * table[token]; the table's gradient, a row summed over its tokens
  head_loss   softmax cross entropy of logits = hidden . weight^T over a large vocabulary, the
              logits never kept; the gradients of hidden and weight, times the step state's loss
              scale.  Tokens without a target (-100) have neither loss nor gradient.

With `own` false every operator is computed from elementary torch operations in 32 bits; with
`own` true the framework's entry points are called.  exact() gives the same outputs in 64 bits
from the operators' definitions.
"""
import math

import torch

own = False

EPS = 1e-5
IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
# rows: tokens of the call; d: the model's width; pad: elements between the rows of activations
# (a slice of a wider buffer); grad: the type of the weights' gradients; acc: gradients are added
# to what an earlier micro-batch (or the other end of a tied embedding) left
def listed():
    return [
        # the small example network's layer norm: a batch of 256, width 512, fp32
        dict(name="layernorm_small_f32", op="layernorm", rows=256, d=512, dtype="f32", pad=0),
        # one of GPT-2 1.5B's 97 layer norms, 8 sequences of 1,024
        dict(name="layernorm_gpt2_1_5b", op="layernorm", rows=8192, d=1600, dtype="bf16", pad=0),
        # odd width in a wider fp16 buffer, fp32 gradients summed over micro-batches
        dict(name="layernorm_backward_odd_f16", op="layernorm_backward", rows=4099, d=641, dtype="f16", pad=7,
             grad="f32", acc=True),
        dict(name="layernorm_backward_gpt2_1_5b", op="layernorm_backward", rows=8192, d=1600, dtype="bf16", pad=0,
             grad="bf16", acc=False),
        # a handful of tokens: one call's latency
        dict(name="embedding_few", op="embedding", rows=16, d=1600, vocab=50257, dtype="bf16", scale=1.0, padded=0.0),
        # Llama 7B's embedding, 16 sequences of 1,024, a tenth of the places padding
        dict(name="embedding_llama_7b", op="embedding", rows=16384, d=4096, vocab=32000, dtype="bf16", scale=1.0,
             padded=0.1),
        # odd sizes in fp16, sqrt(d) on the way in
        dict(name="embedding_backward_odd_f16", op="embedding_backward", rows=1023, d=641, vocab=10007, dtype="f16",
             grad="f16", scale=25.3125, padded=0.1, acc=False),
        # GPT-2 1.5B's table, 8 sequences of 1,024: every row of the gradient is written
        dict(name="embedding_backward_gpt2_1_5b", op="embedding_backward", rows=8192, d=1600, vocab=50257, dtype="bf16",
             grad="bf16", scale=1.0, padded=0.0, acc=False),
        # evaluation of a small batch: odd sizes, fp16
        dict(name="head_loss_odd_f16", op="head_loss", rows=131, d=641, vocab=10007, dtype="f16", masked=0.1),
        # perplexity with Llama 7B's head, 4 sequences of 1,024
        dict(name="head_loss_llama_7b", op="head_loss", rows=4096, d=4096, vocab=32000, dtype="bf16", masked=0.0),
        # fine-tuning a small model in fp16 with a loss scale: half of the tokens are prompts
        # without a target, every answer token has a weight of its own
        dict(name="head_train_small_f16", op="head_train", rows=1024, d=640, vocab=32000, dtype="f16", masked=0.5,
             weighted=True, loss_scale=1024.0, acc=False),
        # one micro-batch of GPT-2 1.5B: 8 sequences of 1,024, forward and backward
        dict(name="head_train_gpt2_1_5b", op="head_train", rows=8192, d=1600, vocab=50257, dtype="bf16", masked=0.0,
             weighted=False, loss_scale=1.0, acc=False),
    ]


OPS = ("layernorm", "layernorm_backward", "embedding", "embedding_backward", "head_loss", "head_train")


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        c = dict(op=rng.choice(OPS), rows=log(1, 32768), d=log(8, 4096), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
        if rng.random() < 0.6:
            c["d"] = -(-c["d"] // 8) * 8
        if c["op"].startswith("layernorm"):
            c["pad"] = rng.choice([0, 0, 0, 8, 7])
        else:
            c["vocab"] = log(17, 50257)
        if c["op"].startswith("embedding"):
            c.update(scale=rng.choice([1.0, 1.0, 25.3125]), padded=rng.choice([0.0, 0.1, 0.5]))
        if c["op"] in ("layernorm_backward", "embedding_backward"):
            c["grad"] = rng.choice([c["dtype"], "f32"])
            c["acc"] = rng.random() < 0.4
        if c["op"].startswith("head"):
            if c["dtype"] == "f32":
                continue
            c["masked"] = rng.choice([0.0, 0.0, 0.1, 0.5])
        if c["op"] == "head_train":
            c.update(weighted=rng.random() < 0.4, loss_scale=1024.0 if c["dtype"] == "f16" else 1.0,
                     acc=rng.random() < 0.3)
        w = work(c)
        if w["bytes"] <= 1 << 30 and w["flops"] <= 6 * 8192 * 50257 * 1600:
            return c


def size_of(name):
    return 4 if name == "f32" else 2


def work(case):
    n, d, e = case["rows"], case["d"], size_of(case["dtype"])
    op, v = case["op"], case.get("vocab", 0)
    if op == "layernorm":               # x in, y out, two numbers a row, weight and bias
        return {"bytes": 2 * n * d * e + 8 * n + 2 * d * e, "flops": 8 * n * d}
    g = size_of(case.get("grad", case["dtype"])) * (2 if case.get("acc") else 1)
    if op == "layernorm_backward":      # x and dy in, dx out
        return {"bytes": 3 * n * d * e + 8 * n + d * e + 2 * d * g, "flops": 14 * n * d}
    if op == "embedding":               # the distinct rows in (at most every row of the table), out
        return {"bytes": (min(n, v) + n) * d * e + 8 * n, "flops": n * d}
    if op == "embedding_backward":      # dout in, the table's gradient out (acc: its touched rows)
        touched = min(n, v) if case["acc"] else v
        return {"bytes": n * d * e + 8 * n + touched * d * g, "flops": n * d}
    valid = int(n * (1.0 - case["masked"]))
    if op == "head_loss":               # one product
        return {"bytes": (n + v) * d * e + 16 * n, "flops": 2 * valid * v * d}
    # three products: logits, hidden's gradient, weight's gradient
    return {"bytes": 2 * n * d * e + v * d * (e + g) + 16 * n, "flops": 6 * valid * v * d}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    n, d, v, op, dt = case["rows"], case["d"], case.get("vocab", 0), case["op"], DTYPES[case["dtype"]]
    gdt = DTYPES[case.get("grad", case["dtype"])]

    def normal(*shape, sigma=1.0, dtype=dt):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, sigma, generator=gen)

    def rows_of(sigma=1.0):             # activations: rows of a buffer that may be wider
        return normal(n, d + case.get("pad", 0), sigma=sigma)[:, :d]

    def before(*shape, sigma):          # what a gradient buffer holds before the call
        return normal(*shape, sigma=sigma, dtype=gdt) if case.get("acc") else torch.empty(shape, dtype=gdt, device=dev)

    def ids(missing, mark):
        """Token ids with frequencies ~ 1 / rank, ranks spread over the ids; some places marked
        (the first is not)."""
        u = torch.rand(n, device=dev, generator=gen, dtype=torch.float64)
        rank = torch.exp(u * math.log(v + 1)).long().clamp(1, v) - 1
        t = rank * 7919 % v if v % 7919 else rank
        there = torch.rand(n, device=dev, generator=gen) >= missing
        there[0] = True
        return torch.where(there, t, torch.full_like(t, mark))

    s = dict(op=op, case=dict(case))
    if op.startswith("layernorm"):
        # a residual stream: a few channels much larger than the others, an offset
        s["x"] = rows_of()
        s["x"][:, ::97] *= 8.0
        s["x"] += 0.25
        s["weight"] = normal(d, sigma=0.1) + 1.0
        s["bias"] = normal(d, sigma=0.1)
        if op == "layernorm_backward":
            s["dy"] = rows_of(0.01)
            s["dweight"], s["dbias"] = before(d, sigma=0.1), before(d, sigma=0.1)
            x = s["x"].double()         # the forward pass's statistics
            s["mean"] = x.mean(1).float()
            s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + EPS).float()
    elif op.startswith("embedding"):
        s["tokens"] = ids(case["padded"], -1)
        if op == "embedding":
            s["table"] = normal(v, d, sigma=0.02)
        else:
            s["dout"] = normal(n, d, sigma=0.01)
            s["dtable"] = before(v, d, sigma=0.01)
    else:
        s["hidden"] = normal(n, d)      # a final layer norm's output
        s["weight"] = normal(v, d, sigma=2.0 / math.sqrt(d))
        s["targets"] = ids(case["masked"], IGNORE)
        if op == "head_train":
            s["dweight"] = before(v, d, sigma=1e-3)
            s["row_scale"] = torch.rand(n, device=dev, generator=gen) + 0.5 if case["weighted"] else None
    if own:
        prepare_own(s, dev, dt)
    return s


def prepare_own(s, dev, dt):
    """The buffers that a user's program keeps: outputs, workspace, step state."""
    import zero_partitioned_optimizer_shard_gb300 as z
    c, op = s["case"], s["op"]
    n, d, v = c["rows"], c["d"], c.get("vocab", 0)
    empty = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
    if op == "layernorm":
        s["y"], s["mean"], s["rstd"] = empty(n, d), empty(n, dtype=torch.float32), empty(n, dtype=torch.float32)
        return
    if op == "embedding":
        s["out"] = empty(n, d)
        return
    if op == "layernorm_backward":
        s["dx"] = empty(n, d)
        need = z.zero_layernorm_workspace_bytes(n, d)
    elif op == "embedding_backward":
        need = z.zero_embedding_workspace_bytes(n, d, v)
    else:
        s["loss"], s["lse"] = empty(n, dtype=torch.float32), empty(n, dtype=torch.float32)
        if op == "head_train":
            s["dhidden"] = empty(n, d)
            s["st"] = empty(z.STATE_BYTES, dtype=torch.uint8)
            z.zero_tensors_state_init(1, c["loss_scale"], False, 0, s["st"])
        need = z.zero_head_workspace_bytes(n, d, v)
    s["work"] = empty(need, dtype=torch.uint8)


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        return run_own(s)
    return {"layernorm": plain_layernorm, "layernorm_backward": plain_layernorm_backward, "embedding": plain_embedding,
            "embedding_backward": plain_embedding_backward, "head_loss": plain_head_loss,
            "head_train": plain_head_train}[s["op"]](s)


def run_own(s):
    import zero_partitioned_optimizer_shard_gb300 as z
    c, op = s["case"], s["op"]
    if op == "layernorm":
        z.zero_layernorm(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=EPS)
        return {k: s[k] for k in ("y", "mean", "rstd")}
    if op == "layernorm_backward":
        z.zero_layernorm_backward(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dweight"], s["dbias"],
                                  s["work"], accumulate=c["acc"])
        return {k: s[k] for k in ("dx", "dweight", "dbias")}
    if op == "embedding":
        z.zero_embedding(s["tokens"], s["table"], s["out"], scale=c["scale"])
        return {"out": s["out"]}
    if op == "embedding_backward":
        z.zero_embedding_backward(s["tokens"], s["dout"], s["dtable"], s["work"], scale=c["scale"], accumulate=c["acc"])
        return {"dtable": s["dtable"]}
    z.zero_head_loss(s["hidden"], s["weight"], s["targets"], s["loss"], s["lse"], s["work"])
    if op == "head_loss":
        return {k: s[k] for k in ("loss", "lse")}
    z.zero_head_loss_backward(s["hidden"], s["weight"], s["targets"], s["lse"], s["dhidden"], s["dweight"], s["work"],
                              scale=1.0 / c["rows"], row_scale=s["row_scale"], st=s["st"], accumulate=c["acc"])
    return {k: s[k] for k in ("loss", "lse", "dhidden", "dweight")}


def plain_layernorm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    y = c * rstd * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def plain_layernorm_backward(s):
    rstd = s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": put(s, "dweight", (dy * xhat).sum(0)),
            "dbias": put(s, "dbias", dy.sum(0))}


def put(s, name, value):
    """A gradient into its buffer, or added to what is there, rounded once."""
    s[name].copy_(s[name].float() + value if s["case"]["acc"] else value)
    return s[name]


def plain_embedding(s):
    t, v = s["tokens"], s["case"]["vocab"]
    there = (t >= 0) & (t < v)
    rows = s["table"][t.clamp(0, v - 1)].float() * s["case"]["scale"]
    return {"out": torch.where(there[:, None], rows, torch.zeros_like(rows)).to(s["table"].dtype)}


def plain_embedding_backward(s):
    t, v, d = s["tokens"], s["case"]["vocab"], s["case"]["d"]
    there = (t >= 0) & (t < v)
    total = torch.zeros(v + 1, d, device=t.device)
    total.index_add_(0, torch.where(there, t, torch.full_like(t, v)), s["dout"].float())
    return {"dtable": put(s, "dtable", total[:v] * s["case"]["scale"])}


def plain_logits(s):
    """The logits, and which tokens have a target, with a safe index for those that do not."""
    t, v = s["targets"], s["case"]["vocab"]
    there = (t >= 0) & (t < v)
    return s["hidden"].float() @ s["weight"].float().t(), there, torch.where(there, t, torch.zeros_like(t))


def plain_loss(logits, there, at):
    top = logits.amax(1)
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    loss = lse - logits.gather(1, at[:, None])[:, 0]
    none = torch.zeros_like(lse)
    return torch.where(there, loss, none), torch.where(there, lse, none)


def plain_head_loss(s):
    loss, lse = plain_loss(*plain_logits(s))
    return {"loss": loss, "lse": lse}


def plain_head_train(s):
    c = s["case"]
    logits, there, at = plain_logits(s)
    loss, lse = plain_loss(logits, there, at)
    p = torch.exp(logits - lse[:, None])
    p.scatter_add_(1, at[:, None], torch.full_like(lse, -1.0)[:, None])
    factor = torch.full_like(lse, c["loss_scale"] / c["rows"])
    if s["row_scale"] is not None:
        factor = factor * s["row_scale"]
    p = torch.where(there[:, None], p * factor[:, None], torch.zeros_like(p))
    dhidden = p @ s["weight"].float()
    dweight = p.t() @ s["hidden"].float()
    return {"loss": loss, "lse": lse, "dhidden": dhidden.to(s["hidden"].dtype), "dweight": put(s, "dweight", dweight)}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, n, d = case["op"], case["rows"], case["d"]
    wide = {k: x.double() for k, x in s.items() if isinstance(x, torch.Tensor) and x.is_floating_point()}
    if op == "layernorm":
        x, y = wide["x"], torch.empty(n, d, dtype=torch.float64, device=s["x"].device)
        variance, mean = torch.var_mean(x, dim=1, correction=0)
        torch.sub(x, mean.unsqueeze(1), out=y)
        y /= torch.sqrt(variance + EPS).unsqueeze(1)
        return {"y": torch.addcmul(wide["bias"].expand(n, d), y, wide["weight"].expand(n, d)), "mean": mean,
                "rstd": 1.0 / torch.sqrt(variance + EPS)}
    if op == "layernorm_backward":
        # the Jacobian of (x - mean) * rstd in its rows: rstd * (I - 1/d - xhat xhat^T / d)
        xhat = (wide["x"] - wide["mean"].unsqueeze(1)) * wide["rstd"].unsqueeze(1)
        g = wide["dy"] * wide["weight"]
        along = torch.einsum("nd,nd->n", g, xhat) / d
        dx = (g - torch.einsum("nd->n", g)[:, None] / d - along[:, None] * xhat) * wide["rstd"][:, None]
        dweight, dbias = torch.einsum("nd,nd->d", wide["dy"], xhat), torch.einsum("nd->d", wide["dy"])
        if case["acc"]:
            dweight, dbias = dweight + wide["dweight"], dbias + wide["dbias"]
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "embedding":
        out = torch.zeros(n, d, dtype=torch.float64, device=s["table"].device)
        at = torch.nonzero(s["tokens"] >= 0)[:, 0]
        out[at] = wide["table"].index_select(0, s["tokens"][at]) * case["scale"]
        return {"out": out}
    if op == "embedding_backward":
        at = torch.nonzero(s["tokens"] >= 0)[:, 0]
        total = wide["dtable"] if case["acc"] else torch.zeros(case["vocab"], d, dtype=torch.float64, device=at.device)
        total.index_put_((s["tokens"][at],), wide["dout"][at] * case["scale"], accumulate=True)
        return {"dtable": total}
    at = torch.nonzero(s["targets"] >= 0)[:, 0]
    h, w, t = wide["hidden"][at], wide["weight"], s["targets"][at]
    z = torch.mm(h, w.T)
    lse, picked = torch.logsumexp(z, 1), z[torch.arange(len(at), device=at.device), t]
    spread = lambda x: torch.zeros(n, *x.shape[1:], dtype=torch.float64, device=x.device).index_copy_(0, at, x)  # noqa: E731
    out = {"loss": spread(lse - picked), "lse": spread(lse)}
    if op == "head_loss":
        return out
    z.sub_(lse[:, None]).exp_()
    z[torch.arange(len(at), device=at.device), t] -= 1.0
    factor = torch.full_like(lse, case["loss_scale"] / n)
    if s["row_scale"] is not None:
        factor *= wide["row_scale"][at]
    z *= factor[:, None]
    dweight = torch.mm(z.T, h)
    return {**out, "dhidden": spread(torch.mm(z, w)), "dweight": wide["dweight"] + dweight if case["acc"] else dweight}
