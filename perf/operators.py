"""The operators of a language model's training step around the KDA mixer, as cases to measure.

Four operators: the norm of a mixer's output with its gate, the residual stream's update with
the next block's norm, the token embedding, and softmax cross entropy over the vocabulary from
the last hidden states (the logits are never an output).  Each has its forward and its backward
pass.  With ``own`` false ``run`` computes them in plain torch operations in 32 bits; with it
true through this package's entry points.  ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
IGNORE = -100
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # A decode step's mixer output (the 256-sequence, 56-head decode workload): latency.
        dict(name="gated_norm decode b256 h56", op="gated_norm", backward=False, dtype="bf16",
             tokens=256, heads=56, width=128, act="sigmoid", sliced=False),
        # The mixer's output in training on the packed 81,920-token batch of 56 heads.
        dict(name="gated_norm train t81920 h56", op="gated_norm", backward=True, dtype="bf16",
             tokens=81920, heads=56, width=128, act="sigmoid", sliced=False),
        # fp32, an odd width, the gate a slice of a wider projection, SiLU.
        dict(name="gated_norm f32 odd", op="gated_norm", backward=True, dtype="f32",
             tokens=1003, heads=3, width=100, act="silu", sliced=True),
        # The residual stream of the decode workload: 56 heads of 128 = 7,168 channels.
        dict(name="residual_norm decode b256", op="residual_norm", backward=False, dtype="bf16",
             tokens=256, width=7168, scale=1.0),
        # The same stream in training, a scaled residual.
        dict(name="residual_norm train t40960", op="residual_norm", backward=True, dtype="bf16",
             tokens=40960, width=7168, scale=0.5),
        # fp32 with an odd width and an odd number of rows.
        dict(name="residual_norm f32 odd", op="residual_norm", backward=False, dtype="f32",
             tokens=20011, width=1001, scale=0.25),
        # A prefill's look-up of 4,096 tokens.
        dict(name="embedding t4096", op="embedding", backward=False, dtype="bf16",
             tokens=4096, vocab=131072, width=4096, scale=1.0),
        # The table's gradient for a training batch: token frequencies as in text (1 / rank).
        dict(name="embedding grad t81920", op="embedding", backward=True, dtype="bf16",
             tokens=81920, vocab=131072, width=4096, scale=1.0),
        # A small table with an odd width: tests, byte-level vocabularies.
        dict(name="embedding grad f32 small", op="embedding", backward=True, dtype="f32",
             tokens=333, vocab=257, width=250, scale=16.0),
        # Scoring 256 positions (one per sequence): the weight's bytes bound it.
        dict(name="cross_entropy score t256", op="cross_entropy", backward=False, dtype="bf16",
             tokens=256, vocab=131072, width=7168),
        # The loss's gradient for a training batch of 8,192 tokens.
        dict(name="cross_entropy grad t8192", op="cross_entropy", backward=True, dtype="bf16",
             tokens=8192, vocab=131072, width=4096),
        # fp32 at odd sizes: what tests and small models use.
        dict(name="cross_entropy grad f32 odd", op="cross_entropy", backward=True, dtype="f32",
             tokens=777, vocab=10007, width=515),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high, even):
    """A size spread over the logarithm of the range; about one in three keeps its odd value."""
    n = _log_int(rng, low, high)
    if n > 2 * even and rng.random() < 0.66:
        n -= n % even
    return n if n != 3072 else n + 1


def draw(rng):
    op = rng.choice(["gated_norm", "residual_norm", "embedding", "cross_entropy"])
    c = dict(op=op, backward=rng.random() < 0.5, dtype="f32" if rng.random() < 0.3 else "bf16")
    if op == "gated_norm":
        c["heads"] = rng.choice([1, 2, 4, 8, 16, 56])
        c["width"] = _size(rng, 16, 512, 16) if rng.random() < 0.5 else rng.choice([64, 128])
        c["tokens"] = _size(rng, 1, max(1, min(81920, 300_000_000 // (c["heads"] * c["width"]))), 64)
        c["act"] = rng.choice(["sigmoid", "silu", "none"])
        c["sliced"] = c["act"] != "none" and rng.random() < 0.3
    elif op == "residual_norm":
        c["width"] = _size(rng, 64, 12288, 64)
        c["tokens"] = _size(rng, 1, min(81920, 300_000_000 // c["width"]), 64)
        c["scale"] = rng.choice([1.0, 0.5, 0.22])
    elif op == "embedding":
        c["vocab"] = _size(rng, 256, 131072, 64)
        c["width"] = _size(rng, 64, 7168, 64)
        c["tokens"] = _size(rng, 1, 81920, 64)
        c["scale"] = rng.choice([1.0, math.sqrt(c["width"])])
    else:
        c["vocab"] = _size(rng, 256, 131072, 64)
        c["width"] = _size(rng, 64, 7168, 64)
        most = 8192 * 131072 * 4096 // (8 if c["dtype"] == "f32" else 1)
        c["tokens"] = _size(rng, 1, max(1, min(8192, most // (c["vocab"] * c["width"]))), 64)
    return c


# ----------------------------------------------------------------- the inputs

def _tokens(count, vocab, gen):
    """Token numbers with text's frequencies: rank r with probability about 1 / r."""
    u = torch.rand(count, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T, D = case["tokens"], case["width"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dt)

    s = dict(case=dict(case))
    if case["op"] == "gated_norm":
        H = case["heads"]
        s["x"] = normal(T, H, D, std=0.3)
        s["gate"] = None
        if case["sliced"]:  # columns of a fused projection's output
            s["gate"] = normal(T, 2, H, D)[:, 1]
        elif case["act"] != "none":
            s["gate"] = normal(T, H, D)
        s["weight"] = 1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        if case["backward"]:
            s["d_out"] = normal(T, H, D, std=0.1)
    elif case["op"] == "residual_norm":
        s["h"] = normal(T, D, std=2.0)
        s["weight"] = 1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        s["y" if not case["backward"] else "d_h"] = normal(T, D, std=0.5)
        if case["backward"]:
            s["d_out"] = normal(T, D, std=0.5)
    elif case["op"] == "embedding":
        s["ids"] = _tokens(T, case["vocab"], gen)
        if case["backward"]:
            s["d_out"] = normal(T, D, std=0.1)
        else:
            s["table"] = normal(case["vocab"], D, std=0.02)
    else:
        V = case["vocab"]
        s["x"] = normal(T, D)
        s["weight"] = normal(V, D, std=2.0 / math.sqrt(D))
        targets = _tokens(T, V, gen)
        masked = torch.rand(T, generator=gen, device="cuda") < 0.1  # a prompt's tokens
        s["targets"] = torch.where(masked, torch.full_like(targets, IGNORE), targets)
        if case["backward"]:
            # the mean over the tokens that count, and the row statistics of the forward pass
            kept = (~masked).float()
            s["d_loss"] = kept / kept.sum().clamp_(min=1.0)
            w = s["weight"].float().T
            s["lse"] = torch.cat([torch.logsumexp(s["x"][i:i + 1024].float() @ w, 1)
                                  for i in range(0, T, 1024)])
    return s


# -------------------------------------------------------------------- one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import kimi_delta_attention_18_gb300 as kda
    c = s["case"]
    if c["op"] == "gated_norm":
        if not c["backward"]:
            return kda.gated_norm(s["x"], s["gate"], s["weight"], act=c["act"], eps=EPS)
        return kda.gated_norm_backward(s["d_out"], s["x"], s["gate"], s["weight"], act=c["act"],
                                       eps=EPS)
    if c["op"] == "residual_norm":
        if not c["backward"]:
            return kda.residual_norm(s["h"], s["y"], s["weight"], scale=c["scale"], eps=EPS)
        return kda.residual_norm_backward(s["d_out"], s["h"], s["weight"], s["d_h"],
                                          scale=c["scale"], eps=EPS)
    if c["op"] == "embedding":
        if not c["backward"]:
            return kda.embedding(s["table"], s["ids"], scale=c["scale"])
        return kda.embedding_backward(s["d_out"], s["ids"], c["vocab"], scale=c["scale"])
    if not c["backward"]:
        return kda.linear_cross_entropy(s["x"], s["weight"], s["targets"], ignore_index=IGNORE)
    return kda.linear_cross_entropy_backward(s["x"], s["weight"], s["targets"], s["lse"],
                                             s["d_loss"], ignore_index=IGNORE)


def _gate(z, act):
    """The gate's factor and its derivative."""
    p = 1.0 / (1.0 + torch.exp(-z))
    if act == "sigmoid":
        return p, p * (1.0 - p)
    return z * p, p * (1.0 + z * (1.0 - p))


def _plain(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if c["op"] == "gated_norm":
        x, w = s["x"].float(), s["weight"]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        x = x * r
        a, da = (1.0, 0.0) if s["gate"] is None else _gate(s["gate"].float(), c["act"])
        if not c["backward"]:
            return (x * w * a).to(dt)
        d = s["d_out"].float()
        d_gate = None if s["gate"] is None else (d * x * w * da).to(dt)
        d = d * a
        d_w = (d * x).sum((0, 1))
        d = d * w
        return (r * (d - x * (d * x).mean(-1, keepdim=True))).to(dt), d_gate, d_w
    if c["op"] == "residual_norm":
        h, w = s["h"].float(), s["weight"]
        if not c["backward"]:
            h = h + c["scale"] * s["y"].float()
            return h.to(dt), (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w).to(dt)
        r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        h, d = h * r, s["d_out"].float()
        d_w = (d * h).sum(0)
        d = d * w
        d = s["d_h"].float() + r * (d - h * (d * h).mean(-1, keepdim=True))
        return d.to(dt), (c["scale"] * d).to(dt), d_w
    if c["op"] == "embedding":
        ids = s["ids"].long()
        if not c["backward"]:
            return (s["table"][ids].float() * c["scale"]).to(dt)
        g = torch.zeros((c["vocab"], c["width"]), device="cuda")
        return (g.index_add_(0, ids, s["d_out"].float()) * c["scale"]).to(dt)
    x, w, y = s["x"].float(), s["weight"].float(), s["targets"].long()
    z = x @ w.T
    kept = y != IGNORE
    at = torch.where(kept, y, torch.zeros_like(y))[:, None]
    if not c["backward"]:
        m = z.max(1, keepdim=True).values
        z_y = z.gather(1, at)[:, 0]
        lse = m[:, 0] + torch.log(torch.exp(z - m).sum(1))
        loss = torch.where(kept, lse - z_y, torch.zeros_like(lse))
        return loss, lse, loss.sum() / kept.sum().clamp(min=1)
    g = torch.where(kept, s["d_loss"], torch.zeros_like(s["d_loss"]))[:, None]
    z = torch.exp(z - s["lse"][:, None]) * g
    z.scatter_add_(1, at, -g)
    return (z @ w).to(dt), (z.T @ x).to(dt)


# --------------------------------------------------------------- what it takes

def work(case):
    b, T, D = BYTES[case["dtype"]], case["tokens"], case["width"]
    if case["op"] == "gated_norm":
        n, gated = T * case["heads"] * D, case["act"] != "none"
        arrays = (3 if not gated else 5) if case["backward"] else (2 if not gated else 3)
        return {"bytes": arrays * n * b + (8 if case["backward"] else 4) * D,
                "flops": (20 if case["backward"] else 8) * n}
    if case["op"] == "residual_norm":
        n = T * D
        return {"bytes": (5 if case["backward"] else 4) * n * b + (8 if case["backward"] else 4) * D,
                "flops": (14 if case["backward"] else 6) * n}
    if case["op"] == "embedding":
        if case["backward"]:
            return {"bytes": T * D * b + 4 * T + case["vocab"] * D * b, "flops": T * D}
        return {"bytes": 2 * T * D * b + 4 * T, "flops": T * D}
    V = case["vocab"]
    if case["backward"]:  # logits again, d_x and d_weight
        return {"bytes": 2 * (T + V) * D * b + 12 * T, "flops": 6 * T * V * D}
    return {"bytes": (T + V) * D * b + 12 * T, "flops": 2 * T * V * D}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    T, D = case["tokens"], case["width"]
    if case["op"] == "cross_entropy" and T * case["vocab"] * D > 2.5e11:
        return None  # the products in 64 bits take too long
    s = prepare(case, seed)
    if case["op"] == "gated_norm":
        return _exact_gated_norm(case, s)
    if case["op"] == "residual_norm":
        return _exact_residual_norm(case, s)
    if case["op"] == "embedding":
        if not case["backward"]:
            return torch.nn.functional.embedding(s["ids"].long(), s["table"]).double() * case["scale"]
        order = torch.argsort(s["ids"].long(), stable=True)
        ids, counts = torch.unique_consecutive(s["ids"].long()[order], return_counts=True)
        ends = counts.cumsum(0).tolist()
        g = torch.zeros((case["vocab"], D), device="cuda", dtype=torch.float64)
        for v, n, e in zip(ids.tolist(), counts.tolist(), ends):
            g[v] = s["d_out"][order[e - n:e]].double().sum(0) * case["scale"]
        return g
    x, w, y = s["x"].double(), s["weight"].double(), s["targets"].long()
    loss, lse, dx = [], [], []
    dw = torch.zeros_like(w)
    for i in range(0, T, 512):
        logits = x[i:i + 512] @ w.t()
        target = y[i:i + 512]
        rows = torch.nonzero(target != IGNORE)[:, 0]
        if not case["backward"]:
            total = torch.logsumexp(logits, 1)
            part = torch.zeros_like(total)
            part[rows] = total[rows] - logits[rows, target[rows]]
            lse.append(total)
            loss.append(part)
            continue
        d = torch.exp(logits - s["lse"][i:i + 512, None].double())
        d[rows, target[rows]] -= 1.0
        g = torch.zeros(len(target), device="cuda", dtype=torch.float64)
        g[rows] = s["d_loss"][i:i + 512].double()[rows]
        d *= g[:, None]
        dx.append(d @ w)
        dw.addmm_(d.t(), x[i:i + 512])
    if case["backward"]:
        return torch.cat(dx), dw
    loss = torch.cat(loss)
    return loss, torch.cat(lse), loss.sum() / max(1, int((y != IGNORE).sum()))


def _exact_gated_norm(case, s):
    """Piece by piece over the tokens; the derivative of x / |x| as a projection."""
    out, d_gate, d_w = [], [], torch.zeros(case["width"], device="cuda", dtype=torch.float64)
    w, step = s["weight"].double(), max(1, 2 ** 26 // (case["heads"] * case["width"]))
    for i in range(0, case["tokens"], step):
        x = s["x"][i:i + step].double()
        rms = torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
        act, slope = torch.ones_like(x), torch.zeros_like(x)
        if s["gate"] is not None:
            z = s["gate"][i:i + step].double()
            act = torch.sigmoid(z) if case["act"] == "sigmoid" else torch.nn.functional.silu(z)
            sg = torch.sigmoid(z)
            slope = sg * torch.sigmoid(-z) if case["act"] == "sigmoid" else sg + act * torch.sigmoid(-z)
        if not case["backward"]:
            out.append(x / rms * w * act)
            continue
        d = s["d_out"][i:i + step].double()
        d_gate.append(d * w * x / rms * slope)
        d_w += (d * act * x / rms).sum((0, 1))
        d = d * act * w
        along = (d * x).sum(-1, keepdim=True) / (case["width"] * rms * rms)
        out.append((d - along * x) / rms)
    if not case["backward"]:
        return torch.cat(out)
    return torch.cat(out), None if s["gate"] is None else torch.cat(d_gate), d_w


def _exact_residual_norm(case, s):
    first, second, d_w = [], [], torch.zeros(case["width"], device="cuda", dtype=torch.float64)
    w, step = s["weight"].double(), max(1, 2 ** 26 // case["width"])
    for i in range(0, case["tokens"], step):
        h = s["h"][i:i + step].double()
        if not case["backward"]:
            h = h + case["scale"] * s["y"][i:i + step].double()
            first.append(h)
            second.append(h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + EPS) * w)
            continue
        rms = torch.sqrt(h.pow(2).mean(-1, keepdim=True) + EPS)
        d = s["d_out"][i:i + step].double()
        d_w += (d * h / rms).sum(0)
        d = d * w
        along = (d * h).sum(-1, keepdim=True) / (case["width"] * rms * rms)
        first.append(s["d_h"][i:i + step].double() + (d - along * h) / rms)
        second.append(case["scale"] * first[-1])
    if case["backward"]:
        return torch.cat(first), torch.cat(second), d_w
    return torch.cat(first), torch.cat(second)
