"""The parts of a recurrent layer beside the KDA mixer, as cases to measure.

Three operators: a gated linear recurrence over packed sequences (every channel its own state,
its gradient, its single-token step), the gated feed-forward block (both projections, the
activation and their product; its gradient), and dropout from a counter-based generator whose
mask is never stored, by itself and in the residual stream's norm.  With ``own`` false ``run``
computes them in plain torch operations in 32 bits; with it true through this package's entry
points.  ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One token of 256 sequences (the decode workload), 56 heads' worth of channels: latency.
        dict(name="recurrence step b256 c7168", op="recurrence", form="step", dtype="bf16",
             seqs=256, channels=7168, write="add"),
        # The packed prefill of four sequences (8,192 to 32,768 tokens), a GRU's update.
        dict(name="recurrence prefill t81920 c7168", op="recurrence", form="forward", dtype="bf16",
             tokens=81920, seqs=4, channels=7168, write="mix", h0=True, sliced=False),
        # One sequence of a million tokens and few channels: only a split over time fills the GPU.
        dict(name="recurrence long t1048576 c512", op="recurrence", form="forward", dtype="bf16",
             tokens=1048576, seqs=1, channels=512, write="add", h0=True, sliced=False),
        # The gradient of a packed training batch.
        dict(name="recurrence grad t81920 c4096", op="recurrence", form="backward", dtype="bf16",
             tokens=81920, seqs=4, channels=4096, write="mix", h0=True, sliced=False),
        # fp32, odd sizes, many short sequences, some of them empty, x a slice of a projection.
        dict(name="recurrence grad f32 odd", op="recurrence", form="backward", dtype="f32",
             tokens=20011, seqs=37, channels=1001, write="add", h0=True, sliced=True),
        # A single request's token: the weight's bytes bound it.
        dict(name="gated_ffn token t1", op="gated_ffn", form="forward", dtype="bf16",
             tokens=1, width=7168, hidden=14336, act="silu"),
        # One token of each of 256 sequences.
        dict(name="gated_ffn decode t256", op="gated_ffn", form="forward", dtype="bf16",
             tokens=256, width=7168, hidden=14336, act="silu"),
        # A training batch's gradient.
        dict(name="gated_ffn grad t8192", op="gated_ffn", form="backward", dtype="bf16",
             tokens=8192, width=4096, hidden=10240, act="silu"),
        # fp32 at odd sizes: what tests and small models use.
        dict(name="gated_ffn grad f32 odd", op="gated_ffn", form="backward", dtype="f32",
             tokens=777, width=515, hidden=1003, act="gelu"),
        # The residual stream in training, the mixer's output dropped out before it is added.
        dict(name="dropout norm t40960", op="dropout", form="norm", dtype="bf16",
             tokens=40960, width=7168, p=0.1, scale=1.0),
        # Its gradient: the mask again from the counter.
        dict(name="dropout norm grad t40960", op="dropout", form="norm_backward", dtype="bf16",
             tokens=40960, width=7168, p=0.1, scale=0.5),
        # By itself, a small model's embeddings at an odd width.
        dict(name="dropout f32 odd", op="dropout", form="alone", dtype="f32",
             tokens=1003, width=1001, p=0.25),
    ]


def _size(rng, low, high, even):
    """A size spread over the logarithm of the range; about one in three keeps its odd value."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if n > 2 * even and rng.random() < 0.66:
        n -= n % even
    return n


def draw(rng):
    op = rng.choice(["recurrence", "gated_ffn", "dropout"])
    c = dict(op=op, dtype="f32" if rng.random() < 0.3 else "bf16")
    if op == "recurrence":
        c["form"] = rng.choice(["step", "forward", "backward"])
        c["channels"] = _size(rng, 64, 8192, 64)
        c["write"] = rng.choice(["add", "mix"])
        if c["form"] == "step":
            c["seqs"] = _size(rng, 1, 4096, 8)
        else:
            c["tokens"] = _size(rng, 1, min(1048576, 300_000_000 // c["channels"]), 64)
            c["seqs"] = min(c["tokens"], _size(rng, 1, 64, 4))
            c["h0"] = rng.random() < 0.7
            c["sliced"] = rng.random() < 0.3
    elif op == "gated_ffn":
        c["form"] = rng.choice(["forward", "backward"])
        c["width"] = _size(rng, 64, 7168, 64)
        c["hidden"] = _size(rng, 64, 14336, 64)
        most = 8192 * 4096 * 10240 // (8 if c["dtype"] == "f32" else 1)
        c["tokens"] = _size(rng, 1, max(1, min(16384, most // (c["width"] * c["hidden"]))), 64)
        c["act"] = rng.choice(["silu", "gelu", "sigmoid"])
    else:
        c["form"] = rng.choice(["norm", "norm_backward", "alone"])
        c["width"] = _size(rng, 64, 12288, 64)
        c["tokens"] = _size(rng, 1, min(81920, 290_000_000 // c["width"]), 64)
        c["p"] = rng.choice([0.05, 0.1, 0.2, 0.5])
        if c["form"] != "alone":
            c["scale"] = rng.choice([1.0, 0.5, 0.22])
    return c


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)

    s = dict(case=dict(case))
    if case["op"] == "recurrence":
        N, C = case["seqs"], case["channels"]
        T = N if case["form"] == "step" else case["tokens"]
        # time constants of one to a thousand tokens, by channel, moved by every token's gate
        rate = torch.exp(torch.rand(C, generator=gen, device="cuda") * 6.9 - 6.9)
        s["g"] = torch.randn((T, C), generator=gen, device="cuda").mul_(0.5).exp_().mul_(rate).neg_()
        s["x"] = normal(T, C)
        if case["form"] == "step":
            s["state"] = normal(N, C, dtype=torch.float32)
            s["next"] = torch.empty_like(s["state"])
            return s
        if case["sliced"]:  # columns of a fused projection's output
            wide = normal(T, 2, C)
            wide[:, 1] = s["x"]
            s["x"] = wide[:, 1]
        if N == 4:
            ends = torch.tensor([0.1, 0.3, 0.6], device="cuda", dtype=torch.float64)
        else:  # cut anywhere: short sequences are empty now and then
            ends = torch.rand(N - 1, generator=gen, device="cuda", dtype=torch.float64).sort().values
        cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
        cu[1:N] = (ends * T + 0.5).to(torch.int32)
        cu[N] = T
        s["cu"] = cu
        s["h0"] = normal(N, C, dtype=torch.float32) if case["h0"] else None
        if case["form"] == "backward":
            s["h"] = _recurrence(s, case["write"])[0]
            s["d_h"] = normal(T, C, std=0.1)
            s["d_h_final"] = normal(N, C, std=0.1, dtype=torch.float32)
    elif case["op"] == "gated_ffn":
        T, D, F = case["tokens"], case["width"], case["hidden"]
        s["x"] = normal(T, D)  # a norm's output
        s["weight"] = normal(2, F, D, std=1.0 / math.sqrt(D))
        if case["form"] == "backward":
            s["d_h"] = normal(T, F, std=0.1)
    else:
        T, D = case["tokens"], case["width"]
        s["rng"] = torch.randint(0, 2 ** 62, (2,), generator=gen, device="cuda")  # seed, offset
        if case["form"] == "alone":
            s["x"] = normal(T, D)
            return s
        s["h"] = normal(T, D, std=2.0)
        s["weight"] = 1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        if case["form"] == "norm":
            s["y"] = normal(T, D, std=0.5)
        else:
            s["d_h"] = normal(T, D, std=0.5)
            s["d_out"] = normal(T, D, std=0.5)
    return s


# -------------------------------------------------------------------- one pass

SITE = 5  # which of a step's dropouts this is


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import kimi_delta_attention_18_gb300 as kda
    c = s["case"]
    if c["op"] == "recurrence":
        if c["form"] == "step":
            return kda.linear_recurrence_step(s["x"], s["g"], s["state"], write=c["write"],
                                              state_out=s["next"])
        if c["form"] == "forward":
            return kda.linear_recurrence(s["x"], s["g"], s["h0"], s["cu"], write=c["write"])
        return kda.linear_recurrence_backward(s["d_h"], s["x"], s["g"], s["h"], s["h0"], s["cu"],
                                              s["d_h_final"], write=c["write"])
    if c["op"] == "gated_ffn":
        if c["form"] == "forward":
            return kda.gated_ffn(s["x"], s["weight"], act=c["act"])
        return kda.gated_ffn_backward(s["d_h"], s["x"], s["weight"], act=c["act"])
    drop = dict(rng=s["rng"], site=SITE)
    if c["form"] == "alone":
        return kda.dropout(s["x"], c["p"], **drop)
    if c["form"] == "norm":
        return kda.residual_norm(s["h"], s["y"], s["weight"], scale=c["scale"], eps=EPS,
                                 dropout=c["p"], **drop)
    return kda.residual_norm_backward(s["d_out"], s["h"], s["weight"], s["d_h"], scale=c["scale"],
                                      eps=EPS, dropout=c["p"], **drop)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first dimension, h_{-1} = 0: spans double."""
    s = 1
    while s < a.shape[0]:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _recurrence(s, write):
    g, x = s["g"], s["x"].float()
    a = torch.exp(g)
    if write == "mix":
        x = x * -torch.expm1(g)
    cu = s["cu"].long()
    full = torch.nonzero(cu[1:] > cu[:-1])[:, 0]
    first, last = cu[:-1][full], cu[1:][full] - 1
    h0 = torch.zeros((len(cu) - 1, g.shape[1]), device="cuda") if s["h0"] is None else s["h0"]
    x = x.index_add(0, first, a[first] * h0[full])
    h = _scan(a.index_fill(0, first, 0.0), x)
    h_final = h0.index_copy(0, full, h[last])
    return h.to(s["x"].dtype), h_final


def _recurrence_grad(s, write):
    g, dt = s["g"], s["x"].dtype
    a = torch.exp(g)
    cu = s["cu"].long()
    full = torch.nonzero(cu[1:] > cu[:-1])[:, 0]
    first, last = cu[:-1][full], cu[1:][full] - 1
    # dh_t = d_t + a_{t+1} dh_{t+1}, from the last token to the first
    d = s["d_h"].float().index_add(0, last, s["d_h_final"][full])
    after = torch.cat([a[1:], a[:1]]).index_fill(0, last, 0.0)
    d = _scan(after.flip(0), d.flip(0)).flip(0)
    h = s["h"].float()
    before = torch.cat([h[:1], h[:-1]])
    h0 = torch.zeros_like(s["d_h_final"]) if s["h0"] is None else s["h0"]
    before = before.index_copy(0, first, h0[full])
    u = a * d
    d_h0 = s["d_h_final"].index_copy(0, full, u[first])
    if write == "mix":
        return (d * -torch.expm1(g)).to(dt), u * (before - s["x"].float()), d_h0
    return d.to(dt), u * before, d_h0


def _act(a, act):
    """The activation and its derivative."""
    if act == "gelu":
        cdf = 0.5 * torch.erfc(a * -math.sqrt(0.5))
        return a * cdf, cdf + a * torch.exp(-0.5 * a * a) * math.sqrt(0.5 / math.pi)
    p = 1.0 / (1.0 + torch.exp(-a))
    if act == "sigmoid":
        return p, p * (1.0 - p)
    return a * p, p * (1.0 + a * (1.0 - p))


def _words(rng, rows, width):
    """Philox 4 x 32 with ten rounds: a 32-bit word for each of rows x width elements."""
    mask, blocks = 0xffffffff, (width + 3) // 4
    c0 = torch.arange(rows * blocks, device="cuda")
    c1 = (c0 >> 32) | (SITE << 16)
    c0 = c0 & mask
    c2, c3 = (rng[1] & mask).expand_as(c0), ((rng[1] >> 32) & mask).expand_as(c0)
    k0, k1 = rng[0] & mask, (rng[0] >> 32) & mask
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((q >> 32) & mask) ^ c1 ^ k0, q & mask, ((p >> 32) & mask) ^ c3 ^ k1, p & mask
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return torch.stack([c0, c1, c2, c3], 1).view(rows, 4 * blocks)[:, :width]


def _dropped(v, s):
    """v / (1 - p) where the element's word says that it stays, else 0."""
    limit = round(s["case"]["p"] * 2.0 ** 32)
    keep = _words(s["rng"], v.shape[0], v.shape[1]) >= limit
    return torch.where(keep, v / (1.0 - limit / 2.0 ** 32), torch.zeros_like(v))


def _plain(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if c["op"] == "recurrence":
        if c["form"] == "step":
            x, a = s["x"].float(), torch.exp(s["g"])
            if c["write"] == "mix":
                x = x * -torch.expm1(s["g"])
            h = a * s["state"] + x
            return h.to(dt), h
        return (_recurrence if c["form"] == "forward" else _recurrence_grad)(s, c["write"])
    if c["op"] == "gated_ffn":
        x, w = s["x"].float(), s["weight"].float()
        a, b = x @ w[0].T, x @ w[1].T
        f, df = _act(a, c["act"])
        if c["form"] == "forward":
            return (f * b).to(dt)
        d = s["d_h"].float()
        da, db = d * b * df, d * f
        return (da @ w[0] + db @ w[1]).to(dt), torch.stack([da.T @ x, db.T @ x]).to(dt)
    if c["form"] == "alone":
        return _dropped(s["x"].float(), s).to(dt)
    h, w = s["h"].float(), s["weight"]
    if c["form"] == "norm":
        h = h + c["scale"] * _dropped(s["y"].float(), s)
        return h.to(dt), (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w).to(dt)
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    h, d = h * r, s["d_out"].float()
    d_w = (d * h).sum(0)
    d = d * w
    d = s["d_h"].float() + r * (d - h * (d * h).mean(-1, keepdim=True))
    return d.to(dt), (c["scale"] * _dropped(d, s)).to(dt), d_w


# --------------------------------------------------------------- what it takes

def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "recurrence":
        N, C, mix = case["seqs"], case["channels"], case["write"] == "mix"
        if case["form"] == "step":
            return {"bytes": N * C * (2 * b + 12), "flops": 4 * N * C}
        n, ends = case["tokens"] * C, N * C * 4
        if case["form"] == "forward":
            return {"bytes": n * (2 * b + 4) + (2 if case["h0"] else 1) * ends, "flops": 4 * n}
        return {"bytes": n * (3 * b + 8 + (b if mix else 0)) + (3 if case["h0"] else 2) * ends,
                "flops": 8 * n}
    if case["op"] == "gated_ffn":
        T, D, F = case["tokens"], case["width"], case["hidden"]
        if case["form"] == "forward":
            return {"bytes": (T * D + 2 * F * D + T * F) * b, "flops": 4 * T * D * F}
        return {"bytes": (2 * T * D + 4 * F * D + T * F) * b, "flops": 12 * T * D * F}
    n, D = case["tokens"] * case["width"], case["width"]
    arrays = {"alone": 2, "norm": 4, "norm_backward": 5}[case["form"]]
    weights = {"alone": 0, "norm": 4, "norm_backward": 8}[case["form"]]
    return {"bytes": arrays * n * b + weights * D, "flops": 20 * n}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    if work(case)["flops"] > 1.5e12:
        return None  # the products in 64 bits take too long
    s = prepare(case, seed)
    if case["op"] == "dropout":
        return _exact_dropout(case, s)
    if case["op"] == "gated_ffn":
        x, w = s["x"].double(), s["weight"].double()
        a, b = torch.nn.functional.linear(x, w[0]), torch.nn.functional.linear(x, w[1])
        if case["act"] == "gelu":
            cdf = torch.special.ndtr(a)
            f, slope = a * cdf, cdf + a * torch.exp(-a.square() / 2) / math.sqrt(2 * math.pi)
        else:
            p = torch.sigmoid(a)
            f = p if case["act"] == "sigmoid" else a * p
            slope = p * torch.sigmoid(-a)
            slope = slope if case["act"] == "sigmoid" else p + a * slope
        if case["form"] == "forward":
            return f * b
        d = s["d_h"].double()
        grads = torch.cat([d * b * slope, d * f], 1)  # [T][2 F]
        w = w.reshape(-1, w.shape[2])
        return grads @ w, (grads.T @ x).view(2, -1, x.shape[1])
    if case["form"] == "step":
        g, x = s["g"].double(), s["x"].double()
        if case["write"] == "mix":
            x = x * (-torch.expm1(g))
        h = torch.addcmul(x, g.exp(), s["state"].double())
        return h, h
    # token by token inside blocks of about sqrt(T) tokens, all blocks at once, then block by
    # block; a few channels at a time
    T, C, N = case["tokens"], case["channels"], case["seqs"]
    L = max(1, math.isqrt(T))
    nb = -(-T // L)
    cu = s["cu"].tolist()
    back = case["form"] == "backward"
    dt = torch.float64
    outs = []
    step = max(1, 2 ** 26 // T)
    for c0 in range(0, C, step):
        cs = slice(c0, min(C, c0 + step))
        g, x = s["g"][:, cs].double(), s["x"][:, cs].double()
        n = g.shape[1]
        h0 = s["h0"][:, cs].double() if s["h0"] is not None else torch.zeros((N, n), device="cuda", dtype=dt)
        write = -torch.expm1(g) if case["write"] == "mix" else torch.ones_like(g)
        a, v = torch.exp(g), s["d_h"][:, cs].double() if back else write * x
        if back:  # time reversed; the factor of a step is the later token's
            a = torch.cat([torch.ones_like(a[:1]), a.flip(0)[:-1]])
            v = v.flip(0)
        for i in range(N):
            if cu[i + 1] > cu[i]:
                at = T - cu[i + 1] if back else cu[i]
                v[at] += s["d_h_final"][i, cs].double() if back else a[at] * h0[i]
                a[at] = 0.0
        pad = nb * L - T
        a = torch.cat([a, torch.zeros((pad, n), device="cuda", dtype=dt)]).view(nb, L, n)
        v = torch.cat([v, torch.zeros((pad, n), device="cuda", dtype=dt)]).view(nb, L, n)
        for j in range(1, L):
            v[:, j] += a[:, j] * v[:, j - 1]
            a[:, j] *= a[:, j - 1]
        for k in range(1, nb):
            v[k] += a[k] * v[k - 1, L - 1]
        v = v.view(nb * L, n)[:T]
        if not back:
            last = torch.stack([v[cu[i + 1] - 1] if cu[i + 1] > cu[i] else h0[i] for i in range(N)])
            outs.append((v, last))
            continue
        dh = v.flip(0)
        before = torch.roll(s["h"][:, cs].double(), 1, 0)
        for i in range(N):
            if cu[i + 1] > cu[i]:
                before[cu[i]] = h0[i]
        u = torch.exp(g) * dh
        first = torch.stack([u[cu[i]] if cu[i + 1] > cu[i] else s["d_h_final"][i, cs].double()
                             for i in range(N)])
        outs.append((write * dh, u * (before - x if case["write"] == "mix" else before), first))
    return tuple(torch.cat(o, 1) for o in zip(*outs))


def _exact_dropout(case, s):
    """The generator with its products in 16-bit limbs, piece by piece over the tokens."""
    T, D, blocks = case["tokens"], case["width"], (case["width"] + 3) // 4
    step = max(1, 2 ** 25 // D)
    seed, offset = (int(v) % 2 ** 64 for v in s["rng"].tolist())
    limit = round(case["p"] * 2.0 ** 32)

    def product(m, c):  # high and low words of m c
        lo, mid = (m & 0xffff) * c, (m >> 16) * c
        low = (mid & 0xffff) * 0x10000 + lo
        return (mid >> 16) + (low >> 32), low & 0xffffffff

    def factor(t0, t1):
        index = torch.arange(t0 * blocks, t1 * blocks, device="cuda")
        word = [index & 0xffffffff, (index >> 32) + (SITE << 16),
                torch.full_like(index, offset % 2 ** 32), torch.full_like(index, offset >> 32)]
        key = [seed % 2 ** 32, seed >> 32]
        for _ in range(10):
            h0, l0 = product(0xD2511F53, word[0])
            h1, l1 = product(0xCD9E8D57, word[2])
            word = [h1 ^ word[1] ^ key[0], l1, h0 ^ word[3] ^ key[1], l0]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        word = torch.stack(word, -1).reshape(t1 - t0, 4 * blocks)[:, :D]
        return (word >= limit).double() / (1.0 - limit / 2.0 ** 32)

    first, second, d_w = [], [], torch.zeros(D, device="cuda", dtype=torch.float64)
    for i in range(0, T, step):
        j = min(T, i + step)
        m = factor(i, j)
        if case["form"] == "alone":
            first.append(s["x"][i:j].double() * m)
            continue
        w, h = s["weight"].double(), s["h"][i:j].double()
        if case["form"] == "norm":
            h = h + case["scale"] * m * s["y"][i:j].double()
            first.append(h)
            second.append(h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + EPS) * w)
            continue
        rms = torch.sqrt(h.pow(2).mean(-1, keepdim=True) + EPS)
        d = s["d_out"][i:j].double()
        d_w += (d * h / rms).sum(0)
        d = d * w
        along = (d * h).sum(-1, keepdim=True) / (D * rms * rms)
        first.append(s["d_h"][i:j].double() + (d - along * h) / rms)
        second.append(case["scale"] * m * first[-1])
    if case["form"] == "alone":
        return torch.cat(first)
    if case["form"] == "norm":
        return torch.cat(first), torch.cat(second)
    return torch.cat(first), torch.cat(second), d_w
