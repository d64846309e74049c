"""The operators around the mixer against their formulas in 64 bits: the norms with
gate and residual, the embedding and the cross entropy, forward and backward.

Bounds.  BF16 has 8 significant bits, so one rounding is up to 2^-8 of the value;
fp32 arithmetic adds a few 2^-24 per operation of the sum behind an output; where
that is a difference of terms (dx of a norm) or a long sum, the bound is relative
to the sum of the terms' magnitudes.  The cross entropy's dz is rounded to BF16
before its products, so there each term of the sum carries 2^-8.
"""
import math

import pytest
import torch

import kimi_delta_attention_18_gb300 as kda

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8}
FP32 = 2.0 ** -18  # rsqrt, exp and division approximations and a row's fp32 sums


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dt, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def _close(got, ref, act, terms=None, extra=0.0):
    """|got - ref| <= one rounding of ref + (FP32 + extra) of the terms behind it."""
    assert got.shape == ref.shape
    terms = ref.abs() if terms is None else terms
    bound = ROUND[act] * ref.abs() + (FP32 + extra) * terms + 1e-30
    bad = (got.double() - ref).abs() > bound
    assert not bad.any(), "%d of %d off, worst %g against %g" % (
        int(bad.sum()), bad.numel(), float((got.double() - ref).abs().max()),
        float(ref.abs().max()))


# -------------------------------------------------------------------- gated norm

def _gate64(z, act):
    s = torch.sigmoid(z)
    if act == "sigmoid":
        return s, s * torch.sigmoid(-z)
    return z * s, s + z * s * torch.sigmoid(-z)


def _gated64(x, z, w, act, eps):
    x = x.double()
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    a, da = (torch.ones_like(x), torch.zeros_like(x)) if z is None else _gate64(z.double(), act)
    w = torch.ones(x.shape[-1], device="cuda", dtype=torch.float64) if w is None else w.double()
    return x * r, r, a, da, w


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,D,act,weight,strided", [
    (1, 1, 1, "sigmoid", True, False),
    (1, 56, 128, "sigmoid", True, False),
    (300, 3, 128, "silu", True, True),
    (5, 2, 7, "silu", True, False),
    (33, 1, 16, "none", False, False),
    (129, 4, 100, "sigmoid", False, True),
    (17, 2, 129, "silu", True, True),
    (7, 1, 1000, "sigmoid", True, False),
    (3, 2, 1032, "sigmoid", True, False),
    (2, 1, 4097, "silu", True, False),
    (5, 1, 16384, "sigmoid", True, False),
    (2, 1, 16383, "sigmoid", True, False),
    (4000, 8, 64, "sigmoid", True, False),
    (1500, 56, 128, "silu", True, True),
    (50001, 1, 128, "sigmoid", True, True),
    (20000, 3, 64, "none", True, True),
    (9000, 5, 100, "silu", True, False),
])
def test_gated_norm(dtype, T, H, D, act, weight, strided):
    g, dt = _gen(T + D), DT[dtype]
    x, z = _randn((T, H, D), g, dt, 2.0), None
    if act != "none":
        z = _randn((T, 3, H, D), g, dt, 2.0)[:, 1] if strided else _randn((T, H, D), g, dt, 2.0)
    if strided:
        x = _randn((T, 2, H, D), g, dt, 2.0)[:, 1]
    w = _randn((D,), g, torch.float32) if weight else None
    d = _randn((T, H, D), g, dt)
    n, r, a, da, w64 = _gated64(x, z, w, act, 1e-5)
    out = kda.gated_norm(x, z, w, act=act, eps=1e-5)
    _close(out, n * w64 * a, dtype)
    dx, dz, dw = kda.gated_norm_backward(d, x, z, w, act=act, eps=1e-5)
    e = d.double() * a * w64
    mean = (e * n).mean(-1, keepdim=True)
    _close(dx, r * (e - n * mean), dtype,
           r * (e.abs() + n.abs() * (e * n).abs().mean(-1, keepdim=True)))
    if z is None:
        assert dz is None
    else:  # 1 - sigmoid and 1 + z (1 - sigmoid) are differences of terms up to 1 + |z|
        _close(dz, d.double() * n * w64 * da, dtype,
               (d.double() * n * w64).abs() * (1.0 + z.double().abs()))
    assert dw.dtype == torch.float32
    _close(dw, (d.double() * a * n).sum((0, 1)), "f32", (d.double() * a * n).abs().sum((0, 1)))


def test_gated_norm_backward_matches_differences():
    """The gradients against central differences of the 64-bit formula."""
    g = _gen(3)
    x, z = _randn((2, 2, 5), g, torch.float32), _randn((2, 2, 5), g, torch.float32)
    w, d = _randn((5,), g, torch.float32), _randn((2, 2, 5), g, torch.float32)

    def f(x, z, w):
        n, _, a, _, w64 = _gated64(x, z, w, "silu", 1e-3)
        return float((d.double() * n * w64 * a).sum())

    got = kda.gated_norm_backward(d, x, z, w, act="silu", eps=1e-3)
    args = [x.double(), z.double(), w.double()]
    for k in range(3):
        for i in range(args[k].numel()):
            vals = []
            for s in (1e-5, -1e-5):
                moved = [t.clone() for t in args]
                moved[k].view(-1)[i] += s
                vals.append(f(*moved))
            # central difference: error 1e-10 of third derivatives, 1e-11 of rounding
            assert abs(float(got[k].view(-1)[i]) - (vals[0] - vals[1]) / 2e-5) < 2e-4


def test_gated_norm_of_zeros_and_large_rows():
    x = torch.zeros((3, 1, 128), device="cuda", dtype=torch.bfloat16)
    x[1] = 3e18  # its square still fits fp32
    z = torch.full_like(x, -200.0)
    z[2] = 200.0
    out = kda.gated_norm(x, z)
    assert torch.isfinite(out.float()).all() and not out.float().abs().max() > 0
    out = kda.gated_norm(x, -z)
    assert torch.equal(out[1].float(), torch.ones((1, 128), device="cuda"))
    dx, dz, dw = kda.gated_norm_backward(torch.ones_like(x), x, z)
    for t in (dx, dz, dw):
        assert torch.isfinite(t.float()).all()


def test_norms_without_tokens():
    x = torch.empty((0, 2, 16), device="cuda")
    assert kda.gated_norm(x, x).shape == (0, 2, 16)
    dx, dz, dw = kda.gated_norm_backward(x, x, x)
    assert dx.numel() == 0 and torch.equal(dw, torch.zeros(16, device="cuda"))
    h = torch.empty((0, 16), device="cuda")
    assert kda.residual_norm(h, h)[1].shape == (0, 16)
    assert torch.equal(kda.residual_norm_backward(h, h)[2], torch.zeros(16, device="cuda"))


# ----------------------------------------------------------------- residual norm

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,scale,weight,with_y", [
    (1, 1, 1.0, True, True),
    (1, 7168, 1.0, True, True),
    (256, 1024, 0.5, True, True),
    (3, 1001, 0.22, True, True),
    (37, 515, -2.0, False, True),
    (9, 12345, 1.0, True, True),
    (64, 4096, 1.0, True, False),
    (1, 33, 1.0, False, False),
    (2049, 192, 0.5, True, True),
    (5003, 1024, 0.5, True, True),
    (5001, 1001, 1.0, True, True),
    (2501, 2560, 0.5, True, False),
    (700, 7168, 0.5, True, True),
    (700, 8192, 1.0, False, True),
])
def test_residual_norm(dtype, T, D, scale, weight, with_y):
    g, dt = _gen(T + D), DT[dtype]
    h, y = _randn((T, D), g, dt, 2.0), _randn((T, D), g, dt) if with_y else None
    w = _randn((D,), g, torch.float32) if weight else None
    w64 = torch.ones(D, device="cuda", dtype=torch.float64) if w is None else w.double()
    h64 = h.double() + (scale * y.double() if with_y else 0.0)
    size = h.double().abs() + (abs(scale) * y.double().abs() if with_y else 0.0)
    r = (h64.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
    h_out, out = kda.residual_norm(h, y, w, scale=scale)
    _close(h_out, h64, dtype, size)
    _close(out, h64 * r * w64, dtype, size * r * w64.abs())
    # backward, from the rounded h_out
    d_out, d_h = _randn((T, D), g, dt), _randn((T, D), g, dt)
    h64 = h_out.double()
    r = (h64.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
    n, e = h64 * r, d_out.double() * w64
    through = r * (e - n * (e * n).mean(-1, keepdim=True))
    terms = r * (e.abs() + n.abs() * (e * n).abs().mean(-1, keepdim=True))
    dw = (d_out.double() * n).sum(0)
    for d in (d_h, None):
        dh, dy, got_w = kda.residual_norm_backward(d_out, h_out, w, d, scale=scale)
        ref = through + (0.0 if d is None else d.double())
        t = terms + (0.0 if d is None else d.double().abs())
        _close(dh, ref, dtype, t)
        _close(dy, scale * ref, dtype, abs(scale) * t)
        _close(got_w, dw, "f32", (d_out.double() * n).abs().sum(0))


def test_residual_norm_in_place_and_on_another_stream():
    g = _gen(5)
    h, y = _randn((64, 512), g, torch.bfloat16), _randn((64, 512), g, torch.bfloat16)
    ref_h, ref = kda.residual_norm(h, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mine = h.clone()
    s.wait_stream(torch.cuda.current_stream())
    h_out, out = kda.residual_norm(mine, y, h_out=mine, stream=s)
    s.synchronize()
    assert h_out is mine and torch.equal(mine, ref_h) and torch.equal(out, ref)


# --------------------------------------------------------------------- embedding

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D,kind,ids_dtype", [
    (1, 1, 1, "same", torch.int32),
    (1, 50, 128, "uniform", torch.int64),
    (333, 257, 250, "text", torch.int32),
    (2047, 1000, 64, "text", torch.int32),
    (2049, 1025, 72, "uniform", torch.int64),
    (5000, 40, 33, "uniform", torch.int32),
    (9000, 3, 8, "same", torch.int32),
    (5000, 100003, 24, "text", torch.int32),
    (3000, (1 << 20) + 5, 2, "uniform", torch.int64),
    (20, 300, 4096, "uniform", torch.int32),
])
def test_embedding(dtype, T, V, D, kind, ids_dtype):
    g, dt = _gen(T + V), DT[dtype]
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    ids = {"same": torch.full_like(u, V - 1), "uniform": u * V,
           "text": (u * math.log(V + 1.0)).exp() - 1.0}[kind].long().clamp(0, V - 1).to(ids_dtype)
    table, d = _randn((V, D), g, dt), _randn((T, D), g, dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kda.embedding(table, ids, scale=1.5, dev_status=status)
    _close(out, 1.5 * table[ids.long()].double(), dtype)
    got = kda.embedding_backward(d, ids, V, scale=1.5, dev_status=status)
    ref = torch.zeros((V, D), device="cuda", dtype=torch.float64).index_add_(0, ids.long(), d.double())
    size = torch.zeros_like(ref).index_add_(0, ids.long(), d.double().abs())
    _close(got, 1.5 * ref, dtype, 1.5 * size)
    assert int(status) == 0
    assert torch.equal(got, kda.embedding_backward(d, ids, V, scale=1.5))  # a fixed order


def test_embedding_gradient_of_one_frequent_token_among_many():
    """An id whose tokens span many parts of the sorted list, absent ids around it."""
    g = _gen(1)
    T, V, D = 30000, 5000, 40
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    ids[::3] = 2500
    d = _randn((T, D), g, torch.float32)
    got = kda.embedding_backward(d, ids, V)
    ref = torch.zeros((V, D), device="cuda", dtype=torch.float64).index_add_(0, ids, d.double())
    size = torch.zeros_like(ref).index_add_(0, ids, d.double().abs())
    _close(got, ref, "f32", size)


def test_embedding_reports_ids_outside_the_table():
    table = torch.ones((4, 8), device="cuda")
    ids = torch.tensor([0, 4, -1, 3], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kda.embedding(table, ids, dev_status=status)
    assert int(status) == 1
    assert out.sum(1).tolist() == [8.0, 0.0, 0.0, 8.0]
    status.zero_()
    got = kda.embedding_backward(torch.ones((4, 8), device="cuda"), ids, 4, dev_status=status)
    assert int(status) == 1
    assert got.sum(1).tolist() == [8.0, 0.0, 0.0, 8.0]


def test_embedding_without_tokens():
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    d = torch.empty((0, 16), device="cuda")
    assert kda.embedding(torch.ones((3, 16), device="cuda"), ids).shape == (0, 16)
    assert torch.equal(kda.embedding_backward(d, ids, 3), torch.zeros((3, 16), device="cuda"))


# ----------------------------------------------------------------- cross entropy

def _check_ce(dtype, x, w, y, d_loss, ignore=-100, piece=0):
    T, V, D = x.shape[0], w.shape[0], x.shape[1]
    x64, w64 = x.double(), w.double()
    z = x64 @ w64.T
    kept = y != ignore
    at = torch.where(kept, y, 0).long()[:, None]
    lse = torch.logsumexp(z, 1)
    loss_ref = torch.where(kept, lse - z.gather(1, at)[:, 0], 0.0)
    loss, got_lse, mean = kda.linear_cross_entropy(x, w, y, ignore_index=ignore)
    # a logit: its D products in fp32, one rounding each step of 16
    steps = (6 if dtype == "f32" else 1) * (D / 16.0) + 16
    size = (x64.abs() @ w64.abs().T).max(1).values
    err = 2.0 ** -23 * (steps * size + 8 * lse.abs() + 8)
    assert ((got_lse.double() - lse).abs() <= err).all()
    assert ((loss.double() - loss_ref).abs() <= 2 * err).all()
    assert not loss[~kept].any()
    n = int(kept.sum())
    ref_mean = float(loss_ref.sum()) / n if n else 0.0
    assert abs(float(mean) - ref_mean) <= 2 * float(err.max()) + 1e-6 * float(loss_ref.abs().max())
    # backward, with the row statistics that the forward gave
    dx, dw = kda.linear_cross_entropy_backward(x, w, y, got_lse, d_loss, ignore_index=ignore,
                                               piece=piece)
    p = torch.exp(z - got_lse.double()[:, None])
    hot = torch.zeros_like(z).scatter_(1, at, 1.0)
    g = torch.where(kept, d_loss, 0.0).double()[:, None]
    dz, dz_size = (p - hot) * g, (p + hot) * g.abs()
    # dz carries its logit's error (relative) and, in BF16, one rounding; the products
    # add one fp32 rounding per step of 16
    for got, ref, terms, k in ((dx, dz @ w64, dz_size @ w64.abs(), V),
                               (dw, dz.T @ x64, dz_size.T @ x64.abs(), T)):
        extra = float(err.max()) + 2.0 ** -23 * ((6 if dtype == "f32" else 1) * (k / 16.0) + 16)
        extra += 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
        _close(got, ref, dtype, terms, extra)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D,piece", [
    (1, 1, 1, 0),
    (1, 5, 8, 0),
    (1, 1000, 64, 0),
    (5, 257, 31, 0),
    (128, 256, 64, 0),
    (129, 255, 72, 0),
    (300, 1000, 520, 256),
    (257, 2049, 128, 512),
    (77, 5003, 100, 0),
    (1000, 700, 1024, 256),
    (2500, 4000, 256, 0),
    (300, 20011, 120, 4096),
    (70, 9000, 643, 4096),
    (6000, 50, 102, 0),
    (3001, 300, 77, 256),
    (513, 1537, 1001, 0),
])
def test_cross_entropy(dtype, T, V, D, piece):
    g, dt = _gen(T + V + D), DT[dtype]
    x, w = _randn((T, D), g, dt), _randn((V, D), g, dt, 2.0 / math.sqrt(D))
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[torch.rand(T, generator=g, device="cuda") < 0.2] = -100
    d = torch.rand(T, generator=g, device="cuda") - 0.3
    _check_ce(dtype, x, w, y.int() if T % 2 else y, d, piece=piece)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cross_entropy_of_large_logits(dtype):
    """Logits of hundreds: exp would overflow without the running maximum."""
    g, dt = _gen(2), DT[dtype]
    x, w = _randn((40, 64), g, dt, 8.0), _randn((600, 64), g, dt, 8.0)
    y = torch.randint(0, 600, (40,), generator=g, device="cuda")
    _check_ce(dtype, x, w, y, torch.ones(40, device="cuda"))


def test_cross_entropy_gradient_of_a_mean_is_not_scaled_by_rounding():
    """d_loss halfway between two BF16 values and equal in all rows: rounded into dz it would
    move every gradient by 2^-8.  The output's own rounding is at most 2^-8 of an element,
    evenly spread at worst: 2^-8 / sqrt 3 of the norm; a tenth more for the softmax's."""
    g = _gen(11)
    x, w = _randn((40, 256), g, torch.bfloat16), _randn((3000, 256), g, torch.bfloat16, 0.1)
    y = torch.randint(0, 3000, (40,), generator=g, device="cuda")
    d = torch.full((40,), 2.0 ** -5 * (1 + 2.0 ** -8), device="cuda")
    _, lse, _ = kda.linear_cross_entropy(x, w, y)
    got = kda.linear_cross_entropy_backward(x, w, y, lse, d)
    z = x.double() @ w.double().T
    dz = (torch.softmax(z, 1) - torch.nn.functional.one_hot(y, 3000)) * d.double()[:, None]
    for a, ref in zip(got, (dz @ w.double(), dz.T @ x.double())):
        assert (a.double() - ref).norm() <= 1.1 * 2.0 ** -8 / math.sqrt(3) * ref.norm()


def test_cross_entropy_with_nothing_to_predict():
    x, w = torch.ones((6, 16), device="cuda"), torch.ones((50, 16), device="cuda")
    y = torch.full((6,), 7, device="cuda")
    loss, lse, mean = kda.linear_cross_entropy(x, w, y, ignore_index=7)
    assert not loss.any() and float(mean) == 0.0
    dx, dw = kda.linear_cross_entropy_backward(x, w, y, lse, torch.ones(6, device="cuda"),
                                               ignore_index=7)
    assert not dx.any() and not dw.any()
    e = torch.empty((0, 16), device="cuda")
    y = torch.empty(0, dtype=torch.int32, device="cuda")
    loss, lse, mean = kda.linear_cross_entropy(e, w, y)
    assert loss.numel() == 0 and float(mean) == 0.0
    dx, dw = kda.linear_cross_entropy_backward(e, w, y, lse, loss)
    assert dx.shape == (0, 16) and not dw.any()


def test_cross_entropy_reports_targets_outside_the_vocabulary():
    g = _gen(4)
    x, w = _randn((4, 32), g, torch.bfloat16), _randn((9, 32), g, torch.bfloat16)
    y = torch.tensor([3, 9, -1, -100], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse, mean = kda.linear_cross_entropy(x, w, y, dev_status=status)
    assert int(status) == 1
    assert loss[1:].tolist() == [0.0, 0.0, 0.0] and float(mean) == float(loss[0])
    status.zero_()
    dx, dw = kda.linear_cross_entropy_backward(x, w, y, lse, torch.ones(4, device="cuda"),
                                               dev_status=status)
    assert int(status) == 1 and not dx[1:].any() and bool(dx[0].any())


def test_cross_entropy_matches_differences():
    """dx and d_weight against central differences of the forward in 64 bits."""
    g = _gen(6)
    x, w = _randn((3, 8), g, torch.float32), _randn((5, 8), g, torch.float32)
    y, d = torch.tensor([1, -100, 4], device="cuda"), torch.tensor([0.5, 9.0, -1.0], device="cuda")

    def f(x, w):
        z = x @ w.T
        rows = torch.tensor([0, 2], device="cuda")
        return float((d[rows].double() * (torch.logsumexp(z, 1)[rows] - z[rows, y[rows]])).sum())

    _, lse, _ = kda.linear_cross_entropy(x, w, y)
    got = kda.linear_cross_entropy_backward(x, w, y, lse, d)
    args = [x.double(), w.double()]
    for k in range(2):
        for i in range(args[k].numel()):
            vals = []
            for s in (1e-5, -1e-5):
                moved = [t.clone() for t in args]
                moved[k].view(-1)[i] += s
                vals.append(f(*moved))
            assert abs(float(got[k].view(-1)[i]) - (vals[0] - vals[1]) / 2e-5) < 2e-4


# --------------------------------------------------------------- refusals, autograd

def test_binding_refuses_what_the_kernels_do_not_take():
    x = torch.zeros((4, 2, 8), device="cuda")
    w, h = torch.ones(8, device="cuda"), torch.zeros((4, 8), device="cuda")
    for bad in (lambda: kda.gated_norm(x, x.bfloat16(), w),
                lambda: kda.gated_norm(x, x[:3], w),
                lambda: kda.gated_norm(x, x, w.double()),
                lambda: kda.gated_norm(x, x, w, act="tanh"),
                lambda: kda.gated_norm(x, None, w),
                lambda: kda.gated_norm(x, x, w, act="none"),
                lambda: kda.gated_norm(x.half(), x.half(), w),
                lambda: kda.gated_norm(x.transpose(0, 1), x.transpose(0, 1), w),
                lambda: kda.gated_norm(x[:, :, ::2], x[:, :, ::2], w[:4]),
                lambda: kda.gated_norm(x, x, w, out=x[:2]),
                lambda: kda.residual_norm(h.T, None),
                lambda: kda.residual_norm(h, h.bfloat16()),
                lambda: kda.residual_norm(h, None, h_out=h),
                lambda: kda.embedding(h, torch.zeros(2, device="cuda")),
                lambda: kda.embedding(h, torch.zeros((2, 2), device="cuda", dtype=torch.int32)),
                lambda: kda.embedding_backward(h, torch.zeros(3, device="cuda", dtype=torch.int32), 5),
                lambda: kda.linear_cross_entropy(h, w[None, :4], torch.zeros(4, device="cuda").long()),
                lambda: kda.linear_cross_entropy(h, h, torch.zeros(3, device="cuda").long()),
                lambda: kda.linear_cross_entropy(h, h.bfloat16(), torch.zeros(4, device="cuda").long())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        kda.gated_norm(x, [1.0], w)
    with pytest.raises(kda.KDAError):
        kda.gated_norm(x, x, w, eps=0.0)
    with pytest.raises(kda.KDAError):  # x is not on a 16-byte boundary
        kda.linear_cross_entropy(torch.zeros(33, device="cuda")[1:].view(4, 8), h,
                                 torch.zeros(4, device="cuda").long())


def test_autograd_matches_torch():
    """The differentiable forms in one small network against torch's own autograd in 64
    bits (fp32 activations)."""
    from kimi_delta_attention_18_gb300 import autograd as ag
    g = _gen(8)
    table, head = _randn((11, 12), g, torch.float32), _randn((11, 12), g, torch.float32)
    z, w1, w2 = _randn((7, 12), g, torch.float32), _randn((4,), g, torch.float32), _randn((12,), g, torch.float32)
    ids = torch.randint(0, 11, (7,), generator=g, device="cuda")
    y = torch.randint(0, 11, (7,), generator=g, device="cuda")
    y[2] = -100
    for reduction in ("mean", "sum", "none"):
        mine = [t.clone().requires_grad_() for t in (table, z, w1, w2, head)]
        e = ag.kda_embedding(mine[0], ids, scale=2.0)
        h, n = ag.kda_residual_norm(e, None, mine[3])
        u = ag.kda_gated_norm(n.view(7, 3, 4), mine[1].view(7, 3, 4), mine[2], act="silu")
        h, n = ag.kda_residual_norm(h, u.view(7, 12), mine[3], scale=0.5)
        loss = ag.kda_linear_cross_entropy(n + h, mine[4], y, reduction=reduction)
        (loss * 3.0).sum().backward()
        ref = [t.double().requires_grad_() for t in (table, z, w1, w2, head)]

        def norm(v):
            return v * (v.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()

        h = 2.0 * ref[0][ids]
        n = norm(h) * ref[3]
        u = norm(n.view(7, 3, 4)) * ref[2] * torch.nn.functional.silu(ref[1].view(7, 3, 4))
        h = h + 0.5 * u.view(7, 12)
        want = torch.nn.functional.cross_entropy((norm(h) * ref[3] + h) @ ref[4].T, y,
                                                 reduction=reduction)
        (want * 3.0).sum().backward()
        assert torch.allclose(loss.double(), want, rtol=1e-5, atol=1e-5)
        for a, b in zip(mine, ref):
            assert a.grad.dtype == torch.float32
            assert torch.allclose(a.grad.double(), b.grad, rtol=1e-4, atol=1e-4)


def test_example_trains():
    """The operators together, as they are used: the loss of the example's model falls
    from that of a uniform guess (log 199 = 5.3)."""
    from examples.train_lm import train
    losses = train(steps=40, log=lambda s: None)
    assert 4.5 < losses[0] < 6.5 and losses[-1] < 0.5 * losses[0]


def test_calls_are_captured_in_a_graph():
    """Nothing is allocated or synchronised behind a capture's back."""
    g = _gen(9)
    x, w = _randn((64, 256), g, torch.bfloat16), _randn((500, 256), g, torch.bfloat16, 0.1)
    y = torch.randint(0, 500, (64,), generator=g, device="cuda")
    d = torch.rand(64, generator=g, device="cuda")

    def run():
        h, n = kda.residual_norm(x, x, None, scale=0.5)
        loss, lse, mean = kda.linear_cross_entropy(n, w, y)
        dx, dw = kda.linear_cross_entropy_backward(n, w, y, lse, d)
        return [mean, dw, kda.residual_norm_backward(dx, h, None)[0],
                kda.embedding_backward(dx, y, 500)]

    want = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D", [(200, 300, 64), (7, 1000, 72), (300, 129, 31)])
def test_cross_entropy_of_rows_with_nan_where_ignored(dtype, T, V, D):
    """Padding may hold anything: an ignored row of NaN and infinities changes nothing."""
    g, dt = _gen(11), DT[dtype]
    x, w = _randn((T, D), g, dt), _randn((V, D), g, dt, 0.1)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::3] = -100
    d = torch.rand(T, generator=g, device="cuda")
    bad = x.clone()
    bad[::3] = float("nan")
    bad[3::6] = float("inf")
    clean = x.clone()
    clean[::3] = 0
    kept = y != -100
    loss, lse, mean = kda.linear_cross_entropy(bad, w, y)
    ref, ref_lse, ref_mean = kda.linear_cross_entropy(clean, w, y)
    assert torch.equal(loss, ref) and torch.equal(mean, ref_mean)
    assert torch.equal(lse[kept], ref_lse[kept])
    dx, dw = kda.linear_cross_entropy_backward(bad, w, y, lse, d)
    ref_dx, ref_dw = kda.linear_cross_entropy_backward(clean, w, y, ref_lse, d)
    assert torch.equal(dw, ref_dw) and torch.equal(dx, ref_dx)
    assert not dx[::3].any()


def test_workspaces_on_another_stream():
    """A call on a stream of its own keeps its workspace until its kernels are done."""
    g = _gen(12)
    x, w = _randn((2000, 512), g, torch.bfloat16), _randn((20000, 512), g, torch.bfloat16, 0.1)
    y = torch.randint(0, 20000, (2000,), generator=g, device="cuda")
    want, _, _ = kda.linear_cross_entropy(x, w, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got, _, _ = kda.linear_cross_entropy(x, w, y, stream=s)
        torch.full((1_000_000,), 7.0, device="cuda")  # would land in a freed workspace
        s.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("T,V,D,piece", [
    (1 << 20, 512, 64, 256),     # d_weight over 2^20 tokens
    (64, 256, 1 << 17, 0),       # logits of 2^17 channels
    (1216, 131072, 4096, 0),     # dx over 131,072 columns
])
def test_cross_entropy_gradient_of_long_sums(T, V, D, piece):
    """BF16 gradients whose sums are long and of one sign (the targets are elsewhere): the
    tensor core's truncation at every step would add up to 0.6 % of d_weight, 0.8 % of the
    logits here.  Bounds: one rounding to BF16 of dz and one of the result, each at most
    2^-8 and evenly spread, so 2^-8 / sqrt 3 of the norm each; a tenth more for the rest."""
    g = _gen(T + D)
    scale = 1.0 + torch.rand(D, generator=g, device="cuda")
    if T > V:  # logits about 1 / 64
        x = ((1.0 + 0.1 * torch.randn((T, D), generator=g, device="cuda")) * scale).bfloat16()
        w = _randn((V, D), g, torch.bfloat16, 1.0 / D)
    elif D > V:  # logits between 10 and 11
        x = ((1.0 + 0.1 * torch.randn((T, D), generator=g, device="cuda")) * scale).bfloat16()
        rows = 10.0 + torch.rand(V, generator=g, device="cuda")
        w = (rows[:, None] / (1.5 * D) * torch.ones(D, device="cuda")).bfloat16()
    else:  # a softmax over many rows of one sign
        x = _randn((T, D), g, torch.bfloat16, 10.0 / math.sqrt(D))
        w = ((1.0 + 0.1 * torch.randn((V, D), generator=g, device="cuda")) * scale).bfloat16()
        w[V - 1] = 0.0
    y = torch.randint(V // 2, V, (T,), generator=g, device="cuda")
    if V > T:
        y.fill_(V - 1)
    d = torch.ones(T, device="cuda")
    _, lse, _ = kda.linear_cross_entropy(x, w, y)
    dx, dw = kda.linear_cross_entropy_backward(x, w, y, lse, d, piece=piece)
    if T < V and V > D:
        rows = torch.arange(16, device="cuda") * (T // 16)
        p = torch.exp(x[rows].double() @ w.double().T - lse[rows, None].double())
        got, ref = dx[rows], p @ w.double()  # the target's row of w is zero
    else:
        cols = torch.arange(32, device="cuda") * (V // 64)
        ref = torch.zeros((32, D), dtype=torch.float64, device="cuda")
        for i in range(0, T, 131072):
            part = x[i:i + 131072].double()
            p = torch.exp(part @ w[cols].double().T - lse[i:i + 131072, None].double())
            ref += p.T @ part
        got = dw[cols]
    bound = 1.1 * math.sqrt(2.0) * 2.0 ** -8 / math.sqrt(3.0)
    assert (got.double() - ref).norm() <= bound * ref.norm()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,D,act,strided", [
    (1500, 56, 128, "sigmoid", False),
    (1500, 56, 128, "silu", False),
    (1500, 56, 128, "none", False),
    (1500, 56, 128, "sigmoid", True),    # tokens apart, more than 2 KB each
    (3200, 1, 1032, "sigmoid", False),   # BF16: 96 threads a row
    (5200, 1, 1024, "silu", False),      # 64 threads a row, 8 rows a tile
    (700, 1, 5120, "sigmoid", False),    # a row a tile, 384 threads
    (700, 1, 7168, "silu", False),       # 512 threads
    (2000, 56, 33, "sigmoid", False),    # rows as pairs
    (25000, 3, 65, "none", False),
])
def test_gated_norm_of_rows_through_shared_memory(dtype, T, H, D, act, strided):
    """Rows enough for the ring in shared memory (four tiles for each of 152 SMs), in each of
    its forms: a row in part of a warp, in several warps, alone in its tile; with the next
    row's sums before this row's outputs (BF16 gradients of rows wider than a warp)."""
    test_gated_norm(dtype, T, H, D, act, True, strided)


def test_tensors_of_calls_on_another_stream_are_kept():
    """With stream=, neither an output that the caller drops before the call's kernels have
    run nor memory that the current stream still writes is shared with anything else."""
    g = _gen(13)
    T, V, D = 1500, 4000, 256
    x, w = _randn((T, D), g, torch.bfloat16), _randn((V, D), g, torch.bfloat16, 0.1)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    d = torch.rand(T, generator=g, device="cuda")
    _, lse, _ = kda.linear_cross_entropy(x, w, y)
    h, wn = x.view(T, 2, 128), torch.ones(128, device="cuda")
    calls = [lambda s: kda.linear_cross_entropy(x, w, y, stream=s),
             lambda s: kda.linear_cross_entropy_backward(x, w, y, lse, d, stream=s),
             lambda s: kda.gated_norm_backward(h, h, h, wn, stream=s),
             lambda s: kda.residual_norm(x, x, None, stream=s),
             lambda s: kda.residual_norm_backward(x, x, None, x, scale=0.5, stream=s),
             lambda s: (kda.embedding(w, y, stream=s), kda.embedding_backward(x, y, V, stream=s))]
    s = torch.cuda.Stream()
    for call in calls:
        want = [t.clone() for t in call(None)]
        sizes = [t.numel() * t.element_size() for t in want] + [1 << 16, 1 << 20, 1 << 22, 1 << 24]
        torch.cuda.synchronize()
        for kept in range(len(want)):
            torch.cuda._sleep(20_000_000)  # late writes of the current stream to memory it gave back
            for n in sizes:
                torch.full((n,), 7, dtype=torch.uint8, device="cuda")
            with torch.cuda.stream(s):
                torch.cuda._sleep(40_000_000)  # the call's kernels come later than what follows
            out = call(s)[kept]  # the others are dropped
            others = [torch.full((n,), 9, dtype=torch.uint8, device="cuda") for n in sizes for _ in (0, 1)]
            torch.cuda.synchronize()
            assert torch.equal(out, want[kept])
            assert all(bool((t == 9).all()) for t in others)
            del out, others


def test_arguments_of_calls_on_another_stream_are_kept():
    """An argument that the caller drops at once (a copy made for the call) stays whole until
    the call's kernels have read it."""
    x = torch.randn((3000, 512), device="cuda")
    want = kda.residual_norm(x, x, scale=0.0)[1]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)
    s.wait_stream(torch.cuda.current_stream())
    copy = x.clone()
    s.wait_stream(torch.cuda.current_stream())
    _, out = kda.residual_norm(copy, copy, stream=s, scale=0.0)
    del copy
    torch.full((3000, 512), 9.0, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("large,small", [(1e30, 1e-20), (1.0, 1e-30), (1.7e38, 1e-3), (3e-36, 1e-36)])
def test_cross_entropy_gradient_of_rows_of_unequal_weight(large, small):
    """BF16: a row's dx does not depend on how large the other rows' d_loss is.  Bound: a
    rounding to BF16 of each term and of the result, 2^-8 each at most."""
    g = _gen(14)
    x, w = _randn((48, 128), g, torch.bfloat16), _randn((300, 128), g, torch.bfloat16, 0.1)
    y = torch.randint(0, 300, (48,), generator=g, device="cuda")
    d = torch.where(torch.arange(48, device="cuda") % 2 == 0, large, small)
    _, lse, _ = kda.linear_cross_entropy(x, w, y)
    dx, dw = kda.linear_cross_entropy_backward(x, w, y, lse, d)
    p = torch.softmax(x.double() @ w.double().T, 1)
    dz = (p - torch.nn.functional.one_hot(y, 300)) * d.double()[:, None]
    for got, ref, terms in ((dx, dz @ w.double(), dz.abs() @ w.double().abs()),
                            (dw, dz.T @ x.double(), dz.T.abs() @ x.double().abs())):
        beyond = ref.abs() > torch.finfo(torch.bfloat16).max  # no BF16 value: infinite
        assert torch.equal(got[beyond].double(), ref[beyond].sign() * math.inf)
        err = torch.where(beyond, 0.0, got.double() - ref).norm(dim=1)
        assert (err <= 2.0 ** -8 * (terms.norm(dim=1) + ref.norm(dim=1)) * 1.01).all()


def test_differentiable_forms_report_errors():
    """An id outside the table, a target outside the vocabulary: in dev_status, from the
    forward pass and again from the backward pass."""
    from kimi_delta_attention_18_gb300 import autograd as ag
    table = torch.ones((4, 8), device="cuda", requires_grad=True)
    bad, good = torch.tensor([0, 4], device="cuda"), torch.tensor([0, 3], device="cuda")
    for f in (lambda ids, s: ag.kda_embedding(table, ids, dev_status=s),
              lambda ids, s: ag.kda_linear_cross_entropy(table[:2], table, ids, dev_status=s)):
        for ids, code in ((bad, 1), (good, 0)):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = f(ids, status)
            assert int(status) == code
            status.zero_()
            out.sum().backward()
            assert int(status) == code


@pytest.mark.parametrize("T,V,D,piece", [
    (96, 4000, 1024, 0),      # the fp32 weight split on its way (up to 128 tokens, whole fours)
    (100, 1500, 256, 256),    # the same in pieces of the vocabulary
    (300, 3001, 515, 0),      # operands stored as terms
    (300, 3001, 515, 512),
])
def test_cross_entropy_of_fp32_is_accurate(T, V, D, piece):
    """fp32 operands are three BF16 terms each and six products.  With the rounding of exp's
    argument (up to 3e-7 of a term) the gradients are within about 6e-7 of the norm; five
    products would be 2.6e-6 off, three 4.5e-6 (in 64 bits, these sizes).  lse: 3e-7 and
    fp32's spacing."""
    g = _gen(T + V)
    x, w = _randn((T, D), g, torch.float32), _randn((V, D), g, torch.float32, 2.0 / math.sqrt(D))
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    d = torch.rand(T, generator=g, device="cuda") - 0.3
    z = x.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    _, got, _ = kda.linear_cross_entropy(x, w, y)
    assert ((got.double() - lse) / lse).pow(2).mean().sqrt() <= 1e-6
    lse = lse.float()
    dz = (torch.exp(z - lse.double()[:, None]) - torch.nn.functional.one_hot(y, V)) * d.double()[:, None]
    dx, dw = kda.linear_cross_entropy_backward(x, w, y, lse, d, piece=piece)
    for got, ref in ((dx, dz @ w.double()), (dw, dz.T @ x.double())):
        assert (got.double() - ref).norm() <= 2e-6 * ref.norm()


def test_cross_entropy_row_statistics_of_a_wide_row_are_accurate():
    """BF16, 7,168 channels: lse within 3e-7 (2.3e-6 if one accumulator took the whole sum,
    which the tensor core truncates at every step)."""
    g = _gen(15)
    x, w = _randn((64, 7168), g, torch.bfloat16), _randn((2000, 7168), g, torch.bfloat16, 2.0 / math.sqrt(7168))
    y = torch.randint(0, 2000, (64,), generator=g, device="cuda")
    lse = torch.logsumexp(x.double() @ w.double().T, 1)
    got = kda.linear_cross_entropy(x, w, y)[1]
    assert ((got.double() - lse) / lse).pow(2).mean().sqrt() <= 1e-6


@pytest.mark.parametrize("dtype,T,V,D,piece", [
    ("f32", 100, 1000, 64, 256),     # an fp32 weight read in pieces, dx added up over them
    ("f32", 128, 700, 132, 512),
    ("bf16", 4100, 131072, 72, 0),   # more than one piece by default
])
def test_cross_entropy_in_pieces(dtype, T, V, D, piece):
    test_cross_entropy(dtype, T, V, D, piece)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D", [(3000, 500, 701), (700, 9000, 517)])
def test_embedding_of_wide_rows_that_are_not_whole_pieces(dtype, T, V, D):
    """Four single columns per thread; frequent ids, and runs of absent ones."""
    test_embedding(dtype, T, V, D, "text", torch.int32)
