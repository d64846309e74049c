"""A recurrent layer's parts beside the mixer against their formulas in 64 bits: the gated
linear recurrence, the gated feed-forward block and dropout, forward and backward.

Bounds.  A rounding to BF16 is up to 2^-8 of the value, to fp32 2^-24.  What an operator
sums in fp32 is held to a number of fp32 roundings of the terms' magnitudes, derived at
each test's reference.
"""
import math

import pytest
import torch

import kimi_delta_attention_18_gb300 as kda
from kimi_delta_attention_18_gb300 import autograd
from oracle.philox import keep_mask

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dt=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def _within(got, ref, bound, what=""):
    assert got.shape == ref.shape
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %g, first at %s" % (
        what, int(bad.sum()), bad.numel(), float((got.double() - ref).abs().max()),
        bad.nonzero()[0].tolist())


# ------------------------------------------------------------ linear recurrence
#
# A step in fp32 multiplies by a factor that is up to 2^-22 of itself off where it comes
# from ex2.approx (its argument's rounding adds |g| e^g 2^-24 < 2^-25; slow decays are off
# by one rounding), adds and rounds; a map's factor and term carry the same errors as the
# steps they stand for, plus one rounding each per join.  Sixteen roundings a step of the
# state that the terms' magnitudes would give (S below) cover it:
#     E_t = e^g E_{t-1} + 16 2^-24 S_t.
STEP = 16 * U


def _recurrence64(x, g, h0, cu, write):
    """h, h_final, and how far they may be off."""
    x, a = x.double(), torch.exp(g.double())
    if write == "mix":
        x = x * -torch.expm1(g.double())
    h, err = torch.empty_like(x), torch.empty_like(x)
    N, C = len(cu) - 1, x.shape[1]
    final = torch.zeros((N, C), device="cuda", dtype=torch.float64)
    final_err = torch.zeros_like(final)
    for n in range(N):
        s = torch.zeros(C, device="cuda", dtype=torch.float64) if h0 is None else h0[n].double()
        size, e = s.abs(), torch.zeros_like(s)
        for t in range(cu[n], cu[n + 1]):
            s = a[t] * s + x[t]
            size = a[t] * size + x[t].abs()
            e = a[t] * e + STEP * size
            h[t], err[t] = s, e
        final[n], final_err[n] = s, e
    return h, err, final, final_err


def _recurrence_grad64(d_h, x, g, h, h0, cu, d_final, write):
    x, h, d, a = x.double(), h.double(), d_h.double(), torch.exp(g.double())
    w = -torch.expm1(g.double()) if write == "mix" else torch.ones_like(a)
    dx, dg, dx_err, dg_err = (torch.empty_like(x) for _ in range(4))
    N, C = len(cu) - 1, x.shape[1]
    d0 = torch.zeros((N, C), device="cuda", dtype=torch.float64)
    d0_err = torch.zeros_like(d0)
    for n in range(N):
        u = torch.zeros(C, device="cuda", dtype=torch.float64) if d_final is None else d_final[n].double()
        size, e = u.abs(), torch.zeros_like(u)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            dh, size = d[t] + u, d[t].abs() + size
            dx[t], dx_err[t] = w[t] * dh, w[t] * (e + STEP * size)
            u, size = a[t] * dh, a[t] * size
            e = a[t] * e + STEP * size
            before = h[t - 1] if t > cu[n] else h[t] * 0 if h0 is None else h0[n].double()
            dg[t] = u * (before - x[t] if write == "mix" else before)
            dg_err[t] = (e + 2 * U * u.abs()) * (before.abs() + (x[t].abs() if write == "mix" else 0))
        d0[n], d0_err[n] = u, e
    return dx, dx_err, dg, dg_err, d0, d0_err


def _gates(T, C, g, slow=True):
    """Log-decays from a thousand tokens to one, some that keep or drop everything."""
    rate = torch.exp(torch.rand(C, generator=g, device="cuda") * 6.9 - (6.9 if slow else 0.0))
    v = -rate * torch.exp(0.5 * torch.randn((T, C), generator=g, device="cuda"))
    pick = torch.rand((T, C), generator=g, device="cuda")
    v = torch.where(pick < 0.01, torch.zeros_like(v), v)
    return torch.where(pick > 0.99, torch.full_like(v, -math.inf), v)


def _cu(lengths):
    return torch.tensor([0] + list(lengths), device="cuda").cumsum(0).to(torch.int32)


CASES = [  # lengths, channels
    ([1], 1), ([0, 3, 0], 2), ([7], 3), ([127, 1], 64), ([128], 65), ([129], 63), ([300, 0, 724], 66),
    ([1024], 2), ([1025], 130), ([0, 1200, 0, 0, 1, 127, 128, 129, 0], 67), ([400] * 5, 4),
    ([4993], 5), ([2100, 37, 2600], 128), ([1] * 1300, 3), ([0] * 40 + [1500] + [0] * 40, 64),
]


@pytest.mark.parametrize("write", ["add", "mix"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,C", CASES, ids=lambda v: str(v) if isinstance(v, int) else "n%d-t%d" % (len(v), sum(v)))
def test_recurrence(lengths, C, act, write):
    g = _gen(sum(lengths) + C)
    T, N, dt = sum(lengths), len(lengths), DT[act]
    cu = _cu(lengths)
    x, gate = _randn((T, C), g, dt), _gates(T, C, g)
    h0 = _randn((N, C), g) if C % 3 else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, h_final = kda.linear_recurrence(x, gate, h0, cu, write=write, dev_status=status)
    ref, err, final, final_err = _recurrence64(x, gate, h0, cu.tolist(), write)
    _within(h, ref, ROUND[act] * ref.abs() * (1 + 2 * U) + 2 * err, "h")
    _within(h_final, final, final_err + U * final.abs(), "h_final")

    d_h, d_final = _randn((T, C), g, dt), _randn((N, C), g) if C % 2 else None
    got = kda.linear_recurrence_backward(d_h, x, gate, h, h0, cu, d_final, write=write,
                                         dev_status=status)
    dx, dx_err, dg, dg_err, d0, d0_err = _recurrence_grad64(d_h, x, gate, h, h0, cu.tolist(),
                                                            d_final, write)
    _within(got[0], dx, ROUND[act] * dx.abs() + 2 * dx_err, "dx")
    _within(got[1], dg, U * dg.abs() + 2 * dg_err, "dg")
    _within(got[2], d0, U * d0.abs() + d0_err, "d_h0")
    assert int(status) == 0
    # the same bits again, whatever order the tiles were worked in
    again = kda.linear_recurrence(x, gate, h0, cu, write=write)
    assert torch.equal(again[0], h) and torch.equal(again[1], h_final)
    more = kda.linear_recurrence_backward(d_h, x, gate, h, h0, cu, d_final, write=write)
    assert all(torch.equal(p, q) for p, q in zip(more, got))


def test_recurrence_gradient_against_differences():
    """Central differences of the library's own forward (fp32; h0, x and g moved by 2^-7: the
    forward is linear in x and h0, and in g the third derivative adds 2^-14 / 6 of it)."""
    g = _gen(3)
    lengths, C = [5, 0, 9], 2
    cu, T = _cu(lengths), 14
    x, h0 = _randn((T, C), g), _randn((3, C), g)
    gate = -torch.rand((T, C), generator=g, device="cuda") - 0.05
    d_h, d_final = _randn((T, C), g), _randn((3, C), g)
    for write in ("add", "mix"):
        def value(x, gate, h0):
            h, last = kda.linear_recurrence(x, gate, h0, cu, write=write)
            return float((h.double() * d_h).sum() + (last.double() * d_final).sum())
        h = kda.linear_recurrence(x, gate, h0, cu, write=write)[0]
        dx, dg, d0 = kda.linear_recurrence_backward(d_h, x, gate, h, h0, cu, d_final, write=write)
        step = 2.0 ** -7
        # a difference divides the forward's fp32 errors (up to 2^-20 of a sum of about 40) by
        # 2 step: 2.5e-3; the gradients are of order 1
        for which, grad in (("x", dx), ("g", dg), ("h0", d0)):
            src = {"x": x, "g": gate, "h0": h0}
            for i in range(0, src[which].numel(), 3):
                moved = []
                for sign in (1, -1):
                    m = dict(src)
                    m[which] = src[which].clone()
                    m[which].view(-1)[i] += sign * step
                    moved.append(value(m["x"], m["g"], m["h0"]))
                slope = (moved[0] - moved[1]) / (2 * step)
                assert abs(slope - float(grad.view(-1)[i])) < 5e-3, (write, which, i)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T", [700, 3000])
def test_recurrence_strided_and_odd_bases(T, act):
    g, dt, C = _gen(T), DT[act], 70
    wide, wide_g = _randn((T, 3, C), g, dt), _gates(T, 2 * C, g).view(T, 2, C)
    for x, gate in ((wide[:, 1], wide_g[:, 1]), (wide.view(T, 3 * C)[:, 1:C + 1], wide_g[:, 0])):
        h, last = kda.linear_recurrence(x, gate, write="mix")
        plain, plain_last = kda.linear_recurrence(x.contiguous(), gate.contiguous(), write="mix")
        assert torch.equal(h, plain) and torch.equal(last, plain_last)
        got = kda.linear_recurrence_backward(h, x, gate, h, write="mix")
        ref = kda.linear_recurrence_backward(h, x.contiguous(), gate.contiguous(), h, write="mix")
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_recurrence_of_growing_factors_and_infinities():
    """Factors whose product overflows do not turn a zero state into NaN; a NaN and an infinity
    stay in their channel and sequence, and g = -inf starts anew."""
    T, C = 2600, 4
    x, g = torch.zeros((T, C), device="cuda"), torch.full((T, C), 3.0, device="cuda")
    cu = _cu([1300, 1300])
    h, last = kda.linear_recurrence(x, g, None, cu)
    assert bool((h == 0).all()) and bool((last == 0).all())
    g.fill_(-0.5)
    x.fill_(1.0)
    x[100, 1] = math.nan
    x[200, 2] = math.inf
    g[700, 1] = g[700, 2] = -math.inf
    h, last = kda.linear_recurrence(x, g, None, cu)
    assert bool(torch.isfinite(h[:, [0, 3]]).all()) and bool(torch.isfinite(h[1300:]).all())
    assert bool(torch.isnan(h[100:700, 1]).all()) and bool(torch.isinf(h[200:205, 2]).all())
    # past the reset 0 * NaN and 0 * inf are NaN, as the formula says
    assert bool(torch.isnan(h[700:1300, 1:3]).all())


def test_recurrence_past_32_bits():
    """More elements than 32 bits count; with e^-1 a step, 64 tokens decide the last ones."""
    T, C = 70001, 65536
    x = torch.empty((T, C), device="cuda", dtype=torch.bfloat16).normal_()
    g = torch.full((T, C), -1.0, device="cuda")
    h, last = kda.linear_recurrence(x, g)
    tail = slice(T - 80, T)
    ref, err, final, final_err = _recurrence64(x[tail], g[tail], None, [0, 80], "add")
    _within(h[T - 16:], ref[64:], ROUND["bf16"] * ref[64:].abs() + 2 * err[64:] + 1e-26, "h")
    _within(last, final, final_err + 1e-26, "h_final")
    del last
    dx, dg, d0 = kda.linear_recurrence_backward(h, x, g, h)
    start = slice(0, 80)
    ref = _recurrence_grad64(h[start], x[start], g[start], h[start], None, [0, 80], None, "add")
    _within(dx[:16], ref[0][:16], ROUND["bf16"] * ref[0][:16].abs() + 2 * ref[1][:16] + 1e-24, "dx")
    _within(dg[:16], ref[2][:16], U * ref[2][:16].abs() + 2 * ref[3][:16] + 1e-24, "dg")
    ref = _recurrence_grad64(h[tail], x[tail], g[tail], h[tail], None, [0, 80], None, "add")
    _within(dx[T - 79:], ref[0][1:], ROUND["bf16"] * ref[0][1:].abs() + 2 * ref[1][1:], "dx")
    _within(dg[T - 79:], ref[2][1:], U * ref[2][1:].abs() + 2 * ref[3][1:], "dg")


@pytest.mark.parametrize("write", ["add", "mix"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("N,C", [(1, 1), (3, 7), (5, 64), (256, 1001), (33, 4096)])
def test_recurrence_step(N, C, act, write):
    g, dt = _gen(N + C), DT[act]
    wide = _randn((N, 2, C), g, dt)
    for x in (wide[:, 0].contiguous(), wide[:, 1]):
        gate, state = _gates(N, C, g), _randn((N, C), g)
        ref, err, final, final_err = _recurrence64(x, gate, state, list(range(N + 1)), write)
        new = torch.full_like(state, math.nan)
        h, got = kda.linear_recurrence_step(x, gate, state, write=write, state_out=new)
        assert got is new
        _within(got, final, final_err + U * final.abs(), "state")
        _within(h, ref, ROUND[act] * ref.abs() * (1 + 2 * U) + 2 * err, "h")
        h2, same = kda.linear_recurrence_step(x, gate, state, write=write)  # in place
        assert same is state and torch.equal(state, new) and torch.equal(h2, h)


def test_recurrence_steps_continue_a_prefill():
    g, C = _gen(5), 96
    lengths = [37, 1500, 4]
    cu, T = _cu(lengths), sum(lengths)
    x, gate = _randn((T, C), g), _gates(T, C, g)
    h, last = kda.linear_recurrence(x, gate, None, cu, write="mix")
    more, more_gate = _randn((6, 3, C), g), _gates(18, C, g).view(6, 3, C)
    state = last.clone()
    steps = [kda.linear_recurrence_step(more[i], more_gate[i], state, write="mix")[0] for i in range(6)]
    one = torch.cat([torch.cat([x[cu[n]:cu[n + 1]], more[:, n]]) for n in range(3)])
    one_gate = torch.cat([torch.cat([gate[cu[n]:cu[n + 1]], more_gate[:, n]]) for n in range(3)])
    cu2 = _cu([n + 6 for n in lengths])
    ref, err, final, final_err = _recurrence64(one, one_gate, None, cu2.tolist(), "mix")
    _within(state, final, final_err, "state")
    for n in range(3):
        at = slice(int(cu2[n + 1]) - 6, int(cu2[n + 1]))
        _within(torch.stack([s[n] for s in steps]), ref[at], err[at] + U * ref[at].abs(), "h")


@pytest.mark.parametrize("T", [900, 5000])
def test_recurrence_bad_sequences_are_reported(T):
    """A malformed cu_seqlens: a status, no access outside the arrays."""
    x, g = torch.zeros((T, 8), device="cuda"), torch.zeros((T, 8), device="cuda")
    for cu in ([0, T - 1], [1, T], [0, 500, 400, T], [0, -3, T], [0, T + 7, T], [0, 2 ** 30, T]):
        for backward in (False, True):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            seqs = torch.tensor(cu, dtype=torch.int32, device="cuda")
            if backward:
                kda.linear_recurrence_backward(x, x, g, x, None, seqs, dev_status=status)
            else:
                kda.linear_recurrence(x, g, None, seqs, dev_status=status)
            assert int(status) == 1, (cu, backward)


def test_recurrence_states_may_be_updated_in_place():
    g, C = _gen(8), 64
    for lengths in ([300, 0, 5], [3000, 0, 41, 900]):
        cu, T, N = _cu(lengths), sum(lengths), len(lengths)
        x, gate, h0 = _randn((T, C), g), _gates(T, C, g), _randn((N, C), g)
        h, last = kda.linear_recurrence(x, gate, h0, cu)
        state = h0.clone()
        h2, same = kda.linear_recurrence(x, gate, state, cu, h_final=state)
        assert same is state and torch.equal(state, last) and torch.equal(h2, h)


def test_recurrence_updates_states_of_short_chains_in_place():
    """Chains of a few tiles: the last tile may be done before the others have read where the
    chain starts.  The C entry points update h0 and d_h_final in place."""
    g, C = _gen(10), 200
    lengths = [300, 700, 1100, 0, 1900, 257] * 20
    cu, T, N = _cu(lengths), sum(lengths), len(lengths)
    x, gate, h0 = _randn((T, C), g), -torch.rand((T, C), generator=g, device="cuda") * 1e-3, _randn((N, C), g)
    h, last = kda.linear_recurrence(x, gate, h0, cu)
    dx, dg, d_h0 = kda.linear_recurrence_backward(x, x, gate, h, h0, cu, last)
    desc = kda._layer.RecurrenceDesc(0, 0, N, T, C, 0, 0)
    ws = torch.empty(kda.lib().kda_recurrence_workspace_size(desc, 1), dtype=torch.uint8, device="cuda")
    for _ in range(10):
        state = h0.clone()
        h2, same = kda.linear_recurrence(x, gate, state, cu, h_final=state)
        assert torch.equal(state, last) and torch.equal(h2, h)
        dx2, dg2 = torch.empty_like(x), torch.empty_like(gate)
        assert kda.lib().kda_recurrence_backward(
            desc, x.data_ptr(), None, gate.data_ptr(), h.data_ptr(), h0.data_ptr(), cu.data_ptr(),
            state.data_ptr(), dx2.data_ptr(), dg2.data_ptr(), state.data_ptr(), ws.data_ptr(),
            ws.numel(), None, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(state, d_h0) and torch.equal(dx2, dx) and torch.equal(dg2, dg)


def test_recurrence_of_no_tokens():
    for write in ("add", "mix"):
        x, g = torch.empty((0, 6), device="cuda"), torch.empty((0, 6), device="cuda")
        h0 = torch.randn((3, 6), device="cuda")
        h, last = kda.linear_recurrence(x, g, h0, _cu([0, 0, 0]), write=write)
        assert h.shape == (0, 6) and torch.equal(last, h0)
        dx, dg, d_h0 = kda.linear_recurrence_backward(x, x, g, h, h0, _cu([0, 0, 0]), last, write=write)
        assert dx.shape == dg.shape == (0, 6) and torch.equal(d_h0, last)
        assert bool((kda.linear_recurrence(x, g)[1] == 0).all())
        state = torch.empty((0, 6), device="cuda")
        assert kda.linear_recurrence_step(x, g, state, write=write)[0].shape == (0, 6)


def test_recurrence_captured_and_on_another_stream():
    g, C, T = _gen(9), 192, 6000
    cu = _cu([2500, 0, 3500])
    x, gate, h0 = _randn((T, C), g, torch.bfloat16), _gates(T, C, g), _randn((3, C), g)
    d_h = _randn((T, C), g, torch.bfloat16)

    def both():
        h, last = kda.linear_recurrence(x, gate, h0, cu, write="mix")
        return (h, last) + kda.linear_recurrence_backward(d_h, x, gate, h, h0, cu, last, write="mix")
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, last = kda.linear_recurrence(x, gate, h0, cu, write="mix", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want[0]) and torch.equal(last, want[1])
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = both()
    for seed in (1, 2):
        x.copy_(_randn((T, C), _gen(seed), torch.bfloat16))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


# ------------------------------------------------------ gated feed-forward block
#
# A projection a = sum x w: the tensor core adds steps of 16 terms with truncation, 2^-23 of
# the running sum each; fp32 operands as three BF16 terms leave 2^-22 of a term, and their
# accumulators of 32 steps are added up with a rounding each:
#     |a - a64| <= (D / 16 + 40) 2^-23 sum |x w|.
# The activation: exp and the reciprocal are within 2^-21, the exponent's rounding adds
# |a| 2^-23, 1 - p is off by 2^-24 of 1; gelu's error function and its density (argument
# a^2 / 2) the same with a^2.  Slopes: |f'| < 1.2, |f''| < 0.8.

def _act64(a, act):
    if act == "gelu":
        cdf = 0.5 * torch.erfc(a * -math.sqrt(0.5))
        return a * cdf, cdf + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    p, q = torch.sigmoid(a), torch.sigmoid(-a)
    return (p, p * q) if act == "sigmoid" else (a * p, p * (1 + a * q))


def _ffn64(x, w, act, d_h=None, kind="f32"):
    """(h, bound) or, with d_h, (dx, bound, dw, bound)."""
    x, w, rnd = x.double(), w.double(), ROUND[kind]
    D, F = x.shape[1], w.shape[1]
    a, b = x @ w[0].T, x @ w[1].T
    acc = (D / 16 + 40) * 2 * U
    ea, eb = acc * (x.abs() @ w[0].abs().T), acc * (x.abs() @ w[1].abs().T)
    f, df = _act64(a, act)
    fuzz = 2.0 ** -20 + (a.abs() + a * a) * 2 * U
    ef = 1.2 * ea + fuzz * torch.maximum(f.abs(), torch.ones_like(f) * 2.0 ** -4)
    if d_h is None:
        ref = f * b
        return ref, b.abs() * ef + f.abs() * eb + ef * eb + (rnd + 2 * U) * ref.abs() + 1e-30
    d = d_h.double()
    da, db = d * b * df, d * f
    eda = d.abs() * (b.abs() * (0.8 * ea + fuzz) + df.abs() * eb + ea * eb) + (rnd + 4 * U) * da.abs()
    edb = d.abs() * ef + (rnd + 4 * U) * db.abs()
    dx = da @ w[0] + db @ w[1]
    sx = da.abs() @ w[0].abs() + db.abs() @ w[1].abs()
    ex = eda @ w[0].abs() + edb @ w[1].abs() + (2 * F / 16 + 40) * 2 * U * sx + (rnd + U) * dx.abs()
    dw = torch.stack([da.T @ x, db.T @ x])
    sw = torch.stack([da.abs().T @ x.abs(), db.abs().T @ x.abs()])
    ew = torch.stack([eda.T @ x.abs(), edb.T @ x.abs()]) + \
        (len(x) / 16 + 40) * 2 * U * sw + (rnd + U) * dw.abs()
    return dx, ex + 1e-30, dw, ew + 1e-30


def _norm_error(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


FFN = [  # T, D, F
    (1, 1, 1), (1, 64, 64), (2, 7, 31), (3, 100, 33), (7, 515, 200), (8, 128, 1003), (9, 129, 65),
    (16, 1000, 300), (31, 72, 257), (65, 64, 8), (128, 256, 640), (129, 520, 96), (256, 264, 1100),
    (300, 90, 513), (700, 448, 2050), (1030, 100, 100),
]


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,F", FFN)
def test_gated_ffn(T, D, F, kind, act):
    g, dt = _gen(T + D + F), DT[kind]
    x, w, d_h = _randn((T, D), g, dt), _randn((2, F, D), g, dt, 1.5 / math.sqrt(D)), _randn((T, F), g, dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    room = torch.full((T + 3, F), 7.0, device="cuda", dtype=dt)
    h = kda.gated_ffn(x, w, act=act, h=room[:T], dev_status=status)
    assert bool((room[T:] == 7).all())
    ref, bound = _ffn64(x, w, act, kind=kind)
    _within(h, ref, bound, "h")
    dx, dw = kda.gated_ffn_backward(d_h, x, w, act=act, dev_status=status)
    rx, bx, rw, bw = _ffn64(x, w, act, d_h, kind)
    _within(dx, rx, bx, "dx")
    _within(dw, rw, bw, "d_weight")
    assert int(status) == 0
    if T * F > 1000:
        # errors at random: the outputs' rounding and, in the gradients, the adjoints' too,
        # each 2^-9 of a value in the mean at most; fp32 a few units of 2^-24
        most = {"bf16": 2.0 ** -8, "f32": 2.0 ** -19}[kind]
        assert max(_norm_error(h, ref), _norm_error(dx, rx), _norm_error(dw, rw)) < most
    only_x = kda.gated_ffn_backward(d_h, x, w, act=act, want_d_weight=False)
    only_w = kda.gated_ffn_backward(d_h, x, w, act=act, want_dx=False)
    assert torch.equal(only_x[0], dx) and only_x[1] is None
    assert torch.equal(only_w[1], dw) and only_w[0] is None


def test_gated_ffn_gradient_against_differences():
    """Central differences of the library's own fp32 forward with steps of 2^-6: the third
    derivative adds about 2^-13, the forward's errors (2^-20 of a sum of about 30) 2^-10."""
    g = _gen(4)
    T, D, F = 5, 12, 9
    x, w, d_h = _randn((T, D), g), _randn((2, F, D), g, std=0.3), _randn((T, F), g)
    for act in ("silu", "gelu", "sigmoid"):
        dx, dw = kda.gated_ffn_backward(d_h, x, w, act=act)
        for src, grad, other in ((x, dx, lambda m: (m, w)), (w, dw, lambda m: (x, m))):
            for i in range(0, src.numel(), 7):
                value = []
                for sign in (1, -1):
                    m = src.clone()
                    m.view(-1)[i] += sign * 2.0 ** -6
                    value.append(float((kda.gated_ffn(*other(m), act=act).double() * d_h).sum()))
                slope = (value[0] - value[1]) * 2.0 ** 5
                assert abs(slope - float(grad.view(-1)[i])) < 4e-3


def test_gated_ffn_of_no_tokens_and_odd_outputs():
    w = torch.randn(2, 24, 16, device="cuda").bfloat16()
    x = torch.randn(40, 16, device="cuda").bfloat16()
    assert kda.gated_ffn(x[:0], w).shape == (0, 24)
    dx, dw = kda.gated_ffn_backward(x.new_empty(0, 24), x[:0], w)
    assert dx.shape == (0, 16) and bool((dw == 0).all())
    room = torch.zeros(40 * 24 + 8, device="cuda", dtype=torch.bfloat16)
    for by in (0, 1, 4):  # an output that starts anywhere
        h = kda.gated_ffn(x, w, h=room[by:by + 960].view(40, 24))
        assert torch.equal(h, kda.gated_ffn(x, w))
        d = room[by:by + 960].view(40, 24)
        assert all(torch.equal(p, q) for p, q in zip(kda.gated_ffn_backward(d, x, w),
                                                     kda.gated_ffn_backward(d.clone(), x, w)))


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_gated_ffn_rows_stay_apart(T):
    """NaN and infinity in a token's x or d_h reach no other token's h or dx."""
    g = _gen(T)
    x, w, d_h = (_randn(s, g, torch.bfloat16) for s in ((T, 64), (2, 96, 64), (T, 96)))
    h, dx = kda.gated_ffn(x, w), kda.gated_ffn_backward(d_h, x, w)[0]
    bad = T // 2
    x2, d2 = x.clone(), d_h.clone()
    x2[bad, 3], d2[bad, 5] = math.nan, math.inf
    h2, dx2 = kda.gated_ffn(x2, w), kda.gated_ffn_backward(d2, x2, w)[0]
    keep = torch.arange(T, device="cuda") != bad
    assert torch.equal(h2[keep], h[keep]) and torch.equal(dx2[keep], dx[keep])
    assert bool(torch.isnan(h2[bad]).all()) and bool(torch.isnan(dx2[bad]).all())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_gated_ffn_in_pieces(kind):
    """More tokens than 1 GiB of adjoints holds: dx adds up over pieces of the channels."""
    g, dt = _gen(6), DT[kind]
    T, D, F = 66000 if kind == "bf16" else 23000, 72, 8200
    x, w = _randn((T, D), g, dt), _randn((2, F, D), g, dt, 0.12)
    d_h = _randn((T, F), g, dt, 0.1)
    dx, dw = kda.gated_ffn_backward(d_h, x, w)
    most = {"bf16": 2.0 ** -8, "f32": 2.0 ** -19}[kind]
    x6, w6, sum_w = x.double(), w.double(), 0
    for i in range(0, T, 8192):
        at = slice(i, i + 8192)
        a, b = x6[at] @ w6[0].T, x6[at] @ w6[1].T
        f, df = _act64(a, "silu")
        da, db = d_h[at].double() * b * df, d_h[at].double() * f
        assert _norm_error(dx[at], da @ w6[0] + db @ w6[1]) < most
        sum_w = sum_w + torch.stack([da.T @ x6[at], db.T @ x6[at]])
    assert _norm_error(dw, sum_w) < most


def test_gated_ffn_past_32_bits():
    """More elements of h than 32 bits count."""
    g = _gen(7)
    T, D, F = 2 ** 20 + 5, 64, 4104
    x, w = _randn((T, D), g, torch.bfloat16), _randn((2, F, D), g, torch.bfloat16, 0.15)
    h = kda.gated_ffn(x, w)
    for at in (slice(0, 64), slice(T - 64, T)):
        ref, bound = _ffn64(x[at], w, "silu", kind="bf16")
        _within(h[at], ref, bound, "h")
    h[:-64] = 0  # as d_h: only the last tokens have a part in d_weight
    dx, dw = kda.gated_ffn_backward(h, x, w)
    at = slice(T - 64, T)
    rx, bx, rw, bw = _ffn64(x[at], w, "silu", h[at], "bf16")
    _within(dx[at], rx, bx, "dx")
    # the accumulators' truncation over the other tokens adds nothing to zeros
    _within(dw, rw, bw, "d_weight")
    assert bool((dx[:1000] == 0).all())


def test_gated_ffn_captured_and_on_another_stream():
    g, T, D, F = _gen(9), 200, 136, 300
    x, w, d_h = (_randn(s, g, torch.bfloat16) for s in ((T, D), (2, F, D), (T, F)))

    def both():
        return (kda.gated_ffn(x, w), kda.gated_ffn(x[:3], w)) + kda.gated_ffn_backward(d_h, x, w)
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = kda.gated_ffn(x, w, stream=side)
    dx, dw = kda.gated_ffn_backward(d_h, x, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip((h, dx, dw), (want[0],) + want[2:]))
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = both()
    for seed in (1, 2):
        x.copy_(_randn((T, D), _gen(seed), torch.bfloat16))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


# ------------------------------------------------------------------------ dropout

def _mask(rows, D, p, rng, site):
    """The mask and its factor from the oracle's generator, as 64-bit tensors."""
    seed, offset = rng.tolist()
    rows = range(rows) if isinstance(rows, int) else rows
    mask, factor = keep_mask(rows, D, p, seed, offset, site)
    return torch.from_numpy(mask).cuda(), factor


def _rng(seed, offset=None):
    return torch.tensor([seed, 3 * seed + 1 if offset is None else offset], device="cuda")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 5), (3, 64), (7, 1001), (33, 250), (257, 4096), (5, 20003)])
def test_dropout(T, D, kind):
    g, dt = _gen(T * D), DT[kind]
    for p, rng, site in ((0.1, _rng(D), 0), (0.5, _rng(-T, 2 ** 62 + 5), 65535), (0.0, _rng(1), 3)):
        x = _randn((T, D), g, dt)
        mask, factor = _mask(T, D, p, rng, site)
        x[~mask] = math.nan  # a dropped element is 0 whatever it was
        room = torch.full((T * D + 9,), 7.0, device="cuda", dtype=dt)
        for by in (0, 1):  # an aligned output and one that is not
            out = kda.dropout(x, p, rng, site=site, out=room[by:by + T * D].view(T, D))
            ref = torch.where(mask, x.double() * factor, 0.0)
            # the factor is rounded to fp32, the product too
            _within(out, ref, (ROUND[kind] + 2 * U) * ref.abs(), "dropout")
            assert bool((room[by + T * D:] == 7).all()) and (by == 0 or float(room[0]) == float(out0))
            out0 = out.view(-1)[0].clone()
        if p == 0:
            assert torch.equal(out, x)
        same = kda.dropout(x, p, rng, site=site, out=x)
        assert same is x and torch.equal(x, out)


def test_dropout_of_almost_everything_and_of_no_rows():
    x = torch.ones((500, 1000), device="cuda")
    assert bool((kda.dropout(x, 1 - 2.0 ** -32, _rng(4)) == 0).all())  # 2^-32 x 5e5 are kept
    assert kda.dropout(x[:0], 0.3, _rng(4)).shape == (0, 1000)


def test_dropout_masks_are_apart():
    """Another seed, offset or site is another mask, whose share of kept elements is as told
    (five deviations)."""
    x = torch.ones((1000, 1000), device="cuda")
    calls = [(_rng(1, 2), 0), (_rng(2, 2), 0), (_rng(1, 3), 0), (_rng(1, 2), 1),
             (_rng(1 + 2 ** 40, 2), 0), (_rng(1, 2 + 2 ** 40), 0)]
    masks = [kda.dropout(x, 0.25, r, site=s) != 0 for r, s in calls]
    for i, m in enumerate(masks):
        assert abs(float(m.double().mean()) - 0.75) < 5 * math.sqrt(0.25 * 0.75 / 1e6)
        for n in masks[:i]:  # both kept: 0.75^2
            assert abs(float((m & n).double().mean()) - 0.5625) < 5 * math.sqrt(0.5625 * 0.4375 / 1e6)


def test_dropout_past_32_bits():
    T, D = 70001, 65540
    x = torch.ones((T, D), device="cuda", dtype=torch.bfloat16)
    out = kda.dropout(x, 0.5, _rng(11), site=9)
    rows = [0, 1, 65535, 65536, 65537, T - 1]
    mask, _ = _mask(rows, D, 0.5, _rng(11), 9)
    assert torch.equal(out[rows], mask.bfloat16() * 2)


NORMS = [  # T, D, elements off the 16-byte boundary
    (1, 1, 0), (5, 64, 0), (3, 250, 0), (6, 1001, 0), (4, 7168, 0), (2, 16384, 0), (9, 100, 1),
    (3, 2000, 1), (10000, 512, 0), (40000, 125, 0), (90000, 33, 0), (5000, 2048, 0), (3000, 7168, 0),
    (1500, 5120, 0), (2600, 1001, 0),
]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,by", NORMS)
def test_residual_norm_with_dropout(T, D, by, kind):
    """Rows in pieces, shifted pieces, pairs and elements, streamed and not.  Bounds: an output's
    rounding, and 2^-18 of the terms behind it for fp32 sums over a row and rsqrt."""
    g, dt, p, scale, site, eps = _gen(T + D), DT[kind], 0.3, 0.5, 7, 1e-5
    rng = _rng(T + D)
    mask, factor = _mask(T, D, p, rng, site)

    def array(std=1.0):
        t = torch.empty(T * D + by, device="cuda", dtype=dt)[by:].view(T, D)
        return t.copy_(_randn((T, D), g, dt, std))
    h, y, d_out, d_h = array(2.0), array(), array(), array()
    y[~mask] = math.nan
    w = 1 + 0.1 * _randn((D,), g)
    drop = dict(dropout=p, rng=rng, site=site, scale=scale, eps=eps)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h_out, out = kda.residual_norm(h, y, w, dev_status=status, h_out=array(), out=array(), **drop)
    add = torch.where(mask, y.double() * (scale * factor), 0.0)
    ref = h.double() + add
    terms = h.double().abs() + add.abs()
    _within(h_out, ref, ROUND[kind] * ref.abs() + 2.0 ** -21 * terms, "h_out")
    r = (ref.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    ref = ref * r * w.double()
    _within(out, ref, ROUND[kind] * ref.abs() + 2.0 ** -18 * terms * r * w.abs(), "out")

    dh, dy, dw = kda.residual_norm_backward(d_out, h_out, w, d_h, dev_status=status, **drop)
    v = h_out.double()
    r = (v.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    n, e = v * r, d_out.double() * w.double()
    ref = d_h.double() + r * (e - n * (e * n).mean(-1, keepdim=True))
    terms = d_h.double().abs() + r * (e.abs() + n.abs() * (e * n).abs().mean(-1, keepdim=True))
    _within(dh, ref, ROUND[kind] * ref.abs() + 2.0 ** -18 * terms, "dh")
    ref = torch.where(mask, ref * (scale * factor), 0.0)
    _within(dy, ref, ROUND[kind] * ref.abs() + 2.0 ** -18 * terms * scale * factor * mask, "dy")
    ref, terms = (d_out.double() * n).sum(0), (d_out.double() * n).abs().sum(0)
    _within(dw, ref, 2.0 ** -18 * terms, "d_weight")
    assert int(status) == 0
    # without dy the mask has no part
    plain = kda.residual_norm_backward(d_out, h_out, w, d_h, want_dy=False, **drop)
    assert torch.equal(plain[0], dh) and plain[1] is None
    # the same norm without dropout: p = 0 through the calls' C form
    zero = kda._lm.DropoutDesc(rng.data_ptr(), 0.0, 0)
    desc = kda._lm.NormDesc(T, 0, 0, 1, D, kda._lm._ACT[dt], 0, eps)
    y = array()
    a, b = kda.residual_norm(h, y, w, scale=scale, eps=eps)
    a2, b2 = torch.empty_like(a), torch.empty_like(b)
    assert kda.lib().kda_residual_norm_dropout_forward(
        desc, zero, h.data_ptr(), y.data_ptr(), w.data_ptr(), scale, a2.data_ptr(), b2.data_ptr(),
        None, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(a, a2) and torch.equal(b, b2)


def test_dropout_captured_with_a_generator_that_moves_on():
    """A graph reads seed and offset when it runs: the captured step moves the offset on."""
    g, T, D = _gen(12), 300, 136
    x, y = _randn((T, D), g, torch.bfloat16), _randn((T, D), g, torch.bfloat16)
    rng = _rng(77, 0)

    def step():
        d = kda.dropout(x, 0.2, rng, site=1)
        h, n = kda.residual_norm(x, y, None, dropout=0.4, rng=rng, site=2)
        return (d, h, n) + kda.residual_norm_backward(y, h, None, x, dropout=0.4, rng=rng, site=2)[:2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    d = kda.dropout(x, 0.2, rng, site=1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(d, step()[0])
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
            rng[1] += 1
    rng[1] = 0
    seen = []
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        seen.append(out[0].clone())
        now = rng.clone()
        rng[1] = i
        want = step()
        rng.copy_(now)
        assert int(now[1]) == i + 1 and all(torch.equal(p, q) for p, q in zip(out, want))
    assert not torch.equal(seen[0], seen[1])


# --------------------------------------------------------- differentiable forms

def test_differentiable_forms_of_a_layer():
    """A layer as it is trained, residual norm with dropout -> recurrence -> residual norm with
    dropout -> feed-forward block -> norm, against the same layer in 64 bits (masks from the
    oracle).  fp32: a chain of operators each within about 2^-20 of its outputs' size."""
    g, T, D, F = _gen(15), 61, 40, 56
    cu = _cu([20, 0, 41])
    rng, p = _rng(5), 0.25
    leaf = lambda *shape, std=1.0: _randn(shape, g, std=std).requires_grad_()  # noqa: E731
    h, y, gate_x = leaf(T, D), leaf(T, D), leaf(T, D)
    w1, w2, ffn, down = leaf(D), leaf(D), leaf(2, F, D, std=0.2), leaf(D, F, std=0.2)
    h0 = leaf(3, D)
    leaves = [h, y, gate_x, w1, w2, ffn, down, h0]
    d_end, d_last = _randn((T, D), g), _randn((3, D), g)

    keep = rng.clone()
    a, n = autograd.kda_residual_norm(h, y, w1, scale=0.5, dropout=p, rng=rng, site=1)
    s, last = autograd.kda_linear_recurrence(n, -torch.nn.functional.softplus(gate_x), h0, cu, write="mix")
    b, n = autograd.kda_residual_norm(a, s, w2, dropout=p, rng=rng, site=2)
    f = autograd.kda_gated_ffn(n, ffn, act="gelu")
    end = b + autograd.kda_dropout(f @ down.T, p, rng, site=3)
    rng += 1  # the program moves on; the backward pass needs what was
    ((end * d_end).sum() + (last * d_last).sum()).backward()
    got = [t.grad.clone() for t in leaves]

    ref = [t.detach().double().requires_grad_() for t in leaves]
    h, y, gate_x, w1, w2, ffn, down, h0 = ref
    m = [torch.where(mask, factor, 0.0) for mask, factor in (_mask(T, D, p, keep, s) for s in (1, 2, 3))]
    norm = lambda v, w: v * (v.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * w  # noqa: E731
    a = h + 0.5 * m[0] * y
    n, decay = norm(a, w1), -torch.nn.functional.softplus(gate_x)
    rows, ends = [], []
    for i in range(3):
        state = h0[i]
        for t in range(int(cu[i]), int(cu[i + 1])):
            state = torch.exp(decay[t]) * state - torch.expm1(decay[t]) * n[t]
            rows.append(state)
        ends.append(state)
    b = a + m[1] * torch.stack(rows)
    n = norm(b, w2)
    f = torch.nn.functional.gelu(n @ ffn[0].T) * (n @ ffn[1].T)
    want = b + m[2] * (f @ down.T)
    ((want * d_end).sum() + (torch.stack(ends) * d_last).sum()).backward()
    assert _norm_error(end.detach(), want.detach()) < 2.0 ** -17
    for name, x, r in zip("h y gate w1 w2 ffn down h0".split(), got, ref):
        assert _norm_error(x, r.grad) < 2.0 ** -16, (name, _norm_error(x, r.grad))


def test_second_derivatives_are_refused():
    x = torch.ones((4, 8), device="cuda", requires_grad=True)
    w = torch.ones((2, 8, 8), device="cuda")
    for y in (autograd.kda_gated_ffn(x, w), autograd.kda_dropout(x, 0.5, _rng(1)),
              autograd.kda_linear_recurrence(x, -torch.ones_like(x))[0]):
        d, = torch.autograd.grad(y.pow(2).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            d.sum().backward()


def test_wrong_tensors_are_refused():
    """The binding's checks beside a GPU: types, shapes, layouts, places."""
    x, g = torch.zeros((6, 8), device="cuda"), torch.zeros((6, 8), device="cuda")
    w, rng = torch.zeros((2, 5, 8), device="cuda"), _rng(1)
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    bad = [
        lambda: kda.linear_recurrence(x.double(), g), lambda: kda.linear_recurrence(x, g.bfloat16()),
        lambda: kda.linear_recurrence(x, g[:5]), lambda: kda.linear_recurrence(x.T, g.T),
        lambda: kda.linear_recurrence(x, g, write="x"), lambda: kda.linear_recurrence(x, g, x),
        lambda: kda.linear_recurrence(x, g, None, cu.long()), lambda: kda.linear_recurrence(x, g, None, cu[:1]),
        lambda: kda.linear_recurrence(x, g, None, cu.cpu()), lambda: kda.linear_recurrence(x, g, h=x[:5]),
        lambda: kda.linear_recurrence(x[:1].expand(6, 8), g),
        lambda: kda.linear_recurrence(x, g, h_final=torch.zeros(2, 8, device="cuda")),
        lambda: kda.linear_recurrence(x, g, dev_status=cu.long()),
        lambda: kda.linear_recurrence_backward(x.bfloat16(), x, g, x),
        lambda: kda.linear_recurrence_backward(x, x, g, x[:5]),
        lambda: kda.linear_recurrence_backward(x, x, g, x, None, None, x),
        lambda: kda.linear_recurrence_step(x, g, x[:5]), lambda: kda.linear_recurrence_step(x, g, x.bfloat16()),
        lambda: kda.linear_recurrence_step(x, g, x, write="x"),
        lambda: kda.gated_ffn(x, w.bfloat16()), lambda: kda.gated_ffn(x, w[:1]),
        lambda: kda.gated_ffn(x, w[:, :, :7]), lambda: kda.gated_ffn(x.T, w), lambda: kda.gated_ffn(x, w, act="x"),
        lambda: kda.gated_ffn(x, w, h=x), lambda: kda.gated_ffn_backward(x, x, w),
        lambda: kda.dropout(x, 0.1, rng.int()), lambda: kda.dropout(x, 0.1, rng.cpu()),
        lambda: kda.dropout(x, 0.1, rng[:1]), lambda: kda.dropout(x.T, 0.1, rng),
        lambda: kda.residual_norm(x, None, dropout=0.1, rng=rng), lambda: kda.residual_norm(x, x, dropout=0.1, rng=cu),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        kda.residual_norm(x, x, dropout=0.1)
    for call in (lambda: kda.dropout(x, 1.0, rng), lambda: kda.dropout(x, 0.1, rng, site=1 << 16),
                 lambda: kda.dropout(x, -0.5, rng), lambda: kda.residual_norm(x, x, dropout=1.5, rng=rng)):
        with pytest.raises(kda.KDAError):
            call()


def test_example_runs_with_all_parts():
    """The example's model with the recurrence, the feed-forward block and dropout: every
    parameter gets a finite gradient, the same one for the same mask, another for another, and
    the steps run."""
    from examples.train_lm import Model, batch, train
    torch.manual_seed(3)
    model = Model(61, 128, 1, 2, full=True, dropout=0.25)
    ids, targets, cu = batch(61, (40, 1, 23), _gen(3))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = []
    for rng in (_rng(1, 5), _rng(1, 5), _rng(1, 6)):
        model.zero_grad()
        model(ids, targets, cu, status, rng).backward()
        rng += 1  # moved on after the backward pass has what it needs
        grads.append([p.grad.clone() for p in model.parameters()])
    names = [n for n, _ in model.named_parameters()]
    assert any("gate_up" in n for n in names) and any("xgz" in n for n in names)
    for n, a, b, c in zip(names, *grads):
        assert bool(torch.isfinite(a).all()) and bool((a != 0).any()), n
        assert torch.equal(a, b), n
        assert not torch.equal(a, c), n
    assert int(status) == 0
    assert len(train(steps=3, layers=2, full=True, dropout=0.1, log=lambda s: None)) == 3


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_the_generator_moves_on_before_the_residual_norms_gradient(p):
    """rng moves on between the passes, also while dropout is 0: the gradients are those of the
    mask that the forward pass had."""
    g = _gen(21)
    h, y = _randn((9, 40), g).requires_grad_(), _randn((9, 40), g).requires_grad_()
    grads = []
    for moves in (0, 1):
        rng = _rng(3)
        out = autograd.kda_residual_norm(h, y, None, scale=0.5, dropout=p, rng=rng, site=2)
        rng[1] += moves
        grads.append(torch.autograd.grad(sum(t.square().sum() for t in out), (h, y)))
    assert all(torch.equal(a, b) and bool((a != 0).any()) for a, b in zip(*grads))


@pytest.mark.parametrize("C", [64, 63])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("backward", [False, True], ids=["forward", "gradient"])
def test_recurrence_gives_up_together(backward, act, C):
    """Blocks without time to wait for one another: some give up in the middle of a long chain,
    the status says so, nothing outside the outputs is written, and the next call is right."""
    T, dt, g = 1 << 20, DT[act], _gen(C)
    x, gate = _randn((T, C), g, dt), _gates(T, C, g)
    want = kda.linear_recurrence(x, gate, want_final_state=False)[0]
    grads = kda.linear_recurrence_backward(x, x, gate, want) if backward else None
    L, desc = kda.lib(), kda._layer.RecurrenceDesc(0, 0, 1, T, C, kda._lm._ACT[dt], 0)
    ws = torch.empty(L.kda_recurrence_workspace_size(desc, int(backward)) + 256, dtype=torch.uint8,
                     device="cuda").fill_(7)
    out = torch.full((T + 1, C), 7.0, device="cuda", dtype=dt)
    dg = torch.full((T + 1, C), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert L.kda_selftest_recurrence_timeout(
        desc, x.data_ptr(), gate.data_ptr(), want.data_ptr() if backward else None, out.data_ptr(),
        dg.data_ptr(), ws.data_ptr(), ws.numel() - 256, status.data_ptr(),
        torch.cuda.current_stream().cuda_stream) == 0
    assert int(status) == 5
    assert bool((out[T] == 7).all()) and bool((dg[T] == 7).all()) and bool((ws[-256:] == 7).all())
    # what a block did write before it gave up is right
    done = out[:T] == (grads[0] if backward else want)
    assert bool((done | (out[:T] == 7)).all())
    assert torch.equal(kda.linear_recurrence(x, gate, want_final_state=False)[0], want)
    if backward:
        again = kda.linear_recurrence_backward(x, x, gate, want)
        assert all(torch.equal(p, q) for p, q in zip(again, grads))


@pytest.mark.parametrize("write", ["add", "mix"])
@pytest.mark.parametrize("C", [128, 63])
def test_recurrence_of_states_that_come_from_far(C, write):
    """Slow gates over several groups of tiles, each state the end of a long look back (copies of
    whole rows and of single channels), and every entry of it: zeros but for the first token."""
    g = _gen(C)
    lengths = [5200, 0, 2300]
    cu, T = _cu(lengths), sum(lengths)
    x, gate, h0 = _randn((T, C), g), -torch.rand((T, C), generator=g, device="cuda") * 1e-3, _randn((3, C), g)
    d_h, d_final = _randn((T, C), g), _randn((3, C), g)
    for zeros in (False, True):
        if zeros:
            x, d_h = torch.zeros_like(x), torch.zeros_like(d_h)
        h, last = kda.linear_recurrence(x, gate, h0, cu, write=write)
        ref, err, final, final_err = _recurrence64(x, gate, h0, cu.tolist(), write)
        _within(h, ref, U * ref.abs() + 2 * err, "h")
        _within(last, final, final_err + U * final.abs(), "h_final")
        got = kda.linear_recurrence_backward(d_h, x, gate, h, h0, cu, d_final, write=write)
        want = _recurrence_grad64(d_h, x, gate, h, h0, cu.tolist(), d_final, write)
        for name, a, r, e in zip(("dx", "dg", "d_h0"), got, want[::2], want[1::2]):
            _within(a, r, U * r.abs() + 2 * e, name)


# Batches of up to 256 tokens have a kernel without a look back; 257 is the first with one.
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 200, 256, 257])
def test_recurrence_of_few_tokens_strided_and_odd_bases(T, act):
    g, dt, C = _gen(T), DT[act], 70
    wide, wide_g = _randn((T, 3, C), g, dt), _gates(T, 2 * C, g).view(T, 2, C)
    h0, d_final = _randn((1, C), g), _randn((1, C), g)
    for x, gate in ((wide[:, 1], wide_g[:, 1]), (wide.view(T, 3 * C)[:, 1:C + 1], wide_g[:, 0]),
                    (wide[:, 2], wide_g.view(T, 2 * C)[:, 3:C + 3])):
        for write in ("add", "mix"):
            h, last = kda.linear_recurrence(x, gate, h0, write=write)
            ref, err, final, final_err = _recurrence64(x, gate, h0, [0, T], write)
            _within(h, ref, ROUND[act] * ref.abs() * (1 + 2 * U) + 2 * err, "h")
            _within(last, final, final_err + U * final.abs(), "h_final")
            got = kda.linear_recurrence_backward(h, x, gate, h, h0, None, d_final, write=write)
            want = _recurrence_grad64(h, x, gate, h, h0, [0, T], d_final, write)
            for name, a, r, e in zip(("dx", "dg", "d_h0"), got, want[::2], want[1::2]):
                _within(a, r, (ROUND[act] if name == "dx" else U) * r.abs() + 2 * e, name)
            plain = kda.linear_recurrence(x.contiguous(), gate.contiguous(), h0, write=write)
            assert torch.equal(h, plain[0]) and torch.equal(last, plain[1])


@pytest.mark.parametrize("T", [3, 200, 256, 257])
def test_bad_sequences_of_few_tokens_are_reported(T):
    """A status, and nothing written outside the outputs."""
    x, g = torch.zeros((T, 70), device="cuda"), torch.zeros((T, 70), device="cuda")
    room = torch.full((T + 2, 70), 7.0, device="cuda")
    for cu in ([0, T - 1], [1, T], [0, T - 1, 1, T], [0, -3, T], [0, T + 7, T], [0, 2 ** 30, T],
               [0, -2 ** 31, T], [0, 2 ** 31 - 1, T]):
        for backward in (False, True):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            seqs = torch.tensor(cu, dtype=torch.int32, device="cuda")
            if backward:
                kda.linear_recurrence_backward(x, x, g, x, None, seqs, dev_status=status)
            else:
                kda.linear_recurrence(x, g, None, seqs, h=room[1:T + 1], dev_status=status)
            assert int(status) == 1, (cu, backward)
    assert bool((room[0] == 7).all()) and bool((room[-1] == 7).all())


@pytest.mark.parametrize("C", [64, 7])
@pytest.mark.parametrize("lengths", [[1], [120, 0, 80], [0, 256], [0, 0], [100, 157]],
                         ids=lambda v: "-".join(map(str, v)))
def test_recurrence_updates_states_of_few_tokens_in_place(lengths, C):
    """h_final may be h0, and (through the C entry point) d_h0 the d_h_final that was given."""
    g, T, N = _gen(sum(lengths)), sum(lengths), len(lengths)
    cu, x, gate, h0 = _cu(lengths), _randn((T, C), g), _gates(T, C, g), _randn((N, C), g)
    h, last = kda.linear_recurrence(x, gate, h0, cu)
    dx, dg, d_h0 = kda.linear_recurrence_backward(x, x, gate, h, h0, cu, last)
    state = h0.clone()
    h2, same = kda.linear_recurrence(x, gate, state, cu, h_final=state)
    assert same is state and torch.equal(state, last) and torch.equal(h2, h)
    desc = kda._layer.RecurrenceDesc(0, 0, N, T, C, 0, 0)
    ws = torch.empty(kda.lib().kda_recurrence_workspace_size(desc, 1) + 16, dtype=torch.uint8, device="cuda")
    dx2, dg2 = torch.empty_like(x), torch.empty_like(gate)
    assert kda.lib().kda_recurrence_backward(
        desc, x.data_ptr(), None, gate.data_ptr(), h.data_ptr(), h0.data_ptr(), cu.data_ptr(),
        state.data_ptr(), dx2.data_ptr(), dg2.data_ptr(), state.data_ptr(), ws.data_ptr(),
        ws.numel(), None, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(state, d_h0) and torch.equal(dx2, dx) and torch.equal(dg2, dg)


@pytest.mark.parametrize("write", ["add", "mix"])
@pytest.mark.parametrize("C", [128, 63])
def test_recurrence_of_growing_states(C, write):
    """Positive gates whose factors' products over 2,048 tokens stay within fp32: states grow by
    e^60 and come back, over several groups of tiles."""
    g, T = _gen(C), 6000
    drift = 0.03 * torch.where(torch.arange(T, device="cuda") // 2000 % 2 == 0, 1.0, -1.0)
    gate = drift[:, None] + 0.02 * (torch.rand((T, C), generator=g, device="cuda") - 0.5)
    x, h0, d_h = _randn((T, C), g), _randn((1, C), g, std=1e-8), _randn((T, C), g)
    h, last = kda.linear_recurrence(x, gate, h0, write=write)
    ref, err, final, final_err = _recurrence64(x, gate, h0, [0, T], write)
    assert float(ref.abs().max()) > 1e20
    _within(h, ref, U * ref.abs() + 2 * err, "h")
    _within(last, final, final_err + U * final.abs(), "h_final")
    got = kda.linear_recurrence_backward(d_h, x, gate, h, h0, write=write)
    want = _recurrence_grad64(d_h, x, gate, h, h0, [0, T], None, write)
    for name, a, r, e in zip(("dx", "dg", "d_h0"), got, want[::2], want[1::2]):
        _within(a, r, U * r.abs() + 2 * e.abs(), name)  # (1 - e^g is negative here)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,F", [
    (150, 24, 1000), (300, 24, 5632), (600, 24, 5632), (130, 24, 10240), (900, 24, 10239), (100, 24, 10240),
    (129, 24, 4097), (400, 24, 2816)])
def test_gated_ffn_of_every_width_of_tile(T, D, F, kind):
    """Few rows take tiles of 64 to 256 columns, of pairs of CTAs or of single ones, by how their
    rounds over the SMs come out."""
    g, dt = _gen(T + F), DT[kind]
    x, w, d_h = _randn((T, D), g, dt), _randn((2, F, D), g, dt, 1.5 / math.sqrt(D)), _randn((T, F), g, dt)
    ref, bound = _ffn64(x, w, "silu", kind=kind)
    _within(kda.gated_ffn(x, w), ref, bound, "h")
    dx, dw = kda.gated_ffn_backward(d_h, x, w)
    rx, bx, rw, bw = _ffn64(x, w, "silu", d_h, kind)
    _within(dx, rx, bx, "dx")
    _within(dw, rw, bw, "d_weight")
