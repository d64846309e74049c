"""A recurrent layer's parts without a GPU: the C ABI refuses bad arguments on the host with
the documented status codes, sizes its workspaces, and the binding refuses bad tensors
before it calls anything."""
import math

import pytest
import torch

import kimi_delta_attention_18_gb300 as kda
from kimi_delta_attention_18_gb300._layer import FFNDesc, RecurrenceDesc
from kimi_delta_attention_18_gb300._lm import DropoutDesc, NormDesc
from oracle.philox import keep_mask, philox

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
A = 0x10000  # an address that is never touched


def _make(cls, base, kw):
    d = dict(base, **kw)
    return cls(*[d[f] for f, _ in cls._fields_])


def _rec(**kw):
    return _make(RecurrenceDesc, dict(x_stride=0, g_stride=0, num_seqs=2, tokens=8, channels=16,
                                      act_dtype=1, write=0), kw)


def _forward(desc, ptrs=None, ws=None, ws_len=0):
    p = dict(x=A, g=A, h0=A, cu=A, h=A, last=A, status=None)
    p.update(ptrs or {})
    return kda.lib().kda_recurrence_forward(desc, p["x"], p["g"], p["h0"], p["cu"], p["h"], p["last"],
                                            ws, ws_len, p["status"], None)


def _backward(desc, ptrs=None, ws=None, ws_len=0):
    p = dict(d_h=A, x=A, g=A, h=A, h0=A, cu=A, d_last=A, dx=A, dg=A, d_h0=A, status=None)
    p.update(ptrs or {})
    return kda.lib().kda_recurrence_backward(desc, p["d_h"], p["x"], p["g"], p["h"], p["h0"], p["cu"],
                                             p["d_last"], p["dx"], p["dg"], p["d_h0"], ws, ws_len,
                                             p["status"], None)


BAD_RECURRENCE = [
    (dict(num_seqs=0), INVALID), (dict(tokens=-1), INVALID), (dict(channels=0), INVALID),
    (dict(x_stride=15), INVALID), (dict(g_stride=-16), INVALID), (dict(act_dtype=2), UNSUPPORTED),
    (dict(write=2), UNSUPPORTED), (dict(write=-1), UNSUPPORTED),
    (dict(tokens=2 ** 30 + 1), UNSUPPORTED), (dict(channels=2 ** 20 + 1), UNSUPPORTED),
    (dict(num_seqs=2 ** 24 + 1), UNSUPPORTED), (dict(x_stride=2 ** 31), UNSUPPORTED),
    (dict(tokens=2 ** 30, channels=2 ** 20), UNSUPPORTED),
    (dict(num_seqs=2 ** 24, channels=2 ** 20), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_RECURRENCE, ids=str)
def test_recurrence_refuses_descriptors(kw, status):
    d = _rec(**kw)
    assert kda.lib().kda_recurrence_workspace_size(d, 0) == kda.lib().kda_recurrence_workspace_size(d, 1) == 0
    assert _forward(d) == status and _backward(d) == status
    assert kda.lib().kda_recurrence_step(d, A, A, A, A, A, None) == status


def test_recurrence_refuses_pointers():
    for name in ("x", "g", "h"):
        assert _forward(_rec(), {name: None}) == INVALID
    for name, off in (("x", 1), ("g", 2), ("h0", 2), ("cu", 2), ("h", 1), ("last", 2), ("status", 2)):
        assert _forward(_rec(), {name: A + off}) == INVALID
    assert _forward(_rec(act_dtype=0), {"x": A + 2}) == INVALID
    assert _forward(_rec(), {"cu": None}) == INVALID  # two sequences need it
    for name in ("d_h", "g", "h", "dx", "dg"):
        assert _backward(_rec(), {name: None}) == INVALID
    assert _backward(_rec(write=1), {"x": None}) == INVALID
    for name, off in (("d_h", 1), ("x", 1), ("g", 2), ("h", 1), ("h0", 2), ("d_last", 2), ("dx", 1),
                      ("dg", 2), ("d_h0", 2), ("cu", 2), ("status", 2)):
        assert _backward(_rec(), {name: A + off}) == INVALID
    step = kda.lib().kda_recurrence_step
    good = [A] * 5
    assert step(_rec(), *good, None) == INVALID  # eight tokens of two sequences
    for i in range(5):
        for bad in (None, A + 1):
            args = list(good)
            args[i] = bad
            assert step(_rec(tokens=2), *args, None) == INVALID


def test_recurrence_workspace():
    size = kda.lib().kda_recurrence_workspace_size
    for backward, tile in ((0, 128), (1, 64)):
        assert size(_rec(tokens=256), backward) == 0 and size(_rec(tokens=0), backward) == 0
        d = _rec(tokens=1025, channels=100)
        need = size(d, backward)
        # tiles (one more for each sequence) x 64 channels: maps and ends
        tiles = 1025 // tile + 2
        states = 2 * 100 * 4  # a copy of them, for calls that update them in place
        least = tiles * (16 + 128 * 12) + states
        assert least <= need <= least + 3 * 256
        call = _backward if backward else _forward
        assert call(d) == WORKSPACE
        assert call(d, ws=A, ws_len=need - 1) == WORKSPACE
        assert call(d, ws=A + 8, ws_len=need) == WORKSPACE
        # sequences of one token each: never more tiles than tokens
        d = _rec(tokens=1025, num_seqs=2 ** 20, channels=100)
        assert size(d, backward) < 1025 * (16 + 128 * 12) + 2 ** 20 * 400 + 4 * 256


def test_recurrence_binding_refuses_tensors():
    x, g = torch.zeros(4, 6), torch.zeros(4, 6)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_recurrence(x, g)
    with pytest.raises(ValueError, match="dimensions"):
        kda.linear_recurrence(x[0], g)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_recurrence_backward(x, x, g, x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_recurrence_step(x, g, g)


def _ffn(**kw):
    return _make(FFNDesc, dict(tokens=4, width=64, hidden=96, act_dtype=1, act=2), kw)


BAD_FFN = [
    (dict(tokens=-1), INVALID), (dict(width=0), INVALID), (dict(hidden=0), INVALID),
    (dict(act_dtype=2), UNSUPPORTED), (dict(act=0), UNSUPPORTED), (dict(act=4), UNSUPPORTED),
    (dict(tokens=2 ** 24 + 1), UNSUPPORTED), (dict(width=2 ** 17 + 1), UNSUPPORTED),
    (dict(hidden=2 ** 20 + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_FFN, ids=str)
def test_gated_ffn_refuses_descriptors(kw, status):
    L, d = kda.lib(), _ffn(**kw)
    assert L.kda_gated_ffn_workspace_size(d, 0) == 0 and L.kda_gated_ffn_workspace_size(d, 1) == 0
    assert L.kda_gated_ffn_forward(d, A, A, A, A, 2 ** 40, None, None) == status
    assert L.kda_gated_ffn_backward(d, A, A, A, A, A, A, 2 ** 40, None, None) == status


def test_gated_ffn_refuses_pointers():
    L = kda.lib()
    for i, bad in ((0, None), (0, A + 8), (1, None), (1, A + 8), (2, None), (2, A + 1), (3, A + 2)):
        p = [A, A, A, None]
        p[i] = bad
        assert L.kda_gated_ffn_forward(_ffn(), p[0], p[1], p[2], None, 0, p[3], None) == INVALID
    for i, bad in ((0, None), (0, A + 1), (1, None), (1, A + 2), (2, None), (2, A + 4), (3, A + 1),
                   (4, A + 1), (5, A + 2)):
        p = [A, A, A, A, A, None]
        p[i] = bad
        assert L.kda_gated_ffn_backward(_ffn(), *p[:5], A, 2 ** 40, p[5], None) == INVALID
    assert L.kda_gated_ffn_backward(_ffn(), A, A, A, None, None, None, 0, None, None) == OK  # nothing wanted
    assert L.kda_gated_ffn_forward(_ffn(tokens=0), None, None, None, None, 0, None, None) == OK


def test_gated_ffn_workspace():
    L = kda.lib()
    size = L.kda_gated_ffn_workspace_size
    assert size(_ffn(), 0) == 0  # BF16 rows of whole 16-byte pieces are read as they are
    assert size(_ffn(width=63, tokens=2), 0) == 0  # one or two tokens read any rows
    d = _ffn(width=63, tokens=16)
    assert size(d, 0) == 16 * 64 * 2 + 2 * 96 * 64 * 2
    assert L.kda_gated_ffn_forward(d, A, A, A, None, 0, None, None) == WORKSPACE
    assert L.kda_gated_ffn_forward(d, A, A, A, A, size(d, 0) - 1, None, None) == WORKSPACE
    assert L.kda_gated_ffn_forward(d, A, A, A, A + 8, 2 ** 40, None, None) == WORKSPACE
    assert size(_ffn(act_dtype=0, tokens=16), 0) == 3 * 16 * 64 * 2  # fp32: x's terms only
    assert size(_ffn(act_dtype=0, tokens=300), 0) == 3 * (300 + 2 * 96) * 64 * 2
    assert L.kda_gated_ffn_backward(_ffn(), A, A, A, A, A, A, size(_ffn(), 1) - 1, None, None) == WORKSPACE
    # the adjoints of a piece: 1 GiB at most, or 512 channels
    assert size(_ffn(tokens=2 ** 18, hidden=2 ** 16), 1) < 2 ** 30 + 2 ** 18 * 64 * 4 + 2 ** 12
    assert size(_ffn(tokens=2 ** 22, hidden=2 ** 16), 1) < 2 ** 22 * 512 * 4 + 2 ** 22 * 64 * 4 + 2 ** 12


def test_gated_ffn_binding_refuses_tensors():
    x, w = torch.zeros(4, 6), torch.zeros(2, 8, 6)
    with pytest.raises(ValueError, match="CUDA"):
        kda.gated_ffn(x, w)
    with pytest.raises(ValueError, match="dimensions"):
        kda.gated_ffn(x[0], w)
    with pytest.raises(ValueError, match="CUDA"):
        kda.gated_ffn_backward(x, x, w)


def test_the_generator_gives_its_published_values():
    """The known answers that its authors publish for ten rounds."""
    for counter, key, words in (
            ([0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
            ([0xffffffff] * 4, [0xffffffff] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
            ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
             "d16cfe09 94fdcceb 5001e420 24126ea1")):
        assert [int(w) for w in philox(counter, key)] == [int(w, 16) for w in words.split()]
    mask, factor = keep_mask(range(1000), 37, 0.3, 5, 6)
    assert abs(mask.mean() - 0.7) < 0.01 and abs(factor - 1 / 0.7) < 1e-9


def _drop(**kw):
    return _make(DropoutDesc, dict(rng=A, p=0.1, site=0), kw)


BAD_DROPOUT = [dict(rng=None), dict(rng=A + 4), dict(p=-0.1), dict(p=1.0), dict(p=math.nan),
               dict(p=1 - 2.0 ** -34), dict(site=-1), dict(site=65536)]


@pytest.mark.parametrize("kw", BAD_DROPOUT, ids=str)
def test_dropout_refuses_descriptors(kw):
    L, n = kda.lib(), NormDesc(4, 0, 0, 1, 64, 1, 0, 1e-6)
    assert L.kda_dropout(_drop(**kw), 4, 64, 1, A, A, None) == INVALID
    assert L.kda_residual_norm_dropout_forward(n, _drop(**kw), A, A, A, 1.0, A, A, None, None) == INVALID
    assert L.kda_residual_norm_dropout_backward(n, _drop(**kw), A, A, A, A, 1.0, A, A, A, A, 2 ** 30,
                                                None, None) == INVALID


def test_dropout_refuses_arguments():
    L, n, d = kda.lib(), NormDesc(4, 0, 0, 1, 64, 1, 0, 1e-6), _drop()
    assert L.kda_dropout(None, 4, 64, 1, A, A, None) == INVALID
    for args, status in (((-1, 64, 1, A, A), INVALID), ((4, 0, 1, A, A), INVALID),
                         ((4, 64, 2, A, A), UNSUPPORTED), ((2 ** 42, 64, 1, A, A), UNSUPPORTED),
                         ((4, 2 ** 30 + 1, 1, A, A), UNSUPPORTED), ((4, 64, 1, None, A), INVALID),
                         ((4, 64, 1, A, None), INVALID), ((4, 64, 1, A + 1, A), INVALID),
                         ((4, 64, 0, A, A + 2), INVALID), ((0, 64, 1, None, None), OK)):
        assert L.kda_dropout(d, *args, None) == status, args
    fwd, bwd = L.kda_residual_norm_dropout_forward, L.kda_residual_norm_dropout_backward
    assert fwd(n, None, A, A, A, 1.0, A, A, None, None) == INVALID
    assert fwd(n, d, A, None, A, 1.0, None, A, None, None) == INVALID  # nothing to drop
    assert fwd(n, d, A, A, A, math.inf, A, A, None, None) == INVALID
    assert fwd(n, _drop(p=0.999), A, A, A, 3e38, A, A, None, None) == INVALID
    assert bwd(n, None, A, A, A, A, 1.0, A, A, A, A, 2 ** 30, None, None) == INVALID
    assert bwd(n, d, A, A, A, A, 1.0, A, None, A, A, 2 ** 30, None, None) == INVALID
    assert bwd(n, d, A, A, A, A, 1.0, A, A, A, None, 0, None, None) == WORKSPACE
    bad = NormDesc(4, 0, 0, 2, 64, 1, 0, 1e-6)  # heads
    assert fwd(bad, d, A, A, A, 1.0, A, A, None, None) == INVALID


def test_dropout_binding_refuses_tensors():
    x, rng = torch.zeros(4, 6), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        kda.dropout(x, 0.1, rng)
    with pytest.raises(ValueError, match="dimensions"):
        kda.dropout(x[0], 0.1, rng)
    from kimi_delta_attention_18_gb300 import autograd
    with pytest.raises(ValueError, match="needs y"):
        autograd.kda_residual_norm(x, dropout=0.5, rng=rng)


def test_a_generator_may_move_on_before_the_gradient(monkeypatch):
    """A step's rng moves on between its forward and its backward pass, with dropout and while a
    schedule holds it at 0; the gradient with dropout has what rng was."""
    from kimi_delta_attention_18_gb300 import autograd
    seen = []

    def backward(d, h, w, dh, want_dy, rng, **k):
        seen.append(rng)
        return d * 1.0, d * 1.0, None
    monkeypatch.setattr(autograd._lm, "residual_norm", lambda h, y, w, **k: (h * 1.0, h * 1.0))
    monkeypatch.setattr(autograd._lm, "residual_norm_backward", backward)
    for p in (0.25, 0.0):
        x, rng = torch.ones((2, 4), requires_grad=True), torch.tensor([3, 5])
        h, out = autograd.kda_residual_norm(x, x * 2.0, None, dropout=p, rng=rng, site=1)
        rng[1] += 1
        (h + out).sum().backward()
        assert bool((x.grad != 0).all())
    assert seen[0].tolist() == [3, 5] and seen[1] is None


def test_gated_ffn_adjoints_stay_within_their_bound():
    """The adjoints of a piece take 1 GiB at most (or 512 channels) where the channels do not
    divide evenly, too.  They lie beside x and weight in terms (fp32) and dx's sums [T, D]."""
    size = kda.lib().kda_gated_ffn_workspace_size
    for tokens, hidden, f32 in ((400000, 8192, False), (81920, 28672, True), (66000, 8200, False),
                                (23000, 8200, True), (300001, 5000, False), (600000, 1000, False)):
        d = _ffn(tokens=tokens, hidden=hidden, act_dtype=0 if f32 else 1)
        planes, D = (3 if f32 else 1), 64
        terms = planes * 2 * D * (tokens + 2 * hidden) if f32 else 0
        adjoints = max(2 ** 30, 512 * 4 * tokens * planes)
        # dx and d_weight of so many tokens are one part each but for a few channels' sums
        assert size(d, 1) <= adjoints + terms + 4 * tokens * D + 2 ** 20, (tokens, hidden)


def test_recurrence_selftest_refuses_arguments():
    call, d = kda.lib().kda_selftest_recurrence_timeout, _rec(num_seqs=1)
    assert call(d, A, A, None, A, None, None, 0, None, None) == INVALID  # nowhere to tell
    assert call(None, A, A, None, A, None, None, 0, A, None) == INVALID
    assert call(_rec(), A, A, None, A, None, None, 0, A, None) == INVALID  # two sequences
    assert call(_rec(num_seqs=1, write=1), A, A, None, A, None, None, 0, A, None) == INVALID
    assert call(d, A, A, A, A, None, None, 0, A, None) == INVALID  # a gradient without dg
    assert call(_rec(num_seqs=1, tokens=1000), A, A, None, A, None, None, 0, A, None) == WORKSPACE


class _Elsewhere:
    """What the binding looks at of a contiguous tensor on a device that is not the current one."""
    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return 4

    def data_ptr(self):
        return A


def test_calls_run_on_their_tensors_device(monkeypatch):
    """Launches and workspace sizes belong to the tensors' device, whichever is current: a launch on
    another one would read addresses that it does not have."""
    from kimi_delta_attention_18_gb300 import _layer, _lm
    current, seen = [0], []

    class Device:
        def __init__(self, dev):
            self.index = dev.index

        def __enter__(self):
            self.was, current[0] = current[0], self.index

        def __exit__(self, *e):
            current[0] = self.was

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, current[0])) or 0
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(_lm, "_several", lambda: True, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    for module in (_lm, _layer):
        monkeypatch.setattr(module, "_lib", lambda: Lib())
        monkeypatch.setattr(module, "_workspace", lambda ws, need, dev: (_Elsewhere(16), 1 << 60))
        monkeypatch.setattr(module, "_out", lambda out, name, like: _Elsewhere(*like.shape, dtype=like.dtype))
    monkeypatch.setattr(_lm, "_stream", lambda dev: None)
    monkeypatch.setattr(_lm._k, "_need", lambda t, *a, **k: t)
    monkeypatch.setattr(torch, "empty", lambda shape, **k: _Elsewhere(*([shape] if isinstance(shape, int) else shape)))
    x, w, rng = _Elsewhere(4, 8), _Elsewhere(2, 6, 8), _Elsewhere(2, dtype=torch.int64)
    ids, vec, heads, h = _Elsewhere(4, dtype=torch.int32), _Elsewhere(4), _Elsewhere(4, 1, 8), _Elsewhere(4, 6)
    drop = dict(dropout=0.5, rng=rng)
    for call in (lambda: kda.gated_norm(heads, heads), lambda: kda.gated_norm_backward(heads, heads, heads),
                 lambda: kda.residual_norm(x, x), lambda: kda.residual_norm_backward(x, x),
                 lambda: kda.residual_norm(x, x, **drop), lambda: kda.residual_norm_backward(x, x, **drop),
                 lambda: kda.embedding(x, ids), lambda: kda.embedding_backward(x, ids, 9),
                 lambda: kda.linear_cross_entropy(x, x, ids),
                 lambda: kda.linear_cross_entropy_backward(x, x, ids, vec, vec),
                 lambda: kda.linear_recurrence(x, x), lambda: kda.linear_recurrence_backward(x, x, x, x),
                 lambda: kda.linear_recurrence_step(x, x, x), lambda: kda.gated_ffn(x, w),
                 lambda: kda.gated_ffn_backward(h, x, w), lambda: kda.dropout(x, 0.5, rng)):
        del seen[:]
        call()
        # (the recurrence's workspace is the same on every device)
        ran = [(name, on) for name, on in seen if name != "kda_recurrence_workspace_size"]
        assert ran and all(on == 1 for _, on in ran), ran
        assert current == [0]
