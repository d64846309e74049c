"""The operators around the mixer without a GPU: the C ABI refuses bad arguments on
the host with the documented status codes, sizes its workspaces, and the binding
refuses bad tensors before it calls anything."""
import ctypes
import math

import pytest
import torch

import kimi_delta_attention_18_gb300 as kda
from kimi_delta_attention_18_gb300 import autograd
from kimi_delta_attention_18_gb300._lm import CrossEntropyDesc, EmbedDesc, NormDesc

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
A = 0x10000  # an address that is never touched


def _make(cls, base, kw):
    d = dict(base, **kw)
    return cls(*[d[f] for f, _ in cls._fields_])


def _norm(**kw):
    return _make(NormDesc, dict(tokens=4, x_stride=0, gate_stride=0, heads=2, width=128, act_dtype=1,
                                gate=1, eps=1e-6), kw)


def _embed(**kw):
    return _make(EmbedDesc, dict(tokens=4, rows=10, width=64, act_dtype=1, id_dtype=0, scale=1.0), kw)


def _ce(**kw):
    return _make(CrossEntropyDesc, dict(ignore_index=-100, tokens=4, vocab=100, width=64, act_dtype=1,
                                        id_dtype=0, piece=0), kw)


def _gated(d, x=A, gate=A, w=A, out=A):
    return kda.lib().kda_gated_norm_forward(d, x, gate, w, out, None, None)


def _gated_bwd(d, d_out=A, x=A, gate=A, w=A, dx=A, dg=A, dw=A, ws=A, n=1 << 30):
    return kda.lib().kda_gated_norm_backward(d, d_out, x, gate, w, dx, dg, dw, ws, n, None, None)


def _resid(d, h=A, y=A, w=A, scale=1.0, h_out=A, out=A):
    return kda.lib().kda_residual_norm_forward(d, h, y, w, scale, h_out, out, None, None)


def _resid_bwd(d, d_out=A, dh_out=A, h=A, w=A, scale=1.0, dh=A, dy=A, dw=A, ws=A, n=1 << 30):
    return kda.lib().kda_residual_norm_backward(d, d_out, dh_out, h, w, scale, dh, dy, dw, ws, n, None,
                                                None)


def _ce_fwd(d, x=A, w=A, y=A, loss=A, lse=A, mean=A, ws=A, n=1 << 40):
    return kda.lib().kda_linear_ce_forward(d, x, w, y, loss, lse, mean, ws, n, None, None)


def _ce_bwd(d, x=A, w=A, y=A, lse=A, dl=A, dx=A, dw=A, ws=A, n=1 << 40):
    return kda.lib().kda_linear_ce_backward(d, x, w, y, lse, dl, dx, dw, ws, n, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID),
    (dict(heads=0), INVALID),
    (dict(width=0), INVALID),
    (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID),
    (dict(act_dtype=2), UNSUPPORTED),
    (dict(gate=3), UNSUPPORTED),
    (dict(width=16385), UNSUPPORTED),
    (dict(x_stride=255), INVALID),      # tokens would overlap
    (dict(gate_stride=100), INVALID),
    (dict(tokens=1 << 40), UNSUPPORTED),
])
def test_norms_reject_bad_descriptors(kw, code):
    d = _norm(**kw)
    assert _gated(d) == code and _gated_bwd(d) == code
    assert _resid(_norm(heads=1, gate=0, **kw) if "heads" not in kw and "gate" not in kw else d) == code
    assert kda.lib().kda_norm_backward_workspace_size(d) == 0


def test_norms_reject_bad_pointers():
    assert _gated(None) == INVALID
    assert _gated(_norm(), x=None) == INVALID and _gated(_norm(), out=None) == INVALID
    assert _gated(_norm(), gate=None) == INVALID            # a gate is wanted
    assert _gated(_norm(gate=0)) == INVALID                 # none is wanted
    assert _gated(_norm(), x=A + 1) == INVALID              # not aligned to an element
    assert _gated(_norm(act_dtype=0), out=A + 2) == INVALID
    assert _gated(_norm(), w=A + 2) == INVALID
    assert _gated_bwd(_norm(), dg=None) == INVALID and _gated_bwd(_norm(), d_out=None) == INVALID
    assert _gated_bwd(_norm(), dw=A + 1) == INVALID
    r = _norm(heads=1, gate=0)
    assert _resid(r, y=None) == INVALID and _resid(r, h_out=None) == INVALID
    assert _resid(r, scale=math.nan) == INVALID
    assert _resid(_norm()) == INVALID                       # heads, gate
    assert _resid(_norm(heads=1, gate=0, x_stride=128)) == INVALID
    assert _resid_bwd(r, h=None) == INVALID and _resid_bwd(r, dh=None) == INVALID


def test_norms_want_their_workspace_and_do_nothing_without_tokens():
    d = _norm(tokens=1000)
    need = kda.lib().kda_norm_backward_workspace_size(d)
    assert need > 0
    assert _gated_bwd(d, ws=None) == WORKSPACE and _gated_bwd(d, n=1) == WORKSPACE
    assert _gated_bwd(d, ws=A + 8) == WORKSPACE
    assert _resid_bwd(_norm(tokens=1000, heads=1, gate=0), n=1) == WORKSPACE
    assert _gated(_norm(tokens=0), x=None, gate=None, out=None) == OK
    assert _resid(_norm(tokens=0, heads=1, gate=0), h=None, out=None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID),
    (dict(rows=0), INVALID),
    (dict(width=0), INVALID),
    (dict(scale=math.inf), INVALID),
    (dict(act_dtype=7), UNSUPPORTED),
    (dict(id_dtype=2), UNSUPPORTED),
    (dict(width=65537), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED),
])
def test_embedding_rejects_bad_descriptors(kw, code):
    L, d = kda.lib(), _embed(**kw)
    assert L.kda_embedding_forward(d, A, A, A, None, None) == code
    assert L.kda_embedding_backward(d, A, A, A, A, 1 << 40, None, None) == code
    assert L.kda_embedding_backward_workspace_size(d) == 0


def test_embedding_rejects_bad_pointers():
    L = kda.lib()
    assert L.kda_embedding_forward(None, A, A, A, None, None) == INVALID
    assert L.kda_embedding_forward(_embed(), None, A, A, None, None) == INVALID
    assert L.kda_embedding_forward(_embed(), A, A + 2, A, None, None) == INVALID
    assert L.kda_embedding_forward(_embed(id_dtype=1), A, A + 4, A, None, None) == INVALID
    assert L.kda_embedding_forward(_embed(), A, A, A + 1, None, None) == INVALID
    assert L.kda_embedding_forward(_embed(tokens=0), None, None, None, None, None) == OK
    assert L.kda_embedding_backward(_embed(), A, A, None, A, 1 << 40, None, None) == INVALID
    assert L.kda_embedding_backward(_embed(), None, A, A, A, 1 << 40, None, None) == INVALID
    need = L.kda_embedding_backward_workspace_size(_embed())
    assert need > 0
    assert L.kda_embedding_backward(_embed(), A, A, A, A, need - 1, None, None) == WORKSPACE
    assert L.kda_embedding_backward(_embed(), A, A, A, None, need, None, None) == WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID),
    (dict(vocab=0), INVALID),
    (dict(width=0), INVALID),
    (dict(piece=-1), INVALID),
    (dict(act_dtype=2), UNSUPPORTED),
    (dict(id_dtype=-1), UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1), UNSUPPORTED),
    (dict(width=(1 << 17) + 1), UNSUPPORTED),
])
def test_cross_entropy_rejects_bad_descriptors(kw, code):
    d = _ce(**kw)
    assert _ce_fwd(d) == code and _ce_bwd(d) == code
    assert kda.lib().kda_linear_ce_workspace_size(d, 0) == 0


def test_cross_entropy_rejects_bad_pointers():
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(loss=None), dict(lse=None),
               dict(x=A + 8), dict(w=A + 2), dict(y=A + 2), dict(loss=A + 1), dict(mean=A + 2)):
        assert _ce_fwd(_ce(), **kw) == INVALID, kw
    for kw in (dict(x=None), dict(lse=None), dict(dl=None), dict(dx=A + 1), dict(dw=A + 1)):
        assert _ce_bwd(_ce(), **kw) == INVALID, kw
    assert _ce_fwd(_ce(), n=16) == WORKSPACE and _ce_bwd(_ce(), ws=None) == WORKSPACE
    assert _ce_bwd(_ce(), dx=None, dw=None) == OK  # nothing asked for
    assert _ce_fwd(None) == INVALID


def test_cross_entropy_workspace_follows_the_piece():
    """The backward's workspace holds dz for one piece of the vocabulary, not for all."""
    size = lambda **kw: kda.lib().kda_linear_ce_workspace_size(  # noqa: E731
        _ce(tokens=4096, vocab=100000, width=512, **kw), 1)
    one, two = size(piece=2048), size(piece=4096)
    assert two - one == 4096 * 2048 * 2
    assert size() < 4096 * 100000 * 2


def test_binding_refuses_tensors_off_the_gpu_and_of_other_shapes():
    x, w = torch.zeros(2, 3, 4), torch.ones(4)
    with pytest.raises(ValueError, match="CUDA"):
        kda.gated_norm(x, x, w)
    with pytest.raises(ValueError, match="dimensions"):
        kda.gated_norm(x[0], x[0], w)
    with pytest.raises(ValueError, match="CUDA"):
        kda.residual_norm(x[0])
    with pytest.raises(ValueError, match="CUDA"):
        kda.embedding(x[0], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_cross_entropy(x[0], x[0], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="dimensions"):
        kda.embedding(3, None)
    with pytest.raises(ValueError, match="reduction"):
        autograd.kda_linear_cross_entropy(x[0], x[0], None, reduction="max")


def test_descriptors_match_the_header():
    """The binding's structures have the header's fields, in its order and sizes."""
    assert ctypes.sizeof(NormDesc) == 48 and NormDesc.eps.offset == 40
    assert ctypes.sizeof(EmbedDesc) == 24 and EmbedDesc.scale.offset == 20
    assert ctypes.sizeof(CrossEntropyDesc) == 32 and CrossEntropyDesc.piece.offset == 28


def _stand_ins(monkeypatch):
    """The library's calls, each as a tensor of the right shape (no GPU here)."""
    def like(*ts):
        return tuple(None if t is None else t.detach() * 0 for t in ts)

    for name, fn in dict(
            gated_norm=lambda x, *a, **k: x * 1.0,
            gated_norm_backward=lambda d, x, gate, w, **k: like(x, gate, w),
            residual_norm=lambda h, y, w, **k: (h * 1.0, h * 1.0),
            residual_norm_backward=lambda d, h, w, dh, want_dy, **k: like(h, h if want_dy else None, w),
            embedding=lambda t, ids, **k: t[ids] * 1.0,
            embedding_backward=lambda d, ids, n, **k: d.new_zeros((n, d.shape[1])),
            linear_cross_entropy=lambda x, w, y, **k: (x.sum(1), x.sum(1), x.sum()),
            linear_cross_entropy_backward=lambda x, w, *a, **k: like(x, w)).items():
        monkeypatch.setattr(autograd._lm, name, fn)
    monkeypatch.setattr(autograd._k, "prefill_chunked", lambda q, k, v, *a, **kw: (v * 1.0, v.sum()))
    monkeypatch.setattr(autograd._k, "prefill_backward",
                        lambda q, k, v, g, beta, *a, **kw: like(q, k, v, g, beta) + (None,))


@pytest.mark.parametrize("op", [
    lambda x, w: autograd.kda_gated_norm(x[:, None], x[:, None] * 2.0, w),
    lambda x, w: autograd.kda_residual_norm(x, x * 2.0, w)[1],
    lambda x, w: autograd.kda_residual_norm(x, None, w)[1],
    lambda x, w: autograd.kda_embedding(x, torch.tensor([1, 0, 1])),
    lambda x, w: autograd.kda_linear_cross_entropy(x, x * 2.0, torch.tensor([1, 0])),
    lambda x, w: autograd.kda_linear_cross_entropy(x, x * 2.0, torch.tensor([1, 0]), reduction="sum"),
    lambda x, w: autograd.kda_prefill(x[:, None], x[:, None], x[:, None], x[:, None], x[:, :1])[0],
])
def test_second_derivatives_are_refused(monkeypatch, op):
    """A gradient of a gradient (a gradient penalty) raises: without the refusal its terms
    through the operation would be dropped and the rest returned as if it were all."""
    _stand_ins(monkeypatch)
    x = torch.randn(2, 4, requires_grad=True)
    y = op(x, torch.ones(4, requires_grad=True))
    grad, = torch.autograd.grad((y * y).sum() + (x * x * x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.pow(2).sum().backward()


class _OnDevice:
    """What the binding looks at of a contiguous tensor on the GPU."""
    is_cuda, device = True, torch.device("cpu")

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A


@pytest.mark.parametrize("n", [1 << 32, (1 << 32) + 3, (1 << 31) + 1])
def test_sizes_beyond_32_bits_are_refused(monkeypatch, n):
    """A length, width or vocabulary whose low 32 bits are a small number is not taken for
    that number (most of the output would stay unwritten)."""
    from kimi_delta_attention_18_gb300 import _lm
    monkeypatch.setattr(_lm, "_stream", lambda dev: None)
    monkeypatch.setattr(_lm, "_workspace", lambda *a: (_OnDevice(16), 1 << 60))
    t, ids = _OnDevice, lambda k: _OnDevice(k, dtype=torch.int32)  # noqa: E731
    vec = dict(loss=t(4), lse=t(4))
    for call in (lambda: kda.gated_norm(t(1, n, 8), t(1, n, 8), out=t(1, n, 8)),
                 lambda: kda.gated_norm(t(1, 1, n), t(1, 1, n), out=t(1, 1, n)),
                 lambda: kda.residual_norm(t(1, n), t(1, n), h_out=t(1, n), out=t(1, n)),
                 lambda: kda.embedding(t(7, 1), ids(n), out=t(n, 1)),
                 lambda: kda.embedding(t(n, 1), ids(7), out=t(7, 1)),
                 lambda: kda.embedding(t(7, n), ids(1), out=t(1, n)),
                 lambda: kda.embedding_backward(t(n, 1), ids(n), 7, d_table=t(7, 1)),
                 lambda: kda.embedding_backward(t(7, 1), ids(7), n, d_table=t(n, 1)),
                 lambda: kda.embedding_backward(t(1, n), ids(1), 7, d_table=t(7, n)),
                 lambda: kda.linear_cross_entropy(t(4, 8), t(n, 8), ids(4), **vec),
                 lambda: kda.linear_cross_entropy(t(4, n), t(9, n), ids(4), **vec),
                 lambda: kda.linear_cross_entropy(t(n, 8), t(9, 8), ids(n), loss=t(n), lse=t(n)),
                 lambda: kda.linear_cross_entropy_backward(t(4, 8), t(n, 8), ids(4), t(4), t(4),
                                                           want_dx=False, want_d_weight=False)):
        with pytest.raises(kda.KDAError) as e:
            call()
        assert e.value.status == UNSUPPORTED


def test_a_piece_beyond_32_bits_is_the_whole_vocabulary(monkeypatch):
    from kimi_delta_attention_18_gb300 import _lm
    desc = _lm._ce(_OnDevice(4, 8), _OnDevice(9, 8), _OnDevice(4, dtype=torch.int32), -100,
                   (1 << 32) + 256)[1]
    assert desc.piece == 0x7fffffff


def test_differentiable_forms_pass_the_status_on(monkeypatch):
    """Forward and backward of each operation give the library the caller's dev_status."""
    _stand_ins(monkeypatch)
    seen = []
    for module, names in ((autograd._lm, ("gated_norm", "residual_norm", "embedding", "linear_cross_entropy",
                                          "gated_norm_backward", "residual_norm_backward",
                                          "embedding_backward", "linear_cross_entropy_backward")),
                          (autograd._k, ("prefill_chunked", "prefill_backward"))):
        for name in names:
            def call(*a, fn=getattr(module, name), name=name, **kw):
                seen.append((name, kw["dev_status"]))
                return fn(*a, **kw)
            monkeypatch.setattr(module, name, call)
    x, w = torch.randn(2, 4, requires_grad=True), torch.ones(4, requires_grad=True)
    ids, status = torch.tensor([1, 0]), torch.zeros(1, dtype=torch.int32)
    s = dict(dev_status=status)
    for out in (autograd.kda_gated_norm(x[:, None], x[:, None], w, **s), autograd.kda_residual_norm(x, x, w, **s)[1],
                autograd.kda_residual_norm(x, None, w, **s)[1], autograd.kda_embedding(x, ids, **s),
                autograd.kda_linear_cross_entropy(x, x, ids, **s),
                autograd.kda_prefill(x[:, None], x[:, None], x[:, None], x[:, None], x[:, :1], **s)[0]):
        out.sum().backward()
    assert len(seen) == 12 and all(t is status for _, t in seen), seen
