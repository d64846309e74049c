"""A recurrent layer's parts without a GPU: the C ABI refuses bad arguments on the host with
the documented status codes, sizes its workspaces, and the binding refuses bad tensors
before it calls anything."""
import math

import pytest
import torch

import kimi_delta_attention_18_gb300 as kda
from kimi_delta_attention_18_gb300._layer import RecurrenceDesc

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
    assert kda.lib().kda_recurrence_workspace_size(d) == 0
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
    assert size(_rec(tokens=1024)) == 0 and size(_rec(tokens=0)) == 0
    d = _rec(tokens=1025, channels=100)
    need = size(d)
    # tiles of 128 tokens (one more for each sequence) x 64 channels: a flag, maps and ends
    tiles = 1025 // 128 + 2
    assert tiles * (16 + 2 * 4 + 128 * 12) <= need <= tiles * (16 + 2 * 4 + 128 * 12) + 5 * 256
    assert _forward(d) == WORKSPACE and _backward(d) == WORKSPACE
    assert _forward(d, ws=A, ws_len=need - 1) == WORKSPACE
    assert _forward(d, ws=A + 8, ws_len=need) == WORKSPACE
    # sequences of one token each: never more tiles than tokens
    assert size(_rec(tokens=1025, num_seqs=2 ** 20, channels=100)) < 1025 * (16 + 8 + 128 * 12) + 5 * 256


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
