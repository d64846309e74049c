"""Calls of the mixer's entry points on a stream of their own: results as on the current
stream, and memory that is shared with nothing else before the call's kernels have run."""
import pytest
import torch

import kimi_delta_attention_18_gb300 as kda
from kimi_delta_attention_18_gb300.inputs import make_decode_inputs, make_prefill_inputs

pytestmark = pytest.mark.gpu


def _calls():
    dev = torch.device("cuda", 0)
    x = make_prefill_inputs([700, 324], 4, 128, 128, "bf16", seed=3, s0_std=0.5, device=dev)
    a = [x[n] for n in ("q", "k", "v", "g", "beta", "S0", "cu_seqlens")]
    d_out = torch.randn((1024, 4, 128), device=dev).bfloat16()
    y = make_decode_inputs(6, 4, 128, 128, 1, "bf16", seed=4, device=dev)
    b = [y[n][0] for n in ("q", "k", "v", "g", "beta")]

    def state(s):  # a decode step changes it in place
        with torch.cuda.stream(s):
            return y["S0"].clone()

    A, B = kda.state_transfer(*a[1:5], a[6], 3)
    U = A.shape[0] * A.shape[1]
    A, B = A.reshape(U, *A.shape[2:]), B.reshape(U, *B.shape[2:])
    return [lambda s: kda.prefill_chunked(*a, num_segments=3, stream=s),
            lambda s: kda.prefill_chunked_ckpt(*a, ckpt_interval=64, num_segments=2, stream=s),
            lambda s: kda.prefill_backward(*a, d_out, stream=s),
            lambda s: kda.state_transfer(*a[1:5], a[6], 3, stream=s),
            lambda s: kda.state_compose(A, B, stream=s),
            lambda s: kda.prefill_segments(*a[:5], None, a[6], 3, stream=s),
            lambda s: (kda.decode_step(*b, state(s), stream=s),)]


def test_tensors_of_calls_on_another_stream_are_kept():
    s = torch.cuda.Stream()
    for call in _calls():
        want = [t.clone() for t in call(None)]
        sizes = [t.numel() * t.element_size() for t in want] + [1 << k for k in (16, 20, 22, 24)]
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
