"""Calls without a stream argument run on torch's current stream, after the work that is already on it: the
inputs are written on a side stream, behind tens of milliseconds of other work there, just before the calls."""
import pytest
import torch

from tests import test_gpu_layer_chain as TC

pytestmark = pytest.mark.gpu


def test_calls_follow_the_current_stream():
    want_step = TC.Step(N=200, seed=31)
    want_step.run()
    want = want_step.snapshot()
    s = TC.Step(N=200, seed=32)
    s.run()                                              # other inputs, and every kernel loaded
    torch.cuda.synchronize()
    for t in s.outputs().values():
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    a = torch.randn(8192, 8192, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(40):                              # tens of milliseconds: a call on another stream overtakes it
            a = (a @ a).mul_(1e-2)
        for name in ("x", "r", "Wb", "b", "gamma"):
            getattr(s, name).copy_(getattr(want_step, name))
        for name in ("W", "idx", "logit", "mask"):
            getattr(s.k, name).copy_(getattr(want_step.k, name))
        s.run()
    assert not side.query()                              # the calls were queued behind the work, not run ahead of it
    side.synchronize()
    for n, t in s.snapshot().items():
        assert torch.equal(t, want[n]), n
