"""CPU tests of where the binding allocates (no GPU): memory that a call
allocates for itself and uses on a caller's stream has to come from that
stream's pool.  Memory from the current stream's may have been freed there by
work that is still to run, and the two streams would use it at the same
time."""

import contextlib

import pytest
import torch

import implicit_gemm_conv_dp_amd as skg

from test_binding import FakeBuffer, FakeStream
from test_lowp_host import P


@pytest.fixture
def allocations(monkeypatch):
    """(bytes, stream of the pool) of each torch.empty; None is the current
    stream's."""
    made, pool = [], [None]

    @contextlib.contextmanager
    def on(stream):
        before, pool[0] = pool[0], stream
        yield
        pool[0] = before

    def empty(n, **kw):
        made.append((n, pool[0]))
        return FakeBuffer(n)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: FakeStream(5))
    return made


@pytest.mark.parametrize("side", [FakeStream(0xABC), None])
def test_workspace_of_a_plan(allocations, side):
    calls = []
    skg._run(lambda *a: calls.append(a), "args", {"workspace_bytes": 4096}, "cuda:0", None, side)
    assert allocations == [(4096, side)]
    assert calls == [("args", 0x10000, 4096, 0xABC if side else 5)]


class Weight:
    device = "cuda:0"

    def data_ptr(self):
        return 0x20000


@pytest.mark.parametrize("side", [FakeStream(0xABC), None])
def test_workspace_of_the_norms_gradient(allocations, monkeypatch, side):
    calls = []
    monkeypatch.setattr(skg, "skg_run_rmsnorm_bwd", lambda *a: calls.append(a))
    monkeypatch.setattr(skg, "_handle", lambda s: s.cuda_stream if s else 5)
    skg.rmsnorm_bwd(P, P, P, P, rows=3000, cols=1024, dtype="bf16", dw=Weight(), stream=side)
    need = skg.skg_rmsnorm_bwd_workspace_bytes(
        skg.rmsnorm_bwd_args(P, P, P, P, rows=3000, cols=1024, dtype="bf16", dw=P))
    assert need > 0 and allocations == [(need, side)]
    assert [c[1:] for c in calls] == [(0x10000, need, 0xABC if side else 5)]
