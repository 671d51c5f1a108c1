"""CPU tests of the binding's edge cases: the router, the experts' forward pass
and the epilogue's backward pass (see test_forward_host)."""

import contextlib

import numpy as np
import pytest
import torch

from oracle import forward as OF
from pruned_expert_backward_lrm_amd import lrm as L


class FakeLibrary:
    """Answers every call with LRM_OK and every size query with 4096."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_workspace_size") else L.LRM_OK


class FakeStream:
    cuda_stream, device_index = 0, 0


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def every_call(stream):
    """Every call that may allocate its workspace, on `stream`."""
    N, T, E = 8, 4, 2
    pr = L.Pairs(i32(N), i32(N), torch.zeros(N), T, E)
    X, W = torch.zeros(T, 8), torch.zeros(E, 12, 8)
    r = L.Router(X, 2)
    f = L.linear_forward(pr, X, "token", W)
    pg = L.pair_grad_problem(pr, X, "token", torch.zeros(N, 8))
    pb = L.linear_problem(pr, X, "token", torch.zeros(T, 12), "token", W, [4, 4])
    m = L.mat(X, "token")
    return {
        "lrm_route": lambda: L.lrm_route(r, i32(8), torch.zeros(8), counts=i32(8), stream=stream),
        "lrm_route_share": lambda: L.lrm_route_share(T, 2, i32(8), torch.zeros(8), 0, E, i32(8), i32(8),
                                                     torch.zeros(8), i32(1), stream=stream),
        "lrm_expert_forward": lambda: L.lrm_expert_forward(f, dict(Y=torch.zeros(T, 12)),
                                                           stream=stream),
        "lrm_pair_grad": lambda: L.lrm_pair_grad(pg, dict(dweight=torch.zeros(N)), stream=stream),
        "lrm_expert_backward": lambda: L.lrm_expert_backward(pb, {}, stream=stream),
        "lrm_expert_backward_events": lambda: L.lrm_expert_backward_events(pb, {}, [], stream=stream),
        "lrm_score": lambda: L.lrm_score(pr, m, m, torch.zeros(N), stream=stream),
        "lrm_score_glu": lambda: L.lrm_score_glu(pr, m, m, m, torch.zeros(N), stream=stream),
        "lrm_select": lambda: L.lrm_select(pr, torch.zeros(N), [4, 4], i32(N), i32(3), i32(N),
                                           stream=stream),
        "lrm_grouped_bwd": lambda: L.lrm_grouped_bwd(E, i32(3), N, X, X, W, 8, 12, W, X, stream=stream),
        "lrm_unpermute": lambda: L.lrm_unpermute(pr, i32(N), X, 8, "token", X, stream=stream),
        "lrm_quota_waterfill_device": lambda: L.lrm_quota_waterfill_device(pr, 4, i32(E),
                                                                           stream=stream),
        "lrm_receiver_layout": lambda: L.lrm_receiver_layout(i32(3), i32(E, 1), 4, stream=stream),
    }


@pytest.mark.parametrize("name", list(every_call(None)))
def test_a_workspace_is_allocated_on_the_stream_that_uses_it(monkeypatch, name):
    s, inside, scratch = FakeStream(), [], []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    empty = torch.empty

    def record(*a, **kw):
        if kw.get("dtype") == torch.uint8:
            scratch.append(inside[-1] if inside else None)
        return empty(*a, **kw)

    call = every_call(s)[name]
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", record)
    monkeypatch.setattr(L, "_lib", FakeLibrary())
    monkeypatch.setattr(L, "_stream", lambda *a: 0)
    call()
    assert scratch == [s]


def test_experts_that_share_weights_are_refused():
    """A W shared over the experts holds one expert's elements: described with
    the stride of a dense W, the kernels would read past it."""
    pr = L.Pairs(i32(8), i32(8), torch.zeros(8), 4, 4)
    X, W = torch.zeros(4, 8), torch.zeros(12, 8)
    with pytest.raises(ValueError):
        L.linear_forward(pr, X, "token", W.expand(4, -1, -1))
    store = torch.zeros(4 * 48 + 96)
    with pytest.raises(ValueError):  # experts that overlap
        L.linear_forward(pr, X, "token", store.as_strided((4, 12, 8), (48, 8, 1)))
    wide = torch.zeros(4, 2, 12, 8)[:, 0]  # a gap between the experts
    assert L.linear_forward(pr, X, "token", wide).c.w_stride == 192
    one = L.Pairs(i32(8), i32(8), torch.zeros(8), 4, 1)  # of one expert any stride will do
    assert L.linear_forward(one, X, "token", W.expand(1, -1, -1)).c.w_stride == 96
    assert L.linear_forward(one, X, "token", store.as_strided((1, 12, 8), (7, 8, 1))).c.w_stride == 96


def test_bias_of_minus_infinity_by_hand():
    """Expert 1 is closed: not chosen, nor counted for its group, but part of the
    softmax."""
    z, b = torch.tensor([[0.0, 2.0, 1.0, 0.0]]), torch.tensor([0.0, -float("inf"), 0.0, 0.0])
    e, w = OF.route(z, 4, renorm=False, bias=b)
    s = torch.softmax(z[0].double(), 0)
    assert e.tolist() == [2, 0, 3, -1]
    assert np.allclose(w, [float(s[2]), float(s[0]), float(s[3]), 0.0])
    e, _ = OF.route(z, 2, n_group=2, topk_group=1, group_rule="max", bias=b)
    assert e.tolist() == [2, 3]
    e, _ = OF.route(torch.tensor([[0.6, 2.0, 0.0, -9.0]]), 2, score="sigmoid", n_group=2, topk_group=1,
                    bias=b)
    assert e.tolist() == [0, -1]


@pytest.mark.parametrize("name", ["lrm_route", "lrm_route_bwd", "lrm_route_share", "lrm_expert_forward",
                                  "lrm_pair_grad"])
def test_tensors_in_host_memory_are_refused(monkeypatch, name):
    """The library would hand their addresses to the GPU."""
    X, n = torch.zeros(4, 8), i32(8)
    calls = dict(every_call(None), lrm_route_bwd=lambda: L.lrm_route_bwd(L.Router(X, 2), n,
                                                                         torch.zeros(8), X))
    monkeypatch.setattr(L, "_lib", FakeLibrary())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream())
    with pytest.raises(ValueError, match="GPU"):
        calls[name]()
    with pytest.raises(ValueError, match="GPU"):
        L._stream(FakeStream(), X.device)


def test_a_call_on_another_device_is_refused(monkeypatch):
    class On(FakeStream):
        def __init__(self, index):
            self.device_index = index

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: On(0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)
    assert L._stream(None, here) == 0 and L._stream(On(0), here) == 0 and L._stream(On(1)) == 0
    for stream, device in ((None, there), (On(1), here), (On(1), there), (On(0), there)):
        with pytest.raises(ValueError, match="device"):
            L._stream(stream, device)
