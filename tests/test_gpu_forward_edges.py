"""Edge cases of the router, the experts' forward pass and the epilogue's
backward pass on the GPU (see test_gpu_forward)."""

import numpy as np
import pytest
import torch

import forward_cases as FC
import forward_edges as FE
from test_gpu_forward import L, dev, filled, make_forward, make_router, run_forward  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("name", list(FE.ONE_TOKEN))
def test_one_token_keeps_its_hidden_values_in_fp32(L, name):  # noqa: F811
    c = FE.one_token_case(name)
    out, _ = run_forward(L, c)
    FE.judge_one_token(c, out)


def gpu_route(L, c):  # noqa: F811
    n, i32 = c["T"] * c["k"], torch.int32
    out = dict(expert=filled((n,), i32), weight=filled((n,), torch.float32), token=filled((n,), i32),
               counts=filled((c["E"],), i32))
    L.lrm_route(make_router(L, c), **out)
    torch.cuda.synchronize()
    return [out[k].cpu() for k in ("expert", "weight", "token", "counts")]


@pytest.mark.parametrize("name", list(FE.ZERO_TIES))
def test_zeros_of_both_signs_tie(L, name):  # noqa: F811
    c = FE.zero_case(name)
    FC.judge_route(c, *gpu_route(L, c))


def test_workspaces_of_another_stream_are_not_handed_out(L):  # noqa: F811
    """Calls on a side stream that is still busy allocate their own workspaces;
    the current stream then allocates and fills memory of the same sizes."""
    T, E, k = 40_000, 64, 4
    g = FC.gen("busy")
    z = FC.normal(g, T, E)
    r = L.Router(dev(z), k)
    n, i32, f32 = T * k, torch.int32, torch.float32
    expert, weight, counts = filled((n,), i32), filled((n,), f32), filled((E,), i32)
    out = dict(out_token=filled((n,), i32), out_expert=filled((n,), i32),
               out_weight=filled((n,), f32), out_n=filled((1,), i32))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    L.lrm_route(r, expert, weight, counts=counts, stream=side)
    L.lrm_route_share(T, k, expert, weight, 8, 16, **out, stream=side)
    for size in (r.ws_bytes, int(L._lib.lrm_route_share_workspace_size(T, k))):
        for _ in range(4):
            torch.full((size,), 0x7F, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    want = dev(z).sort(dim=1, descending=True, stable=True).indices[:, :k].int().reshape(-1)
    assert torch.equal(expert, want)
    assert torch.equal(counts, torch.bincount(want.long(), minlength=E).int())
    here = ((want >= 8) & (want < 24)).nonzero()[:, 0]
    m = here.numel()
    assert int(out["out_n"]) == m
    assert torch.equal(out["out_expert"][:m], want[here] - 8)
    assert torch.equal(out["out_token"][:m], (here // k).int())
