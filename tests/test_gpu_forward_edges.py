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
