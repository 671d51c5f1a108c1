"""Edge cases of the router, the experts' forward pass and the epilogue's
backward pass on the GPU (see test_gpu_forward)."""

import numpy as np
import pytest
import torch

import forward_cases as FC
import forward_edges as FE
from test_gpu_forward import L, dev, filled, make_forward, run_forward  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("name", list(FE.ONE_TOKEN))
def test_one_token_keeps_its_hidden_values_in_fp32(L, name):  # noqa: F811
    c = FE.one_token_case(name)
    out, _ = run_forward(L, c)
    FE.judge_one_token(c, out)
