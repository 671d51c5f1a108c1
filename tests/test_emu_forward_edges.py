"""Edge cases of the router, the experts' forward pass and the epilogue's
backward pass on the unchanged kernels in the CPU emulation (see
test_emu_forward)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import forward_cases as FC
import forward_edges as FE
from test_emu_forward import FULL, call, driver, held, nbytes, router_nums, stored  # noqa: F401


def emu(driver, tmp_path, c, expect=(0, 0), env_extra=None):  # noqa: F811
    """The forward call's outputs by name."""
    shapes = FC.forward_shapes(c)
    order = ("Y", "Yp", "Z", "A", "B", "h_sumsq")
    pr = c["pairs"]
    nums = [3, c["T"], c["N"], c["E"], int(c["kind"] != "linear"), int(c["dtype"] == "bf16"),
            ("none", "relu", "gelu", "silu").index(c["act"]), c["d_in"], c["d"],
            int(c["x_rows"] == "pair"), c["ldx"], c["d_out"], c["d_in"] * c["d"]]
    nums += [nbytes(*shapes[k]) if k in shapes else -1 for k in order]
    w = [c["W"], c["bias_t"]] if c["kind"] == "linear" else [c["W_gate"], c["W_up"], c["W_down"]]
    got = call(driver, tmp_path, nums,
               [pr["token"], pr["expert"], pr["weight"], c["X_store"].reshape(-1), c["R"], *w],
               [shapes[k] for k in order if k in shapes], expect=expect, env_extra=env_extra)
    return dict(zip([k for k in order if k in shapes], got))


@pytest.mark.parametrize("name", list(FE.ONE_TOKEN))
def test_emu_one_token_keeps_its_hidden_values_in_fp32(driver, tmp_path, name):  # noqa: F811
    c = FE.one_token_case(name)
    FE.judge_one_token(c, emu(driver, tmp_path, c))


def emu_route(driver, tmp_path, c):  # noqa: F811
    n, i32 = c["T"] * c["k"], torch.int32
    return call(driver, tmp_path, router_nums(0, c) + [4 * n, 4 * n, 4 * c["E"]],
                [stored(c), c["bias_t"], c["emask"], c["tmask"]],
                [((n,), i32), ((n,), torch.float32), ((n,), i32), ((c["E"],), i32)])


@pytest.mark.parametrize("name", list(FE.ZERO_TIES))
def test_emu_zeros_of_both_signs_tie(driver, tmp_path, name):  # noqa: F811
    c = FE.zero_case(name)
    FC.judge_route(c, *emu_route(driver, tmp_path, c))


@pytest.mark.parametrize("name", [n for n in FE.BAD_TOKENS if FULL or n != "many_blocks"])
@pytest.mark.parametrize("path", ["own", "tiles"])
def test_emu_tokens_out_of_range_are_absent(driver, tmp_path, name, path):  # noqa: F811
    c = FE.bad_token_case(name)
    got = emu(driver, tmp_path, c, expect=(0, 8),
              env_extra={"LRM_FWD_TILE": "64"} if path == "tiles" else None)
    FC.judge_forward(c, got, {k: held(*v) for k, v in FC.forward_shapes(c).items()})


@pytest.mark.parametrize("name", list(FE.OVERFLOW))
def test_emu_overflow_stays_infinite(driver, tmp_path, name):  # noqa: F811
    c = FE.overflow_case(name)
    FE.judge_overflow(c, emu(driver, tmp_path, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_emu_relu_keeps_nan(driver, tmp_path, dtype):  # noqa: F811
    c = FC._g(12, 3, 2, 24, dtype, act="relu")
    c.update(pairs=FC.make_pairs(12, 3, 2, 1), N=24)
    g, dt = FC.gen("relu nan"), FC.DT[dtype]
    c["Z"], c["dY"] = FC.normal(g, 24, 24, dtype=dt), FC.normal(g, 12, 24, dtype=dt)
    c["Z"][5, 7] = float("nan")
    pr, f32 = c["pairs"], torch.float32
    nums = [4, 12, 24, 3, 0, int(dtype == "bf16"), 1, 0, 24, 0, 24, 24, 0, 4 * 24,
            nbytes((24, 24), dt), -1]
    dw, G = call(driver, tmp_path, nums, [pr["token"], pr["expert"], pr["weight"], c["dY"], c["Z"]],
                 [((24,), f32), ((24, 24), dt)])
    assert torch.isnan(dw).nonzero()[:, 0].tolist() == [5]
    assert G[5, 7] == 0 and not torch.isnan(G).any()


@pytest.mark.parametrize("name", list(FE.CLOSED))
def test_emu_bias_of_minus_infinity_closes_an_expert(driver, tmp_path, name):  # noqa: F811
    c = FE.closed_case(name)
    FC.judge_route(c, *emu_route(driver, tmp_path, c))


@pytest.mark.parametrize("name", [n for n in FE.SPARSE if n != "many" and (FULL or n != "spread")])
def test_emu_long_runs_of_tokens_without_pairs(driver, tmp_path, name):  # noqa: F811
    c = FE.sparse_case(name)
    FC.judge_forward(c, emu(driver, tmp_path, c, env_extra={"LRM_FWD_TILE": "64"}))
