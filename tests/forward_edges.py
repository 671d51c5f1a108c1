"""Inputs and references of the edge cases of the router, the experts' forward
pass and the epilogue's backward pass, shared by the emulated and the GPU tests
(see forward_cases, whose notation the bounds take)."""

from __future__ import annotations

import numpy as np
import torch

import forward_cases as FC
from oracle import forward as OF

U = FC.U


# ------------------------------------------------- one token's hidden values
ONE_TOKEN = {
    "one": FC._f("swiglu", 1, 16, 8, 24, 264),
    "two": FC._f("swiglu", 2, 64, 8, 16, 72),
    "long": FC._f("swiglu", 1, 5, 2, 8, 1544),
    "f32": FC._f("swiglu", 1, 16, 4, 20, 516, "f32"),
}


def one_token_case(name):
    """The residual takes nearly all of Y away, so that Y's own rounding does not
    hide those of the sums."""
    c = FC.build_forward(ONE_TOKEN[name], "one token " + name)
    ref = OF.forward("swiglu", c["pairs"], c["T"], c["E"], c["X"], W_gate=c["W_gate"],
                     W_up=c["W_up"], W_down=c["W_down"])
    c["R"] = (-ref["Y"]).to(c["X"].dtype)
    return c


def judge_one_token(c, got):
    """silu(a) b held in fp32 between the products: FC.judge_forward's bounds
    without the rounding to the inputs' type (half |h|) and with one of fp32
    (U |h|) in its place."""
    pr, T, E, N = c["pairs"], c["T"], c["E"], c["N"]
    ref = OF.forward("swiglu", pr, T, E, c["X"], W_gate=c["W_gate"], W_up=c["W_up"],
                     W_down=c["W_down"], residual=c["R"])
    half = FC.HALF[c["X"].dtype]
    h, d = c["d_in"], c["d"]
    ax = c["X"].double().abs()[torch.from_numpy(pr["token"]).long()]
    ex = pr["expert"]

    def absdot(W, v):
        return torch.stack([W[int(ex[p])].double().abs() @ v[p] for p in range(N)])

    ta, tb = ((h + 4) * U * absdot(c[w], ax) for w in ("W_gate", "W_up"))
    a, b = ref["A"], ref["B"]
    s = OF.act(a, "silu")
    hv = (s * b).abs()
    th = 1.13 * ta * (b.abs() + tb) + s.abs() * tb + 16 * U * (1 + a.abs()) * b.abs()
    th = th + U * (hv + th)
    ty = absdot(c["W_down"], th + (d + 4) * U * (hv + th))
    FC.close("Yp", got["Yp"].cpu(), ref["Yp"], ty + half * (ref["Yp"].abs() + ty))
    FC.close("h_sumsq", got["h_sumsq"].cpu(), (hv * hv).sum(1),
             (2 * hv * th + th * th).sum(1) + 4 * d * U * (hv * hv).sum(1))
    tY = (c["k"] + 4) * U * c["R"].double().abs()
    for p in range(N):
        t, w = int(pr["token"][p]), abs(float(pr["weight"][p]))
        tY[t] += w * (ty[p] + (c["k"] + 4) * U * ref["Yp"][p].abs())
    FC.close("Y", got["Y"].cpu(), ref["Y"], tY + half * (ref["Y"].abs() + tY))
