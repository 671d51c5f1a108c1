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


# ------------------------------------------------------- zeros of both signs
# -0 and +0 are equal logits: the border of the choice lies between them (z1 of
# a row's zeros, the rest below), or between groups whose best are zeros.
ZERO_TIES = {
    "direct": dict(T=40, E=16, k=1, dtype="bf16"),
    "direct_mid": dict(T=40, E=136, k=3, dtype="bf16"),
    "direct_wide": dict(T=20, E=512, k=4, dtype="bf16"),
    "not_renormed": dict(T=40, E=16, k=2, dtype="bf16", renorm=False),
    "odd": dict(T=40, E=15, k=2, dtype="bf16"),
    "sigmoid": dict(T=40, E=15, k=1, dtype="bf16", score="sigmoid"),
    "f32": dict(T=40, E=16, k=2, dtype="f32"),
    "f32_odd": dict(T=40, E=61, k=3, dtype="f32"),
    "f32_wide": dict(T=12, E=600, k=2, dtype="f32"),
    "wide": dict(T=12, E=600, k=2, dtype="bf16"),
    "widest": dict(T=4, E=1100, k=2, dtype="f32"),
    "bias": dict(T=40, E=24, k=2, dtype="f32", bias=True, score="sigmoid"),
    "groups_lanes": dict(T=40, E=64, k=2, dtype="bf16", n_group=8, topk_group=1, group_rule="max"),
    "groups_lanes_f32": dict(T=40, E=64, k=2, dtype="f32", n_group=4, topk_group=2,
                             group_rule="max"),
    "groups_odd": dict(T=40, E=60, k=2, dtype="f32", n_group=10, topk_group=2, group_rule="max"),
    "groups_wide": dict(T=8, E=600, k=2, dtype="f32", n_group=50, topk_group=2, group_rule="max"),
    "groups_top2": dict(T=40, E=64, k=3, dtype="f32", n_group=8, topk_group=2),
    "masked": dict(T=40, E=16, k=2, dtype="bf16", emask=True),
}


def zero_case(name):
    c = dict(score="softmax", renorm=True, scale=1.0, n_group=1, topk_group=1, group_rule="top2",
             bias=False, emask=False)
    c.update(ZERO_TIES[name])
    T, E = c["T"], c["E"]
    g = FC.gen("zeros", name)
    z = -1.0 - torch.rand(T, E, generator=g)
    rng = np.random.default_rng(T + E)
    for t in range(T):
        at = np.sort(rng.choice(E, size=min(E, c["k"] + 4), replace=False))
        sign = rng.random(at.size) < 0.5
        sign[0], sign[-1] = True, False  # the lowest is -0, the highest +0
        z[t, torch.from_numpy(at)] = torch.from_numpy(np.where(sign, -0.0, 0.0).astype(np.float32))
    c["bias_t"] = torch.zeros(E) if c["bias"] else None
    c["tmask"] = None
    c["emask"] = (torch.rand(E, generator=g) < 0.7).to(torch.uint8) if c["emask"] else None
    c["logits"] = z.to(FC.DT[c["dtype"]])
    c["ld"] = E
    return c


# ------------------------------------------------------ tokens out of range
# where: the pairs whose token is out of range, as a share of the list
BAD_TOKENS = {
    "middle": (FC._f("linear", 20, 8, 2, 24, 16, residual=True), ((0.5, -1), (0.7, 1 << 20))),
    "past_t": (FC._f("linear", 20, 8, 2, 24, 16), ((0.5, 20),)),
    "ends": (FC._f("linear", 20, 8, 2, 24, 16, "f32", residual=True), ((0.0, -5), (0.999, -5))),
    "runs": (FC._f("linear", 90, 5, 2, 16, 24), ((slice(0.2, 0.4), -1), (slice(0.7, 0.73), 90))),
    "padded": (FC._f("linear", 90, 5, 2, 16, 24, residual=True), ((slice(0.6, 1.0), -1),)),
    "padded_high": (FC._f("linear", 90, 5, 2, 16, 24), ((slice(0.6, 1.0), 90),)),
    "all": (FC._f("linear", 40, 5, 2, 16, 24, residual=True), ((slice(0.0, 1.0), -1),)),
    "swiglu": (FC._f("swiglu", 60, 5, 2, 24, 16, residual=True), ((0.3, -1), (slice(0.5, 0.6), 60))),
    "swiglu_few": (FC._f("swiglu", 3, 64, 4, 24, 16), ((0.5, -1), (0.7, 3))),
    "swiglu_sum": (FC._f("swiglu", 9, 8, 4, 24, 16), ((0.5, -1), (0.7, 9))),
    "many_blocks": (FC._f("linear", 4500, 7, 2, 16, 8, empty=0.1), ((slice(0.3, 0.5), -1), (0.9, -2))),
}


def bad_token_case(name):
    case, where = BAD_TOKENS[name]
    c = FC.build_forward(case, "bad tokens " + name)
    N, tok = c["N"], c["pairs"]["token"]
    for at, t in where:
        if isinstance(at, slice):
            tok[int(at.start * N):max(int(at.stop * N), int(at.start * N) + 1)] = t
        else:
            tok[int(at * N)] = t
    return c


# ------------------------------------------- products past fp32, and no numbers
# Column 0 of some tokens is huge, and so is some weight rows' column 0: their
# product passes fp32 (upwards only where the activation of -inf is no number).
# One token holds a NaN.
OVERFLOW = {
    "none": FC._f("linear", 90, 5, 2, 16, 24, residual=True),
    "relu": FC._f("linear", 90, 5, 2, 16, 40, act="relu", bias=True),
    "gelu": FC._f("linear", 90, 5, 2, 24, 24, act="gelu"),
    "silu": FC._f("linear", 90, 5, 2, 16, 24, act="silu", residual=True),
    "f32": FC._f("linear", 90, 5, 2, 16, 24, "f32", act="relu", residual=True),
    "gelu_f32": FC._f("linear", 90, 5, 2, 16, 24, "f32", act="gelu"),
    "few": FC._f("linear", 9, 5, 2, 16, 24, act="relu"),
}


def overflow_case(name):
    c = FC.build_forward(OVERFLOW[name], "overflow " + name)
    c["X_store"][1::4, 0] = 3e38
    c["W"][:, ::5, 0] = 4.0
    if c["act"] in ("none", "relu"):
        c["W"][:, 1::5, 0] = -4.0
    c["X_store"][2, 3] = float("nan")
    return c


def judge_overflow(c, got):
    """Z, Yp and Y: infinities and NaN where the formula in fp32 has them; the
    finite ones in coarse bounds (the other tests have the fine ones)."""
    ref = OF.forward("linear", c["pairs"], c["T"], c["E"], c["X"], W=c["W"], bias=c["bias_t"],
                     act_name=c["act"], residual=c["R"])
    for k in ("Z", "Yp", "Y"):
        want, v = ref[k].float(), got[k].cpu().float()
        assert torch.isinf(want).any() and torch.isnan(want).any()
        assert torch.equal(torch.isnan(v), torch.isnan(want)), k
        inf = torch.isinf(want)
        assert torch.equal(v[inf], want[inf]) and not torch.isinf(v[~inf]).any(), k
        fin = torch.isfinite(want)
        assert ((v - want).abs()[fin] <= 2.0 ** -6 * (want.abs()[fin] + 1)).all(), k


# ------------------------------------------------- biases of minus infinity
# They close an expert to the choice alone.
CLOSED = {
    "few_left": dict(T=30, E=16, k=4, dtype="f32", score="sigmoid", open=3),
    "some": dict(T=30, E=40, k=4, dtype="bf16", score="sigmoid", open=30),
    "softmax": dict(T=30, E=40, k=4, dtype="f32", open=20, renorm=False),
    "groups": dict(T=30, E=64, k=4, dtype="f32", score="sigmoid", open=20, n_group=8, topk_group=2),
    "groups_max": dict(T=30, E=60, k=4, dtype="bf16", open=20, n_group=10, topk_group=2,
                       group_rule="max"),
    "wide": dict(T=8, E=600, k=6, dtype="f32", score="sigmoid", open=300),
    "none_left": dict(T=8, E=16, k=2, dtype="f32", open=0),
}


def closed_case(name):
    c = dict(score="softmax", renorm=True, scale=1.0, n_group=1, topk_group=1, group_rule="top2")
    c.update(CLOSED[name])
    T, E = c["T"], c["E"]
    g = FC.gen("closed", name)
    c["logits"] = FC.normal(g, T, E, std=2.0, dtype=FC.DT[c["dtype"]])
    c["bias_t"] = FC.normal(g, E, std=0.3)
    c["bias_t"][torch.randperm(E, generator=g)[c["open"]:]] = -float("inf")
    c["tmask"] = c["emask"] = None
    c["ld"] = E
    return c


# --------------------------------------------- long runs of tokens without pairs
def sparse_case(name):
    """`tail`, `head`: all pairs in 40 neighbouring tokens of 1000; `spread`: about 90
    pairs over 6000 tokens, a third of the gaps long ones; `many`: more long gaps
    than a workgroup notes; `none`."""
    T, k, drop = {"tail": (40, 2, 0.0), "head": (40, 2, 0.0), "spread": (6000, 1, 0.985),
                  "many": (60000, 1, 0.99), "none": (40, 2, 1.0)}[name]
    c = FC.build_forward(FC._f("linear", T, 5, k, 8, 8, residual=name != "head", drop=drop,
                               outs=("Y",)), "sparse " + name)
    if name not in ("spread", "many"):  # the same pairs among more tokens
        more, dt = 1000 - T, c["X"].dtype
        g = FC.gen("sparse more", name)
        first = name != "head"

        def grow(m):
            new = FC.normal(g, more, m.shape[1], dtype=dt)
            return torch.cat([m, new] if first else [new, m])

        c["X_store"] = grow(c["X_store"])
        c["X"] = c["X_store"][:, :c["d_in"]]
        if c["R"] is not None:
            c["R"] = grow(c["R"])
        if not first:
            c["pairs"] = dict(c["pairs"], token=c["pairs"]["token"] + np.int32(more))
        c["T"] = 1000
    return c


SPARSE = ("tail", "head", "spread", "none", "many")
