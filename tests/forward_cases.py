"""Inputs, fp64 references and tolerances shared by the tests of the router,
the experts' forward pass and the epilogue's backward pass (on the GPU and in
the CPU emulation).

Tolerances are elementwise bounds derived from the arithmetic, with u = 2^-24
(half a step of fp32, relative) and half = half a step of the output type:

* a sum of n products held in fp32 is off by at most (n + 4) u sum |terms|
  (bf16 products are exact in fp32);
* activations and their derivatives are Lipschitz with constants below 1.13
  and evaluated to 16 u of (1 + |z|) or better;
* silu(a) b is rounded to the input type before the down product: half |h|;
* the rows that are joined keep 24 bits: 2^-16 |y|;
* exp(z - m) is off by (|z - m| + 4) u of its value.
"""

from __future__ import annotations

import zlib

import numpy as np
import torch

from oracle import forward as OF

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def make_pairs(T, E, k, seed, drop=0.0, skew=0.0, empty_tokens=0.0):
    """Token-major pairs, k distinct experts per token; `drop` of them left out,
    `empty_tokens` of the tokens without any."""
    rng = np.random.default_rng(seed)
    logits = rng.normal(size=(T, E)) - skew * np.log1p(np.arange(E))
    ex = np.argsort(-logits, axis=1)[:, :k].reshape(-1)
    tok = np.repeat(np.arange(T), k)
    keep = rng.random(tok.size) >= drop
    keep &= ~np.isin(tok, np.nonzero(rng.random(T) < empty_tokens)[0])
    w = rng.random(tok.size) + 0.1
    return dict(token=tok[keep].astype(np.int32), expert=ex[keep].astype(np.int32),
                weight=w[keep].astype(np.float32))


def close(name, got, ref, tol):
    got, ref, tol = (torch.as_tensor(v).double() for v in (got, ref, tol))
    assert got.shape == ref.shape, f"{name}: shape {tuple(got.shape)} != {tuple(ref.shape)}"
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}{list(i)}: {float(got[i])!r} for {float(ref[i])!r}, tolerance "
                             f"{float(tol[i]):.3g} ({int(bad.sum())} of {bad.numel()} off)")


# ------------------------------------------------------------------ router
ROUTE_CASES = {
    "one": dict(T=1, E=1, k=1),
    "t1": dict(T=1, E=128, k=8),
    "odd": dict(T=37, E=61, k=5, dtype="f32"),
    "odd_bf16": dict(T=37, E=63, k=7, renorm=False, scale=2.5),
    "all": dict(T=9, E=12, k=12, dtype="f32"),
    "ties": dict(T=64, E=96, k=8, coarse=True),
    "ties_bias": dict(T=64, E=96, k=8, coarse=True, bias=True, score="sigmoid"),
    "equal_bias": dict(T=40, E=128, k=8, dtype="f32", near=True, bias=True, score="sigmoid"),
    "softmax_bias": dict(T=50, E=72, k=4, dtype="f32", bias=True, near=True),
    "groups_top2": dict(T=50, E=64, k=6, n_group=8, topk_group=3, score="sigmoid", bias=True),
    "groups_max": dict(T=50, E=60, k=6, n_group=5, topk_group=2, group_rule="max", dtype="f32"),
    "groups_softmax": dict(T=50, E=66, k=4, n_group=22, topk_group=9, dtype="f32", coarse=True),
    "groups_one_each": dict(T=30, E=40, k=4, n_group=40, topk_group=6, score="sigmoid"),
    "masks": dict(T=60, E=50, k=6, score="sigmoid", padded=0.3, down=20, minus_inf=0.5),
    "masks_softmax": dict(T=60, E=50, k=6, padded=0.3, down=46, renorm=False),
    "masks_groups": dict(T=60, E=48, k=8, n_group=6, topk_group=2, down=30, minus_inf=0.5,
                         score="sigmoid", bias=True),
    "lowest": dict(T=20, E=33, k=4, dtype="f32", lowest=True),
    "lowest_sigmoid": dict(T=20, E=33, k=4, lowest=True, score="sigmoid"),
    "wide": dict(T=20, E=160, k=20, dtype="f32", score="sigmoid", renorm=True),
    "wider": dict(T=7, E=700, k=40, bias=True, score="sigmoid"),
    "widest": dict(T=5, E=4096, k=64, dtype="f32"),
    "widest_groups": dict(T=3, E=4096, k=8, n_group=64, topk_group=4, score="sigmoid", bias=True),
    "strided": dict(T=33, E=40, k=3, ld=43, dtype="bf16"),
}


def route_case(name):
    c = dict(dtype="bf16", score="softmax", renorm=True, scale=1.0, n_group=1, topk_group=1,
             group_rule="top2", bias=False, padded=0.0, down=0, minus_inf=0.0, coarse=False,
             near=False, lowest=False, ld=0)
    c.update(ROUTE_CASES[name])
    T, E = c["T"], c["E"]
    g = gen("route", name)
    z = torch.randn(T, E, generator=g) * 2
    if c["coarse"]:  # many exact ties
        z = torch.round(z)
    if c["near"]:  # neighbours that 32 bits cannot tell apart, or barely
        z = torch.round(z) + 2e-7 * torch.randint(-3, 4, (T, E), generator=g)
    lo = torch.finfo(DT[c["dtype"]]).min
    if c["lowest"]:  # the type's lowest value as a mask; one row holds nothing else
        z[torch.rand(T, E, generator=g) < 0.8] = lo
        z[0] = lo
    if c["minus_inf"]:
        z[torch.rand(T, E, generator=g) < c["minus_inf"]] = -float("inf")
        z[T // 2] = -float("inf")
    c["bias_t"] = None
    if c["bias"]:
        c["bias_t"] = torch.randn(E, generator=g) * 0.3
        if c["coarse"]:
            c["bias_t"] = torch.zeros(E)
    c["tmask"] = c["emask"] = None
    if c["padded"]:
        c["tmask"] = (torch.rand(T, generator=g) >= c["padded"]).to(torch.uint8)
        z[c["tmask"] == 0] = float("nan")
    if c["down"]:
        c["emask"] = torch.ones(E, dtype=torch.uint8)
        c["emask"][torch.randperm(E, generator=g)[:c["down"]]] = 0
        z[:, c["emask"] == 0] = float("inf")
        z[::2, c["emask"] == 0] = float("nan")
    c["logits"] = z.to(DT[c["dtype"]])
    c["ld"] = c["ld"] or E
    return c


def route_kw(c):
    return dict(score=c["score"], renorm=c["renorm"], scale=c["scale"], n_group=c["n_group"],
                topk_group=c["topk_group"], group_rule=c["group_rule"], bias=c["bias_t"],
                expert_mask=c["emask"], token_mask=c["tmask"])


def _spread(c):
    """Largest |z - m| that a score's exponential sees (finite ones, capped where
    the result underflows anyway)."""
    z = c["logits"].double()
    z = z[torch.isfinite(z)]
    return min(float(z.max() - z.min()), 110.0) if z.numel() else 0.0


def judge_route(c, expert, weight, token=None, counts=None):
    e, w = OF.route(c["logits"], c["k"], **route_kw(c))
    expert = np.asarray(expert, np.int64)
    assert np.array_equal(expert, e), f"slots {np.nonzero(expert != e)[0][:8]} differ"
    w = torch.from_numpy(w)
    tol = (2 * _spread(c) + c["k"] + c["E"] + 32) * U * w.abs() + 1e-37
    close("weight", weight, w, tol)
    if token is not None:
        assert np.array_equal(np.asarray(token), np.repeat(np.arange(c["T"]), c["k"]))
    if counts is not None:
        assert np.array_equal(np.asarray(counts), np.bincount(e[e >= 0], minlength=c["E"]))


def route_grad_inputs(c, name):
    e, _ = OF.route(c["logits"], c["k"], **route_kw(c))
    g = gen("dw", name)
    dw = torch.randn(c["T"] * c["k"], generator=g)
    dw[torch.from_numpy(e < 0)] = float("nan")  # empty slots are not read
    return torch.from_numpy(e.astype(np.int32)), dw


def judge_route_bwd(c, e, dw, dlogits):
    T, k = c["T"], c["k"]
    dw0 = torch.nan_to_num(dw)
    ref = OF.route_bwd(c["logits"], k, e.numpy(), dw0, score=c["score"], renorm=c["renorm"],
                       scale=c["scale"], expert_mask=c["emask"], token_mask=c["tmask"])
    big = c["scale"] * dw0.abs().double().view(T, k).amax(1, keepdim=True)
    tol = (2 * _spread(c) + c["k"] + c["E"] + 32) * U * big + HALF[DT[c["dtype"]]] * ref.abs()
    close("dlogits", dlogits, ref, tol.expand_as(ref))


# ---------------------------------------------------------- experts forward
def _f(kind, T, E, k, d_in, d, dtype="bf16", **kw):
    c = dict(kind=kind, T=T, E=E, k=k, d_in=d_in, d=d, dtype=dtype, act="none", bias=False,
             residual=False, x_rows="token", drop=0.0, skew=0.0, empty=0.0, bad=False, ldx=0,
             twice=False, outs=None)
    c.update(kw)
    return c


FORWARD_CASES = {
    "lin_one": _f("linear", 1, 1, 1, 8, 8),
    "lin_one_f32": _f("linear", 1, 1, 1, 4, 4, "f32", bias=True, act="relu", residual=True),
    "lin_tiny_f32": _f("linear", 256, 8, 2, 64, 128, "f32", bias=True, act="gelu", residual=True),
    "lin_odd": _f("linear", 93, 5, 2, 136, 72, bias=True, act="silu", skew=1.0, empty=0.2),
    "lin_odd_f32": _f("linear", 93, 5, 2, 132, 76, "f32", act="gelu", bias=True, skew=2.0),
    "lin_pair_rows": _f("linear", 50, 4, 3, 40, 264, x_rows="pair", act="relu", bias=True,
                        residual=True, drop=0.3),
    "lin_skew": _f("linear", 700, 3, 1, 72, 40, skew=3.0, act="gelu"),
    "lin_strided": _f("linear", 40, 4, 2, 64, 64, ldx=72, residual=True),
    "lin_pairs_only": _f("linear", 40, 4, 2, 64, 64, bias=True, act="gelu", outs=("Yp", "Z")),
    "lin_none": _f("linear", 30, 4, 2, 64, 64, residual=True, drop=1.0),
    "lin_bad": _f("linear", 40, 6, 2, 64, 64, residual=True, bad=True, bias=True, act="silu"),
    "glu_t1": _f("swiglu", 1, 16, 8, 64, 48),
    "glu_t1_f32": _f("swiglu", 1, 16, 8, 64, 48, "f32", residual=True),
    "glu_t3": _f("swiglu", 3, 16, 4, 136, 72, residual=True),
    "glu_t17": _f("swiglu", 17, 24, 6, 264, 200, residual=True),
    "glu_small": _f("swiglu", 90, 6, 2, 136, 72, residual=True, skew=1.5, empty=0.1),
    "glu_small_f32": _f("swiglu", 90, 6, 2, 68, 36, "f32", residual=True, skew=1.5),
    "glu_mid": _f("swiglu", 600, 5, 2, 200, 264, skew=1.0, drop=0.1),
    "glu_pairs_only": _f("swiglu", 40, 5, 2, 72, 40, outs=("A", "B", "h_sumsq")),
    "glu_y_only": _f("swiglu", 40, 5, 2, 72, 40, outs=("Y",), residual=True),
    "glu_bad": _f("swiglu", 40, 6, 2, 64, 40, bad=True),
    "glu_bad_t1": _f("swiglu", 2, 16, 4, 64, 40, bad=True, residual=True),
    "lin_many": _f("linear", 4500, 7, 2, 16, 24, skew=0.5, drop=0.02, empty=0.05, bad=True),
    "lin_one_block": _f("linear", 4096, 9, 2, 16, 24, skew=0.5, bad=True),
    "lin_512_experts": _f("linear", 700, 512, 3, 16, 24, skew=0.3, bad=True),
    "lin_513_experts": _f("linear", 700, 513, 3, 16, 24, skew=0.3, bad=True),
    "lin_no_tokens": _f("linear", 0, 4, 2, 64, 64, residual=True, bias=True),
    "glu_no_tokens": _f("swiglu", 0, 4, 2, 64, 40, residual=True),
    "lin_twice": _f("linear", 40, 3, 3, 64, 72, twice=True, act="gelu", residual=True),
    "glu_twice": _f("swiglu", 5, 8, 4, 64, 40, twice=True, residual=True),
}


def forward_case(name):
    return build_forward(FORWARD_CASES[name], name)


def build_forward(case, name):
    c = dict(case)
    T, E, dt = c["T"], c["E"], DT[c["dtype"]]
    g = gen("fwd", name)
    c["pairs"] = p = make_pairs(T, E, c["k"], 5 + len(name), c["drop"], c["skew"], c["empty"])
    N = c["N"] = p["token"].size
    if c["twice"]:  # every token names one expert twice
        p["expert"][1::c["k"]] = p["expert"][0::c["k"]]
    if c["bad"] and N > 3:  # experts out of range: absent, reported
        p["expert"][1] = -1
        p["expert"][N // 2] = E
        p["weight"][1] = float("nan")
    rows = T if c["x_rows"] == "token" else N
    ldx = c["ldx"] or c["d_in"]
    c["ldx"] = ldx
    c["X_store"] = normal(g, rows, ldx, dtype=dt)
    c["X"] = c["X_store"][:, :c["d_in"]]
    h, d = c["d_in"], c["d"]
    if c["kind"] == "linear":
        c["W"] = normal(g, E, d, h, std=h ** -0.5, dtype=dt)
        c["bias_t"] = normal(g, E, d, std=0.5, dtype=dt) if c["bias"] else None
        c["d_out"] = d
        full = ("Y", "Yp", "Z")
    else:
        c["W_gate"] = normal(g, E, d, h, std=h ** -0.5, dtype=dt)
        c["W_up"] = normal(g, E, d, h, std=h ** -0.5, dtype=dt)
        c["W_down"] = normal(g, E, h, d, std=d ** -0.5, dtype=dt)
        c["d_out"] = h
        full = ("Y", "Yp", "A", "B", "h_sumsq")
    c["outs"] = c["outs"] or full
    c["R"] = normal(g, T, c["d_out"], dtype=dt) if c["residual"] else None
    return c


def forward_shapes(c):
    """Output name -> (shape, dtype)."""
    N, T, dt = c["N"], c["T"], DT[c["dtype"]]
    s = dict(Y=((T, c["d_out"]), dt), Yp=((N, c["d_out"]), dt), Z=((N, c["d"]), dt),
             A=((N, c["d"]), dt), B=((N, c["d"]), dt), h_sumsq=((N,), torch.float64))
    return {k: s[k] for k in c["outs"]}


def _by_pair(fn, pairs, here, n, cols):
    out = torch.full((n, cols), float("nan"), dtype=torch.float64)
    for p in np.nonzero(here)[0]:
        out[p] = fn(int(p), int(pairs["expert"][p]), int(pairs["token"][p]))
    return out


def judge_forward(c, got, before=None):
    """`got`: the outputs; `before`: what they held (rows of absent pairs stay)."""
    pr, T, E, N = c["pairs"], c["T"], c["E"], c["N"]
    lin = c["kind"] == "linear"
    ref = OF.forward(c["kind"], pr, T, E, c["X"], c["x_rows"], c.get("W"), c.get("bias_t"), c["act"],
                     c.get("W_gate"), c.get("W_up"), c.get("W_down"), c["R"])
    here = OF.present(pr, T, E)
    half = HALF[DT[c["dtype"]]]
    h, d = c["d_in"], c["d"]
    aX = c["X"].double().abs()

    def absdot(W):
        aW = W.double().abs()
        return _by_pair(lambda p, e, t: aW[e] @ aX[t if c["x_rows"] == "token" else p], pr, here, N,
                        W.shape[1])

    tol = {}
    if lin:
        mag = absdot(c["W"])
        if c["bias_t"] is not None:
            mag = mag + c["bias_t"].double().abs()[torch.from_numpy(
                np.clip(pr["expert"], 0, E - 1)).long()]
        tz = (h + 4) * U * mag
        tol["Z"] = tz + half * ref["Z"].abs()
        ty = 1.13 * tz + 16 * U * (1 + ref["Z"].abs())
    else:
        ta, tb = ((h + 4) * U * absdot(c[w]) for w in ("W_gate", "W_up"))
        a, b = ref["A"], ref["B"]
        tol["A"], tol["B"] = ta + half * a.abs(), tb + half * b.abs()
        s = OF.act(a, "silu")
        hv = s * b
        th = 1.13 * ta * (b.abs() + tb) + s.abs() * tb + 16 * U * (1 + a.abs()) * b.abs()
        th = th + half * (hv.abs() + th)
        aD = c["W_down"].double().abs()
        ty = _by_pair(lambda p, e, t: aD[e] @ (th[p] + (d + 4) * U * (hv[p].abs() + th[p])), pr, here,
                      N, c["d_out"])
        tol["h_sumsq"] = (2 * hv.abs() * th + th * th).sum(1) + 4 * d * U * (hv * hv).sum(1)
        ref["h_sumsq"] = (hv * hv).sum(1)
    tol["Yp"] = ty + half * ref["Yp"].abs()
    tY = U * (c["R"].double().abs() if c["R"] is not None else torch.zeros_like(ref["Y"]))
    for p in np.nonzero(here)[0]:
        t, w = int(pr["token"][p]), abs(float(pr["weight"][p]))
        tY[t] += w * (ty[p] + (2.0 ** -16 + (c["k"] + 4) * U) * ref["Yp"][p].abs())
    tol["Y"] = tY + half * (ref["Y"].abs() + tY)
    rows = torch.from_numpy(here)
    for k, v in got.items():
        v = v.cpu()
        if k == "Y":
            close(k, v, ref[k], tol[k])
            continue
        close(k, v[rows], ref[k][rows], tol[k][rows])
        if before is not None and bool((~rows).any()):
            assert torch.equal(v[~rows].view(torch.uint8), before[k][~rows].view(torch.uint8)), \
                f"{k}: a row of an absent pair was written"


# ------------------------------------------------------ epilogue backward
def _g(T, E, k, d, dtype="bf16", **kw):
    c = dict(T=T, E=E, k=k, d=d, dtype=dtype, act="none", dy_rows="token", drop=0.0, skew=0.0,
             empty=0.0, bad=False, outs=("dweight", "G", "dbias"))
    c.update(kw)
    return c


PAIR_GRAD_CASES = {
    "one": _g(1, 1, 1, 8),
    "weights": _g(33, 6, 3, 72, outs=("dweight",)),
    "weights_f32": _g(33, 6, 3, 76, "f32", outs=("dweight",), act="gelu"),
    "no_bias": _g(20, 6, 3, 520, act="silu", outs=("dweight", "G"), bad=True),
    "gelu": _g(90, 5, 2, 136, act="gelu", skew=1.5),
    "gelu_f32": _g(90, 5, 2, 132, "f32", act="gelu", skew=1.5),
    "silu_pair": _g(60, 7, 2, 264, act="silu", dy_rows="pair", drop=0.2),
    "relu": _g(60, 40, 2, 1032, act="relu", empty=0.3),
    "none_wide": _g(24, 3, 2, 1544, bad=True),
    "silu_2048": _g(40, 3, 2, 2048, act="silu", skew=1.0),
    "gelu_over": _g(30, 3, 2, 2184, act="gelu", bad=True),
    "over_f32": _g(12, 2, 1, 4100, "f32", act="relu"),
    "bias_only": _g(50, 4, 2, 72, act="gelu", outs=("dbias",)),
    "none_left": _g(10, 4, 2, 72, act="gelu", drop=1.0),
}


def pair_grad_case(name):
    c = dict(PAIR_GRAD_CASES[name])
    T, E, dt = c["T"], c["E"], DT[c["dtype"]]
    g = gen("pg", name)
    c["pairs"] = p = make_pairs(T, E, c["k"], 11 + len(name), c["drop"], c["skew"], c["empty"])
    N = c["N"] = p["token"].size
    c["Z"] = normal(g, N, c["d"], std=1.5, dtype=dt)
    c["dY"] = normal(g, T if c["dy_rows"] == "token" else N, c["d"], dtype=dt)
    if c["bad"]:
        p["expert"][1] = -1
        p["expert"][N // 2] = E + 3
        p["weight"][1] = float("nan")
        c["Z"][1] = float("nan")
    return c


def pair_grad_shapes(c):
    s = dict(dweight=((c["N"],), torch.float32), G=((c["N"], c["d"]), DT[c["dtype"]]),
             dbias=((c["E"], c["d"]), torch.float32))
    return {k: s[k] for k in c["outs"]}


def judge_pair_grad(c, got):
    pr, T, E, N, d = c["pairs"], c["T"], c["E"], c["N"], c["d"]
    ref = OF.pair_grad(pr, T, E, c["dY"], c["dy_rows"], c["Z"], c["act"])
    here = OF.present(pr, T, E)
    rows = torch.from_numpy(np.clip(pr["token"], 0, T - 1) if c["dy_rows"] == "token"
                            else np.arange(N)).long()
    dy = c["dY"].double().abs()[rows]
    z = torch.nan_to_num(c["Z"].double()).abs()
    y = OF.act(torch.nan_to_num(c["Z"].double()), c["act"]).abs()
    t_el = dy * 16 * U * (1 + z)
    tol = dict(dweight=t_el.sum(1) + (d + 4) * U * (dy * y).sum(1),
               G=t_el + HALF[DT[c["dtype"]]] * ref["G"].abs())
    tb = torch.zeros(E, d, dtype=torch.float64)
    counts = np.bincount(pr["expert"][here], minlength=E)
    for p in np.nonzero(here)[0]:
        e, w = int(pr["expert"][p]), abs(float(pr["weight"][p]))
        tb[e] += w * (t_el[p] + (counts[e] + 4) * U * ref["G"][p].abs())
    tol["dbias"] = tb
    for k, v in got.items():
        close(k, v.cpu(), ref[k], tol[k])
