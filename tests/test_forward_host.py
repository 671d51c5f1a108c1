"""CPU tests of the router and the experts' forward pass: the fp64 oracle is
pinned against hand values, differences and automatic differentiation, and
the C ABI refuses bad arguments before any HIP call."""

import ctypes as C

import numpy as np
import pytest
import torch

import forward_cases as FC
from oracle import forward as OF
from pruned_expert_backward_lrm_amd import lrm as L

lib = L._lib


# ------------------------------------------------------------- oracle pins
def test_route_by_hand():
    z = torch.tensor([[0.0, 2.0, 2.0, -1.0], [float("-inf")] * 4])
    e, w = OF.route(z, 2)
    assert e.tolist() == [1, 2, -1, -1]  # a tie goes to the lower index; an empty row
    assert np.allclose(w, [0.5, 0.5, 0, 0])
    # the bias chooses but does not weigh
    e, w = OF.route(z[:1], 2, score="sigmoid", renorm=False, bias=torch.tensor([0.9, 0, 0, 0.9]))
    assert e.tolist() == [0, 3]
    assert np.allclose(w, [0.5, 1 / (1 + np.e)])
    # groups {0, 1}, {2, 3}: the sum of two against the maximum
    z = torch.tensor([[3.0, -9.0, 2.9, 2.9]])
    assert OF.route(z, 1, n_group=2, topk_group=1, group_rule="max")[0].tolist() == [0]
    assert OF.route(z, 1, n_group=2, topk_group=1, group_rule="top2")[0].tolist() == [2]
    # more slots than eligible experts
    e, w = OF.route(z, 3, expert_mask=torch.tensor([0, 1, 0, 0]))
    assert e.tolist() == [1, -1, -1] and np.allclose(w, [1, 0, 0])


def test_sigmoid_weights_do_not_underflow():
    e, w = OF.route(torch.tensor([[-400.0, -401.0, -900.0]]), 2, score="sigmoid")
    assert np.allclose(w, [1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_is_the_difference_quotient(score, renorm):
    g = FC.gen("fd", score, renorm)
    z = torch.randn(3, 7, generator=g, dtype=torch.float64) * 3
    kw = dict(score=score, renorm=renorm, scale=1.7)
    e, w = OF.route(z, 3, **kw)
    dw = torch.randn(9, generator=g, dtype=torch.float64)
    grad = OF.route_bwd(z, 3, e, dw, **kw)
    step = 1e-5
    for t in range(3):
        for c in range(7):
            lo, hi = z.clone(), z.clone()
            lo[t, c] -= step
            hi[t, c] += step
            (e0, w0), (e1, w1) = OF.route(lo, 3, **kw), OF.route(hi, 3, **kw)
            assert np.array_equal(e0, e) and np.array_equal(e1, e)
            fd = float(((w1 - w0) * dw.numpy()).sum() / (2 * step))
            assert abs(fd - float(grad[t, c])) < 1e-8


def test_pair_grad_is_the_difference_quotient():
    pr = FC.make_pairs(4, 3, 2, 1)
    g = FC.gen("fdp")
    Z, dY = torch.randn(8, 3, generator=g).double(), torch.randn(4, 3, generator=g).double()
    for name in ("gelu", "silu", "relu", "none"):
        got = OF.pair_grad(pr, 4, 3, dY, "token", Z, name)

        def loss(zz, ww):
            return sum(float(ww[p]) * float((dY[int(pr["token"][p])] * OF.act(zz[p], name)).sum())
                       for p in range(8))

        for p in range(8):
            for c in range(3):
                lo, hi = Z.clone(), Z.clone()
                lo[p, c] -= 1e-6
                hi[p, c] += 1e-6
                fd = (loss(hi, pr["weight"]) - loss(lo, pr["weight"])) / 2e-6
                assert abs(fd - float(pr["weight"][p]) * float(got["G"][p, c])) < 1e-7
            w = pr["weight"].astype(np.float64)
            w1 = w.copy()
            w1[p] += 1e-3
            assert abs((loss(Z, w1) - loss(Z, w)) / 1e-3 - float(got["dweight"][p])) < 1e-9
        for e in range(3):
            ref = sum(float(pr["weight"][p]) * got["G"][p] for p in range(8) if pr["expert"][p] == e)
            assert torch.allclose(got["dbias"][e], torch.as_tensor(ref, dtype=torch.float64)
                                  .expand(3) if isinstance(ref, int) else ref)


def test_gelu_is_exact():
    x = torch.linspace(-6, 6, 101, dtype=torch.float64)
    assert torch.allclose(OF.act(x, "gelu"), torch.nn.functional.gelu(x), atol=1e-15)


def test_swiglu_forward_matches_dense_algebra():
    c = FC.forward_case("glu_small_f32")
    pr = c["pairs"]
    out = OF.forward("swiglu", pr, c["T"], c["E"], c["X"], W_gate=c["W_gate"], W_up=c["W_up"],
                     W_down=c["W_down"], residual=c["R"])
    X = c["X"].double()
    Y = c["R"].double().clone()
    for e in range(c["E"]):
        h = torch.nn.functional.silu(X @ c["W_gate"][e].double().T) * (X @ c["W_up"][e].double().T)
        y = h @ c["W_down"][e].double().T
        wt = torch.zeros(c["T"], dtype=torch.float64)
        for t, ex, w in zip(pr["token"], pr["expert"], pr["weight"]):
            if ex == e:
                wt[int(t)] += float(w)
        Y += wt[:, None] * y
    assert torch.allclose(out["Y"], Y, atol=1e-12)


# ---------------------------------------------------------------- refusals
P = 0x1000  # an aligned address; nothing is launched


def router(**kw):
    v = dict(T=4, E=8, k=2, score=0, flags=0, n_group=1, topk_group=1, group_rule=0, scale=1.0,
             dtype=L.LRM_BF16, logits=P, ld=8, bias=None, expert_mask=None, token_mask=None)
    v.update(kw)
    return L.lrm_router(*v.values())


ROUTER_REFUSALS = [
    (dict(T=-1), 2), (dict(E=0), 2), (dict(E=4097, ld=4097), 2), (dict(k=0), 2), (dict(k=9), 2),
    (dict(E=100, ld=100, k=65), 2), (dict(T=1 << 30, k=2), 2), (dict(n_group=0), 2),
    (dict(n_group=3), 2), (dict(n_group=128, E=128, ld=128), 2), (dict(topk_group=0), 2),
    (dict(topk_group=2), 2), (dict(ld=7), 2), (dict(dtype=5), 3), (dict(score=2), 10),
    (dict(group_rule=2), 10), (dict(flags=2), 10), (dict(scale=float("nan")), 10),
    (dict(scale=float("inf")), 10), (dict(logits=None), 1), (dict(logits=P + 1), 5),
    (dict(dtype=L.LRM_F32, logits=P + 2), 5), (dict(bias=P + 2), 5),
]


@pytest.mark.parametrize("kw,status", ROUTER_REFUSALS)
def test_route_refusals(kw, status):
    r = router(**kw)
    assert lib.lrm_route(C.byref(r), P, P, None, None, None, 0, None) == status
    assert lib.lrm_route_bwd(C.byref(r), P, P, P, 5000, None) == status
    assert lib.lrm_route_workspace_size(C.byref(r)) == 0


def test_route_argument_refusals():
    r = router()
    assert lib.lrm_route(None, P, P, None, None, None, 0, None) == 1
    assert lib.lrm_route(C.byref(r), None, P, None, None, None, 0, None) == 1
    assert lib.lrm_route(C.byref(r), P, None, None, None, None, 0, None) == 1
    assert lib.lrm_route(C.byref(r), P + 2, P, None, None, None, 0, None) == 5
    need = lib.lrm_route_workspace_size(C.byref(r))
    assert need > 0
    assert lib.lrm_route(C.byref(r), P, P, None, P, None, 0, None) == 7
    assert lib.lrm_route(C.byref(r), P, P, None, P, P, need - 1, None) == 7
    assert lib.lrm_route_bwd(C.byref(r), None, P, P, 8, None) == 1
    assert lib.lrm_route_bwd(C.byref(r), P, None, P, 8, None) == 1
    assert lib.lrm_route_bwd(C.byref(r), P, P, None, 8, None) == 1
    assert lib.lrm_route_bwd(C.byref(r), P, P, P, 7, None) == 2
    assert lib.lrm_route_bwd(C.byref(r), P, P, P + 1, 8, None) == 5


def test_share_refusals():
    need = lib.lrm_route_share_workspace_size(4, 2)
    assert need > 0 and lib.lrm_route_share_workspace_size(-1, 2) == 0

    def share(T=4, k=2, e=P, w=P, e0=0, E=8, oe=P, ow=P, n=P, ws=P, size=need):
        return lib.lrm_route_share(T, k, e, w, e0, E, None, oe, ow, None, n, ws, size, None)

    assert share(T=-1) == 2 and share(k=0) == 2 and share(T=1 << 30, k=4) == 2
    assert share(e0=-1) == 2 and share(E=0) == 2 and share(E=4097) == 2
    assert share(e=None) == 1 and share(w=None) == 1 and share(oe=None) == 1
    assert share(ow=None) == 1 and share(n=None) == 1
    assert share(ws=None) == 7 and share(size=need - 1) == 7
    assert share(e=P + 2) == 5 and share(n=P + 2) == 5


def pairs(T=4, N=8, E=2, ptr=P):
    return L.lrm_pairs(T, N, E, 0, ptr, ptr, ptr)


def m(ptr=P, dtype=L.LRM_BF16, rows=0, cols=64, ld=None):
    return L.lrm_mat(ptr, dtype, rows, cols, 0, ld or cols)


def fwd(which="linear", **kw):
    f = L.lrm_forward()
    f.dtype, f.pairs, f.X, f.R = L.LRM_BF16, pairs(), m(), m(None)
    if which == "linear":
        f.W, f.w_stride, f.d_in, f.d_out = P, 64 * 32, 64, 32
    else:
        f.kind = 1
        f.W_gate = f.W_up = f.W_down = P
        f.H, f.I = 64, 32
    for k, v in kw.items():
        setattr(f, k, v)
    return f


def fout(**kw):
    return L.lrm_forward_outputs(**(kw or dict(Y=P)))


FORWARD_REFUSALS = [
    ("linear", dict(kind=7), 10), ("linear", dict(act=4), 10), ("linear", dict(act=-1), 10),
    ("linear", dict(dtype=9), 3), ("linear", dict(pairs=pairs(E=0)), 2),
    ("linear", dict(pairs=pairs(ptr=None)), 1), ("linear", dict(d_in=0), 2),
    ("linear", dict(d_out=1 << 20), 2), ("linear", dict(d_out=36), 10), ("linear", dict(W=None), 1),
    ("linear", dict(W=P + 8), 5), ("linear", dict(bias=P + 8), 5),
    ("linear", dict(w_stride=64 * 32 - 8), 2), ("linear", dict(w_stride=64 * 32 + 4), 5),
    ("linear", dict(X=m(cols=72)), 2), ("linear", dict(X=m(dtype=L.LRM_F32)), 3),
    ("linear", dict(X=m(rows=3)), 4), ("linear", dict(X=m(ptr=P + 8)), 5),
    ("linear", dict(X=m(ld=60)), 2), ("linear", dict(X=m(ld=68)), 5), ("linear", dict(R=m()), 2),
    ("linear", dict(R=m(cols=32, rows=1)), 4),
    ("swiglu", dict(act=3), 10), ("swiglu", dict(bias=P), 10), ("swiglu", dict(X=m(rows=1)), 4),
    ("swiglu", dict(I=36), 10), ("swiglu", dict(H=0), 2), ("swiglu", dict(W_up=None), 1),
    ("swiglu", dict(W_down=P + 8), 5), ("swiglu", dict(R=m(cols=32)), 2),
]


@pytest.mark.parametrize("kind,kw,status", FORWARD_REFUSALS)
def test_forward_refusals(kind, kw, status):
    f = fwd(kind, **kw)
    assert lib.lrm_expert_forward(C.byref(f), C.byref(fout()), P, 1 << 40, None) == status
    assert lib.lrm_forward_workspace_size(C.byref(f)) == 0


def test_forward_output_refusals():
    f, s = fwd(), fwd("swiglu")
    ok = C.byref(f)
    assert lib.lrm_expert_forward(None, C.byref(fout()), P, 1 << 40, None) == 1
    assert lib.lrm_expert_forward(ok, None, P, 1 << 40, None) == 1
    assert lib.lrm_expert_forward(ok, C.byref(fout(Y=None)), P, 1 << 40, None) == 1
    assert lib.lrm_expert_forward(ok, C.byref(fout(Y=P + 8)), P, 1 << 40, None) == 5
    assert lib.lrm_expert_forward(ok, C.byref(fout(Y=P, A=P)), P, 1 << 40, None) == 10
    assert lib.lrm_expert_forward(C.byref(s), C.byref(fout(Z=P)), P, 1 << 40, None) == 10
    assert lib.lrm_expert_forward(C.byref(s), C.byref(fout(h_sumsq=P + 4)), P, 1 << 40, None) == 5
    r = fwd(R=m(cols=32))  # a residual without the output that it joins
    assert lib.lrm_expert_forward(C.byref(r), C.byref(fout(Yp=P)), P, 1 << 40, None) == 10
    need = lib.lrm_forward_workspace_size(ok)
    assert need > 0
    assert lib.lrm_expert_forward(ok, C.byref(fout()), None, need, None) == 7
    assert lib.lrm_expert_forward(ok, C.byref(fout()), P, need - 1, None) == 7
    assert lib.lrm_expert_forward(ok, C.byref(fout()), P + 64, need, None) == 5


def test_pair_grad_refusals():
    def problem(act=0, dtype=L.LRM_BF16, pr=None, dY=None, Z=None):
        return L.lrm_pair_grad_problem(act, dtype, pr or pairs(), dY or m(), Z or m(rows=1))

    def run(g, ws=P, size=1 << 40, **outs):
        o = L.lrm_pair_grad_outputs(**(outs or dict(dweight=P)))
        return lib.lrm_pair_grad(C.byref(g) if g else None, C.byref(o), ws, size, None)

    assert run(None) == 1
    assert run(problem(act=4)) == 10 and run(problem(dtype=3)) == 3
    assert run(problem(pr=pairs(E=0))) == 2 and run(problem(Z=m())) == 4
    assert run(problem(dY=m(cols=72))) == 2 and run(problem(dY=m(rows=4))) == 4
    assert run(problem(dY=m(ptr=P + 8))) == 5 and run(problem(Z=m(rows=1, cols=1 << 20))) == 2
    assert run(problem(), dweight=None) == 1
    assert run(problem(), dweight=P + 2) == 5 and run(problem(), G=P + 8) == 5
    g = problem()
    need = lib.lrm_pair_grad_workspace_size(C.byref(g))
    assert need > 0
    assert run(g, ws=None) == 7 and run(g, size=need - 1) == 7 and run(g, ws=P + 64) == 5


def test_struct_layouts():
    assert C.sizeof(L.lrm_router) == 80
    assert C.sizeof(L.lrm_forward) == 16 + 40 + 64 + 32 + 24 + 8
    assert C.sizeof(L.lrm_forward_outputs) == 48
    assert C.sizeof(L.lrm_pair_grad_problem) == 8 + 40 + 64
    assert C.sizeof(L.lrm_pair_grad_outputs) == 24


def test_binding_refuses_bad_tensors():
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        L.Router(z.t(), 2)
    with pytest.raises(ValueError):
        L.Router(z, 2, bias=torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        L.Router(z, 2, token_mask=torch.zeros(5, dtype=torch.uint8))
    with pytest.raises(TypeError):
        L.Router(z.half(), 2)
    r = L.Router(z, 2)
    i, f = torch.zeros(8, dtype=torch.int32), torch.zeros(8)
    for e, w, kw in ((i[:7], f, {}), (i.long(), f, {}), (i, f.double(), {}),
                     (i, f, dict(counts=i[:7])), (i, f, dict(token=f))):
        with pytest.raises(ValueError):
            L.lrm_route(r, e, w, stream=None, **kw)
    with pytest.raises(ValueError):
        L.lrm_route_bwd(r, i, f, torch.zeros(4, 7))
    with pytest.raises(ValueError):
        L.lrm_route_bwd(r, i, f, torch.zeros(4, 8, dtype=torch.bfloat16))
    pr = L.Pairs(i, i, f, 4, 2)
    with pytest.raises(ValueError):
        L.linear_forward(pr, z, "token", torch.zeros(3, 8, 8))
    with pytest.raises(ValueError):
        L.linear_forward(pr, z, "token", torch.zeros(2, 8, 8), bias=torch.zeros(2, 7))
    with pytest.raises(ValueError):
        L.swiglu_forward(pr, z, torch.zeros(2, 4, 8), torch.zeros(2, 4, 8), torch.zeros(2, 4, 8))


def test_binding_refuses_outputs_that_do_not_fit():
    i, f = torch.zeros(8, dtype=torch.int32), torch.zeros(8)
    pr = L.Pairs(i, i, f, 4, 2)
    X, W = torch.zeros(4, 8), torch.zeros(2, 12, 8)
    with pytest.raises(ValueError):
        L.linear_forward(pr, X[:3], "token", W)
    with pytest.raises(ValueError):
        L.linear_forward(pr, X, "pair", W)
    with pytest.raises(ValueError):
        L.linear_forward(pr, X, "token", W, residual=torch.zeros(3, 12))
    with pytest.raises(ValueError):
        L.linear_forward(pr, X, "token", W.to("meta"))
    lin = L.linear_forward(pr, X, "token", W)
    for out in (dict(Y=torch.zeros(4, 11)), dict(Yp=torch.zeros(7, 12)),
                dict(Y=torch.zeros(4, 12, dtype=torch.bfloat16)),
                dict(Y=torch.zeros(4, 12), Z=torch.zeros(9, 12)),
                dict(Y=torch.zeros(4, 12, device="meta"))):
        with pytest.raises(ValueError):
            L.lrm_expert_forward(lin, out)
        with pytest.raises(ValueError):  # marshalled before
            L.lrm_expert_forward(lin, L.forward_outputs(out))
    glu = L.swiglu_forward(pr, X, torch.zeros(2, 4, 8), torch.zeros(2, 4, 8), torch.zeros(2, 8, 4))
    for out in (dict(Y=torch.zeros(4, 4)), dict(A=torch.zeros(8, 8)), dict(h_sumsq=torch.zeros(8))):
        with pytest.raises(ValueError):
            L.lrm_expert_forward(glu, out)
    with pytest.raises(ValueError):
        L.pair_grad_problem(pr, X, "token", torch.zeros(7, 8))
    with pytest.raises(ValueError):
        L.pair_grad_problem(pr, X, "pair", torch.zeros(8, 8))
    pg = L.pair_grad_problem(pr, X, "token", torch.zeros(8, 8))
    for out in (dict(dweight=torch.zeros(7)), dict(G=torch.zeros(8, 4)), dict(dbias=torch.zeros(3, 8)),
                dict(dweight=torch.zeros(8, dtype=torch.float64))):
        with pytest.raises(ValueError):
            L.lrm_pair_grad(pg, out)
    r = L.Router(X, 2)
    with pytest.raises(ValueError):
        L.lrm_route(r, i.to("meta"), f)
    with pytest.raises(ValueError):
        L.lrm_route_bwd(r, i, f, torch.zeros(4, 8, device="meta"))
