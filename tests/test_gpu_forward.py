"""GPU parity of the router, the experts' forward pass and its epilogue's
backward pass against the fp64 oracle, through the Python binding of the
C ABI; and the calls together, as a training step makes them."""

import numpy as np
import pytest
import torch

import forward_cases as FC
from oracle import forward as OF

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pruned_expert_backward_lrm_amd import lrm
    return lrm


def dev(t):
    return None if t is None else t.to(DEV)


def filled(shape, dt):
    """A device output that holds bytes 0xCD."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dt).element_size()
    raw = torch.full((n,), 0xCD, dtype=torch.uint8, device=DEV)
    return raw.view(dt).reshape(shape) if n else torch.empty(shape, dtype=dt, device=DEV)


# ------------------------------------------------------------------ router
def make_router(L, c):
    T, E, ld = c["T"], c["E"], c["ld"]
    store = torch.zeros(T, ld, dtype=c["logits"].dtype, device=DEV)
    store[:, :E] = dev(c["logits"])
    kw = FC.route_kw(c)
    for k in ("bias", "expert_mask", "token_mask"):
        kw[k] = dev(kw[k])
    return L.Router(store[:, :E], c["k"], **kw)


@pytest.mark.parametrize("name", list(FC.ROUTE_CASES))
def test_route(L, name):
    c = FC.route_case(name)
    n = c["T"] * c["k"]
    r = make_router(L, c)
    out = dict(expert=filled((n,), torch.int32), weight=filled((n,), torch.float32),
               token=filled((n,), torch.int32), counts=filled((c["E"],), torch.int32))
    L.lrm_route(r, **out)
    torch.cuda.synchronize()
    FC.judge_route(c, *(out[k].cpu() for k in ("expert", "weight", "token", "counts")))
    # without the optional outputs, on another stream
    s = torch.cuda.Stream()
    e2, w2 = filled((n,), torch.int32), filled((n,), torch.float32)
    s.wait_stream(torch.cuda.current_stream())
    L.lrm_route(r, e2, w2, stream=s)
    s.synchronize()
    assert torch.equal(e2, out["expert"]) and torch.equal(w2, out["weight"])


@pytest.mark.parametrize("name", list(FC.ROUTE_CASES))
def test_route_bwd(L, name):
    c = FC.route_case(name)
    e, dw = FC.route_grad_inputs(c, name)
    r = make_router(L, c)
    T, E = c["T"], c["E"]
    gap = 3 if name in ("odd", "strided") else 0
    store = filled((T, E + gap), c["logits"].dtype)
    L.lrm_route_bwd(r, dev(e), dev(dw), store[:, :E])
    torch.cuda.synchronize()
    FC.judge_route_bwd(c, e, dw, store[:, :E].cpu())
    assert (store[:, E:].contiguous().view(torch.uint8) == 0xCD).all()


def test_route_many_tokens_against_sorting(L):
    """Many rows (several per block) against a stable sort of the exact keys."""
    T, E, k = 70001, 128, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn(T, E, generator=g, device=DEV).to(torch.bfloat16)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    for kw, key in ((dict(), z.double()),
                    (dict(score="sigmoid", bias=bias), torch.sigmoid(z.double()) + bias.double())):
        r = L.Router(z, k, **kw)
        e = filled((T * k,), torch.int32)
        w = filled((T * k,), torch.float32)
        cnt = filled((E,), torch.int32)
        L.lrm_route(r, e, w, counts=cnt)
        want = key.sort(dim=1, descending=True, stable=True).indices[:, :k].int().reshape(-1)
        assert torch.equal(e, want)
        assert torch.equal(cnt, torch.bincount(want.long(), minlength=E).int())
        assert torch.allclose(w.view(T, k).sum(1), torch.ones(T, device=DEV), atol=2e-6)


def test_route_no_tokens(L):
    r = L.Router(torch.empty(0, 16, device=DEV), 2)
    z = torch.empty(0, dtype=torch.int32, device=DEV)
    cnt = filled((16,), torch.int32)
    L.lrm_route(r, z, z.float(), counts=cnt)
    L.lrm_route_bwd(r, z, z.float(), torch.empty(0, 16, device=DEV))
    torch.cuda.synchronize()
    assert not cnt.any()


def test_route_bwd_same_expert_twice(L):
    """A choice that names an expert twice: its slots' gradients add up."""
    z = FC.normal(FC.gen("twice"), 3, 20)
    e = torch.tensor([4, 4, 7, 0, 19, 19, 19, 3, 25], dtype=torch.int32)
    dw = FC.normal(FC.gen("twice_dw"), 9)
    for kw in (dict(score="sigmoid", renorm=False), dict(renorm=False)):
        got = filled((3, 20), torch.float32)
        L.lrm_route_bwd(L.Router(dev(z), 3, **kw), dev(e), dev(dw), got)
        ref = OF.route_bwd(z, 3, e.numpy(), dw, **kw)
        FC.close("dlogits", got.cpu(), ref, torch.full_like(ref, 2e-6 * float(dw.abs().max())))


@pytest.mark.parametrize("T,k,e0,E", [(1, 1, 0, 1), (300, 3, 4, 5), (3001, 2, 2, 3), (50, 4, 90, 8),
                                      (0, 4, 0, 8), (300007, 8, 3, 4)])
def test_share(L, T, k, e0, E):
    rng = np.random.default_rng(T)
    n = T * k
    ex, w = rng.integers(-1, 12, n).astype(np.int32), rng.random(n).astype(np.float32)
    i32, f32 = torch.int32, torch.float32
    ot, oe, os_ = (filled((n,), i32) for _ in range(3))
    ow, on = filled((n,), f32), filled((1,), i32)
    L.lrm_route_share(T, k, dev(torch.from_numpy(ex)), dev(torch.from_numpy(w)), e0, E, ot, oe, ow, on,
                      out_slot=os_)
    torch.cuda.synchronize()
    t, e, wr, s = OF.route_share(k, ex, w, e0, E)
    assert int(on) == s.size
    for got, ref in ((ot, t), (oe, e), (ow, wr), (os_, s)):
        assert np.array_equal(got[:s.size].cpu().numpy(), ref)
        assert (got[s.size:].contiguous().view(torch.uint8) == 0xCD).all()


# ---------------------------------------------------------- experts forward
def gpu_pairs(L, c):
    p = c["pairs"]
    return L.Pairs(*(dev(torch.from_numpy(p[k])) for k in ("token", "expert", "weight")), c["T"],
                   c["E"])


def make_forward(L, c):
    pairs = gpu_pairs(L, c)
    X = dev(c["X_store"])[:, :c["d_in"]]
    if c["kind"] == "linear":
        return L.linear_forward(pairs, X, c["x_rows"], dev(c["W"]), act=c["act"],
                                bias=dev(c["bias_t"]), residual=dev(c["R"]))
    return L.swiglu_forward(pairs, X, dev(c["W_gate"]), dev(c["W_up"]), dev(c["W_down"]),
                            residual=dev(c["R"]))


def run_forward(L, c, stream=None):
    f = make_forward(L, c)
    out = {k: filled(*v) for k, v in FC.forward_shapes(c).items()}
    before = {k: v.cpu().clone() for k, v in out.items()}
    ws = torch.full((max(L.lrm_forward_workspace_size(f), 1),), 0xCD, dtype=torch.uint8, device=DEV)
    L.lrm_expert_forward(f, out, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert L.lrm_check_device_errors(ws) == (L.LRM_ERR_INDEX if c["bad"] else L.LRM_OK)
    return out, before


@pytest.mark.parametrize("name", list(FC.FORWARD_CASES))
def test_forward(L, name):
    c = FC.forward_case(name)
    out, before = run_forward(L, c)
    FC.judge_forward(c, out, before)
    again, _ = run_forward(L, c)
    for k in out:  # bit for bit, whatever the workspace held
        assert torch.equal(out[k].view(torch.uint8), again[k].view(torch.uint8)), k


@pytest.mark.parametrize("tile", ["64", "128", "256"])
@pytest.mark.parametrize("name", ["lin_one", "lin_tiny_f32", "lin_odd", "lin_odd_f32", "lin_skew",
                                  "lin_bad", "glu_t17", "glu_small", "glu_small_f32", "glu_mid"])
def test_forward_tiles(L, monkeypatch, name, tile):
    """Every row tile of the products on every kind of case."""
    monkeypatch.setenv("LRM_FWD_TILE", tile)
    c = FC.forward_case(name)
    out, before = run_forward(L, c)
    FC.judge_forward(c, out, before)


def test_forward_input_past_2_gib(L):
    """X of more than 2 GiB: byte offsets of its last rows pass 31 bits."""
    T, H, d, k = 540_000, 2048, 64, 1
    rng = np.random.default_rng(1)
    rows = np.unique(np.concatenate([[0, 1, T - 1], rng.integers(0, T, 90)])).astype(np.int32)
    N = rows.size
    c = dict(kind="linear", T=T, E=2, k=k, d_in=H, d=d, dtype="bf16", act="none", x_rows="token",
             N=N, bias_t=None, R=None, d_out=d, bad=False, outs=("Yp",))
    c["pairs"] = dict(token=rows, expert=rng.integers(0, 2, N).astype(np.int32),
                      weight=np.ones(N, np.float32))
    g = FC.gen("big")
    c["W"] = FC.normal(g, 2, d, H, std=0.02, dtype=torch.bfloat16)
    small = FC.normal(g, N, H, dtype=torch.bfloat16)
    X = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)  # rows no pair reads
    X[dev(torch.from_numpy(rows)).long()] = dev(small)
    f = L.linear_forward(gpu_pairs(L, c), X, "token", dev(c["W"]))
    out = dict(Yp=filled((N, d), torch.bfloat16))
    L.lrm_expert_forward(f, out)
    torch.cuda.synchronize()
    # the same pairs over the rows alone
    c["pairs"] = dict(c["pairs"], token=np.arange(N, dtype=np.int32))
    c.update(T=N, X=small)
    FC.judge_forward(c, out)


def test_forward_in_place_residual(L):
    c = FC.forward_case("glu_small")
    f = make_forward(L, c)
    Y = dev(c["R"]).clone()
    f2 = L.swiglu_forward(f.pairs, f.keep[1], dev(c["W_gate"]), dev(c["W_up"]), dev(c["W_down"]),
                          residual=Y)
    L.lrm_expert_forward(f2, dict(Y=Y))
    torch.cuda.synchronize()
    FC.judge_forward(c, dict(Y=Y))


def test_forward_graph_replays(L):
    """One captured call replayed over new inputs equals the eager call."""
    for name in ("glu_small", "glu_t1", "lin_odd"):
        c = FC.forward_case(name)
        f = make_forward(L, c)
        out = {k: filled(*v) for k, v in FC.forward_shapes(c).items()}
        ws = torch.empty(L.lrm_forward_workspace_size(f), dtype=torch.uint8, device=DEV)
        marshalled = L.forward_outputs(out)
        L.lrm_expert_forward(f, marshalled, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lrm_expert_forward(f, marshalled, ws=ws)
        X = f.keep[1]
        for step in range(3):
            X.copy_(FC.normal(FC.gen("replay", name, step), *X.shape).to(X.dtype))
            graph.replay()
            torch.cuda.synchronize()
            got = {k: v.clone() for k, v in out.items()}
            L.lrm_expert_forward(f, marshalled, ws=ws)
            torch.cuda.synchronize()
            for k in out:
                assert torch.equal(got[k].view(torch.uint8), out[k].view(torch.uint8)), (name, k)


@pytest.mark.parametrize("name", ["lin_none", "lin_no_tokens", "glu_no_tokens", "lin_twice",
                                  "glu_twice"])
def test_forward_tiles_of_little(L, monkeypatch, name):
    monkeypatch.setenv("LRM_FWD_TILE", "64")
    c = FC.forward_case(name)
    out, before = run_forward(L, c)
    FC.judge_forward(c, out, before)


@pytest.mark.parametrize("name", list(FC.PAIR_GRAD_CASES))
def test_pair_grad(L, name):
    c = FC.pair_grad_case(name)
    g = L.pair_grad_problem(gpu_pairs(L, c), dev(c["dY"]), c["dy_rows"], dev(c["Z"]), act=c["act"])
    out = {k: filled(*v) for k, v in FC.pair_grad_shapes(c).items()}
    ws = torch.full((L.lrm_pair_grad_workspace_size(g),), 0xCD, dtype=torch.uint8, device=DEV)
    L.lrm_pair_grad(g, out, ws=ws)
    torch.cuda.synchronize()
    bad = c["bad"] and "dbias" in out
    assert L.lrm_check_device_errors(ws) == (L.LRM_ERR_INDEX if bad else L.LRM_OK)
    FC.judge_pair_grad(c, out)


# ----------------------------------------------------------------- together
def test_training_step_together(L):
    """Router, forward, and both backward passes of one layer call: the loss
    <Y, V> of the whole chain, differentiated, equals the calls' gradients."""
    T, E, k, H, I = 96, 8, 2, 64, 48  # noqa: E741
    g = FC.gen("together")
    X, V = FC.normal(g, T, H), FC.normal(g, T, H)
    z = FC.normal(g, T, E)
    Wg, Wu = FC.normal(g, E, I, H, std=H ** -0.5), FC.normal(g, E, I, H, std=H ** -0.5)
    Wd = FC.normal(g, E, H, I, std=I ** -0.5)
    n = T * k
    i32, f32 = torch.int32, torch.float32
    expert, token, weight = filled((n,), i32), filled((n,), i32), filled((n,), f32)
    counts, quota = filled((E,), i32), filled((E,), i32)
    r = L.Router(dev(z), k, score="sigmoid", scale=1.5)
    L.lrm_route(r, expert, weight, token=token, counts=counts)
    pairs = L.Pairs(token, expert, weight, T, E)
    L.lrm_quota_waterfill_device(pairs, n, quota, counts=counts)  # a budget that keeps all
    Xd, dY = dev(X), dev(V)
    W = [dev(w) for w in (Wg, Wu, Wd)]
    out = dict(Y=filled((T, H), f32), Yp=filled((n, H), f32), A=filled((n, I), f32),
               B=filled((n, I), f32), h_sumsq=filled((n,), torch.float64))
    L.lrm_expert_forward(L.swiglu_forward(pairs, Xd, *W, residual=Xd), out)
    dweight = filled((n,), f32)
    L.lrm_pair_grad(L.pair_grad_problem(pairs, dY, "token", out["Yp"]), dict(dweight=dweight))
    dz = filled((T, E), f32)
    L.lrm_route_bwd(r, expert, dweight, dz)
    pb = L.swiglu_problem(pairs, Xd, "token", dY, "token", out["A"], out["B"], *W, quota, quota, quota,
                          flags=L.LRM_QUOTA_ON_DEVICE, h_sumsq=out["h_sumsq"])
    back = dict(dW_gate=filled((E, I, H), f32), dW_up=filled((E, I, H), f32),
                dW_down=filled((E, H, I), f32), dX=filled((T, H), f32))
    ws = L.lrm_expert_backward(pb, back)
    torch.cuda.synchronize()
    assert L.lrm_check_device_errors(ws) == L.LRM_OK
    # the same chain by automatic differentiation in 64 bits
    leaves = [t.double().requires_grad_(True) for t in (z, X, Wg, Wu, Wd)]
    zz, xx, wg, wu, wd = leaves
    e = expert.cpu().long().view(T, k)
    s = torch.sigmoid(zz).gather(1, e)
    w = 1.5 * s / s.sum(1, keepdim=True)
    Y = xx.clone()
    for j in range(k):
        ej = e[:, j]
        a, b = torch.einsum("th,tih->ti", xx, wg[ej]), torch.einsum("th,tih->ti", xx, wu[ej])
        y = torch.einsum("ti,thi->th", torch.nn.functional.silu(a) * b, wd[ej])
        Y = Y + w[:, j:j + 1] * y
    (Y * V.double()).sum().backward()
    # the residual's own gradient is V and is not the layer's to return
    want = dict(dz=zz.grad, dX=xx.grad - V.double(), dW_gate=wg.grad, dW_up=wu.grad, dW_down=wd.grad)
    got = dict(back, dz=dz)
    for name, ref in want.items():
        err = float((got[name].cpu().double() - ref).norm() / ref.norm())
        assert err < 1e-5, (name, err)
    assert float((out["Y"].cpu().double() - Y.detach()).norm() / Y.detach().norm()) < 1e-6


def test_share_of_a_padded_batch_together(L):
    """A padded batch routed over all experts; one GPU's share of the pairs goes
    through the forward pass; the gradient of the weights returns by slot."""
    T, E, k, H, d = 200, 16, 4, 64, 72
    g = FC.gen("share")
    z = FC.normal(g, T, E)
    keep = (torch.arange(T) % 7 != 3).to(torch.uint8)
    z[keep == 0] = float("nan")
    e0, El, n = 4, 6, T * k
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    expert, weight = filled((n,), i32), filled((n,), f32)
    r = L.Router(dev(z), k, token_mask=dev(keep))
    L.lrm_route(r, expert, weight)
    tok, ex, slot = (filled((n,), i32) for _ in range(3))
    wt, cnt = filled((n,), f32), filled((1,), i32)
    L.lrm_route_share(T, k, expert, weight, e0, El, tok, ex, wt, cnt, out_slot=slot)
    N = int(cnt)
    pairs = L.Pairs(tok[:N], ex[:N], wt[:N], T, El)
    X, W, dY = FC.normal(g, T, H, dtype=bf), FC.normal(g, El, d, H, std=0.1, dtype=bf), \
        FC.normal(g, T, d, dtype=bf)
    out = dict(Y=filled((T, d), bf), Z=filled((N, d), bf))
    ws = L.lrm_expert_forward(L.linear_forward(pairs, dev(X), "token", dev(W), act="silu"), out)
    assert L.lrm_check_device_errors(ws) == L.LRM_OK
    dw = filled((N,), f32)
    L.lrm_pair_grad(L.pair_grad_problem(pairs, dev(dY), "token", out["Z"], act="silu"),
                    dict(dweight=dw))
    dslot = torch.zeros(n, device=DEV)
    dslot[slot[:N].long()] = dw
    dz = filled((T, E), f32)
    L.lrm_route_bwd(r, expert, dslot, dz)
    torch.cuda.synchronize()
    we, ww = OF.route(z, k, token_mask=keep)
    assert np.array_equal(expert.cpu().numpy(), we)
    t2, e2, w2, s2 = OF.route_share(k, we, ww, e0, El)
    c = dict(kind="linear", T=T, E=El, k=k, d_in=H, d=d, dtype="bf16", act="silu", x_rows="token",
             pairs=dict(token=t2, expert=e2, weight=weight.cpu().numpy()[s2]), N=N, X=X, W=W,
             bias_t=None, R=None, d_out=d)
    FC.judge_forward(c, out)
    assert not out["Y"][dev(keep) == 0].any()  # padding gets nothing
    zr = OF.act(out["Z"].cpu().double(), "silu")
    ref_dw = (zr * dY.double()[torch.from_numpy(t2)]).sum(1)
    assert float((dw.cpu().double() - ref_dw).norm() / ref_dw.norm()) < 1e-5
    dref = torch.zeros(n, dtype=torch.float64)
    dref[torch.from_numpy(s2)] = ref_dw
    ref = OF.route_bwd(z, k, we, dref, token_mask=keep)
    assert float((dz.cpu().double() - ref).norm() / ref.norm()) < 1e-5


def _bits(out):
    return {k: v.clone().view(torch.uint8) for k, v in out.items()}


def test_calls_of_a_layer_in_one_graph(L):
    """Route, share, forward, both epilogue gradients and the routing gradient,
    captured in one graph over one workspace: every replay, with the program's
    own eager calls in the same workspace between, equals the eager calls."""
    T, E, k, H, d = 130, 12, 3, 64, 72
    g = FC.gen("graph")
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    n = T * k
    z, X, dY = dev(FC.normal(g, T, E)), dev(FC.normal(g, T, H, dtype=bf)), \
        dev(FC.normal(g, T, d, dtype=bf))
    W, bias = dev(FC.normal(g, E, d, H, std=0.1, dtype=bf)), dev(FC.normal(g, E, d, dtype=bf))
    out = dict(expert=filled((n,), i32), weight=filled((n,), f32), token=filled((n,), i32),
               counts=filled((E,), i32), st=filled((n,), i32), se=filled((n,), i32),
               sw=filled((n,), f32), ss=filled((n,), i32), sn=filled((1,), i32),
               Y=filled((T, d), bf), Z=filled((n, d), bf), dweight=filled((n,), f32),
               G=filled((n, d), bf), dbias=filled((E, d), f32), dz=filled((T, E), f32))
    r = L.Router(z, k, score="sigmoid")
    pairs = L.Pairs(out["token"], out["expert"], out["weight"], T, E)
    f = L.linear_forward(pairs, X, "token", W, act="gelu", bias=bias)
    pg = L.pair_grad_problem(pairs, dY, "token", out["Z"], act="gelu")
    fo = L.forward_outputs(dict(Y=out["Y"], Z=out["Z"]))
    po = L.pair_grad_outputs(dict(dweight=out["dweight"], G=out["G"], dbias=out["dbias"]))
    ws = torch.empty(max(L.lrm_forward_workspace_size(f), L.lrm_pair_grad_workspace_size(pg), 1 << 16),
                     dtype=torch.uint8, device=DEV)

    def calls():
        L.lrm_route(r, out["expert"], out["weight"], token=out["token"], counts=out["counts"], ws=ws)
        L.lrm_route_share(T, k, out["expert"], out["weight"], 2, 6, out["st"], out["se"], out["sw"],
                          out["sn"], out_slot=out["ss"], ws=ws)
        L.lrm_expert_forward(f, fo, ws=ws)
        L.lrm_pair_grad(pg, po, ws=ws)
        L.lrm_route_bwd(r, out["expert"], out["dweight"], out["dz"])

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for step in range(4):
        gs = FC.gen("graph", step)
        z.copy_(FC.normal(gs, T, E))
        X.copy_(FC.normal(gs, T, H).to(bf))
        dY.copy_(FC.normal(gs, T, d).to(bf))
        for v in out.values():
            v.view(torch.uint8).fill_(0xCD)
        graph.replay()
        torch.cuda.synchronize()
        got = _bits(out)
        for v in out.values():
            v.view(torch.uint8).fill_(0xCD)
        calls()
        torch.cuda.synchronize()
        want = _bits(out)
        for name in out:
            assert torch.equal(got[name], want[name]), (step, name)
        assert L.lrm_check_device_errors(ws) == L.LRM_OK


def test_two_streams_at_once(L):
    """Two calls on two streams, each with its own workspace and outputs."""
    todo = []
    for name in ("glu_mid", "lin_odd"):
        c = FC.forward_case(name)
        f = make_forward(L, c)
        out = {k: filled(*v) for k, v in FC.forward_shapes(c).items()}
        ws = torch.empty(L.lrm_forward_workspace_size(f), dtype=torch.uint8, device=DEV)
        rc = FC.route_case("groups_top2")
        r = make_router(L, rc)
        ex, wt = filled((rc["T"] * rc["k"],), torch.int32), filled((rc["T"] * rc["k"],), torch.float32)
        todo.append((c, f, out, ws, r, ex, wt, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, f, out, ws, r, ex, wt, s in todo:
            L.lrm_expert_forward(f, out, ws=ws, stream=s)
            L.lrm_route(r, ex, wt, stream=s)
    torch.cuda.synchronize()
    for c, f, out, ws, r, ex, wt, s in todo:
        FC.judge_forward(c, out)
        alone = {k: filled(*v) for k, v in FC.forward_shapes(c).items()}
        ex1, wt1 = torch.empty_like(ex), torch.empty_like(wt)
        L.lrm_expert_forward(f, alone)
        L.lrm_route(r, ex1, wt1)
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k].view(torch.uint8), alone[k].view(torch.uint8)), k
        assert torch.equal(ex, ex1) and torch.equal(wt, wt1)


def test_pair_grad_without_tokens(L):
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    pairs = L.Pairs(filled((0,), i32), filled((0,), i32), filled((0,), f32), 0, 5)
    out = dict(dweight=filled((0,), f32), G=filled((0, 72), bf), dbias=filled((5, 72), f32))
    L.lrm_pair_grad(L.pair_grad_problem(pairs, filled((0, 72), bf), "token", filled((0, 72), bf),
                                        act="gelu"), out)
    torch.cuda.synchronize()
    assert not out["dbias"].any()
    L.lrm_pair_grad(L.pair_grad_problem(pairs, filled((0, 72), bf), "pair", filled((0, 72), bf)),
                    dict(dweight=out["dweight"]))
    torch.cuda.synchronize()
