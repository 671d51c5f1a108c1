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


@pytest.mark.parametrize("name", list(FE.BAD_TOKENS))
@pytest.mark.parametrize("tile", [None, "64", "256"])
def test_tokens_out_of_range_are_absent(L, monkeypatch, name, tile):  # noqa: F811
    if tile:
        monkeypatch.setenv("LRM_FWD_TILE", tile)
    c = dict(FE.bad_token_case(name), bad=True)
    out, before = run_forward(L, c)
    FC.judge_forward(c, out, before)


@pytest.mark.parametrize("one_launch", ["0", "1"])
@pytest.mark.parametrize("name", ["middle", "runs", "padded", "many_blocks"])
def test_backward_of_tokens_out_of_range(L, monkeypatch, name, one_launch):  # noqa: F811
    """dX of a call with absent pairs equals that of the call without them (both
    keep every pair: every row's sums have the same terms in the same order)."""
    monkeypatch.setenv("LRM_SELECT_ONE_LAUNCH", one_launch)
    c = FE.bad_token_case(name)
    T, E, N, bf = c["T"], c["E"], c["N"], torch.bfloat16
    g = FC.gen("bad tokens back", name)
    G = FC.normal(g, T, c["d"], dtype=bf)
    X, W = c["X"].to(bf).contiguous(), c["W"].to(bf)
    p = c["pairs"]
    here = (p["token"] >= 0) & (p["token"] < T)

    def back(pick):
        pr = L.Pairs(*(dev(torch.from_numpy(p[k][pick])) for k in ("token", "expert", "weight")), T, E)
        pb = L.linear_problem(pr, dev(X), "token", dev(G), "token", dev(W), [N] * E)
        out = dict(dW=filled((E, c["d"], c["d_in"]), torch.float32),
                   dX=filled((T, c["d_in"]), torch.float32))
        ws = L.lrm_expert_backward(pb, out)
        torch.cuda.synchronize()
        return out, L.lrm_check_device_errors(ws)

    got, status = back(np.ones(N, bool))
    want, ok = back(here)
    assert (status, ok) == (L.LRM_ERR_INDEX, L.LRM_OK)
    assert torch.equal(got["dX"], want["dX"])
    assert float((got["dW"] - want["dW"]).abs().max()) <= 1e-5 * float(want["dW"].abs().max())


@pytest.mark.parametrize("tile", [None, "128", "256"])
@pytest.mark.parametrize("name", list(FE.OVERFLOW))
def test_overflow_stays_infinite(L, monkeypatch, name, tile):  # noqa: F811
    if tile:
        monkeypatch.setenv("LRM_FWD_TILE", tile)
    c = FE.overflow_case(name)
    out, _ = run_forward(L, c)
    FE.judge_overflow(c, out)


@pytest.mark.parametrize("name", list(FE.CLOSED))
def test_bias_of_minus_infinity_closes_an_expert(L, name):  # noqa: F811
    c = FE.closed_case(name)
    FC.judge_route(c, *gpu_route(L, c))


@pytest.mark.parametrize("T", [65535, 65536])
def test_few_pairs_among_many_tokens(L, T):  # noqa: F811
    """A GPU's share of a batch may hold next to nothing: the tokens without pairs
    cost what a copy of the residual costs, not a product each."""
    case = FC._f("swiglu", 3, 32, 2, 2048, 64, residual=True, outs=("Y",))
    c = FC.build_forward(case, "few among many")
    where = np.array([5, 40000, T - 1])
    pr = dict(c["pairs"], token=where[c["pairs"]["token"]].astype(np.int32))
    bf = torch.bfloat16
    X, R = torch.zeros(T, 2048, dtype=bf, device=DEV), torch.randn(T, 2048, device=DEV).to(bf)
    at = dev(torch.from_numpy(where))
    X[at], R[at] = dev(c["X"]), dev(c["R"])
    pairs = L.Pairs(*(dev(torch.from_numpy(pr[k])) for k in ("token", "expert", "weight")), T, 32)
    f = L.swiglu_forward(pairs, X, *(dev(c[w]) for w in ("W_gate", "W_up", "W_down")), residual=R)
    Y = filled((T, 2048), bf)
    ws = L.lrm_expert_forward(f, dict(Y=Y))
    torch.cuda.synchronize()
    FC.judge_forward(c, dict(Y=Y[at]))
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert torch.equal(Y[rest], R[rest])

    copy = time_of(lambda: Y.copy_(R))
    assert time_of(lambda: L.lrm_expert_forward(f, dict(Y=Y), ws=ws)) < 20 * copy + 0.2


@pytest.mark.parametrize("name", FE.SPARSE)
def test_long_runs_of_tokens_without_pairs(L, monkeypatch, name):  # noqa: F811
    monkeypatch.setenv("LRM_FWD_TILE", "128")
    c = FE.sparse_case(name)
    out, _ = run_forward(L, c)
    FC.judge_forward(c, out)


def time_of(call):
    """The least of five, ms."""
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("N", [0, 512, 16384])
def test_tokens_behind_the_last_pair_cost_little(L, N):  # noqa: F811
    """262144 tokens with pairs of the first ones only, forward and backward: Y is
    the residual and dX is 0 there, without a thread that writes them one by one
    (7 ms)."""
    T, E, d, bf = 1 << 18, 8, 64, torch.bfloat16
    g = FC.gen("behind", N)
    tok = torch.arange(N, dtype=torch.int32) // 2
    pairs = L.Pairs(dev(tok), dev(torch.randint(0, E, (N,), generator=g).int()),
                    dev(torch.rand(N, generator=g)), T, E)
    X, W = dev(FC.normal(g, T, d, dtype=bf)), dev(FC.normal(g, E, d, d, std=0.1, dtype=bf))
    f = L.linear_forward(pairs, X, "token", W, residual=X)
    Y = filled((T, d), bf)
    ws = L.lrm_expert_forward(f, dict(Y=Y))
    pb = L.linear_problem(pairs, X, "token", X, "token", W, [max(N // E, 1)] * E)
    out = dict(dW=filled((E, d, d), torch.float32), dX=filled((T, d), torch.float32))
    wb = L.lrm_expert_backward(pb, out)
    torch.cuda.synchronize()
    used = N // 2
    assert torch.equal(Y[used:], X[used:]) and not out["dX"][used:].any()
    if N:
        assert not torch.equal(Y[:used], X[:used]) and out["dX"][:used].any()
    assert time_of(lambda: L.lrm_expert_forward(f, dict(Y=Y), ws=ws)) < 1.5
    assert time_of(lambda: L.lrm_expert_backward(pb, out, ws=wb)) < 1.5
