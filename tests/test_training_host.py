"""CPU tests of the balance losses and the update of the parameters: the fp64
oracle is pinned against hand values, differences and automatic differentiation,
and the C ABI and its binding refuse bad arguments before any HIP call."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import training_cases as TC
from oracle import forward as OF
from oracle import training as OT
from pruned_expert_backward_lrm_amd import lrm as L

lib = L._lib


# ------------------------------------------------------------- oracle pins
def test_balance_by_hand():
    z = torch.log(torch.tensor([[3.0, 1.0], [1.0, 1.0]]))
    f = OT.balance(z, 1, expert=np.array([0, 0]), coef=1.0, z_coef=0.5)
    # all slots on expert 0: f = (1, 0), P = (0.75 + 0.5) / 2, M = 2
    assert np.allclose(f["loss"], [2 * 0.625, 0.5 * (math.log(4) ** 2 + math.log(2) ** 2) / 2])
    assert np.allclose(f["saved"], [1.0, 0.0, 1.0, 0.5]) and f["counts"].tolist() == [[2, 0]]
    # balanced: 1
    f = OT.balance(torch.zeros(4, 2), 1, expert=np.array([0, 1, 0, 1]), coef=1.0)
    assert np.allclose(f["loss"], [1.0, 0.0])
    # by sequence, one of them empty, one token of none
    f = OT.balance(torch.zeros(4, 2), 1, expert=np.array([0, 0, 1, 1]), seq=[0, 2, 2, 3], coef=1.0)
    assert np.allclose(f["loss"][0], 1.0) and f["counts"].tolist() == [[2, 0], [0, 0], [0, 1]]
    assert np.allclose(f["saved"][:6], [1, 0, 0, 0, 0, 2]) and f["saved"][6] == 0.5


@pytest.mark.parametrize("name", ["seqs", "sigmoid", "shifted", "sigmoid_low", "row_of_none"])
def test_balance_gradient_is_the_difference_quotient(name):
    c = TC.balance_case(name)
    z, f = c["clean"].double(), c["fwd"]
    kw = dict(c["kw"], expert=c["expert"].numpy(), seq=c["seq"], coef=c["coef"], z_coef=c["z_coef"])
    grad = OT.balance_bwd(z, c["k"], f, (1.0, 1.0), c["score"], **{k: v for k, v in c["kw"].items()
                                                                  if k != "score"})
    rng = np.random.default_rng(1)
    for _ in range(25):
        t, e = int(rng.integers(c["T"])), int(rng.integers(c["E"]))
        if z[t, e] == -math.inf:
            assert grad[t, e] == 0
            continue
        d, h = [], 1e-4
        for s in (-h, h):
            y = z.clone()
            y[t, e] += s
            d.append(OT.balance(y, c["k"], **kw)["loss"].sum())
        assert abs((d[1] - d[0]) / (2 * h) - float(grad[t, e])) <= 1e-8


def test_balance_gradient_is_the_derivative():
    """Against automatic differentiation of the losses and the routing weights."""
    for name in ("small_bf16", "sigmoid_seqs"):
        c = TC.balance_case(name)
        z = c["clean"].double().clamp_min(-1e3).requires_grad_(True)
        p = torch.softmax(z, 1) if c["score"] == "softmax" else \
            torch.sigmoid(z) / torch.sigmoid(z).sum(1, keepdim=True)
        cuts = c["seq"] or [0, c["T"]]
        bal = sum((torch.as_tensor(c["fwd"]["a"][s]) * p[i:j].sum(0)).sum()
                  for s, (i, j) in enumerate(zip(cuts, cuts[1:]))) * c["fwd"]["saved"][-2]
        zl = 0.5 * c["fwd"]["saved"][-1] * torch.logsumexp(z, 1)[cuts[0]:cuts[-1]].square().sum()
        assert abs(bal.item() - c["fwd"]["loss"][0]) < 1e-12
        assert abs(zl.item() - c["fwd"]["loss"][1]) < 1e-12
        e = c["expert"].view(c["T"], c["k"]).long()
        s = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
        w = s.gather(1, e)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
        d = c["dloss"].tolist()
        total = d[0] * bal + d[1] * zl + (w.reshape(-1) * c["dweight"].double()).sum()
        ref = torch.autograd.grad(total, z)[0]
        got = OT.balance_bwd(c["clean"], c["k"], c["fwd"], d, c["score"], c["expert"].numpy(),
                             c["dweight"], c["renorm"])
        assert torch.allclose(got, ref, atol=1e-12)


def test_codes_by_hand():
    # a largest element of 1.5: exponent 127, codes 31 octaves and a half
    assert OT.block_exponent([1.5, 0.1], True) == 127 and OT.encode(1.5, 127, True, 0)[0] == 31 * 8 + 4
    assert OT.decode(31 * 8 + 4, 127, True) == 1.5 and OT.decode(0, 127, True) == 0.0
    # above 7/8 of an octave the block moves up, so that rounding up stays inside
    assert OT.block_exponent([1.9], False) == 128 and OT.block_exponent([1.875], False) == 127
    assert OT.decode(OT.encode(-1.99, 128, False, 0xFFFF)[0], 128, False) == -2.0
    # exact values stay, whatever the random bits
    for r in (0, 0x7FFF, 0xFFFF):
        for code in (1, 7, 8, 200, 255):
            assert OT.encode(OT.decode(code, 140, True), 140, True, r)[0] == code
        for code in (1, 100, 127, 129, 255):
            assert OT.encode(OT.decode(code, 140, False), 140, False, r)[0] == code
    # below the least code: v stays positive, m is dropped
    assert OT.encode(1e-30, 127, True, 0)[0] == 1 and OT.encode(1e-30, 127, False, 0xFFFF)[0] == 0


def test_random_bits_are_even_and_independent():
    """Means, correlations between the three numbers, neighbours and steps: within
    5 deviations of what even, independent numbers have."""
    n = 4096
    a = np.array([OT.random_bits(7, 3, i) for i in range(n)], np.float64) / 65536 - 0.5
    b = np.array([OT.random_bits(7, 4, i) for i in range(n)], np.float64) / 65536 - 0.5
    assert (np.abs(a.mean(0)) < 5 / math.sqrt(12 * n)).all()
    pairs = [(a[:, i], a[:, j]) for i, j in ((0, 1), (0, 2), (1, 2))]
    pairs += [(a[:-1, i], a[1:, i]) for i in range(3)] + [(a[:, i], b[:, i]) for i in range(3)]
    pairs += [(a[:-32, i], a[32:, i]) for i in range(3)]
    for x, y in pairs:
        assert abs((x * y).mean()) < 5 / 12 / math.sqrt(len(x))
    for i in range(3):
        assert (np.bincount(((a[:, i] + 0.5) * 16).astype(int), minlength=16) > n / 16 - 5 * 16).all()


def test_adamw_is_the_formula():
    w, m, v = OT.adamw(np.array([1.0]), np.array([0.5]), np.zeros(1), np.zeros(1), 1, 0.1, decay=0.2)
    # the first step is lr sign(g), and the decay
    assert abs(float(w[0]) - (1.0 - 0.1 - 0.02)) < 1e-7
    assert np.allclose(m, 0.05) and np.allclose(v, 0.00025)
    p = torch.tensor([1.0, -2.0], dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=0.03, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    x = np.array([1.0, -2.0])
    m = v = np.zeros(2)
    for s in range(1, 6):
        g = np.array([0.3 * s, -0.1])
        p.grad = torch.as_tensor(g)
        opt.step()
        x, m, v = OT.adamw(x, g, m, v, s, 0.03, 0.8, 0.95, 1e-6, 0.1)
        assert np.allclose(p.detach().numpy(), x, atol=1e-14)


# ---------------------------------------------------------------- refusals
P = 0x1000  # an aligned address; nothing is launched


def balance(router=None, **kw):
    r = dict(T=4, E=8, k=2, score=0, flags=0, n_group=1, topk_group=1, group_rule=0, scale=1.0,
             dtype=L.LRM_BF16, logits=P, ld=8, bias=None, expert_mask=None, token_mask=None)
    r.update(router or {})
    v = dict(router=L.lrm_router(*r.values()), expert=P, counts=None, seq=None, S=1, coef=1.0,
             z_coef=0.1, _pad=0)
    v.update(kw)
    return L.lrm_balance(*v.values())


BALANCE_REFUSALS = [
    (dict(router=dict(T=-1)), 2), (dict(router=dict(ld=7)), 2), (dict(router=dict(dtype=4)), 3),
    (dict(router=dict(logits=None)), 1), (dict(S=0, seq=P), 2), (dict(S=2), 2),
    (dict(S=(1 << 20) + 1, seq=P), 2), (dict(S=1 << 20, seq=P, router=dict(E=4096, ld=4096)), 2),
    (dict(coef=float("nan")), 10), (dict(z_coef=float("inf")), 10),
    (dict(router=dict(score=1)), 10), (dict(expert=P + 2), 5), (dict(counts=P + 1), 5),
    (dict(seq=P + 2, S=3), 5),
]


@pytest.mark.parametrize("kw,status", BALANCE_REFUSALS)
def test_balance_refusals(kw, status):
    b = balance(**kw)
    assert lib.lrm_balance_loss(C.byref(b), P, P, None, P, 1 << 40, None) == status
    assert lib.lrm_balance_bwd(C.byref(b), P, None, None, P, 5000, None) == status
    assert lib.lrm_balance_workspace_size(C.byref(b)) == 0


def test_balance_call_refusals():
    b, ref = balance(), C.byref
    big = 1 << 40
    assert lib.lrm_balance_loss(None, P, P, None, P, big, None) == 1
    assert lib.lrm_balance_loss(ref(b), None, P, None, P, big, None) == 1
    assert lib.lrm_balance_loss(ref(b), P, None, None, P, big, None) == 1
    assert lib.lrm_balance_loss(ref(b), P + 2, P, None, P, big, None) == 5
    assert lib.lrm_balance_loss(ref(b), P, P, P + 1, P, big, None) == 5
    assert lib.lrm_balance_loss(ref(b), P, P, None, None, big, None) == 7
    assert lib.lrm_balance_loss(ref(b), P, P, None, P, 16, None) == 7
    assert lib.lrm_balance_loss(ref(b), P, P, None, P + 64, big, None) == 5
    assert lib.lrm_balance_loss(ref(balance(expert=None)), P, P, None, P, big, None) == 1
    assert lib.lrm_balance_loss(ref(balance(counts=P)), P, P, P, P, big, None) == 10
    assert lib.lrm_balance_bwd(None, P, None, None, P, 8, None) == 1
    assert lib.lrm_balance_bwd(ref(b), None, None, None, P, 8, None) == 1
    assert lib.lrm_balance_bwd(ref(b), P, None, None, None, 8, None) == 1
    assert lib.lrm_balance_bwd(ref(balance(expert=None)), P, None, P, P, 8, None) == 1
    assert lib.lrm_balance_bwd(ref(b), P, None, None, P, 7, None) == 2
    assert lib.lrm_balance_bwd(ref(b), P, P + 2, None, P, 8, None) == 5
    assert lib.lrm_balance_bwd(ref(b), P, None, None, P + 1, 8, None) == 5


def params(n=1, table=P, param=True, **kw):
    v = dict(p=P, g=P, master=None, m=P, v=P, m_exp=None, v_exp=None, n=100, lr=1.0, weight_decay=0.0)
    top = dict(p_dtype=0, g_dtype=0, moments=0, masters=0)
    top.update({k: kw.pop(k) for k in list(kw) if k in top})
    v.update(kw)
    arr = (L.lrm_param * max(n, 1))(*[L.lrm_param(*v.values()) for _ in range(max(n, 1))])
    ps = L.lrm_params(n, *top.values(), 0, arr if param else None, table, 1)
    ps._arr = arr
    return ps


PARAM_REFUSALS = [
    (dict(n=-1), 2), (dict(n=65537, param=False), 2), (dict(p_dtype=2), 3), (dict(g_dtype=-1), 3),
    (dict(moments=2), 10), (dict(masters=2), 10), (dict(masters=1, master=P), 10), (dict(table=None), 1),
    (dict(param=False), 1), (dict(table=P + 128), 5), (dict(n=1, lr=float("nan")), 10),
    (dict(lr=-1.0), 10), (dict(weight_decay=float("inf")), 10), (dict(g=None), 1), (dict(g=P + 2), 5),
    (dict(p=None), 1), (dict(m=None), 1), (dict(v=None), 1), (dict(master=P), 1),
    (dict(masters=1, p_dtype=1), 1), (dict(moments=1), 1), (dict(moments=1, m_exp=P), 1),
    (dict(m_exp=P), 1), (dict(p=P + 2), 5), (dict(m=P + 1), 5), (dict(v=P + 2), 5),
    (dict(p_dtype=1, p=P + 1), 5), (dict(p_dtype=1, masters=1, master=P + 2), 5),
]


def step(**kw):
    v = dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, grad_scale=1.0, max_norm=0.0, step=1, seed=0,
             sumsq=None, n_sumsq=0, _pad=0, lr_dev=None, steps=None)
    v.update(kw)
    return L.lrm_adamw_step(*v.values())


@pytest.mark.parametrize("kw,status", PARAM_REFUSALS)
def test_params_refusals(kw, status):
    ps, a = params(**kw), step()
    assert lib.lrm_params_table(C.byref(ps), 1 << 40, None) == status
    assert lib.lrm_grad_sumsq(C.byref(ps), P, P, 1 << 40, None) == status
    assert lib.lrm_sumsq_workspace_size(C.byref(ps)) == 0
    assert lib.lrm_adamw(C.byref(ps), C.byref(a), None) == status


def test_params_call_refusals():
    ps, ref = params(), C.byref
    big = 1 << 40
    assert lib.lrm_params_table_size(-1) == 0 and lib.lrm_params_table_size(65537) == 0
    assert lib.lrm_params_table_size(0) > 0
    assert lib.lrm_params_table(None, big, None) == 1
    assert lib.lrm_params_table(ref(ps), 64, None) == 7
    assert lib.lrm_grad_sumsq(ref(ps), None, P, big, None) == 1
    assert lib.lrm_grad_sumsq(ref(ps), P + 4, P, big, None) == 5
    assert lib.lrm_grad_sumsq(ref(ps), P, None, big, None) == 7
    assert lib.lrm_grad_sumsq(ref(ps), P, P, 8, None) == 7
    assert lib.lrm_grad_sumsq(ref(ps), P, P + 4, big, None) == 5
    ps.chunks = 2  # another table's
    assert lib.lrm_grad_sumsq(ref(ps), P, P, big, None) == 2
    a = step()
    assert lib.lrm_adamw(ref(ps), ref(a), None) == 2
    ps.chunks = 1
    # gradients alone: to be read, not updated
    only = params(p=None, m=None, v=None)
    assert lib.lrm_sumsq_workspace_size(ref(only)) > 0
    a = step()
    assert lib.lrm_adamw(ref(only), ref(a), None) == 1
    assert lib.lrm_adamw(ref(ps), None, None) == 1


STEP_REFUSALS = [
    (dict(lr=-0.1), 10), (dict(lr=float("nan")), 10), (dict(eps=0.0), 10), (dict(eps=1e-17), 10), (dict(eps=float("inf")), 10),
    (dict(beta1=1.0), 10), (dict(beta1=-0.1), 10), (dict(beta2=1.5), 10), (dict(beta2=float("nan")), 10),
    (dict(grad_scale=float("inf")), 10), (dict(max_norm=-1.0, sumsq=P, n_sumsq=1), 10),
    (dict(step=0), 2), (dict(step=(1 << 53) + 1), 2), (dict(n_sumsq=1), 2), (dict(sumsq=P), 2),
    (dict(sumsq=P, n_sumsq=65), 2), (dict(max_norm=1.0), 1), (dict(sumsq=P + 4, n_sumsq=1), 5),
    (dict(lr_dev=P + 2), 5), (dict(steps=P + 4), 5),
]


@pytest.mark.parametrize("kw,status", STEP_REFUSALS)
def test_step_refusals(kw, status):
    ps, a = params(), step(**kw)
    assert lib.lrm_adamw(C.byref(ps), C.byref(a), None) == status


def test_moment_read_refusals():
    f = lib.lrm_moment_read
    assert f(-1, 0, P, P, 0, P, None) == 2
    assert f(4, 2, P, P, 0, P, None) == 10
    assert f(4, 0, P, P, 3, P, None) == 3
    assert f(4, 0, None, P, 0, P, None) == 1 and f(4, 0, P, None, 0, P, None) == 1
    assert f(4, 0, P, P, 0, None, None) == 1
    assert f(4, 1, P, P, 0, P + 2, None) == 5 and f(4, 1, P, P, 1, P + 1, None) == 5


def test_struct_layouts():
    assert C.sizeof(L.lrm_balance) == 120 and L.lrm_balance.S.offset == 104
    assert C.sizeof(L.lrm_param) == 72 and L.lrm_param.n.offset == 56
    assert C.sizeof(L.lrm_params) == 48 and L.lrm_params.chunks.offset == 40
    assert C.sizeof(L.lrm_adamw_step) == 96 and L.lrm_adamw_step.sumsq.offset == 64


def test_binding_refuses_what_does_not_fit():
    z = torch.zeros(4, 8)
    r = L.Router(z, 2)
    e = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="expert"):
        L.Balance(r, expert=e[:7])
    with pytest.raises(ValueError, match="expert"):
        L.Balance(r, expert=e.long())
    with pytest.raises(ValueError, match="seq"):
        L.Balance(r, expert=e, seq=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="counts"):
        L.Balance(r, counts=torch.zeros(8, dtype=torch.int32), seq=torch.zeros(3, dtype=torch.int32))
    b = L.Balance(r, expert=e)
    f = torch.zeros(10)
    with pytest.raises(ValueError, match="saved"):
        L.lrm_balance_loss(b, f[:2], f[:9])
    with pytest.raises(ValueError, match="loss"):
        L.lrm_balance_loss(b, f[:1], f)
    with pytest.raises(ValueError, match="dlogits"):
        L.lrm_balance_bwd(b, f, torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dweight"):
        L.lrm_balance_bwd(b, f, z, dweight=torch.zeros(7))
    with pytest.raises(ValueError, match="not on a GPU"):
        L.lrm_balance_loss(b, f[:2], f, ws=torch.zeros(1 << 16, dtype=torch.uint8))


def test_binding_refuses_lists_that_do_not_fit():
    t = lambda n=8, dt=torch.float32: torch.zeros(n, dtype=dt)  # noqa: E731
    good = dict(g=[t()], p=[t()], m=[t()], v=[t()])

    def bad(match, **kw):
        with pytest.raises(ValueError, match=match):
            L.Params(**dict(good, **kw))

    bad("at least one", g=[])
    bad("p must have 1", p=[t(), t()])
    bad(r"m\[0\]", m=[t(9)])
    bad(r"v\[0\]", v=[t(dt=torch.bfloat16)])
    bad(r"p\[0\]", p=[torch.zeros(8, 2)[:, 0]])
    bad("lr must", lr=[1.0, 2.0])
    bad("shares memory", p=good["m"])
    x = t(40)
    bad("shares memory", g=[x[:8]], p=[x[4:12]])
    bad("shares memory", g=[t(), t()], p=[x[:8], x[7:15]], m=[t(), t()], v=[t(), t()])
    # the same tensor twice
    y = {k: v * 2 for k, v in good.items()}
    with pytest.raises(ValueError, match="shares memory"):
        L.Params(**y)
    # (gradients may: only the device is wrong here)
    with pytest.raises(ValueError, match="not on a GPU"):
        L.Params(g=[x[:8], x[:8]])
    c8 = dict(m=[t(dt=torch.uint8)], v=[t(dt=torch.uint8)])
    bad(r"v\[0\]", m=[t(dt=torch.uint8)], m_exp=[t(1, torch.uint8)], v_exp=[t(1, torch.uint8)])
    bad(r"m_exp\[0\]", **c8, m_exp=[t(2, torch.uint8)], v_exp=[t(1, torch.uint8)])
    with pytest.raises(ValueError, match="sumsq"):
        L.AdamW(sumsq=t())
    with pytest.raises(ValueError, match="steps"):
        L.AdamW(steps=t(1))
    with pytest.raises(ValueError, match="lr"):
        L.AdamW(lr=t(2))
    with pytest.raises(ValueError, match="codes"):
        L.lrm_moment_read(t(8), t(1, torch.uint8), t(8), "m")
