"""Inputs, fp64 references and tolerances shared by the tests of the balance
losses and the update of the parameters (on the GPU and in the CPU emulation).

Tolerances are derived from the arithmetic, with u = 2^-24 (half a step of fp32,
relative) and half = half a step of the output type:

* a share p is off by (R + 80) u of itself, R the spread of the row's logits (the
  exponent's product is rounded to 2^-24 of it; sums of up to 4096 experts are
  added in at most 64 + 6 steps);
* the log of the exps' sum is off by (R + 80) u + 3 u |lse|;
* a sum over tokens is fp32 over at most 256 of them, in at most 64 + 6 steps, then fp64;
* the sums of the gradient, one term at a time: every factor's error times the others;
* an AdamW step: m and v are off by 6 u of their terms (the factors' and three
  roundings), the update by what that makes of it and 10 u, the weight by 3 u more;
* a code, or a bf16 weight, that is rounded by random bits is the reference's
  unless its place lies within that error of a border: then it may be a neighbour.
"""

from __future__ import annotations

import math

import numpy as np
import torch

from forward_cases import DT, HALF, U, close, gen, normal
from oracle import forward as OF
from oracle import training as OT

__all__ = ["DT", "HALF", "U", "close", "gen", "normal"]

# --------------------------------------------------------------- balance
BALANCE = {
    # name: T, E, k, dtype, and more
    "one_token": dict(T=1, E=4, k=1),
    "small_bf16": dict(T=37, E=16, k=2, dtype="bf16"),
    "seqs": dict(T=70, E=24, k=3, seq=[3, 3, 4, 40, 40, 66]),
    "one_seq": dict(T=30, E=16, k=2, seq=[5, 22]),
    "one_empty_seq": dict(T=9, E=8, k=2, seq=[4, 4]),
    "one_seq_wide": dict(T=150, E=300, k=2, seq=[2, 147], dtype="bf16"),
    "garbage_outside": dict(T=40, E=16, k=2, seq=[3, 20, 31], garbage=True),
    "garbage_outside_dense": dict(T=40, E=24, k=2, seq=[3, 20, 31], garbage=True, renorm=False,
                                  dtype="bf16"),
    "seqs_bf16": dict(T=70, E=40, k=3, dtype="bf16", seq=[0, 1, 33, 70]),
    "sigmoid": dict(T=45, E=33, k=4, score="sigmoid", padded=0.2, down=3),
    "sigmoid_seqs": dict(T=66, E=40, k=2, score="sigmoid", dtype="bf16", seq=[0, 30, 64], renorm=False),
    "sigmoid_low": dict(T=9, E=12, k=3, score="sigmoid", shift=-200.0),
    "shifted": dict(T=33, E=20, k=3, shift=70.0, renorm=False),
    "counts_given": dict(T=50, E=16, k=2, counts=True),
    "strided": dict(T=21, E=19, k=3, ld=29, dtype="bf16", renorm=False, padded=0.3),
    "nobody": dict(T=12, E=8, k=2, padded=1.0),
    "row_of_none": dict(T=10, E=8, k=2, closed_rows=3),
    "wide": dict(T=20, E=200, k=20, renorm=False, dtype="bf16"),
    "wider": dict(T=12, E=300, k=5, seq=[0, 5, 12]),
    "thousand": dict(T=9, E=700, k=6, score="sigmoid", dtype="bf16"),
    "aligned_thousand": dict(T=6, E=528, k=3),
    "aligned_1104": dict(T=5, E=1104, k=3, dtype="bf16"),
    "most": dict(T=6, E=1100, k=33, renorm=False),
    "twice": dict(T=17, E=12, k=5, repeat=True, renorm=False),
}


def balance_case(name, **over):
    c = dict(dtype="f32", score="softmax", renorm=True, seq=None, padded=0.0, down=0, shift=0.0,
             counts=False, ld=None, closed_rows=0, repeat=False, garbage=False, coef=0.5,
             **{k: v for k, v in BALANCE.get(name, {}).items()
                if k not in ("dtype", "score", "renorm", "seq", "padded", "down", "shift", "counts",
                             "ld", "closed_rows", "repeat", "garbage")})
    c.update(BALANCE.get(name, {}))
    c.update(over)
    g = gen("balance", name)
    T, E, k = c["T"], c["E"], c["k"]
    z = torch.randn(T, E, generator=g) * 2 + c["shift"]
    c["z_coef"] = 0.03 if c["score"] == "softmax" else 0.0
    c["token_mask"] = c["expert_mask"] = None
    if c["padded"]:
        c["token_mask"] = (torch.rand(T, generator=g) >= c["padded"]).to(torch.uint8)
    if c["down"]:
        m = torch.ones(E, dtype=torch.uint8)
        m[torch.randperm(E, generator=g)[:c["down"]]] = 0
        c["expert_mask"] = m
    for t in range(c["closed_rows"]):
        z[2 * t] = -math.inf
    if T > 4 and E > 4:
        z[3, 1] = -math.inf
    z = z.to(DT[c["dtype"]])
    c["clean"] = z.clone()
    # what masked places hold is not used
    if c["token_mask"] is not None:
        z[c["token_mask"] == 0] = float("nan")
    if c["expert_mask"] is not None:
        z[:, c["expert_mask"] == 0] = float("inf")
    c["logits"] = z
    kw = dict(score=c["score"], expert_mask=c["expert_mask"], token_mask=c["token_mask"])
    e, _ = OF.route(c["clean"], k, renorm=c["renorm"], **kw)
    if c["repeat"]:  # a choice that names an expert more than once, and one that is none
        e = e.reshape(T, k)
        e[::2, 1] = e[::2, 0]
        e[::4, 3] = e[::4, 0]
        e[1, 0], e[1, 1] = E, -7
        e = e.reshape(-1)
    if c["garbage"]:  # tokens of no sequence, without slots: their logits may be anything
        e = e.reshape(T, k)
        for t in (*range(c["seq"][0]), *range(c["seq"][-1], T)):
            e[t] = -1
            z[t] = float("nan")
        e = e.reshape(-1)
    c["expert"] = torch.as_tensor(e).int()
    if c["counts"]:
        c["counts_in"] = torch.randint(0, 100, (1 if c["seq"] is None else len(c["seq"]) - 1, E),
                                       generator=g).int()
        c["counts_in"][:, 0] = 0
    else:
        c["counts_in"] = None
    c["dweight"] = torch.randn(T * k, generator=g) * 0.1
    c["dloss"] = torch.tensor([0.75, 1.5])
    c["kw"] = kw
    # (the kernels take the coefficients in fp32)
    c["coef"], c["z_coef"] = float(np.float32(c["coef"])), float(np.float32(c["z_coef"]))
    c["fwd"] = OT.balance(c["clean"], k, expert=c["expert"].numpy(), counts=c["counts_in"],
                          seq=c["seq"], coef=c["coef"], z_coef=c["z_coef"], **kw)
    return c


def _spread(c):
    z = c["clean"].double()
    z = torch.where(z == -math.inf, torch.nan, z)
    z = torch.nan_to_num(z, nan=float(torch.nan_to_num(z).mean()))
    return float((z.max(1).values - z.min(1).values).max())


def check_balance(c, loss, saved, counts=None):
    f = c["fwd"]
    R = _spread(c)
    close("saved", saved, f["saved"], 2 * U * np.abs(f["saved"]) + 1e-45)
    used = (f["at"] >= 0) & f["live"]
    lse = np.abs(f["lse"][used])
    dz = f["saved"][-1] * float((lse * ((R + 80) * U + 3 * U * lse)).sum())
    close("loss", loss, f["loss"], [(R + 80 + 64 + 4) * U * abs(f["loss"][0]) + 1e-45,
                                    dz + 4 * U * abs(f["loss"][1]) + 1e-45])
    if counts is not None:
        assert torch.equal(counts.long(), torch.as_tensor(f["counts"])), "counts"


def check_balance_bwd(c, dlogits, dweight=True, dloss=True):
    f = c["fwd"]
    T, E, k = c["T"], c["E"], c["k"]
    d = c["dloss"].tolist() if dloss else [1.0, 1.0]
    ref = OT.balance_bwd(c["clean"], k, f, d, c["score"], c["expert"].numpy(),
                         c["dweight"] if dweight else None, c["renorm"],
                         expert_mask=c["expert_mask"], token_mask=c["token_mask"])
    R = _spread(c)
    p, lse = f["p"], np.abs(f["lse"])[:, None]
    a = np.where((f["at"] >= 0)[:, None], f["a"][f["at"]], 0.0)
    size = np.abs(d[0] * f["saved"][-2]) * p * (np.abs(a) + (p * np.abs(a)).sum(1, keepdims=True))
    size = size + np.abs(d[1] * f["saved"][-1]) * p * (lse + R + 3)
    if dweight:
        # every slot's part is at most its |weight gradient| twice (the softmax's two
        # terms), on its expert and, not renormalised, times p on every expert
        dw = np.abs(c["dweight"].numpy().reshape(T, k)).sum(1, keepdims=True)
        hit = np.zeros((T, E))
        for t in range(T):
            for e in c["expert"].numpy().reshape(T, k)[t]:
                if 0 <= e < E:
                    hit[t, e] += 1
        size = size + 2 * dw * (hit + p)
    tol = (R + lse + 80) * U * size + HALF[DT[c["dtype"]]] * np.abs(ref.numpy()) + 1e-38
    assert dlogits.dtype == DT[c["dtype"]]
    close("dlogits", dlogits, ref, tol)


# ------------------------------------------------------------- parameters
PARAMS = {
    # name: sizes of the tensors, and more
    "one": dict(sizes=[1]),
    "odd_f32": dict(sizes=[5, 0, 33, 2049, 8]),
    "bf16_g": dict(sizes=[40, 100], g="bf16"),
    "bf16": dict(sizes=[70, 3], p="bf16"),
    "bf16_bf16": dict(sizes=[64, 257], p="bf16", g="bf16", clip=True),
    "master": dict(sizes=[130, 31], p="bf16", master=True, clip=True),
    "eight": dict(sizes=[1, 31, 32, 33, 100], bits=8),
    "eight_bf16": dict(sizes=[300, 7], bits=8, p="bf16", g="bf16", clip=True),
    "eight_master": dict(sizes=[65], bits=8, p="bf16", master=True),
    "unaligned": dict(sizes=[45, 77], offset=3),
    "unaligned_eight": dict(sizes=[45, 77], offset=3, bits=8, p="bf16", g="bf16"),
    "forty": dict(sizes=[(7 * i) % 45 for i in range(70)], bits=8),
    "first_step": dict(sizes=[100], bits=8, fresh=True, step=1),
}


def param_case(name, **over):
    c = dict(p="f32", g="f32", master=False, bits=32, clip=False, offset=0, fresh=False, step=37,
             seed=0x123456789ABCDEF)
    c.update(PARAMS.get(name, {}))
    c.update(over)
    g = gen("params", name)
    c["lr"], c["beta1"], c["beta2"], c["eps"], c["scale"] = 3e-3, 0.9, 0.99, 1e-8, 0.5
    c["max_norm"] = 0.05 if c["clip"] else 0.0
    c["lrs"] = [1.0 + 0.5 * (i % 2) for i in range(len(c["sizes"]))]
    c["decays"] = [0.1 * (i % 3) for i in range(len(c["sizes"]))]
    t = []
    for i, n in enumerate(c["sizes"]):
        w = normal(g, n, std=0.1)
        q = dict(n=n, g=normal(g, n, std=0.02, dtype=DT[c["g"]]), p=w.to(DT[c["p"]]),
                 master=w if c["master"] else None, m_exp=None, v_exp=None)
        m, v = normal(g, n, std=0.005), normal(g, n, std=0.02).square()
        if n > 2:  # moments that are nothing yet, and far below their block's
            m[0] = v[0] = 0.0
            m[1], v[1] = 1e-12, 1e-30
            q["g"][0] = 0.0
        if c["fresh"]:
            m, v = torch.zeros(n), torch.zeros(n)
        if c["bits"] == 8:
            nb = (n + 31) // 32
            for key, x, second in (("m", m, False), ("v", v, True)):
                codes, exps = np.zeros(n, np.uint8), np.zeros(nb, np.uint8)
                for b in range(nb):
                    xs = [float(y) for y in x[32 * b:32 * b + 32]]
                    exps[b] = 0 if c["fresh"] else OT.block_exponent(xs, second)
                    for j, y in enumerate(xs):
                        if y:
                            codes[32 * b + j] = OT.encode(y, int(exps[b]), second, 0x7FFF)[0]
                q[key], q[key + "_exp"] = torch.from_numpy(codes), torch.from_numpy(exps)
        else:
            q["m"], q["v"] = m, v
        t.append(q)
    c["t"] = t
    c["sumsq"] = math.fsum(float((q["g"].double() ** 2).sum()) for q in t)
    c["factor"] = c["scale"]
    norm = c["scale"] * math.sqrt(c["sumsq"])
    if c["clip"] and norm > c["max_norm"]:
        c["factor"] *= c["max_norm"] / norm
    return c


def values(codes, exps, second):
    return np.array([OT.decode(int(x), int(exps[i // 32]), second) for i, x in enumerate(codes)])


def check_adamw(c, got):
    """got: a list of dicts like c["t"], after one step on c's inputs."""
    place0 = 0
    for i, (q, r) in enumerate(zip(c["t"], got)):
        n = q["n"]
        eight = c["bits"] == 8
        m0, v0 = (values(q[k].numpy(), q[k + "_exp"].numpy(), k == "v") if eight
                  else q[k].double().numpy() for k in ("m", "v"))
        w0 = (q["p"] if q["master"] is None else q["master"]).double().numpy()
        g = q["g"].double().numpy()
        lr, decay = c["lr"] * c["lrs"][i], float(np.float32(c["decays"][i]))
        w, m, v = OT.adamw(w0, g, m0, v0, c["step"], lr, c["beta1"], c["beta2"], c["eps"], decay,
                           c["factor"])
        x = np.abs(c["factor"] * g)
        em = 6 * U * (c["beta1"] * np.abs(m0) + (1 - c["beta1"]) * x) + 1e-44
        ev = 8 * U * (c["beta2"] * v0 + (1 - c["beta2"]) * x * x) + 1e-44
        den = np.sqrt(v / (1 - c["beta2"] ** c["step"])) + c["eps"]
        up = lr / (1 - c["beta1"] ** c["step"])
        ew = up * em / den + 12 * U * np.abs(up * m / den) + 3 * U * (np.abs(w0) + np.abs(w))
        rel_v = np.where(v > 0, ev / np.maximum(v, 1e-300), 0.0)
        ew = ew + np.abs(up * m / den) * rel_v
        if not eight:
            close(f"m[{i}]", r["m"], m, em)
            close(f"v[{i}]", r["v"], v, ev)
        else:
            bits = [OT.random_bits(c["seed"], c["step"], place0 + j) for j in range(n)]
            for key, x0, e0, second in (("m", m, em, False), ("v", v, ev, True)):
                exps = r[key + "_exp"].numpy()
                for b in range((n + 31) // 32):
                    at = slice(32 * b, min(32 * b + 32, n))
                    want = OT.block_exponent([float(y) for y in x0[at]], second)
                    assert int(exps[b]) == want, f"{key}_exp[{i}][{b}]"
                    for j in range(at.start, at.stop):
                        code, far = OT.encode(float(x0[j]), want, second, bits[j][1 if second else 0])
                        have = int(r[key][j])
                        # the place of x is off by its error in steps (x of 8 to 16 of them)
                        near = 16 * e0[j] / max(abs(x0[j]), 1e-300)
                        off = abs((have & 127 if not second else have) - (code & 127 if not second else code))
                        assert have == code or (off == 1 and far <= near), \
                            f"{key}[{i}][{j}]: {have} for {code}, {far:.3g} from the border"
        if c["p"] == "bf16" and q["master"] is None:
            for j in range(n):
                ref, far = OT.round_bf16(float(w[j]), OT.random_bits(c["seed"], c["step"], place0 + j)[2])
                have = float(r["p"][j])
                step = 2.0 ** (OT.octave(float(w[j])) - 7)
                assert have == ref or (abs(have - ref) <= 1.01 * step and far <= ew[j] / step), \
                    f"p[{i}][{j}]: {have!r} for {ref!r}"
        elif q["master"] is not None:
            close(f"master[{i}]", r["master"], w, ew)
            assert torch.equal(r["p"], r["master"].to(torch.bfloat16)), f"p[{i}]"
        else:
            close(f"p[{i}]", r["p"], w, ew)
        place0 += (n + 31) // 32 * 32
