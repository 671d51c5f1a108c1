"""fp64 CPU oracle of the router, the experts' forward pass and the backward
pass of its epilogue -- TEST INFRASTRUCTURE ONLY.

Written from the definitions, one token or one pair at a time, without any of
the product's code.  Tensors are CPU torch tensors; results are float64.
"""

from __future__ import annotations

import math

import numpy as np
import torch


# ------------------------------------------------------------------ router
def _scores(z, on, score):
    """Scores of one row: list of floats, None where not eligible."""
    if score == "sigmoid":
        return [1.0 / (1.0 + math.exp(-v)) if v > -700 else math.exp(v) if o else 0.0
                for v, o in zip(z, on)]
    if not any(on):
        return [0.0] * len(z)
    m = max(v for v, o in zip(z, on) if o)
    ex = [math.exp(v - m) if o else 0.0 for v, o in zip(z, on)]
    s = math.fsum(ex)
    return [v / s for v in ex]


def route(logits, k, score="softmax", renorm=True, scale=1.0, n_group=1, topk_group=1,
          group_rule="top2", bias=None, expert_mask=None, token_mask=None):
    """(expert [T*k] int64 with -1 in empty slots, weight [T*k] float64)."""
    T, E = logits.shape
    z = logits.double().tolist()
    b = bias.double().tolist() if bias is not None else None
    em = [bool(v) for v in expert_mask.tolist()] if expert_mask is not None else [True] * E
    tm = [bool(v) for v in token_mask.tolist()] if token_mask is not None else [True] * T
    experts, weights = [], []
    for t in range(T):
        on = [tm[t] and em[e] and z[t][e] > -math.inf for e in range(E)]
        row = [z[t][e] if on[e] else 0.0 for e in range(E)]
        s = _scores(row, on, score)
        # without a bias the exact scores order like the logits
        key = row if b is None else [s[e] + b[e] for e in range(E)]
        if b is not None:  # a bias of -inf closes its expert to the choice
            on = [on[e] and b[e] > -math.inf for e in range(E)]
        if n_group > 1:
            per = E // n_group
            best = []
            for g in range(n_group):
                have = [e for e in range(g * per, (g + 1) * per) if on[e]]
                if not have:
                    continue
                val = key if b is not None or group_rule == "max" else s
                top = sorted((val[e] for e in have), reverse=True)
                best.append((-(top[0] if group_rule == "max" else sum(top[:2])), g))
            keep = {g for _, g in sorted(best)[:topk_group]}
            on = [on[e] and e // per in keep for e in range(E)]
        order = sorted((e for e in range(E) if on[e]), key=lambda e: (-key[e], e))[:k]
        if renorm and order:
            # s / sum of s, with the common factor of tiny scores taken out
            if score == "softmax":
                m = max(row[e] for e in order)
                f = [math.exp(row[e] - m) for e in order]
            else:
                m = min(0.0, max(row[e] for e in order))
                f = [math.exp(row[e] - m) / (1.0 + math.exp(row[e])) if row[e] < 0
                     else math.exp(-m) / (1.0 + math.exp(-row[e])) for e in order]
            w = [scale * v / math.fsum(f) for v in f]
        else:
            w = [scale * s[e] for e in order]
        experts += order + [-1] * (k - len(order))
        weights += w + [0.0] * (k - len(order))
    return np.array(experts, np.int64).reshape(-1), np.array(weights, np.float64).reshape(-1)


def route_bwd(logits, k, expert, dweight, score="softmax", renorm=True, scale=1.0,
              expert_mask=None, token_mask=None):
    """Gradient of the logits, by automatic differentiation of the definition."""
    T, E = logits.shape
    out = torch.zeros(T, E, dtype=torch.float64)
    ex = np.asarray(expert).reshape(T, k)
    dw = torch.as_tensor(dweight).double().reshape(T, k)
    for t in range(T):
        if token_mask is not None and not token_mask[t]:
            continue
        on = [e for e in range(E) if (expert_mask is None or expert_mask[e])
              and float(logits[t, e]) > -math.inf]
        where = {e: i for i, e in enumerate(on)}
        slots = [j for j in range(k) if int(ex[t, j]) in where]
        if not slots:
            continue
        z = logits[t, on].double().requires_grad_(True)
        sel = torch.tensor([where[int(ex[t, j])] for j in slots])
        if score == "softmax":
            ls = torch.log_softmax(z, 0)[sel]
        else:
            ls = torch.nn.functional.logsigmoid(z)[sel]
        w = scale * (torch.softmax(ls, 0) if renorm else torch.exp(ls))
        (w * dw[t, slots]).sum().backward()
        out[t, on] = z.grad
    return out


def route_share(k, expert, weight, e0, E):
    slot = [i for i, e in enumerate(np.asarray(expert).tolist()) if e0 <= e < e0 + E]
    slot = np.array(slot, np.int64)
    return slot // k, np.asarray(expert)[slot] - e0, np.asarray(weight)[slot], slot


# ---------------------------------------------------------- experts forward
def act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def present(pairs, T, E):
    tok, ex = np.asarray(pairs["token"]), np.asarray(pairs["expert"])
    return (tok >= 0) & (tok < T) & (ex >= 0) & (ex < E)


def forward(kind, pairs, T, E, X, x_rows="token", W=None, bias=None, act_name="none",
            W_gate=None, W_up=None, W_down=None, residual=None):
    """dict of float64: Y [T][d], Yp [N][d], Z or A, B [N][.] and `h` (SwiGLU);
    rows of absent pairs are NaN in the PAIR arrays."""
    tok, ex = np.asarray(pairs["token"]), np.asarray(pairs["expert"])
    wt = np.asarray(pairs["weight"], np.float64)
    here = present(pairs, T, E)
    N = tok.shape[0]
    d = W.shape[1] if kind == "linear" else W_down.shape[1]
    nan = float("nan")
    Yp = torch.full((N, d), nan, dtype=torch.float64)
    Y = residual.double().clone() if residual is not None else torch.zeros(T, d, dtype=torch.float64)
    if kind == "linear":
        Z = torch.full((N, d), nan, dtype=torch.float64)
    else:
        I = W_gate.shape[1]  # noqa: E741
        A = torch.full((N, I), nan, dtype=torch.float64)
        B = torch.full((N, I), nan, dtype=torch.float64)
    for p in np.nonzero(here)[0]:
        e = int(ex[p])
        x = X[int(tok[p]) if x_rows == "token" else int(p)].double()
        if kind == "linear":
            z = W[e].double() @ x
            if bias is not None:
                z = z + bias[e].double()
            Z[p] = z
            y = act(z, act_name)
        else:
            a, b = W_gate[e].double() @ x, W_up[e].double() @ x
            A[p], B[p] = a, b
            y = W_down[e].double() @ (act(a, "silu") * b)
        Yp[p] = y
        Y[int(tok[p])] += wt[p] * y
    out = {"Y": Y, "Yp": Yp}
    out.update({"Z": Z} if kind == "linear" else {"A": A, "B": B})
    return out


def pair_grad(pairs, T, E, dY, dy_rows, Z, act_name):
    """dict of float64: dweight [N], G [N][d], dbias [E][d] (absent pairs: 0)."""
    tok, ex = np.asarray(pairs["token"]), np.asarray(pairs["expert"])
    wt = np.asarray(pairs["weight"], np.float64)
    N, d = Z.shape
    dw = torch.zeros(N, dtype=torch.float64)
    G = torch.zeros(N, d, dtype=torch.float64)
    db = torch.zeros(E, d, dtype=torch.float64)
    for p in np.nonzero(present(pairs, T, E))[0]:
        z = Z[p].double().requires_grad_(True)
        dy = dY[int(tok[p]) if dy_rows == "token" else int(p)].double()
        y = act(z, act_name)
        (y * dy).sum().backward()
        dw[p] = (y.detach() * dy).sum()
        G[p] = z.grad
        db[int(ex[p])] += wt[p] * z.grad
    return {"dweight": dw, "G": G, "dbias": db}
