"""fp64 CPU oracle of the balance losses, their gradient and the update of the
parameters -- TEST INFRASTRUCTURE ONLY.

Written from the definitions, one token or one element at a time, without any
of the product's code.
"""

from __future__ import annotations

import math

import numpy as np
import torch

from oracle import forward as OF


# ----------------------------------------------------------------- balance
def _row(z, on, score):
    """Shares of one row's experts (0 where not eligible) and log of the exps' sum."""
    if not any(on):
        return None, 0.0
    top = max(v for v, o in zip(z, on) if o)
    if score == "softmax":
        f = [math.exp(v - top) if o else 0.0 for v, o in zip(z, on)]
        return [v / math.fsum(f) for v in f], top + math.log(math.fsum(f))
    # sigmoid, the common factor of tiny scores taken out
    m = min(top, 0.0)
    f = [0.0 if not o else math.exp(v - m) / (1.0 + math.exp(v)) if v < 0
         else math.exp(-m) / (1.0 + math.exp(-v)) for v, o in zip(z, on)]
    return [v / math.fsum(f) for v in f], 0.0


def _masks(T, E, expert_mask, token_mask):
    em = [bool(v) for v in expert_mask.tolist()] if expert_mask is not None else [True] * E
    tm = [bool(v) for v in token_mask.tolist()] if token_mask is not None else [True] * T
    return em, tm


def balance(logits, k, expert=None, counts=None, seq=None, coef=1.0, z_coef=0.0, score="softmax",
            expert_mask=None, token_mask=None):
    """dict(loss [2], saved [S*E + 2], counts [S][E], p [T][E], lse [T], live [T], at [T]): at is the
    sequence of a token, -1 for none."""
    T, E = logits.shape
    z = logits.double().tolist()
    em, tm = _masks(T, E, expert_mask, token_mask)
    cuts = [0, T] if seq is None else [int(v) for v in seq]
    S = len(cuts) - 1
    at = [-1] * T
    for s in range(S):
        for t in range(cuts[s], cuts[s + 1]):
            at[t] = s
    p, lse, live = np.zeros((T, E)), np.zeros(T), np.zeros(T, bool)
    for t in range(T):
        on = [tm[t] and em[e] and z[t][e] > -math.inf for e in range(E)]
        got, lse[t] = _row(z[t], on, score)
        if got is not None:
            p[t], live[t] = got, True
    own = np.zeros((S, E), np.int64)
    if counts is None:
        ex = np.asarray(expert).reshape(T, k)
        for t in range(T):
            for e in ex[t]:
                if at[t] >= 0 and tm[t] and 0 <= e < E and em[e]:
                    own[at[t], e] += 1
    c = own if counts is None else np.asarray(counts).reshape(S, E)
    n = np.array([sum(live[t] for t in range(T) if at[t] == s) for s in range(S)], np.float64)
    full, total = int((n > 0).sum()), float(n.sum())
    a, bal, zl = np.zeros((S, E)), 0.0, 0.0
    for s in range(S):
        if n[s] > 0 and c[s].sum() > 0:
            a[s] = sum(em) * (c[s] / c[s].sum()) / n[s]
    for t in range(T):
        if at[t] >= 0 and live[t]:
            bal += float((a[at[t]] * p[t]).sum())
            zl += lse[t] ** 2
    fb, fz = coef / max(full, 1), z_coef / max(total, 1.0)
    return dict(loss=np.array([fb * bal, fz * zl]), counts=own, p=p, lse=lse, live=live,
                at=np.array(at), a=a, saved=np.concatenate([a.reshape(-1), [fb, 2 * fz]]))


def balance_bwd(logits, k, fwd, dloss=(1.0, 1.0), score="softmax", expert=None, dweight=None,
                renorm=True, scale=1.0, expert_mask=None, token_mask=None):
    """Gradient of the logits, from the results of balance."""
    T, E = logits.shape
    z = logits.double().numpy()
    out = np.zeros((T, E))
    for t in range(T):
        s = fwd["at"][t]
        if s < 0 or not fwd["live"][t]:
            continue
        p, a = fwd["p"][t], fwd["a"][s]
        g = dloss[0] * fwd["saved"][-2] * (a - (p * a).sum())
        if score == "sigmoid":
            with np.errstate(over="ignore", invalid="ignore"):
                g = np.where(p > 0, g / (1.0 + np.exp(np.where(p > 0, z[t], 0.0))), 0.0)
        else:
            g = g + dloss[1] * fwd["saved"][-1] * fwd["lse"][t]
        out[t] = p * g
    out = torch.as_tensor(out)
    if dweight is not None:
        out = out + OF.route_bwd(logits, k, expert, dweight, score=score, renorm=renorm, scale=scale,
                                 expert_mask=expert_mask, token_mask=token_mask)
    return out


# ------------------------------------------------------------ the roundings
WORD = 2 ** 32


def _mix(x):
    """Multiply-xorshift mixing with the fractional bits of sqrt 2 and sqrt 3."""
    for shift, root in ((16, 2), (15, 3)):
        x = (x ^ (x >> shift)) * (math.isqrt(root << 64) % WORD) % WORD
    return x ^ (x >> 16)


# 2^32 over the golden ratio, rounded down: floor((sqrt 5 - 1) 2^31)
GOLD = (math.isqrt(5 << 62) - (1 << 31)) % WORD


def random_bits(seed, step, place):
    """The 16 random bits of m, v and p at element `place` (of tensors padded to 32)."""
    key = 0
    for part in (seed % WORD, seed >> 32, step % WORD, step >> 32):
        key = _mix(((key ^ part) + GOLD) % WORD)
    block, j = divmod(place, 32)
    h = _mix((key + block % WORD * GOLD + (block >> 32) * (math.isqrt(3 << 64) % WORD)) % WORD)
    h = (h + j * GOLD) % WORD
    h = (h ^ (h >> 16)) * (math.isqrt(2 << 64) % WORD) % WORD
    h ^= h >> 15
    q = h * (math.isqrt(3 << 64) % WORD) % WORD
    return h % 65536, h >> 16, (q ^ (q >> 16)) % 65536


def octave(x):
    """floor(log2 |x|) of x != 0."""
    return math.frexp(x)[1] - 1


def block_exponent(xs, second):
    """The shared exponent byte of a block."""
    top = 31 if second else 15
    most = max(abs(x) for x in xs)
    if most == 0:
        return top + 1
    mant, e = math.frexp(most)
    return max(top + 1, e - 1 + (1 if mant > 0.9375 else 0) + 127)


def encode(x, byte, second, r):
    """(code, distance of the place from the next border, in steps)."""
    top = 31 if second else 15
    if x == 0:
        return 0, 1.0
    e = octave(x)
    place = abs(x) / 2.0 ** (e - 3) + (16 * r + 8) / 2.0 ** 20  # in [8, 17)
    c = math.floor(place) - 8 + 8 * (e - (byte - 127 - top))
    c = min(max(c, 1 if second else 0), 8 * top + 7)
    return (c + 128 if x < 0 and c > 0 and not second else c), abs(place - round(place))


def decode(code, byte, second):
    top = 31 if second else 15
    c = code if second else code & 127
    if c == 0:
        return 0.0
    x = (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - top + byte - 127)
    return -x if not second and code > 127 else x


def round_bf16(x, r):
    """x rounded up (in magnitude) to bf16 with random bits r, and the distance to the border."""
    if x == 0:
        return 0.0, 1.0
    step = 2.0 ** (max(octave(x), -126) - 7)
    place = abs(x) / step + r / 65536
    return math.copysign(math.floor(place) * step, x), abs(place - round(place))


# ------------------------------------------------------------------- AdamW
def adamw(w, g, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, decay=0.0, factor=1.0):
    """One step in fp64 (NumPy arrays): the new w, m, v before any rounding."""
    g = factor * np.asarray(g, np.float64)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = m / (1 - beta1 ** step)
    den = np.sqrt(v / (1 - beta2 ** step)) + eps
    return w - lr * (decay * w + hat / den), m, v
