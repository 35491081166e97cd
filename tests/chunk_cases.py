"""Inputs that show single bits of the chunked form's operand splits, and a
model of that form in numpy.

The chunked form of ss_prefill cuts fp32 operands into three bf16 parts: the
state S, the residuals R, the stacked [P T; T] and t o U; R with [P T; T]
takes the six products whose parts' numbers add up to at most 2.  On random
tokens a lost part hides behind sums of many roundings.  Here keys and queries
are rows of the identity, so that every sum has one or two terms that are not
zero and what is left is the operand itself, with all its 24 bits:

  read     S <- S, o = a row of S                                (S)
  write    S[r] <- S[r] + b (v - S[r]), o = the new row          (S, R, t o U)
  pair     o = a u_0 from a zero state, u_0 = b v                (R with P T)
  solve    two tokens with one key, from a zero state            (R with T)
  decay    Mamba-2: o = dt v, S[r] = dt v, from a zero state     (P, t o U)

Room.  e = 2^-24.  An elementwise fp32 operation is off by at most e of its
result; an MMA adds to an fp32 accumulator, which may drop what lies below its
last place (2 e of the accumulator, whatever the hardware's rounding); terms
that are zero add nothing.  A contraction with three parts is three such
additions, the first onto zero: 4 e.  R with [P T; T]: six additions, 12 e, and
the products left out, 8 e (2^-21).
  read     S^T q 4, the sum's rounding 1                                 5 e |S[r]|
  write    S^T k 4, R 2, with T's 1: 4, t o U 1 + 4, the sum's 1: 16     16 e (|S[r]| + |v|)
           o: S^T q 4, R's share 10, the sum's 1 more                    16 e (|S[r]| + |v|)
  pair     R 2, with a 12 + 8, the sum's 1: 23; S: y 1 + 4, 1: 29        30 e |u_0|
  solve    T and P T 2 each, R 2, products 20, sums as above: 33         36 e M
  decay    P 2 (D and dt), 4 with v, the sum's 1: 7; S: 1 + 4 + 1        8 e dt |v|
M adds the magnitudes of the terms.  Losing a part costs 2^-17 of the operand
on average, 2^-15 at worst: 128 e and more.
"""
import numpy as np

from ssm_decode_b200 import synth
from tests import many_token_util as U

E = 2.0 ** -24
C = 64
PAIRS = [(i, j) for i in range(3) for j in range(3 - i)]


def make(name, family, dk, dv, lead, seed=0, heads=4):
    """Inputs of one sequence of lead + 64 tokens (see many_token_util.draw), its
    state, and the room of the outputs [T][H][dv] and of the state [H][dk][dv]."""
    r = np.random.default_rng([seed, dk, dv, lead, len(name)])
    T = lead + C
    S = r.standard_normal((heads, dk, dv)).astype(np.float32)
    q, k = np.zeros((T, heads, dk)), np.zeros((T, heads, dk))
    q[:, :, 0] = 1
    d = {"gate": np.full((T, heads), 0 if family == synth.MAMBA2 else 1, np.float32), "beta": np.zeros((T, heads), np.float32),
         "A": np.full(heads, -1, np.float32)}
    d["v"], d["v_"] = U.bf16(r.standard_normal((T, heads, dv)))
    frac = lambda *s: r.uniform(0.25, 1, s).astype(np.float32)  # noqa: E731
    out_room, S_room = np.zeros((T, heads, dv)), np.zeros((heads, dk, dv))
    i = np.arange(C)
    if name == "read":
        k[:] = r.standard_normal(k.shape)
        q[:] = 0
        for t in range(T):
            q[t, :, (5 * t) % dk] = 1
            out_room[t] = 5 * E * np.abs(S[:, (5 * t) % dk])
    elif name == "write":
        rows = r.permutation(dk)[:C]
        q[lead:] = 0
        q[lead + i, :, rows] = k[lead + i, :, rows] = 1
        d["beta"][lead:] = frac(C, heads)
        q[:lead] = 0
        M = np.abs(S[:, rows].transpose(1, 0, 2)) + np.abs(d["v_"][lead:])
        out_room[lead:] = 16 * E * M
        S_room[:, rows] = 16 * E * M.transpose(1, 0, 2)
    else:
        S[:] = 0
        k[lead, :, 0] = 1
        v0 = np.abs(d["v_"][lead])
        if name == "decay":
            d["gate"][lead] = frac(heads)
            M = d["gate"][lead].astype(np.float64)[:, None] * v0
            out_room[lead:], S_room[:, 0] = 8 * E * M, 8 * E * M
        else:
            d["beta"][lead] = frac(heads)
            d["gate"][lead + 1] = frac(heads)
            u0 = d["beta"][lead].astype(np.float64)[:, None] * v0
            room = 30 * E * u0
            if name == "solve":
                k[lead + 1, :, 0] = 1
                d["beta"][lead + 1] = frac(heads)
                b1 = d["beta"][lead + 1].astype(np.float64)[:, None]
                room = 36 * E * (u0 * (1 + b1) + b1 * np.abs(d["v_"][lead + 1]))
            out_room[lead:], S_room[:, 0] = room, room
    for n, x in (("q", q), ("k", k)):
        d[n], d[n + "_"] = U.bf16(x)
    return d, S, out_room, S_room


def names(family):
    return ["read", "decay"] if family == synth.MAMBA2 else ["read", "write", "pair", "solve"]


def parts(x, n=3):
    """The first n bf16 parts of fp32 values, each the leading 16 bits of what is left."""
    x, out = np.asarray(x, np.float32), []
    for _ in range(n):
        p = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out.append(p.astype(np.float64))
        x = x - p
    return out


def model(family, d, S, cut_S=3, cut_U=3, pairs=PAIRS):
    """The chunked form with exact sums and the kernel's elementwise roundings:
    out [T][H][dv] and the state behind the last token."""
    f = lambda x: np.asarray(x, np.float32).astype(np.float64)  # noqa: E731
    T, H = d["gate"].shape
    group = H // d["q_"].shape[1]
    out = np.zeros((T, H, S.shape[2]))
    S = S.astype(np.float64).copy()
    m2 = family == synth.MAMBA2
    for h in range(H):
        for c in range(0, T, C):
            s = slice(c, c + C)
            q, k, v = d["q_"][s, h // group], d["k_"][s, h // group], d["v_"][s, h]
            x = d["gate"][s, h].astype(np.float64)
            a, b = (f(np.exp(f(x * d["A"][h]))), x) if m2 else (x, d["beta"][s, h].astype(np.float64))
            n = len(a)
            g = f(np.cumprod(a))
            t = f(np.append(np.cumprod(a[::-1])[::-1][1:], 1))
            D = np.zeros((n, n))
            for i in range(n):
                D[i, :i + 1] = f(np.append(np.cumprod(a[i:0:-1])[::-1], 1))
            P, A = f(D * (q @ k.T)), f(np.tril(b[:, None] * D * (k @ k.T), -1))
            S_ = sum(parts(S[h], cut_S))
            if m2:
                Y, inner, whole = f(b[:, None] * v), f(P * b), sum(parts(f(P * b), 1 + max(j for i, j in pairs if i == 0))) @ v
            else:
                inv = f(np.linalg.inv(np.eye(n) + A))
                R = f(b[:, None] * f(v - g[:, None] * f(k @ S_)))
                rp, pt, tt = parts(R), parts(f(P @ inv)), parts(inv)
                whole = f(sum(pt[j] @ rp[i] for i, j in pairs))
                Y = f(sum(tt[j] @ rp[i] for i, j in pairs))
            out[s, h] = f(g[:, None] * f(q @ S_) + f(whole))
            S[h] = f(g[-1] * S[h] + f(k.T @ sum(parts(f(t[:, None] * Y), cut_U))))
    return out, S
