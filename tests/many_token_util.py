"""Plain 64-bit forms of the many-token calls, for the tests: one token, one
head at a time, straight from the definitions in include/sketchssm.h.

Tolerances.  The kernels keep states, products and sums in fp32 (unit
round-off e = 2^-24) or in operand splits whose dropped part is below it.  A
state entry is a sum over T tokens of products of contractions of dk terms;
each of the T + dk roundings on the way is off by at most e relative to the
largest magnitude it meets, and the decays (<= 1 here) shrink earlier ones, so
the worst error is (T + dk) e of the head's largest entry; ROOM = 4 covers the
erase term's echo of an error through k . S and the output's own sum.
"""
import numpy as np

from ssm_decode_b200 import synth

ROOM = 4.0


def tolerance(tokens, dk):
    return ROOM * (tokens + dk) * 2.0 ** -24


def bf16(x):
    """float array -> (bf16 bits, the values they hold as fp64)."""
    bits = synth.f32_to_bf16_bits(np.asarray(x, np.float32))
    return bits, synth.bf16_bits_to_f32(bits).astype(np.float64)


def run_tokens(family, S, q, k, v, gate, beta, A):
    """Tokens q, k [T][H][dk], v [T][H][dv] through state S [H][dk][dv], all
    fp64 values; returns (out [T][H][dv], the state behind them)."""
    S = S.copy()
    out = np.zeros(v.shape)
    for t in range(v.shape[0]):
        for h in range(S.shape[0]):
            if family == synth.MAMBA2:
                S[h] = np.exp(gate[t, h] * A[h]) * S[h] + gate[t, h] * np.outer(k[t, h], v[t, h])
            else:
                S[h] = gate[t, h, :, None] * S[h] if family == synth.KDA else gate[t, h] * S[h]
                S[h] = S[h] + np.outer(k[t, h], beta[t, h] * (v[t, h] - k[t, h] @ S[h]))
            out[t, h] = q[t, h] @ S[h]
    return out, S


def draw(family, rows, heads, qk_heads, dk, dv, seed):
    """Inputs of `rows` tokens: bf16 bits and fp64 values of q, k, v; gate, beta, A fp32."""
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    q, k = unit(r.standard_normal((rows, qk_heads, dk))), unit(r.standard_normal((rows, qk_heads, dk)))
    v = r.standard_normal((rows, heads, dv))
    if family == synth.MAMBA2:
        gate = np.logaddexp(0, r.standard_normal((rows, heads)) - 2)
    else:
        gate = 1 / (1 + np.exp(-r.standard_normal((rows, heads, dk) if family == synth.KDA else (rows, heads)) - 1))
    beta = 1 / (1 + np.exp(-r.standard_normal((rows, heads))))
    A = -np.exp(r.uniform(0, 2, heads))
    d = {"gate": gate.astype(np.float32), "beta": beta.astype(np.float32), "A": A.astype(np.float32)}
    for name, x in (("q", q), ("k", k), ("v", v)):
        d[name], d[name + "_"] = bf16(x)
    return d


def reference(family, state, d, lengths, fresh, first=0):
    """Expected output rows (fp64, NaN where no sequence has the row) and states."""
    heads = state.shape[1]
    rows = d["v_"].shape[0]
    group = heads // d["q_"].shape[1]
    out = np.full((rows, heads, state.shape[3]), np.nan)
    S = state.astype(np.float64).copy()
    at = first
    for b, n in enumerate(lengths):
        s = slice(at, at + n)
        q, k = (np.repeat(d[x][s], group, axis=1) for x in ("q_", "k_"))
        out[s], S[b] = run_tokens(family, np.zeros_like(S[b]) if fresh[b] else S[b], q, k, d["v_"][s],
                                  d["gate"][s].astype(np.float64), d["beta"][s].astype(np.float64),
                                  d["A"].astype(np.float64))
        at += n
    return out, S


def quantise(x, bits):
    """(codes, scales fp64) of values whose last axis is a multiple of 32, by exact quotients."""
    m = 127 if bits == 8 else 7
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(g).max(-1)
        scale = synth.bf16_bits_to_f32(synth.f32_to_bf16_bits((top / np.float32(m)).astype(np.float32))).astype(np.float64)
    scale = np.where(np.isfinite(top), scale, np.nan)
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.clip(np.rint(g.astype(np.float64) / scale[..., None]), -m, m)
    c = np.where((scale > 0)[..., None], c, 0)
    return c.astype(np.int64).reshape(x.shape), scale


def held(x, bits):
    """The values a slot holds of x."""
    c, s = quantise(x, bits)
    return (c.reshape(*x.shape[:-1], -1, 32) * s[..., None]).reshape(x.shape)
