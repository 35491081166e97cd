"""Cases of the operators that carry a linear-attention layer's state over many tokens and in and out of a cache.

Two entry points of a decode layer are called: `prefill` (the recurrence over a packed, ragged batch of token rows; the
chunked form for prompts and the recurrent one for the few tokens of a verification step) and `save` / `restore` (the
states of the batch into and out of slots that hold them in 8 or 4 bits).

  prefill   per token, S <- M S + b k v^T and o = S^T q, with
            mamba2: M = a, a = exp(dt A), b = dt;  gdn: M = a (I - beta k k^T), b = beta;
            kda: M = (I - beta k k^T) Diag(a), b = beta
  cache     groups of 32 values along dv: scale = bf16(fp32(max|x| / m)), m = 127 or 7; code = the whole number nearest
            to x / scale (ties to even); the value held is code * scale
"""
import math

import numpy as np
import torch

own = False

FAMILIES = {"mamba2": 0, "gdn": 1, "kda": 2}
GROUP = 32


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one long prompt of a single user: 32 heads are all the parallelism there is
        dict(name="gdn_prompt_8k", op="prefill", family="gdn", batch=1, heads=32, qk_heads=32, dk=128, dv=128,
             lo=8192, hi=8192, out="bf16", fresh=1.0, pad=0),
        # prompts of unequal lengths packed into one call, some continued from a cached prefix, the rows padded behind them
        dict(name="gdn_ragged_16", op="prefill", family="gdn", batch=16, heads=32, qk_heads=32, dk=128, dv=128,
             lo=1, hi=4096, out="f32", fresh=0.5, pad=37),
        # a layer whose key heads are shared by two value heads, odd lengths
        dict(name="gdn_shared_keys_8", op="prefill", family="gdn", batch=8, heads=32, qk_heads=16, dk=128, dv=128,
             lo=900, hi=1100, out="bf16", fresh=1.0, pad=0),
        # the 128-head Mamba-2 layer on a few prompts
        dict(name="mamba2_prompt_2k", op="prefill", family="mamba2", batch=4, heads=128, qk_heads=128, dk=128, dv=64,
             lo=1900, hi=2048, out="bf16", fresh=1.0, pad=0),
        # per-channel decay
        dict(name="kda_prompt_512", op="prefill", family="kda", batch=8, heads=32, qk_heads=32, dk=128, dv=128,
             lo=300, hi=512, out="bf16", fresh=1.0, pad=0),
        # verifying a draft of four tokens on the full decode batch
        dict(name="gdn_verify_4", op="prefill", family="gdn", batch=256, heads=32, qk_heads=32, dk=128, dv=128,
             lo=4, hi=4, out="f32", fresh=0.0, pad=0),
        # one token for every sequence of the Mamba-2 decode batch
        dict(name="mamba2_one_token", op="prefill", family="mamba2", batch=320, heads=128, qk_heads=128, dk=128, dv=64,
             lo=1, hi=1, out="f32", fresh=0.0, pad=0),
        # the smallest call: four small sequences, up to three tokens each; latency is all there is
        dict(name="gdn_tiny_verify", op="prefill", family="gdn", batch=4, heads=4, qk_heads=4, dk=64, dv=64,
             lo=0, hi=3, out="f32", fresh=0.25, pad=0),
        # the whole decode batch swapped out and in again
        dict(name="swap_8bit_gdn", op="swap", family="gdn", batch=256, heads=32, dk=128, dv=128, bits=8, skip=0.0),
        # part of a Mamba-2 batch preempted, at 4 bits
        dict(name="swap_4bit_mamba2", op="swap", family="mamba2", batch=100, heads=128, dk=128, dv=64, bits=4, skip=0.3),
        # new sequences that share a few cached prefixes
        dict(name="restore_4bit_shared", op="restore", family="gdn", batch=128, heads=32, dk=128, dv=128, bits=4,
             slots=5, skip=0.0),
        # a single sequence resumed from its prefix
        dict(name="restore_8bit_one", op="restore", family="gdn", batch=1, heads=32, dk=128, dv=128, bits=8, slots=3,
             skip=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    family = rng.choice(["gdn", "gdn", "mamba2", "kda"])
    dk, dv = rng.choice([(128, 128), (128, 128), (128, 64), (64, 128), (64, 64)])
    op = rng.choice(["prefill", "prefill", "few", "swap", "restore"])
    heads = _log(rng, 1, 128 if family == "mamba2" else 48)
    if op == "prefill":
        shared = rng.choice([1, 1, 2])
        heads = max(shared, heads // shared * shared)
        batch = _log(rng, 1, 48)
        hi = _log(rng, 17, 600 if family == "kda" else 8192)
        hi = max(17, min(hi, 500_000 // (batch * heads)))
        lo = rng.choice([0, 1, hi, max(1, hi - rng.randrange(1, 100))])
        return dict(op="prefill", family=family, batch=batch, heads=heads, qk_heads=heads // shared, dk=dk, dv=dv,
                    lo=lo, hi=hi, out=rng.choice(["bf16", "f32"]), fresh=rng.choice([0.0, 0.5, 1.0]),
                    pad=rng.choice([0, 5]))
    batch = _log(rng, 1, 320)
    batch = max(1, min(batch, 8192 // heads))
    if op == "few":
        hi = rng.randrange(1, 17)
        return dict(op="prefill", family=family, batch=batch, heads=heads, qk_heads=heads, dk=dk, dv=dv,
                    lo=rng.choice([0, hi]), hi=hi, out=rng.choice(["bf16", "f32"]), fresh=rng.choice([0.0, 0.5]),
                    pad=rng.choice([0, 3]))
    c = dict(op=op, family=family, batch=batch, heads=heads, dk=dk, dv=dv, bits=rng.choice([8, 4]),
             skip=rng.choice([0.0, 0.0, 0.3]))
    if op == "restore":
        c["slots"] = rng.randrange(1, 20)
    return c


# --------------------------------------------------------------------------- inputs
def _lengths(case):
    """The lengths of a case's sequences: a user's batch, not a random input, so the same for every seed."""
    r = np.random.default_rng(case["batch"] * 1000 + case["hi"])
    lo, hi, B = case["lo"], case["hi"], case["batch"]
    if hi - lo < 256 or lo > 1:
        n = r.integers(lo, hi + 1, size=B)
    else:                                                  # spread over the logarithm
        n = np.exp(r.uniform(0, math.log(hi + 1), size=B)).astype(np.int64)
        n = np.clip(n, lo, hi)
    if lo != hi:
        n[0] = hi
        n[1:2] = lo
    return n


def _mask(case, key, share):
    return np.random.default_rng(case["batch"] * 7 + key).random(case["batch"]) < share


def _rand(seed, key):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 64 + key)
    return lambda *shape: torch.randn(shape, device="cuda", generator=g)


def _state(case, seed):
    return _rand(seed, 0)(case["batch"], case["heads"], case["dk"], case["dv"]) * math.sqrt(0.1)


def _slots(case):
    """Slot of each sequence (-1: not moved) and the number of slots."""
    B = case["batch"]
    r = np.random.default_rng(B * 11 + 1)
    n = B + 3 if case["op"] == "swap" else case["slots"]
    s = r.permutation(n)[:B] if case["op"] == "swap" else r.integers(0, n, size=B)
    s[_mask(case, 3, case["skip"])] = -1
    return s.astype(np.int32), n


def prepare(case, seed):
    if case["op"] == "prefill":
        n = _lengths(case)
        rows, H, Hq, K, V = int(n.sum()) + case["pad"], case["heads"], case["qk_heads"], case["dk"], case["dv"]
        unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
        s = {"case": case, "max": int(n.max())}
        q, k = _rand(seed, 1)(rows, Hq, K), _rand(seed, 2)(rows, Hq, K)
        if case["family"] == "mamba2":
            s["q"], s["k"] = (q / math.sqrt(K)).bfloat16(), (k / math.sqrt(K)).bfloat16()
            s["gate"] = torch.nn.functional.softplus(_rand(seed, 4)(rows, H) - 2)
            s["beta"] = None
            s["A"] = -torch.exp(2 * torch.rand(H, device="cuda", generator=torch.Generator("cuda").manual_seed(seed * 64 + 6)))
        else:
            s["q"], s["k"] = unit(q).bfloat16(), unit(k).bfloat16()
            shape = (rows, H, K) if case["family"] == "kda" else (rows, H)
            s["gate"] = torch.sigmoid(_rand(seed, 4)(*shape))        # exp(-softplus(-x))
            s["beta"] = torch.sigmoid(_rand(seed, 5)(rows, H))
            s["A"] = None
        s["v"] = _rand(seed, 3)(rows, H, V).bfloat16()
        s["out"] = torch.zeros(rows, H, V, device="cuda", dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        s["start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
        s["fresh"] = torch.from_numpy(_mask(case, 2, case["fresh"]).astype(np.int32)).cuda()
        s["state"] = _state(case, seed)
    else:
        slots, count = _slots(case)
        s = {"case": case, "A": None, "slots": torch.from_numpy(slots).cuda(), "state": _state(case, seed)}
        H, K, V = case["heads"], case["dk"], case["dv"]
        held = _rand(seed, 7)(count, H, K, V) if case["op"] == "restore" else None
    if own:
        import ssm_decode_b200 as ss
        layer = lambda batch: ss.DecodeLayer(FAMILIES[case["family"]], batch, case["heads"], case["dk"], case["dv"], 16,  # noqa: E731
                                             [1] * case["heads"])
        s["layer"] = layer(case["batch"])
        s["layer"].load(state=s.pop("state"), A=s["A"])
        if case["op"] != "prefill":
            s["cache"] = ss.StateCache(s["layer"], count, bits=case["bits"])
        if case["op"] == "restore":
            filler = layer(count)
            filler.load(state=held)
            filler.save(s["cache"], torch.arange(count, device="cuda", dtype=torch.int32))
    elif case["op"] != "prefill":
        s["codes"] = torch.zeros(count + 1, H, K, V, device="cuda", dtype=torch.int8)
        s["scales"] = torch.zeros(count + 1, H, K, V // GROUP, device="cuda", dtype=torch.bfloat16)
        if held is not None:
            s["codes"], s["scales"] = _quantise(held, case["bits"])
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        layer = s["layer"]
        if case["op"] == "prefill":
            layer.prefill(s["q"], s["k"], s["v"], s["gate"], s["beta"], s["start"], max_tokens=s["max"],
                          fresh=s["fresh"], out=s["out"])
            return {"out": s["out"], "state": layer.state}
        if case["op"] == "swap":
            layer.save(s["cache"], s["slots"])
        layer.restore(s["cache"], s["slots"])
        return {"state": layer.state}
    if case["op"] == "prefill":
        _tokens(s) if case["family"] == "kda" or s["max"] <= 16 else _chunks(s)
        return {"out": s["out"], "state": s["state"]}
    slots = s["slots"].long()
    if case["op"] == "swap":
        codes, scales = _quantise(s["state"], case["bits"])
        # sequences with no slot write the row behind the last slot
        to = torch.where(slots >= 0, slots, len(s["codes"]) - 1)
        s["codes"][to], s["scales"][to] = codes, scales
    at = slots.clamp_min(0)
    values = s["codes"][at].float().unflatten(-1, (-1, GROUP)) * s["scales"][at].float().unsqueeze(-1)
    s["state"].copy_(torch.where((slots >= 0)[:, None, None, None], values.flatten(-2), s["state"]))
    return {"state": s["state"]}


def _quantise(x, bits):
    m = 127 if bits == 8 else 7
    g = x.unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1).double() / m).float().bfloat16()
    # 64 bits: the quotient next to a border between two codes
    codes = torch.round(g.double() / scale.double().unsqueeze(-1)).clamp(-m, m)
    return torch.where(scale.unsqueeze(-1) > 0, codes, 0).to(torch.int8).flatten(-2), scale


def _rows(s, at, n):
    """Rows at..at+n-1 of every sequence in 32 bits, [B, heads, n, ...]: those behind its end are rows that change nothing."""
    case = s["case"]
    first, last = s["start"][:-1].long(), s["start"][1:].long()
    idx = first[:, None] + torch.arange(at, at + n, device="cuda")
    ok = idx < last[:, None]
    idx = torch.where(ok, idx, 0)
    live = ok[:, None, :, None]
    take = lambda x, r: torch.where(live, x[idx].float().transpose(1, 2).repeat_interleave(r, 1), 0)  # noqa: E731
    r = case["heads"] // case["qk_heads"]
    gate = s["gate"][idx].transpose(1, 2)
    if case["family"] == "mamba2":
        a, b = torch.exp(gate * s["A"][None, :, None]), gate
    else:
        a, b = gate, s["beta"][idx].transpose(1, 2)
    ok = ok[:, None, :]
    a = torch.where(ok[..., None] if a.dim() == 4 else ok, a, 1)
    return idx, ok, take(s["q"], r), take(s["k"], r), take(s["v"], 1), a, torch.where(ok, b, 0)


def _put(s, idx, ok, o):
    """Rows o [B, heads, n, dv] into the output; those behind a sequence's end go nowhere."""
    rows = torch.where(ok[:, 0], idx, len(s["out"])).reshape(-1)
    wide = torch.cat([s["out"], s["out"][:1]]) if len(s["out"]) else s["out"].new_zeros(1, *s["out"].shape[1:])
    wide[rows] = o.transpose(1, 2).reshape(-1, *o.shape[1:2], o.shape[-1]).to(wide.dtype)
    s["out"].copy_(wide[:-1])


def _first_state(s):
    return torch.where((s["fresh"] > 0)[:, None, None, None], 0, s["state"])


def _tokens(s):
    S, family = _first_state(s), s["case"]["family"]
    idx, ok, Q, K, V, a, b = _rows(s, 0, max(1, s["max"]))
    outs = []
    for t in range(Q.shape[2]):
        k, v, q = K[:, :, t], V[:, :, t], Q[:, :, t]
        S = S * (a[:, :, t, :, None] if family == "kda" else a[:, :, t, None, None])
        u = v if family == "mamba2" else v - (k.unsqueeze(-2) @ S).squeeze(-2)
        S = S + k.unsqueeze(-1) * (b[:, :, t, None] * u).unsqueeze(-2)
        outs.append((q.unsqueeze(-2) @ S).squeeze(-2))
    _put(s, idx, ok, torch.stack(outs, 2))
    s["state"].copy_(S)


def _chunks(s, C=64):
    S, family = _first_state(s), s["case"]["family"]
    lower = torch.ones(C, C, device="cuda").tril()
    eye = torch.eye(C, device="cuda")
    out, put, good = [], [], []
    for at in range(0, s["max"], C):
        idx, ok, Q, K, V, a, b = _rows(s, at, C)
        g = torch.cumsum(torch.log(a.double()), -1)                       # 64 bits: a long sum of logarithms
        D = torch.where(lower > 0, torch.exp(torch.where(lower > 0, g[..., :, None] - g[..., None, :], 0)), 0).float()
        tail, whole, g = torch.exp(g[..., -1:] - g).float(), torch.exp(g[..., -1]).float(), torch.exp(g).float()
        U = b[..., None] * V
        if family != "mamba2":
            U = U - (b * g)[..., None] * (K @ S)
            P = -(b[..., None] * (K @ K.mT) * D).tril(-1)                 # (I - P)^-1 = (I + P)(I + P^2)(I + P^4)...
            T = eye + P
            for _ in range(int(math.log2(C)) - 1):
                P = P @ P
                T = T + T @ P
            U = T @ U
        out.append((g[..., None] * (Q @ S) + ((Q @ K.mT) * D) @ U).to(s["out"].dtype))
        put.append(idx)
        good.append(ok)
        S = whole[..., None, None] * S + (K * tail[..., None]).mT @ U
    _put(s, torch.cat(put, 1), torch.cat(good, 2), torch.cat(out, 2))
    s["state"].copy_(S)


# --------------------------------------------------------------------------- floor and exact values
def work(case):
    B, H, K, V = case["batch"], case["heads"], case["dk"], case["dv"]
    values = B * H * K * V
    if case["op"] == "prefill":
        lengths = _lengths(case)
        n, fresh = int(lengths.sum()), _mask(case, 2, case["fresh"])
        e = 2 if case["out"] == "bf16" else 4
        gate = K * 4 if case["family"] == "kda" else 4
        token = case["qk_heads"] * 2 * K * 2 + H * (V * 2 + V * e + gate + (0 if case["family"] == "mamba2" else 4))
        # a state is read unless the sequence starts afresh, and written unless nothing changes it
        states = (lengths[~fresh] > 0).sum() + ((lengths > 0) | fresh).sum()
        per = 4 if case["family"] == "mamba2" else 6          # the recurrence's products: S^T k, + k u^T, S^T q
        return {"bytes": n * token + int(states) * (values // B) * 4, "flops": n * H * K * V * per}
    moved = float((_slots(case)[0] >= 0).mean()) * values
    held = case["bits"] / 8 + 2 / GROUP
    if case["op"] == "swap":
        return {"bytes": moved * (8 + 2 * held), "flops": moved * 4}
    # a slot that several sequences share is read once
    s = _slots(case)[0]
    return {"bytes": moved * 4 + len(set(s[s >= 0])) * H * K * V * held, "flops": moved}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    S = s["state"].double()
    if case["op"] != "prefill":
        slots = _slots(case)[0]
        m = 127 if case["bits"] == 8 else 7
        for b, slot in enumerate(slots.tolist()):
            if slot < 0:
                continue
            if case["op"] == "restore":                       # what the slot was given, as prepare() gave it
                codes, scale = s["codes"][slot].double(), s["scales"][slot].double()
            else:
                rows = S[b].reshape(*S[b].shape[:-1], -1, GROUP)
                scale = (rows.abs().amax(-1) / m).float().bfloat16().double()
                codes = (rows / scale[..., None]).round().clamp(-m, m).reshape(S[b].shape)
            S[b] = codes * scale.repeat_interleave(GROUP, -1)
        return {"state": S}
    n = _lengths(case)
    H, family, r = case["heads"], case["family"], case["heads"] // case["qk_heads"]
    S[torch.from_numpy(_mask(case, 2, case["fresh"]))] = 0
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])[:-1]).cuda()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    # sequences by falling length: those still running are the first ones, and their states a slice
    order = np.argsort(-n, kind="stable")
    S, first = S[order], first[order]
    for t in range(int(n.max(initial=0))):
        m = int((n > t).sum())
        row = first[:m] + t
        q, k = (s[x][row].double().repeat_interleave(r, 1) for x in "qk")
        v, gate = s["v"][row].double(), s["gate"][row].double()
        T = S[:m]
        if family == "mamba2":
            T *= torch.exp(gate * s["A"].double())[..., None, None]
            u = gate[..., None] * v
        else:
            T *= gate[..., None] if family == "kda" else gate[..., None, None]
            u = s["beta"][row].double()[..., None] * (v - torch.einsum("bhk,bhkv->bhv", k, T))
        T += k[..., None] * u[..., None, :]
        out[row] = torch.einsum("bhk,bhkv->bhv", q, T)
    back = torch.empty_like(S)
    back[order] = S
    return {"out": out, "state": back}
