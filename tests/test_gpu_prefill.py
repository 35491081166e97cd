"""GPU parity of ss_prefill against the plain 64-bit recurrence (needs a B200).

Both forms of the call run on the same cases: token by token (max_tokens = 1
asks for it) and the form the library picks for long sequences (max_tokens
far above them).  Lengths from zero on, around the chunk length and odd; sequences
that start afresh or go on; rows of no sequence, which hold NaN; shared key
heads, strided rows, both output types; decays of exactly 0 and 1.
"""
import numpy as np
import pytest

from ssm_decode_b200 import binding as B
from ssm_decode_b200 import synth
from ssm_decode_b200.layer import DecodeLayer, StateCache
from tests import many_token_util as U

pytestmark = pytest.mark.gpu

FAM = {"mamba2": synth.MAMBA2, "gdn": synth.GDN, "kda": synth.KDA}
LENGTHS = [65, 0, 1, 130, 64, 7, 63]


def dev(x):
    import torch
    x = np.ascontiguousarray(x)
    return torch.from_numpy(x.view(np.int16) if x.dtype == np.uint16 else x).cuda()


def make_layer(family, batch, heads, dk, dv, A, seed, window=4):
    rng = np.random.default_rng(seed)
    state = (rng.standard_normal((batch, heads, dk, dv)) * 0.3).astype(np.float32)
    lay = DecodeLayer(family, batch, heads, dk, dv, window, [2] * heads)
    basis = rng.standard_normal((2 * heads, dk)).astype(np.float32)
    lay.load(state=state, basis=basis, coef=basis, A=A)
    return lay, state


def starts(lengths, first=0):
    return dev((first + np.concatenate([[0], np.cumsum(lengths)])).astype(np.int32))


def check(got, ref, tol, out_bf16=False):
    """Elementwise against the largest entry of the reference."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    if not ref.size:
        return
    room = tol * max(np.abs(ref).max(), 1e-30) + (2.0 ** -8 * np.abs(ref) if out_bf16 else 0)
    bad = ~(np.abs(got - ref) <= room)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref)):.3e} of {np.abs(ref).max():.3e}"


def run_case(family, heads, qk_heads, dk, dv, lengths, fresh, seed, form, out_dtype="f32", first=0, pad=3,
             change=None, layer=None):
    import torch
    rows = first + sum(lengths) + pad
    d = U.draw(family, rows, heads, qk_heads, dk, dv, seed)
    if change:
        change(d)
    lay, state = layer or make_layer(family, len(lengths), heads, dk, dv, d["A"], seed)
    ref_out, ref_S = U.reference(family, state, d, lengths, fresh, first)
    used = np.zeros(rows, bool)
    used[first:first + sum(lengths)] = True
    nan16 = np.uint16(0x7FC0)
    for n in ("q", "k", "v"):
        d[n][~used] = nan16
    d["gate"][~used] = np.nan
    d["beta"][~used] = np.nan
    out = torch.full((rows, heads, dv), 7.0, device="cuda",
                     dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32)
    lay.prefill(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["gate"]),
                None if family == synth.MAMBA2 else dev(d["beta"]), starts(lengths, first),
                max_tokens=1 if form == "tokens" else 1 << 20, fresh=dev(np.asarray(fresh, np.int32)), out=out)
    torch.cuda.synchronize()
    o, S = out.float().cpu().numpy(), lay.state.cpu().numpy()
    tol = U.tolerance(max(list(lengths) + [1]), dk)
    assert (o[~used] == 7.0).all(), "rows of no sequence were written"
    for b in range(len(lengths)):
        check(S[b], ref_S[b], tol)
        if lengths[b] == 0:
            assert (S[b] == (0 if fresh[b] else state[b])).all()
    for h in range(heads):
        check(o[used][:, h], ref_out[used][:, h], tol, out_dtype == "bf16")
    assert int(lay.status[0]) == 0
    return lay


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("family", list(FAM))
def test_ragged_batch(cuda_ok, family, dk, dv, form):
    run_case(FAM[family], 3, 3, dk, dv, LENGTHS, [0, 1, 0, 1, 0, 0, 1], 40 + dk + dv, form)


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 127, 128, 129, 200])
@pytest.mark.parametrize("family", list(FAM))
def test_lengths(cuda_ok, family, n, form):
    run_case(FAM[family], 2, 2, 128, 128, [n], [0], 100 + n, form, pad=0)


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("family", list(FAM))
def test_shared_key_heads_bf16_out_and_offset_rows(cuda_ok, family, form):
    run_case(FAM[family], 4, 2, 128, 128, [70, 5], [0, 1], 7, form, out_dtype="bf16", first=2)
    run_case(FAM[family], 4, 1, 64, 64, [3, 66], [0, 1], 8, form, out_dtype="bf16", first=1)


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("family", ["gdn", "kda"])
def test_decays_of_zero_and_one_and_no_update(cuda_ok, family, form):
    def change(d):
        r = np.random.default_rng(5)
        d["gate"][r.random(d["gate"].shape) < 0.1] = 0
        d["gate"][r.random(d["gate"].shape) < 0.3] = 1
        d["beta"][r.random(d["beta"].shape) < 0.2] = 0
        d["beta"][r.random(d["beta"].shape) < 0.2] = 1
    run_case(FAM[family], 3, 3, 128, 128, [100, 64, 20], [0, 0, 1], 9, form, change=change)


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("family", ["gdn", "kda"])
def test_tiny_decays(cuda_ok, family, form):
    """Products of decays that leave the fp32 range."""
    def change(d):
        d["gate"][:] = np.where(np.random.default_rng(6).random(d["gate"].shape) < 0.7, 1e-12, 0.9)
    run_case(FAM[family], 2, 2, 128, 128, [90, 64], [0, 1], 10, form, change=change)


@pytest.mark.parametrize("form", ["tokens", "long"])
def test_equal_keys(cuda_ok, form):
    """One key for every token, beta = 1: each token replaces what the last one stored."""
    def change(d):
        for n in ("k", "k_"):
            d[n][:] = d[n][:1]
        d["gate"][:] = 1
        d["beta"][:] = 1
    run_case(synth.GDN, 2, 2, 128, 128, [150], [0], 11, form, change=change)


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("family", list(FAM))
def test_strided_rows(cuda_ok, family, form):
    """Column ranges of fused projections; the result is that of dense rows bit for bit."""
    import torch
    fam, H, K, V, n = FAM[family], 2, 64, 64, 81
    d = U.draw(fam, n, H, H, K, V, 12)
    t = {x: dev(d[x]) for x in ("q", "k", "v", "gate", "beta")}
    got = []
    for strided in (False, True):
        lay, _ = make_layer(fam, 1, H, K, V, d["A"], 12)
        out = torch.zeros(n, H, V, device="cuda")
        if strided:
            qkv = torch.cat([t["q"].flatten(1), t["k"].flatten(1), t["v"].flatten(1)], 1)
            q, k, v = (qkv[:, i * H * K:(i + 1) * H * K].view(n, H, K) for i in range(3))
            ab = torch.cat([t["gate"].flatten(1), t["beta"]] + ([] if family != "kda" else [t["beta"]]), 1)
            gate = ab[:, :t["gate"].flatten(1).shape[1]].view(t["gate"].shape)
            beta = ab[:, t["gate"].flatten(1).shape[1]:][:, :H]
            wide = torch.zeros(n, 3, H, V, device="cuda")
            out = wide[:, 1]
        else:
            q, k, v, gate, beta = (t[x] for x in ("q", "k", "v", "gate", "beta"))
        lay.prefill(q, k, v, gate, None if family == "mamba2" else beta, starts([n]),
                    max_tokens=1 if form == "tokens" else 1 << 20, out=out)
        torch.cuda.synchronize()
        if strided:
            assert (wide[:, 0] == 0).all() and (wide[:, 2] == 0).all()
        got.append((out.cpu(), lay.state.cpu()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_another_current_device_or_stream_handle(cuda_ok):
    """A raw stream handle (0: the default stream) and an allocated output, under another stream's context."""
    import torch
    d = U.draw(synth.GDN, 40, 2, 2, 64, 64, 23)
    args = [dev(d[x]) for x in ("q", "k", "v", "gate", "beta")] + [starts([40])]
    outs = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (None, 0, side.cuda_stream, side):
        lay, _ = make_layer(synth.GDN, 1, 2, 64, 64, d["A"], 23)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            outs.append((lay.prefill(*args, stream=handle), lay))
        torch.cuda.synchronize()
    assert all(torch.equal(outs[0][0], o) and torch.equal(outs[0][1].state, lay.state) for o, lay in outs)
    assert outs[0][0].dtype == torch.bfloat16


def test_a_layer_on_a_device_that_is_not_current(cuda_ok):
    """prefill in both forms, save and restore on the second device while the first is current, against the first."""
    import torch
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two devices")
    d = U.draw(synth.GDN, 90, 2, 2, 64, 64, 28)
    got = []
    for device, stream in (("cuda:0", None), ("cuda:1", None), ("cuda:1", torch.cuda.Stream("cuda:1"))):
        lay = DecodeLayer(synth.GDN, 1, 2, 64, 64, 4, [2] * 2, device=torch.device(device))
        cache = StateCache(lay, 1)
        args = [dev(d[x]).to(device) for x in ("q", "k", "v", "gate", "beta")] + [starts([90]).to(device)]
        slots = torch.zeros(1, dtype=torch.int32, device=device)
        torch.cuda.synchronize(device)
        assert torch.cuda.current_device() == 0
        outs = [lay.prefill(*args, max_tokens=1, stream=stream), lay.prefill(*args, max_tokens=1 << 20, stream=stream)]
        lay.save(cache, slots, stream=stream)
        lay.restore(cache, slots, stream=stream)
        torch.cuda.synchronize(device)
        assert int(lay.status[0]) == 0
        got.append([x.cpu() for x in outs + [lay.state, cache.codes, cache.scales]])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("family", list(FAM))
def test_no_token_reaches_another_sequence(cuda_ok, family):
    """A sequence of NaN and infinities between two others in the same chunk's rows leaves them bit for bit as without it."""
    import torch
    fam, H, K, V, lens = FAM[family], 2, 64, 128, [70, 20, 75]
    d = U.draw(fam, sum(lens), H, H, K, V, 24)
    got = []
    for bad in (False, True):
        t = {x: dev(d[x]) for x in ("q", "k", "v", "gate", "beta")}
        if bad:
            for x in ("q", "k", "v"):
                t[x][70:90] = 0x7F80                       # infinity
            t["gate"][70:90] = float("nan")
        for form in (1, 1 << 20):
            lay, _ = make_layer(fam, 3, H, K, V, d["A"], 24)
            out = lay.prefill(*(t[x] for x in ("q", "k", "v", "gate")), None if family == "mamba2" else t["beta"], starts(lens),
                              max_tokens=form)
            torch.cuda.synchronize()
            got.append((out[:70].cpu(), out[90:].cpu(), lay.state[0].cpu(), lay.state[2].cpu()))
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(got[i], got[i + 2]))


def test_no_rows(cuda_ok):
    import torch
    lay, state = make_layer(synth.GDN, 3, 2, 64, 64, np.ones(2, np.float32), 13)
    e = lambda *s, dtype=torch.int16: torch.zeros(0, *s, dtype=dtype, device="cuda")  # noqa: E731
    lay.prefill(e(2, 64), e(2, 64), e(2, 64), e(2, dtype=torch.float32), e(2, dtype=torch.float32), starts([0, 0, 0]),
                fresh=dev(np.asarray([0, 1, 0], np.int32)))
    got = lay.state.cpu().numpy()
    state[1] = 0
    assert (got == state).all()


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("table", [[0, 5, 3, 8], [-1, 4, 6, 8], [0, 4, 9, 9], [0, 4, 2 ** 31 - 1, 8]])
def test_bad_rows_are_left_out(cuda_ok, table, form):
    """A sequence whose rows are no range of the call's sets the status bit and nothing else; the others run."""
    import torch
    d = U.draw(synth.GDN, 8, 2, 2, 64, 64, 14)
    lay, state = make_layer(synth.GDN, 3, 2, 64, 64, d["A"], 14)
    out = torch.full((8, 2, 64), 7.0, device="cuda")
    lay.prefill(*(dev(d[x]) for x in ("q", "k", "v", "gate", "beta")), dev(np.asarray(table, np.int32)),
                max_tokens=1 if form == "tokens" else 1 << 20, fresh=dev(np.ones(3, np.int32)), out=out)
    torch.cuda.synchronize()
    assert int(lay.status[0]) == B.SS_DEVICE_BAD_ROWS
    o, S = out.cpu().numpy(), lay.state.cpu().numpy()
    touched = np.zeros(8, int)
    fine = [b for b in range(3) if 0 <= table[b] <= table[b + 1] <= 8]
    for b in fine:
        touched[table[b]:table[b + 1]] += 1
    for b in range(3):
        s, e = table[b], table[b + 1]
        if b not in fine:
            assert (S[b] == state[b]).all()
            continue
        cut = {x: d[x][s:e] for x in ("q_", "k_", "v_", "gate", "beta")}
        ref, ref_S = U.reference(synth.GDN, state[b:b + 1], {**cut, "A": d["A"]}, [e - s], [1])
        check(S[b], ref_S[0], U.tolerance(8, 64))
        own = touched[s:e] == 1                # a row of two sequences holds either's output
        check(o[s:e][own], ref[own], U.tolerance(8, 64))
    assert (o[touched == 0] == 7.0).all()


@pytest.mark.parametrize("family", list(FAM))
def test_prompt_in_parts_then_decode(cuda_ok, family):
    """A prompt in two parts with its state swapped out at 8 bits between them,
    then drafts of three tokens, a sketch and a window of decode steps: the
    outputs are the 64-bit recurrence's (ranks = dk: the sketch is exact)."""
    import torch
    fam, Bt, H, K, V, W = FAM[family], 2, 2, 64, 64, 4
    lens = [[70, 33], [5, 64], [3, 3]]
    total = sum(map(sum, lens)) + Bt * W
    d = U.draw(fam, total, H, H, K, V, 15)
    state = np.zeros((Bt, H, K, V), np.float32)
    lay = DecodeLayer(fam, Bt, H, K, V, W, [K] * H)
    eye = np.concatenate([np.eye(K, dtype=np.float32)] * H)
    lay.load(state=state + 9, basis=eye, coef=eye, A=d["A"])
    cache = StateCache(lay, 3, bits=8)
    S, at = state.astype(np.float64), 0
    for part, n in enumerate(lens):
        cut = {x: d[x][at:at + sum(n)] for x in ("q", "k", "v", "gate", "beta", "q_", "k_", "v_")}
        out = lay.prefill(*(dev(cut[x]) for x in ("q", "k", "v", "gate")),
                          None if family == "mamba2" else dev(cut["beta"]), starts(n), max_tokens=max(n),
                          fresh=dev(np.full(Bt, int(part == 0), np.int32)), out_dtype=torch.float32)
        ref, S = U.reference(fam, S, {**cut, "A": d["A"]}, n, [0] * Bt)
        torch.cuda.synchronize()
        # the quantised hand-over is followed from the state the device holds
        check(out.cpu().numpy(), ref, U.tolerance(max(n), K))
        check(lay.state.cpu().numpy(), S, U.tolerance(max(n), K))
        if part == 0:
            gpu = lay.state.cpu().numpy()
            lay.save(cache, dev(np.asarray([2, 0], np.int32)))
            lay.load(state=state - 5)
            lay.restore(cache, dev(np.asarray([2, 0], np.int32)))
            torch.cuda.synchronize()
            S = U.held(gpu, 8)
            assert (lay.state.cpu().numpy() == S.astype(np.float32)).all()
        at += sum(n)
    lay.prime()
    for w in range(W):
        tok = {x: d[x][at:at + Bt] for x in ("q", "k", "v", "gate", "beta")}
        lay.step(lay.token(tok))
        torch.cuda.synchronize()
        for b in range(Bt):
            cut = {x: d[x][at + b:at + b + 1] for x in ("q_", "k_", "v_", "gate", "beta")}
            ref, S_b = U.reference(fam, S[b:b + 1], {**cut, "A": d["A"]}, [1], [0])
            S[b] = S_b[0]
            check(lay.out[b].cpu().numpy(), ref[0], 1e-4)
        at += Bt
    assert int(lay.status[0]) == 0


@pytest.mark.parametrize("family", list(FAM))
def test_new_sequence_joins_a_mixed_batch(cuda_ok, family):
    """Continuous batching: while sequence 0 sits inside its window, sequence 1
    ends and a new prompt takes its place; after prime() both go on, sequence 0
    with the tokens it had buffered (ranks = dk: the sketch is exact)."""
    import torch
    fam, H, K, V, W, n = FAM[family], 2, 64, 64, 4, 40
    d = U.draw(fam, 2 * 7 + n, H, H, K, V, 25)
    lay = DecodeLayer(fam, 2, H, K, V, W, [K] * H)
    eye = np.concatenate([np.eye(K, dtype=np.float32)] * H)
    S = np.random.default_rng(25).standard_normal((2, H, K, V)).astype(np.float32) * 0.3
    lay.load(state=S, basis=eye, coef=eye, A=d["A"])
    S = S.astype(np.float64)
    fills = [torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2)]
    cut = lambda a, b: {x: d[x][a:b] for x in ("q", "k", "v", "gate", "beta", "q_", "k_", "v_")}  # noqa: E731

    def steps(at, count):
        for i in range(count):
            c = cut(at + 2 * i, at + 2 * i + 2)
            lay.step_mixed(lay.token({x: c[x] for x in ("q", "k", "v", "gate", "beta")}), *fills)
            torch.cuda.synchronize()
            fills.reverse()
            for b in range(2):
                one = {x: c[x][b:b + 1] for x in c}
                ref, S_b = U.reference(fam, S[b:b + 1], {**one, "A": d["A"]}, [1], [0])
                S[b] = S_b[0]
                check(lay.out[b].cpu().numpy(), ref[0], 1e-4)

    lay.prime()
    steps(0, 2)
    c = cut(4, 4 + n)
    out = lay.prefill(*(dev(c[x]) for x in ("q", "k", "v", "gate")), None if family == "mamba2" else dev(c["beta"]),
                      starts([0, n]), max_tokens=n, fresh=dev(np.asarray([0, 1], np.int32)), out_dtype=torch.float32)
    ref, S_1 = U.reference(fam, S[1:2], {**c, "A": d["A"]}, [n], [1])
    S[1] = S_1[0]
    torch.cuda.synchronize()
    check(out.cpu().numpy(), ref, U.tolerance(n, K))
    fills[0][1] = 0
    lay.prime()
    steps(4 + n, 5)
    assert fills[0].tolist() == [3, 1] and int(lay.status[0]) == 0


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("family", list(FAM))
def test_captured_and_on_another_stream(cuda_ok, family, form):
    """A call captured into a graph, replayed twice while another layer's call
    runs on a second stream, gives what the same calls give one after the other."""
    import torch
    fam, H, K, V, lens = FAM[family], 3, 128, 128, [70, 9]
    d = U.draw(fam, sum(lens), H, H, K, V, 16)
    t = [dev(d[x]) for x in ("q", "k", "v", "gate")] + [None if family == "mamba2" else dev(d["beta"])]
    st = starts(lens)
    mt = 1 if form == "tokens" else 1 << 20
    layers = [make_layer(fam, 2, H, K, V, d["A"], 16)[0] for _ in range(3)]
    outs = [torch.zeros(sum(lens), H, V, device="cuda") for _ in range(3)]
    for _ in range(2):
        layers[0].prefill(*t, st, max_tokens=mt, out=outs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layers[1].prefill(*t, st, max_tokens=mt, out=outs[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        g.replay()
        layers[2].prefill(*t, st, max_tokens=mt, out=outs[2], stream=side)
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(outs[0], outs[i]) and torch.equal(layers[0].state, layers[i].state)


@pytest.mark.parametrize("family", ["mamba2", "gdn"])
def test_more_heads_than_sms_and_many_lengths(cuda_ok, family):
    """Several units follow one another on an SM; every length modulo the chunk's 64 occurs near its ends."""
    lens = [1, 62, 63, 64, 65, 66, 126, 128, 130, 191, 192, 193, 0, 40, 320, 257]
    heads = 11
    run_case(FAM[family], heads, heads, 64, 64, lens, [i % 3 == 0 for i in range(len(lens))], 18, "long")


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("batch", [200, 512, 600])
def test_few_sequences_of_a_large_batch(cuda_ok, batch, form):
    """Prompts for a few places of a large batch (put in order up to 512 sequences): the others keep their state or start afresh."""
    r = np.random.default_rng(batch)
    lens = np.zeros(batch, int)
    lens[r.choice(batch, 9, replace=False)] = [1, 70, 5, 70, 64, 130, 2, 33, 70]
    lens[-1] = 3
    run_case(synth.GDN, 2, 1, 64, 64, lens.tolist(), (r.random(batch) < 0.5).astype(int).tolist(), 26, form, first=1)


@pytest.mark.parametrize("form", ["tokens", "long"])
def test_large_and_small_values(cuda_ok, form):
    """Values far from one: the split operands keep fp32's relative accuracy over the exponents."""
    for scale in (2.0 ** 60, 2.0 ** -60):
        def change(d):
            d["v"], d["v_"] = U.bf16(d["v_"] * scale)
        lay, state = make_layer(synth.GDN, 1, 2, 64, 64, np.ones(2, np.float32), 19)
        state = (state * scale).astype(np.float32)
        lay.load(state=state)
        run_case(synth.GDN, 2, 2, 64, 64, [100], [0], 19, form, change=change, layer=(lay, state))


@pytest.mark.parametrize("form", ["tokens", "long"])
def test_row_offsets_beyond_32_bits(cuda_ok, form):
    """Rows 2^25 elements apart: the last ones lie more than 2^31 elements behind the first."""
    import torch
    H, K, n = 2, 64, 70
    d = U.draw(synth.GDN, n, H, H, K, K, 21)
    wide = torch.zeros(n << 25, dtype=torch.bfloat16, device="cuda").view(n, 1 << 25)
    views = []
    for i, x in enumerate(("q", "k", "v")):
        view = wide[:, 256 * i:256 * i + H * K].view(n, H, K)
        view.copy_(dev(d[x]).view(torch.bfloat16))
        views.append(view)
    out = wide[:, 1024:1024 + H * K].view(n, H, K)
    lay, state = make_layer(synth.GDN, 1, H, K, K, d["A"], 21)
    lay.prefill(*views, dev(d["gate"]), dev(d["beta"]), starts([n]), max_tokens=1 if form == "tokens" else 1 << 20, out=out)
    torch.cuda.synchronize()
    ref, ref_S = U.reference(synth.GDN, state, d, [n], [0])
    check(out.float().cpu().numpy(), ref, U.tolerance(n, K), True)
    check(lay.state[0].cpu().numpy(), ref_S[0], U.tolerance(n, K))


@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("family", list(FAM))
def test_nothing_outside_the_buffers_is_written(cuda_ok, family, form):
    """Canary-padded state, output, slots, status and inputs around ragged calls and a swap."""
    import torch
    from tests.test_gpu_canary import Guarded
    fam, H, lens = FAM[family], 3, [65, 0, 7, 130]
    for K, V in ((128, 128), (64, 128), (128, 64)):
        d = U.draw(fam, sum(lens), H, H, K, V, 22)
        lay, _ = make_layer(fam, 4, H, K, V, d["A"], 22)
        g = Guarded()
        for x in ("state", "A", "status"):
            setattr(lay, x, g.view(getattr(lay, x)))
        lay._bufs = {w: lay._make_bufs(w) for w in (True, False)}
        args = [g.view(dev(d[x])) for x in ("q", "k", "v", "gate", "beta")]
        if family == "mamba2":
            args[4] = None
        st, fresh, slots = (g.view(dev(np.asarray(x, np.int32))) for x in (np.cumsum([0] + lens), [0, 1, 0, 1], [2, -1, 0, 1]))
        for dt in (torch.float32, torch.bfloat16):
            out = g.view(torch.zeros(sum(lens), H, V, dtype=dt, device="cuda"))
            lay.prefill(*args, st, max_tokens=1 if form == "tokens" else 1 << 20, fresh=fresh, out=out)
        for bits in (8, 4):
            cache = StateCache(lay, 3, bits=bits)
            cache.codes, cache.scales = g.view(cache.codes), g.view(cache.scales)
            cache._arg = B.make_cache(cache.codes, cache.scales, 3, bits)
            lay.save(cache, slots)
            lay.restore(cache, slots)
        assert int(lay.status[0]) == 0
        g.check()


@pytest.mark.parametrize("family", ["mamba2", "gdn"])
def test_wait_that_runs_out(cuda_ok, family):
    """A copy that one CTA waits for in vain: the call ends, says so, leaves that
    head's state as it was and completes the others; the next call is sound."""
    import torch
    fam, H, lens = FAM[family], 3, [70, 200]
    d = U.draw(fam, sum(lens), H, H, 64, 64, 20)
    lay, state = make_layer(fam, 2, H, 64, 64, d["A"], 20)
    args = [dev(d[x]) for x in ("q", "k", "v", "gate")] + [None if family == "mamba2" else dev(d["beta"]), starts(lens)]
    B.ss_debug_stall_next_copy(lay.plan)
    lay.prefill(*args, max_tokens=1 << 20, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert int(lay.status[0]) == B.SS_DEVICE_TIMEOUT
    _, ref = U.reference(fam, state, d, lens, [0, 0])
    got = lay.state.cpu().numpy()
    stalled = [(b, h) for b in range(2) for h in range(H) if (got[b, h] == state[b, h]).all()]
    assert len(stalled) == 1
    for b in range(2):
        for h in range(H):
            if (b, h) not in stalled:
                check(got[b, h], ref[b, h], U.tolerance(200, 64))
    lay.status.zero_()
    lay.load(state=state)
    lay.prefill(*args, max_tokens=1 << 20, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert int(lay.status[0]) == 0
    for b in range(2):
        check(lay.state[b].cpu().numpy(), ref[b], U.tolerance(200, 64))


def test_stall_hook_waits_for_a_call_with_bulk_copies(cuda_ok):
    """The testing hook stays armed over calls that wait for no bulk copy."""
    import torch
    d = U.draw(synth.GDN, 70, 2, 2, 64, 64, 27)
    lay, _ = make_layer(synth.GDN, 1, 2, 64, 64, d["A"], 27)
    args = [dev(d[x]) for x in ("q", "k", "v", "gate", "beta")] + [starts([70])]
    cache, slots = StateCache(lay, 1), dev(np.zeros(1, np.int32))
    B.ss_debug_stall_next_copy(lay.plan)
    lay.prefill(*args, max_tokens=1)
    lay.save(cache, slots)
    lay.restore(cache, slots)
    torch.cuda.synchronize()
    assert int(lay.status[0]) == 0
    lay.prefill(*args, max_tokens=1 << 20)
    torch.cuda.synchronize()
    assert int(lay.status[0]) == B.SS_DEVICE_TIMEOUT
    lay.status.zero_()
    lay.prefill(*args, max_tokens=1 << 20)
    torch.cuda.synchronize()
    assert int(lay.status[0]) == 0


def test_argument_checks(cuda_ok):
    import torch
    lay, _ = make_layer(synth.GDN, 2, 4, 64, 64, np.ones(4, np.float32), 17)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    good = dict(q=bf(6, 4, 64), k=bf(6, 4, 64), v=bf(6, 4, 64), gate=f(6, 4), beta=f(6, 4), seq_start=starts([4, 2]))
    lay.prefill(**good)
    for kw, err in ((dict(q=f(6, 4, 64)), TypeError), (dict(k=bf(5, 4, 64)), ValueError),
                    (dict(q=bf(6, 3, 64), k=bf(6, 3, 64)), ValueError), (dict(v=bf(6, 4, 128)), ValueError),
                    (dict(k=bf(6, 64, 4).mT), ValueError), (dict(gate=f(6, 4, 64)), ValueError),
                    (dict(beta=None), TypeError), (dict(v=bf(1, 4, 64).expand(6, 4, 64)), ValueError),
                    (dict(q=bf(6, 4, 64).cpu()), ValueError), (dict(seq_start=starts([6])), ValueError),
                    (dict(seq_start=starts([4, 2]).long()), TypeError), (dict(fresh=f(2)), TypeError),
                    (dict(seq_start=starts([4, 2]).cpu()), ValueError), (dict(out=f(6, 4, 32)), ValueError),
                    (dict(out=f(6, 4, 64).double()), TypeError), (dict(max_tokens=-1), B.SSError),
                    (dict(out=f(6, 4, 64), out_dtype=torch.bfloat16), TypeError),
                    (dict(v=bf(6, 4 * 64 + 4)[:, :256].view(6, 4, 64)), B.SSError)):
        with pytest.raises(err):
            lay.prefill(**{**good, **kw})
    B.ss_set_phase(lay.plan, 1, True)
    with pytest.raises(B.SSError) as e:
        lay.prefill(**good)
    assert e.value.status == B.SS_ERR_SCHEDULE
    B.ss_set_phase(lay.plan, 0, True)
    B.ss_debug_fail_launch(lay.plan, 1)
    with pytest.raises(B.SSError) as e:
        lay.prefill(**good)
    assert e.value.status == B.SS_ERR_CUDA and B.ss_get_phase(lay.plan) == (0, True)
    lay.prefill(**good)
    assert B.ss_get_phase(lay.plan) == (0, False)      # the sketch is stale now
