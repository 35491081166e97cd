"""The chunked form of ss_prefill: the bits its operand splits keep, and long prompts (needs a B200)."""
import numpy as np
import pytest

from ssm_decode_b200 import synth
from ssm_decode_b200.layer import DecodeLayer
from tests import chunk_cases as cases
from tests import many_token_util as U
from tests.test_gpu_prefill import check, dev, make_layer, starts

pytestmark = pytest.mark.gpu

FAM = {"mamba2": synth.MAMBA2, "gdn": synth.GDN}


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("lead", [0, 64])
@pytest.mark.parametrize("form", ["tokens", "long"])
@pytest.mark.parametrize("family", list(FAM))
def test_split_operands_keep_every_bit(cuda_ok, family, form, lead, dk, dv):
    """The cases of tests/chunk_cases.py in their room, in the first chunk and behind another
    (the token form, which cuts nothing, has the same room)."""
    import torch
    fam = FAM[family]
    for name in cases.names(fam):
        d, S, out_room, S_room = cases.make(name, fam, dk, dv, lead)
        T, H = d["gate"].shape
        lay = DecodeLayer(fam, 1, H, dk, dv, 4, [2] * H)
        lay.load(state=S[None], A=d["A"])
        out = lay.prefill(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["gate"]), None if family == "mamba2" else dev(d["beta"]),
                          starts([T]), max_tokens=1 if form == "tokens" else T, out_dtype=torch.float32)
        torch.cuda.synchronize()
        ref, ref_S = U.reference(fam, S[None], d, [T], [0])
        for what, got, want, room in (("out", out.cpu().numpy(), ref, out_room), ("state", lay.state[0].cpu().numpy(), ref_S[0], S_room)):
            off = np.abs(got.astype(np.float64) - want)
            assert (off <= room).all(), f"{name}, {what}: {(off > room).sum()} beyond the room, {(off - room).max():.2e} at most"
        assert int(lay.status[0]) == 0


@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64)])
@pytest.mark.parametrize("family", list(FAM))
def test_long_prompts(cuda_ok, family, dk, dv):
    """65 chunks beside shorter prompts, against 64 bits.  The decays over 64 tokens are below 2^-10, so an error
    more than a chunk old no longer counts: the tolerance is that of 128 tokens."""
    import torch
    fam, H, lens = FAM[family], 2, [4133, 1, 2048, 1000]
    d = U.draw(fam, sum(lens), H, 1, dk, dv, 31)
    a = np.exp(d["gate"] * d["A"]) if family == "mamba2" else d["gate"]
    g = np.cumsum(np.log(a.astype(np.float64)), 0)
    assert (g[64:] - g[:-64]).max() < np.log(2.0 ** -10)
    lay, state = make_layer(fam, len(lens), H, dk, dv, d["A"], 31)
    out = lay.prefill(*(dev(d[x]) for x in ("q", "k", "v", "gate")), None if family == "mamba2" else dev(d["beta"]), starts(lens),
                      max_tokens=max(lens), out_dtype=torch.float32)
    torch.cuda.synchronize()
    ref, ref_S = U.reference(fam, state, d, lens, [0] * len(lens))
    tol = U.tolerance(128, dk) * (1 + 2.0 ** -9)
    for h in range(H):
        check(out[:, h].cpu().numpy(), ref[:, h], tol)
    for b in range(len(lens)):
        check(lay.state[b].cpu().numpy(), ref_S[b], tol)


@pytest.mark.parametrize("family", list(FAM))
def test_a_prompt_in_parts_of_whole_chunks_is_the_same_bits(cuda_ok, family):
    """2500 tokens in one call and in three, cut between chunks: the state handed over is the one the kernel kept."""
    import torch
    fam, H, K, V, n = FAM[family], 3, 128, 128, 2500
    d = U.draw(fam, n, H, H, K, V, 32)
    args = [dev(d[x]) for x in ("q", "k", "v", "gate")] + [None if family == "mamba2" else dev(d["beta"])]
    got = []
    for cuts in ([0, n], [0, 64 * 13, 64 * 14, n]):
        lay, _ = make_layer(fam, 1, H, K, V, d["A"], 32)
        out = torch.zeros(n, H, V, device="cuda")
        for s, e in zip(cuts, cuts[1:]):
            lay.prefill(*args, dev(np.asarray([s, e], np.int32)), max_tokens=n, out=out)
        torch.cuda.synchronize()
        got.append((out.cpu(), lay.state.cpu()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dk,dv,batch,heads,tokens,chunks", [
    (128, 128, 1, 2, 24, True), (128, 128, 1, 2, 16, False), (128, 128, 64, 32, 28, False), (128, 128, 64, 32, 40, True),
    (64, 64, 1, 2, 32, True), (64, 64, 64, 32, 64, False), (128, 64, 64, 32, 52, False), (128, 64, 64, 32, 70, False),
    (64, 128, 16, 32, 40, True)])
def test_the_faster_form_runs(cuda_ok, dk, dv, batch, heads, tokens, chunks):
    """Which form a call takes, by the shape, the number of units and the longest sequence: the testing hook that
    delays a bulk copy reaches the chunked form only.  (Measured both ways at each of these; the two differ by 5 to 50 %.)"""
    import torch
    from ssm_decode_b200 import binding as B
    d = U.draw(synth.GDN, tokens, heads, 1, dk, dv, 33)
    lay = DecodeLayer(synth.GDN, batch, heads, dk, dv, 4, [2] * heads)
    st = starts([tokens] + [0] * (batch - 1))
    B.ss_debug_stall_next_copy(lay.plan)
    lay.prefill(*(dev(d[x]) for x in ("q", "k", "v", "gate", "beta")), st, max_tokens=tokens)
    torch.cuda.synchronize()
    assert int(lay.status[0]) == (B.SS_DEVICE_TIMEOUT if chunks else 0)
