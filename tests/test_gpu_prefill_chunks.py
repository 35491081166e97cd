"""The chunked form of ss_prefill: the bits its operand splits keep (needs a B200)."""
import numpy as np
import pytest

from ssm_decode_b200 import synth
from ssm_decode_b200.layer import DecodeLayer
from tests import chunk_cases as cases
from tests import many_token_util as U
from tests.test_gpu_prefill import dev, starts

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
