"""ss_cache_write / ss_cache_read against exact quantisation (needs a B200): every code and scale bit for bit."""
import numpy as np
import pytest

from ssm_decode_b200 import binding as B
from ssm_decode_b200 import synth
from ssm_decode_b200.layer import DecodeLayer, StateCache
from tests import many_token_util as U
from tests.test_gpu_prefill import dev, make_layer

pytestmark = pytest.mark.gpu


def codes_of(cache):
    raw = cache.codes.cpu().numpy()
    if cache.bits == 8:
        return raw.view(np.int8).astype(np.int64)
    both = np.stack([raw & 15, raw >> 4], -1).reshape(*raw.shape[:-1], -1).astype(np.int64)
    return np.where(both > 7, both - 16, both)


def bits16(cache):
    import torch
    return cache.scales.view(torch.int16).cpu().numpy().view(np.uint16)


def save(state, bits, slots, count):
    import torch
    Bt, H, K, V = state.shape
    lay = DecodeLayer(synth.GDN, Bt, H, K, V, 4, [1] * H)
    lay.load(state=state)
    cache = StateCache(lay, count, bits=bits)
    cache.codes.fill_(0x33)
    cache.scales.fill_(3.0)
    lay.save(cache, dev(np.asarray(slots, np.int32)))
    torch.cuda.synchronize()
    return lay, cache


def states(kind, shape, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal(shape)
    if kind == "wide":                      # every exponent, groups of zeros, -0.0
        x = x * np.exp2(r.integers(-126, 120, size=(*shape[:-1], 1)))
        x[..., ::7, :] = 0.0
        x[..., 1::7, :] *= -0.0
    if kind == "subnormal":
        x = x * np.exp2(r.integers(-149, -118, size=(*shape[:-1], 1)).astype(np.float64))
    if kind == "ties":                      # whole and half codes of a power-of-two scale
        m = {0: 127, 1: 7}[seed % 2]
        x = r.integers(-2 * m, 2 * m + 1, size=shape) / 2.0
        x[..., ::32] = m
        x = x * np.exp2(r.integers(-9, 9, size=(*shape[:-1], 1)))
    return x.astype(np.float32)


@pytest.mark.parametrize("kind,seed", [("plain", 2), ("wide", 3), ("subnormal", 4), ("ties", 0), ("ties", 1)])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("bits", [8, 4])
def test_codes_and_values(cuda_ok, bits, dk, dv, kind, seed):
    import torch
    state = states(kind, (3, 3, dk, dv), seed)
    lay, cache = save(state, bits, [4, -1, 0], 5)
    c, s = U.quantise(state, bits)
    got, sc = codes_of(cache), bits16(cache)
    for b, slot in ((0, 4), (2, 0)):
        assert (sc[slot] == synth.f32_to_bf16_bits(s[b].astype(np.float32))).all()
        assert (got[slot] == c[b]).all()
    for slot in (1, 2, 3):                  # untouched slots
        assert (cache.codes[slot] == 0x33).all() and (cache.scales[slot] == 3.0).all()
    lay.load(state=state * 0 + 1)
    lay.restore(cache, dev(np.asarray([0, -3, 4], np.int32)))
    torch.cuda.synchronize()
    h = U.held(state, bits).astype(np.float32)
    out = lay.state.cpu().numpy()
    assert (out[0] == h[2]).all() and (out[2] == h[0]).all() and (out[1] == 1).all()
    assert int(lay.status[0]) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_infinities_and_nan(cuda_ok, bits):
    """A group that holds one reads back as NaN; its neighbours are not touched by it."""
    import torch
    state = states("plain", (1, 2, 64, 64), 5)
    state[0, 0, 3, 5], state[0, 1, 9, 40], state[0, 1, 10, 0] = np.inf, np.nan, -np.inf
    lay, cache = save(state, bits, [0], 1)
    lay.restore(cache, dev(np.asarray([0], np.int32)))
    torch.cuda.synchronize()
    out = lay.state.cpu().numpy()
    ref = U.held(np.where(np.isfinite(state), state, 0), bits).astype(np.float32)
    bad = np.zeros(state.shape, bool)
    bad[0, 0, 3, :32] = bad[0, 1, 9, 32:] = bad[0, 1, 10, :32] = True
    assert np.isnan(out[bad]).all() and (out[~bad] == ref[~bad]).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_same_slot_twice_and_bad_slots(cuda_ok, bits):
    """Of several sequences that name a slot the last is kept; one slot is read
    by several; a slot behind the last one sets the status bit and is left out."""
    import torch
    n = 300                                  # more sequences than a block has threads
    state = states("plain", (n, 1, 64, 64), 6)
    slots = np.full(n, -1)
    slots[[0, 7, 299]], slots[[3, 258]], slots[5] = 1, 0, 9
    lay, cache = save(state, bits, slots, 2)
    assert int(lay.status[0]) == B.SS_DEVICE_BAD_SLOT
    lay.status.zero_()
    lay.load(state=state * 0)
    back = np.full(n, 1)
    back[4], back[8], back[9] = 0, 2, -1
    lay.restore(cache, dev(back.astype(np.int32)))
    torch.cuda.synchronize()
    h = U.held(state[[299, 258]], bits).astype(np.float32)
    out = lay.state.cpu().numpy()
    rest = np.setdiff1d(np.arange(n), [4, 8, 9])
    assert (out[rest] == h[0]).all() and (out[4] == h[1]).all() and (out[[8, 9]] == 0).all()
    assert int(lay.status[0]) == B.SS_DEVICE_BAD_SLOT


def test_offsets_beyond_32_bits(cuda_ok):
    """A cache of more than 2^32 codes: the slots at its end are their own."""
    import torch
    H, K, V = 128, 128, 128                  # 2 MB a slot in 8 bits
    count = 2200
    lay = DecodeLayer(synth.GDN, 2, H, K, V, 4, [1] * H)
    x = torch.randn(2, H, K, V, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    lay.state.copy_(x)
    cache = StateCache(lay, count, bits=8)
    lay.save(cache, dev(np.asarray([count - 1, 3], np.int32)))
    assert not cache.codes[:3].any() and not cache.codes[4:count - 1].any()
    lay.state.zero_()
    lay.restore(cache, dev(np.asarray([3, count - 1], np.int32)))
    torch.cuda.synchronize()
    err = (lay.state.flip(0) - x).abs().amax()
    assert float(err) <= float(x.abs().amax()) / 127 * 0.51 and bool((lay.state != 0).any(-1).all())


def test_captured(cuda_ok):
    import torch
    lay, state = make_layer(synth.KDA, 2, 2, 64, 128, np.ones(2, np.float32), 7)
    cache = StateCache(lay, 2, bits=4)
    slots = dev(np.asarray([1, 0], np.int32))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lay.save(cache, slots)
        lay.restore(cache, slots)
    for _ in range(2):                       # what a slot held is held exactly again
        g.replay()
        torch.cuda.synchronize()
        assert (lay.state.cpu().numpy() == U.held(state, 4).astype(np.float32)).all()


def test_argument_checks(cuda_ok):
    lay, _ = make_layer(synth.GDN, 2, 2, 64, 64, np.ones(2, np.float32), 8)
    other, _ = make_layer(synth.GDN, 2, 2, 64, 128, np.ones(2, np.float32), 8)
    for kw in (dict(bits=5), dict(slots=0)):
        with pytest.raises(B.SSError):
            StateCache(lay, **{"slots": 2, **kw})
    cache = StateCache(lay, 2)
    ok = dev(np.zeros(2, np.int32))
    for bad, err in ((ok.long(), TypeError), (ok[:1], ValueError), (ok.cpu(), ValueError)):
        with pytest.raises(err):
            lay.save(cache, bad)
        with pytest.raises(err):
            lay.restore(cache, bad)
    with pytest.raises(ValueError):
        other.save(cache, ok)
    B.ss_set_phase(lay.plan, 2, True)
    for call in (lay.save, lay.restore):
        with pytest.raises(B.SSError) as e:
            call(cache, ok)
        assert e.value.status == B.SS_ERR_SCHEDULE
    B.ss_set_phase(lay.plan, 0, True)
    lay.save(cache, ok)
    assert B.ss_get_phase(lay.plan) == (0, True)       # saving changes nothing
    lay.restore(cache, ok)
    assert B.ss_get_phase(lay.plan) == (0, False)
