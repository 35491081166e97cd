"""Refusals of ss_prefill and the state cache calls that need no GPU: every
call here fails a check before anything is launched."""
import ctypes

import numpy as np
import pytest

from ssm_decode_b200 import binding as B
from ssm_decode_b200 import build, synth
from tests import many_token_util as U
from tests.test_abi_host import _fake_bufs, _no_gpu

cpu_only = pytest.mark.skipif(not _no_gpu(), reason="fake-pointer validation tests run on CPU hosts only")


@pytest.fixture(scope="module")
def L():
    build.build()
    return B.lib()


def _io(**kw):
    f = dict(q=0x10000, k=0x20000, v=0x30000, gate=0x40000, beta=0x50000, out=0x60000, q_stride=0, k_stride=0,
             v_stride=0, gate_stride=0, beta_stride=0, out_stride=0, rows=8, max_tokens=0, seq_start=0x70000,
             fresh=None, qk_heads=0, out_dtype=0)
    f.update(kw)
    return B.ss_prefill_io(*[f[n] for n, _ in B.ss_prefill_io._fields_])


@cpu_only
@pytest.mark.parametrize("family", [B.SS_MAMBA2, B.SS_GDN, B.SS_KDA])
def test_prefill_refusals(L, family):
    p = B.Plan(family, 2, 4, 128, 64, 4, [2] * 4)
    ok = _fake_bufs()

    def rc(io, bufs=ok):
        return L.ss_prefill(p.handle, ctypes.byref(bufs), ctypes.byref(io), None)

    inv, ali, uns = B.SS_ERR_INVALID_ARG, B.SS_ERR_ALIGNMENT, B.SS_ERR_UNSUPPORTED
    cases = [(dict(rows=-1), inv), (dict(rows=2 ** 31), inv), (dict(max_tokens=-1), inv), (dict(out_dtype=2), inv),
             (dict(qk_heads=3), inv), (dict(qk_heads=-1), inv), (dict(qk_heads=8), inv), (dict(seq_start=None), inv),
             (dict(seq_start=0x70002), ali), (dict(fresh=0x70001), ali), (dict(q=None), inv), (dict(q=0x10008), ali),
             (dict(k=None), inv), (dict(k=0x20002), ali), (dict(v=None), inv), (dict(v=0x30004), ali),
             (dict(out=None), inv), (dict(out=0x60004), ali), (dict(gate=None), inv), (dict(gate=0x40002), ali),
             (dict(q_stride=511), inv), (dict(q_stride=516), ali), (dict(k_stride=-512), inv),
             (dict(v_stride=248), inv), (dict(v_stride=260), ali), (dict(out_stride=257), ali),
             (dict(q_stride=2 ** 30 + 8), uns), (dict(gate_stride=1), inv), (dict(gate_stride=2 ** 31), uns)]
    if family != B.SS_MAMBA2:
        cases += [(dict(beta=None), inv), (dict(beta=0x50001), ali), (dict(beta_stride=3), inv)]
    if family == B.SS_KDA:
        cases += [(dict(gate=0x40004), ali), (dict(gate_stride=514), ali)]
    for kw, code in cases:
        assert rc(_io(**kw)) == code, kw
    assert rc(_io(), _fake_bufs(null="state")) == inv
    assert rc(_io(), _fake_bufs(bad="state")) == ali
    if family == B.SS_MAMBA2:
        assert rc(_io(), _fake_bufs(null="A")) == inv
    assert L.ss_prefill(p.handle, ctypes.byref(ok), None, None) == inv
    assert L.ss_prefill(p.handle, None, ctypes.byref(_io()), None) == inv
    assert L.ss_prefill(None, ctypes.byref(ok), ctypes.byref(_io()), None) == inv
    B.ss_set_phase(p, 1, True)
    assert rc(_io()) == B.SS_ERR_SCHEDULE
    assert B.ss_get_phase(p) == (1, True)


@cpu_only
def test_prefill_launch_failure_leaves_the_plan(L):
    p = B.Plan(B.SS_GDN, 2, 4, 128, 64, 4, [2] * 4)
    B.ss_set_phase(p, 0, True)
    B.ss_debug_fail_launch(p, 1)
    assert L.ss_prefill(p.handle, ctypes.byref(_fake_bufs()), ctypes.byref(_io()), None) == B.SS_ERR_CUDA
    assert B.ss_get_phase(p) == (0, True)


@cpu_only
def test_cache_refusals(L):
    p = B.Plan(B.SS_GDN, 2, 4, 64, 64, 4, [2] * 4)
    good = dict(codes=0x10000, scales=0x20000, slots=3, bits=8)

    def rc(fn, cache=None, slots=0x30000, bufs=None):
        c = B.ss_cache(*[{**good, **(cache or {})}[n] for n, _ in B.ss_cache._fields_])
        return fn(p.handle, ctypes.byref(bufs or _fake_bufs()), ctypes.byref(c), ctypes.c_void_p(slots), None)

    for fn in (L.ss_cache_write, L.ss_cache_read):
        for kw, code in ((dict(codes=None), 1), (dict(codes=0x10008), 2), (dict(scales=None), 1),
                         (dict(scales=0x20002), 2), (dict(slots=0), 1), (dict(bits=16), 3)):
            assert rc(fn, kw) == code, kw
        assert rc(fn, slots=None) == B.SS_ERR_INVALID_ARG
        assert rc(fn, slots=0x30002) == B.SS_ERR_ALIGNMENT
        assert rc(fn, bufs=_fake_bufs(null="state")) == B.SS_ERR_INVALID_ARG
        B.ss_set_phase(p, 1, True)
        assert rc(fn) == B.SS_ERR_SCHEDULE
        B.ss_set_phase(p, 0, True)
        B.ss_debug_fail_launch(p, 1)
        assert rc(fn) == B.SS_ERR_CUDA
        assert B.ss_get_phase(p) == (0, True)


def test_cache_sizes(L):
    p = B.Plan(B.SS_KDA, 2, 3, 128, 64, 4, [2] * 3)
    assert B.ss_cache_sizes(p, 8, 5) == (5 * 3 * 128 * 64, 5 * 3 * 128 * 2 * 2)
    assert B.ss_cache_sizes(p, 4, 5) == (5 * 3 * 128 * 32, 5 * 3 * 128 * 2 * 2)
    assert B.ss_cache_sizes(p, 8, 2 ** 31 - 1)[0] == (2 ** 31 - 1) * 3 * 128 * 64
    for bits, slots in ((2, 1), (8, 0), (4, -1)):
        with pytest.raises(B.SSError):
            B.ss_cache_sizes(p, bits, slots)


def test_plain_quantiser():
    """The tests' own quantiser: codes by exact fractions, ties to even."""
    from fractions import Fraction
    r = np.random.default_rng(0)
    x = (r.standard_normal((4, 32)) * np.exp2(r.integers(-40, 40, (4, 1)))).astype(np.float32)
    x[1] = np.arange(32) / 2 - 8
    x[1, 0] = 7
    for bits, m in ((8, 127), (4, 7)):
        c, s = U.quantise(x, bits)
        for i in range(4):
            for j in range(32):
                want = round(Fraction(float(x[i, j])) / Fraction(float(s[i, 0])))     # ties to even
                assert c[i, j] == max(-m, min(m, want))


@pytest.mark.parametrize("family", [synth.MAMBA2, synth.GDN, synth.KDA])
def test_plain_recurrence_is_the_oracles(family):
    """The tests' token loop against the oracle's exact step on the same inputs."""
    from oracle import sketchssm_oracle as orc
    H, K, V, T = 2, 64, 64, 5
    d = U.draw(family, T, H, H, K, V, 3)
    S0 = np.random.default_rng(1).standard_normal((1, H, K, V)).astype(np.float32)
    out, S = U.reference(family, S0, d, [T], [0])
    sess = orc.Session(family, S0, 1, d["A"], np.zeros((H, K), np.float32), np.zeros((H, K), np.float32),
                       np.arange(H + 1, dtype=np.int32))
    for t in range(T):
        o = sess.flush({x: d[x][t:t + 1] for x in ("q", "k", "v", "gate", "beta")})
        np.testing.assert_allclose(out[t], o[0], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S, sess.S, rtol=1e-12, atol=1e-12)


def test_calls_go_to_the_layers_device(L, monkeypatch):
    """prefill, save and restore of a layer whose device is not the current one: that device is current while the
    call's output is allocated and the kernel launched, on its own current stream or the stream given."""
    import contextlib

    import torch
    from ssm_decode_b200 import layer as M
    now, seen = {"device": 0, "stream": {0: "s0", 1: "s1"}}, []

    @contextlib.contextmanager
    def on(key, value):
        was, now[key] = now[key], value
        yield
        now[key] = was

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now["device"])
    monkeypatch.setattr(torch.cuda, "device", lambda d: on("device", torch.device(d).index))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: on("stream", {**now["stream"], now["device"]: s}))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now["stream"][now["device"]])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: "raw " + now["stream"][i], raising=False)
    monkeypatch.setattr(torch, "zeros", lambda *a, device, **kw: seen.append(("zeros", device.index, now["device"], torch.cuda.current_stream())))
    monkeypatch.setattr(M.B, "make_prefill_io", lambda *a: None)
    monkeypatch.setattr(M.B, "_index", lambda *a: None)
    for f in ("ss_prefill", "ss_cache_write", "ss_cache_read"):
        monkeypatch.setattr(M.B, f, lambda *a, f=f: seen.append((f, now["device"], a[-1])))
    lay = M.DecodeLayer.__new__(M.DecodeLayer)
    lay.plan, lay.heads, lay.dv, lay.batch, lay._bufs = None, 2, 64, 1, {False: None}
    lay.state = type("State", (), {"device": torch.device("cuda:1")})()
    cache = type("Cache", (), {"arg": lambda self, layer: None})()
    q = torch.empty(3, 2, 64)
    for current in (0, 1):
        now["device"] = current
        for given in (None, "mine"):
            del seen[:]
            lay.prefill(q, q, q, None, None, None, stream=given)
            lay.save(cache, None, stream=given)
            lay.restore(cache, None, stream=given)
            own = given or "s1"
            handle = "raw s1" if given is None and current == 1 else own
            assert seen == [("zeros", 1, 1, own), ("ss_prefill", 1, handle), ("ss_cache_write", 1, handle),
                            ("ss_cache_read", 1, handle)]
            assert now["device"] == current and now["stream"] == {0: "s0", 1: "s1"}
