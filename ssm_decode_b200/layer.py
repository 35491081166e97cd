"""One layer's decode buffers on the device, driven through the C ABI.

PyTorch only allocates device memory and supplies the stream; every step of
the decode path runs in libsketchssm.so's kernels.  The layout of each buffer
is the one include/sketchssm.h documents.
"""
from __future__ import annotations

import contextlib
import weakref

import numpy as np

from . import binding as B


def _dev(x, dtype, device):
    import torch
    if isinstance(x, np.ndarray):
        if x.dtype == np.uint16:
            x = x.view(np.int16)
        x = torch.from_numpy(np.ascontiguousarray(x))
    return x.to(device=device, dtype=dtype).contiguous()


class Token(dict):
    """One step's inputs on the device (q, k, v, gate, beta tensors).  The
    C-ABI argument structs built from it are cached per layer, so a step
    costs one library call; update the tensors in place (copy_) to reuse it."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self._io = {}


class DecodeLayer:
    """Plan plus caller-owned device buffers for one linear-attention layer."""

    def __init__(self, family, batch, heads, dk, dv, window, ranks, sketch_dtype=B.SS_F32,
                 device="cuda", coef_mode=B.SS_COEF_FIXED, coef_ridge=0.0, dense_heads=None):
        import torch
        self.plan = B.Plan(family, batch, heads, dk, dv, window, ranks, sketch_dtype, coef_mode, coef_ridge,
                           dense_heads)
        self.family, self.batch, self.heads, self.dk, self.dv, self.window = family, batch, heads, dk, dv, window
        self.device = device
        sz = B.ss_buffer_sizes(self.plan)
        self.R = sz["total_rank"]
        Wg = (window + 3) & ~3
        f32, i16 = torch.float32, torch.int16
        z = lambda *shape, dtype=f32: torch.zeros(shape, dtype=dtype, device=device)
        self.state = z(batch, heads, dk, dv)
        self.ring_k = z(batch, heads, window, dk, dtype=i16)
        self.ring_v = z(batch, heads, window, dv, dtype=i16)
        self.ring_gate = z(batch, heads, window, dk) if family == B.SS_KDA else z(batch, heads, Wg)
        self.ring_beta = None if family == B.SS_MAMBA2 else z(batch, heads, Wg)
        sk_dtype = torch.float32 if sketch_dtype == B.SS_F32 else torch.bfloat16
        self.sketch = torch.zeros((batch, max(self.R, 1), dv), dtype=sk_dtype, device=device)
        self.basis = z(max(self.R, 1), dk)
        self.coef = z(max(self.R, 1), dk)
        # per-(sequence, head) coefficient maps of SS_COEF_STATE / SS_COEF_LRD, sketch dtype
        self.coef_state = (torch.zeros((batch, max(self.R, 1), dk), dtype=sk_dtype, device=device)
                           if coef_mode in (B.SS_COEF_STATE, B.SS_COEF_LRD) else None)
        self.A = z(heads)
        self.out = z(batch, heads, dv)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)   # device status word (+ padding)
        self.sketch_dtype = sketch_dtype
        # The buffers stay in place for the layer's life (load() copies into
        # them), so their argument structs are built once.
        self._bufs = {w: self._make_bufs(w) for w in (True, False)}

    # -- data -------------------------------------------------------------------
    def load(self, state=None, basis=None, coef=None, A=None):
        if state is not None:
            self.state.copy_(_dev(state, self.state.dtype, self.device))
        if basis is not None and self.R:
            self.basis.copy_(_dev(basis, self.basis.dtype, self.device))
        if coef is not None and self.R:
            self.coef.copy_(_dev(coef, self.coef.dtype, self.device))
        if A is not None:
            self.A.copy_(_dev(A, self.A.dtype, self.device))

    def token(self, inp):
        """Move one step's raw inputs (numpy or torch) to the device."""
        import torch
        t = Token((k, _dev(inp[k], torch.int16, self.device)) for k in ("q", "k", "v"))
        t["gate"] = _dev(inp["gate"], torch.float32, self.device)
        t["beta"] = _dev(inp["beta"], torch.float32, self.device)
        return t

    def bufs(self, with_sketch=True):
        return self._bufs[bool(with_sketch)]

    def _make_bufs(self, with_sketch):
        return B.make_buffers(self.state, self.ring_k, self.ring_v, self.ring_gate, self.ring_beta,
                              self.sketch if with_sketch else None, self.basis, self.coef, self.A,
                              self.status, self.coef_state)

    def io(self, tok, out=None):
        cache = getattr(tok, "_io", None) if out is None else None
        if cache is not None:
            hit = cache.get(id(self))
            if hit is not None and hit[0]() is self:      # guard against a reused id()
                return hit[1]
        beta = tok["beta"] if self.family != B.SS_MAMBA2 else None
        io = B.make_step_io(tok["q"], tok["k"], tok["v"], tok["gate"], beta,
                            self.out if out is None else out)
        if cache is not None:
            cache[id(self)] = (weakref.ref(self), io)
        return io

    @property
    def phase(self):
        return B.ss_get_phase(self.plan)[0]

    # -- calls --------------------------------------------------------------------
    def prime(self, stream=None):
        B.ss_prime(self.plan, self.bufs(), stream)

    def decode(self, tok, out=None, stream=None):
        B.ss_decode_step(self.plan, self.bufs(), self.io(tok, out), stream)

    def flush(self, tok=None, with_sketch=True, out=None, stream=None):
        io = None if tok is None else self.io(tok, out)
        B.ss_flush(self.plan, self.bufs(with_sketch), io, stream)

    def step(self, tok, out=None, stream=None):
        """One SketchSSM step: non-flush until the window's last token, then flush."""
        if self.phase == self.window - 1:
            self.flush(tok, out=out, stream=stream)
        else:
            self.decode(tok, out=out, stream=stream)

    def exact_step(self, tok, out=None, stream=None):
        B.ss_exact_step(self.plan, self.bufs(False), self.io(tok, out), stream)

    def step_mixed(self, tok, fill_in, fill_out, out=None, stream=None):
        """One step with a window position per sequence (int32 device tensors
        of `batch` entries): sequences at W-1 flush, the rest decode;
        fill_out receives (fill_in + 1) mod W."""
        B.ss_step_mixed(self.plan, self.bufs(), self.io(tok, out), fill_in, fill_out, stream)

    def prefill(self, q, k, v, gate, beta, seq_start, max_tokens=None, fresh=None, out=None,
                out_dtype=None, stream=None):
        """Runs a packed, ragged batch of token rows through the exact
        recurrence, from each sequence's state (zero where fresh[b] != 0) to
        the state behind its last token: prompts, parts of prompts, drafts.

        q, k [rows][qk_heads][dk] and v [rows][heads][dv] bf16, gate fp32
        [rows][heads] (KDA [rows][heads][dk]), beta fp32 [rows][heads] (None
        for Mamba-2); sequence b has rows seq_start[b] .. seq_start[b+1]-1
        (device int32 [batch + 1]).  Rows may be strided, and qk_heads may
        divide heads (shared keys).  max_tokens (a host int, at least the
        longest sequence) lets the library pick the faster form; None takes
        the number of rows, so give it for short drafts of many sequences, and
        give prompts and drafts in calls of their own.  Returns out
        [rows][heads][dv], allocated in `out_dtype` (bf16 unless given) when
        not passed; rows of no sequence are left as they were (zero in an
        allocated one).  The state is updated in place: clone it first to be
        able to reject part of a draft.  Needs phase 0; prime(), over the
        whole batch, comes before the next sketched step."""
        import torch
        with self._on_device(stream) as st:
            if out is None:
                out = torch.zeros((q.shape[0], self.heads, self.dv), device=self.state.device,
                                  dtype=out_dtype or torch.bfloat16)
            elif out_dtype not in (None, out.dtype):
                raise TypeError(f"out: dtype {out.dtype}, out_dtype {out_dtype}")
            B.ss_prefill(self.plan, self._bufs[False],
                         B.make_prefill_io(self.plan, q, k, v, gate, beta, out, seq_start, fresh, max_tokens,
                                           self.state.device), st)
        return out

    def save(self, cache, slots, stream=None):
        """Quantises the state of sequence b into cache slot slots[b] (device
        int32 [batch]; negative: left out).  Of several sequences that name
        one slot the last is kept.  Needs phase 0."""
        with self._on_device(stream) as st:
            B.ss_cache_write(self.plan, self.bufs(False), cache.arg(self), self._slot_index(slots), st)

    def restore(self, cache, slots, stream=None):
        """Sets the state of sequence b to what cache slot slots[b] holds
        (negative: left as it is; a slot may be read by several).  Needs
        phase 0; prime() comes before the next sketched step."""
        with self._on_device(stream) as st:
            B.ss_cache_read(self.plan, self.bufs(False), cache.arg(self), self._slot_index(slots), st)

    def _slot_index(self, slots):
        return B._index(slots, "slots", self.batch, self.state.device)

    def _on_device(self, stream):
        """Context that makes the layer's device current and gives the stream a
        call runs on there: `stream`, or the device's current stream.  An
        allocation inside belongs to that stream."""
        import torch
        index = self.state.device.index
        if stream is None and torch.cuda.current_device() == index:
            return contextlib.nullcontext(torch._C._cuda_getCurrentRawStream(index))
        return self._switch(stream)

    @contextlib.contextmanager
    def _switch(self, stream):
        import torch
        with torch.cuda.device(self.state.device):
            if stream is None:
                yield torch.cuda.current_stream()
                return
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
            with torch.cuda.stream(stream):
                yield stream

    def replay_step(self, tok, out=None, stream=None):
        if self.phase == self.window - 1:
            self.flush(tok, with_sketch=False, out=out, stream=stream)
        else:
            B.ss_replay_step(self.plan, self.bufs(False), self.io(tok, out), stream)


class StateCache:
    """Quantised states of one layer's sequences in `slots` slots, 8 or 4 bits
    a value with a bf16 scale per 32 (see ss_cache in include/sketchssm.h):
    prefixes kept for later sequences, or sequences swapped out.  Written and
    read by DecodeLayer.save and .restore of any layer of the same heads and
    dk x dv on the same device."""

    def __init__(self, layer, slots, bits=8):
        import torch
        codes, scales = B.ss_cache_sizes(layer.plan, bits, slots)
        self.slots, self.bits = int(slots), int(bits)
        self.shape = (layer.heads, layer.dk, layer.dv)
        device = layer.state.device
        self.codes = torch.zeros((slots, layer.heads, layer.dk, layer.dv * bits // 8), dtype=torch.uint8, device=device)
        self.scales = torch.zeros((slots, layer.heads, layer.dk, layer.dv // 32), dtype=torch.bfloat16, device=device)
        assert self.codes.numel() == codes and self.scales.numel() * 2 == scales
        self._arg = B.make_cache(self.codes, self.scales, self.slots, self.bits)

    def arg(self, layer):
        if (layer.heads, layer.dk, layer.dv) != self.shape or layer.state.device != self.codes.device:
            raise ValueError(f"cache of {self.shape} on {self.codes.device}, layer of "
                             f"{(layer.heads, layer.dk, layer.dv)} on {layer.state.device}")
        return self._arg
