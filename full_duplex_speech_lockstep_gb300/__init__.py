"""GB300-native lockstep decode tick of the PersonaPlex / Moshi RQ-Transformer.

Thin Python binding of ``libpp.so`` (``include/pp.h``): the functions below have the C
ABI's names and only marshal arguments; every step of the tick runs in the library's
CUDA kernels.  PyTorch is used for device memory and streams only.

    import full_duplex_speech_lockstep_gb300 as pp
    eng = pp.Engine(shape, max_batch, weights)   # weights: dict of device tensors
    eng.open(0)
    col = eng.step(prev_column, user_codes)      # int32 [max_batch, 17] device tensor

There is no CPU fallback: if the library is missing or fails to load, this module
raises.
"""
import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
SO = os.path.join(HERE, "libpp.so")

ROWS = 17
PP_OK, PP_EINVAL, PP_E_BUSY, PP_E_RANGE, PP_E_NOTLIVE, PP_E_CUDA, PP_E_NOSPACE = 0, -1, -2, -3, -4, -5, -6
PP_S_NAN, PP_S_INDEX, PP_S_TIMEOUT = 0x1, 0x2, 0x4
ERRORS = {PP_EINVAL: "PP_EINVAL", PP_E_BUSY: "PP_E_BUSY", PP_E_RANGE: "PP_E_RANGE",
          PP_E_NOTLIVE: "PP_E_NOTLIVE", PP_E_CUDA: "PP_E_CUDA", PP_E_NOSPACE: "PP_E_NOSPACE"}

# Order of enum pp_weight in pp.h.
WEIGHT_NAMES = ["emb_text", "emb_audio", "attn_alpha", "wqkv", "wo", "mlp_alpha", "wgu",
                "wdown", "out_alpha", "wtext", "dep_inproj", "dep_emb_text", "dep_emb_audio",
                "dep_attn_alpha", "dep_wqkv", "dep_wo", "dep_mlp_alpha", "dep_wgu",
                "dep_wdown", "dep_out_alpha", "dep_heads"]
PP_W_COUNT = len(WEIGHT_NAMES)

# Every function pp.h declares (checked against the header and the library by the tests).
EXPORTS = ["pp_weight_shape", "pp_workspace_bytes", "pp_create", "pp_destroy",
           "pp_session_open", "pp_session_close", "pp_session_import", "pp_session_pos",
           "pp_ring_block", "pp_step", "pp_step_host", "pp_status", "pp_step_kernel_count",
           "pp_profile_step", "pp_ring_attention_scratch_bytes", "pp_ring_attention",
           "pp_ring_attention_noalloc", "pp_rvq_dequantize", "pp_driver_create",
           "pp_driver_destroy", "pp_driver_open", "pp_driver_close", "pp_driver_phase",
           "pp_driver_prepare", "pp_driver_absorb", "pp_driver_tick", "pp_session_sampling",
           "pp_sample", "pp_test_faults", "pp_paged_append",
           "pp_paged_attention_scratch_bytes", "pp_paged_attention", "pp_paged_mass",
           "pp_paged_evict", "pp_test_paged_faults"]

# enum pp_kernel_kind
KERNEL_KINDS = ["begin", "norm", "qkv", "rope_ring", "attn", "oproj", "gateup", "down",
                "text_head", "dep_inproj", "dep_norm", "dep_qkv", "dep_attn", "dep_oproj",
                "dep_gateup", "dep_down", "dep_head", "finish", "dep_persist"]


class PPError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__("%s failed: %s (%d)" % (fn, ERRORS.get(code, "?"), code))
        self.code = code


class pp_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ["d_model", "n_layers", "n_heads", "ffn", "text_vocab", "audio_card", "n_q",
                 "dep_d", "dep_layers", "dep_heads", "dep_ffn", "window", "max_batch"]] + [
        ("eps", ctypes.c_float), ("rope_base", ctypes.c_float), ("flags", ctypes.c_int32)]

PP_FLAG_CUDA_CORE_GEMM = 0x1
PP_FLAG_NO_PDL = 0x2
PP_FLAG_TWO_GROUPS = 0x4
PP_FLAG_SKIP_USER_STEPS = 0x8
PP_FLAG_SEQUENTIAL_USER_STEPS = 0x10
PP_FLAG_WIDE_TILES = 0x20
PP_FLAG_LOW_LATENCY = 0x40


class pp_sampling(ctypes.Structure):
    """Per-session sampling parameters (temperature <= 0 keeps a stream greedy)."""
    _fields_ = [("text_temperature", ctypes.c_float), ("text_top_k", ctypes.c_int32),
                ("text_top_p", ctypes.c_float), ("repetition_penalty", ctypes.c_float),
                ("penalty_window", ctypes.c_int32), ("audio_temperature", ctypes.c_float),
                ("audio_top_k", ctypes.c_int32), ("audio_top_p", ctypes.c_float),
                ("seed", ctypes.c_uint64)]


SAMPLE_HISTORY = 256   # the longest repetition-penalty window


PP_F32, PP_BF16, PP_F16 = 0, 1, 2


class pp_paged_kv(ctypes.Structure):
    """One cache of pages with its block table (device pointers)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("mass", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("page_stride", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ["n_pages", "page_size", "n_kv_heads", "head_dim", "type",
                                      "n_seqs", "table_ld"]]


class pp_weights(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p * PP_W_COUNT)]


_lib = None


def lib():
    """Load libpp.so (building it first if it is missing or older than its sources)."""
    global _lib
    if _lib is None:
        from . import build
        build.build()
        if not os.path.exists(SO):
            raise RuntimeError("libpp.so is missing; run __graft_entry__.build()")
        L = ctypes.CDLL(SO)
        P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.pp_weight_shape.argtypes = [P, I, P, P, P]
        L.pp_weight_shape.restype = I
        L.pp_workspace_bytes.argtypes = [P]
        L.pp_workspace_bytes.restype = ctypes.c_size_t
        L.pp_create.argtypes = [P, P, P, ctypes.c_size_t, P]
        L.pp_create.restype = I
        L.pp_destroy.argtypes = [P]
        L.pp_destroy.restype = None
        for f in ["pp_session_open", "pp_session_close"]:
            getattr(L, f).argtypes = [P, I]
            getattr(L, f).restype = I
        L.pp_session_import.argtypes = [P, I, I64]
        L.pp_session_import.restype = I
        L.pp_session_pos.argtypes = [P, I, P]
        L.pp_session_pos.restype = I
        L.pp_ring_block.argtypes = [P, I, I, I, P]
        L.pp_ring_block.restype = I
        L.pp_step.argtypes = [P] * 8
        L.pp_step.restype = I
        L.pp_step_host.argtypes = [P] * 8
        L.pp_step_host.restype = I
        L.pp_status.argtypes = [P, P, P]
        L.pp_status.restype = I
        L.pp_step_kernel_count.argtypes = [P]
        L.pp_step_kernel_count.restype = I
        L.pp_test_faults.argtypes = [P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P]
        L.pp_test_faults.restype = I
        L.pp_profile_step.argtypes = [P] * 10
        L.pp_profile_step.restype = I
        L.pp_ring_attention_scratch_bytes.argtypes = [I, I, I, I]
        L.pp_ring_attention_scratch_bytes.restype = ctypes.c_size_t
        L.pp_ring_attention.argtypes = [P, P, P, I64, P, I, I, I, I, P, P, P, ctypes.c_size_t, P]
        L.pp_ring_attention.restype = I
        L.pp_ring_attention_noalloc.argtypes = [P, P, P, I64, P, I, I, I, I, P, P, P]
        L.pp_ring_attention_noalloc.restype = I
        L.pp_rvq_dequantize.argtypes = [P, I, I, I, P, I, I, P, P, P]
        L.pp_rvq_dequantize.restype = I
        L.pp_driver_create.argtypes = [I, I, I, ctypes.POINTER(P)]
        L.pp_driver_create.restype = I
        L.pp_driver_destroy.argtypes = [P]
        L.pp_driver_destroy.restype = None
        L.pp_driver_open.argtypes = [P, P, ctypes.POINTER(pp_prompt), ctypes.POINTER(I)]
        L.pp_driver_open.restype = I
        L.pp_driver_close.argtypes = [P, P, I]
        L.pp_driver_close.restype = I
        L.pp_driver_phase.argtypes = [P, I]
        L.pp_driver_phase.restype = I
        L.pp_driver_prepare.argtypes = [P, P, P, P, P, P]
        L.pp_driver_prepare.restype = I
        L.pp_driver_absorb.argtypes = [P, P, P, P]
        L.pp_driver_absorb.restype = I
        L.pp_driver_tick.argtypes = [P, P, P, P, P, P]
        L.pp_session_sampling.argtypes = [P, I, ctypes.POINTER(pp_sampling)]
        L.pp_session_sampling.restype = I
        F = ctypes.c_float
        L.pp_sample.argtypes = [P, I64, I, I, F, I, F, F, P, I, P, P, P, P, P]
        L.pp_sample.restype = I
        L.pp_driver_tick.restype = I
        KV = ctypes.POINTER(pp_paged_kv)
        L.pp_paged_append.argtypes = [KV, P, I64, P, I64, P, I64, I, P, P, F, F, I, I, P, P, P, I,
                                      I, P, P, P]
        L.pp_paged_append.restype = I
        L.pp_paged_attention_scratch_bytes.argtypes = [KV, I, I, I, I]
        L.pp_paged_attention_scratch_bytes.restype = ctypes.c_size_t
        L.pp_paged_attention.argtypes = [KV, P, I64, P, P, I, I, I, F, I, P, P, P, P,
                                         ctypes.c_size_t, P]
        L.pp_paged_attention.restype = I
        L.pp_paged_mass.argtypes = [KV, P, I64, P, P, P, I, I, I, F, I, F, P, P]
        L.pp_paged_mass.restype = I
        L.pp_paged_evict.argtypes = [KV, P, I, I, KV, P, P, P, P]
        L.pp_paged_evict.restype = I
        L.pp_test_paged_faults.argtypes = [ctypes.c_int32, ctypes.c_int32]
        L.pp_test_paged_faults.restype = I
        _lib = L
    return _lib


def _check(fn, rc):
    if rc != PP_OK:
        raise PPError(fn, rc)
    return rc


def make_config(shape, max_batch, flags=0):
    """pp_config from an object with the model's dimensions (by attribute name)."""
    return pp_config(shape.d, shape.n_layers, shape.n_heads, shape.ffn, shape.text_vocab,
                     shape.audio_card, shape.n_q, shape.dep_d, shape.dep_layers,
                     shape.dep_heads, shape.dep_ffn, shape.window, int(max_batch),
                     float(shape.eps), float(shape.rope_base), int(flags))


# ---- the C ABI, one wrapper per entry point -------------------------------------------

def pp_weight_shape(cfg, which):
    dims = (ctypes.c_int64 * 4)()
    nd, f32 = ctypes.c_int(), ctypes.c_int()
    _check("pp_weight_shape", lib().pp_weight_shape(ctypes.byref(cfg), which, dims,
                                                    ctypes.byref(nd), ctypes.byref(f32)))
    return tuple(dims[:nd.value]), bool(f32.value)


def pp_workspace_bytes(cfg):
    n = lib().pp_workspace_bytes(ctypes.byref(cfg))
    if n == 0:
        raise PPError("pp_workspace_bytes", PP_EINVAL)
    return n


def pp_create(cfg, weight_ptrs, workspace_ptr, ws_bytes):
    w = pp_weights()
    for i, p in enumerate(weight_ptrs):
        w.ptr[i] = p
    h = ctypes.c_void_p()
    _check("pp_create", lib().pp_create(ctypes.byref(cfg), ctypes.byref(w), workspace_ptr,
                                        ws_bytes, ctypes.byref(h)))
    return h


def pp_destroy(h):
    lib().pp_destroy(h)


def pp_session_open(h, slot):
    return _check("pp_session_open", lib().pp_session_open(h, slot))


def pp_session_close(h, slot):
    return _check("pp_session_close", lib().pp_session_close(h, slot))


def pp_session_import(h, slot, pos):
    return _check("pp_session_import", lib().pp_session_import(h, slot, pos))


def pp_session_pos(h, slot):
    v = ctypes.c_int64()
    _check("pp_session_pos", lib().pp_session_pos(h, slot, ctypes.byref(v)))
    return v.value


def pp_ring_block(h, layer, slot, kv):
    p = ctypes.c_void_p()
    _check("pp_ring_block", lib().pp_ring_block(h, layer, slot, kv, ctypes.byref(p)))
    return p.value


def pp_step(h, prev_column, user_codes, force_mask, forced_tokens, column, logits, stream):
    return _check("pp_step", lib().pp_step(h, prev_column, user_codes, force_mask,
                                           forced_tokens, column, logits, stream))


def pp_step_host(h, prev_column, user_codes, force_mask, forced_tokens, column, logits, stream):
    return _check("pp_step_host", lib().pp_step_host(h, prev_column, user_codes, force_mask,
                                                     forced_tokens, column, logits, stream))


def pp_status(h, stream):
    v = ctypes.c_uint32()
    _check("pp_status", lib().pp_status(h, stream, ctypes.byref(v)))
    return v.value


def pp_step_kernel_count(h):
    return lib().pp_step_kernel_count(h)


PP_TEST_UMMA, PP_TEST_ATTN, PP_TEST_PERSIST = 0x1, 0x2, 0x4


def pp_test_faults(h, wait_polls, withhold, kinds, stream):
    """Failure-detection tests only: lower the bounded waits' poll budget and have
    producers of the named kernel families withhold copies (0, 0, 0 resets)."""
    return _check("pp_test_faults", lib().pp_test_faults(h, wait_polls, withhold, kinds, stream))


def pp_profile_step(h, prev_column, user_codes, force_mask, forced_tokens, column, logits,
                    stream, kind_ms, kind_launches):
    """kind_ms: ctypes double array, kind_launches: ctypes int64 array (accumulated)."""
    return _check("pp_profile_step", lib().pp_profile_step(
        h, prev_column, user_codes, force_mask, forced_tokens, column, logits, stream,
        kind_ms, kind_launches))


def pp_ring_attention_scratch_bytes(B, H, head_dim, window):
    n = lib().pp_ring_attention_scratch_bytes(B, H, head_dim, window)
    if n == 0:
        raise PPError("pp_ring_attention_scratch_bytes", PP_EINVAL)
    return n


def pp_ring_attention(q, k, v, slot_stride, n_valid, B, H, head_dim, window, out, status,
                      scratch, scratch_bytes, stream):
    return _check("pp_ring_attention", lib().pp_ring_attention(
        q, k, v, slot_stride, n_valid, B, H, head_dim, window, out, status, scratch,
        scratch_bytes, stream))


def pp_ring_attention_noalloc(q, k, v, slot_stride, n_valid, B, H, head_dim, window, out,
                              status, stream):
    """pp_ring_attention with the library's built-in scratch (no allocation)."""
    return _check("pp_ring_attention_noalloc", lib().pp_ring_attention_noalloc(
        q, k, v, slot_stride, n_valid, B, H, head_dim, window, out, status, stream))


PP_DRV_FREE, PP_DRV_VOICE, PP_DRV_SILENCE, PP_DRV_PERSONA, PP_DRV_LIVE = 0, 1, 2, 3, 4


class pp_prompt(ctypes.Structure):
    _fields_ = [("voice_frames", ctypes.c_void_p), ("n_voice", ctypes.c_int),
                ("persona_tokens", ctypes.c_void_p), ("n_persona", ctypes.c_int),
                ("silence_frame", ctypes.c_void_p), ("silence_ticks", ctypes.c_int)]


class Driver:
    """The session driver (admission, prefill, acoustic delay) over host numpy buffers.
    With an Engine, tick() runs pp_step through it; without one, prepare()/absorb() give
    the bookkeeping alone."""

    def __init__(self, max_batch, text_vocab, audio_card):
        h = ctypes.c_void_p()
        _check("pp_driver_create", lib().pp_driver_create(max_batch, text_vocab, audio_card,
                                                          ctypes.byref(h)))
        self.h, self.B = h, max_batch

    def close_driver(self):
        if self.h:
            lib().pp_driver_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close_driver()
        except Exception:
            pass

    def open(self, voice=None, persona=None, silence=None, silence_ticks=0, engine=None,
             sampling=None):
        """Admit a session (lowest free slot) and open it on `engine`; `sampling` (a
        pp_sampling) sets its sampling parameters there."""
        if sampling is not None and engine is None:
            raise ValueError("sampling parameters live on the engine: pass engine=")
        keep = []
        def arr(a):
            if a is None:
                return None, 0
            a = np.ascontiguousarray(a, dtype=np.int32)
            keep.append(a)
            return a.ctypes.data, a.shape[0]
        v, nv = arr(voice)
        p_, np_ = arr(persona)
        s_, _ = arr(silence)
        pr = pp_prompt(v, nv, p_, np_, s_, silence_ticks)
        slot = ctypes.c_int(-1)
        _check("pp_driver_open", lib().pp_driver_open(self.h, engine.h if engine else None,
                                                      ctypes.byref(pr), ctypes.byref(slot)))
        if sampling is not None:
            engine.set_sampling(slot.value, sampling)
        return slot.value

    def close(self, slot, engine=None):
        return _check("pp_driver_close",
                      lib().pp_driver_close(self.h, engine.h if engine else None, slot))

    def phase(self, slot):
        return lib().pp_driver_phase(self.h, slot)

    def prepare(self, user_frames):
        u = np.ascontiguousarray(user_frames, dtype=np.int32)
        prev = np.empty((self.B, 17), np.int32)
        user = np.empty((self.B, 8), np.int32)
        mask = np.empty((self.B, 17), np.uint8)
        forced = np.empty((self.B, 17), np.int32)
        _check("pp_driver_prepare", lib().pp_driver_prepare(
            self.h, u.ctypes.data, prev.ctypes.data, user.ctypes.data, mask.ctypes.data,
            forced.ctypes.data))
        return prev, user, mask, forced

    def absorb(self, user_frames, column):
        u = np.ascontiguousarray(user_frames, dtype=np.int32)
        c = np.ascontiguousarray(column, dtype=np.int32)
        out = np.empty((self.B, 9), np.int32)
        _check("pp_driver_absorb", lib().pp_driver_absorb(self.h, u.ctypes.data, c.ctypes.data,
                                                          out.ctypes.data))
        return out

    def tick(self, engine, user_frames):
        u = np.ascontiguousarray(user_frames, dtype=np.int32)
        out = np.empty((self.B, 9), np.int32)
        col = np.empty((self.B, 17), np.int32)
        _check("pp_driver_tick", lib().pp_driver_tick(self.h, engine.h, u.ctypes.data,
                                                      out.ctypes.data, col.ctypes.data,
                                                      engine._stream()))
        return out, col


def pp_rvq_dequantize(codes, code_stride, n_frames, n_books, codebooks, card, dim, out, status,
                      stream):
    """Latent of each frame = sum of the codebook entries its codes select (device)."""
    return _check("pp_rvq_dequantize", lib().pp_rvq_dequantize(
        codes, code_stride, n_frames, n_books, codebooks, card, dim, out, status, stream))


def pp_session_sampling(h, slot, params=None):
    """Sampling parameters of an open slot (a pp_sampling, or None for greedy)."""
    return _check("pp_session_sampling", lib().pp_session_sampling(
        h, slot, None if params is None else ctypes.byref(params)))


def pp_sample(logits, ld, rows, n, temperature, top_k, top_p, penalty, hist, hist_ld, hist_n,
              uniforms, tokens, status, stream):
    """One token per row of device logits with the caller's uniforms (device pointers)."""
    return _check("pp_sample", lib().pp_sample(logits, ld, rows, n, temperature, top_k, top_p,
                                               penalty, hist, hist_ld, hist_n, uniforms, tokens,
                                               status, stream))


def sampling(text_temperature=0.0, text_top_k=0, text_top_p=1.0, repetition_penalty=1.0,
             penalty_window=0, audio_temperature=0.0, audio_top_k=0, audio_top_p=1.0, seed=0):
    """A pp_sampling with greedy defaults."""
    return pp_sampling(text_temperature, text_top_k, text_top_p, repetition_penalty,
                       penalty_window, audio_temperature, audio_top_k, audio_top_p,
                       int(seed) & (2**64 - 1))


def pp_paged_append(kv, q, q_stride, k, k_stride, v, v_stride, in_type, q_alpha, k_alpha, eps,
                    rope_base, rot_dim, halves, positions, cu, kv_len, T, n_heads, q_out, status,
                    stream):
    """Norm and rotation of new queries and keys; keys and values into the paged cache."""
    return _check("pp_paged_append", lib().pp_paged_append(
        ctypes.byref(kv), q, q_stride, k, k_stride, v, v_stride, in_type, q_alpha, k_alpha, eps,
        rope_base, rot_dim, halves, positions, cu, kv_len, T, n_heads, q_out, status, stream))


def pp_paged_attention_scratch_bytes(kv, n_heads, T, max_q, window):
    n = lib().pp_paged_attention_scratch_bytes(ctypes.byref(kv), n_heads, T, max_q, window)
    if n == 0:
        raise PPError("pp_paged_attention_scratch_bytes", PP_EINVAL)
    return n


def pp_paged_attention(kv, q, q_stride, cu, kv_len, T, max_q, n_heads, scale, window, out, lse,
                       status, scratch, scratch_bytes, stream):
    """Attention of new rows over the paged cache."""
    return _check("pp_paged_attention", lib().pp_paged_attention(
        ctypes.byref(kv), q, q_stride, cu, kv_len, T, max_q, n_heads, scale, window, out, lse,
        status, scratch, scratch_bytes, stream))


def pp_paged_mass(kv, q, q_stride, lse, cu, kv_len, T, max_q, n_heads, scale, window, decay, status,
                  stream):
    """The attention weight that new rows give to each entry, added to the cache's mass."""
    return _check("pp_paged_mass", lib().pp_paged_mass(
        ctypes.byref(kv), q, q_stride, lse, cu, kv_len, T, max_q, n_heads, scale, window, decay,
        status, stream))


def pp_test_paged_faults(wait_polls, withhold):
    """Failure-detection tests of the paged calls of this thread; reset with (0, 0)."""
    return _check("pp_test_paged_faults", lib().pp_test_paged_faults(wait_polls, withhold))


def pp_paged_evict(kv, kv_len, budget, recent, to, to_len, kept, status, stream):
    """The newest and heaviest entries of the paged cache into another's pages."""
    return _check("pp_paged_evict", lib().pp_paged_evict(
        ctypes.byref(kv), kv_len, budget, recent, ctypes.byref(to), to_len, kept, status, stream))


# ---- convenience wrapper over torch device memory ---------------------------------------

class Engine:
    """One engine over torch-owned device memory (weights dict + workspace)."""

    def __init__(self, shape, max_batch, weights, device="cuda", flags=0):
        import torch
        self.torch = torch
        self.shape = shape
        self.B = int(max_batch)
        self.cfg = make_config(shape, max_batch, flags)
        self.weights = weights
        ptrs = []
        for i, name in enumerate(WEIGHT_NAMES):
            t = weights[name]
            dims, f32 = pp_weight_shape(self.cfg, i)
            if tuple(t.shape) != dims or t.element_size() != (4 if f32 else 2):
                raise ValueError("weight %s: shape %s, expected %s" % (name, tuple(t.shape), dims))
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("weight %s must be a contiguous CUDA tensor" % name)
            ptrs.append(t.data_ptr())
        self.ws_bytes = pp_workspace_bytes(self.cfg)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.h = pp_create(self.cfg, ptrs, self.workspace.data_ptr(), self.ws_bytes)
        self.logits_ld = shape.text_vocab + shape.n_q * shape.audio_card
        self.column = torch.empty((self.B, ROWS), dtype=torch.int32, device=device)

    def close_engine(self):
        if self.h:
            pp_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close_engine()
        except Exception:
            pass

    def _stream(self):
        return self.torch.cuda.current_stream().cuda_stream

    def open(self, slot):
        pp_session_open(self.h, slot)

    def close(self, slot):
        pp_session_close(self.h, slot)

    def set_sampling(self, slot, params=None, **kw):
        """Sampling parameters of an open slot: a pp_sampling, keyword fields of one, or
        nothing for greedy."""
        if params is None and kw:
            params = sampling(**kw)
        pp_session_sampling(self.h, slot, params)

    def import_session(self, slot, pos):
        pp_session_import(self.h, slot, pos)

    def pos(self, slot):
        return pp_session_pos(self.h, slot)

    def ring_block(self, layer, slot, kv):
        return pp_ring_block(self.h, layer, slot, kv)

    def kernel_count(self):
        return pp_step_kernel_count(self.h)

    def status(self):
        return pp_status(self.h, self._stream())

    def test_faults(self, wait_polls=0, withhold=0, kinds=0):
        pp_test_faults(self.h, wait_polls, withhold, kinds, self._stream())

    def step(self, prev_column, user_codes, force_mask=None, forced=None, logits=None,
             out=None):
        """One tick on device tensors; returns the column tensor (``out`` or the
        engine's own buffer, overwritten by the next step)."""
        col = self.column if out is None else out
        pp_step(self.h, prev_column.data_ptr(), user_codes.data_ptr(),
                None if force_mask is None else force_mask.data_ptr(),
                None if forced is None else forced.data_ptr(), col.data_ptr(),
                None if logits is None else logits.data_ptr(), self._stream())
        return col

    def profile_step(self, prev_column, user_codes, kind_ms, kind_launches, out=None):
        """One tick through the profiling graph; accumulates per-kind ms / launches."""
        col = self.column if out is None else out
        pp_profile_step(self.h, prev_column.data_ptr(), user_codes.data_ptr(), None, None,
                        col.data_ptr(), None, self._stream(), kind_ms, kind_launches)
        return col

    def step_host(self, prev_column, user_codes, force_mask, forced, column, logits=None):
        """One tick on host (numpy or pinned torch) buffers; blocks until done."""
        def ptr(a):
            if a is None:
                return None
            return a.data_ptr() if hasattr(a, "data_ptr") else a.ctypes.data
        pp_step_host(self.h, ptr(prev_column), ptr(user_codes), ptr(force_mask), ptr(forced),
                     ptr(column), ptr(logits), self._stream())
        return column


class PagedKV:
    """One layer's paged cache over torch-owned device memory.

    ``k`` and ``v`` are [pages, kv_heads, page_size, head_dim] in bf16 or fp16, ``table``
    [sequences, table width] int32 page numbers, ``mass`` (optional) f32 [pages, kv_heads,
    page_size].  ``cu`` is int32 [sequences + 1] row offsets and ``kv_len`` int32 [sequences]
    entry counts, the new entries included.  Every call runs on the cache's device, on its
    current stream.  Tensors that do not fit raise ValueError; what the library refuses
    raises PPError."""

    def __init__(self, k, v, table, mass=None, status=None):
        import torch
        self.torch = torch
        self.types = {torch.float32: PP_F32, torch.bfloat16: PP_BF16, torch.float16: PP_F16}
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise ValueError("k and v must be [pages, heads, rows, dims] of one layout and type")
        if k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("the cache holds bf16 or fp16, not %s" % k.dtype)
        if not k.is_cuda or v.device != k.device:
            raise ValueError("k and v must be on one CUDA device")
        n_pages, heads, rows, dim = k.shape
        if n_pages and not k[0].is_contiguous():
            raise ValueError("each page of k and v must be contiguous")
        if table.dim() != 2:
            raise ValueError("table must be [sequences, width]")
        self.device, self.index, self.dtype = k.device, k.get_device(), k.dtype
        self.k, self.v, self.table, self.mass = k, v, table, mass
        self.heads, self.dim, self.n = heads, dim, table.shape[0]
        self._fits("table", table, torch.int32, table.shape)
        self.mass_shape = (n_pages, heads, rows)
        if mass is not None:
            self._fits("mass", mass, torch.float32, self.mass_shape)
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._fits("status", status, torch.int32, (1,))
        self.status = status
        # stands in for a scratch that a call asks for but does not use (the smallest size)
        self.unused = torch.empty(256, dtype=torch.uint8, device=self.device)
        stride = k.stride(0) if n_pages > 1 else heads * rows * dim
        self.c = pp_paged_kv(k.data_ptr(), v.data_ptr(), self._ptr(mass), table.data_ptr(),
                             stride, n_pages, rows, heads, dim, self.types[k.dtype],
                             table.shape[0], table.shape[1])
        self.ref, self.lib, self.sizes = ctypes.byref(self.c), lib(), {}
        # the current stream's handle without building a stream object, where torch offers it
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)

    @staticmethod
    def _ptr(t):
        return None if t is None else t.data_ptr()

    def _fits(self, name, t, dtype, shape):
        """Raise unless t is a contiguous tensor of this cache's device, of this type and shape."""
        if (t.get_device() != self.index or t.dtype is not dtype or t.shape != shape
                or not t.is_contiguous()):
            raise ValueError("%s: %s %s on %s, expected contiguous %s %s on %s" % (
                name, t.dtype, tuple(t.shape), t.device, dtype, tuple(shape), self.device))
        return t

    def _rows(self, name, t, dtype):
        """(rows, heads, row stride) of a [rows, heads, dims] tensor whose rows are contiguous."""
        if t.get_device() != self.index or t.dtype is not dtype or t.dim() != 3:
            raise ValueError("%s: %s %s on %s, expected [rows, heads, %d] in %s on %s" % (
                name, t.dtype, tuple(t.shape), t.device, self.dim, dtype, self.device))
        T, H, D = t.shape
        row, head, one = t.stride()
        if D != self.dim or (T and H and (one != 1 or (H > 1 and head != D))):
            raise ValueError("%s: shape %s, strides %s: the heads of a row must be contiguous, of "
                             "%d values" % (name, tuple(t.shape), t.stride(), self.dim))
        return T, H, row if T > 1 else H * D

    def _batch(self, cu, kv_len):
        self._fits("cu", cu, self.torch.int32, (self.n + 1,))
        self._fits("kv_len", kv_len, self.torch.int32, (self.n,))

    def _call(self, name, *args):
        """One library call on the cache's device and that device's current stream."""
        cuda, fn = self.torch.cuda, getattr(self.lib, name)
        if cuda.current_device() == self.index:
            rc = fn(*args, self.raw_stream(self.index))
        else:
            with cuda.device(self.index):
                rc = fn(*args, self.raw_stream(self.index))
        if rc != PP_OK:
            raise PPError(name, rc)

    def _scratch_bytes(self, *shape):
        """Scratch of an attention call, by its shape (heads, rows, max_q, window)."""
        n = self.sizes.get(shape)
        if n is None:
            if len(self.sizes) >= 1024:
                self.sizes.clear()
            n = self.sizes[shape] = pp_paged_attention_scratch_bytes(self.c, *shape)
        return n

    @staticmethod
    def _longest(max_q, T):
        # The library's hint is an int32 of at least 1.  A caller's is handed on whatever T is: it
        # picks the kernel and its tiles, and with them a sequence's bits, which must not depend on
        # how many rows the rest of the batch has.
        return max(1, min(T if max_q is None else max_q, 2 ** 31 - 1))

    def read_status(self):
        """Wait for the current stream, then read and clear the status word."""
        bits = int(self.status.item())
        self.status.zero_()
        return bits

    def append(self, q, k, v, cu, kv_len, positions=None, q_alpha=None, k_alpha=None, eps=1e-5,
               rope_base=10000.0, rot_dim=None, halves=False, out=None):
        """New queries normed and rotated ([rows, heads, dims], returned in the cache's type);
        new keys, the same way, and values become cache entries."""
        torch, dtype = self.torch, q.dtype
        if dtype not in self.types:
            raise ValueError("q must be f32 or the cache's type, not %s" % dtype)
        T, H, qs = self._rows("q", q, dtype)
        kT, kH, ks = self._rows("k", k, dtype)
        vT, vH, vs = self._rows("v", v, dtype)
        if kT != T or vT != T or kH != self.heads or vH != self.heads:
            raise ValueError("k and v must have %d rows of %d heads" % (T, self.heads))
        self._batch(cu, kv_len)
        if q_alpha is not None:
            self._fits("q_alpha", q_alpha, torch.float32, (self.dim,))
        if k_alpha is not None:
            self._fits("k_alpha", k_alpha, torch.float32, (self.dim,))
        if positions is not None:
            self._fits("positions", positions, torch.int32, (T,))
        if out is None:
            out = torch.empty((T, H, self.dim), dtype=self.dtype, device=self.device)
        else:
            self._fits("out", out, self.dtype, (T, H, self.dim))
        self._call("pp_paged_append", self.ref, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                   self.types[dtype], self._ptr(q_alpha), self._ptr(k_alpha), eps, rope_base,
                   self.dim if rot_dim is None else rot_dim, int(halves), self._ptr(positions),
                   cu.data_ptr(), kv_len.data_ptr(), T, H, out.data_ptr(), self.status.data_ptr())
        return out

    def attention(self, q, cu, kv_len, max_q=None, scale=None, window=0, with_lse=False,
                  out=None):
        """Attention of the new rows over the cache: out, or (out, lse) on request.  max_q is
        the longest chunk as far as the host knows.  It picks the kernel: give it where chunks are
        short.  Without it all rows count as one chunk, so the kernel, and with it a sequence's
        bits, goes by the batch's row count.  out must not lie over q."""
        torch = self.torch
        T, H, qs = self._rows("q", q, self.dtype)
        self._batch(cu, kv_len)
        if out is None:
            out = torch.empty((T, H, self.dim), dtype=self.dtype, device=self.device)
        else:
            self._fits("out", out, self.dtype, (T, H, self.dim))
        lse = torch.empty((T, H), dtype=torch.float32, device=self.device) if with_lse else None
        max_q = self._longest(max_q, T)
        nbytes = self._scratch_bytes(H, T, max_q, window)
        scratch = self.unused if nbytes <= 256 else \
            torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self._call("pp_paged_attention", self.ref, q.data_ptr(), qs, cu.data_ptr(), kv_len.data_ptr(),
                   T, max_q, H, self.dim ** -0.5 if scale is None else scale, window,
                   out.data_ptr(), self._ptr(lse), self.status.data_ptr(), scratch.data_ptr(),
                   nbytes)
        return (out, lse) if with_lse else out

    def attention_mass(self, q, lse, cu, kv_len, max_q=None, scale=None, window=0, decay=1.0,
                       mass=None):
        """Add the attention weight of the new rows to the cache's mass (or to ``mass``, of the
        same layout)."""
        T, H, qs = self._rows("q", q, self.dtype)
        self._fits("lse", lse, self.torch.float32, (T, H))
        self._batch(cu, kv_len)
        c = self.ref
        if mass is not None:
            self._fits("mass", mass, self.torch.float32, self.mass_shape)
            other = pp_paged_kv.from_buffer_copy(self.c)
            other.mass = mass.data_ptr()
            c = ctypes.byref(other)
        elif self.mass is None:
            raise ValueError("this cache keeps no mass")
        self._call("pp_paged_mass", c, q.data_ptr(), qs, lse.data_ptr(), cu.data_ptr(),
                   kv_len.data_ptr(), T, self._longest(max_q, T), H,
                   self.dim ** -0.5 if scale is None else scale, window, decay,
                   self.status.data_ptr())

    def evict(self, kv_len, budget, recent, to):
        """Keep the newest `recent` and the heaviest other entries, `budget` in all, in the
        PagedKV `to`; returns (lengths there, the entries kept)."""
        torch = self.torch
        if self.mass is None:
            raise ValueError("this cache keeps no mass")
        if to.index != self.index:
            raise ValueError("both caches must be on one device")
        self._fits("kv_len", kv_len, torch.int32, (self.n,))
        to_len = torch.empty(self.n, dtype=torch.int32, device=self.device)
        kept = torch.empty((self.n, self.heads, max(budget, 0)), dtype=torch.int32,
                           device=self.device)
        self._call("pp_paged_evict", self.ref, kv_len.data_ptr(), budget, recent, to.ref,
                   to_len.data_ptr(), kept.data_ptr(), self.status.data_ptr())
        return to_len, kept
