"""Thin ctypes binding of libmac_gb300.so (the C ABI in include/mac.h).

The functions keep the C names and only marshal arguments: every step of
the decode path runs in the library's CUDA kernels.  PyTorch provides the
device memory and streams (``MacLayer`` allocates the workspaces).  There is
no fallback: loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

MAC_OK, MAC_ERR_INVALID_ARG, MAC_ERR_UNSUPPORTED, MAC_ERR_CUDA = 0, -1, -2, -3
MAC_DEV_BAD_SEQ_LEN, MAC_DEV_BAD_PAGE, MAC_DEV_WAIT_TIMEOUT, MAC_DEV_NONFINITE_Q, MAC_DEV_BAD_COPY = 1, 2, 4, 8, 16
MAC_DEV_NO_ROOM, MAC_DEV_BAD_PARENT, MAC_DEV_NONFINITE_LOGIT = 32, 64, 128
MAC_MAX_BEAMS, MAC_MAX_CANDIDATES = 16, 32
MAC_TRACE_POINTS = 32
MAC_BF16, MAC_F32 = 0, 1
MAC_THR_ONE_MINUS_TAU, MAC_THR_TAU = 0, 1
MAC_ROPE_HALF, MAC_ROPE_INTERLEAVED, MAC_ROPE_NONE = 0, 1, 2

# every function the header declares (checked against include/mac.h by the tests)
EXPORTS = ("mac_workspace_size", "mac_ring_layout_of", "mac_init_rings", "mac_decode_step",
           "mac_full_attention", "mac_full_attention_noalloc", "mac_join_aux", "mac_release_ring",
           "mac_last_status", "mac_set_phase_events", "mac_set_trace", "mac_status_string",
           "mac_threshold_sq", "mac_reset_requests", "mac_test_wait_budget",
           "mac_chunk_workspace_size", "mac_build_tables", "mac_write_kv", "mac_chunk_attention",
           "mac_cross_attention", "mac_beam_workspace_size", "mac_beam_select",
           "mac_reorder_tables", "mac_reorder_state")
MAC_NOALLOC_SCRATCH_BYTES = 16 << 20


class mac_config(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("ring_k", ctypes.c_int32), ("band_r", ctypes.c_int32),
        ("tau", ctypes.c_double), ("thr_mode", ctypes.c_int32), ("rope_base", ctypes.c_double),
        ("rope_mode", ctypes.c_int32), ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("min_context", ctypes.c_int32), ("max_context", ctypes.c_int64),
        ("front_sink", ctypes.c_int32),
    ]


class mac_kv(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("capacity", ctypes.c_int64), ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int32),
    ]


class mac_pages(ctypes.Structure):
    _fields_ = [
        ("page_table", ctypes.c_void_p), ("free_pages", ctypes.c_void_p), ("n_free_in", ctypes.c_void_p),
        ("n_free_out", ctypes.c_void_p), ("capacity", ctypes.c_int64), ("max_pages", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
    ]


class mac_ring_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("pos", "q", "o", "lse", "stage_q", "stage_o", "stage_lse", "ctl", "total")]


class MacError(RuntimeError):
    pass


_LIB = None


def lib_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libmac_gb300.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise MacError(f"{path} is missing: build it with long_context_decode_gb300.build.build()")
    L = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    P = ctypes.POINTER
    L.mac_workspace_size.argtypes = [P(mac_config), P(ctypes.c_size_t), P(ctypes.c_size_t)]
    L.mac_ring_layout_of.argtypes = [P(mac_config), P(mac_ring_layout)]
    L.mac_init_rings.argtypes = [P(mac_config), vp, vp, vp, vp, i32, P(mac_kv), vp]
    L.mac_decode_step.argtypes = [P(mac_config), vp, vp, vp, vp, P(mac_kv), vp, vp, vp, vp]
    L.mac_full_attention.argtypes = [P(mac_config), vp, vp, vp, P(mac_kv), vp, vp, vp]
    L.mac_full_attention_noalloc.argtypes = [P(mac_config), vp, vp, P(mac_kv), vp, vp, vp]
    L.mac_join_aux.argtypes = [vp, vp]
    L.mac_release_ring.argtypes = [vp]
    L.mac_last_status.argtypes = [P(mac_config), vp, P(i32), vp]
    L.mac_set_phase_events.argtypes = [vp, vp, vp]
    L.mac_set_trace.argtypes = [vp]
    L.mac_reset_requests.argtypes = [P(mac_config), vp, vp, vp]
    L.mac_test_wait_budget.argtypes = [i64, i32]
    L.mac_chunk_workspace_size.argtypes = [P(mac_config), i32, P(ctypes.c_size_t)]
    L.mac_build_tables.argtypes = [P(mac_config), vp, P(mac_pages), vp, vp, vp, i32, vp, vp, vp, vp, vp]
    L.mac_write_kv.argtypes = [P(mac_config), vp, vp, i64, vp, i64, vp, i64, vp, vp, i32, P(mac_kv), vp, vp]
    L.mac_chunk_attention.argtypes = [P(mac_config), vp, vp, vp, vp, i32, P(mac_kv), vp, vp, vp]
    L.mac_cross_attention.argtypes = [P(mac_config), vp, vp, vp, i32, vp, i32, P(mac_kv), vp, vp, vp]
    L.mac_beam_workspace_size.argtypes = [P(mac_config), i32, i32, i32, P(ctypes.c_size_t)]
    L.mac_beam_select.argtypes = [P(mac_config), vp, i32, vp, i32, i64, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
    L.mac_reorder_tables.argtypes = [P(mac_config), vp, P(mac_pages), i32, vp, vp, vp, vp, vp, vp, vp]
    L.mac_reorder_state.argtypes = [P(mac_config), vp, vp, i32, vp, P(mac_kv), vp]
    L.mac_status_string.argtypes = [ctypes.c_int]
    L.mac_status_string.restype = ctypes.c_char_p
    L.mac_threshold_sq.argtypes = [P(mac_config)]
    L.mac_threshold_sq.restype = ctypes.c_float
    for n in EXPORTS:
        if n not in ("mac_status_string", "mac_threshold_sq"):
            getattr(L, n).restype = ctypes.c_int
    _LIB = L
    return L


def _check(code: int, what: str) -> None:
    if code != MAC_OK:
        raise MacError(f"{what}: {load().mac_status_string(code).decode()} ({code})")


def _ptr(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


# ---------------------------------------------------------------------------
# the C entry points, same names, marshalling only
# ---------------------------------------------------------------------------

def mac_workspace_size(cfg: mac_config) -> tuple[int, int]:
    ring, scratch = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().mac_workspace_size(ctypes.byref(cfg), ctypes.byref(ring), ctypes.byref(scratch)),
           "mac_workspace_size")
    return ring.value, scratch.value


def mac_ring_layout_of(cfg: mac_config) -> mac_ring_layout:
    lay = mac_ring_layout()
    _check(load().mac_ring_layout_of(ctypes.byref(cfg), ctypes.byref(lay)), "mac_ring_layout_of")
    return lay


def mac_init_rings(cfg, ring, scratch, q_seed, prompt_len, n_seed, kv: mac_kv, stream=None):
    _check(load().mac_init_rings(ctypes.byref(cfg), _ptr(ring), _ptr(scratch), _ptr(q_seed),
                                 _ptr(prompt_len), int(n_seed),
                                 ctypes.byref(kv) if kv is not None else None, _stream(stream)),
           "mac_init_rings")


def mac_decode_step(cfg, ring, scratch, q_pre, seq_len, kv: mac_kv, out, match_pos=None,
                    stream_main=None, stream_aux=None):
    _check(load().mac_decode_step(ctypes.byref(cfg), _ptr(ring), _ptr(scratch), _ptr(q_pre),
                                  _ptr(seq_len), ctypes.byref(kv), _ptr(out), _ptr(match_pos),
                                  _stream(stream_main), _stream(stream_aux)), "mac_decode_step")


def mac_full_attention(cfg, scratch, q_pre, seq_len, kv: mac_kv, out, lse=None, stream=None):
    _check(load().mac_full_attention(ctypes.byref(cfg), _ptr(scratch), _ptr(q_pre), _ptr(seq_len),
                                     ctypes.byref(kv), _ptr(out), _ptr(lse), _stream(stream)),
           "mac_full_attention")


def mac_full_attention_noalloc(cfg, q_pre, seq_len, kv: mac_kv, out, lse=None, stream=None):
    """mac_full_attention with its scratch in the library's fixed array
    (for callers that cannot allocate device memory; see include/mac.h)."""
    _check(load().mac_full_attention_noalloc(ctypes.byref(cfg), _ptr(q_pre), _ptr(seq_len),
                                             ctypes.byref(kv), _ptr(out), _ptr(lse), _stream(stream)),
           "mac_full_attention_noalloc")


def mac_join_aux(ring, stream_main=None):
    _check(load().mac_join_aux(_ptr(ring), _stream(stream_main)), "mac_join_aux")


def mac_release_ring(ring):
    _check(load().mac_release_ring(_ptr(ring)), "mac_release_ring")


def mac_last_status(cfg, scratch, stream=None) -> int:
    st = ctypes.c_int32()
    _check(load().mac_last_status(ctypes.byref(cfg), _ptr(scratch), ctypes.byref(st), _stream(stream)),
           "mac_last_status")
    return st.value


def mac_set_phase_events(before_match=None, after_match=None, after_attend=None):
    """Arm the next mac_decode_step on this thread to record these
    torch.cuda.Event objects (or raw cudaEvent_t handles)."""
    def h(e):
        if e is None or isinstance(e, int):
            return e
        return e.cuda_event
    _check(load().mac_set_phase_events(h(before_match), h(after_match), h(after_attend)),
           "mac_set_phase_events")


def mac_set_trace(buffer):
    """Arm the next step kernel on this thread to write per-CTA phase
    timestamps into ``buffer`` (a torch uint64/int64 tensor of >= 8 * SMs)."""
    _check(load().mac_set_trace(_ptr(buffer)), "mac_set_trace")


def mac_reset_requests(cfg: mac_config, ring, reset_flags, stream=None):
    """Requests whose flag (device int32 tensor [B]) is set start over with
    empty rings: their next step misses on every head; the flags are
    cleared on the device."""
    _check(load().mac_reset_requests(ctypes.byref(cfg), _ptr(ring), _ptr(reset_flags), _stream(stream)),
           "mac_reset_requests")


def mac_test_wait_budget(cycles: int, withhold_use: int = -1):
    """Test hook: the next step kernel on this thread gives every bounded
    wait ``cycles`` SM cycles and never copies stage use ``withhold_use``."""
    _check(load().mac_test_wait_budget(int(cycles), int(withhold_use)), "mac_test_wait_budget")


def mac_chunk_workspace_size(cfg: mac_config, n_tokens: int) -> int:
    n = ctypes.c_size_t()
    _check(load().mac_chunk_workspace_size(ctypes.byref(cfg), int(n_tokens), ctypes.byref(n)),
           "mac_chunk_workspace_size")
    return n.value


def mac_build_tables(cfg, chunk_ws, pages: mac_pages, reset_flags, len_in, new_len, n_tokens, len_out, q_start, pos,
                     slot, stream=None):
    """Pages, packed rows, positions and slots of a batch of new tokens,
    from device lengths (see include/mac.h)."""
    _check(load().mac_build_tables(ctypes.byref(cfg), _ptr(chunk_ws), ctypes.byref(pages) if pages is not None else None,
                                   _ptr(reset_flags), _ptr(len_in), _ptr(new_len), int(n_tokens), _ptr(len_out),
                                   _ptr(q_start), _ptr(pos), _ptr(slot), _stream(stream)), "mac_build_tables")


def _row_stride(t, heads, head_dim, rows=0) -> int:
    """Elements between rows of [T, heads, d] whose rows are whole, T >= rows
    (a raw pointer's rows lie end to end)."""
    if t is None or isinstance(t, int):
        return heads * head_dim
    try:
        (n, h, d), (row, head, one) = t.shape, t.stride()
    except ValueError:
        n = h = d = row = head = one = 0
    if n < rows or h < heads or d != head_dim:
        raise MacError(f"mac_write_kv: {rows} rows of {heads} heads of {head_dim} are needed, not {tuple(t.shape)}")
    if (head != d and h != 1) or one != 1:
        raise MacError("mac_write_kv: a row's heads must lie end to end")
    return row if n != 1 else heads * head_dim  # (one row's stride may be anything)


def _whole(t, n, what) -> int | None:
    """Pointer of a tensor that the library takes as n elements end to end."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_contiguous() or t.numel() < n:
        raise MacError(f"{what} must be {n} elements end to end")
    return t.data_ptr()


def mac_write_kv(cfg, chunk_ws, q, k, v, pos, slot, n_tokens, kv: mac_kv, q_out, stream=None):
    """Rotate and store the rows of a batch.  q, k, v: [T, heads, d] tensors,
    strided views of a fused projection included, or pointers to contiguous
    rows; q_out contiguous; q and q_out None for keys and values only."""
    d, hq, hkv, n = cfg.head_dim, cfg.n_q_heads, cfg.n_kv_heads, int(n_tokens)
    _check(load().mac_write_kv(ctypes.byref(cfg), _ptr(chunk_ws), _ptr(q), _row_stride(q, hq, d, n), _ptr(k),
                               _row_stride(k, hkv, d, n), _ptr(v), _row_stride(v, hkv, d, n), _ptr(pos), _ptr(slot), n,
                               ctypes.byref(kv) if kv is not None else None, _whole(q_out, n * hq * d, "mac_write_kv: q_out"),
                               _stream(stream)), "mac_write_kv")


def mac_chunk_attention(cfg, chunk_ws, q, q_start, seq_len, n_tokens, kv: mac_kv, out, lse=None, stream=None):
    """Exact causal attention of a batch's rotated rows over the cache; q, out
    and lse contiguous."""
    n = int(n_tokens)
    rows = n * cfg.n_q_heads
    _check(load().mac_chunk_attention(ctypes.byref(cfg), _ptr(chunk_ws), _whole(q, rows * cfg.head_dim, "mac_chunk_attention: q"),
                                      _ptr(q_start), _ptr(seq_len), n, ctypes.byref(kv) if kv is not None else None,
                                      _whole(out, rows * cfg.head_dim, "mac_chunk_attention: out"),
                                      _whole(lse, rows, "mac_chunk_attention: lse"), _stream(stream)), "mac_chunk_attention")


def mac_cross_attention(cfg, chunk_ws, q, q_start, group, mem_len, n_tokens, kv: mac_kv, out, lse=None, stream=None):
    """Attention of the rows of each source's ``group`` slots over the whole of
    that source's memory; q, out and lse contiguous."""
    n = int(n_tokens)
    rows = n * cfg.n_q_heads
    _check(load().mac_cross_attention(ctypes.byref(cfg), _ptr(chunk_ws), _whole(q, rows * cfg.head_dim, "mac_cross_attention: q"),
                                      _ptr(q_start), int(group), _ptr(mem_len), n, ctypes.byref(kv) if kv is not None else None,
                                      _whole(out, rows * cfg.head_dim, "mac_cross_attention: out"),
                                      _whole(lse, rows, "mac_cross_attention: lse"), _stream(stream)), "mac_cross_attention")


def mac_beam_workspace_size(cfg: mac_config, n_beams: int, vocab: int, n_out: int) -> int:
    n = ctypes.c_size_t()
    _check(load().mac_beam_workspace_size(ctypes.byref(cfg), int(n_beams), int(vocab), int(n_out), ctypes.byref(n)),
           "mac_beam_workspace_size")
    return n.value


_LOGITS: dict = {}  # torch dtype -> MAC_*, filled at the first call


def mac_beam_select(cfg, beam_ws, n_beams, logits, scores, done, end_token, n_out, placed, scores_out, parent, token, done_out=None,
                    stream=None):
    """The n_out best next tokens of every group's beams.  logits: a [slots,
    vocab] tensor of bf16 or fp32, its rows any distance apart."""
    if not _LOGITS:
        import torch
        _LOGITS.update({torch.bfloat16: MAC_BF16, torch.float32: MAC_F32})
    S, kind = cfg.batch, _LOGITS.get(logits.dtype)
    groups = S // n_beams * n_out if n_beams > 0 else 0
    try:
        (rows, vocab), (stride, one) = logits.shape, logits.stride()
    except ValueError:
        rows = vocab = stride = one = 0
    if kind is None or rows < S or (one != 1 and vocab > 1):
        raise MacError(f"mac_beam_select: logits must be {S} rows of bf16 or fp32, a row's elements end to end")
    if rows == 1:
        stride = vocab  # (one row's stride may be anything)
    _check(load().mac_beam_select(ctypes.byref(cfg), _ptr(beam_ws), n_beams, logits.data_ptr(), kind, stride, vocab,
                                  _whole(scores, S, "mac_beam_select: scores"), _whole(done, S, "mac_beam_select: done"), end_token, n_out,
                                  int(placed), _whole(scores_out, groups, "mac_beam_select: scores_out"),
                                  _whole(parent, groups, "mac_beam_select: parent"), _whole(token, groups, "mac_beam_select: token"),
                                  _whole(done_out, groups, "mac_beam_select: done_out"), _stream(stream)), "mac_beam_select")


def mac_reorder_tables(cfg, chunk_ws, pages: mac_pages | None, n_beams, parent, len_in, len_out, shared_in, shared_out, moves,
                       stream=None):
    """Slots take over their parents' pages, lengths and common positions; moves
    ([slots, 8] int32) says what mac_reorder_state has to move.  A slot begins
    anew with parent -1; one that does so in another way (reset flags, where it
    shares no page) gets its row and its column of the common positions cleared
    by the caller first."""
    S = cfg.batch
    pairs = S * n_beams
    _check(load().mac_reorder_tables(ctypes.byref(cfg), _ptr(chunk_ws), ctypes.byref(pages) if pages is not None else None, n_beams,
                                     _whole(parent, S, "mac_reorder_tables: parent"), _whole(len_in, S, "mac_reorder_tables: len_in"),
                                     _whole(len_out, S, "mac_reorder_tables: len_out"), _whole(shared_in, pairs, "mac_reorder_tables: shared_in"),
                                     _whole(shared_out, pairs, "mac_reorder_tables: shared_out"), _whole(moves, S * 8, "mac_reorder_tables: moves"),
                                     _stream(stream)), "mac_reorder_tables")


def mac_reorder_state(cfg, chunk_ws, ring, n_beams, moves, kv: mac_kv | None, stream=None):
    """One layer's part of the moves: its rings (or None) and its cache (or None), in place."""
    _check(load().mac_reorder_state(ctypes.byref(cfg), _ptr(chunk_ws), _ptr(ring), int(n_beams),
                                    _whole(moves, cfg.batch * 8, "mac_reorder_state: moves"),
                                    ctypes.byref(kv) if kv is not None else None, _stream(stream)), "mac_reorder_state")


def mac_status_string(code: int) -> str:
    return load().mac_status_string(code).decode()


def mac_threshold_sq(cfg: mac_config) -> float:
    return float(load().mac_threshold_sq(ctypes.byref(cfg)))


# ---------------------------------------------------------------------------
# convenience: configuration and torch-allocated workspaces
# ---------------------------------------------------------------------------

def config(batch, n_q_heads, n_kv_heads, head_dim=128, ring_k=1024, band_r=256, tau=0.6,
           thr_mode=MAC_THR_ONE_MINUS_TAU, rope_base=10000.0, rope_mode=MAC_ROPE_HALF,
           dtype=MAC_BF16, page_size=0, min_context=0, max_context=131072, front_sink=0) -> mac_config:
    return mac_config(batch, n_q_heads, n_kv_heads, head_dim, ring_k, band_r, float(tau), thr_mode,
                      float(rope_base), rope_mode, dtype, page_size, min_context, int(max_context),
                      int(front_sink))


def kv_view(k, v, page_table=None, capacity=0, max_pages=0, n_pages=0) -> mac_kv:
    """K/V descriptor from torch tensors (contiguous [B, Hkv, cap, d] or
    paged [n_pages, Hkv, 16, d] + page table [B, max_pages])."""
    if page_table is None:
        capacity = capacity or k.shape[2]
    else:
        max_pages = max_pages or page_table.shape[1]
        n_pages = n_pages or k.shape[0]
    return mac_kv(_ptr(k), _ptr(v), _ptr(page_table), int(capacity), int(max_pages), int(n_pages))


def pages_view(page_table=None, free_pages=None, n_free_in=None, n_free_out=None, capacity=0, max_pages=0,
               n_pages=0) -> mac_pages:
    """Page pool descriptor from torch tensors: page table [B, max_pages], free
    stack [n_pages] and its counts (n_free_out defaults to n_free_in), or
    just the capacity of a contiguous cache."""
    if page_table is not None:
        max_pages = max_pages or page_table.shape[1]
        n_pages = n_pages or free_pages.shape[0]
        n_free_out = n_free_in if n_free_out is None else n_free_out
    view = mac_pages(_ptr(page_table), _ptr(free_pages), _ptr(n_free_in), _ptr(n_free_out), int(capacity),
                     int(max_pages), int(n_pages))
    view.tensors = (page_table, free_pages, n_free_in, n_free_out)  # alive as long as the view
    return view


class MacLayer:
    """One layer's ring workspace plus a (possibly shared) scratch workspace,
    allocated with torch on the current CUDA device."""

    def __init__(self, cfg: mac_config, scratch=None, device="cuda"):
        import torch
        self.cfg = cfg
        ring_bytes, scratch_bytes = mac_workspace_size(cfg)
        self.ring = torch.zeros(ring_bytes, dtype=torch.uint8, device=device)
        self.scratch = scratch if scratch is not None else torch.zeros(scratch_bytes, dtype=torch.uint8,
                                                                        device=device)
        self.layout = mac_ring_layout_of(cfg)

    def ring_view(self, part: str):
        """A typed torch view of one part of the ring workspace."""
        import torch
        c, L = self.cfg, self.layout
        B, H, K, d = c.batch, c.n_q_heads, c.ring_k, c.head_dim
        qdt = torch.bfloat16 if c.dtype == MAC_BF16 else torch.float32
        spec = {
            "pos": (L.pos, torch.int32, (B, K)),
            "q": (L.q, qdt, (B, H, K, d)),
            "o": (L.o, torch.float32, (B, H, K, d)),
            "lse": (L.lse, torch.float32, (B, H, K)),
            "stage_q": (L.stage_q, qdt, (B, H, d)),
            "stage_o": (L.stage_o, torch.float32, (B, H, d)),
            "stage_lse": (L.stage_lse, torch.float32, (B, H)),
        }[part]
        off, dt, shape = spec
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        return self.ring[off:off + nbytes].view(dt).view(shape)

    def release(self):
        mac_release_ring(self.ring)
