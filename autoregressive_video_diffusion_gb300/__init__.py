"""Python binding of libdcp, the GB300 (sm_103a) DeCoPrune history-KV prune step.

Argument marshalling only: every function here passes tensor addresses and sizes to the C ABI declared in
``include/dcp.h`` (same names) on torch's current CUDA stream, and raises :class:`DcpError` on a non-zero status.
Every step of the prune runs in the library's CUDA kernels; there is no CPU or PyTorch fallback, and importing this
package fails if ``libdcp.so`` has not been built (``python autoregressive_video_diffusion_gb300/build.py``).

The method (page "DeCoPrune이 디노이징 불일치로 비디오 KV 캐시를 85% 줄인다", onedev.kr/papers/726): score each
token of the chunk that leaves the dense window by l = (1/d)||x0hat(tau*) - x_final||^2, keep the tokens with
l > gamma (one mask for every layer), physically gather K[m], V[m] into the compacted history, and re-index the
temporal RoPE phase of history keys to t~(t) = q0 - g(q0 - t).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdcp.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python autoregressive_video_diffusion_gb300/build.py` "
                      "(nvcc, sm_103a).  There is no fallback implementation.")

lib = ctypes.CDLL(LIB_PATH)

DCP_OK, DCP_EINVAL, DCP_ECAPACITY, DCP_ECUDA, DCP_ETIMEOUT, DCP_EDEVICE = range(6)
DCP_BF16, DCP_F32 = 0, 1

# The page's fixed choices (section "premises and limits"): 4-step schedule, probe at zero-based index 2, gamma.
SCHEDULE = (999, 957, 899, 702)
PROBE_INDEX = 2
TAU_STAR = SCHEDULE[PROBE_INDEX]
GAMMA = 0.10


class DcpCacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("L", ctypes.c_int32), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("cap", ctypes.c_int64),
                ("hist_cap", ctypes.c_int64), ("hist_len", ctypes.c_void_p), ("hist_t", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class DcpConfigC(ctypes.Structure):
    _fields_ = [("gamma", ctypes.c_float), ("keep_rule", ctypes.c_int32), ("sink_chunks", ctypes.c_int32),
                ("window_chunks", ctypes.c_int32), ("tokens_per_frame", ctypes.c_int32),
                ("frames_per_chunk", ctypes.c_int32), ("n_temporal_pairs", ctypes.c_int32),
                ("pair_layout", ctypes.c_int32), ("rope_base", ctypes.c_double), ("g_recent_R", ctypes.c_double),
                ("g_span_S", ctypes.c_double), ("g_mode", ctypes.c_int32), ("rephase_sink", ctypes.c_int32),
                ("max_frames", ctypes.c_int32), ("random_seed", ctypes.c_uint32), ("reindex_mode", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class DcpPagedCacheC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("L", ctypes.c_int32),
                ("H", ctypes.c_int32), ("D", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("layout", ctypes.c_int32), ("n_blocks", ctypes.c_int64),
                ("hist_cap", ctypes.c_int64), ("hist_blocks", ctypes.c_void_p), ("window_blocks", ctypes.c_void_p),
                ("hist_len", ctypes.c_void_p), ("hist_t", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class DcpKvPoolC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("block_size", ctypes.c_int32), ("n_blocks", ctypes.c_int64),
                ("s_block", ctypes.c_int64), ("s_head", ctypes.c_int64), ("s_row", ctypes.c_int64)]


class DcpSeqBatchC(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("total_q", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("kv_len_per_head", ctypes.c_int32), ("max_kv", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("kv_len_add", ctypes.c_int64), ("q_start", ctypes.c_void_p), ("tables", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("status", ctypes.c_void_p)]


DCP_ROPE_MAX_PAIRS = 64


class DcpRopeConfigC(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("pair_layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("amplitude", ctypes.c_double)]


class DcpRopePlanC(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("pair_layout", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("ready", ctypes.c_int32), ("turns", ctypes.c_uint64 * DCP_ROPE_MAX_PAIRS)]


class DcpAttnConfigC(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class DcpPagePoolC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("L", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("n_blocks", ctypes.c_int64), ("page_bytes", ctypes.c_int64), ("status", ctypes.c_void_p)]


class DcpPrCounter(ctypes.Structure):
    _fields_ = [("visible", ctypes.c_int64), ("full", ctypes.c_int64)]


_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_pc, _pg = ctypes.POINTER(DcpCacheC), ctypes.POINTER(DcpConfigC)
_pk, _pb, _pa = ctypes.POINTER(DcpKvPoolC), ctypes.POINTER(DcpSeqBatchC), ctypes.POINTER(DcpAttnConfigC)
_pp = ctypes.POINTER(DcpPagePoolC)
_SIGS = {
    "dcp_workspace_size": ([_pc, _pg], _sz),
    "dcp_score_workspace_size": ([_i32], _sz),
    "dcp_workspace_init": ([_vp, _sz, _vp], _i32),
    "dcp_score_mask": ([_vp, _vp, _i32, _i32, _f32, _i32, ctypes.c_uint64, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                        _vp], _i32),
    "dcp_compact_layers": ([_pc, _pg, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp], _i32),
    "dcp_rope_reindex": ([_pc, _pg, _i32, _i32, _vp, _sz, _vp], _i32),
    "dcp_prune_step": ([_pc, _pg, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "dcp_workspace_outputs": ([_pc, _pg, _vp, _vp, _vp, _vp], _i32),
    "dcp_get_status": ([_vp, _vp], _i32),
    "dcp_reset_status": ([_vp, _vp], _i32),
    "dcp_status_string": ([_i32], ctypes.c_char_p),
    "dcp_pr_add_chunk": ([ctypes.POINTER(DcpPrCounter), _i64, _i64, _i64, _i64, _i64], None),
    "dcp_pr_value": ([ctypes.POINTER(DcpPrCounter)], ctypes.c_double),
    "dcp_abi_struct_sizes": ([], ctypes.c_uint32),
    "dcp_set_phase_events": ([_vp, _vp], _i32),
    "dcp_prune_step_noalloc": ([_pc, _pg, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp], _i32),
    "dcp_paged_workspace_size": ([ctypes.POINTER(DcpPagedCacheC), _pg], _sz),
    "dcp_paged_prune_step": ([ctypes.POINTER(DcpPagedCacheC), _pg, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp,
                              _vp, _vp, _sz, _vp], _i32),
    "dcp_paged_prune_step_shared": ([ctypes.POINTER(DcpPagedCacheC), _pg, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                     _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "dcp_abi_paged_cache_size": ([], ctypes.c_uint32),
    "dcp_read_history_keys": ([_pc, _pg, _i32, _i32, _i32, _vp, _vp, _sz, _vp], _i32),
    "dcp_phase_table": ([_pg, _i32, _i32, _i32, _vp, _vp], _i32),
    "dcp_paged_read_history_keys": ([ctypes.POINTER(DcpPagedCacheC), _pg, _i32, _i32, _i32, _vp, _vp, _sz, _vp],
                                    _i32),
    "dcp_snapshot_max_bytes": ([_pc, _pg, ctypes.c_uint32], _sz),
    "dcp_snapshot": ([_pc, _pg, ctypes.c_uint32, _i32, _vp, _sz, _vp, _sz, _vp], _i32),
    "dcp_restore": ([_pc, _pg, _vp, _sz, ctypes.POINTER(_i32), ctypes.POINTER(ctypes.c_uint32), _vp, _sz, _vp],
                    _i32),
    "dcp_rope_plan_init": ([ctypes.POINTER(DcpRopeConfigC), ctypes.POINTER(DcpRopePlanC)], _i32),
    "dcp_rope_append": ([_pk, _pb, ctypes.POINTER(DcpRopePlanC), _vp, _i64, _i32, _vp, _vp, _i64, _vp, _vp, _vp],
                        _i32),
    "dcp_attention_workspace_size": ([_pk, _pb, _pa, _i32], _sz),
    "dcp_paged_attention": ([_pk, _pb, _pa, _vp, _i64, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "dcp_pages_workspace_size": ([_pp, _i32, _i32], _sz),
    "dcp_pages_copy": ([_pp, _vp, _vp, _i32, _vp], _i32),
    "dcp_pages_fork": ([_pp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "dcp_pages_free": ([_pp, _vp, _i32, _i32, _vp, _vp, _vp, _vp], _i32),
    "dcp_pages_compact": ([_pp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "dcp_abi_serving_struct_size": ([_i32], ctypes.c_uint32),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

_sizes = lib.dcp_abi_struct_sizes()
if (_sizes >> 16) != ctypes.sizeof(DcpCacheC) or (_sizes & 0xFFFF) != ctypes.sizeof(DcpConfigC) or \
        lib.dcp_abi_paged_cache_size() != ctypes.sizeof(DcpPagedCacheC):
    raise ImportError("libdcp struct layout does not match the binding")
for _i, _t in enumerate((DcpKvPoolC, DcpSeqBatchC, DcpRopeConfigC, DcpRopePlanC, DcpAttnConfigC, DcpPagePoolC)):
    if lib.dcp_abi_serving_struct_size(_i) != ctypes.sizeof(_t):
        raise ImportError(f"libdcp struct layout does not match the binding: {_t.__name__}")


class DcpError(RuntimeError):
    def __init__(self, what: str, status: int):
        super().__init__(f"{what}: {dcp_status_string(status)} ({status})")
        self.status = status


def dcp_status_string(status: int) -> str:
    return lib.dcp_status_string(status).decode()


def _check(rc: int, what: str) -> None:
    if rc != DCP_OK:
        raise DcpError(what, rc)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# The current stream's handle without building a Stream object, where torch offers that (a few microseconds a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device_index = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _device_index is not None and torch.cuda.is_initialized():
        return _raw_stream(_device_index())
    return torch.cuda.current_stream().cuda_stream


@dataclass
class Config:
    """Method parameters (dcp_config)."""
    gamma: float = GAMMA
    keep_rule: int = 0
    sink_chunks: int = 1
    window_chunks: int = 3
    tokens_per_frame: int = 1560
    frames_per_chunk: int = 4
    n_temporal_pairs: int = 22
    rope_base: float = 10000.0
    g_recent_R: float = 12.0
    g_span_S: float = 24.0
    g_mode: int = 0
    max_frames: int = 256
    pair_layout: int = 0
    rephase_sink: int = 0
    random_seed: int = 0
    reindex_mode: int = 0

    @property
    def C(self) -> int:
        return self.tokens_per_frame * self.frames_per_chunk

    def c(self) -> DcpConfigC:
        return DcpConfigC(self.gamma, self.keep_rule, self.sink_chunks, self.window_chunks, self.tokens_per_frame,
                          self.frames_per_chunk, self.n_temporal_pairs, self.pair_layout, self.rope_base,
                          self.g_recent_R, self.g_span_S, self.g_mode, self.rephase_sink, self.max_frames,
                          self.random_seed & 0xFFFFFFFF, self.reindex_mode, 0)

    def random_stream(self, evict_first_frame: int) -> int:
        """SplitMix64 seed a prune step under keep_rule 2 draws from (as dcp_prune_step forms it)."""
        return ((self.random_seed & 0xFFFFFFFF) << 32) | (evict_first_frame & 0xFFFFFFFF)


class KVCache:
    """Device tensors of one KV cache in the sink | history | window-ring layout (dcp_cache)."""

    def __init__(self, L: int, H: int, D: int, dtype: int, cap: int, hist_cap: int, device="cuda"):
        tdt = torch.bfloat16 if dtype == DCP_BF16 else torch.float32
        self.L, self.H, self.D, self.dtype, self.cap, self.hist_cap = L, H, D, dtype, cap, hist_cap
        self.k = torch.empty((L, H, cap, D), dtype=tdt, device=device)
        self.v = torch.empty((L, H, cap, D), dtype=tdt, device=device)
        self.hist_len = torch.zeros(L * H, dtype=torch.int32, device=device)
        self.hist_t = torch.zeros(max(hist_cap, 1), dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def c(self) -> DcpCacheC:
        return DcpCacheC(_ptr(self.k), _ptr(self.v), self.L, self.H, self.D, self.dtype, self.cap, self.hist_cap,
                         _ptr(self.hist_len), _ptr(self.hist_t), _ptr(self.status))


def dcp_workspace_size(cache: KVCache, cfg: Config) -> int:
    cc, gc = cache.c(), cfg.c()
    n = lib.dcp_workspace_size(ctypes.byref(cc), ctypes.byref(gc))
    if n == 0:
        raise DcpError("dcp_workspace_size", DCP_EINVAL)
    return n


def dcp_score_workspace_size(n_tok: int) -> int:
    return lib.dcp_score_workspace_size(n_tok)


def dcp_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check(lib.dcp_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "dcp_workspace_init")


def new_workspace(nbytes: int, device="cuda", stream=None) -> torch.Tensor:
    """A zero-initialised, 256-byte aligned device workspace (torch allocation; not on the hot path)."""
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + nbytes]
    dcp_workspace_init(ws, stream)
    return ws


def dcp_score_mask(x0hat: torch.Tensor, xref: torch.Tensor, gamma: float, keep_rule: int, ell, mask, idx, kept,
                   status: torch.Tensor, ws: torch.Tensor, stream=None, random_stream: int = 0) -> None:
    n_tok, d = x0hat.shape
    _check(lib.dcp_score_mask(_ptr(x0hat), _ptr(xref), n_tok, d, gamma, keep_rule, random_stream, _ptr(ell),
                              _ptr(mask), _ptr(idx), _ptr(kept), _ptr(status), _ptr(ws), ws.numel(), _stream(stream)),
           "dcp_score_mask")


def dcp_compact_layers(cache: KVCache, cfg: Config, evict_slot: int, evict_first_frame: int, mask: torch.Tensor,
                       head_is_static, q0: int, kept, ws: torch.Tensor, stream=None) -> None:
    cc, gc = cache.c(), cfg.c()
    _check(lib.dcp_compact_layers(ctypes.byref(cc), ctypes.byref(gc), evict_slot, evict_first_frame, _ptr(mask),
                                  _ptr(head_is_static), q0, _ptr(kept), _ptr(ws), ws.numel(), _stream(stream)),
           "dcp_compact_layers")


def dcp_rope_reindex(cache: KVCache, cfg: Config, q0_prev: int, q0: int, ws: torch.Tensor, stream=None) -> None:
    cc, gc = cache.c(), cfg.c()
    _check(lib.dcp_rope_reindex(ctypes.byref(cc), ctypes.byref(gc), q0_prev, q0, _ptr(ws), ws.numel(),
                                _stream(stream)), "dcp_rope_reindex")


def dcp_prune_step(cache: KVCache, cfg: Config, x0hat: torch.Tensor, xref: torch.Tensor, evict_slot: int,
                   evict_first_frame: int, q0_prev: int, q0: int, head_is_static, kept_dev, kept_host_pinned,
                   ws: torch.Tensor, stream=None) -> None:
    cc, gc = cache.c(), cfg.c()
    _check(lib.dcp_prune_step(ctypes.byref(cc), ctypes.byref(gc), _ptr(x0hat), _ptr(xref), x0hat.shape[1],
                              evict_slot, evict_first_frame, q0_prev, q0, _ptr(head_is_static), _ptr(kept_dev),
                              _ptr(kept_host_pinned), _ptr(ws), ws.numel(), _stream(stream)), "dcp_prune_step")


DCP_NOALLOC_WORKSPACE_BYTES = (4 << 20) + (8 << 10)


def dcp_prune_step_noalloc(cache: KVCache, cfg: Config, x0hat: torch.Tensor, xref: torch.Tensor, evict_slot: int,
                           evict_first_frame: int, q0_prev: int, q0: int, head_is_static, kept_dev, kept_host_pinned,
                           stream=None) -> None:
    """dcp_prune_step without a workspace, for callers that cannot allocate device memory: the library's own fixed
    scratch array (DCP_NOALLOC_WORKSPACE_BYTES per GPU) is used instead.  Calls that overlap on the GPU race."""
    cc, gc = cache.c(), cfg.c()
    _check(lib.dcp_prune_step_noalloc(ctypes.byref(cc), ctypes.byref(gc), _ptr(x0hat), _ptr(xref), x0hat.shape[1],
                                      evict_slot, evict_first_frame, q0_prev, q0, _ptr(head_is_static),
                                      _ptr(kept_dev), _ptr(kept_host_pinned), _stream(stream)),
           "dcp_prune_step_noalloc")


def dcp_workspace_outputs(cache: KVCache, cfg: Config, ws: torch.Tensor):
    """Views of the workspace where the last prune/compact call left l (fp32), the mask (uint8), the index list."""
    cc, gc = cache.c(), cfg.c()
    pe, pm, pi = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib.dcp_workspace_outputs(ctypes.byref(cc), ctypes.byref(gc), _ptr(ws), ctypes.byref(pe),
                                     ctypes.byref(pm), ctypes.byref(pi)), "dcp_workspace_outputs")
    C, base = cfg.C, ws.data_ptr()
    ell = ws[pe.value - base: pe.value - base + 4 * C].view(torch.float32)
    mask = ws[pm.value - base: pm.value - base + C]
    idx = ws[pi.value - base: pi.value - base + 4 * C].view(torch.int32)
    return ell, mask, idx


def dcp_get_status(status: torch.Tensor, stream=None) -> int:
    return lib.dcp_get_status(_ptr(status), _stream(stream))


def dcp_reset_status(status: torch.Tensor, stream=None) -> None:
    _check(lib.dcp_reset_status(_ptr(status), _stream(stream)), "dcp_reset_status")


def dcp_pr_add_chunk(acc: DcpPrCounter, n_planes: int, hist_len_sum: int, sink_visible: int, window_visible: int,
                     prior_tokens: int) -> None:
    lib.dcp_pr_add_chunk(ctypes.byref(acc), n_planes, hist_len_sum, sink_visible, window_visible, prior_tokens)


def dcp_pr_value(acc: DcpPrCounter) -> float:
    return lib.dcp_pr_value(ctypes.byref(acc))


def dcp_set_phase_events(ev_after_scan, ev_after_gather) -> None:
    """Record torch.cuda.Event objects (or None) after the scan and gather kernels of each dcp_prune_step."""
    a = None if ev_after_scan is None else ev_after_scan.cuda_event
    b = None if ev_after_gather is None else ev_after_gather.cuda_event
    _check(lib.dcp_set_phase_events(a, b), "dcp_set_phase_events")


# ------------------------------------------------------------------------------------------ host snapshot
def dcp_snapshot_max_bytes(cache: KVCache, cfg: Config, live_slots: int) -> int:
    cc, gc = cache.c(), cfg.c()
    n = lib.dcp_snapshot_max_bytes(ctypes.byref(cc), ctypes.byref(gc), live_slots)
    if n == 0:
        raise DcpError("dcp_snapshot_max_bytes", DCP_EINVAL)
    return n


def new_snapshot_image(nbytes: int) -> torch.Tensor:
    """Page-locked, 256-byte aligned host buffer for a snapshot image (torch allocation; not on the hot path)."""
    buf = torch.empty(nbytes + 256, dtype=torch.uint8, pin_memory=True)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + nbytes]


def snapshot_total_bytes(image: torch.Tensor) -> int:
    """Size written by the snapshot held in `image` (its header's total_bytes; read after the stream synced)."""
    return int(image[88:96].view(torch.int64).item())


def dcp_snapshot(cache: KVCache, cfg: Config, live_slots: int, q0: int, image: torch.Tensor, ws: torch.Tensor,
                 stream=None) -> None:
    cc, gc = cache.c(), cfg.c()
    _check(lib.dcp_snapshot(ctypes.byref(cc), ctypes.byref(gc), live_slots, q0, _ptr(image), image.numel(),
                            _ptr(ws), ws.numel(), _stream(stream)), "dcp_snapshot")


def dcp_restore(cache: KVCache, cfg: Config, image: torch.Tensor, ws: torch.Tensor, stream=None):
    """Returns (q0, live_slots) of the image."""
    cc, gc = cache.c(), cfg.c()
    q0, live = ctypes.c_int32(0), ctypes.c_uint32(0)
    _check(lib.dcp_restore(ctypes.byref(cc), ctypes.byref(gc), _ptr(image), image.numel(), ctypes.byref(q0),
                           ctypes.byref(live), _ptr(ws), ws.numel(), _stream(stream)), "dcp_restore")
    return q0.value, live.value


# ------------------------------------------------------------------------------------------ paged variant
DCP_PAGED_HND, DCP_PAGED_NHD = 0, 1


class PagedKVCache:
    """Device block pools and block tables of one paged KV cache (dcp_paged_cache).

    Pools are [L][n_blocks][H][block_size][D] (HND) or [L][n_blocks][block_size][H][D] (NHD); hist_blocks and
    window_blocks are int32 device tensors the caller fills (block ids of the history positions and of the ring
    slots, slot s owning entries [s * C / block_size, (s + 1) * C / block_size)).  block_ref may be set to the blocks'
    reference counts (int32 [n_blocks], as the dcp_pages_* calls keep them): a prune step that would write a history
    block that another sequence holds too is then refused on the device (DCP_EDEVICE)."""

    def __init__(self, L: int, H: int, D: int, dtype: int, block_size: int, layout: int, n_blocks: int,
                 hist_cap: int, n_window_blocks: int, device="cuda"):
        tdt = torch.bfloat16 if dtype == DCP_BF16 else torch.float32
        shape = (L, n_blocks, H, block_size, D) if layout == DCP_PAGED_HND else (L, n_blocks, block_size, H, D)
        self.L, self.H, self.D, self.dtype = L, H, D, dtype
        self.block_size, self.layout, self.n_blocks, self.hist_cap = block_size, layout, n_blocks, hist_cap
        self.k_pool = torch.empty(shape, dtype=tdt, device=device)
        self.v_pool = torch.empty(shape, dtype=tdt, device=device)
        self.hist_blocks = torch.zeros(max(hist_cap // block_size, 1), dtype=torch.int32, device=device)
        self.window_blocks = torch.zeros(max(n_window_blocks, 1), dtype=torch.int32, device=device)
        self.block_ref = None
        self.hist_len = torch.zeros(L * H, dtype=torch.int32, device=device)
        self.hist_t = torch.zeros(max(hist_cap, 1), dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def c(self) -> DcpPagedCacheC:
        return DcpPagedCacheC(_ptr(self.k_pool), _ptr(self.v_pool), self.L, self.H, self.D, self.dtype,
                              self.block_size, self.layout, self.n_blocks, self.hist_cap, _ptr(self.hist_blocks),
                              _ptr(self.window_blocks), _ptr(self.hist_len), _ptr(self.hist_t), _ptr(self.status))


def dcp_paged_workspace_size(cache: PagedKVCache, cfg: Config) -> int:
    cc, gc = cache.c(), cfg.c()
    n = lib.dcp_paged_workspace_size(ctypes.byref(cc), ctypes.byref(gc))
    if n == 0:
        raise DcpError("dcp_paged_workspace_size", DCP_EINVAL)
    return n


def dcp_paged_prune_step(cache: PagedKVCache, cfg: Config, x0hat: torch.Tensor, xref: torch.Tensor, evict_slot: int,
                         evict_first_frame: int, q0_prev: int, q0: int, head_is_static, kept, kept_host,
                         ws: torch.Tensor, stream=None) -> None:
    """With cache.block_ref set: dcp_paged_prune_step_shared, which refuses to write history blocks held in common."""
    cc, gc = cache.c(), cfg.c()
    args = (_ptr(x0hat), _ptr(xref), x0hat.shape[1], evict_slot, evict_first_frame, q0_prev, q0, _ptr(head_is_static),
            _ptr(kept), _ptr(kept_host), _ptr(ws), ws.numel(), _stream(stream))
    ref = cache.block_ref
    if ref is None:
        _check(lib.dcp_paged_prune_step(ctypes.byref(cc), ctypes.byref(gc), *args), "dcp_paged_prune_step")
        return
    if ref.dtype != torch.int32 or not ref.is_contiguous() or not ref.is_cuda or ref.numel() != cache.n_blocks:
        raise DcpError("dcp_paged_prune_step", DCP_EINVAL)
    _check(lib.dcp_paged_prune_step_shared(ctypes.byref(cc), ctypes.byref(gc), _ptr(ref), *args),
           "dcp_paged_prune_step_shared")


def paged_row_map(cfg: Config, hist_cap: int, block_size: int, sink_blocks: torch.Tensor, hist_blocks: torch.Tensor,
                  window_blocks: torch.Tensor):
    """(block, row-in-block) of every row of the contiguous layout sink | history | ring, as int64 tensors on the
    tables' device.  For moving caches between the two layouts (set-up and checks; not on the prune path)."""
    C = cfg.C
    sink = cfg.sink_chunks * C
    dev = hist_blocks.device
    pos = torch.arange(sink + hist_cap + (cfg.window_chunks + 1) * C, device=dev)
    block = torch.empty_like(pos)
    region = [(0, sink, sink_blocks), (sink, sink + hist_cap, hist_blocks),
              (sink + hist_cap, pos.numel(), window_blocks)]
    for lo, hi, tbl in region:
        i = pos[lo:hi] - lo
        if hi > lo:
            block[lo:hi] = tbl.to(device=dev, dtype=torch.int64)[i // block_size]
    return block, pos % block_size


def paged_pack(pool: torch.Tensor, t: torch.Tensor, block: torch.Tensor, off: torch.Tensor, layout: int) -> None:
    """Write a contiguous [L][H][rows][D] tensor into a block pool through a row map."""
    if layout == DCP_PAGED_HND:
        pool[:, block, :, off, :] = t.permute(2, 0, 1, 3)
    else:
        pool[:, block, off] = t.permute(0, 2, 1, 3)


def paged_unpack(pool: torch.Tensor, block: torch.Tensor, off: torch.Tensor, layout: int) -> torch.Tensor:
    """Read a block pool back into a contiguous [L][H][rows][D] tensor through a row map."""
    if layout == DCP_PAGED_HND:
        return pool[:, block, :, off, :].permute(1, 2, 0, 3).contiguous()
    return pool[:, block, off].permute(0, 2, 1, 3).contiguous()


# ------------------------------------------------------------------------------------------ read-time re-index
def dcp_read_history_keys(cache, cfg: Config, q0: int, plane0: int, n_planes: int, out: torch.Tensor,
                          ws: torch.Tensor, stream=None) -> None:
    """History keys of planes [plane0, plane0 + n_planes) turned to t~(t; q0) into out [n_planes][hist_cap][D]
    (reindex_mode 1).  `cache` is a KVCache or a PagedKVCache."""
    cc, gc = cache.c(), cfg.c()
    fn = lib.dcp_paged_read_history_keys if isinstance(cache, PagedKVCache) else lib.dcp_read_history_keys
    _check(fn(ctypes.byref(cc), ctypes.byref(gc), q0, plane0, n_planes, _ptr(out), _ptr(ws), ws.numel(),
              _stream(stream)), "dcp_read_history_keys")


def dcp_phase_table(cfg: Config, q0: int, frame_lo: int, frame_hi: int, out: torch.Tensor, stream=None) -> None:
    """cos/sin entries {c_hi, c_lo, s_hi, s_lo} of the turn t -> t~(t; q0) for frames [frame_lo, frame_hi) and every
    temporal pair, into out (float32 [(frame_hi - frame_lo) * n_t * 4], device)."""
    gc = cfg.c()
    _check(lib.dcp_phase_table(ctypes.byref(gc), q0, frame_lo, frame_hi, _ptr(out), _stream(stream)),
           "dcp_phase_table")


# ------------------------------------------------------------------------------------------ serving operators
DCP_ROPE_INTERLEAVED, DCP_ROPE_HALF = 0, 1
DCP_ROPE_PLAIN, DCP_ROPE_LINEAR, DCP_ROPE_BASE, DCP_ROPE_PARTS = range(4)


class KVPool:
    """One layer's pages (dcp_kv_pool).  k, v: [n_blocks][H][block_size][D] (DCP_PAGED_HND) or
    [n_blocks][block_size][H][D] (DCP_PAGED_NHD), bf16 or fp32; views with other strides are fine as long as both
    have the same and D is dense."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, layout: int):
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.dim() != 4 or \
                k.stride(3) != 1 or k.dtype not in (torch.bfloat16, torch.float32) or not (k.is_cuda and v.is_cuda):
            raise DcpError("KVPool", DCP_EINVAL)
        h, r = (1, 2) if layout == DCP_PAGED_HND else (2, 1)
        self.k, self.v, self.D, self.H, self.dtype = k, v, k.shape[3], k.shape[h], k.dtype
        self._c = DcpKvPoolC(_ptr(k), _ptr(v), k.shape[h], k.shape[3],
                             DCP_BF16 if k.dtype == torch.bfloat16 else DCP_F32, k.shape[r], k.shape[0], k.stride(0),
                             k.stride(h), k.stride(r))
        self.ref = ctypes.byref(self._c)

    def c(self) -> DcpKvPoolC:
        return self._c


def layer_pool(cache, layer: int, block_size: int = 0) -> KVPool:
    """Layer `layer` of a PagedKVCache, or of a KVCache cut into pages of block_size rows (a divisor of cap): page b
    of the latter holds rows [b * block_size, (b + 1) * block_size) of every plane."""
    if isinstance(cache, PagedKVCache):
        return KVPool(cache.k_pool[layer], cache.v_pool[layer], cache.layout)
    if block_size < 1 or cache.cap % block_size:
        raise DcpError("layer_pool", DCP_EINVAL)
    k, v = (x[layer].view(cache.H, cache.cap // block_size, block_size, cache.D).transpose(0, 1)
            for x in (cache.k, cache.v))
    return KVPool(k, v, DCP_PAGED_HND)


class SeqBatch:
    """The ragged batch (dcp_seq_batch).  Device int32 tensors: q_start [n + 1], tables [n][stride], kv_len [n] (or
    [n][H]), status [1].  max_q and max_kv are bounds the host knows."""

    def __init__(self, q_start: torch.Tensor, tables: torch.Tensor, kv_len: torch.Tensor, status: torch.Tensor,
                 total_q: int, max_q: int, max_kv: int, kv_len_add: int = 0):
        n = tables.shape[0] if tables.dim() == 2 else -1
        if any(t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda
               for t in (q_start, tables, kv_len, status)) or q_start.numel() != n + 1 or \
                kv_len.dim() not in (1, 2) or kv_len.shape[0] != n:
            raise DcpError("SeqBatch", DCP_EINVAL)
        self.tensors = (q_start, tables, kv_len, status)
        self.n_seqs, self.total_q, self.kv_heads = n, total_q, kv_len.shape[1] if kv_len.dim() == 2 else 0
        self._c = DcpSeqBatchC(n, total_q, max_q, int(kv_len.dim() == 2), max_kv, tables.shape[1], kv_len_add,
                               _ptr(q_start), _ptr(tables), _ptr(kv_len), _ptr(status))
        self.ref = ctypes.byref(self._c)

    def c(self) -> DcpSeqBatchC:
        return self._c


@dataclass
class RopeConfig:
    """Rotary positions (dcp_rope_config)."""
    rot_dim: int
    pair_layout: int = DCP_ROPE_INTERLEAVED
    base: float = 10000.0
    scaling: int = DCP_ROPE_PLAIN
    factor: float = 1.0
    orig_len: float = 4096.0
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    amplitude: float = 1.0

    def c(self) -> DcpRopeConfigC:
        return DcpRopeConfigC(self.rot_dim, self.pair_layout, self.scaling, 0, self.base, self.factor, self.orig_len,
                              self.beta_fast, self.beta_slow, self.amplitude)


def dcp_rope_plan(cfg: RopeConfig) -> DcpRopePlanC:
    """The rotary plan of a config: made once, kept by the caller, passed to every dcp_rope_append."""
    plan, c = DcpRopePlanC(), cfg.c()
    _check(lib.dcp_rope_plan_init(ctypes.byref(c), ctypes.byref(plan)), "dcp_rope_plan_init")
    return plan


def _rows_of(t: torch.Tensor, pool: KVPool, batch: SeqBatch, heads: int, what: str) -> int:
    """Token stride of a [total_q][heads][D] tensor of the pool's type whose heads are dense."""
    n, D = batch.total_q, pool.D
    if t.dtype is not pool.dtype or t.shape != (n, heads, D) or not t.is_cuda:
        raise DcpError(what, DCP_EINVAL)
    token, head, dim = t.stride()
    if dim != 1 or (head != D and heads > 1):
        raise DcpError(what, DCP_EINVAL)
    return token if n > 1 else heads * D


def dcp_rope_append(pool: KVPool, batch: SeqBatch, plan: DcpRopePlanC, q, k: torch.Tensor, v: torch.Tensor,
                    positions, q_out, stream=None) -> None:
    """Turn q and k of the new tokens, put k and v into the pool's pages; q_out gets the turned q.  q, k, v are
    [total_q][heads][D] (views of one fused projection are fine), positions int32 [total_q] or None."""
    kv_stride = _rows_of(k, pool, batch, pool.H, "dcp_rope_append")
    if _rows_of(v, pool, batch, pool.H, "dcp_rope_append") != kv_stride or \
            (positions is not None and (positions.dtype != torch.int32 or not positions.is_contiguous() or
                                        not positions.is_cuda or positions.numel() != batch.total_q)):
        raise DcpError("dcp_rope_append", DCP_EINVAL)
    hq, q_stride = 0, 0
    if q is not None:
        hq = q.shape[1]
        q_stride = _rows_of(q, pool, batch, hq, "dcp_rope_append")
        if q_out is None or _rows_of(q_out, pool, batch, hq, "dcp_rope_append") != hq * pool.D:
            raise DcpError("dcp_rope_append", DCP_EINVAL)
    _check(lib.dcp_rope_append(pool.ref, batch.ref, plan, _ptr(q), q_stride, hq, _ptr(k), _ptr(v), kv_stride,
                               _ptr(positions), _ptr(q_out), _stream(stream)), "dcp_rope_append")


@dataclass
class AttnConfig:
    """Attention over the paged cache (dcp_attn_config); scale None: D ** -0.5."""
    scale: float | None = None
    causal: bool = True
    window: int = -1

    def c(self, D: int) -> DcpAttnConfigC:
        return DcpAttnConfigC(D ** -0.5 if self.scale is None else self.scale, int(self.causal), self.window, 0)


def dcp_attention_workspace_size(pool: KVPool, batch: SeqBatch, cfg: AttnConfig, Hq: int) -> int:
    n = lib.dcp_attention_workspace_size(pool.ref, batch.ref, cfg.c(pool.D), Hq)
    if n == 0:
        raise DcpError("dcp_attention_workspace_size", DCP_EINVAL)
    return n


def dcp_paged_attention(pool: KVPool, batch: SeqBatch, cfg: AttnConfig, q: torch.Tensor, out: torch.Tensor, lse,
                        ws: torch.Tensor, stream=None) -> None:
    """out [total_q][Hq][D] = attention of the new tokens q over the cache; lse (or None): fp32 [total_q][Hq]."""
    hq = q.shape[1]
    q_stride = _rows_of(q, pool, batch, hq, "dcp_paged_attention")
    if _rows_of(out, pool, batch, hq, "dcp_paged_attention") != hq * pool.D or batch.kv_heads not in (0, pool.H) or \
            (lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or not lse.is_cuda or
                                  lse.numel() != batch.total_q * hq)) or not ws.is_cuda:
        raise DcpError("dcp_paged_attention", DCP_EINVAL)
    _check(lib.dcp_paged_attention(pool.ref, batch.ref, cfg.c(pool.D), _ptr(q), q_stride, hq, _ptr(out), _ptr(lse),
                                   _ptr(ws), ws.numel(), _stream(stream)), "dcp_paged_attention")


class PagePool:
    """Every layer's pages (dcp_page_pool).  k, v: [L][n_blocks][...] contiguous, a page of block_size positions in
    the trailing dims (either layout of PagedKVCache)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, block_size: int, status: torch.Tensor):
        if k.shape != v.shape or k.dtype != v.dtype or k.dim() < 3 or not k.is_contiguous() or \
                not v.is_contiguous() or status.dtype != torch.int32 or not (k.is_cuda and v.is_cuda and status.is_cuda):
            raise DcpError("PagePool", DCP_EINVAL)
        self.tensors, self.n_blocks = (k, v, status), k.shape[1]
        self._c = DcpPagePoolC(_ptr(k), _ptr(v), k.shape[0], block_size, k.shape[1],
                               k.stride(1) * k.element_size(), _ptr(status))
        self.ref = ctypes.byref(self._c)

    @classmethod
    def of(cls, cache: PagedKVCache) -> "PagePool":
        return cls(cache.k_pool, cache.v_pool, cache.block_size, cache.status)

    def c(self) -> DcpPagePoolC:
        return self._c


def _ints(what: str, *tensors) -> None:
    for t in tensors:
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda):
            raise DcpError(what, DCP_EINVAL)


def dcp_pages_workspace_size(pool: PagePool, n_rows: int, stride: int) -> int:
    n = lib.dcp_pages_workspace_size(pool.ref, n_rows, stride)
    if n == 0:
        raise DcpError("dcp_pages_workspace_size", DCP_EINVAL)
    return n


def dcp_pages_copy(pool: PagePool, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Block dst[i] = block src[i] in every layer."""
    _ints("dcp_pages_copy", src, dst)
    if src.numel() != dst.numel():
        raise DcpError("dcp_pages_copy", DCP_EINVAL)
    _check(lib.dcp_pages_copy(pool.ref, _ptr(src), _ptr(dst), src.numel(), _stream(stream)), "dcp_pages_copy")


def dcp_pages_fork(pool: PagePool, tables: torch.Tensor, lens: torch.Tensor, parent: torch.Tensor, shared, reserve,
                   ref: torch.Tensor, child_tables: torch.Tensor, ref_out: torch.Tensor, ws: torch.Tensor,
                   stream=None) -> None:
    """Branch rows parent[c] of `tables` into child_tables; shared and reserve (int32 [n_children]) may be None.  Pages
    that will be written must not be shared: of a cache whose prune steps turn the history's keys (reindex_mode 0, q0 - T_s
    past the span) only those before the history are.  Set PagedKVCache.block_ref to `ref` to have this checked."""
    _ints("dcp_pages_fork", tables, lens, parent, shared, reserve, ref, child_tables, ref_out)
    if tables.dim() != 2 or not ws.is_cuda:
        raise DcpError("dcp_pages_fork", DCP_EINVAL)
    (rows, stride), n = tables.shape, parent.numel()
    if child_tables.shape != (n, stride) or lens.numel() != rows or ref.numel() != pool.n_blocks or \
            ref_out.numel() != pool.n_blocks or any(t is not None and t.numel() != n for t in (shared, reserve)):
        raise DcpError("dcp_pages_fork", DCP_EINVAL)
    _check(lib.dcp_pages_fork(pool.ref, _ptr(tables), _ptr(lens), rows, stride, _ptr(parent), _ptr(shared),
                              _ptr(reserve), n, _ptr(ref), _ptr(child_tables), _ptr(ref_out), _ptr(ws), ws.numel(),
                              _stream(stream)), "dcp_pages_fork")


def _tables_and_counts(what: str, pool: PagePool, tables, ref, tables_out, ref_out) -> None:
    _ints(what, tables, ref, tables_out, ref_out)
    if tables.dim() != 2 or tables_out.shape != tables.shape or ref.numel() != pool.n_blocks or \
            ref_out.numel() != pool.n_blocks:
        raise DcpError(what, DCP_EINVAL)


def dcp_pages_free(pool: PagePool, tables: torch.Tensor, ref: torch.Tensor, tables_out: torch.Tensor,
                   ref_out: torch.Tensor, stream=None) -> None:
    """Drop every row of `tables`."""
    _tables_and_counts("dcp_pages_free", pool, tables, ref, tables_out, ref_out)
    _check(lib.dcp_pages_free(pool.ref, _ptr(tables), tables.shape[0], tables.shape[1], _ptr(ref), _ptr(tables_out),
                              _ptr(ref_out), _stream(stream)), "dcp_pages_free")


def dcp_pages_compact(pool: PagePool, tables: torch.Tensor, ref: torch.Tensor, tables_out: torch.Tensor,
                      ref_out: torch.Tensor, n_live, ws: torch.Tensor, stream=None) -> None:
    """Pack the live blocks to the front of the pool; tables and counts follow, n_live (int32 [1] or None)."""
    _tables_and_counts("dcp_pages_compact", pool, tables, ref, tables_out, ref_out)
    _ints("dcp_pages_compact", n_live)
    if not ws.is_cuda or (n_live is not None and n_live.numel() < 1):
        raise DcpError("dcp_pages_compact", DCP_EINVAL)
    _check(lib.dcp_pages_compact(pool.ref, _ptr(tables), tables.shape[0], tables.shape[1], _ptr(ref),
                                 _ptr(tables_out), _ptr(ref_out), _ptr(n_live), _ptr(ws), ws.numel(),
                                 _stream(stream)), "dcp_pages_compact")
