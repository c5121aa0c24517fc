"""Thin ctypes binding of libqsa (include/qsa.h).

Argument marshalling only: every step of the QSA decode path runs in the CUDA
kernels of libqsa.so.  PyTorch supplies device memory and the current stream.
The functions keep the C names; they take torch tensors, check dtype / device /
shape / contiguity, pass raw pointers, and raise :class:`QSAError` on a
non-zero status.  There is no fallback: if libqsa.so is missing, importing this
module raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqsa.so")

HEAD_DIM = 256
IDX_HEADS = 8
IDX_DIM = 128
RATIO = 4
PAGE_TOKENS = 64
BLOCKS_PER_PAGE = 16
MAX_TOPK = 2048
MAX_GROUP = 16

QSA_OK, QSA_ERR_INVALID_ARG, QSA_ERR_UNSUPPORTED, QSA_ERR_CUDA = 0, -1, -2, -3
DEV_BITS = {1: "BAD_PAGE", 2: "BAD_SEQ", 4: "BAD_POS", 8: "BAD_SEL", 16: "BAD_COUNT", 32: "BAD_ORDER",
            64: "TIMEOUT", 128: "SCORES_LD"}


class QSAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


class qsa_cache_t(ctypes.Structure):
    _fields_ = [("kv_pages", ctypes.c_void_p), ("kc_pages", ctypes.c_void_p),
                ("kc_partial", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("max_seqs", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("kv_dtype", ctypes.c_int32)]


ROPE_MAX_PAIRS, ROPE_MAX_AXES, ROPE_MAX_TENSORS = 128, 3, 4


class qsa_rope_plan_t(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32), ("adjacent", ctypes.c_int32),
                ("axis", ctypes.c_uint8 * ROPE_MAX_PAIRS), ("freq", ctypes.c_double * ROPE_MAX_PAIRS)]


class qsa_rope_tensor_t(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("in_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


KV_BF16 = 0
KV_FP8_E4M3 = 1
_KV_TORCH = {KV_BF16: torch.bfloat16, KV_FP8_E4M3: torch.float8_e4m3fn}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libqsa.so not built at {LIB_PATH}; run `python sparse_attention_decode_03_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    PC = ctypes.POINTER(qsa_cache_t)
    sig = {
        "qsa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "qsa_abi_version": (ctypes.c_int, []),
        "qsa_append_kv": (ctypes.c_int, [PC, P, P, P, P, P, I32, P, P]),
        "qsa_index_scores": (ctypes.c_int, [PC, P, P, P, P, I32, P, I64, P, P]),
        "qsa_topk_blocks": (ctypes.c_int, [P, I64, P, I32, I32, P, P, P, P]),
        "qsa_index_topk": (ctypes.c_int, [PC, P, P, P, P, I32, I32, P, I64, P, P, P, P]),
        "qsa_index_topk_smem_bytes": (ctypes.c_int, [PC, I64]),
        "qsa_index_topk_resident_queries": (ctypes.c_int, [PC, I64]),
        "qsa_decode_plan": (ctypes.c_int, [I32, I32, I32, I32, ctypes.POINTER(I32), ctypes.POINTER(I32)]),
        "qsa_sparse_decode": (ctypes.c_int, [PC, P, I32, I32, P, P, P, P, I32, F, I32, I32, P, P, P, P]),
        "qsa_sparse_attention": (ctypes.c_int, [PC, P, I32, I32, P, P, P, P, I32, F, I32, I32, P, P, P, P, P, P, P]),
        "qsa_combine": (ctypes.c_int, [P, P, I32, I32, I32, P, P, P]),
        "qsa_combine_strided": (ctypes.c_int, [P, P, I32, I32, I32, I64, I64, I64, I64, P, I32, P, P]),
        "qsa_dcp_localize_tokens": (ctypes.c_int, [P, P, I32, I32, I32, I32, P, P, P]),
        "qsa_dcp_localize_selection": (ctypes.c_int, [P, P, P, I32, I32, I32, I32, I32, P, P, P, P, P]),
        "qsa_sparse_attention_noalloc": (ctypes.c_int, [PC, P, I32, I32, P, P, P, P, I32, F, I32, P, P, P, P]),
        "qsa_rope": (ctypes.c_int, [ctypes.POINTER(qsa_rope_plan_t), ctypes.POINTER(qsa_rope_tensor_t), I32, P, I64,
                                    I32, P]),
        "qsa_dense_decode_workspace_bytes": (I64, [PC, I32, I32, I32]),
        "qsa_dense_decode": (ctypes.c_int, [PC, P, I32, I32, P, P, F, P, P, P, P, I64, F, P, I64, P, P]),
        "qsa_evict_workspace_bytes": (I64, [PC, I32, I32]),
        "qsa_evict": (ctypes.c_int, [PC, P, P, P, I32, P, P, I64, I32, I32, I32, P, P, P, P, I64, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


LIB = _load()
ABI_VERSION = LIB.qsa_abi_version()


def status_string(status: int) -> str:
    return LIB.qsa_status_string(int(status)).decode()


def _check(fn: str, rc: int) -> None:
    if rc != QSA_OK:
        raise QSAError(fn, rc)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _req(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None:
        if t.dim() != len(shape) or any(s is not None and a != s for a, s in zip(t.shape, shape)):
            raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    return t


# ----------------------------------------------------------------------------
# cache group


class PagedCache:
    """Device buffers of one cache group: main K/V pages and the compressed-indexer
    side cache, paged by the same page ids, plus the per-sequence open-block sum.

    kv_pages holds, per page and KV head, 16 micro-blocks of 4 tokens, each one
    contiguous run (one selected micro-block of one KV head is one copy):
    BF16 (kv_dtype KV_BF16): [page][Hkv][16][4 dim atoms][8 rows][64], rows 0-3
    the K rows and 4-7 the V rows, the 16-byte chunk c of row r at chunk
    position c ^ r (the tensor cores' 128-byte swizzled operand layout);
    FP8 e4m3 (KV_FP8_E4M3): [page][Hkv][16][2 (K, V)][4 rows][256].
    with_kv=False leaves out the main K/V (a selector-only group),
    with_kc=False the side cache (a K/V-only group, e.g. a DCP rank's shard)."""

    def __init__(self, num_pages: int, max_seqs: int, max_pages_per_seq: int, num_kv_heads: int,
                 block_table: torch.Tensor | None = None, device="cuda", kv_dtype: int = KV_BF16,
                 with_kv: bool = True, with_kc: bool = True):
        dev = torch.device(device)
        if kv_dtype not in _KV_TORCH:
            raise ValueError(f"kv_dtype must be KV_BF16 or KV_FP8_E4M3, got {kv_dtype}")
        self.num_pages, self.max_seqs, self.max_pages_per_seq, self.num_kv_heads = (
            int(num_pages), int(max_seqs), int(max_pages_per_seq), int(num_kv_heads))
        self.kv_dtype = int(kv_dtype)
        if not (with_kv or with_kc):
            raise ValueError("a cache group needs the main K/V, the side cache, or both")
        shape = ((num_pages, num_kv_heads, BLOCKS_PER_PAGE, 4, 2 * RATIO, HEAD_DIM // 4) if self.kv_dtype == KV_BF16
                 else (num_pages, num_kv_heads, BLOCKS_PER_PAGE, 2, RATIO, HEAD_DIM))
        self.kv_pages = torch.empty(shape, dtype=_KV_TORCH[self.kv_dtype], device=dev) if with_kv else None
        self.kc_pages = torch.empty((num_pages, BLOCKS_PER_PAGE, IDX_DIM), dtype=torch.bfloat16,
                                    device=dev) if with_kc else None
        self.kc_partial = torch.zeros((max_seqs, IDX_DIM), dtype=torch.float32, device=dev) if with_kc else None
        self.device = dev
        if block_table is None:
            block_table = torch.full((max_seqs, max_pages_per_seq), -1, dtype=torch.int32)
        self.block_table = block_table.to(device=dev, dtype=torch.int32).contiguous()
        assert tuple(self.block_table.shape) == (max_seqs, max_pages_per_seq)
        self._struct = None

    def struct(self) -> qsa_cache_t:
        if self._struct is None:
            dp = lambda t: None if t is None else t.data_ptr()
            self._struct = qsa_cache_t(dp(self.kv_pages), dp(self.kc_pages), dp(self.kc_partial),
                                       self.block_table.data_ptr(), self.num_pages, self.max_seqs,
                                       self.max_pages_per_seq, self.num_kv_heads, self.kv_dtype)
        return self._struct

    def _rows(self, kv: int) -> torch.Tensor:
        if self.kv_dtype != KV_BF16:
            return self.kv_pages[:, :, :, kv].reshape(self.num_pages, self.num_kv_heads, PAGE_TOKENS, HEAD_DIM)
        # [page][Hkv][blk][atom][row][chunk position][8]: row r's chunk c sits at position c ^ r
        x = self.kv_pages.view(self.num_pages, self.num_kv_heads, BLOCKS_PER_PAGE, 4, 2 * RATIO, 8, 8)
        r = torch.arange(2 * RATIO, device=x.device)
        pos = (torch.arange(8, device=x.device)[None, :] ^ r[:, None])      # [row][chunk] -> position
        x = torch.gather(x, 5, pos[None, None, None, None, :, :, None].expand(x.shape))
        x = x[:, :, :, :, kv * RATIO:(kv + 1) * RATIO]                       # [page][Hkv][blk][atom][4][8][8]
        return x.permute(0, 1, 2, 4, 3, 5, 6).reshape(self.num_pages, self.num_kv_heads, PAGE_TOKENS, HEAD_DIM)

    def k_view(self) -> torch.Tensor:
        """K as [page][Hkv][64][256] (a copy in logical order, for inspection)."""
        return self._rows(0)

    def v_view(self) -> torch.Tensor:
        """V as [page][Hkv][64][256] (a copy in logical order, for inspection)."""
        return self._rows(1)

    @property
    def capacity_tokens(self) -> int:
        return self.max_pages_per_seq * PAGE_TOKENS


# ----------------------------------------------------------------------------
# the five calls


def qsa_append_kv(cache: PagedCache, k_new, v_new, kidx_new, seq_id, pos, dev_status=None, stream=None):
    n = int(seq_id.shape[0]) if isinstance(seq_id, torch.Tensor) else -1
    hkv = cache.num_kv_heads
    _req(k_new, "k_new", torch.bfloat16, (n, hkv, HEAD_DIM))
    _req(v_new, "v_new", torch.bfloat16, (n, hkv, HEAD_DIM))
    _req(kidx_new, "kidx_new", torch.bfloat16, (n, IDX_DIM))
    _req(seq_id, "seq_id", torch.int32, (n,))
    _req(pos, "pos", torch.int32, (n,))
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, (1,))
    _check("qsa_append_kv", LIB.qsa_append_kv(ctypes.byref(cache.struct()), _ptr(k_new), _ptr(v_new), _ptr(kidx_new),
                                              _ptr(seq_id), _ptr(pos), n, _ptr(dev_status), _stream(stream)))


def qsa_index_scores(cache: PagedCache, q_idx, w, q_seq, q_pos, scores, dev_status=None, stream=None):
    nq = int(q_seq.shape[0])
    _req(q_idx, "q_idx", torch.bfloat16, (nq, IDX_HEADS, IDX_DIM))
    _req(w, "w", torch.float32, (nq, IDX_HEADS))
    _req(q_seq, "q_seq", torch.int32, (nq,))
    _req(q_pos, "q_pos", torch.int32, (nq,))
    _req(scores, "scores", torch.float32, (nq, None))
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, (1,))
    _check("qsa_index_scores", LIB.qsa_index_scores(ctypes.byref(cache.struct()), _ptr(q_idx), _ptr(w), _ptr(q_seq),
                                                    _ptr(q_pos), nq, _ptr(scores), int(scores.shape[1]),
                                                    _ptr(dev_status), _stream(stream)))


def qsa_topk_blocks(scores, q_pos, k: int, sel, count, dev_status=None, stream=None):
    nq = int(q_pos.shape[0])
    _req(scores, "scores", torch.float32, (nq, None))
    _req(q_pos, "q_pos", torch.int32, (nq,))
    _req(sel, "sel", torch.int32, (nq, k))
    _req(count, "count", torch.int32, (nq,))
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, (1,))
    _check("qsa_topk_blocks", LIB.qsa_topk_blocks(_ptr(scores), int(scores.shape[1]), _ptr(q_pos), nq, int(k),
                                                  _ptr(sel), _ptr(count), _ptr(dev_status), _stream(stream)))


def qsa_index_topk(cache: PagedCache, q_idx, w, q_seq, q_pos, k: int, scores, sel, count, dev_status=None,
                   stream=None):
    """qsa_index_scores + qsa_topk_blocks in one kernel (a cluster of 8 CTAs per
    query keeps the score row on chip while it selects from it)."""
    nq = int(q_seq.shape[0])
    _req(q_idx, "q_idx", torch.bfloat16, (nq, IDX_HEADS, IDX_DIM))
    _req(w, "w", torch.float32, (nq, IDX_HEADS))
    _req(q_seq, "q_seq", torch.int32, (nq,))
    _req(q_pos, "q_pos", torch.int32, (nq,))
    _req(scores, "scores", torch.float32, (nq, None))
    _req(sel, "sel", torch.int32, (nq, k))
    _req(count, "count", torch.int32, (nq,))
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, (1,))
    _check("qsa_index_topk", LIB.qsa_index_topk(ctypes.byref(cache.struct()), _ptr(q_idx), _ptr(w), _ptr(q_seq),
                                                _ptr(q_pos), nq, int(k), _ptr(scores), int(scores.shape[1]),
                                                _ptr(sel), _ptr(count), _ptr(dev_status), _stream(stream)))


def index_topk_smem_bytes(cache: PagedCache, scores_ld: int) -> int:
    r = LIB.qsa_index_topk_smem_bytes(ctypes.byref(cache.struct()), int(scores_ld))
    _check("qsa_index_topk_smem_bytes", r if r < 0 else QSA_OK)
    return r


def index_topk_resident_queries(cache: PagedCache, scores_ld: int) -> int:
    r = LIB.qsa_index_topk_resident_queries(ctypes.byref(cache.struct()), int(scores_ld))
    _check("qsa_index_topk_resident_queries", r if r < 0 else QSA_OK)
    return r


FUSED_CLUSTER_CTAS = 8  # CTAs per query of qsa_index_topk (one cluster)


def fused_selection_pays(nq: int, max_seqs: int, sms: int, resident: int) -> bool:
    """Whether a step of nq queries should run the fused indexer + selection:
    its clusters fill the GPU (nq * FUSED_CLUSTER_CTAS >= the SM count) and all
    fit at once (nq <= resident: with a second wave the longest rows start late
    and the two-call form, which spreads a row over many CTAs, is faster), and
    the call is decode-shaped (fewer than 8 queries per sequence on average;
    prefill calls take the tensor-core query-tiled indexer)."""
    return nq * FUSED_CLUSTER_CTAS >= sms and nq <= resident and nq < 8 * max_seqs


def fused_default(cache: PagedCache, scores_ld: int, nq: int, sms: int) -> bool:
    """The Decoder's default selection form for a step of up to nq queries.  A
    device that cannot place the fused kernel's clusters (the occupancy query
    fails, or the clusters do not fit) keeps the two calls; an invalid cache or
    scores_ld is the caller's error and raises QSAError."""
    if cache.kc_pages is None:
        return False
    try:
        resident = index_topk_resident_queries(cache, scores_ld)
    except QSAError as e:
        if e.status not in (QSA_ERR_UNSUPPORTED, QSA_ERR_CUDA):
            raise
        resident = 0
    return fused_selection_pays(nq, cache.max_seqs, sms, resident)


def qsa_decode_plan(nq: int, hkv: int, k: int, target_ctas: int) -> tuple[int, int]:
    c, s = ctypes.c_int32(), ctypes.c_int32()
    _check("qsa_decode_plan", LIB.qsa_decode_plan(int(nq), int(hkv), int(k), int(target_ctas), ctypes.byref(c),
                                                  ctypes.byref(s)))
    return c.value, s.value


def qsa_sparse_decode(cache: PagedCache, q, q_seq, q_pos, sel, count, k: int, scale: float, chunk_units: int,
                      max_splits: int, part_o, part_lse, dev_status=None, stream=None):
    nq = int(q_seq.shape[0])
    hq = int(q.shape[1]) if q.dim() == 3 else -1
    _req(q, "q", torch.bfloat16, (nq, hq, HEAD_DIM))
    _req(q_seq, "q_seq", torch.int32, (nq,))
    _req(q_pos, "q_pos", torch.int32, (nq,))
    _req(sel, "sel", torch.int32, (nq, k))
    _req(count, "count", torch.int32, (nq,))
    _req(part_o, "part_o", torch.float32, (nq, max_splits, hq, HEAD_DIM))
    _req(part_lse, "part_lse", torch.float32, (nq, max_splits, hq))
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, (1,))
    _check("qsa_sparse_decode", LIB.qsa_sparse_decode(
        ctypes.byref(cache.struct()), _ptr(q), nq, hq, _ptr(q_seq), _ptr(q_pos), _ptr(sel), _ptr(count), int(k),
        float(scale), int(chunk_units), int(max_splits), _ptr(part_o), _ptr(part_lse), _ptr(dev_status),
        _stream(stream)))


def qsa_sparse_attention(cache: PagedCache, q, q_seq, q_pos, sel, count, k: int, scale: float, chunk_units: int,
                         max_splits: int, part_o, part_lse, pair_done, out, lse, dev_status=None, stream=None):
    """qsa_sparse_decode + qsa_combine in one kernel: the CTA that writes a
    (query, KV head) pair's last split merges it.  pair_done (int32 [nq][Hkv])
    must be zero on entry and is zero again afterwards."""
    nq = int(q_seq.shape[0])
    hq = int(q.shape[1]) if q.dim() == 3 else -1
    _req(q, "q", torch.bfloat16, (nq, hq, HEAD_DIM))
    _req(q_seq, "q_seq", torch.int32, (nq,))
    _req(q_pos, "q_pos", torch.int32, (nq,))
    _req(sel, "sel", torch.int32, (nq, k))
    _req(count, "count", torch.int32, (nq,))
    _req(part_o, "part_o", torch.float32, (nq, max_splits, hq, HEAD_DIM))
    _req(part_lse, "part_lse", torch.float32, (nq, max_splits, hq))
    _req(pair_done, "pair_done", torch.int32, (nq * cache.num_kv_heads,))
    _req(out, "out", torch.bfloat16, (nq, hq, HEAD_DIM))
    _req(lse, "lse", torch.float32, (nq, hq))
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, (1,))
    _check("qsa_sparse_attention", LIB.qsa_sparse_attention(
        ctypes.byref(cache.struct()), _ptr(q), nq, hq, _ptr(q_seq), _ptr(q_pos), _ptr(sel), _ptr(count), int(k),
        float(scale), int(chunk_units), int(max_splits), _ptr(part_o), _ptr(part_lse), _ptr(pair_done), _ptr(out),
        _ptr(lse), _ptr(dev_status), _stream(stream)))


def qsa_combine(part_o, part_lse, out, lse, stream=None):
    nq, S, hq = (int(x) for x in part_lse.shape)
    _req(part_o, "part_o", torch.float32, (nq, S, hq, HEAD_DIM))
    _req(part_lse, "part_lse", torch.float32, (nq, S, hq))
    _req(out, "out", torch.bfloat16, (nq, hq, HEAD_DIM))
    _req(lse, "lse", torch.float32, (nq, hq))
    _check("qsa_combine", LIB.qsa_combine(_ptr(part_o), _ptr(part_lse), nq, S, hq, _ptr(out), _ptr(lse),
                                          _stream(stream)))


OUT_BF16 = 0
OUT_F32 = 1


def qsa_combine_ranks(part_o, part_lse, out, lse, stream=None):
    """Merge results laid out split-major: part_o [S][nq][hq][256] fp32 and
    part_lse [S][nq][hq] (e.g. one fp32 result per DCP rank, gathered rank-major).
    out: bf16 or fp32 [nq][hq][256]; lse fp32 [nq][hq]."""
    S, nq, hq = (int(x) for x in part_lse.shape)
    _req(part_o, "part_o", torch.float32, (S, nq, hq, HEAD_DIM))
    _req(part_lse, "part_lse", torch.float32, (S, nq, hq))
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out must be bf16 or fp32")
    _req(out, "out", out.dtype, (nq, hq, HEAD_DIM))
    _req(lse, "lse", torch.float32, (nq, hq))
    od = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _check("qsa_combine_strided", LIB.qsa_combine_strided(
        _ptr(part_o), _ptr(part_lse), nq, S, hq, hq * HEAD_DIM, nq * hq * HEAD_DIM, hq, nq * hq, _ptr(out), od,
        _ptr(lse), _stream(stream)))


def qsa_combine_f32(part_o, part_lse, out, lse, stream=None):
    """qsa_combine with an fp32 result (part_o [nq][S][hq][256]); the result can
    be one split of a later merge."""
    nq, S, hq = (int(x) for x in part_lse.shape)
    _req(part_o, "part_o", torch.float32, (nq, S, hq, HEAD_DIM))
    _req(part_lse, "part_lse", torch.float32, (nq, S, hq))
    _req(out, "out", torch.float32, (nq, hq, HEAD_DIM))
    _req(lse, "lse", torch.float32, (nq, hq))
    _check("qsa_combine_strided", LIB.qsa_combine_strided(
        _ptr(part_o), _ptr(part_lse), nq, S, hq, S * hq * HEAD_DIM, hq * HEAD_DIM, S * hq, hq, _ptr(out), OUT_F32,
        _ptr(lse), _stream(stream)))


def qsa_dcp_localize_tokens(seq_id, pos, nranks: int, rank: int, interleave_pages: int, seq_id_local, pos_local,
                            stream=None):
    n = int(seq_id.shape[0])
    for t, nm in ((seq_id, "seq_id"), (pos, "pos"), (seq_id_local, "seq_id_local"), (pos_local, "pos_local")):
        _req(t, nm, torch.int32, (n,))
    _check("qsa_dcp_localize_tokens", LIB.qsa_dcp_localize_tokens(
        _ptr(seq_id), _ptr(pos), n, int(nranks), int(rank), int(interleave_pages), _ptr(seq_id_local),
        _ptr(pos_local), _stream(stream)))


def qsa_dcp_localize_selection(sel, count, q_pos, k: int, nranks: int, rank: int, interleave_pages: int, sel_local,
                               count_local, q_pos_local, dev_status=None, stream=None):
    nq = int(q_pos.shape[0])
    _req(sel, "sel", torch.int32, (nq, k))
    _req(sel_local, "sel_local", torch.int32, (nq, k))
    for t, nm in ((count, "count"), (q_pos, "q_pos"), (count_local, "count_local"), (q_pos_local, "q_pos_local")):
        _req(t, nm, torch.int32, (nq,))
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, (1,))
    _check("qsa_dcp_localize_selection", LIB.qsa_dcp_localize_selection(
        _ptr(sel), _ptr(count), _ptr(q_pos), nq, int(k), int(nranks), int(rank), int(interleave_pages),
        _ptr(sel_local), _ptr(count_local), _ptr(q_pos_local), _ptr(dev_status), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 16 << 20


def qsa_sparse_attention_noalloc(cache: PagedCache, q, q_seq, q_pos, sel, count, k: int, scale: float,
                                 chunk_units: int, out, lse, dev_status=None, stream=None):
    """qsa_sparse_decode + qsa_combine for callers that cannot allocate device
    memory: the split partials live in a fixed device array of
    NOALLOC_SCRATCH_BYTES inside libqsa.  Calls on one device share that array,
    so calls that can overlap on the GPU must be ordered (one stream).  The
    first call on each device looks up the array's address; make it before any
    stream capture."""
    nq = int(q_seq.shape[0])
    hq = int(q.shape[1]) if q.dim() == 3 else -1
    _req(q, "q", torch.bfloat16, (nq, hq, HEAD_DIM))
    _req(q_seq, "q_seq", torch.int32, (nq,))
    _req(q_pos, "q_pos", torch.int32, (nq,))
    _req(sel, "sel", torch.int32, (nq, k))
    _req(count, "count", torch.int32, (nq,))
    _req(out, "out", torch.bfloat16, (nq, hq, HEAD_DIM))
    _req(lse, "lse", torch.float32, (nq, hq))
    if dev_status is not None:
        _req(dev_status, "dev_status", torch.int32, (1,))
    _check("qsa_sparse_attention_noalloc", LIB.qsa_sparse_attention_noalloc(
        ctypes.byref(cache.struct()), _ptr(q), nq, hq, _ptr(q_seq), _ptr(q_pos), _ptr(sel), _ptr(count), int(k),
        float(scale), int(chunk_units), _ptr(out), _ptr(lse), _ptr(dev_status), _stream(stream)))


# ----------------------------------------------------------------------------
# pre-bound launches: validate once, then call the C entry point directly


class BoundCall:
    """A C entry point with its arguments marshalled once.  Calling it only
    enqueues the kernels (a few microseconds of host time), so a step of
    several launches keeps the GPU fed.  The tensors must stay alive and
    unchanged in shape while the call is used."""

    def __init__(self, name: str, args: tuple, keep: tuple):
        self.name = name
        self.fn = getattr(LIB, name)
        self.args = args
        self._keep = keep  # tensors / structs referenced by raw pointers

    def __call__(self):
        rc = self.fn(*self.args)
        if rc != QSA_OK:
            raise QSAError(self.name, rc)


def bind_append_kv(cache: PagedCache, k_new, v_new, kidx_new, seq_id, pos, dev_status=None, stream=None):
    n = int(seq_id.shape[0])
    hkv = cache.num_kv_heads
    _req(k_new, "k_new", torch.bfloat16, (n, hkv, HEAD_DIM))
    _req(v_new, "v_new", torch.bfloat16, (n, hkv, HEAD_DIM))
    _req(kidx_new, "kidx_new", torch.bfloat16, (n, IDX_DIM))
    _req(seq_id, "seq_id", torch.int32, (n,))
    _req(pos, "pos", torch.int32, (n,))
    st = cache.struct()
    return BoundCall("qsa_append_kv", (ctypes.byref(st), _ptr(k_new), _ptr(v_new), _ptr(kidx_new), _ptr(seq_id),
                                       _ptr(pos), n, _ptr(dev_status), _stream(stream)),
                     (cache, st, k_new, v_new, kidx_new, seq_id, pos, dev_status))


# ----------------------------------------------------------------------------
# a decode step: its calls on preallocated buffers


class Decoder:
    """Holds the per-step buffers (scores, selection, split partials, outputs) for
    up to `max_nq` queries and runs index_scores -> topk -> sparse_decode ->
    combine on the current stream, with no host synchronisation.

    ``fused=True`` runs the first two as the one fused call qsa_index_topk,
    ``fused=False`` as the two calls; the default chooses the fused call when
    fused_selection_pays(max_nq, ...).  ``merged=True`` runs the last two as
    the one call qsa_sparse_attention (the split kernel merges each pair's
    splits itself), the default ``merged=False`` as qsa_sparse_decode +
    qsa_combine (faster on B200: the merge's fences and L2 round trips in the
    split kernel cost more than the separate launch)."""

    def __init__(self, cache: PagedCache, hq: int, max_nq: int, k: int = 512, scale: float = 1.0 / 16.0,
                 target_ctas: int | None = None, chunk_units: int | None = None, scores_ld: int | None = None,
                 fused: bool | None = None, merged: bool = False):
        dev = cache.device
        self.cache, self.hq, self.k, self.scale, self.max_nq = cache, hq, k, scale, max_nq
        sms = torch.cuda.get_device_properties(dev).multi_processor_count
        if target_ctas is None:
            target_ctas = sms
        self.scores_ld = scores_ld or cache.max_pages_per_seq * BLOCKS_PER_PAGE
        if fused is None:
            fused = fused_default(cache, self.scores_ld, max_nq, sms)
        self.fused = bool(fused)
        if chunk_units is None:
            chunk_units, self.max_splits = qsa_decode_plan(max_nq, cache.num_kv_heads, k, target_ctas)
        else:
            self.max_splits = splits_bound(k, chunk_units)
        self.chunk_units = chunk_units
        self.scores = torch.empty((max_nq, self.scores_ld), dtype=torch.float32, device=dev)
        self.sel = torch.empty((max_nq, k), dtype=torch.int32, device=dev)
        self.count = torch.empty((max_nq,), dtype=torch.int32, device=dev)
        self.part_o = torch.empty((max_nq, self.max_splits, hq, HEAD_DIM), dtype=torch.float32, device=dev)
        self.part_lse = torch.empty((max_nq, self.max_splits, hq), dtype=torch.float32, device=dev)
        # out and lse share one allocation, so a full batch reads back in one copy
        out_bytes = max_nq * hq * HEAD_DIM * 2
        self._out_arena = torch.empty(_align(out_bytes) + max_nq * hq * 4, dtype=torch.uint8, device=dev)
        self.out = self._out_arena[:out_bytes].view(torch.bfloat16).view(max_nq, hq, HEAD_DIM)
        self.lse = self._out_arena[_align(out_bytes):].view(torch.float32).view(max_nq, hq)
        self.merged = bool(merged)
        self.pair_done = torch.zeros((max_nq * cache.num_kv_heads,), dtype=torch.int32, device=dev)
        self.dev_status = torch.zeros((1,), dtype=torch.int32, device=dev)

    def bind(self, q, q_idx, w, q_seq, q_pos, stream=None) -> list:
        """Validate the step inputs once and return the pre-bound launches for
        them: (index_scores, topk, sparse_decode, combine), or (index_topk,
        sparse_decode, combine) when fused."""
        nq = int(q_seq.shape[0])
        assert nq <= self.max_nq
        hq = self.hq
        _req(q_idx, "q_idx", torch.bfloat16, (nq, IDX_HEADS, IDX_DIM))
        _req(w, "w", torch.float32, (nq, IDX_HEADS))
        _req(q_seq, "q_seq", torch.int32, (nq,))
        _req(q_pos, "q_pos", torch.int32, (nq,))
        _req(q, "q", torch.bfloat16, (nq, hq, HEAD_DIM))
        sc, se, cn = self.scores[:nq], self.sel[:nq], self.count[:nq]
        po, pl = self.part_o[:nq], self.part_lse[:nq]
        out, lse = self.out[:nq], self.lse[:nq]
        st = self.cache.struct()
        ds, sp = _ptr(self.dev_status), _stream(stream)
        keep = (self.cache, st, q, q_idx, w, q_seq, q_pos, self.dev_status)
        if self.fused:
            select = [BoundCall("qsa_index_topk", (ctypes.byref(st), _ptr(q_idx), _ptr(w), _ptr(q_seq), _ptr(q_pos),
                                                   nq, self.k, _ptr(sc), int(sc.shape[1]), _ptr(se), _ptr(cn), ds,
                                                   sp), keep)]
        else:
            select = [
                BoundCall("qsa_index_scores", (ctypes.byref(st), _ptr(q_idx), _ptr(w), _ptr(q_seq), _ptr(q_pos), nq,
                                               _ptr(sc), int(sc.shape[1]), ds, sp), keep),
                BoundCall("qsa_topk_blocks", (_ptr(sc), int(sc.shape[1]), _ptr(q_pos), nq, self.k, _ptr(se),
                                              _ptr(cn), ds, sp), keep)]
        if self.merged:
            return select + [
                BoundCall("qsa_sparse_attention", (ctypes.byref(st), _ptr(q), nq, hq, _ptr(q_seq), _ptr(q_pos),
                                                   _ptr(se), _ptr(cn), self.k, float(self.scale), self.chunk_units,
                                                   self.max_splits, _ptr(po), _ptr(pl), _ptr(self.pair_done),
                                                   _ptr(out), _ptr(lse), ds, sp), keep + (self.pair_done,))]
        return select + [
            BoundCall("qsa_sparse_decode", (ctypes.byref(st), _ptr(q), nq, hq, _ptr(q_seq), _ptr(q_pos), _ptr(se),
                                            _ptr(cn), self.k, float(self.scale), self.chunk_units, self.max_splits,
                                            _ptr(po), _ptr(pl), ds, sp), keep),
            BoundCall("qsa_combine", (_ptr(po), _ptr(pl), nq, self.max_splits, hq, _ptr(out), _ptr(lse), sp), keep),
        ]

    def host_outputs(self):
        """Pinned host buffers laid out like the device outputs: (arena, out, lse)."""
        arena = torch.empty(self._out_arena.shape, dtype=torch.uint8).pin_memory()
        out = arena[:self.out.numel() * 2].view(torch.bfloat16).view(self.out.shape)
        lse = arena[self._out_arena.numel() - self.lse.numel() * 4:].view(torch.float32).view(self.lse.shape)
        return arena, out, lse

    def download(self, host, nq: int, stream=None) -> int:
        """Enqueue the device-to-host copy of out[:nq] and lse[:nq] into `host`
        (from host_outputs()): one copy for a full batch, two otherwise.
        Returns the bytes copied."""
        arena, out, lse = host
        s = stream or torch.cuda.current_stream()
        with torch.cuda.stream(s):
            if nq == self.max_nq:
                arena.copy_(self._out_arena, non_blocking=True)
                return arena.numel()
            out[:nq].copy_(self.out[:nq], non_blocking=True)
            lse[:nq].copy_(self.lse[:nq], non_blocking=True)
        return out[:nq].numel() * 2 + lse[:nq].numel() * 4

    def run(self, q, q_idx, w, q_seq, q_pos, stream=None):
        nq = int(q_seq.shape[0])
        assert nq <= self.max_nq
        sc, se, cn = self.scores[:nq], self.sel[:nq], self.count[:nq]
        po, pl = self.part_o[:nq], self.part_lse[:nq]
        if self.fused:
            qsa_index_topk(self.cache, q_idx, w, q_seq, q_pos, self.k, sc, se, cn, self.dev_status, stream)
        else:
            qsa_index_scores(self.cache, q_idx, w, q_seq, q_pos, sc, self.dev_status, stream)
            qsa_topk_blocks(sc, q_pos, self.k, se, cn, self.dev_status, stream)
        if self.merged:
            qsa_sparse_attention(self.cache, q, q_seq, q_pos, se, cn, self.k, self.scale, self.chunk_units,
                                 self.max_splits, po, pl, self.pair_done[:nq * self.cache.num_kv_heads],
                                 self.out[:nq], self.lse[:nq], self.dev_status, stream)
        else:
            qsa_sparse_decode(self.cache, q, q_seq, q_pos, se, cn, self.k, self.scale, self.chunk_units,
                              self.max_splits, po, pl, self.dev_status, stream)
            qsa_combine(po, pl, self.out[:nq], self.lse[:nq], stream)
        return self.out[:nq], self.lse[:nq]


def _align(n: int, a: int = 256) -> int:
    return (n + a - 1) // a * a


class StepIO:
    """The inputs of one step (the appended tokens and the queries) staged in one
    pinned host buffer and one device buffer, 256-byte aligned fields, so that
    sending a step's inputs is a single host-to-device copy.  `host[name]` and
    `dev[name]` are views of the same field; bind the step to the `dev` views,
    fill the `host` views, then upload()."""

    def __init__(self, n_new: int, nq: int, hq: int, hkv: int, device="cuda"):
        fields = [("k_new", torch.bfloat16, (n_new, hkv, HEAD_DIM)), ("v_new", torch.bfloat16, (n_new, hkv, HEAD_DIM)),
                  ("kidx_new", torch.bfloat16, (n_new, IDX_DIM)), ("seq_id", torch.int32, (n_new,)),
                  ("pos", torch.int32, (n_new,)), ("q", torch.bfloat16, (nq, hq, HEAD_DIM)),
                  ("q_idx", torch.bfloat16, (nq, IDX_HEADS, IDX_DIM)), ("w", torch.float32, (nq, IDX_HEADS)),
                  ("q_seq", torch.int32, (nq,)), ("q_pos", torch.int32, (nq,))]
        off, spans = 0, []
        for name, dt, shape in fields:
            nbytes = torch.Size(shape).numel() * torch.empty((), dtype=dt).element_size()
            spans.append((name, dt, shape, off, nbytes))
            off = _align(off + nbytes)
        self.nbytes = off
        self.host_buf = torch.empty(off, dtype=torch.uint8).pin_memory()
        self.dev_buf = torch.empty(off, dtype=torch.uint8, device=device)
        self.host, self.dev = {}, {}
        for name, dt, shape, o, nb in spans:
            self.host[name] = self.host_buf[o:o + nb].view(dt).view(shape)
            self.dev[name] = self.dev_buf[o:o + nb].view(dt).view(shape)

    def upload(self, stream=None):
        """Enqueue the single host-to-device copy of every field."""
        s = stream or torch.cuda.current_stream()
        with torch.cuda.stream(s):
            self.dev_buf.copy_(self.host_buf, non_blocking=True)


class StepGraph:
    """The pre-bound launches of one step captured once into a CUDA graph and
    replayed with a single launch, so a step costs no per-kernel host work.
    The library calls only enqueue kernels (no allocation, no host
    synchronisation), which is what lets them be captured.  The calls must have
    been bound to `stream` (a side stream, not the legacy default stream).

    With ``timing=True`` a timing event is captured before every call and
    after the last one; after a replay, :meth:`kernel_ms` gives each call's
    device time for that replay."""

    def __init__(self, calls, stream: torch.cuda.Stream, timing: bool = False):
        self.calls = list(calls)
        self.stream = stream
        self.events = ([torch.cuda.Event(enable_timing=True, external=True) for _ in range(len(self.calls) + 1)]
                       if timing else None)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            for k, c in enumerate(self.calls):
                if self.events:
                    self.events[k].record(stream)
                c()
            if self.events:
                self.events[-1].record(stream)

    def replay(self):
        """Enqueue one replay on the graph's stream (stream-ordered after the
        work already enqueued there)."""
        with torch.cuda.stream(self.stream):
            self.graph.replay()

    def kernel_ms(self) -> list:
        """Device time of each call in the last replay (synchronises on it)."""
        self.events[-1].synchronize()
        return [self.events[k].elapsed_time(self.events[k + 1]) for k in range(len(self.calls))]


class StepPipeline:
    """Serving-style double buffering of whole steps.  Two slots, each with its
    own staged inputs (a StepIO), Decoder, pinned host outputs and step graph;
    step i runs in slot i % 2.  The inputs of a step go up on one copy stream
    while the previous step computes, and its outputs come back on another
    while the next one computes.  Events order every reuse of a slot:
      upload(i)   after compute(i - 2) has read the slot's inputs,
      compute(i)  after upload(i) and after download(i - 2) has read the
                  slot's outputs,
      download(i) after compute(i).
    `calls[s]` are slot s's pre-bound launches (bound to `compute`, reading
    ios[s].dev and writing decs[s]'s buffers); `before(stream)`, if given,
    enqueues work on the compute stream ahead of every step's graph.  Nothing
    synchronises the host."""

    def __init__(self, ios, decs, calls, compute: torch.cuda.Stream, before=None, nq: int | None = None):
        assert len(ios) == len(decs) == len(calls) == 2
        self.ios, self.decs, self.compute, self.before = ios, decs, compute, before
        self.nq = decs[0].max_nq if nq is None else nq
        self.up_stream = torch.cuda.Stream(device=compute.device)
        self.down_stream = torch.cuda.Stream(device=compute.device)
        self.hosts = [d.host_outputs() for d in decs]
        self.graphs = [StepGraph(c, compute) for c in calls]
        self._up = [torch.cuda.Event() for _ in range(2)]
        self._done = [torch.cuda.Event() for _ in range(2)]
        self._down = [torch.cuda.Event() for _ in range(2)]
        self._used = [False, False]
        self.d2h_bytes = 0

    def step(self, i: int):
        """Enqueue step i (inputs already in ios[i % 2].host)."""
        s = i % 2
        if self._used[s]:
            self.up_stream.wait_event(self._done[s])
        self.ios[s].upload(self.up_stream)
        self._up[s].record(self.up_stream)
        self.compute.wait_event(self._up[s])
        if self._used[s]:
            self.compute.wait_event(self._down[s])
        if self.before is not None:
            self.before(self.compute)
        self.graphs[s].replay()
        self._done[s].record(self.compute)
        self.down_stream.wait_event(self._done[s])
        self.d2h_bytes = self.decs[s].download(self.hosts[s], self.nq, self.down_stream)
        self._down[s].record(self.down_stream)
        self._used[s] = True

    def uploaded(self, i: int) -> bool:
        """Whether step i's inputs have left ios[i % 2].host (the slot's host
        inputs may be refilled for step i + 2 only then)."""
        return self._up[i % 2].query()

    def wait_outputs(self, i: int):
        """Block the host until step i's outputs are in host memory; return them
        as (out, lse).  Step i + 2 reuses the slot's host outputs."""
        self._down[i % 2].synchronize()
        return self.outputs(i)

    def outputs(self, i: int):
        """Host (out, lse) of step i: valid once its download has completed."""
        _, out, lse = self.hosts[i % 2]
        return out, lse


# ----------------------------------------------------------------------------
# layers that attend to everything they hold: rotary positions, dense decode,
# eviction.  Every call has a bind_* form that checks its arguments once.


def _as_c(fn: str, t, x):
    """x as the C type t; an integer that t cannot hold is refused (ctypes would cut it to t's bits)."""
    v = t(x)
    if isinstance(x, int) and v.value != x:
        raise ValueError(f"{fn}: {x} is beyond the {8 * ctypes.sizeof(t)} bits of its argument")
    return v


class LaunchCall:
    """A bound C entry point (see :class:`BoundCall`) that takes its stream when
    it is called: the one it was bound to, or the caller's current stream.  It
    runs on its tensors' device whichever device is current.  The tensors must
    stay alive and unchanged in shape while the call is used."""

    def __init__(self, name: str, args: tuple, keep: tuple, device: torch.device, stream=None):
        self.name = name
        self.fn = LIB[name]  # a function object of its own: its arguments are converted here, once
        self.fn.restype = ctypes.c_int
        self.args = tuple(_as_c(name, t, x) if isinstance(x, (int, float, type(None))) else x
                          for x, t in zip(args, getattr(LIB, name).argtypes))
        self._keep = keep
        self.device = device.index if device.index is not None else torch.cuda.current_device()
        self.stream = stream

    def __call__(self):
        if torch._C._cuda_getDevice() != self.device:
            with torch.cuda.device(self.device):
                return self()
        s = (self.stream.cuda_stream if self.stream is not None else torch._C._cuda_getCurrentRawStream(self.device))
        rc = self.fn(*self.args, ctypes.c_void_p(s))
        if rc != QSA_OK:
            raise QSAError(self.name, rc)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _status(dev_status):
    return None if dev_status is None else _req(dev_status, "dev_status", torch.int32, (1,))


def _workspace_ptr(workspace, need: int, name: str = "workspace"):
    _req(workspace, name, torch.uint8, (None,))
    if workspace.numel() < need:
        raise ValueError(f"{name}: {workspace.numel()} bytes, needs {need}")
    return _ptr(workspace)


class RopePlan:
    """What qsa_rope rotates and how fast.  `sections` holds the number of pairs
    of each axis (time, height, width; one axis for plain text); rot_dim is
    twice their sum.  Pair i turns by base ** (-2 i / rot_dim) per position, or
    by freqs[i] where given.  `cycled` deals the pairs to the axes in turn
    (0, 1, 2, 0, 1, 2, ...) as long as axes 1 and 2 have pairs left, the rest to
    axis 0; otherwise the sections follow one another.  `adjacent` pairs dims
    (2i, 2i + 1) instead of (i, i + rot_dim / 2)."""

    def __init__(self, rot_dim: int, sections=None, base: float = 1.0e4, cycled: bool = False,
                 adjacent: bool = False, freqs=None):
        half = int(rot_dim) // 2
        if rot_dim < 16 or rot_dim % 16 or half > ROPE_MAX_PAIRS:
            raise ValueError(f"rot_dim must be a multiple of 16 in [16, {2 * ROPE_MAX_PAIRS}], got {rot_dim}")
        sections = (half,) if sections is None else tuple(int(x) for x in sections)
        if not 1 <= len(sections) <= ROPE_MAX_AXES or any(x < 0 for x in sections) or sum(sections) != half:
            raise ValueError(f"sections {sections} must be 1 to {ROPE_MAX_AXES} counts that add up to rot_dim / 2 = "
                             f"{half}")
        if cycled:
            k = len(sections)
            axis = [i % k if i % k and i < k * sections[i % k] else 0 for i in range(half)]
            if [axis.count(a) for a in range(k)] != list(sections):
                raise ValueError(f"sections {sections} cannot be dealt in turn over {half} pairs")
        else:
            axis = [a for a, x in enumerate(sections) for _ in range(x)]
        if freqs is None:
            freqs = [float(base) ** (-2.0 * i / rot_dim) for i in range(half)]
        freqs = [float(f) for f in freqs]
        if len(freqs) != half or not all(math.isfinite(f) for f in freqs):
            raise ValueError(f"freqs must be {half} finite numbers")
        self.rot_dim, self.num_axes, self.adjacent = int(rot_dim), len(sections), bool(adjacent)
        self.axis, self.freqs = axis, freqs
        self._struct = qsa_rope_plan_t(self.rot_dim, self.num_axes, int(self.adjacent),
                                       (ctypes.c_uint8 * ROPE_MAX_PAIRS)(*axis),
                                       (ctypes.c_double * ROPE_MAX_PAIRS)(*freqs))

    def struct(self) -> qsa_rope_plan_t:
        return self._struct


def _rope_rows(t, name: str, n: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3 or t.shape[0] != n:
        raise ValueError(f"{name}: expected shape ({n}, heads, head_dim), got {tuple(t.shape)}")
    if t.numel() and ((t.shape[2] > 1 and t.stride(2) != 1) or (t.shape[1] > 1 and t.stride(1) != t.shape[2])):
        raise ValueError(f"{name}: heads and dims must be dense (only the token stride is free)")
    return t


def bind_rope(plan: RopePlan, pos, inputs, outputs=None, stream=None) -> LaunchCall:
    """qsa_rope with its arguments checked once; see :func:`qsa_rope`."""
    _req(pos, "pos", torch.int32, (plan.num_axes, None))
    n = int(pos.shape[1])
    inputs = list(inputs)
    outputs = inputs if outputs is None else list(outputs)
    if not 1 <= len(inputs) <= ROPE_MAX_TENSORS or len(outputs) != len(inputs):
        raise ValueError(f"1 to {ROPE_MAX_TENSORS} inputs and as many outputs")
    arr = (qsa_rope_tensor_t * len(inputs))()
    for k, (x, y) in enumerate(zip(inputs, outputs)):
        _rope_rows(x, f"inputs[{k}]", n)
        _rope_rows(y, f"outputs[{k}]", n)
        if x.shape != y.shape:
            raise ValueError(f"outputs[{k}]: expected shape {tuple(x.shape)}, got {tuple(y.shape)}")
        _same_device(pos.device, **{f"inputs[{k}]": x, f"outputs[{k}]": y})
        arr[k] = qsa_rope_tensor_t(x.data_ptr(), y.data_ptr(), int(x.shape[1]), int(x.shape[2]), x.stride(0),
                                   y.stride(0))
    st = plan.struct()
    return LaunchCall("qsa_rope", (ctypes.byref(st), arr, len(inputs), _ptr(pos), n, n),
                      (plan, st, arr, pos, inputs, outputs), pos.device, stream)


def qsa_rope(plan: RopePlan, pos, inputs, outputs=None, stream=None):
    """Rotate bf16 tensors [n][heads][head_dim] (q, k, the indexer's, ...) by the
    positions pos int32 [axes][n]; in place unless `outputs` are given.  Only the
    token stride is free, so slices of a fused projection can be passed.  Returns
    the outputs."""
    outputs = list(inputs) if outputs is None else list(outputs)
    bind_rope(plan, pos, inputs, outputs, stream)()
    return outputs


def dense_decode_workspace_bytes(cache: PagedCache, nq: int, hq: int, with_mass: bool = False) -> int:
    fn = "qsa_dense_decode_workspace_bytes"
    r = LIB.qsa_dense_decode_workspace_bytes(ctypes.byref(cache.struct()), _as_c(fn, ctypes.c_int32, int(nq)),
                                             _as_c(fn, ctypes.c_int32, int(hq)), int(with_mass))
    _check(fn, r if r < 0 else QSA_OK)
    return r


def _mass_args(cache: PagedCache, mass_in, mass_out):
    ld = cache.max_pages_per_seq * BLOCKS_PER_PAGE
    for t, nm in ((mass_in, "mass_in"), (mass_out, "mass_out")):
        _req(t, nm, torch.float32, (cache.max_seqs, None))
        if t.shape[1] < ld:
            raise ValueError(f"{nm}: {t.shape[1]} blocks per sequence, needs {ld}")
    if mass_in.shape != mass_out.shape:
        raise ValueError("mass_in and mass_out must have the same shape")
    return int(mass_in.shape[1])


def bind_dense_decode(cache: PagedCache, q, q_seq, q_pos, scale: float, out, lse, workspace, mass_in=None,
                      mass_out=None, decay: float = 1.0, dev_status=None, stream=None) -> LaunchCall:
    """qsa_dense_decode with its arguments checked once; see :func:`qsa_dense_decode`."""
    nq = int(q_seq.shape[0])
    hq = int(q.shape[1]) if q.dim() == 3 else -1
    _req(q, "q", torch.bfloat16, (nq, hq, HEAD_DIM))
    _req(q_seq, "q_seq", torch.int32, (nq,))
    _req(q_pos, "q_pos", torch.int32, (nq,))
    _req(out, "out", torch.bfloat16, (nq, hq, HEAD_DIM))
    _req(lse, "lse", torch.float32, (nq, hq))
    ld = 0
    if mass_in is not None or mass_out is not None:
        ld = _mass_args(cache, mass_in, mass_out)
    _status(dev_status)
    ws = _workspace_ptr(workspace, dense_decode_workspace_bytes(cache, nq, hq, ld > 0))
    _same_device(q.device, q_seq=q_seq, q_pos=q_pos, out=out, lse=lse, workspace=workspace, mass_in=mass_in,
                 mass_out=mass_out, dev_status=dev_status, kv_pages=cache.kv_pages, block_table=cache.block_table)
    st = cache.struct()
    return LaunchCall("qsa_dense_decode",
                      (ctypes.byref(st), _ptr(q), nq, hq, _ptr(q_seq), _ptr(q_pos), float(scale), _ptr(out),
                       _ptr(lse), _ptr(mass_in), _ptr(mass_out), ld, float(decay), ws, int(workspace.numel()),
                       _ptr(dev_status)),
                      (cache, st, q, q_seq, q_pos, out, lse, mass_in, mass_out, workspace, dev_status), q.device,
                      stream)


def qsa_dense_decode(cache: PagedCache, q, q_seq, q_pos, scale: float, out, lse, workspace, mass_in=None,
                     mass_out=None, decay: float = 1.0, dev_status=None, stream=None):
    """Attention of one token per query over all the tokens its sequence holds
    (positions 0 .. q_pos); with mass_in / mass_out (fp32 [max_seqs][blocks]) also
    the attention weight of every micro-block, added into a running total.
    `workspace`: uint8, dense_decode_workspace_bytes(...) of them."""
    bind_dense_decode(cache, q, q_seq, q_pos, scale, out, lse, workspace, mass_in, mass_out, decay, dev_status,
                      stream)()


def evict_workspace_bytes(cache: PagedCache, n: int, budget: int) -> int:
    fn = "qsa_evict_workspace_bytes"
    r = LIB.qsa_evict_workspace_bytes(ctypes.byref(cache.struct()), _as_c(fn, ctypes.c_int32, int(n)),
                                      _as_c(fn, ctypes.c_int32, int(budget)))
    _check(fn, r if r < 0 else QSA_OK)
    return r


def bind_evict(cache: PagedCache, seq_ids, seq_len, mass_in, mass_out, budget: int, sink: int, recent: int, keep,
               keep_count, new_len, workspace, dst_table=None, dev_status=None, stream=None) -> LaunchCall:
    """qsa_evict with its arguments checked once; see :func:`qsa_evict`."""
    n = int(seq_ids.shape[0])
    for t, nm in ((seq_ids, "seq_ids"), (seq_len, "seq_len"), (keep_count, "keep_count"), (new_len, "new_len")):
        _req(t, nm, torch.int32, (n,))
    _req(keep, "keep", torch.int32, (n, int(budget)))
    ld = _mass_args(cache, mass_in, mass_out)
    if dst_table is not None:
        _req(dst_table, "dst_table", torch.int32, (cache.max_seqs, cache.max_pages_per_seq))
    _status(dev_status)
    ws = _workspace_ptr(workspace, evict_workspace_bytes(cache, n, budget))
    _same_device(seq_ids.device, seq_len=seq_len, mass_in=mass_in, mass_out=mass_out, keep=keep,
                 keep_count=keep_count, new_len=new_len, workspace=workspace, dst_table=dst_table,
                 dev_status=dev_status, block_table=cache.block_table, kv_pages=cache.kv_pages,
                 kc_pages=cache.kc_pages)
    st = cache.struct()
    return LaunchCall("qsa_evict",
                      (ctypes.byref(st), _ptr(dst_table), _ptr(seq_ids), _ptr(seq_len), n, _ptr(mass_in),
                       _ptr(mass_out), ld, int(budget), int(sink), int(recent), _ptr(keep), _ptr(keep_count),
                       _ptr(new_len), ws, int(workspace.numel()), _ptr(dev_status)),
                      (cache, st, seq_ids, seq_len, mass_in, mass_out, keep, keep_count, new_len, workspace,
                       dst_table, dev_status), seq_ids.device, stream)


def qsa_evict(cache: PagedCache, seq_ids, seq_len, mass_in, mass_out, budget: int, sink: int, recent: int, keep,
              keep_count, new_len, workspace, dst_table=None, dev_status=None, stream=None):
    """Cut sequences down to `budget` complete micro-blocks by accumulated
    attention weight: the first `sink`, the last `recent` and the heaviest
    between them, moved together in order (in place, or into the pages of
    dst_table).  Fills keep [n][budget], keep_count and new_len."""
    bind_evict(cache, seq_ids, seq_len, mass_in, mass_out, budget, sink, recent, keep, keep_count, new_len,
               workspace, dst_table, dev_status, stream)()


def _capturing(stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


class DenseDecoder:
    """Outputs and workspace of qsa_dense_decode for up to `max_nq` queries.  With
    ``track=True`` it also holds `mass`, the running attention weight of every
    micro-block (``decay`` of the old total is kept at each step), and
    :meth:`evict` cuts sequences to a budget by it.  A row of `mass` belongs to
    the sequence in its slot: zero it when the slot goes to another.

    Calls share `mass`, the outputs and the workspace: :meth:`run` and
    :meth:`evict` may take any stream, and each waits for the object's last call
    and, given a stream, for the caller's current one.  Launches from
    :meth:`bind`, and calls that are captured, are put on their stream as they
    are (one given a stream inside a capture branches off it); order those
    yourself."""

    def __init__(self, cache: PagedCache, hq: int, max_nq: int, scale: float = 1.0 / 16.0, track: bool = False,
                 decay: float = 1.0):
        dev = cache.device
        self.cache, self.hq, self.max_nq, self.scale, self.decay = cache, hq, max_nq, float(scale), float(decay)
        self.out = torch.empty((max_nq, hq, HEAD_DIM), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((max_nq, hq), dtype=torch.float32, device=dev)
        self.mass = (torch.zeros((cache.max_seqs, cache.max_pages_per_seq * BLOCKS_PER_PAGE), dtype=torch.float32,
                                 device=dev) if track else None)
        self.workspace = torch.empty(dense_decode_workspace_bytes(cache, max_nq, hq, track), dtype=torch.uint8,
                                     device=dev)
        self.dev_status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self._last = None  # the stream of the last run or evict

    def _enter(self, stream, *tensors):
        """Order a call behind the last one and the caller's current stream; `tensors`, allocated on that
        stream, stay theirs until a call on another one has used them."""
        raw = torch._C._cuda_getCurrentRawStream(self.workspace.device.index)
        leaves = stream is not None and stream.cuda_stream != raw
        if not leaves and self._last is not None and self._last.cuda_stream == raw:
            return  # the usual call, on the stream of the last one
        current = torch.cuda.current_stream(self.workspace.device)
        s = stream if leaves else current
        if _capturing(current):
            if leaves:
                s.wait_stream(current)  # a branch of the capture, which the caller joins
        elif not _capturing(s):
            for other in (current, self._last):
                if other is not None and other != s:
                    s.wait_stream(other)
            self._last = s
        if leaves:
            for t in tensors:
                if t is not None:
                    t.record_stream(s)

    def bind(self, q, q_seq, q_pos, stream=None) -> list:
        """The pre-bound launch of a step's attention, for a StepGraph."""
        nq = int(q_seq.shape[0])
        if nq > self.max_nq:
            raise ValueError(f"{nq} queries, at most {self.max_nq}")
        return [bind_dense_decode(self.cache, q, q_seq, q_pos, self.scale, self.out[:nq], self.lse[:nq],
                                  self.workspace, self.mass, self.mass, self.decay, self.dev_status, stream)]

    def run(self, q, q_seq, q_pos, stream=None):
        """out [nq][hq][256] and lse [nq][hq] of the queries (views of this object's buffers)."""
        call = self.bind(q, q_seq, q_pos, stream)[0]
        self._enter(stream, q, q_seq, q_pos)
        call()
        nq = int(q_seq.shape[0])
        return self.out[:nq], self.lse[:nq]

    def evict(self, seq_ids, seq_len, budget: int, sink: int = 0, recent: int = 0, dst_table=None, stream=None):
        """Cut the listed sequences (seq_len tokens each) to `budget` complete
        micro-blocks by `mass`.  Returns (new_len, keep, keep_count), device
        tensors; the caller appends at new_len and frees the pages behind it."""
        if self.mass is None:
            raise ValueError("evict needs track=True")
        n, dev = int(seq_ids.shape[0]), self.cache.device
        keep = torch.empty((n, int(budget)), dtype=torch.int32, device=dev)
        count = torch.empty((n,), dtype=torch.int32, device=dev)
        new_len = torch.empty((n,), dtype=torch.int32, device=dev)
        ws = torch.empty(evict_workspace_bytes(self.cache, n, budget), dtype=torch.uint8, device=dev)
        self._enter(stream, seq_ids, seq_len, dst_table, keep, count, new_len, ws)
        qsa_evict(self.cache, seq_ids, seq_len, self.mass, self.mass, budget, sink, recent, keep, count, new_len, ws,
                  dst_table, self.dev_status, stream)
        return new_len, keep, count


def splits_bound(k: int, chunk_units: int) -> int:
    """Most KV chunks one (query, KV head) pair's k+1 unit slots can touch."""
    return (k + 1 + chunk_units - 2) // chunk_units + 1


def dev_status_names(v: int) -> list[str]:
    return [n for b, n in DEV_BITS.items() if v & b]


def pages_for(tokens: int) -> int:
    return math.ceil(tokens / PAGE_TOKENS)
