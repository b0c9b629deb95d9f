"""suffix_match_drafter_amd -- MI355X (gfx950) suffix-match drafter.

Thin ctypes binding over ``libsfx.so`` (C-ABI in ``include/sfx.h``).  This module only
marshals arguments: every step of the drafter runs in the library's HIP kernels.  PyTorch is
used for device memory and streams.  There is no CPU fallback: if the library is missing the
calls raise.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsfx.so")

MODE_LONGEST_FILL = 0
MODE_SCORED = 1

OK, EINVAL, ENOMEM, ECAPACITY, EHIP, ESTATE, EIO = 0, -1, -2, -3, -4, -5, -6
_NAMES = {EINVAL: "EINVAL", ENOMEM: "ENOMEM", ECAPACITY: "ECAPACITY", EHIP: "EHIP",
          ESTATE: "ESTATE", EIO: "EIO"}

# every entry point declared in include/sfx.h
EXPORTS = ("sfx_create", "sfx_destroy", "sfx_last_error", "sfx_propose", "sfx_propose_masked",
           "sfx_propose_counts",
           "sfx_update_state", "sfx_harvest_finished", "sfx_ingest_inflight", "sfx_ingest",
           "sfx_rebuild", "sfx_rebuild_async", "sfx_poll", "sfx_wait_rebuild",
           "sfx_accept_estimate", "sfx_accept_feedback", "sfx_accept_reset", "sfx_accept_counts",
           "sfx_corpus_snapshot", "sfx_save", "sfx_load", "sfx_debug_errors",
           "sfx_debug_fail_next_rebuild", "sfx_debug_index", "sfx_rebuild_stats",
           "sfx_suffix_array_workspace_bytes", "sfx_build_suffix_array",
           "sfx_build_suffix_array_noalloc", "sfx_graphs_create", "sfx_graphs_propose",
           "sfx_graphs_stats", "sfx_graphs_destroy", "sfx_kv_write", "sfx_kv_read",
           "sfx_kv_attention_workspace_bytes", "sfx_kv_attention",
           "sfx_verify_workspace_bytes", "sfx_verify")


FLAG_STREAM_CONTEXT = 1  # read contexts from device memory instead of staging them in LDS
FLAG_CHECK_INPUTS = 2    # check device-resident inputs into the sticky error word
FLAG_TREE_DEPTH_CAP = 4  # match length plus draft length at most max_tree_depth

# flags of a batch-bucketed graph set (include/sfx.h)
GRAPHS_EAGER = 1             # capture nothing: every call runs eagerly
GRAPHS_UPDATE_STATE = 2      # the chain ends with the state update
GRAPHS_DELTA_INDEX = 4       # every chain groups the delta by tail pair first
GRAPHS_DEBUG_BREAK_ODD = 8   # test hook: captures of odd-indexed buckets fail

# bits of the sticky error word (include/sfx.h)
ERR_LENGTH, ERR_NEGATIVE_TOKEN, ERR_SAMPLED_AFTER_PAD, ERR_ROW_INDEX = 1, 2, 4, 8
ERR_SYNC_TIMEOUT = 16    # a propose workgroup's bounded internal wait ran out

# element types of the verification step's arrays (include/sfx.h)
_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class SfxError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{_NAMES.get(code, code)}: {msg}")
        self.code = code


class _Config(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_int32),
        ("max_tree_depth", ctypes.c_int32),
        ("num_backoff", ctypes.c_int32),
        ("max_occurrences", ctypes.c_int32),
        ("mode", ctypes.c_int32),
        ("min_self_match", ctypes.c_int32),
        ("min_corpus_match", ctypes.c_int32),
        ("max_batch", ctypes.c_int32),
        ("max_seq", ctypes.c_int32),
        ("max_sampled", ctypes.c_int32),
        ("spec_factor_ppm", ctypes.c_int64),
        ("spec_offset_ppm", ctypes.c_int64),
        ("min_token_prob_ppm", ctypes.c_int64),
        ("corpus_capacity", ctypes.c_int64),
        ("flags", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class _KvCache(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]


@dataclasses.dataclass
class Config:
    k: int
    max_tree_depth: int = 24
    num_backoff: int = 1
    max_occurrences: int = 128
    mode: int = MODE_LONGEST_FILL
    min_self_match: int = 1
    min_corpus_match: int = 2
    max_batch: int = 256
    max_seq: int = 16384
    max_sampled: int = 1
    spec_factor_ppm: int = 1_000_000
    spec_offset_ppm: int = 0
    min_token_prob_ppm: int = 100_000
    corpus_capacity: int = 0
    flags: int = 0
    reserved: int = 0

    def _c(self) -> _Config:
        return _Config(*[getattr(self, f[0]) for f in _Config._fields_])


_V = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SIZE_P = ctypes.POINTER(ctypes.c_size_t)
_lib = None


def load(path: str = LIB_PATH):
    """Load libsfx.so (torch is imported first so both share one HIP runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m suffix_match_drafter_amd.build` (hipcc, gfx950)")
    L = ctypes.CDLL(path)
    sig = {
        "sfx_create": (ctypes.c_int, [ctypes.POINTER(_Config), ctypes.POINTER(_V)]),
        "sfx_destroy": (None, [_V]),
        "sfx_last_error": (ctypes.c_char_p, []),
        "sfx_propose": (ctypes.c_int, [_V, _I32, _I32, _I32, _V, _V, _V, _V, _V, _V]),
        "sfx_propose_masked": (ctypes.c_int, [_V, _I32, _I32, _V, _V, _V, _V, _V, _V]),
        "sfx_propose_counts": (ctypes.c_int, [_V, _I32, _I32, _I32, _I32, _V, _V, _V, _V, _V,
                                              _V, _V]),
        "sfx_update_state": (ctypes.c_int, [_I32, _I32, _I32, _V, _V, _V, _V, _V]),
        "sfx_harvest_finished": (ctypes.c_int, [_V, _I32, _V, _V, _V, _I32, _I32, _V]),
        "sfx_ingest": (ctypes.c_int, [_V, _I32, _V, _V, _V]),
        "sfx_ingest_inflight": (ctypes.c_int, [_V, _I32, _V, _V, _V, _V, _I32, _I32, _I32, _V]),
        "sfx_rebuild": (ctypes.c_int, [_V, _V]),
        "sfx_rebuild_async": (ctypes.c_int, [_V, _V]),
        "sfx_poll": (ctypes.c_int, [_V, ctypes.POINTER(_I32), _V]),
        "sfx_wait_rebuild": (ctypes.c_int, [_V, _V]),
        "sfx_corpus_snapshot": (ctypes.c_int, [_V, _V, _I64, ctypes.POINTER(_I64), _V]),
        "sfx_accept_estimate": (ctypes.c_int, [_V, _I32, _V, _V]),
        "sfx_accept_feedback": (ctypes.c_int, [_V, _I32, _V, _V]),
        "sfx_accept_reset": (ctypes.c_int, [_V, _V]),
        "sfx_accept_counts": (ctypes.c_int, [_V, _V, _V]),
        "sfx_save": (ctypes.c_int, [_V, ctypes.c_char_p, _V]),
        "sfx_load": (ctypes.c_int, [_V, ctypes.c_char_p, _V]),
        "sfx_debug_errors": (ctypes.c_int, [_V, ctypes.POINTER(ctypes.c_uint32), _V]),
        "sfx_debug_fail_next_rebuild": (ctypes.c_int, [_V]),
        "sfx_debug_index": (ctypes.c_int, [_V, _V, _V, _I64, ctypes.POINTER(_I64), _V]),
        "sfx_rebuild_stats": (ctypes.c_int, [_V, ctypes.POINTER(_I32), ctypes.POINTER(_I64)]),
        "sfx_suffix_array_workspace_bytes": (ctypes.c_size_t, [_I64]),
        "sfx_build_suffix_array": (ctypes.c_int, [_V, _I64, _V, _V, ctypes.c_size_t, _V]),
        "sfx_build_suffix_array_noalloc": (ctypes.c_int, [_V, _I64, _V, _V]),
        "sfx_graphs_create": (ctypes.c_int, [_V, _I32, ctypes.POINTER(_I32), _I32, _I32, _V, _V,
                                             _V, _V, _V, _V, _I32, _V, ctypes.POINTER(_V)]),
        "sfx_graphs_propose": (ctypes.c_int, [_V, _I32, _V]),
        "sfx_graphs_stats": (ctypes.c_int, [_V, ctypes.POINTER(_I32),
                                            ctypes.POINTER(ctypes.c_uint64),
                                            ctypes.POINTER(ctypes.c_uint64),
                                            ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
        "sfx_graphs_destroy": (None, [_V]),
        "sfx_kv_write": (ctypes.c_int, [_V, _I32, _I32, _I32, _V, _V, _V, _V, _V, _V, _V, _I32,
                                        _V]),
        "sfx_kv_read": (ctypes.c_int, [_V, _I32, _I32, _I32, _V, _V, _V, _V, _V, _V, _V, _I32,
                                       _V]),
        "sfx_kv_attention_workspace_bytes": (ctypes.c_int, [_V, _I32, _I32, _I32, _I32, _I32,
                                                            _I32, _SIZE_P]),
        "sfx_kv_attention": (ctypes.c_int, [_V, _I32, _I32, _I32, _I32, _V, _V, _V, _V, _V, _V,
                                            _I32, ctypes.c_float, _I32, _I32, _V,
                                            ctypes.c_size_t, _V]),
        "sfx_verify_workspace_bytes": (ctypes.c_int, [_I32, _I32, _I32, _I32, _SIZE_P]),
        "sfx_verify": (ctypes.c_int, [_I32, _I32, _I32, _V, _I64, _I64, _I32, _V, _V, _V, _V,
                                      _V, _V, _V, _V, ctypes.c_size_t, _V]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(rc):
    if rc != OK:
        raise SfxError(rc, load().sfx_last_error().decode())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return _V(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _i32(t: torch.Tensor, name: str, ndim: int) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda:
        raise TypeError(f"{name} must be an int32 CUDA/HIP tensor")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor")
    return t


def _ptr(t):
    return _V(t.data_ptr()) if t is not None and t.numel() else _V(0)


class Drafter:
    """One drafter context: configuration, corpus ring and double-buffered corpus index."""

    def __init__(self, cfg: Config):
        L = load()
        self.cfg = cfg
        h = _V()
        _check(L.sfx_create(ctypes.byref(cfg._c()), ctypes.byref(h)))
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            load().sfx_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def propose(self, num_tokens, token_ids, sampled, draft=None, num_valid=None, stream=None):
        tok = _i32(token_ids, "token_ids", 2)
        B, S = tok.shape
        samp = _i32(sampled, "sampled", 2)
        nt = _i32(num_tokens, "num_tokens_no_spec", 1)
        if samp.shape[0] != B or nt.shape[0] != B:
            raise ValueError("batch sizes differ")
        if draft is None:
            draft = torch.empty((B, self.cfg.k), dtype=torch.int32, device=tok.device)
        if num_valid is None:
            num_valid = torch.empty((B,), dtype=torch.int32, device=tok.device)
        _i32(draft, "draft", 2)
        _i32(num_valid, "num_valid", 1)
        if draft.shape != (B, self.cfg.k) or num_valid.shape != (B,):
            raise ValueError("draft must be [B,k] and num_valid [B]")
        _check(load().sfx_propose(self._h, B, S, samp.shape[1], _ptr(nt), _ptr(tok), _ptr(samp),
                                  _ptr(draft), _ptr(num_valid), _stream(stream)))
        return draft, num_valid

    def propose_masked(self, num_tokens, token_ids, mask, draft=None, num_valid=None,
                       stream=None):
        """The masked form: contexts are the rows themselves; rows with mask 0 get no draft."""
        tok = _i32(token_ids, "token_ids", 2)
        B, S = tok.shape
        nt = _i32(num_tokens, "num_tokens_no_spec", 1)
        m = _i32(mask, "mask", 1)
        if nt.shape[0] != B or m.shape[0] != B:
            raise ValueError("num_tokens_no_spec, mask and token_ids disagree on B")
        if draft is None:
            draft = torch.empty((B, self.cfg.k), dtype=torch.int32, device=tok.device)
        if num_valid is None:
            num_valid = torch.empty((B,), dtype=torch.int32, device=tok.device)
        _check(load().sfx_propose_masked(self._h, B, S, _ptr(nt), _ptr(tok), _ptr(m),
                                         _ptr(draft), _ptr(num_valid), _stream(stream)))
        return draft, num_valid

    def propose_counts(self, k, num_tokens, token_ids, sampled, counts, draft=None,
                       num_valid=None, stream=None):
        """The counted form: counts[b] valid entries of sampled[b]; drafts of width k."""
        tok = _i32(token_ids, "token_ids", 2)
        B, S = tok.shape
        samp = _i32(sampled, "sampled", 2)
        nt = _i32(num_tokens, "num_tokens_no_spec", 1)
        cnt = _i32(counts, "counts", 1)
        if samp.shape[0] != B or nt.shape[0] != B or cnt.shape[0] != B:
            raise ValueError("num_tokens_no_spec, token_ids, sampled and counts disagree on B")
        if draft is None:
            draft = torch.empty((B, k), dtype=torch.int32, device=tok.device)
        if num_valid is None:
            num_valid = torch.empty((B,), dtype=torch.int32, device=tok.device)
        _check(load().sfx_propose_counts(self._h, int(k), B, S, samp.shape[1], _ptr(nt),
                                         _ptr(tok), _ptr(samp), _ptr(cnt), _ptr(draft),
                                         _ptr(num_valid), _stream(stream)))
        return draft, num_valid

    def graphs(self, buckets, num_tokens, token_ids, sampled, draft, num_valid,
               num_tokens_out=None, flags=0, stream=None) -> "GraphSet":
        """Pre-capture the step for each batch bucket over these persistent buffers."""
        return GraphSet(self, buckets, num_tokens, token_ids, sampled, draft, num_valid,
                        num_tokens_out, flags, stream)

    def propose_with_update(self, num_tokens, token_ids, sampled, stream=None):
        draft, nv = self.propose(num_tokens, token_ids, sampled, stream=stream)
        new_n = update_state(token_ids, num_tokens, sampled, stream=stream)
        return draft, nv, new_n

    def harvest_finished(self, row_indices, lengths, token_ids, stream=None):
        rows = _i32(row_indices, "row_indices", 1)
        lens = _i32(lengths, "lengths", 1)
        tok = _i32(token_ids, "token_ids", 2)
        if rows.shape != lens.shape:
            raise ValueError("row_indices and lengths differ in size")
        _check(load().sfx_harvest_finished(self._h, rows.shape[0], _ptr(rows), _ptr(lens),
                                           _ptr(tok), tok.shape[0], tok.shape[1],
                                           _stream(stream)))

    def ingest_inflight(self, row_indices, lengths, token_ids, final=None, min_chunk=1,
                        stream=None):
        """Append each listed row's tokens past its ingest cursor as one document once at least
        min_chunk have accumulated; rows with final != 0 flush what is left and restart."""
        rows = _i32(row_indices, "row_indices", 1)
        lens = _i32(lengths, "lengths", 1)
        tok = _i32(token_ids, "token_ids", 2)
        if rows.shape != lens.shape:
            raise ValueError("row_indices and lengths differ in size")
        fin = None
        if final is not None:
            fin = _i32(final, "final", 1)
            if fin.shape != rows.shape:
                raise ValueError("final and row_indices differ in size")
        _check(load().sfx_ingest_inflight(self._h, rows.shape[0], _ptr(rows), _ptr(lens),
                                          _ptr(fin), _ptr(tok), tok.shape[0], tok.shape[1],
                                          int(min_chunk), _stream(stream)))

    def ingest(self, doc_offsets, tokens, stream=None):
        offs = doc_offsets
        if offs.dtype != torch.int64 or not offs.is_cuda or offs.dim() != 1:
            raise TypeError("doc_offsets must be a 1-D int64 CUDA/HIP tensor")
        tok = _i32(tokens, "tokens", 1)
        _check(load().sfx_ingest(self._h, offs.shape[0] - 1, _ptr(offs), _ptr(tok),
                                 _stream(stream)))

    def ingest_docs(self, docs, stream=None):
        """Convenience: ingest a list of 1-D int sequences (host) as packed documents."""
        import numpy as np

        lens = [len(d) for d in docs]
        offs = np.zeros(len(docs) + 1, np.int64)
        offs[1:] = np.cumsum(lens)
        flat = np.concatenate([np.asarray(d, np.int32) for d in docs]) if docs else \
            np.zeros(0, np.int32)
        dev = torch.device("cuda")
        self.ingest(torch.from_numpy(offs).to(dev), torch.from_numpy(flat).to(dev), stream)

    def rebuild(self, stream=None):
        _check(load().sfx_rebuild(self._h, _stream(stream)))

    def rebuild_async(self, stream=None):
        _check(load().sfx_rebuild_async(self._h, _stream(stream)))

    def poll(self, stream=None) -> bool:
        sw = _I32(0)
        _check(load().sfx_poll(self._h, ctypes.byref(sw), _stream(stream)))
        return bool(sw.value)

    def wait_rebuild(self, stream=None):
        _check(load().sfx_wait_rebuild(self._h, _stream(stream)))

    def accept_estimate(self, B, est_ppm=None, stream=None):
        """[B, k] int32 per-slot acceptance estimates (ppm) of the last propose's drafts."""
        if est_ppm is None:
            est_ppm = torch.empty((B, self.cfg.k), dtype=torch.int32, device="cuda")
        _check(load().sfx_accept_estimate(self._h, B, _ptr(est_ppm), _stream(stream)))
        return est_ppm

    def accept_feedback(self, num_accepted, stream=None):
        """Count the verifier's accepted tokens [B] against the last propose's drafts."""
        na = _i32(num_accepted, "num_accepted", 1)
        _check(load().sfx_accept_feedback(self._h, na.shape[0], _ptr(na), _stream(stream)))

    def accept_reset(self, stream=None):
        _check(load().sfx_accept_reset(self._h, _stream(stream)))

    def accept_counts(self, stream=None) -> torch.Tensor:
        """The counts table as int64 [2, 65, 32, 2] (proposed, accepted)."""
        out = torch.empty((2, 65, 32, 2), dtype=torch.int64, device="cuda")
        _check(load().sfx_accept_counts(self._h, _ptr(out), _stream(stream)))
        return out

    def save(self, path, stream=None):
        """Write the corpus (live documents, counters, live index) to the host file `path`."""
        _check(load().sfx_save(self._h, os.fsencode(path), _stream(stream)))

    def load(self, path, stream=None):
        """Replace the corpus with the one saved in `path` (same corpus_capacity)."""
        _check(load().sfx_load(self._h, os.fsencode(path), _stream(stream)))

    def debug_fail_next_rebuild(self):
        """Test hook: the next rebuild fails with EHIP before its swap (the live index stays)."""
        _check(load().sfx_debug_fail_next_rebuild(self._h))

    def debug_errors(self, stream=None) -> int:
        """Read and clear the sticky ERR_* bits raised since the last read (synchronises)."""
        v = ctypes.c_uint32(0)
        _check(load().sfx_debug_errors(self._h, ctypes.byref(v), _stream(stream)))
        return v.value

    def corpus_snapshot(self, stream=None) -> torch.Tensor:
        cap = max(int(self.cfg.corpus_capacity), 1)
        out = torch.empty(cap, dtype=torch.int32, device="cuda")
        n = _I64(0)
        _check(load().sfx_corpus_snapshot(self._h, _ptr(out), cap, ctypes.byref(n),
                                          _stream(stream)))
        return out[: n.value]

    def rebuild_stats(self):
        """sfx_rebuild_stats: (doubling rounds, snapshot tokens) of the last index build."""
        r, n = _I32(0), _I64(0)
        _check(load().sfx_rebuild_stats(self._h, ctypes.byref(r), ctypes.byref(n)))
        return r.value, n.value

    def debug_index(self, stream=None):
        """sfx_debug_index: (snapshot text, suffix array) of the live corpus index."""
        cap = max(int(self.cfg.corpus_capacity), 1)
        text = torch.empty(cap, dtype=torch.int32, device="cuda")
        sa = torch.empty(cap, dtype=torch.int32, device="cuda")
        n = _I64(0)
        _check(load().sfx_debug_index(self._h, _ptr(text), _ptr(sa), cap, ctypes.byref(n),
                                      _stream(stream)))
        return text[: n.value], sa[: n.value]


class GraphSet:
    """Graphs of the drafter step captured per batch-size bucket over persistent buffers
    (sfx_graphs_create); propose(B) replays the smallest bucket >= B with rows B.. emptied, or
    runs eagerly where no graph was captured."""

    def __init__(self, drafter, buckets, num_tokens, token_ids, sampled, draft, num_valid,
                 num_tokens_out=None, flags=0, stream=None):
        buckets = [int(x) for x in buckets]
        nt = _i32(num_tokens, "num_tokens", 1)
        tok = _i32(token_ids, "token_ids", 2)
        smp = _i32(sampled, "sampled", 2)
        dr = _i32(draft, "draft", 2)
        nv = _i32(num_valid, "num_valid", 1)
        nout = None if num_tokens_out is None else _i32(num_tokens_out, "num_tokens_out", 1)
        rows = max(buckets) if buckets else 0
        for name, t in (("num_tokens", nt), ("token_ids", tok), ("sampled", smp),
                        ("draft", dr), ("num_valid", nv), ("num_tokens_out", nout)):
            if t is not None and t.shape[0] < rows:
                raise ValueError(f"{name} has {t.shape[0]} rows, the largest bucket {rows}")
        if dr.shape[1] != drafter.cfg.k:
            raise ValueError(f"draft must have k={drafter.cfg.k} columns")
        # the buffers stay referenced while the graphs exist
        self._keep = (drafter, nt, tok, smp, dr, nv, nout)
        arr = (_I32 * max(len(buckets), 1))(*buckets)
        h = _V()
        _check(load().sfx_graphs_create(drafter._h, len(buckets), arr, tok.shape[1],
                                        smp.shape[1], _ptr(nt), _ptr(tok), _ptr(smp), _ptr(dr),
                                        _ptr(nv), _ptr(nout), int(flags), _stream(stream),
                                        ctypes.byref(h)))
        self._h = h

    def propose(self, B, stream=None):
        _check(load().sfx_graphs_propose(self._h, int(B), _stream(stream)))

    def stats(self):
        nb, em, pm = _I32(), ctypes.c_uint64(), ctypes.c_uint64()
        rep, eag = _I64(), _I64()
        _check(load().sfx_graphs_stats(self._h, ctypes.byref(nb), ctypes.byref(em),
                                       ctypes.byref(pm), ctypes.byref(rep), ctypes.byref(eag)))
        return {"buckets": nb.value, "exact_mask": em.value, "padded_mask": pm.value,
                "replays": rep.value, "eager_calls": eag.value}

    def close(self):
        if getattr(self, "_h", None):
            load().sfx_graphs_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def update_state(token_ids, num_tokens, sampled, num_tokens_out=None, stream=None):
    tok = _i32(token_ids, "token_ids", 2)
    samp = _i32(sampled, "sampled", 2)
    nt = _i32(num_tokens, "num_tokens_no_spec", 1)
    B, S = tok.shape
    if num_tokens_out is None:
        num_tokens_out = torch.empty((B,), dtype=torch.int32, device=tok.device)
    _check(load().sfx_update_state(B, S, samp.shape[1], _ptr(tok), _ptr(nt), _ptr(samp),
                                   _ptr(num_tokens_out), _stream(stream)))
    return num_tokens_out


NOALLOC_MAX_TOKENS = 1 << 20  # largest text of build_suffix_array_noalloc


def build_suffix_array_noalloc(text: torch.Tensor, sa: torch.Tensor, stream=None) -> None:
    """sfx_build_suffix_array_noalloc: the suffix array of text into the caller's sa (same
    length), with no allocation; sa is ready once `stream` reaches the call."""
    t = _i32(text, "text", 1)
    out = _i32(sa, "sa", 1)
    if out.shape[0] != t.shape[0]:
        raise ValueError("sa must have text's length")
    _check(load().sfx_build_suffix_array_noalloc(_ptr(t), t.shape[0], _ptr(out), _stream(stream)))


def build_suffix_array(text: torch.Tensor, stream=None) -> torch.Tensor:
    t = _i32(text, "text", 1)
    n = t.shape[0]
    sa = torch.empty(n, dtype=torch.int32, device=t.device)
    L = load()
    wsb = L.sfx_suffix_array_workspace_bytes(n)
    ws = torch.empty(wsb, dtype=torch.uint8, device=t.device)
    _check(L.sfx_build_suffix_array(_ptr(t), n, _ptr(sa), _ptr(ws), wsb, _stream(stream)))
    return sa


# ------------------------------------------------------------------ the verification step
# These calls are short (a few microseconds on the device), so their checks are written to be
# cheap: device indexes instead of device objects, addresses as plain integers.
def _on(index):
    """The kernels run on the current device: the tensors have to be there."""
    if index < 0:
        raise TypeError("tensors must be on a CUDA/HIP device")
    cur = torch.cuda.current_device()
    if index != cur:
        raise ValueError(f"tensors are on cuda:{index}, the current device is cuda:{cur}")


def _raw_stream(stream, index):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to `stream` (the current one if None), so that its memory is
    not handed to other work while a kernel there still uses it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(
            stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _array(t, name, shape, dtype, index):
    """A contiguous tensor of this shape, type and device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
        raise TypeError(f"{name} must be a {dtype} tensor on cuda:{index}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {tuple(shape)}, got "
                         f"{tuple(t.shape)}")
    return t.data_ptr()


def _too_large(*sizes):
    """Sizes go to the library as int32, where larger ones would arrive as others."""
    raise ValueError(f"sizes {sizes}: each must be in [0, 2^31)")


def _heads(t, name, heads, dim, index):
    """A [B, T, heads, dim] tensor of any batch, token and head strides."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _TYPES or t.get_device() != index:
        raise TypeError(f"{name} must be a bfloat16, float16 or float32 tensor on cuda:{index}")
    shape = t.shape
    if len(shape) != 4 or shape[2] != heads or shape[3] != dim:
        raise ValueError(f"{name} must be [B, T, {heads}, {dim}], got {tuple(shape)}")
    if t.stride(3) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if t.requires_grad and torch.is_grad_enabled():
        raise RuntimeError(f"{name} requires grad, which ends here: these calls have no backward "
                           "(detach it, or call under torch.no_grad())")
    return shape


def _strides(t):
    return None if t.is_contiguous() else (_I64 * 3)(t.stride(0), t.stride(1), t.stride(2))


class KVCache:
    """A paged 8-bit KV cache: e4m3 codes with a power-of-two scale for each block of 32 tokens
    and head, in the layout that the attention reads (sfx_kv_cache in include/sfx.h).

    The buffers are allocated here, or given as ``buffers = (k, v, k_scale, v_scale)``: uint8 (or
    float8_e4m3fn) codes and float32 scales of the shapes of :meth:`shapes`; they stay the
    cache's.  Page tables, starts and lengths are contiguous int32 tensors in device memory; which
    pages a request owns is the caller's business.  There is no backward."""

    def __init__(self, num_pages, page_size, kv_heads, head_dim, device="cuda", buffers=None):
        if head_dim not in (64, 128, 256):
            raise ValueError("head_dim must be 64, 128 or 256")
        if page_size % 32 or not 32 <= page_size <= 2048:
            raise ValueError("page_size must be a multiple of 32 in [32, 2048]")
        if num_pages < 0 or kv_heads < 1:
            raise ValueError("num_pages must not be negative, kv_heads at least 1")
        if (num_pages | kv_heads) >> 31:
            _too_large(num_pages, kv_heads)
        codes = self.shapes(num_pages, page_size, kv_heads, head_dim)
        if buffers is None:
            dev = torch.device(device)
            self.k, self.v = (torch.zeros(s, dtype=torch.uint8, device=dev) for s in codes[:2])
            self.k_scale, self.v_scale = (torch.zeros(s, dtype=torch.float32, device=dev)
                                          for s in codes[2:])
        else:
            for t, s, name in zip(buffers, codes, ("k", "v", "k_scale", "v_scale")):
                kinds = (torch.float32,) if name.endswith("scale") else \
                    (torch.uint8, torch.float8_e4m3fn)
                if t.dtype not in kinds or not t.is_cuda or t.device != buffers[0].device:
                    raise TypeError(f"{name} must be a {kinds[0]} CUDA/HIP tensor")
                if t.shape != s or not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous of shape {tuple(s)}")
            self.k, self.v, self.k_scale, self.v_scale = buffers
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.kv_heads, self.head_dim = int(kv_heads), int(head_dim)
        self.device = self.k.device
        self._index = self.k.get_device()
        self._c = _KvCache(self.num_pages, self.page_size, self.kv_heads, self.head_dim,
                           self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(),
                           self.v_scale.data_ptr())
        self._p = ctypes.addressof(self._c)
        self._bytes = {}  # workspace sizes of the attention's shapes

    def __setattr__(self, name, value):
        # the library has the buffers' addresses and the sizes from the constructor
        if name in self.__dict__:
            raise AttributeError(f"{name} stays as it was made; write into the tensor, or make "
                                 "another KVCache")
        super().__setattr__(name, value)

    @staticmethod
    def shapes(num_pages, page_size, kv_heads, head_dim):
        """Shapes of k, v, k_scale and v_scale."""
        s = torch.Size((num_pages, kv_heads, page_size // 32))
        return (torch.Size((num_pages, kv_heads, head_dim // 64, page_size, 64)),
                torch.Size((num_pages, kv_heads, page_size // 32, head_dim // 32, 16, 4, 2, 2,
                            4)), s, s)

    def _table(self, page_table, B):
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be [B, pages]")
        pages = page_table.shape[1]
        return _array(page_table, "page_table", (B, pages), torch.int32, self._index), pages

    def write(self, k, v, page_table, start, count=None, stream=None):
        """sfx_kv_write: quantise k, v [B, T, kv_heads, head_dim] into positions start[b] .."""
        i = self._index
        _on(i)
        shape = _heads(k, "k", self.kv_heads, self.head_dim, i)
        if _heads(v, "v", self.kv_heads, self.head_dim, i) != shape or v.dtype is not k.dtype:
            raise ValueError("k and v differ in shape or type")
        B, T = shape[0], shape[1]
        tab, pages = self._table(page_table, B)
        if (B | T | pages) >> 31:
            _too_large(B, T, pages)
        st = _array(start, "start", (B,), torch.int32, i)
        ct = None if count is None else _array(count, "count", (B,), torch.int32, i)
        _check(load().sfx_kv_write(self._p, B, T, pages, tab, st, ct, k.data_ptr(),
                                   _strides(k), v.data_ptr(), _strides(v), _TYPES[k.dtype],
                                   _raw_stream(stream, i)))

    def read(self, page_table, start, count, T, dtype=torch.bfloat16, k=None, v=None,
             stream=None):
        """sfx_kv_read: positions start[b] .. start[b] + T - 1 as k, v [B, T, kv_heads,
        head_dim]; zero past count[b]."""
        i = self._index
        _on(i)
        if dtype not in _TYPES:
            raise TypeError("dtype must be bfloat16, float16 or float32")
        B, T = page_table.shape[0], int(T)
        tab, pages = self._table(page_table, B)
        if (B | T | pages) >> 31:
            _too_large(B, T, pages)
        st = _array(start, "start", (B,), torch.int32, i)
        ct = None if count is None else _array(count, "count", (B,), torch.int32, i)
        shape = (B, T, self.kv_heads, self.head_dim)
        if k is None:
            k = _empty(shape, dtype, self.device, stream)
        elif _heads(k, "k", self.kv_heads, self.head_dim, i) != shape or k.dtype is not dtype:
            raise ValueError(f"k must be {shape} of {dtype}")
        if v is None:
            v = torch.empty_like(k) if stream is None and k.is_contiguous() else \
                _empty(shape, dtype, self.device, stream)
        elif _heads(v, "v", self.kv_heads, self.head_dim, i) != shape or v.dtype is not dtype:
            raise ValueError(f"v must be {shape} of {dtype}")
        _check(load().sfx_kv_read(self._p, B, T, pages, tab, st, ct, k.data_ptr(),
                                  _strides(k), v.data_ptr(), _strides(v), _TYPES[dtype],
                                  _raw_stream(stream, i)))
        return k, v

    def attend(self, q, page_table, seq_lens, q_lens=None, scale=None, window=0, sinks=0,
               out=None, stream=None):
        """sfx_kv_attention: rows t < q_lens[b] of q [B, T, heads, head_dim] (bf16 or fp16), the
        newest tokens of seq_lens[b] cached ones, attend causally over the cache; window and
        sinks restrict what they see (0: everything).  scale defaults to head_dim ** -0.5."""
        i = self._index
        _on(i)
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise ValueError("q must be [B, T, heads, head_dim]")
        B, T, H, _ = shape = _heads(q, "q", q.shape[2], self.head_dim, i)
        if q.dtype is torch.float32:
            raise TypeError("q must be bfloat16 or float16")
        tab, pages = self._table(page_table, B)
        sl = _array(seq_lens, "seq_lens", (B,), torch.int32, i)
        ql = None if q_lens is None else _array(q_lens, "q_lens", (B,), torch.int32, i)
        L = load()
        window, sinks = int(window), int(sinks)
        if window >> 31 or sinks >> 31:
            raise ValueError("window and sinks must be in [0, 2^31)")
        key = (B, T, H, pages, window, sinks)
        n = self._bytes.get(key)
        if n is None:
            if (B | T | H | pages) >> 31:
                _too_large(B, T, H, pages)
            size = ctypes.c_size_t(0)
            _check(L.sfx_kv_attention_workspace_bytes(self._p, *key, ctypes.byref(size)))
            if len(self._bytes) >= 1024:
                self._bytes.clear()
            n = self._bytes[key] = size.value
        if out is None:
            out = torch.empty_like(q) if stream is None and q.is_contiguous() else \
                _empty(shape, q.dtype, self.device, stream)
        to = _array(out, "out", shape, q.dtype, i)
        ws = _empty((n,), torch.uint8, self.device, stream) if n else None
        _check(L.sfx_kv_attention(self._p, B, T, H, pages, tab, sl, ql, q.data_ptr(),
                                  _strides(q), to, _TYPES[q.dtype],
                                  self.head_dim ** -0.5 if scale is None else float(scale),
                                  window, sinks, ws.data_ptr() if n else None, n,
                                  _raw_stream(stream, i)))
        return out


_verify_bytes = {}  # workspace sizes of verify's shapes


def verify(logits, draft, num_valid, u_accept, u_sample, temperature=None, sampled=None,
           num_accepted=None, stream=None):
    """sfx_verify: accept or reject drafts [B, k] against the target's logits [B, k + 1, V] with
    the given uniform numbers u_accept [B, k] and u_sample [B].  Returns sampled [B, k + 1]
    (accepted tokens, one drawn token, then -1) and num_accepted [B]: the next inputs of
    propose / update_state and accept_feedback."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _TYPES or not logits.is_cuda:
        raise TypeError("logits must be a bfloat16, float16 or float32 CUDA/HIP tensor")
    if logits.dim() != 3 or logits.shape[1] < 1 or (logits.shape[2] > 1 and
                                                    logits.stride(2) != 1):
        raise ValueError("logits must be [B, k + 1, V] with V contiguous")
    i = logits.get_device()
    _on(i)
    B, k1, V = logits.shape
    dr = _array(draft, "draft", (B, k1 - 1), torch.int32, i)
    nv = None if num_valid is None else _array(num_valid, "num_valid", (B,), torch.int32, i)
    ua = _array(u_accept, "u_accept", (B, k1 - 1), torch.float32, i)
    us = _array(u_sample, "u_sample", (B,), torch.float32, i)
    tp = None if temperature is None else _array(temperature, "temperature", (B,),
                                                 torch.float32, i)
    if sampled is None:
        sampled = draft.new_empty(B, k1) if stream is None else \
            _empty((B, k1), torch.int32, logits.device, stream)
    if num_accepted is None:
        num_accepted = draft.new_empty(B) if stream is None else \
            _empty((B,), torch.int32, logits.device, stream)
    so = _array(sampled, "sampled", (B, k1), torch.int32, i)
    no = _array(num_accepted, "num_accepted", (B,), torch.int32, i)
    L = load()
    key = (B, k1 - 1, V, _TYPES[logits.dtype])
    n = _verify_bytes.get(key)
    if n is None:
        if (B | k1 | V) >> 31:
            _too_large(B, k1, V)
        size = ctypes.c_size_t(0)
        _check(L.sfx_verify_workspace_bytes(*key, ctypes.byref(size)))
        if len(_verify_bytes) >= 1024:
            _verify_bytes.clear()
        n = _verify_bytes[key] = size.value
    ws = _empty((n,), torch.uint8, logits.device, stream) if n else None
    _check(L.sfx_verify(B, k1 - 1, V, logits.data_ptr(), logits.stride(0), logits.stride(1),
                        key[3], tp, dr, nv, ua, us, so, no, ws.data_ptr() if n else None, n,
                        _raw_stream(stream, i)))
    return sampled, num_accepted
