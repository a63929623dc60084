"""Python front end of the C ABI: torch tensors in, raw pointers out.

PyTorch provides device memory and the current CUDA stream; every step of the
path runs in libpagedattn's kernels.  Argument checks here only guard the
pointer marshalling (device, dtype, contiguity, shape).
"""
import ctypes

import numpy as np
import torch

from . import _lib as L

# pool element type -> (torch type of k/v/q inputs, torch type of the stored elements)
_TORCH = {L.PA_F32: (torch.float32, torch.float32), L.PA_BF16: (torch.bfloat16, torch.bfloat16),
          L.PA_FP8E4M3: (torch.bfloat16, torch.uint8),
          L.PA_FP8E4M3_BLOCK: (torch.bfloat16, torch.uint8)}
_CODE = {torch.float32: L.PA_F32, torch.bfloat16: L.PA_BF16, "f32": L.PA_F32,
         "bf16": L.PA_BF16, "fp8": L.PA_FP8E4M3, "fp8e4m3": L.PA_FP8E4M3, "fp8b": L.PA_FP8E4M3_BLOCK}
# element types an attention output may have
_OUT = {torch.float32: L.PA_F32, torch.bfloat16: L.PA_BF16}


# torch's own query for a raw handle: 0.1 us, where the public one takes 2 us of a call's 4 to
# 12.  It is no public name, so a torch without it is asked the public way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    """The current stream of `device`, as a raw handle."""
    if _raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def _dev(t, dtype, name, device):
    """The address of a tensor, checked."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _span(x):
    """A count of positions for a C int: no context reaches beyond 2^30, and a negative
    one (refused there) stays negative."""
    return max(min(int(x), 1 << 30), -(1 << 31))


def _i32p(a):
    return a.ctypes.data_as(L.c_i32p)


class KVPool:
    """A pool of fixed-size physical KV blocks on one GPU (one layer).

    K is [num_blocks, kv_heads, block_size, head_dim]; V is stored transposed
    per tile, [num_blocks, kv_heads, head_dim, block_size].  dtype "fp8" keeps
    one e4m3 code per element (stored as uint8; a code stands for its value
    times the pool's K or V scale) and takes bf16 k, v and q.  dtype "fp8b" does
    the same with one power-of-two scale per (block, KV head), K and V apart,
    chosen by the appends from their data.
    """

    def __init__(self, num_blocks, block_size, kv_heads, head_dim, dtype="bf16", device=None):
        dev = torch.device("cuda") if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError("KVPool lives on a CUDA device")
        self.device = dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())
        self.dtype_code = _CODE[dtype]
        self.dtype, self.storage_dtype = _TORCH[self.dtype_code]
        self.fp8 = self.dtype_code == L.PA_FP8E4M3
        self.block_scaled = self.dtype_code == L.PA_FP8E4M3_BLOCK
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)
        self.kv_heads, self.head_dim = int(kv_heads), int(head_dim)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            L.check(L.pa_pool_create(self.num_blocks, self.block_size, self.kv_heads,
                                     self.head_dim, self.dtype_code, ctypes.byref(h)),
                    "pa_pool_create")
        self.handle = h

    def set_kv_scales(self, k_scale, v_scale):
        """Scales of an fp8 pool (set them before the first append)."""
        L.check(L.pa_pool_set_kv_scales(self.handle, float(k_scale), float(v_scale)),
                "pa_pool_set_kv_scales")

    def kv_scales(self):
        k, v = ctypes.c_float(), ctypes.c_float()
        L.check(L.pa_pool_kv_scales(self.handle, ctypes.byref(k), ctypes.byref(v)),
                "pa_pool_kv_scales")
        return k.value, v.value

    OPTIONS = {"partition_cap": L.PA_OPT_PARTITION_CAP, "shared_kernel": L.PA_OPT_SHARED_KERNEL,
               "prefill_kernel": L.PA_OPT_PREFILL_KERNEL}

    def set_option(self, name, value):
        """Kernel-choice option of this pool (pa_pool_set_option): partition_cap
        (tokens; 0 none, -1 automatic), shared_kernel / prefill_kernel (0
        tcgen05 where eligible, 1 mma.sync)."""
        L.check(L.pa_pool_set_option(self.handle, self.OPTIONS[name], int(value)),
                "pa_pool_set_option")

    def get_option(self, name):
        v = ctypes.c_int()
        L.check(L.pa_pool_get_option(self.handle, self.OPTIONS[name], ctypes.byref(v)),
                "pa_pool_get_option")
        return v.value

    def close(self):
        if getattr(self, "handle", None):
            L.pa_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- data movement ---------------------------------------------------
    def append_kv(self, k, v, slot_mapping):
        T = int(slot_mapping.shape[0])
        shape = (T, self.kv_heads, self.head_dim)
        if k.shape != shape or v.shape != shape:
            raise ValueError(f"k/v must be {shape}")
        L.check(L.pa_append_kv(self.handle, _dev(k, self.dtype, "k", self.device),
                               _dev(v, self.dtype, "v", self.device),
                               _dev(slot_mapping, torch.int64, "slot_mapping", self.device), T,
                               _stream(self.device)), "pa_append_kv")

    def append_rope(self, q, k, v, slot_mapping, positions, inv_freq, axis=None,
                    interleaved=False, q_out=None):
        """Rotate q and k by their tokens' positions, store k and v at
        slot_mapping and return the rotated queries (pa_append_rope).

        positions is int32 [T] or [num_axes, T]; axis (int32, one per pair) names
        the axis of each pair, all 0 when not given.  q, k and v may be slices of
        one projection's output: only a token's heads have to be contiguous.
        q None: keys and values only, returns None."""
        if slot_mapping.dim() != 1:
            raise ValueError("slot_mapping must be [T]")
        T, hkv, d = slot_mapping.shape[0], self.kv_heads, self.head_dim
        if k.shape != (T, hkv, d) or v.shape != (T, hkv, d):
            raise ValueError(f"k/v must be {(T, hkv, d)}")
        axes = 1
        if positions.dim() == 2:
            axes = positions.shape[0]
        if positions.dim() not in (1, 2) or positions.shape[-1] != T:
            raise ValueError("positions must be [T] or [num_axes, T]")
        if inv_freq.dim() != 1 or (axis is not None and axis.shape != inv_freq.shape):
            raise ValueError("inv_freq and axis must be [rotary_dim / 2]")
        qp, qs, hq, op = None, 0, 0, None
        if q is not None:
            hq = q.shape[1]
            if q.shape != (T, hq, d):
                raise ValueError("q must be [T, Hq, D]")
            qp, qs = self._rows(q, "q")
            if q_out is None:
                q_out = torch.empty((T, hq, d), dtype=self.dtype, device=self.device)
                op = q_out.data_ptr()
            elif q_out.shape != (T, hq, d):
                raise ValueError("q_out must be [T, Hq, D]")
            else:
                op = _dev(q_out, self.dtype, "q_out", self.device)
        kp, ks = self._rows(k, "k")
        vp, vs = self._rows(v, "v")
        L.check(L.pa_append_rope(
            self.handle, qp, qs, hq, kp, ks, vp, vs,
            _dev(slot_mapping, torch.int64, "slot_mapping", self.device), T,
            _dev(positions, torch.int32, "positions", self.device), axes,
            _dev(inv_freq, torch.float32, "inv_freq", self.device),
            _dev(axis, torch.int32, "axis", self.device) if axis is not None else None,
            2 * inv_freq.shape[0], 1 if interleaved else 0, op, _stream(self.device)),
            "pa_append_rope")
        return q_out if q is not None else None

    def _rows(self, t, name):
        """(address, elements between tokens) of [T, heads, D] whose heads are packed."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.device != self.device:
            raise ValueError(f"{name} must live on {self.device}, got {t.device}")
        if t.dtype != self.dtype:
            raise TypeError(f"{name} must be {self.dtype}, got {t.dtype}")
        T, h, d = t.shape
        if t.is_contiguous():
            return t.data_ptr(), h * d
        s0, s1, s2 = t.stride()
        if T and ((h > 1 and s1 != d) or s2 != 1 or (T > 1 and s0 < h * d)):
            raise ValueError(f"{name}: a token's heads must be contiguous")
        return t.data_ptr(), s0 if T > 1 else h * d

    def read_kv(self, slots):
        """(k, v), [n, Hkv, D] each, of the tokens stored at slots (int64 [n])."""
        if slots.dim() != 1:
            raise ValueError("slots must be [n]")
        n = slots.shape[0]
        k = torch.empty((n, self.kv_heads, self.head_dim), dtype=self.dtype, device=self.device)
        v = torch.empty_like(k)
        L.check(L.pa_read_kv(self.handle, _dev(slots, torch.int64, "slots", self.device), n,
                             k.data_ptr(), v.data_ptr(), _stream(self.device)), "pa_read_kv")
        return k, v

    def copy_blocks(self, pairs):
        P = int(pairs.shape[0]) if pairs.numel() else 0
        if P and tuple(pairs.shape) != (P, 2):
            raise ValueError("pairs must be [P, 2]")
        ptr = _dev(pairs, torch.int64, "pairs", self.device) if P else None
        L.check(L.pa_copy_blocks(self.handle, ptr, P, _stream(self.device)), "pa_copy_blocks")

    def decode(self, q, block_tables, context_lens, scale, out=None, out_dtype=torch.float32,
               window=None, sinks=0):
        """Decode attention; window (and sinks): only the last `window` positions and
        the first `sinks` are seen (pa_decode_window)."""
        S, hq, d = q.shape
        if d != self.head_dim:
            raise ValueError("q head_dim does not match the pool")
        if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
            raise ValueError("block_tables [S, max_blocks] / context_lens [S]")
        if out is None:
            out = torch.empty((S, hq, d), dtype=out_dtype, device=self.device)
        if out.shape != (S, hq, d):
            raise ValueError("out must be [S, Hq, D]")
        if window is not None:
            L.check(L.pa_decode_window(
                self.handle, _dev(q, self.dtype, "q", self.device), S, hq,
                _dev(block_tables, torch.int32, "block_tables", self.device),
                int(block_tables.shape[1]),
                _dev(context_lens, torch.int32, "context_lens", self.device), _span(window),
                _span(sinks), float(scale), _dev(out, out.dtype, "out", self.device),
                _OUT[out.dtype], _stream(self.device)), "pa_decode_window")
            return out
        if sinks:
            raise ValueError("sinks need a window")
        L.check(L.pa_decode(self.handle, _dev(q, self.dtype, "q", self.device), S, hq,
                            _dev(block_tables, torch.int32, "block_tables", self.device),
                            int(block_tables.shape[1]),
                            _dev(context_lens, torch.int32, "context_lens", self.device),
                            float(scale), _dev(out, out.dtype, "out", self.device),
                            _CODE[out.dtype], _stream(self.device)), "pa_decode")
        return out

    def append_decode(self, k, v, slot_mapping, q, block_tables, context_lens, scale, out=None,
                      out_dtype=torch.float32):
        """Write each sequence's new token (k[s], v[s] at slot_mapping[s]), then decode."""
        S, hq, d = q.shape
        shape = (S, self.kv_heads, self.head_dim)
        if k.shape != shape or v.shape != shape or slot_mapping.shape != (S,):
            raise ValueError(f"k/v must be {shape}, slot_mapping [S]")
        if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
            raise ValueError("block_tables [S, max_blocks] / context_lens [S]")
        if out is None:
            out = torch.empty((S, hq, d), dtype=out_dtype, device=self.device)
        L.check(L.pa_append_decode(self.handle, _dev(k, self.dtype, "k", self.device),
                                   _dev(v, self.dtype, "v", self.device),
                                   _dev(slot_mapping, torch.int64, "slot_mapping", self.device),
                                   _dev(q, self.dtype, "q", self.device), S, hq,
                                   _dev(block_tables, torch.int32, "block_tables", self.device),
                                   int(block_tables.shape[1]),
                                   _dev(context_lens, torch.int32, "context_lens", self.device),
                                   float(scale), _dev(out, out.dtype, "out", self.device),
                                   _CODE[out.dtype], _stream(self.device)), "pa_append_decode")
        return out

    def decode_shared(self, q, block_tables, context_lens, scale, groups, out=None,
                      out_dtype=torch.float32):
        """Decode with shared leading blocks read once per group.

        groups = (offsets, seqs, shared_blocks) host int32 arrays, as returned by
        BlockManager.prefix_groups.
        """
        offs, seqs, nsh = (np.ascontiguousarray(a, dtype=np.int32) for a in groups)
        S, hq, d = q.shape
        if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
            raise ValueError("block_tables [S, max_blocks] / context_lens [S]")
        if out is None:
            out = torch.empty((S, hq, d), dtype=out_dtype, device=self.device)
        ng = len(nsh)
        if len(offs) != ng + 1:
            raise ValueError("group offsets must have num_groups + 1 entries")
        L.check(L.pa_decode_shared(self.handle, _dev(q, self.dtype, "q", self.device), S, hq,
                                   _dev(block_tables, torch.int32, "block_tables", self.device),
                                   int(block_tables.shape[1]),
                                   _dev(context_lens, torch.int32, "context_lens", self.device),
                                   float(scale), _dev(out, out.dtype, "out", self.device),
                                   _CODE[out.dtype], _i32p(offs), _i32p(seqs) if len(seqs) else None,
                                   _i32p(nsh) if ng else None, ng, _stream(self.device)),
                "pa_decode_shared")
        return out

    def prefill(self, q, cu_seqlens_q, block_tables, context_lens, scale, max_q_len=None,
                out=None, out_dtype=torch.float32, window=None, sinks=0):
        """Chunked prefill: the packed chunk queries q [T, Hq, D] (sequence s owns
        rows cu_seqlens_q[s] .. cu_seqlens_q[s+1]-1) attend to the cached prefix
        and causally to their chunk.  The chunk's keys and values must already
        be appended.  max_q_len (longest chunk) is read from cu_seqlens_q when
        not given (one device-to-host copy).  window (and sinks): each query sees
        only the last `window` positions up to its own and the first `sinks`
        (pa_prefill_window)."""
        T, hq, d = q.shape
        S = int(cu_seqlens_q.shape[0]) - 1
        if d != self.head_dim or S < 0:
            raise ValueError("q head_dim / cu_seqlens_q [S+1]")
        if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
            raise ValueError("block_tables [S, max_blocks] / context_lens [S]")
        if max_q_len is None:
            max_q_len = int((cu_seqlens_q[1:] - cu_seqlens_q[:-1]).max().item()) if S else 0
        if out is None:
            out = torch.empty((T, hq, d), dtype=out_dtype, device=self.device)
        if out.shape != (T, hq, d):
            raise ValueError("out must be [T, Hq, D]")
        if window is not None:
            L.check(L.pa_prefill_window(
                self.handle, _dev(q, self.dtype, "q", self.device), T, hq,
                _dev(cu_seqlens_q, torch.int32, "cu_seqlens_q", self.device), S, int(max_q_len),
                _dev(block_tables, torch.int32, "block_tables", self.device),
                int(block_tables.shape[1]),
                _dev(context_lens, torch.int32, "context_lens", self.device), _span(window),
                _span(sinks), float(scale), _dev(out, out.dtype, "out", self.device),
                _OUT[out.dtype], _stream(self.device)), "pa_prefill_window")
            return out
        if sinks:
            raise ValueError("sinks need a window")
        L.check(L.pa_prefill(self.handle, _dev(q, self.dtype, "q", self.device), T, hq,
                             _dev(cu_seqlens_q, torch.int32, "cu_seqlens_q", self.device), S,
                             int(max_q_len),
                             _dev(block_tables, torch.int32, "block_tables", self.device),
                             int(block_tables.shape[1]),
                             _dev(context_lens, torch.int32, "context_lens", self.device),
                             float(scale), _dev(out, out.dtype, "out", self.device),
                             _CODE[out.dtype], _stream(self.device)), "pa_prefill")
        return out

    def reserve(self, max_seqs, max_q_heads, window=False):
        """Size the decode workspace (window: that of windowed decodes)."""
        if window:
            L.check(L.pa_decode_window_reserve(self.handle, int(max_seqs), int(max_q_heads)),
                    "pa_decode_window_reserve")
            return
        L.check(L.pa_decode_reserve(self.handle, int(max_seqs), int(max_q_heads)),
                "pa_decode_reserve")

    def get_error(self):
        """Synchronise the current stream; return the recorded error code (0 = none)."""
        return L.pa_get_error(self.handle, _stream(self.device))

    def check_error(self):
        code = self.get_error()
        if code:
            raise L.PagedAttnError(code, "device")

    # -- snapshots ---------------------------------------------------------
    def export(self):
        """Copies of (K, V) as device tensors in the pool's own layout."""
        k = torch.empty((self.num_blocks, self.kv_heads, self.block_size, self.head_dim),
                        dtype=self.storage_dtype, device=self.device)
        v = torch.empty((self.num_blocks, self.kv_heads, self.head_dim, self.block_size),
                        dtype=self.storage_dtype, device=self.device)
        L.check(L.pa_pool_export(self.handle, ctypes.c_void_p(k.data_ptr()),
                                 ctypes.c_void_p(v.data_ptr()), _stream(self.device)), "pa_pool_export")
        return k, v

    def import_(self, k, v):
        L.check(L.pa_pool_import(self.handle, _dev(k, self.storage_dtype, "k", self.device),
                                 _dev(v, self.storage_dtype, "v", self.device), _stream(self.device)),
                "pa_pool_import")


    def export_scales(self):
        """Biased exponents [num_blocks, Hkv, 2] (K, V) of a block-scaled pool, uint8."""
        e = torch.empty((self.num_blocks, self.kv_heads, 2), dtype=torch.uint8, device=self.device)
        L.check(L.pa_pool_export_scales(self.handle, ctypes.c_void_p(e.data_ptr()), _stream(self.device)),
                "pa_pool_export_scales")
        return e

    def import_scales(self, exps):
        if tuple(exps.shape) != (self.num_blocks, self.kv_heads, 2):
            raise ValueError("scales must be [num_blocks, Hkv, 2]")
        L.check(L.pa_pool_import_scales(self.handle,
                                        _dev(exps, torch.uint8, "scales", self.device), _stream(self.device)),
                "pa_pool_import_scales")


class BlockManager:
    """Host free pool, reference counts, copy-on-write and prefix hash (C++)."""

    def __init__(self, num_blocks, block_size, free_order=None):
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)
        h = ctypes.c_void_p()
        order = None
        if free_order is not None:
            self._order = np.ascontiguousarray(free_order, dtype=np.int32)
            order = _i32p(self._order)
        L.check(L.pa_bm_create(self.num_blocks, self.block_size, order, ctypes.byref(h)),
                "pa_bm_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            L.pa_bm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_request(self, tokens, salt=0):
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        rid, cached = ctypes.c_int(), ctypes.c_int()
        L.check(L.pa_bm_add_request(self.handle, _i32p(t), len(t), ctypes.c_uint64(salt),
                                    ctypes.byref(rid), ctypes.byref(cached)), "pa_bm_add_request")
        return rid.value, cached.value

    def fork(self, parent):
        c = ctypes.c_int()
        L.check(L.pa_bm_fork(self.handle, int(parent), ctypes.byref(c)), "pa_bm_fork")
        return c.value

    def append_slot(self, req, token):
        slot, s, d = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        L.check(L.pa_bm_append_slot(self.handle, int(req), int(token), ctypes.byref(slot),
                                    ctypes.byref(s), ctypes.byref(d)), "pa_bm_append_slot")
        return slot.value, s.value, d.value

    def append_slots(self, reqs, tokens):
        """Batched appends: returns (slots int64 [n], pairs int64 [P, 2])."""
        r = np.ascontiguousarray(reqs, dtype=np.int32)
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        n = len(r)
        slots = np.empty(n, dtype=np.int64)
        pairs = np.empty((max(n, 1), 2), dtype=np.int64)
        npairs, done = ctypes.c_int(), ctypes.c_int()
        L.check(L.pa_bm_append_slots(self.handle, n, _i32p(r), _i32p(t),
                                     slots.ctypes.data_as(L.c_i64p),
                                     pairs.ctypes.data_as(L.c_i64p), ctypes.byref(npairs),
                                     ctypes.byref(done)), "pa_bm_append_slots")
        return slots, pairs[:npairs.value].copy()

    def free_request(self, req):
        L.check(L.pa_bm_free_request(self.handle, int(req)), "pa_bm_free_request")

    def block_table(self, req):
        n = ctypes.c_int()
        L.check(L.pa_bm_block_table(self.handle, int(req), None, 0, ctypes.byref(n)),
                "pa_bm_block_table")
        out = np.empty(max(n.value, 1), dtype=np.int32)
        L.check(L.pa_bm_block_table(self.handle, int(req), _i32p(out), n.value, ctypes.byref(n)),
                "pa_bm_block_table")
        return out[:n.value].tolist()

    def batch_tables(self, reqs, width=None):
        r = np.ascontiguousarray(reqs, dtype=np.int32)
        if width is None:
            w = ctypes.c_int()
            L.check(L.pa_bm_batch_width(self.handle, len(r), _i32p(r), ctypes.byref(w)),
                    "pa_bm_batch_width")
            width = max(1, w.value)
        tables = np.empty((len(r), width), dtype=np.int32)
        lens = np.empty(len(r), dtype=np.int32)
        L.check(L.pa_bm_batch_tables(self.handle, len(r), _i32p(r), int(width), _i32p(tables),
                                     _i32p(lens)), "pa_bm_batch_tables")
        return tables, lens

    def seq_len(self, req):
        return L.pa_bm_seq_len(self.handle, int(req))

    def refcount(self, block):
        return L.pa_bm_refcount(self.handle, int(block))

    def num_free(self):
        return L.pa_bm_num_free(self.handle)

    def free_list(self):
        n = ctypes.c_int()
        out = np.empty(self.num_blocks, dtype=np.int32)
        L.check(L.pa_bm_free_list(self.handle, _i32p(out), self.num_blocks, ctypes.byref(n)),
                "pa_bm_free_list")
        return out[:n.value].tolist()

    def prefix_groups(self, reqs):
        """(offsets, seqs, shared_blocks) of the batch's sharing groups."""
        r = np.ascontiguousarray(reqs, dtype=np.int32)
        n = len(r)
        offs = np.zeros(n + 1, dtype=np.int32)
        seqs = np.zeros(max(n, 1), dtype=np.int32)
        nsh = np.zeros(max(n, 1), dtype=np.int32)
        ng = ctypes.c_int()
        L.check(L.pa_bm_prefix_groups(self.handle, n, _i32p(r), _i32p(offs), _i32p(seqs),
                                      _i32p(nsh), ctypes.byref(ng)), "pa_bm_prefix_groups")
        g = ng.value
        return offs[:g + 1].copy(), seqs[:offs[g]].copy(), nsh[:g].copy()

    def is_cached(self, block):
        return L.pa_bm_is_cached(self.handle, int(block)) == 1

    def set_retention(self, on):
        L.check(L.pa_bm_set_retention(self.handle, 1 if on else 0), "pa_bm_set_retention")

    def num_evictable(self):
        return L.pa_bm_num_evictable(self.handle)

    def evictable_list(self):
        n = ctypes.c_int()
        out = np.empty(self.num_blocks, dtype=np.int32)
        L.check(L.pa_bm_evictable_list(self.handle, _i32p(out), self.num_blocks, ctypes.byref(n)),
                "pa_bm_evictable_list")
        return out[:n.value].tolist()


def fnv1a64(data: bytes) -> int:
    buf = (ctypes.c_uint8 * max(len(data), 1)).from_buffer_copy(data or b"\0")
    return int(L.pa_bm_fnv1a64(buf, len(data)))


def launch_count() -> int:
    return int(L.pa_launch_count())
