"""The paged cache's operators beside attention, over the C ABI of include/rpa.h.

Argument checks and marshalling only, as in ``binding``: every step of the
computation runs in the CUDA library.  Each class owns one library handle,
made on the current device from the keywords of ``RaggedPagedAttention``
(shapes, types and scales of the cache and of q) and its own.  Calls on one
object share its workspace and must be serialised on the GPU; a CUDA graph of
its calls uses that workspace too, so the object has to outlive the replays.
"""

from __future__ import annotations

import ctypes

import numpy as np

from .binding import (RPA_DT_BF16, RPA_DT_F16, RPA_DT_F32, RPA_KV_LATENT, RPA_OK, RpaError, RpaEvictCfg,
                      RpaRopeCfg, cache_shape, lib, make_cfg)

ROPE_PAIRINGS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "rotations": 3, "index": 4}


def _q_type(code):
    import torch

    return {RPA_DT_BF16: torch.bfloat16, RPA_DT_F16: torch.float16, RPA_DT_F32: torch.float32}[code]


class _Handle:
    """A library handle on the device that was current when it was made."""

    _prefix = ""  # of the C entry points
    _names = ()   # of the calls among them

    def _create(self, cfg, *more):
        import torch

        h = ctypes.c_void_p()
        r = getattr(lib(), self._prefix + "create")(ctypes.byref(cfg), *more, ctypes.byref(h))
        if r != RPA_OK:
            raise RpaError(r, self._prefix + "create")
        self._h = h
        self._device = torch.cuda.current_device()
        self._current = torch._C._cuda_getCurrentRawStream  # what torch.cuda.current_stream(device).cuda_stream is
        self._calls = {name: getattr(lib(), self._prefix + name) for name in self._names}

    def _checks(self, c):
        """What the calls' tensors have to be, from the RpaCfg."""
        import torch

        self._latent = c.kv_layout == RPA_KV_LATENT
        self._i32, self._f32 = torch.int32, torch.float32
        self._q_dtype = _q_type(c.q_dtype)
        self._q_shape = (c.num_q_tokens, c.num_q_heads, c.head_dim)
        self._kv_rows = (c.num_q_tokens, c.num_kv_heads, c.head_dim)  # of new keys
        self._kv_shape = cache_shape(c)
        self._kv_dtype = {RPA_DT_BF16: torch.bfloat16, RPA_DT_F16: torch.float16}.get(c.kv_dtype)  # None: one byte
        self._table_shape = (c.max_num_seqs, c.pages_per_seq)
        self._lens_shape, self._cu_shape = (c.max_num_seqs,), (c.max_num_seqs + 1,)
        self._scores_shape = (c.total_num_pages, c.num_kv_heads, c.page_size)

    def _need(self, name, t, dtype, shape):
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)}")

    def _need_cache(self, kv_pages):
        if kv_pages.shape != self._kv_shape or not kv_pages.is_contiguous():
            raise ValueError(f"kv_pages must be contiguous {self._kv_shape}")
        if (kv_pages.dtype != self._kv_dtype) if self._kv_dtype else (kv_pages.element_size() != 1):
            raise ValueError(f"kv_pages must hold {self._kv_dtype or 'one byte'} elements")

    def _need_lengths(self, kv_lens, page_indices, cu_q_lens):
        self._need("kv_lens", kv_lens, self._i32, self._lens_shape)
        self._need("page_indices", page_indices, self._i32, self._table_shape)
        if cu_q_lens is not None:
            self._need("cu_q_lens", cu_q_lens, self._i32, self._cu_shape)

    def _need_here(self, tensors):
        here = self._device
        for t in tensors:
            if t is not None and t.get_device() != here:
                raise ValueError(f"every tensor must be on cuda:{here}, where the handle was made")

    def _stream(self, stream, tensors=()):
        """The stream's pointer.  On another stream than the current one the tensors' memory is kept until it is done."""
        here = self._current(self._device)
        if stream is None:
            return here
        if stream.device.index != self._device:  # (every device's default stream has the same pointer)
            raise ValueError(f"the stream must be one of cuda:{self._device}, where the handle was made")
        if stream.cuda_stream == here:
            return here
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return stream.cuda_stream

    def _fits(self, kv_pages, kinds, plain):
        """Whether the cache and the plain tensors, whose (dtype, shape) are `kinds`, are contiguous, of their types and shapes, and
        here: all that the _need functions ask of them, in less time.  Where they are not, those say what is wrong."""
        here, kv_dtype = self._device, self._kv_dtype
        for t, (dtype, shape) in zip(plain, kinds):
            if t.dtype is not dtype or t.shape != shape or t.get_device() != here or not t.is_contiguous():
                return False
        return (kv_pages.shape == self._kv_shape and (kv_pages.dtype is kv_dtype if kv_dtype else kv_pages.element_size() == 1)
                and kv_pages.get_device() == here and kv_pages.is_contiguous())

    def _call(self, name, *args):
        if not self._h:
            raise ValueError("the handle is closed")
        r = self._calls[name](self._h, *args)
        if r != RPA_OK:
            raise RpaError(r, self._prefix + name)

    def status(self, stream=None) -> int:
        """The first device-detected error since the last status(), which this clears; synchronises the stream."""
        if not self._h:
            raise ValueError("the handle is closed")
        return int(getattr(lib(), self._prefix + "get_status")(self._h, self._stream(stream)))

    def close(self):
        if getattr(self, "_h", None):
            getattr(lib(), self._prefix + "destroy")(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def make_rope_cfg(*, rotary_dim=None, rotary_offset=0, pairing="half", scaling="none", base=10000.0, factor=1.0,
                  trained_len=0, low=1.0, high=4.0, magnitude=1.0, **cfg) -> RpaRopeCfg:
    c = RpaRopeCfg()
    c.cache = make_cfg(**dict(cfg, sinks=None))  # attention's alone: an append reads none
    c.rotary_dim = c.cache.head_dim if rotary_dim is None else int(rotary_dim)
    c.rotary_offset = int(rotary_offset)
    c.pairing, c.scaling = ROPE_PAIRINGS[pairing], ROPE_SCALINGS[scaling]
    c.base, c.factor, c.trained_len = float(base), float(factor), float(trained_len)
    c.low, c.high, c.magnitude = float(low), float(high), float(magnitude)
    return c


def validate_rope_cfg(**cfg) -> int:
    """Host-only check of RopeAppend's keywords: the status code."""
    return int(lib().rpa_rope_validate_cfg(ctypes.byref(make_rope_cfg(**cfg))))


def rope_frequencies(**cfg) -> np.ndarray:
    """Radians a position turns each pair by (float64 [rotary_dim / 2]) for RopeAppend's keywords."""
    c = make_rope_cfg(**cfg)
    w = np.zeros(max(1, c.rotary_dim // 2), np.float64)
    r = lib().rpa_rope_frequencies(ctypes.byref(c), w.ctypes.data)
    if r != RPA_OK:
        raise RpaError(r, "rpa_rope_frequencies")
    return w


class RopeAppend(_Handle):
    """Rotary positions on q and the new keys, and the write of the new K/V rows to the paged cache (``append``); its rows as
    values (``read``).

    Keywords beside RaggedPagedAttention's: ``rotary_dim`` (a multiple of 16; default the head) and
    ``rotary_offset`` (a multiple of 8) say which part of a head turns, ``pairing`` "half" or
    "interleaved" which elements form a pair; ``base``, ``scaling`` ("none", "linear", "base",
    "rotations", "index"), ``factor``, ``trained_len``, ``low`` and ``high`` the frequencies
    (include/rpa.h, RpaRopeScaling), ``magnitude`` a factor of the rotated values.
    """

    _prefix = "rpa_rope_"
    _names = ("append", "read")

    def __init__(self, **cfg):
        self._h = None
        self._c = make_rope_cfg(**cfg)
        self._create(self._c)
        self._checks(self._c.cache)
        self._append_kinds = ((self._i32, self._lens_shape), (self._i32, self._table_shape), (self._i32, self._cu_shape),
                              (self._q_dtype, self._q_shape))

    def _check(self, q, k, v, kv_pages, kv_lens, page_indices, cu_q_lens, positions, q_out):
        T, Hq, D = self._q_shape
        rows = self._kv_rows
        if (v is None) != self._latent:
            raise ValueError("v is None with the latent layout, whose rows are k, and only there")
        for name, t, shape in (("q", q, self._q_shape), ("k", k, rows), ("v", v, rows)):
            if t is None:
                continue
            # (one head has no distance to another)
            if t.dtype is not self._q_dtype or t.shape != shape or (T and (t.stride(2) != 1 or (shape[1] > 1 and t.stride(1) != D))):
                raise ValueError(f"{name} must be a {self._q_dtype} tensor {tuple(shape)} whose tokens' heads are contiguous")
        self._need_cache(kv_pages)
        self._need_lengths(kv_lens, page_indices, cu_q_lens)
        if positions is not None:
            self._need("positions", positions, self._i32, (T,))
        self._need("q_out", q_out, self._q_dtype, self._q_shape)

    def append(self, q, k, v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, positions=None, q_out=None, stream=None):
        """Write the tokens' K/V rows into kv_pages and return the rotated q (q_out; q itself where that is given).

        q [T, Hq, D], k and v [T, Hkv, D] in q's type: tokens may be any multiple of 16 bytes apart (slices of a
        fused projection).  kv_lens counts the new tokens: token i of a sequence goes to slot kv_len - q_len + i,
        which is its position too unless ``positions`` (int32 [T]) gives another.
        """
        if q_out is None:
            import torch

            with torch.cuda.stream(stream):
                q_out = torch.zeros(self._q_shape, dtype=self._q_dtype, device=q.device)
        dtype, D, here = self._q_dtype, self._q_shape[2], self._device
        tensors = (q, k, v, kv_pages, kv_lens, page_indices, cu_q_lens, positions, q_out)
        q_far = k_far = v_far = 0  # the distance of two tokens
        if v is not None and positions is None and self._q_shape[0] > 1:
            (q_far, q1, q2), (k_far, k1, k2), (v_far, v1, v2) = q.stride(), k.stride(), v.stride()
            fits = (q.dtype is k.dtype is v.dtype is dtype and q1 == k1 == v1 == D and q2 == k2 == v2 == 1 and not self._latent
                    and q.shape == self._q_shape and k.shape == v.shape == self._kv_rows
                    and q.get_device() == k.get_device() == v.get_device() == here
                    and self._fits(kv_pages, self._append_kinds, (kv_lens, page_indices, cu_q_lens, q_out)))
        else:
            fits = False
        if not fits:
            self._check(q, k, v, kv_pages, kv_lens, page_indices, cu_q_lens, positions, q_out)
            self._need_here(tensors)
            # (with one token any distance will do)
            far = self._q_shape[0] > 1
            rows = self._kv_rows[1] * self._kv_rows[2]
            q_far, k_far = (q.stride(0), k.stride(0)) if far else (self._q_shape[1] * D, rows)
            v_far = 0 if v is None else v.stride(0) if far else rows
        self._call("append", q.data_ptr(), q_far, k.data_ptr(), k_far, None if v is None else v.data_ptr(), v_far, kv_pages.data_ptr(),
                   kv_lens.data_ptr(), page_indices.data_ptr(), cu_q_lens.data_ptr(), None if positions is None else positions.data_ptr(),
                   int(num_seqs), q_out.data_ptr(), self._stream(stream, tensors))
        return q_out

    def _check_read(self, kv_pages, kv_lens, page_indices, cu_q_lens, k_out, v_out):
        self._need_cache(kv_pages)
        self._need_lengths(kv_lens, page_indices, cu_q_lens)
        self._need("k_out", k_out, self._q_dtype, self._kv_rows)
        if (v_out is None) != self._latent:
            raise ValueError("v_out is None with the latent layout, whose rows are k, and only there")
        if v_out is not None:
            self._need("v_out", v_out, self._q_dtype, self._kv_rows)

    def read(self, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, k_out=None, v_out=None, stream=None):
        """The cached rows of each sequence's last q_len keys as values: (k_out, v_out), [T, Hkv, D] in q's type, whatever
        wrote them (v_out None with the latent layout).  With cu_q_lens the running sum of kv_lens, whole sequences."""
        if k_out is None or (v_out is None and not self._latent):
            import torch

            with torch.cuda.stream(stream):
                new = lambda: torch.zeros(self._kv_rows, dtype=self._q_dtype, device=kv_pages.device)  # noqa: E731
                k_out = new() if k_out is None else k_out
                v_out = new() if v_out is None and not self._latent else v_out
        self._check_read(kv_pages, kv_lens, page_indices, cu_q_lens, k_out, v_out)
        tensors = (kv_pages, kv_lens, page_indices, cu_q_lens, k_out, v_out)
        self._need_here(tensors)
        self._call("read", kv_pages.data_ptr(), kv_lens.data_ptr(), page_indices.data_ptr(), cu_q_lens.data_ptr(), int(num_seqs),
                   k_out.data_ptr(), None if v_out is None else v_out.data_ptr(), self._stream(stream, tensors))
        return k_out, v_out


def make_evict_cfg(*, budget, protect=0, recent=0, **cfg) -> RpaEvictCfg:
    c = RpaEvictCfg()
    c.cache = make_cfg(**cfg)
    c.budget, c.protect, c.recent = int(budget), int(protect), int(recent)
    return c


def validate_evict_cfg(**cfg) -> int:
    """Host-only check of CacheEviction's keywords: the status code."""
    return int(lib().rpa_evict_validate_cfg(ctypes.byref(make_evict_cfg(_host_ok=True, **cfg))))


class CacheEviction(_Handle):
    """Eviction from the paged cache by accumulated attention weight.

    Keywords beside RaggedPagedAttention's: ``budget``, the keys a sequence keeps, of them the first
    ``protect`` and the last ``recent`` always.  ``scores`` [total_num_pages, Hkv, page_size] float32 lies
    beside kv_pages: ``accumulate`` adds to it, ``compact`` goes by it.
    """

    _prefix = "rpa_evict_"
    _names = ("accumulate", "compact")

    def __init__(self, **cfg):
        import torch

        self._h = None
        if isinstance(cfg.get("sinks"), np.ndarray):
            cfg["sinks"] = torch.from_numpy(np.ascontiguousarray(cfg["sinks"], np.float32)).cuda()
        self._sinks = cfg.get("sinks")  # read by every accumulate: kept alive
        self._c = make_evict_cfg(**cfg)
        self._create(self._c)
        self._checks(self._c.cache)

    def _check_accumulate(self, q, kv_pages, kv_lens, page_indices, cu_q_lens, scores):
        self._need("q", q, self._q_dtype, self._q_shape)
        self._need_cache(kv_pages)
        self._need_lengths(kv_lens, page_indices, cu_q_lens)
        self._need("scores", scores, self._f32, self._scores_shape)

    def accumulate(self, q, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, scores, stream=None):
        """Add the softmax weight each key gets from the call's queries to ``scores``, and return it.  The keys of
        the call's own tokens (each sequence's last q_len) start from 0."""
        self._check_accumulate(q, kv_pages, kv_lens, page_indices, cu_q_lens, scores)
        tensors = (q, kv_pages, kv_lens, page_indices, cu_q_lens, scores)
        self._need_here(tensors)
        self._call("accumulate", q.data_ptr(), kv_pages.data_ptr(), kv_lens.data_ptr(), page_indices.data_ptr(),
                   cu_q_lens.data_ptr(), int(num_seqs), scores.data_ptr(), self._stream(stream, tensors))
        return scores

    def _check_compact(self, kv_pages, scores, kv_lens, page_indices, new_page_indices, new_kv_lens, kept):
        self._need_cache(kv_pages)
        self._need("scores", scores, self._f32, self._scores_shape)
        self._need_lengths(kv_lens, page_indices, None)
        self._need("new_page_indices", new_page_indices, self._i32, self._table_shape)
        self._need("new_kv_lens", new_kv_lens, self._i32, self._lens_shape)
        if kept is not None:
            self._need("kept", kept, self._i32, (self._table_shape[0], self._c.cache.num_kv_heads, self._c.budget))

    def compact(self, kv_pages, scores, kv_lens, page_indices, num_seqs, new_page_indices=None, new_kv_lens=None, kept=None,
                stream=None):
        """Cut every sequence to the budget and return its new length (new_kv_lens, int32 [max_num_seqs]).

        The kept keys' rows and scores move, in order, to the first slots of new_page_indices' pages (default:
        page_indices, in place, where rows wait for each other: fresh pages are faster).  ``kept`` (int32
        [max_num_seqs, Hkv, budget]) receives the slots they had.  An object made for about as many and as long
        sequences as a call has is fastest.
        """
        if new_page_indices is None:
            new_page_indices = page_indices
        if new_kv_lens is None:
            import torch

            with torch.cuda.stream(stream):
                new_kv_lens = kv_lens.clone()
        self._check_compact(kv_pages, scores, kv_lens, page_indices, new_page_indices, new_kv_lens, kept)
        tensors = (kv_pages, scores, kv_lens, page_indices, new_page_indices, new_kv_lens, kept)
        self._need_here(tensors)
        self._call("compact", kv_pages.data_ptr(), scores.data_ptr(), kv_lens.data_ptr(), page_indices.data_ptr(), int(num_seqs),
                   new_page_indices.data_ptr(), new_kv_lens.data_ptr(), None if kept is None else kept.data_ptr(),
                   self._stream(stream, tensors))
        return new_kv_lens


def validate_prefix_cfg(*, max_groups=1, **cfg) -> int:
    """Host-only check of SharedPrefixAttention's keywords: the status code."""
    return int(lib().rpa_prefix_validate_cfg(ctypes.byref(make_cfg(_host_ok=True, **cfg)), int(max_groups)))


class SharedPrefixAttention(_Handle):
    """RaggedPagedAttention for batches whose sequences share their first keys: a group's prefix is read once for
    all of its query tokens.  Keywords beside RaggedPagedAttention's: ``max_groups``, the most groups of a call.
    """

    _prefix = "rpa_prefix_"
    _names = ("forward",)

    def __init__(self, *, max_groups=1, **cfg):
        import torch

        self._h = None
        if isinstance(cfg.get("sinks"), np.ndarray):
            cfg["sinks"] = torch.from_numpy(np.ascontiguousarray(cfg["sinks"], np.float32)).cuda()
        self._sinks = cfg.get("sinks")  # read by every call: kept alive
        self._c = make_cfg(**cfg)
        self._max_groups = int(max_groups)
        self._create(self._c, self._max_groups)
        self._checks(self._c)

    def _check(self, q, kv_pages, kv_lens, page_indices, cu_q_lens, cu_groups, prefix_lens, num_groups, out):
        self._need("q", q, self._q_dtype, self._q_shape)
        self._need("out", out, self._q_dtype, self._q_shape)
        self._need_cache(kv_pages)
        self._need_lengths(kv_lens, page_indices, cu_q_lens)
        for name, t, n in (("cu_groups", cu_groups, num_groups + 1), ("prefix_lens", prefix_lens, num_groups)):
            if t.dtype is not self._i32 or t.dim() != 1 or t.shape[0] < n or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor of at least {n}")

    def forward(self, q, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, cu_groups, prefix_lens, num_groups, out=None,
                stream=None):
        """RaggedPagedAttention.forward's result.  Group g is the sequences [cu_groups[g], cu_groups[g + 1]), which have
        their first prefix_lens[g] keys in common, read through the first one's page table."""
        num_groups = int(num_groups)
        if out is None:
            import torch

            with torch.cuda.stream(stream):
                out = torch.empty(self._q_shape, dtype=self._q_dtype, device=q.device)
        self._check(q, kv_pages, kv_lens, page_indices, cu_q_lens, cu_groups, prefix_lens, num_groups, out)
        tensors = (q, kv_pages, kv_lens, page_indices, cu_q_lens, cu_groups, prefix_lens, out)
        self._need_here(tensors)
        self._call("forward", q.data_ptr(), kv_pages.data_ptr(), kv_lens.data_ptr(), page_indices.data_ptr(), cu_q_lens.data_ptr(),
                   int(num_seqs), cu_groups.data_ptr(), prefix_lens.data_ptr(), num_groups, out.data_ptr(),
                   self._stream(stream, tensors))
        return out
