"""TurboQuant-prod / QJL compressed KV cache and decode attention on B200 (sm_100a).

The compute lives in ``libtq.so`` (hand-written CUDA kernels behind the C ABI
of ``include/tq.h``); ``native`` is its ctypes binding and this module adds
small owners of the device buffers (allocated with PyTorch) around it.
``native`` is loaded on first use (so that ``build`` can run before the library
exists); using any class here without a built ``libtq.so`` raises ImportError.
"""
from __future__ import annotations

import contextlib
import importlib
import math
from typing import Optional

import torch

__all__ = ["native", "TQError", "Codebook", "Projections", "CompressedKVCache", "PagedKVCache",
           "LayerGroups", "key_variance", "stack_partials", "gather_partials", "merge_partials"]


def __getattr__(name):
    if name == "TQError":
        return importlib.import_module(".native", __name__).TQError
    raise AttributeError(name)


class _Native:
    def __getattr__(self, name):
        return getattr(importlib.import_module(".native", __package__), name)


native = _Native()


class Codebook:
    """Lloyd-Max centroids/boundaries for head dim d and b1 bits, built on the GPU."""

    def __init__(self, d: int, bits: int, device="cuda"):
        self.d, self.bits = d, bits
        L = 1 << bits
        self.centroids = torch.empty(L, dtype=torch.float32, device=device)
        self.boundaries = torch.empty(max(L - 1, 1), dtype=torch.float32, device=device)
        native.tq_codebook_build(d, bits, self.centroids, self.boundaries)


class Projections:
    """Per-layer Pi (d x d), S (m x d) and T = S Pi^T, generated on the GPU.
    structured: the Hadamard rotation Pi = H diag(s) / sqrt(d) instead of the QR one."""

    def __init__(self, d: int, m: int, layer: int, rotation: bool = True, device="cuda",
                 base_seed: int = 42, stride: int = 7, structured: bool = False):
        self.d, self.m, self.layer = d, m, layer
        f32 = dict(dtype=torch.float32, device=device)
        self.Pi = torch.empty(d, d, **f32) if rotation else None
        self.S = torch.empty(m, d, **f32)
        self.T = torch.empty(m, d, **f32)
        if rotation and structured:
            native.tq_make_projections_hadamard(d, m, layer, self.Pi, self.S, self.T, base_seed, stride)
            return
        ws = None
        if rotation:
            ws = torch.empty(native.tq_projections_workspace_bytes(d), dtype=torch.uint8, device=device)
        native.tq_make_projections(d, m, layer, self.Pi, self.S, self.T, ws, base_seed, stride)


class LayerGroups:
    """A-QJL per-layer-group sketch dims from the config strings ("8,16,24", "512,384,256,192")."""

    def __init__(self, boundaries: str, sketch_dims: str):
        self._g = native.tq_layer_groups_parse(boundaries, sketch_dims)

    @classmethod
    def from_variances(cls, layer_var, num_groups: int, m_avg: int, m_min: int = 32,
                       m_max: int = 1024) -> "LayerGroups":
        """Sensitivity profile: groups and sketch dims from per-layer key variances."""
        obj = cls.__new__(cls)
        obj._g = native.tq_sensitivity_profile(layer_var, num_groups, m_avg, m_min, m_max)
        return obj

    @property
    def boundaries(self):
        return [int(self._g.bound[i]) for i in range(self._g.n - 1)]

    @property
    def sketch_dims(self):
        return [int(self._g.m[i]) for i in range(self._g.n)]

    def m_for_layer(self, layer: int) -> int:
        return native.tq_m_for_layer(self._g, layer)


def key_variance(K: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> float:
    """Population variance of every entry of one layer's calibration keys
    (tq_key_moments, one streaming pass on the device; waits for the result)."""
    out = torch.empty(2, dtype=torch.float64, device=K.device)
    if workspace is None:
        workspace = torch.empty(native.tq_key_moments_workspace_bytes(), dtype=torch.uint8,
                                device=K.device)
    native.tq_key_moments(K, out, workspace)
    return float(out[1].item())


class CompressedKVCache:
    """A packed cache of B x Hkv sequences plus its full-precision ring."""

    def __init__(self, B, Hkv, d, b1, m, vbits, group, W, capacity, dtype=torch.bfloat16,
                 device="cuda", structured: bool = False):
        """structured: the projections come from Projections(..., structured=True);
        the rotations on CUDA cores then run as fast Walsh-Hadamard transforms."""
        rot = native.TQ_ROTATION_HADAMARD if structured else native.TQ_ROTATION_DENSE
        self.desc = native.make_desc(B, Hkv, d, b1, m, vbits, group, W, capacity, dtype, rot)
        self.dtype = dtype
        nbytes = native.tq_cache_bytes(self.desc)
        if nbytes == 0:
            native.tq_cache_layout(self.desc)      # raises with the reason
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.state = native.tq_cache()
        native.tq_cache_init(self.state, self.desc, self.buffer)
        self._ws = None

    @property
    def n_total(self) -> int:
        return self.state.n_total

    @property
    def n_comp(self) -> int:
        return native.lib.tq_cache_compressed_tokens(self.state)

    @property
    def n_ring(self) -> int:
        return native.lib.tq_cache_ring_tokens(self.state)

    def append(self, K: torch.Tensor, V: torch.Tensor, proj: Projections, cb: Optional[Codebook]):
        native.tq_append(self.state, K, V, proj.Pi, proj.T,
                         cb.centroids if cb is not None else None,
                         cb.boundaries if cb is not None else None)

    def workspace(self, Hq: int, num_splits: int = 0) -> torch.Tensor:
        need = native.tq_decode_workspace_bytes(self.state, Hq, num_splits)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=self.buffer.device)
        return self._ws

    def decode_step(self, K: torch.Tensor, V: torch.Tensor, Q: torch.Tensor, proj: Projections,
                    cb: Optional[Codebook], softmax_scale: Optional[float] = None,
                    want_logits: bool = False, num_splits: int = 0,
                    out: Optional[torch.Tensor] = None):
        """append(K, V) then decode(Q) as one call (fused when the shapes allow)."""
        B, Hq, d = Q.shape
        scale = 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale
        out = torch.empty_like(Q) if out is None else out
        logits = None
        if want_logits:        # compressed + ring tokens after the append
            logits = torch.empty(B, Hq, self.n_total + K.shape[2], dtype=torch.float32,
                                 device=Q.device)
        ws = self.workspace(Hq, num_splits)
        native.tq_decode_step(self.state, K, V, Q, scale, proj.Pi, proj.S, proj.T,
                              cb.centroids if cb is not None else None,
                              cb.boundaries if cb is not None else None, out, logits, num_splits, ws)
        return (out, logits) if want_logits else out

    def prefill(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, proj: Projections,
                cb: Optional[Codebook], softmax_scale: Optional[float] = None, num_splits: int = 0,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        """Attention of a chunk of n new tokens before it is appended: Q [B, n, Hq, d]
        (token-major), K, V [B, Hkv, n, d]; query i sees the history, the ring and
        chunk tokens 0..i.  The cache is unchanged (call append(K, V) afterwards)."""
        B, n, Hq, d = Q.shape
        scale = 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale
        out = torch.empty_like(Q) if out is None else out
        if workspace is None:
            need = native.tq_prefill_workspace_bytes(self.state, Hq, n, num_splits)
            workspace = torch.empty(need, dtype=torch.uint8, device=self.buffer.device)
        native.tq_prefill_attention(self.state, Q, K, V, scale, proj.Pi, proj.S,
                                    cb.centroids if cb is not None else None, out, num_splits,
                                    workspace)
        return out

    def decode_partials(self, Q: torch.Tensor, proj: Projections, cb: Optional[Codebook],
                        softmax_scale: Optional[float] = None, num_splits: int = 0,
                        workspace: Optional[torch.Tensor] = None):
        """This cache's share of a context-sharded decode: query preparation and the
        split partials, not merged.  Returns (part_ml [B*Hq, S, 2], part_o
        [B*Hq, S, d]), float32 views into the workspace (valid until it is reused)."""
        B, Hq, d = Q.shape
        scale = 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale
        ws = self.workspace(Hq, num_splits) if workspace is None else workspace
        cent = cb.centroids if cb is not None else None
        native.tq_decode_prep(self.state, Q, scale, proj.Pi, proj.S, cent, num_splits, ws)
        native.tq_decode_partial(self.state, Hq, scale, cent, None, num_splits, ws)
        return native.tq_decode_partials_view(self.state, Hq, num_splits, ws)

    def decode(self, Q: torch.Tensor, proj: Projections, cb: Optional[Codebook],
               softmax_scale: Optional[float] = None, want_logits: bool = False,
               num_splits: int = 0, out: Optional[torch.Tensor] = None):
        B, Hq, d = Q.shape
        scale = 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale
        out = torch.empty_like(Q) if out is None else out
        logits = None
        if want_logits:
            logits = torch.empty(B, Hq, self.n_comp + self.n_ring, dtype=torch.float32, device=Q.device)
        ws = self.workspace(Hq, num_splits)
        native.tq_decode_attention(self.state, Q, scale, proj.Pi, proj.S,
                                   cb.centroids if cb is not None else None, out, logits,
                                   num_splits, ws)
        return (out, logits) if want_logits else out


_CURRENT = contextlib.nullcontext()       # a call on the current device needs no switch


class PagedKVCache:
    """Keys and values in 8 bits, in pages of `page` tokens with one scale per page and KV head;
    sequences of any lengths, named by slots 0 .. slots-1, that fork, copy and free.

    Slots and offsets are int32 CUDA tensors: row i of a call is slot slots[i] with the packed
    tokens cu[i] .. cu[i+1]-1 (token-major [tokens, heads, d]).  Checks that need the state on
    the device report through check(); see tq.h."""

    CODES = {"int8": 0, "e4m3": 1}

    def __init__(self, Hkv, d, pages, slots, max_pages, page: int = 64, code: str = "int8",
                 dtype=torch.bfloat16, layers: int = 1, device="cuda"):
        if code not in self.CODES:
            raise ValueError(f"code {code!r} is not one of {sorted(self.CODES)}")
        self.desc = native.make_paged_desc(layers, Hkv, d, page, pages, slots, max_pages, dtype,
                                           self.CODES[code])
        self.dtype = dtype
        nbytes = native.tq_paged_bytes(self.desc)
        if nbytes == 0:
            native.tq_paged_layout(self.desc)      # raises with the reason
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self._index = self.buffer.device.index
        self.state = native.tq_paged()
        with torch.cuda.device(self.buffer.device):
            native.tq_paged_init(self.state, self.desc, self.buffer)
        self._ws = {}
        self._cu = {}

    def _on(self, *tensors):
        """The cache's device made current; every tensor of the call has to be on it."""
        for t in tensors:
            if t is not None and t.get_device() != self._index:
                raise ValueError(f"tensor on {t.device}, the cache is on {self.buffer.device}")
        if torch.cuda.current_device() == self._index:
            return _CURRENT
        return torch.cuda.device(self.buffer.device)

    def _typed(self, *tensors):
        for t in tensors:
            if t.dtype != self.dtype:
                raise ValueError(f"expected {self.dtype}, got {t.dtype}")

    def workspace(self) -> torch.Tensor:
        """The attention workspace of the current stream (calls on different streams may run
        at the same time, so each has its own).  In a capture: one of the graph's own, made
        ready by the graph itself."""
        if torch.cuda.is_current_stream_capturing():
            return self.make_workspace()
        key = native.raw_stream(self._index)
        if key not in self._ws:
            self._ws[key] = self.make_workspace()
        return self._ws[key]

    def make_workspace(self) -> torch.Tensor:
        """A new workspace, for attend(workspace=...)."""
        with torch.cuda.device(self.buffer.device):
            ws = torch.empty(native.tq_paged_workspace_bytes(self.state), dtype=torch.uint8,
                             device=self.buffer.device)
            native.tq_paged_workspace_init(self.state, ws)
        return ws

    # ---- tokens in, floats out
    def extend(self, slots: torch.Tensor, cu: torch.Tensor, total: Optional[int] = None):
        """Take pages for cu[i+1]-cu[i] new tokens of each slot; then write() every layer.  total:
        the tokens that write() will be given, so that offsets past them are refused here, where
        the cache stays as it was (in write() they store zeros)."""
        with self._on(slots, cu):
            if total is None:
                native.tq_paged_extend(self.state, slots, cu)
            else:
                native.tq_paged_extend_within(self.state, slots, cu, total)

    def write(self, K: torch.Tensor, V: torch.Tensor, layer: int = 0):
        """The tokens of the last extend(), quantised into `layer`."""
        self._typed(K, V)
        with self._on(K, V):
            native.tq_paged_write(self.state, layer, K, V)

    def append(self, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, cu: torch.Tensor):
        """extend() and write() of a cache of one layer."""
        if self.desc.layers != 1:
            raise ValueError("a cache of several layers takes extend() and a write() per layer")
        self._typed(K, V)
        with self._on(K, V, slots, cu):
            native.tq_paged_append(self.state, slots, cu, K, V)

    def read(self, slots: torch.Tensor, cu: torch.Tensor, total: int, layer: int = 0):
        """The first cu[i+1]-cu[i] tokens of each slot as floats: (K, V), [total, Hkv, d]."""
        K, V = (torch.empty(total, self.desc.Hkv, self.desc.d, dtype=self.dtype,
                            device=self.buffer.device) for _ in range(2))
        with self._on(slots, cu):
            native.tq_paged_read(self.state, layer, slots, cu, K, V)
        return K, V

    # ---- attention
    def _queries(self, Q, slots, cu, out=None, lse=None, workspace=None):
        """What can be checked of an attention call without the library; (the device made current,
        what native.check_queries gives)."""
        queries = native.check_queries(self.state, Q, slots, cu)
        if Q.dtype != self.dtype:
            raise ValueError(f"expected {self.dtype}, got {Q.dtype}")
        if out is not None and (out.shape != Q.shape or out.dtype != self.dtype or not out.is_contiguous()):
            raise ValueError("out must be contiguous, of Q's shape and dtype")
        if lse is not None and (lse.shape != Q.shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous()):
            raise ValueError("lse must be contiguous float32 [tokens, Hq]")
        return self._on(Q, slots, cu, out, lse, workspace), queries

    def attend(self, Q: torch.Tensor, slots: torch.Tensor, cu: torch.Tensor, max_q: int,
               causal: bool = True, softmax_scale: Optional[float] = None, layer: int = 0,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None):
        """Row i's queries Q[cu[i]:cu[i+1]] over the tokens of slots[i].  causal: they are the
        sequence's last tokens, each sees the tokens up to itself.  out and lse (float32
        [tokens, Hq], log-sum-exp of the scaled logits) may be given."""
        on, queries = self._queries(Q, slots, cu, out, lse, workspace)
        with on:
            return self._attend(queries, Q, slots, cu, max_q, causal, softmax_scale, layer, out, lse,
                                workspace)

    def _attend(self, queries, Q, slots, cu, max_q, causal, softmax_scale, layer, out, lse, workspace):
        scale = 1.0 / math.sqrt(self.desc.d) if softmax_scale is None else softmax_scale
        if out is None:
            out = torch.empty(Q.shape, dtype=self.dtype, device=Q.device)
        ws = self.workspace() if workspace is None else workspace
        native.tq_paged_attention(self.state, layer, Q, slots, cu, max_q, causal, scale, out, lse, ws,
                                  queries=queries)
        return out

    def _ones(self, n: int) -> torch.Tensor:
        """Offsets of n rows of one token, made once (in a capture: the graph's own)."""
        if n not in self._cu:
            if torch.cuda.is_current_stream_capturing():
                return torch.arange(n + 1, dtype=torch.int32, device=self.buffer.device)
            # a copy that the host waits for: there for every stream
            self._cu[n] = torch.arange(n + 1, dtype=torch.int32).to(self.buffer.device)
        return self._cu[n]

    def decode(self, Q: torch.Tensor, slots: torch.Tensor, softmax_scale: Optional[float] = None,
               layer: int = 0, cu: Optional[torch.Tensor] = None, **kw):
        """One query per slot, Q [n, Hq, d], over all of its tokens."""
        cu = self._ones(slots.numel()) if cu is None else cu
        return self.attend(Q, slots, cu, 1, True, softmax_scale, layer, **kw)

    def decode_step(self, K: torch.Tensor, V: torch.Tensor, Q: torch.Tensor, slots: torch.Tensor,
                    cu: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                    layer: int = 0, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        """append() one token per slot (K, V [n, Hkv, d]), then decode().  What can be said of Q
        without the library is checked before the append."""
        cu = self._ones(slots.numel()) if cu is None else cu
        if softmax_scale is not None and not math.isfinite(softmax_scale):
            raise ValueError(f"softmax_scale {softmax_scale} is not finite")
        on, queries = self._queries(Q, slots, cu, out, lse, workspace)
        _, heads, at, stride, _ = queries
        if heads % self.desc.Hkv or not 1 <= heads // self.desc.Hkv <= 8:
            raise ValueError(f"{heads} query heads over {self.desc.Hkv} KV heads")
        if at % 16 or stride * Q.element_size() % 16 or (out is not None and out.data_ptr() % 16):
            raise ValueError("Q's tokens and out must be 16-byte aligned")
        with on:
            self.append(K, V, slots, cu)
            return self._attend(queries, Q, slots, cu, 1, True, softmax_scale, layer, out, lse,
                                workspace)

    def cross(self, Q: torch.Tensor, slots: torch.Tensor, cu: torch.Tensor, max_q: int,
              softmax_scale: Optional[float] = None, layer: int = 0, **kw):
        """Cross attention: the slots hold an encoder's states, every query sees all of them."""
        return self.attend(Q, slots, cu, max_q, False, softmax_scale, layer, **kw)

    # ---- pages
    def fork(self, src: torch.Tensor, dst: torch.Tensor):
        """Sequence src[i] also becomes dst[i] (an empty slot); full pages are shared."""
        with self._on(src, dst):
            native.tq_paged_fork(self.state, src, dst)

    def copy(self, src: torch.Tensor, dst: torch.Tensor, to: Optional["PagedKVCache"] = None):
        """Sequence src[i] copied to the empty slot dst[i] of `to` (default: this cache)."""
        other = self if to is None else to
        if other.buffer.device != self.buffer.device:
            raise ValueError("the caches are on different devices")
        with self._on(src, dst):
            native.tq_paged_copy(self.state, other.state, src, dst)

    def free(self, slots: torch.Tensor):
        with self._on(slots):
            native.tq_paged_free(self.state, slots)

    def compact(self):
        """Move the live pages to the front of the pool."""
        with self._on():
            native.tq_paged_compact(self.state)

    def page_table(self, slots: torch.Tensor) -> torch.Tensor:
        """int32 [n, max_pages]: the pages of each slot, -1 where it has none."""
        out = torch.empty(slots.numel(), self.desc.max_pages, dtype=torch.int32,
                          device=self.buffer.device)
        with self._on(slots):
            native.tq_paged_table(self.state, slots, out)
        return out

    @property
    def lengths(self) -> torch.Tensor:
        """int32 [slots], a view of the state on the device: tokens of each sequence."""
        o = self.state.o_len
        return self.buffer[o:o + 4 * self.desc.slots].view(torch.int32)

    def check(self) -> int:
        """Raise if a call failed a check on the device since the last check (waits for the
        stream); returns the number of free pages."""
        with self._on():
            return native.tq_paged_check(self.state)


# ----------------------------------------------------------------------------- sharded context
def stack_partials(parts, slots: int):
    """Split partials of several context shards side by side: parts = [(part_ml
    [rows, S_i, 2], part_o [rows, S_i, d]), ...] with S_i <= slots; a shard with
    fewer splits is padded with empty slots (m = -inf, l = 0, o = 0).  Returns
    (part_ml [rows, R * slots, 2], part_o [rows, R * slots, d]), contiguous."""
    mls, os_ = [], []
    for ml, o in parts:
        rows, s, d = o.shape
        if s > slots:
            raise ValueError(f"a shard has {s} splits, more than slots={slots}")
        pm = torch.zeros(rows, slots, 2, dtype=torch.float32, device=ml.device)
        pm[:, :, 0] = float("-inf")
        pm[:, :s] = ml
        po = torch.zeros(rows, slots, d, dtype=torch.float32, device=o.device)
        po[:, :s] = o
        mls.append(pm)
        os_.append(po)
    return torch.cat(mls, dim=1).contiguous(), torch.cat(os_, dim=1).contiguous()


def gather_partials(part_ml: torch.Tensor, part_o: torch.Tensor, slots: int, group=None):
    """All-gather every rank's split partials of one decode (each rank holds one shard
    of the context) and stack them as ``stack_partials`` does.  Every rank passes
    the same ``slots`` (at least its own split count)."""
    import torch.distributed as dist
    ml, o = stack_partials([(part_ml, part_o)], slots)
    R = dist.get_world_size(group)
    mls = [torch.empty_like(ml) for _ in range(R)]
    os_ = [torch.empty_like(o) for _ in range(R)]
    dist.all_gather(mls, ml, group=group)
    dist.all_gather(os_, o, group=group)
    return torch.cat(mls, dim=1).contiguous(), torch.cat(os_, dim=1).contiguous()


def merge_partials(part_ml: torch.Tensor, part_o: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """out [rows, d] (any float dtype): the softmax merge of the slots of each row."""
    native.tq_merge_partials(part_ml, part_o, out)
    return out
