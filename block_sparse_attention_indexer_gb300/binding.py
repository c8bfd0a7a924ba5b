"""Thin ctypes binding of libmsa.so (include/msa.h).

Argument marshalling only: every function takes torch tensors, checks dtype / device /
contiguity, passes data pointers and the current CUDA stream to the C entry point of the
same name, and raises MsaError on a non-OK status.  All compute happens in the library's
CUDA kernels; there is no Python or CPU fallback.  If libmsa.so has not been built the
import fails loudly (build with `python block_sparse_attention_indexer_gb300/build.py`).
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python block_sparse_attention_indexer_gb300/build.py` "
        "(the MSA path has no CPU fallback)")
_lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------------------- C types
MSA_OK, MSA_ERR_INVALID_ARG, MSA_ERR_UNSUPPORTED, MSA_ERR_WORKSPACE, MSA_ERR_CUDA = range(5)
MSA_OP_INDEXER_SCORES, MSA_OP_SELECT_BLOCKS, MSA_OP_SPARSE_ATTN, MSA_OP_DECODE = range(4)
MSA_OP_FP8_APPEND, MSA_OP_FP8_ATTN, MSA_OP_FP8_ATTN_WEIGHTS, MSA_OP_EVICT = range(4, 8)
MSA_OP_PROMPT_ATTN = 8
MSA_DEVERR_BAD_PAGE, MSA_DEVERR_BAD_SEQLEN, MSA_DEVERR_TIMEOUT, MSA_DEVERR_BAD_SCALE = 0x1, 0x2, 0x4, 0x8
MSA_DEVERR_NO_PAGE, MSA_DEVERR_BAD_PARENT = 0x10, 0x20
MSA_SCORE_MAX, MSA_SCORE_LSE = 0, 1
MSA_TYPE_F32, MSA_TYPE_BF16, MSA_TYPE_E4M3 = range(3)
MSA_E8M0_MIN, MSA_E8M0_MAX = 87, 167


class _Config(ctypes.Structure):
    _fields_ = [("num_kv_groups", ctypes.c_int32), ("heads_per_group", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("index_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("init_blocks", ctypes.c_int32), ("local_blocks", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("score_type", ctypes.c_int32)]


class _Cache(ctypes.Structure):
    _fields_ = [("k_data", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_data", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("idx_data", ctypes.c_void_p), ("idx_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64)]


class _Fp8Cache(ctypes.Structure):
    _fields_ = [("k_data", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_data", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64)]


class _Batch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("q_len", ctypes.c_int32)]


class _Packed(ctypes.Structure):
    _fields_ = [("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("q_tokens", ctypes.c_int64), ("k_tokens", ctypes.c_int64)]


class _PageBuffer(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("token_bytes", ctypes.c_int32)]


class _PagePool(ctypes.Structure):
    _fields_ = [("refs", ctypes.c_void_p), ("refs_out", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("buffers", ctypes.POINTER(_PageBuffer)), ("num_buffers", ctypes.c_int32)]


_P = ctypes.c_void_p
_CP, _CC, _CB = ctypes.POINTER(_Config), ctypes.POINTER(_Cache), ctypes.POINTER(_Batch)
_CF = ctypes.POINTER(_Fp8Cache)
_CK, _CG = ctypes.POINTER(_Packed), ctypes.POINTER(_PagePool)
_SIGS = {
    "msa_abi_version": (ctypes.c_int32, []),
    "msa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "msa_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, _CP, _CB]),
    "msa_nvfp4_insert": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P, _P,
                                        ctypes.c_int64, ctypes.c_int32, _P]),
    "msa_fp8_quantize": (ctypes.c_int, [_P, ctypes.c_int64, _P, _P]),
    "msa_indexer_scores": (ctypes.c_int, [_CP, _CC, _CB, _P, _P, _P, ctypes.c_size_t, _P]),
    "msa_select_blocks": (ctypes.c_int, [_CP, _CB, _P, _P, _P]),
    "msa_dcp_local_candidates": (ctypes.c_int, [_CP, _CC, _CB, _P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P,
                                                ctypes.c_size_t, _P]),
    "msa_dcp_merge": (ctypes.c_int, [_CP, _CB, ctypes.c_int32, _P, _P, _P, _P]),
    "msa_sparse_attn_decode": (ctypes.c_int, [_CP, _CC, _CB, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "msa_decode": (ctypes.c_int, [_CP, _CC, _CB, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "msa_fp8_append": (ctypes.c_int, [_CP, _CF, _CB, _P, _P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, _P,
                                      ctypes.c_size_t, _P]),
    "msa_fp8_attn": (ctypes.c_int, [_CP, _CF, _CB, _P, ctypes.c_int32, ctypes.c_int64, _P, _P, _P, _P, ctypes.c_float,
                                    _P, _P, ctypes.c_size_t, _P]),
    "msa_evict_blocks": (ctypes.c_int, [_CB, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P,
                                        _P, ctypes.c_size_t, _P]),
    "msa_prompt_workspace_bytes": (ctypes.c_size_t, [_CP, _CK]),
    "msa_prompt_attn": (ctypes.c_int, [_CP, _CK, _P, ctypes.c_int64, _P, ctypes.c_int64, _P, ctypes.c_int64, _P, _P, _P,
                                       ctypes.c_size_t, _P]),
    "msa_page_workspace_bytes": (ctypes.c_size_t, [_CG, ctypes.c_int32]),
    "msa_extend_pages": (ctypes.c_int, [_CG, _CB, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "msa_fork_pages": (ctypes.c_int, [_CG, _CB, _P, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]),
    "msa_free_pages": (ctypes.c_int, [_CG, _P, _P, ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "msa_compact_pages": (ctypes.c_int, [_CG, _CB, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "msa_sparse_attn_decode_noalloc": (ctypes.c_int, [_CP, _CC, _CB, _P, _P, _P, _P, _P]),
    "msa_noalloc_read_device_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), _P]),
    "msa_test_indexer_stall": (ctypes.c_int, [_CP, _CC, _CB, _P, _P, _P, ctypes.c_size_t, ctypes.c_uint32, _P]),
    "msa_test_attention_stall": (ctypes.c_int, [_CP, _CC, _CB, _P, _P, _P, _P, _P, ctypes.c_size_t, ctypes.c_uint32,
                                                _P]),
    "msa_read_device_error": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_uint32), _P]),
    "msa_clear_device_error": (ctypes.c_int, [_P, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


class MsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {_lib.msa_status_string(status).decode()}")


def _check(fn: str, status: int):
    if status != MSA_OK:
        raise MsaError(fn, status)


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _on(t: torch.Tensor, name: str) -> int:
    """Index of the CUDA device that t is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _at(t: Optional[torch.Tensor], shape, dtype, dev: int, name: str):
    """Pointer of a contiguous tensor that must have exactly this shape and type and be on
    device `dev` (None passes).  The calls below make these checks for up to nine tensors, so
    each is a plain comparison: a decode step's launch is a few microseconds."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on CUDA device {dev} like the block table, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _space(t: torch.Tensor, dev: int):
    """(pointer, bytes) of a workspace."""
    if t.get_device() != dev:
        raise ValueError(f"workspace must be on CUDA device {dev} like the block table, got {t.device}")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _launch(name: str, fn, dev: int, stream, *args):
    """Calls the C entry point with device `dev` current, on `stream` or that device's current
    stream."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if dev == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    _check(name, status)


def _token_rows(t: torch.Tensor, shape, dev: int, name: str):
    """(pointer, token stride in elements) of a [B, T, heads, dim] tensor whose heads are
    contiguous within a token and whose tokens are evenly spaced, b * T + t in order: a
    contiguous tensor, or a slice of the heads of one (no copy is made)."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on CUDA device {dev} like the block table, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    B, T, heads, dim = shape
    sb, st, sh, sd = t.stride()
    if sd != 1 or (heads > 1 and sh != dim) or (B > 1 and T > 1 and sb != T * st):
        raise ValueError(f"{name} must hold each token's heads contiguously and its tokens evenly spaced, "
                         f"got strides {t.stride()}")
    return t.data_ptr(), st if T > 1 else sb if B > 1 else heads * dim


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ---------------------------------------------------------------------------- Python-side views
@dataclasses.dataclass
class Config:
    num_kv_groups: int = 4
    heads_per_group: int = 8
    head_dim: int = 128
    index_dim: int = 128
    block_size: int = 128
    top_k: int = 16
    init_blocks: int = 0
    local_blocks: int = 1
    softmax_scale: float = 0.0      # 0 = 1/sqrt(head_dim)
    score_type: int = 0             # MSA_SCORE_MAX (0) or MSA_SCORE_LSE (1)

    def c(self):
        return ctypes.byref(_Config(self.num_kv_groups, self.heads_per_group, self.head_dim, self.index_dim,
                                    self.block_size, self.top_k, self.init_blocks, self.local_blocks,
                                    self.softmax_scale, self.score_type))

    @property
    def num_heads(self):
        return self.num_kv_groups * self.heads_per_group


class PagedCache:
    """The six NVFP4 page pools (device tensors, uint8), allocated by torch."""

    def __init__(self, num_pages: int, groups: int = 4, dim: int = 128, index_dim: int = 128, block: int = 128,
                 device="cuda"):
        u8 = dict(dtype=torch.uint8, device=device)
        self.num_pages, self.groups, self.block = num_pages, groups, block
        self.k_data = torch.zeros(num_pages, groups, block, dim // 2, **u8)
        self.k_scale = torch.zeros(num_pages, groups, block, dim // 16, **u8)
        self.v_data = torch.zeros(num_pages, groups, block, dim // 2, **u8)
        self.v_scale = torch.zeros(num_pages, groups, block, dim // 16, **u8)
        self.idx_data = torch.zeros(num_pages, block, index_dim // 2, **u8)
        self.idx_scale = torch.zeros(num_pages, block, index_dim // 16, **u8)

    def tensors(self):
        return (self.k_data, self.k_scale, self.v_data, self.v_scale, self.idx_data, self.idx_scale)

    def c(self):
        ps = [_ptr(t, torch.uint8, "cache") for t in self.tensors()]
        return ctypes.byref(_Cache(*ps, self.num_pages))

    @property
    def nbytes(self):
        return sum(t.numel() for t in self.tensors())


class Fp8Cache:
    """The FP8 K/V page pools (device tensors, uint8): E4M3 codes [P, groups, 128, 128] and
    E8M0 scales [P, groups] (value = code * 2^(scale - 127)); new pages hold zeros."""

    def __init__(self, num_pages: int, groups: int = 4, dim: int = 128, block: int = 128, device="cuda"):
        u8 = dict(dtype=torch.uint8, device=device)
        pool, heads = (num_pages, groups, block, dim), (num_pages, groups)
        self._hold(torch.zeros(pool, **u8), torch.full(heads, MSA_E8M0_MIN, **u8),
                   torch.zeros(pool, **u8), torch.full(heads, MSA_E8M0_MIN, **u8))

    @classmethod
    def from_tensors(cls, k_data: torch.Tensor, k_scale: torch.Tensor, v_data: torch.Tensor, v_scale: torch.Tensor):
        """A cache over pools the caller holds (no copy)."""
        self = cls.__new__(cls)
        self._hold(k_data, k_scale, v_data, v_scale)
        return self

    def _hold(self, k_data, k_scale, v_data, v_scale):
        # checked once: the pools of a cache are not replaced, so a call takes the struct as it is
        if k_data.dim() != 4:
            raise ValueError("k_data must be [pages, groups, block, dim]")
        pool, heads, self.device_index = k_data.shape, k_data.shape[:2], _on(k_data, "k_data")
        self._tensors = (k_data, k_scale, v_data, v_scale)
        u8 = torch.uint8
        self._c = _Fp8Cache(_at(k_data, pool, u8, self.device_index, "k_data"),
                            _at(k_scale, heads, u8, self.device_index, "k_scale"),
                            _at(v_data, pool, u8, self.device_index, "v_data"),
                            _at(v_scale, heads, u8, self.device_index, "v_scale"), pool[0])
        self._pages = tuple(pool[1:])

    k_data = property(lambda self: self._tensors[0])
    k_scale = property(lambda self: self._tensors[1])
    v_data = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])
    num_pages = property(lambda self: self._c.num_pages)
    groups = property(lambda self: self._pages[0])

    def tensors(self):
        return self._tensors

    def c(self):
        return ctypes.byref(self._c)

    @property
    def nbytes(self):
        return sum(t.numel() for t in self._tensors)


def _fp8_call(cfg: Config, cache: Fp8Cache, batch: Batch) -> int:
    """Checks that the configuration fits the cache, and both tensors of the batch: their device."""
    if cache._pages != (cfg.num_kv_groups, cfg.block_size, cfg.head_dim):
        raise ValueError(f"the cache's pages are {cache._pages}, the configuration's "
                         f"{(cfg.num_kv_groups, cfg.block_size, cfg.head_dim)}")
    dev = _batch_device(batch)
    if cache.device_index != dev:
        raise ValueError(f"the cache is on CUDA device {cache.device_index}, the block table on {dev}")
    return dev


def _batch_device(batch: Batch) -> int:
    dev = _on(batch.block_table, "block_table")
    if batch.seq_lens.get_device() != dev or batch.seq_lens.shape != (batch.block_table.shape[0],):
        raise ValueError(f"seq_lens must be [batch] on CUDA device {dev} like the block table, "
                         f"got {tuple(batch.seq_lens.shape)} on {batch.seq_lens.device}")
    return dev


@dataclasses.dataclass
class Batch:
    block_table: torch.Tensor     # int32 [B, max_blocks] on the device
    seq_lens: torch.Tensor        # int32 [B] on the device
    q_len: int = 1

    def c(self):
        B, MB = self.block_table.shape
        return ctypes.byref(_Batch(_ptr(self.block_table, torch.int32, "block_table"),
                                   _ptr(self.seq_lens, torch.int32, "seq_lens"), B, MB, self.q_len))

    @property
    def batch(self):
        return self.block_table.shape[0]

    @property
    def max_blocks(self):
        return self.block_table.shape[1]


@dataclasses.dataclass
class Packed:
    """Packed prompts: sequence b's query tokens are cu_q[b] .. cu_q[b + 1] - 1 of a list of q_tokens, its keys
    cu_k[b] .. cu_k[b + 1] - 1 of one of k_tokens."""
    cu_q: torch.Tensor            # int32 [B + 1] on the device
    cu_k: torch.Tensor            # int32 [B + 1] on the device (cu_q itself where every token is both)
    q_tokens: int
    k_tokens: int

    def c(self):
        n = self.cu_q.numel()
        if self.cu_q.dim() != 1 or n < 1:
            raise ValueError(f"cu_q must be [batch + 1], got {tuple(self.cu_q.shape)}")
        dev = _on(self.cu_q, "cu_q")
        return ctypes.byref(_Packed(_at(self.cu_q, (n,), torch.int32, dev, "cu_q"),
                                    _at(self.cu_k, (n,), torch.int32, dev, "cu_k"), n - 1, self.q_tokens, self.k_tokens))

    @property
    def batch(self):
        return self.cu_q.numel() - 1


class PagePool:
    """A pool of pages: refs (int32 [num_pages] on the device, 0 for a free page), and the caches
    whose pools hold the pages (of every layer that goes by the same block table).  refs may be replaced by
    another such tensor, a call's refs_out for example; the tensors of a PagedCache too: the next call goes by the new ones."""

    def __init__(self, caches=(), refs: Optional[torch.Tensor] = None, num_pages: Optional[int] = None, device=None):
        self.caches = tuple(caches)
        counts = {c.num_pages for c in self.caches} | ({int(num_pages)} if num_pages is not None else set())
        if refs is None:
            if len(counts) != 1:
                raise ValueError(f"the pool needs one number of pages, got {sorted(counts)}")
            where = self.caches[0].tensors()[0].device if device is None and self.caches else device or "cuda"
            refs = torch.zeros(counts.pop(), dtype=torch.int32, device=where)
        elif counts - {refs.numel()}:
            raise ValueError(f"refs counts {refs.numel()} pages, the caches have {sorted(counts)}")
        if refs.dim() != 1:
            raise ValueError(f"refs must be [num_pages], got {tuple(refs.shape)}")
        self.num_pages, self.device_index = refs.numel(), _on(refs, "refs")
        self._c = _PagePool(None, None, self.num_pages, None, 0)
        self.refs = refs
        self._take_buffers()

    @property
    def refs(self):
        return self._refs

    @refs.setter
    def refs(self, refs: torch.Tensor):
        self._c.refs = self._c.refs_out = _at(refs, (self.num_pages,), torch.int32, self.device_index, "refs")
        self._refs = refs

    def _take_buffers(self):
        buffers, held = [], []
        for c in self.caches:
            held.append(c.tensors())
            for t in held[-1]:
                if t.dtype != torch.uint8 or t.get_device() != self.device_index or not t.is_contiguous():
                    raise ValueError("the caches' pools must be contiguous uint8 tensors on the device of refs")
                if t.shape[0] != self.num_pages:
                    raise ValueError(f"the pool has {self.num_pages} pages, a cache's tensor {t.shape[0]}")
                page = t.numel() // self.num_pages if self.num_pages else 0
                # [P, groups, block, bytes] or [P, block, bytes]; FP8 scales [P, groups] belong to whole pages
                buffers.append(_PageBuffer(t.data_ptr(), page, t.shape[-1] if t.dim() > 2 else 0))
        self._buffers = (_PageBuffer * max(1, len(buffers)))(*buffers)
        self._held = held  # (the C structs have their addresses)
        self._c.buffers, self._c.num_buffers = self._buffers, len(buffers)

    def c(self, refs_out: Optional[torch.Tensor] = None, pages=False):
        """The C struct for a call that leaves the new counts in refs_out (None: in refs); pages: one that copies pages."""
        if pages:
            for c, held in zip(self.caches, self._held):
                now = c.tensors()
                if now is not held and (len(now) != len(held) or any(x is not y for x, y in zip(now, held))):
                    self._take_buffers()
                    break
        if refs_out is None:
            return ctypes.byref(self._c)
        out = _at(refs_out, (self.num_pages,), torch.int32, self.device_index, "refs_out")
        return ctypes.byref(_PagePool(self._c.refs, out, self.num_pages, self._buffers, self._c.num_buffers))


def _pool_batch(pool: PagePool, batch: Batch) -> int:
    dev = _batch_device(batch)
    if pool.device_index != dev:
        raise ValueError(f"the page pool is on CUDA device {pool.device_index}, the block table on {dev}")
    return dev


# ---------------------------------------------------------------------------- entry points
def msa_abi_version() -> int:
    return _lib.msa_abi_version()


def msa_workspace_bytes(op: int, cfg: Config, batch: Batch) -> int:
    return int(_lib.msa_workspace_bytes(op, cfg.c(), batch.c()))


def alloc_workspace(op: int, cfg: Config, batch, device="cuda") -> torch.Tensor:
    """Zero-filled workspace of the size `op` needs (the zero fill clears the error word).
    `batch` is a Batch, or for MSA_OP_PROMPT_ATTN a Packed."""
    size = msa_prompt_workspace_bytes(cfg, batch) if isinstance(batch, Packed) else msa_workspace_bytes(op, cfg, batch)
    return torch.zeros(max(size, 256), dtype=torch.uint8, device=device)


def msa_prompt_workspace_bytes(cfg: Config, packed: Packed) -> int:
    return int(_lib.msa_prompt_workspace_bytes(cfg.c(), packed.c()))


def msa_page_workspace_bytes(pool: PagePool, rows: int) -> int:
    return int(_lib.msa_page_workspace_bytes(pool.c(), rows))


def alloc_page_workspace(pool: PagePool, rows: int) -> torch.Tensor:
    """Zero-filled workspace of the page operators for calls of up to `rows` sequences (or children)."""
    return torch.zeros(max(msa_page_workspace_bytes(pool, rows), 256), dtype=torch.uint8, device=pool.refs.device)


def msa_nvfp4_insert(x: torch.Tensor, slots: torch.Tensor, data: torch.Tensor, scale: torch.Tensor,
                     block_size: int = 128, stream=None):
    """x float32 [n_tokens, rows_per_token, dim]; slots int64 [n_tokens]; data/scale are a
    cache pool pair ([P, rows, block, dim/2] and [P, rows, block, dim/16])."""
    n, rows, dim = x.shape
    num_pages = data.shape[0]
    _check("msa_nvfp4_insert", _lib.msa_nvfp4_insert(
        _ptr(x, torch.float32, "x"), n, rows, dim, _ptr(slots, torch.int64, "slots"),
        _ptr(data, torch.uint8, "data"), _ptr(scale, torch.uint8, "scale"), num_pages, block_size,
        _stream(stream)))


def msa_fp8_quantize(x: torch.Tensor, out: torch.Tensor, stream=None):
    _check("msa_fp8_quantize", _lib.msa_fp8_quantize(_ptr(x, torch.float32, "x"), x.numel(),
                                                     _ptr(out, torch.uint8, "out"), _stream(stream)))


def msa_indexer_scores(cfg: Config, cache: PagedCache, batch: Batch, index_q: torch.Tensor,
                       block_scores: torch.Tensor, workspace: torch.Tensor, stream=None):
    _check("msa_indexer_scores", _lib.msa_indexer_scores(
        cfg.c(), cache.c(), batch.c(), _ptr(index_q, torch.uint8, "index_q"),
        _ptr(block_scores, torch.float32, "block_scores"), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def msa_select_blocks(cfg: Config, batch: Batch, block_scores: torch.Tensor, selection: torch.Tensor, stream=None):
    _check("msa_select_blocks", _lib.msa_select_blocks(
        cfg.c(), batch.c(), _ptr(block_scores, torch.float32, "block_scores"),
        _ptr(selection, torch.int32, "selection"), _stream(stream)))


def msa_dcp_local_candidates(cfg: Config, cache: PagedCache, batch: Batch, index_q: torch.Tensor, block_lo: int,
                             block_hi: int, block_scores: torch.Tensor, cand_scores: torch.Tensor,
                             cand_blocks: torch.Tensor, workspace: torch.Tensor, stream=None):
    _check("msa_dcp_local_candidates", _lib.msa_dcp_local_candidates(
        cfg.c(), cache.c(), batch.c(), _ptr(index_q, torch.uint8, "index_q"), block_lo, block_hi,
        _ptr(block_scores, torch.float32, "block_scores"), _ptr(cand_scores, torch.float32, "cand_scores"),
        _ptr(cand_blocks, torch.int32, "cand_blocks"), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def msa_dcp_merge(cfg: Config, batch: Batch, cand_scores: torch.Tensor, cand_blocks: torch.Tensor,
                  selection: torch.Tensor, stream=None):
    """cand_scores / cand_blocks: [num_shards, B, T, G, 15] (the shards' outputs stacked)."""
    _check("msa_dcp_merge", _lib.msa_dcp_merge(
        cfg.c(), batch.c(), int(cand_scores.shape[0]), _ptr(cand_scores, torch.float32, "cand_scores"),
        _ptr(cand_blocks, torch.int32, "cand_blocks"), _ptr(selection, torch.int32, "selection"), _stream(stream)))


def msa_sparse_attn_decode(cfg: Config, cache: PagedCache, batch: Batch, q: torch.Tensor, selection: torch.Tensor,
                           out: torch.Tensor, lse: Optional[torch.Tensor], workspace: torch.Tensor, stream=None):
    _check("msa_sparse_attn_decode", _lib.msa_sparse_attn_decode(
        cfg.c(), cache.c(), batch.c(), _ptr(q, torch.uint8, "q"), _ptr(selection, torch.int32, "selection"),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def msa_sparse_attn_decode_noalloc(cfg: Config, cache: PagedCache, batch: Batch, q: torch.Tensor,
                                   selection: torch.Tensor, out: torch.Tensor, lse: Optional[torch.Tensor],
                                   stream=None):
    """msa_sparse_attn_decode without a workspace, for callers that cannot allocate device
    memory: the scratch is the library's own 8 MiB device array (see include/msa.h).  Calls
    that overlap on the GPU share that array and race."""
    _check("msa_sparse_attn_decode_noalloc", _lib.msa_sparse_attn_decode_noalloc(
        cfg.c(), cache.c(), batch.c(), _ptr(q, torch.uint8, "q"), _ptr(selection, torch.int32, "selection"),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"), _stream(stream)))


def msa_noalloc_read_device_error(stream=None) -> int:
    """The device error word of the no-allocation entry point's array (the last call's)."""
    flags = ctypes.c_uint32(0)
    _check("msa_noalloc_read_device_error", _lib.msa_noalloc_read_device_error(ctypes.byref(flags), _stream(stream)))
    return int(flags.value)


def msa_test_indexer_stall(cfg: Config, cache: PagedCache, batch: Batch, index_q: torch.Tensor,
                           block_scores: torch.Tensor, workspace: torch.Tensor, spin_limit: int, stream=None):
    """Test hook: the streaming indexer with its page copies withheld and its waits capped at
    spin_limit polls (include/msa.h)."""
    _check("msa_test_indexer_stall", _lib.msa_test_indexer_stall(
        cfg.c(), cache.c(), batch.c(), _ptr(index_q, torch.uint8, "index_q"),
        _ptr(block_scores, torch.float32, "block_scores"), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), spin_limit, _stream(stream)))


def msa_test_attention_stall(cfg: Config, cache: PagedCache, batch: Batch, q: torch.Tensor, selection: torch.Tensor,
                             out: torch.Tensor, lse: Optional[torch.Tensor], workspace: torch.Tensor, spin_limit: int,
                             stream=None):
    """Test hook: the team attention with its page copies withheld and every wait capped at
    spin_limit polls (the waits run out; MSA_DEVERR_TIMEOUT is set)."""
    _check("msa_test_attention_stall", _lib.msa_test_attention_stall(
        cfg.c(), cache.c(), batch.c(), _ptr(q, torch.uint8, "q"), _ptr(selection, torch.int32, "selection"),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), spin_limit, _stream(stream)))


def msa_decode(cfg: Config, cache: PagedCache, batch: Batch, q: torch.Tensor, index_q: torch.Tensor,
               out: torch.Tensor, lse: Optional[torch.Tensor], selection_out: Optional[torch.Tensor],
               workspace: torch.Tensor, stream=None):
    _check("msa_decode", _lib.msa_decode(
        cfg.c(), cache.c(), batch.c(), _ptr(q, torch.uint8, "q"), _ptr(index_q, torch.uint8, "index_q"),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(selection_out, torch.int32, "selection_out"), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


_ROW_TYPES = {torch.float32: MSA_TYPE_F32, torch.bfloat16: MSA_TYPE_BF16}
_QUERY_TYPES = {torch.uint8: MSA_TYPE_E4M3, torch.bfloat16: MSA_TYPE_BF16}


def msa_fp8_append(cfg: Config, cache: Fp8Cache, batch: Batch, k: torch.Tensor, v: torch.Tensor,
                   workspace: torch.Tensor, stream=None):
    """The q_len newest K and V rows of every sequence into their FP8 pages (include/msa.h).
    k, v: float32 or bfloat16 [B, T, G, 128], contiguous or a slice of the heads of a fused
    projection's rows.  workspace: alloc_workspace(MSA_OP_FP8_APPEND, ...)."""
    dev = _fp8_call(cfg, cache, batch)
    kind = _ROW_TYPES.get(k.dtype)
    if kind is None or v.dtype != k.dtype:
        raise TypeError(f"k and v must both be float32 or both bfloat16, got {k.dtype} and {v.dtype}")
    shape = (batch.batch, batch.q_len, cfg.num_kv_groups, cfg.head_dim)
    kp, ks = _token_rows(k, shape, dev, "k")
    vp, vs = _token_rows(v, shape, dev, "v")
    _launch("msa_fp8_append", _lib.msa_fp8_append, dev, stream, cfg.c(), cache.c(), batch.c(), kp, vp, kind, ks, vs,
            *_space(workspace, dev))


def msa_fp8_attn(cfg: Config, cache: Fp8Cache, batch: Batch, q: torch.Tensor, out: torch.Tensor,
                 lse: Optional[torch.Tensor], workspace: torch.Tensor, selection: Optional[torch.Tensor] = None,
                 weight_in: Optional[torch.Tensor] = None, weight_out: Optional[torch.Tensor] = None,
                 weight_decay: float = 1.0, stream=None):
    """Attention over the FP8 pages (include/msa.h): dense causal, or over selection
    [B, T, G, 16].  q: uint8 (E4M3 codes) or bfloat16 [B, T, H, 128], contiguous or a slice of the
    heads of wider rows; out: bfloat16 [B, T, H, 128]; lse: float32 [B, T, H] or None.
    weight_out (float32 [B, max_blocks]) receives weight_decay * weight_in plus the attention
    weight that each block collected; it may be weight_in.  workspace:
    alloc_workspace(MSA_OP_FP8_ATTN_WEIGHTS, ...) with weight_out, else MSA_OP_FP8_ATTN."""
    dev = _fp8_call(cfg, cache, batch)
    kind = _QUERY_TYPES.get(q.dtype)
    if kind is None:
        raise TypeError(f"q must be uint8 (E4M3 codes) or bfloat16, got {q.dtype}")
    table, T, H = batch.block_table.shape, batch.q_len, cfg.num_heads
    B = table[0]
    rows = (B, T, H, cfg.head_dim)
    qp, qs = _token_rows(q, rows, dev, "q")
    _launch("msa_fp8_attn", _lib.msa_fp8_attn, dev, stream, cfg.c(), cache.c(), batch.c(), qp, kind, qs,
            _at(selection, (B, T, cfg.num_kv_groups, 16), torch.int32, dev, "selection"),
            _at(out, rows, torch.bfloat16, dev, "out"), _at(lse, rows[:3], torch.float32, dev, "lse"),
            _at(weight_in, table, torch.float32, dev, "weight_in"), weight_decay,
            _at(weight_out, table, torch.float32, dev, "weight_out"), *_space(workspace, dev))


def msa_evict_blocks(batch: Batch, weight: torch.Tensor, budget: int, keep_first: int, keep_last: int,
                     table_out: torch.Tensor, seq_lens_out: torch.Tensor, weight_out: torch.Tensor,
                     freed: torch.Tensor, freed_count: torch.Tensor, workspace: torch.Tensor, stream=None):
    """Cuts every sequence to at most `budget` blocks by dropping those of least weight
    (include/msa.h).  table_out, seq_lens_out and weight_out may be batch.block_table,
    batch.seq_lens and weight.  workspace: alloc_workspace(MSA_OP_EVICT, ...)."""
    dev = _batch_device(batch)
    table = batch.block_table.shape
    rows, i32, f32 = table[:1], torch.int32, torch.float32
    _launch("msa_evict_blocks", _lib.msa_evict_blocks, dev, stream, batch.c(), _at(weight, table, f32, dev, "weight"),
            budget, keep_first, keep_last, _at(table_out, table, i32, dev, "table_out"),
            _at(seq_lens_out, rows, i32, dev, "seq_lens_out"), _at(weight_out, table, f32, dev, "weight_out"),
            _at(freed, table, i32, dev, "freed"), _at(freed_count, rows, i32, dev, "freed_count"),
            *_space(workspace, dev))


def _flat_rows(t: torch.Tensor, shape, dev: int, name: str):
    """(pointer, token stride in elements) of a bfloat16 [tokens, heads, dim] tensor whose heads are contiguous
    within a token (a slice of the heads of wider rows is: no copy is made)."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on CUDA device {dev} like cu_q, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    tokens, heads, dim = shape
    st, sh, sd = t.stride()
    if tokens and (sd != 1 or (heads > 1 and sh != dim)):
        raise ValueError(f"{name} must hold each token's heads contiguously, got strides {t.stride()}")
    return t.data_ptr(), st if tokens > 1 else heads * dim


def msa_prompt_attn(cfg: Config, packed: Packed, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                    lse: Optional[torch.Tensor], workspace: torch.Tensor, stream=None):
    """Causal attention of packed prompts over their own keys and values (include/msa.h).
    q: bfloat16 [q_tokens, H, 128]; k, v: bfloat16 [k_tokens, G, 128]; each contiguous or a slice of
    the heads of a fused projection's rows; out: bfloat16 [q_tokens, H, 128]; lse: float32
    [q_tokens, H] or None.  workspace: alloc_workspace(MSA_OP_PROMPT_ATTN, cfg, packed)."""
    dev = _on(packed.cu_q, "cu_q")
    rows = (packed.q_tokens, cfg.num_heads, cfg.head_dim)
    keys = (packed.k_tokens, cfg.num_kv_groups, cfg.head_dim)
    _launch("msa_prompt_attn", _lib.msa_prompt_attn, dev, stream, cfg.c(), packed.c(), *_flat_rows(q, rows, dev, "q"),
            *_flat_rows(k, keys, dev, "k"), *_flat_rows(v, keys, dev, "v"), _at(out, rows, torch.bfloat16, dev, "out"),
            _at(lse, rows[:2], torch.float32, dev, "lse"), *_space(workspace, dev))


def msa_extend_pages(pool: PagePool, batch: Batch, workspace: torch.Tensor, new_tokens: Optional[torch.Tensor] = None,
                     table_out: Optional[torch.Tensor] = None, seq_lens_out: Optional[torch.Tensor] = None,
                     refs_out: Optional[torch.Tensor] = None, stream=None):
    """Pages for the next new_tokens (int32 [B]; None: batch.q_len for every sequence that has tokens) of
    every sequence (include/msa.h), in place unless other outputs are given.  workspace:
    alloc_page_workspace(pool, B)."""
    dev = _pool_batch(pool, batch)
    table, i32 = batch.block_table.shape, torch.int32
    to = batch.block_table if table_out is None else table_out
    lens = batch.seq_lens if seq_lens_out is None else seq_lens_out
    _launch("msa_extend_pages", _lib.msa_extend_pages, dev, stream, pool.c(refs_out), batch.c(),
            _at(new_tokens, table[:1], i32, dev, "new_tokens"), _at(to, table, i32, dev, "table_out"),
            _at(lens, table[:1], i32, dev, "seq_lens_out"), *_space(workspace, dev))


def msa_fork_pages(pool: PagePool, batch: Batch, parents: torch.Tensor, table_out: torch.Tensor,
                   seq_lens_out: torch.Tensor, workspace: torch.Tensor, refs_out: Optional[torch.Tensor] = None,
                   stream=None):
    """Sequences that go on from batch's sequences parents (int32 [children]; -1: empty): table_out [children,
    max_blocks] and seq_lens_out [children] (include/msa.h).  workspace: alloc_page_workspace(pool, children)."""
    dev = _pool_batch(pool, batch)
    if parents.dim() != 1:
        raise ValueError(f"parents must be [children], got {tuple(parents.shape)}")
    n, i32 = parents.shape[0], torch.int32
    _launch("msa_fork_pages", _lib.msa_fork_pages, dev, stream, pool.c(refs_out, True), batch.c(),
            _at(parents, (n,), i32, dev, "parents"), n, _at(table_out, (n, batch.max_blocks), i32, dev, "table_out"),
            _at(seq_lens_out, (n,), i32, dev, "seq_lens_out"), *_space(workspace, dev))


def msa_free_pages(pool: PagePool, pages: torch.Tensor, workspace: torch.Tensor, counts: Optional[torch.Tensor] = None,
                   refs_out: Optional[torch.Tensor] = None, stream=None):
    """One reference to every listed page given back (include/msa.h): the first counts[r] entries of each
    row of pages (int32 [rows, width]; counts int32 [rows], None: all), msa_evict_blocks' freed and
    freed_count for example.  workspace: alloc_page_workspace(pool, 0)."""
    dev = pool.device_index
    if pages.dim() != 2:
        raise ValueError(f"pages must be [rows, width], got {tuple(pages.shape)}")
    rows, width = pages.shape
    _launch("msa_free_pages", _lib.msa_free_pages, dev, stream, pool.c(refs_out),
            _at(pages, (rows, width), torch.int32, dev, "pages"), _at(counts, (rows,), torch.int32, dev, "counts"), rows,
            width, *_space(workspace, dev))


def msa_compact_pages(pool: PagePool, batch: Batch, page_map: torch.Tensor, live_count: torch.Tensor,
                      workspace: torch.Tensor, table_out: Optional[torch.Tensor] = None,
                      refs_out: Optional[torch.Tensor] = None, stream=None):
    """The pages in use moved to the lowest numbers, the block table renamed in place or into table_out
    (include/msa.h).  page_map: int32 [num_pages], every page's new number; live_count: int32 [1].
    workspace: alloc_page_workspace(pool, 0)."""
    dev = _pool_batch(pool, batch)
    to, i32 = batch.block_table if table_out is None else table_out, torch.int32
    _launch("msa_compact_pages", _lib.msa_compact_pages, dev, stream, pool.c(refs_out, True), batch.c(),
            _at(to, batch.block_table.shape, i32, dev, "table_out"),
            _at(page_map, (pool.num_pages,), i32, dev, "page_map"), _at(live_count, (1,), i32, dev, "live_count"),
            *_space(workspace, dev))


def msa_read_device_error(workspace: torch.Tensor, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check("msa_read_device_error", _lib.msa_read_device_error(_ptr(workspace, None, "workspace"),
                                                               ctypes.byref(flags), _stream(stream)))
    return int(flags.value)


def msa_clear_device_error(workspace: torch.Tensor, stream=None):
    _check("msa_clear_device_error", _lib.msa_clear_device_error(_ptr(workspace, None, "workspace"),
                                                                 _stream(stream)))


def default_softmax_scale(head_dim: int = 128) -> float:
    return 1.0 / math.sqrt(head_dim)
