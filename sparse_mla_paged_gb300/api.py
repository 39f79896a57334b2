"""Python binding of the C ABI (include/dsa_mla.h): argument marshalling only.

Every step of the decode runs in the library's sm_103a kernels; these functions pass
torch tensors' device pointers, sizes and the current CUDA stream through ctypes and
raise DsaError on a non-OK status.
"""
from __future__ import annotations

import contextlib
import threading
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import DsaError, check  # noqa: F401

LATENT = 512
INDEX = 128


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {dtype}")


def abi_version() -> int:
    return int(_lib.load().dsa_abi_version())


def status_string(status: int) -> str:
    return _lib.load().dsa_status_string(int(status)).decode()


def _decode_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, sel_indices, num_seqs,
                 rows_per_seq, num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale, sm_scale, out):
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.uint8, "k_cache")
    _need(v_cache, torch.uint8, "v_cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(sel_indices, torch.int32, "sel_indices")
    _need(out, torch.bfloat16, "out")
    return [_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), int(max_blocks_per_seq), _ptr(seq_lens),
            _ptr(sel_indices), int(sel_indices.shape[-1]), int(num_seqs), int(rows_per_seq), int(num_q_heads),
            int(block_size), int(cache_stride_bytes), float(k_scale), float(v_scale), float(sm_scale), _ptr(out)]


def _out_like(q, out):
    return torch.empty_like(q) if out is None else out


def decode(q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, sel_indices, num_seqs,
           rows_per_seq, num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale, sm_scale,
           out=None, stream=None) -> torch.Tensor:
    """dsa_mla_decode: per-row seq_lens; returns out (bf16 [R, H, 512])."""
    out = _out_like(q, out)
    a = _decode_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, sel_indices, num_seqs,
                     rows_per_seq, num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale, sm_scale, out)
    check(_lib.load().dsa_mla_decode(*a, _stream(stream)), "dsa_mla_decode")
    return out


def decode_k(q, k_cache, v_cache, block_tables, max_blocks_per_seq, base_lens, sel_indices, num_seqs, k,
             num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale, sm_scale, out=None,
             stream=None) -> torch.Tensor:
    """dsa_mla_decode_k: k verify rows per sequence; base_lens is per sequence."""
    out = _out_like(q, out)
    a = _decode_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq, base_lens, sel_indices, num_seqs, k,
                     num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale, sm_scale, out)
    check(_lib.load().dsa_mla_decode_k(*a, _stream(stream)), "dsa_mla_decode_k")
    return out


def workspace_bytes(num_seqs, rows_per_seq, num_q_heads, sel_width, num_ctas=0) -> int:
    return int(_lib.load().dsa_mla_decode_workspace_bytes(int(num_seqs), int(rows_per_seq), int(num_q_heads),
                                                          int(sel_width), int(num_ctas)))


def decode_grid(num_seqs, rows_per_seq, num_q_heads, sel_width, num_ctas=0) -> int:
    """Decode grid size a call of this shape runs with (dsa_mla_decode_grid; 0 = none)."""
    return int(_lib.load().dsa_mla_decode_grid(int(num_seqs), int(rows_per_seq), int(num_q_heads),
                                               int(sel_width), int(num_ctas)))


def alloc_workspace(num_seqs, rows_per_seq, num_q_heads, sel_width, num_ctas=0, device=None) -> torch.Tensor:
    n = workspace_bytes(num_seqs, rows_per_seq, num_q_heads, sel_width, num_ctas)
    if n == 0:
        raise DsaError(2, "dsa_mla_decode_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def options(num_ctas=0, tile_tokens=0, wait_limit_ns=0, ev_begin=None, ev_end=None,
            gather_mode=0) -> "_lib.DecodeOptions":
    """A dsa_decode_options struct (zero fields take the library defaults)."""
    o = _lib.DecodeOptions()
    o.num_ctas = int(num_ctas)
    o.tile_tokens = int(tile_tokens)
    o.gather_mode = int(gather_mode)
    o.wait_limit_ns = int(wait_limit_ns)
    o.ev_begin = None if ev_begin is None else ev_begin.cuda_event
    o.ev_end = None if ev_end is None else ev_end.cuda_event
    return o


def decode_ws(q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, sel_indices, num_seqs,
              rows_per_seq, num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale, sm_scale, out,
              workspace: torch.Tensor, verify_rows=0, num_ctas=0, ev_begin=None, ev_end=None,
              tile_tokens=0, wait_limit_ns=0, gather_mode=0, stream=None) -> torch.Tensor:
    """dsa_mla_decode_ws: caller workspace (capturable) and per-call options."""
    a = _decode_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, sel_indices, num_seqs,
                     rows_per_seq, num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale, sm_scale, out)
    _need(workspace, torch.uint8, "workspace")
    o = options(num_ctas, tile_tokens, wait_limit_ns, ev_begin, ev_end, gather_mode)
    check(_lib.load().dsa_mla_decode_ws(*a, int(verify_rows), _ptr(workspace), workspace.numel(),
                                        _lib.ctypes.byref(o), _stream(stream)), "dsa_mla_decode_ws")
    return out


def host_workspace_bytes(num_seqs, rows_per_seq, num_q_heads, sel_width, table_rows, max_blocks_per_seq,
                         verify_rows=0, num_ctas=0) -> int:
    return int(_lib.load().dsa_mla_decode_host_workspace_bytes(
        int(num_seqs), int(rows_per_seq), int(num_q_heads), int(sel_width), int(table_rows),
        int(max_blocks_per_seq), int(verify_rows), int(num_ctas)))


def decode_host(q_host, k_cache, v_cache, block_tables_host, max_blocks_per_seq, seq_lens_host, sel_host,
                num_seqs, rows_per_seq, num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale, sm_scale,
                out_host, workspace, verify_rows=0, num_ctas=0, stream=None) -> torch.Tensor:
    """dsa_mla_decode_host: per-step inputs and output in (pinned) host memory."""
    for t, n in ((q_host, "q_host"), (block_tables_host, "block_tables_host"), (seq_lens_host, "seq_lens_host"),
                 (sel_host, "sel_host"), (out_host, "out_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host tensor")
    _need(k_cache, torch.uint8, "k_cache")
    _need(v_cache, torch.uint8, "v_cache")
    check(_lib.load().dsa_mla_decode_host(
        _ptr(q_host), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables_host), int(block_tables_host.shape[0]),
        int(max_blocks_per_seq), _ptr(seq_lens_host), _ptr(sel_host), int(sel_host.shape[-1]), int(num_seqs),
        int(rows_per_seq), int(num_q_heads), int(block_size), int(cache_stride_bytes), float(k_scale),
        float(v_scale), float(sm_scale), _ptr(out_host), int(verify_rows), _ptr(workspace), workspace.numel(),
        int(num_ctas), _stream(stream)), "dsa_mla_decode_host")
    return out_host


def resolve_indices(sel_indices: torch.Tensor, seq_lens: torch.Tensor, stream=None):
    """dsa_resolve_indices -> (ids int32 [rows, W], counts int32 [rows])."""
    _need(sel_indices, torch.int32, "sel_indices")
    _need(seq_lens, torch.int32, "seq_lens")
    rows, width = sel_indices.shape
    ids = torch.empty((rows, width), dtype=torch.int32, device=sel_indices.device)
    counts = torch.empty(rows, dtype=torch.int32, device=sel_indices.device)
    check(_lib.load().dsa_resolve_indices(_ptr(sel_indices), _ptr(seq_lens), int(width), int(rows), _ptr(ids),
                                          _ptr(counts), _stream(stream)), "dsa_resolve_indices")
    return ids, counts


def latent_write(kv_a: torch.Tensor, norm_weight: torch.Tensor, slots: torch.Tensor, rms_eps: float,
                 kv_scale: float, block_size: int, cache_stride_bytes: int, cache: torch.Tensor,
                 stream=None) -> torch.Tensor:
    """dsa_latent_write: RMSNorm(kv_a) * weight * (1/kv_scale) as E4M3 into each row's slot of
    the paged cache (negative slot: skipped). Returns cache."""
    _need(kv_a, torch.bfloat16, "kv_a")
    _need(norm_weight, torch.bfloat16, "norm_weight")
    _need(slots, torch.int64, "slots")
    _need(cache, torch.uint8, "cache")
    if kv_a.shape[-1] != LATENT or norm_weight.numel() != LATENT or slots.numel() != kv_a.numel() // LATENT:
        raise ValueError("kv_a [rows, 512], norm_weight [512], slots [rows]")
    check(_lib.load().dsa_latent_write(_ptr(kv_a), _ptr(norm_weight), _ptr(slots), int(slots.numel()),
                                       float(rms_eps), float(kv_scale), int(block_size), int(cache_stride_bytes),
                                       _ptr(cache), _stream(stream)), "dsa_latent_write")
    return cache


def select_pools(scores: torch.Tensor, q_pos: torch.Tensor, kpool: int, topk: int, out=None,
                 stream=None) -> torch.Tensor:
    """dsa_select_pools: per row the topk highest-scoring pools ending at or before q_pos, as
    ascending token ids (kpool per pool), -1 padded; returns int32 [rows, topk * kpool]."""
    _need(scores, torch.float32, "scores")
    _need(q_pos, torch.int32, "q_pos")
    rows, n_pools = scores.shape
    if out is None:
        out = torch.empty((rows, topk * kpool), dtype=torch.int32, device=scores.device)
    _need(out, torch.int32, "out")
    check(_lib.load().dsa_select_pools(_ptr(scores), _ptr(q_pos), int(rows), int(n_pools), int(kpool), int(topk),
                                       _ptr(out), _stream(stream)), "dsa_select_pools")
    return out


def _absorb_out(shape, dtype, device, out):
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("absorb output must be float32 or bfloat16")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    _need(out, dtype, "out")
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must have shape {tuple(shape)}")
    return out, 0 if dtype == torch.float32 else 1


def absorb_q(q_b: torch.Tensor, kv_b: torch.Tensor, heads: int, nope: int, vd: int, dtype=torch.float32, out=None,
             stream=None) -> torch.Tensor:
    """dsa_absorb_q (build.rs absorb_q): q_b bf16 [heads*nope, q_lora_rank], kv_b bf16
    [heads*(nope+vd), kvl] -> [heads*kvl, q_lora_rank] in `dtype` (float32 or bfloat16)."""
    _need(q_b, torch.bfloat16, "q_b")
    _need(kv_b, torch.bfloat16, "kv_b")
    ql, kvl = q_b.shape[1], kv_b.shape[1]
    if q_b.shape[0] != heads * nope or kv_b.shape[0] != heads * (nope + vd):
        raise ValueError("absorb_q: shapes do not match heads/nope/vd")
    out, code = _absorb_out((heads * kvl, ql), dtype, q_b.device, out)
    check(_lib.load().dsa_absorb_q(_ptr(q_b), _ptr(kv_b), heads, nope, vd, kvl, ql, _ptr(out), code,
                                   _stream(stream)), "dsa_absorb_q")
    return out


def absorb_o(o_proj: torch.Tensor, kv_b: torch.Tensor, heads: int, nope: int, vd: int, dtype=torch.float32,
             out=None, stream=None) -> torch.Tensor:
    """dsa_absorb_o (build.rs absorb_o): o_proj bf16 [hidden, heads*vd], kv_b bf16
    [heads*(nope+vd), kvl] -> [hidden, heads*kvl] in `dtype` (float32 or bfloat16)."""
    _need(o_proj, torch.bfloat16, "o_proj")
    _need(kv_b, torch.bfloat16, "kv_b")
    hidden, kvl = o_proj.shape[0], kv_b.shape[1]
    if o_proj.shape[1] != heads * vd or kv_b.shape[0] != heads * (nope + vd):
        raise ValueError("absorb_o: shapes do not match heads/nope/vd")
    out, code = _absorb_out((hidden, heads * kvl), dtype, o_proj.device, out)
    check(_lib.load().dsa_absorb_o(_ptr(o_proj), _ptr(kv_b), heads, nope, vd, kvl, hidden, _ptr(out), code,
                                   _stream(stream)), "dsa_absorb_o")
    return out


def _device_of(t: torch.Tensor, name: str) -> int:
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return i


def _need_on(t: torch.Tensor, dtype, name: str, index: int):
    if t.get_device() != index or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {dtype} on cuda:{index}")


def _fit(*sizes):
    # ctypes would cut a larger number to its low 32 bits.
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise ValueError("sizes must be 32-bit numbers")


class _Launch:
    """What a call needs of its device: makes it current for the call (when it is not), and
    gives the raw stream and the context in which its outputs are allocated (the given
    stream's, so that their memory is not handed out again while that stream uses it)."""
    __slots__ = ("index", "raw", "stream", "guard")

    def __init__(self, index: int, stream):
        self.index = index
        self.guard = None
        if stream is None:
            self.stream = None
            self.raw = torch._C._cuda_getCurrentRawStream(index)
        else:
            self.raw = _stream(stream)
            self.stream = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(self.raw, device=index)

    def __enter__(self):
        if torch.cuda.current_device() != self.index:
            self.guard = torch.cuda.device(self.index)
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False

    def allocating(self):
        return contextlib.nullcontext() if self.stream is None else torch.cuda.stream(self.stream)


class StepPlan(NamedTuple):
    """dsa_plan_step's outputs, a row per new token: slots int64, positions, row_lens and row_seqs
    int32 [rows]; info int32 [4] (rows with a token, pages taken, status, 0)."""
    slots: torch.Tensor
    positions: torch.Tensor
    row_lens: torch.Tensor
    row_seqs: torch.Tensor
    info: torch.Tensor


def alloc_step_plan(rows: int, device=None) -> StepPlan:
    """Output buffers of plan_step, to be kept from step to step (a captured step needs fixed ones)."""
    device, i32 = device or "cuda", torch.int32
    return StepPlan(torch.empty(rows, dtype=torch.int64, device=device), torch.empty(rows, dtype=i32, device=device),
                    torch.empty(rows, dtype=i32, device=device), torch.empty(rows, dtype=i32, device=device),
                    torch.empty(4, dtype=i32, device=device))


def plan_step(base_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor, block_size: int,
              block_tables: torch.Tensor, rows_per_seq: int = 0, max_rows: Optional[int] = None,
              out: Optional[StepPlan] = None, stream=None) -> StepPlan:
    """dsa_plan_step: pages for every request's new tokens into block_tables (in place), and each
    new token's slot, position, visible length and request. rows_per_seq 0 packs the rows
    (max_rows is then needed, unless out gives it), else row s*rows_per_seq + i is token i of
    request s."""
    i = _device_of(base_lens, "base_lens")
    for t, n in ((base_lens, "base_lens"), (new_lens, "new_lens"), (free_pages, "free_pages"),
                 (block_tables, "block_tables")):
        _need_on(t, torch.int32, n, i)
    n = base_lens.numel()
    if new_lens.numel() != n or block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise ValueError("base_lens [num_seqs], new_lens [num_seqs], block_tables [num_seqs, max_blocks_per_seq]")
    rows = n * rows_per_seq if rows_per_seq else (max_rows if out is None else out.slots.numel())
    if rows is None or (max_rows is not None and max_rows != rows):
        raise ValueError("max_rows must be the number of rows to write (num_seqs*rows_per_seq unless packed)")
    _fit(rows, rows_per_seq, free_pages.numel(), block_size, block_tables.shape[1])
    with _Launch(i, stream) as at:
        if out is None:
            with at.allocating():
                out = alloc_step_plan(rows, base_lens.device)
        else:
            _need_on(out.slots, torch.int64, "out.slots", i)
            for t in out[1:]:
                _need_on(t, torch.int32, "out", i)
            if out.info.numel() < 4 or any(t.numel() != rows for t in out[:4]):
                raise ValueError(f"out must hold {rows} rows")
        check(_lib.load().dsa_plan_step(base_lens.data_ptr(), new_lens.data_ptr(), n, rows_per_seq, rows,
                                        free_pages.data_ptr(), free_pages.numel(), block_size, block_tables.data_ptr(),
                                        block_tables.shape[1], out.slots.data_ptr(), out.positions.data_ptr(),
                                        out.row_lens.data_ptr(), out.row_seqs.data_ptr(), out.info.data_ptr(), at.raw),
              "dsa_plan_step")
    return out


def index_page_stride(block_size: int) -> int:
    """Smallest page stride of the index cache: block_size*(128 codes + a float32 scale), in 16s."""
    return (block_size * (INDEX + 4) + 15) // 16 * 16


def index_write(keys: torch.Tensor, slots: torch.Tensor, block_size: int, page_stride_bytes: int,
                index_cache: torch.Tensor, norm_weight: Optional[torch.Tensor] = None,
                norm_bias: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None) -> torch.Tensor:
    """dsa_index_write: the (layer-normalised) index keys bf16 [rows, 128] as E4M3 codes and a
    float32 scale per row into each row's slot (negative: skipped). Returns index_cache."""
    i = _device_of(index_cache, "index_cache")
    _need_on(keys, torch.bfloat16, "keys", i)
    _need_on(slots, torch.int64, "slots", i)
    _need_on(index_cache, torch.uint8, "index_cache", i)
    rows = slots.numel()
    if keys.shape[-1] != INDEX or rows * INDEX != keys.numel():
        raise ValueError("keys [rows, 128], slots [rows]")
    for t, n in ((norm_weight, "norm_weight"), (norm_bias, "norm_bias")):
        if t is not None:
            _need_on(t, torch.bfloat16, n, i)
            if t.numel() != INDEX:
                raise ValueError(f"{n} [128]")
    _fit(rows, block_size)
    with _Launch(i, stream) as at:
        check(_lib.load().dsa_index_write(keys.data_ptr(), _ptr(norm_weight), _ptr(norm_bias), slots.data_ptr(), rows,
                                          eps, block_size, page_stride_bytes, index_cache.data_ptr(), at.raw),
              "dsa_index_write")
    return index_cache


_wait_limits = threading.local()


@contextlib.contextmanager
def wait_limit(limit_ns: int):
    """dsa_set_wait_limit for this thread's pool_scores and decode_full calls inside the block
    (0: the default), the limit outside it after that."""
    if not 0 <= limit_ns < 1 << 64:
        raise ValueError("limit_ns must be a 64-bit number of nanoseconds")
    outer = getattr(_wait_limits, "ns", 0)
    check(_lib.load().dsa_set_wait_limit(limit_ns), "dsa_set_wait_limit")
    _wait_limits.ns = limit_ns
    try:
        yield
    finally:
        _wait_limits.ns = outer
        check(_lib.load().dsa_set_wait_limit(outer), "dsa_set_wait_limit")


def _table_rows(block_tables, max_blocks_per_seq, num_seqs):
    need = num_seqs * max_blocks_per_seq if max_blocks_per_seq > 0 else 1
    if block_tables.numel() < need:
        raise ValueError(f"block_tables must hold {need} entries")


def pool_scores(q: torch.Tensor, head_weights: torch.Tensor, index_cache: torch.Tensor, block_tables: torch.Tensor,
                max_blocks_per_seq: int, q_pos: torch.Tensor, num_seqs: int, rows_per_seq: int, num_heads: int,
                block_size: int, page_stride_bytes: int, kpool: int, n_pools: int, out=None, device_status=None,
                stream=None) -> torch.Tensor:
    """dsa_pool_scores: float32 [R, n_pools], per row the maximum over each pool's kpool positions of
    scale_j * sum_h head_weights[h] * max(0, q[h] . k_j); -inf for pools that end after q_pos.
    Without a device_status word (int32 [1]) step_device_status tells of bad pages."""
    i = _device_of(q, "q")
    _need_on(q, torch.bfloat16, "q", i)
    _need_on(head_weights, torch.float32, "head_weights", i)
    _need_on(index_cache, torch.uint8, "index_cache", i)
    _need_on(block_tables, torch.int32, "block_tables", i)
    _need_on(q_pos, torch.int32, "q_pos", i)
    _fit(num_seqs, rows_per_seq, num_heads, max_blocks_per_seq, block_size, kpool, n_pools)
    rows = num_seqs * rows_per_seq
    if q.numel() != rows * num_heads * INDEX or head_weights.numel() != rows * num_heads or q_pos.numel() != rows:
        raise ValueError("q [R, num_heads, 128], head_weights [R, num_heads], q_pos [R]")
    _table_rows(block_tables, max_blocks_per_seq, num_seqs)
    if device_status is not None:
        _need_on(device_status, torch.int32, "device_status", i)
    with _Launch(i, stream) as at:
        if out is None:
            with at.allocating():
                out = torch.empty((rows, n_pools), dtype=torch.float32, device=q.device)
        else:
            _need_on(out, torch.float32, "out", i)
            if out.numel() != rows * n_pools:
                raise ValueError(f"out must hold [{rows}, {n_pools}]")
        check(_lib.load().dsa_pool_scores(q.data_ptr(), head_weights.data_ptr(), index_cache.data_ptr(),
                                          block_tables.data_ptr(), max_blocks_per_seq, q_pos.data_ptr(), num_seqs,
                                          rows_per_seq, num_heads, block_size, page_stride_bytes, kpool, n_pools,
                                          out.data_ptr(), _ptr(device_status), at.raw), "dsa_pool_scores")
    return out


def full_workspace_bytes(num_seqs: int, rows_per_seq: int, num_q_heads: int) -> int:
    return int(_lib.load().dsa_mla_decode_full_workspace_bytes(int(num_seqs), int(rows_per_seq), int(num_q_heads)))


def alloc_full_workspace(num_seqs: int, rows_per_seq: int, num_q_heads: int, device=None) -> torch.Tensor:
    """A workspace for decode_full, to be kept from call to call (one per stream or captured graph)."""
    device = torch.device(device or "cuda")
    with torch.cuda.device(device):
        n = full_workspace_bytes(num_seqs, rows_per_seq, num_q_heads)
    if n == 0:
        raise DsaError(2, "dsa_mla_decode_full_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_full(q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, num_seqs, rows_per_seq, num_q_heads,
                block_size, cache_stride_bytes, k_scale, v_scale, sm_scale, out=None, verify_rows=0, workspace=None,
                stream=None) -> torch.Tensor:
    """dsa_mla_decode_full: every row attends to its whole cache; seq_lens per row, or with
    verify_rows per sequence before its rows. Returns out (bf16 [R, H, 512]). Without a
    workspace one is allocated for the call. step_device_status tells of bad pages and lengths."""
    i = _device_of(q, "q")
    _need_on(q, torch.bfloat16, "q", i)
    _need_on(k_cache, torch.uint8, "k_cache", i)
    _need_on(v_cache, torch.uint8, "v_cache", i)
    _need_on(block_tables, torch.int32, "block_tables", i)
    _need_on(seq_lens, torch.int32, "seq_lens", i)
    _fit(num_seqs, rows_per_seq, num_q_heads, max_blocks_per_seq, block_size)
    rows = num_seqs * rows_per_seq
    if q.numel() != rows * num_q_heads * LATENT or seq_lens.numel() != (num_seqs if verify_rows else rows):
        raise ValueError("q [R, num_q_heads, 512], seq_lens [R] ([num_seqs] for verify rows)")
    _table_rows(block_tables, max_blocks_per_seq, num_seqs)
    with _Launch(i, stream) as at:
        if out is None or workspace is None:
            with at.allocating():
                out = torch.empty_like(q) if out is None else out
                if workspace is None:
                    workspace = alloc_full_workspace(num_seqs, rows_per_seq, num_q_heads, q.device)
        _need_on(out, torch.bfloat16, "out", i)
        _need_on(workspace, torch.uint8, "workspace", i)
        if out.numel() != q.numel():
            raise ValueError("out [R, num_q_heads, 512]")
        check(_lib.load().dsa_mla_decode_full(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), max_blocks_per_seq,
            seq_lens.data_ptr(), num_seqs, rows_per_seq, num_q_heads, block_size, cache_stride_bytes, k_scale, v_scale,
            sm_scale, out.data_ptr(), verify_rows, workspace.data_ptr(), workspace.numel(), at.raw), "dsa_mla_decode_full")
    return out


def read_device_status(workspace: torch.Tensor, stream=None) -> int:
    v = _lib.ctypes.c_int32(0)
    check(_lib.load().dsa_read_device_status(_ptr(workspace), _lib.ctypes.byref(v), _stream(stream)),
          "dsa_read_device_status")
    return int(v.value)


def last_device_status(stream=None) -> int:
    v = _lib.ctypes.c_int32(0)
    check(_lib.load().dsa_last_device_status(_lib.ctypes.byref(v), _stream(stream)), "dsa_last_device_status")
    return int(v.value)


def step_device_status(stream=None) -> int:
    """First device status of pool_scores calls without a device_status and of decode_full calls on
    the current device since this was last called; clears it."""
    v = _lib.ctypes.c_int32(0)
    check(_lib.load().dsa_step_device_status(_lib.ctypes.byref(v), _stream(stream)), "dsa_step_device_status")
    return int(v.value)


def static_device_status(stream=None) -> int:
    """Device status word of the latest dsa_mla_decode_static call on the current device."""
    v = _lib.ctypes.c_int32(0)
    check(_lib.load().dsa_static_device_status(_lib.ctypes.byref(v), _stream(stream)), "dsa_static_device_status")
    return int(v.value)


# ----------------------------------------------------------------------------------------
# Workload conveniences (a workloads.Workload holds the tensors and the scalars).
# ----------------------------------------------------------------------------------------

def _workload_args(w):
    vc = w.k_cache if w.v_cache is None else w.v_cache
    return (w.q, w.k_cache, vc, w.block_tables, w.max_blocks_per_seq)


def decode_workload(w, out=None, workspace=None, num_ctas=0, verify=None, stream=None, ev_begin=None,
                    ev_end=None, tile_tokens=0, wait_limit_ns=0, gather_mode=0) -> torch.Tensor:
    """Run the decode on a Workload. verify=True uses the k-row entry point with the
    workload's per-sequence base lengths. Per-call options (num_ctas, tile_tokens,
    wait_limit_ns, gather_mode, events) go through dsa_mla_decode_ws; without a workspace one is
    allocated for the call."""
    q, kc, vc, bt, mbps = _workload_args(w)
    out = torch.empty_like(q) if out is None else out
    verify = (w.base_lens is not None) if verify is None else verify
    lens = w.base_lens if verify else w.seq_lens
    if workspace is None and (num_ctas or tile_tokens or wait_limit_ns or gather_mode or ev_begin is not None):
        workspace = alloc_workspace(w.num_seqs, w.rows_per_seq, w.num_q_heads, w.sel_width, num_ctas,
                                    device=q.device)
    if workspace is None:
        fn = decode_k if verify else decode
        return fn(q, kc, vc, bt, mbps, lens, w.sel_indices, w.num_seqs, w.rows_per_seq, w.num_q_heads,
                  w.block_size, w.cache_stride_bytes, w.k_scale, w.v_scale, w.sm_scale, out=out, stream=stream)
    return decode_ws(q, kc, vc, bt, mbps, lens, w.sel_indices, w.num_seqs, w.rows_per_seq, w.num_q_heads,
                     w.block_size, w.cache_stride_bytes, w.k_scale, w.v_scale, w.sm_scale, out, workspace,
                     verify_rows=1 if verify else 0, num_ctas=num_ctas, ev_begin=ev_begin, ev_end=ev_end,
                     tile_tokens=tile_tokens, wait_limit_ns=wait_limit_ns, gather_mode=gather_mode,
                     stream=stream)
