"""Python binding of the DFlash 2 draft-block head (argument marshalling only).

Every function has the name of the C entry point it calls (without the
``dflash2_`` prefix) and runs entirely in the CUDA library: torch tensors only
supply device memory and the current stream.  The arguments of the cache operators, and of
rope, logits_adjust and token_counts, are checked and passed on by the compiled module _dflash2_bind.  bf16 tensors may be given as
torch.bfloat16 or as int16/uint16 bit patterns.  Outputs that are not passed in
are allocated with torch before the call (the library itself never allocates).
"""
import ctypes
from functools import cached_property

import torch

from . import _lib

K = 16
EMBED = 256

STATUS = {0: "OK", -1: "INVALID_ARG", -2: "UNSUPPORTED", -3: "MISALIGNED", -4: "CUDA",
          -5: "TIMEOUT", -6: "DEVICE", -7: "WORKSPACE"}
DEVERR_BAD_TOKEN = 0x1
DEVERR_TIMEOUT = 0x2
DEVERR_BAD_SLOT = 0x4
DEVERR_BAD_PAGE = 0x8
DEVERR_BAD_LENGTH = 0x10
DEVERR_BAD_NODE = 0x20


class Dflash2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.load().dflash2_status_string(status).decode()
        super().__init__(f"{where}: {STATUS.get(status, status)} ({msg})")


def _check(status: int, where: str):
    if status != 0:
        raise Dflash2Error(status, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _is16(t):
    return t.dtype in (torch.bfloat16, torch.int16, torch.uint16)


def _need(cond, what):
    if not cond:
        raise ValueError(what)


class Handle:
    """Owns a dflash2_handle (device error word) bound to one CUDA device."""

    def __init__(self, device: int = None):
        self._lib = _lib.load()
        if device is None:
            device = torch.cuda.current_device()
        self.device = device
        h = ctypes.c_void_p()
        _check(self._lib.dflash2_create(device, ctypes.byref(h)), "dflash2_create")
        self._h = h
        self.raw = h.value

    @cached_property
    def _bind(self):
        """The compiled half of the binding, loaded by the handle's first cache operator: the others do without it."""
        return _lib.load_bind()

    @property
    def ptr(self):
        return self._h

    @property
    def num_sms(self) -> int:
        return int(self._lib.dflash2_num_sms(self._h))

    def device_error(self, stream=None, clear: bool = True) -> int:
        bits = ctypes.c_uint32(0)
        _check(self._lib.dflash2_get_device_error(self._h, _stream(stream), ctypes.byref(bits),
                                                  1 if clear else 0), "dflash2_get_device_error")
        return int(bits.value)

    def close(self):
        if self._h is not None and self._h.value:
            _check(self._lib.dflash2_destroy(self._h), "dflash2_destroy")
        self._h = None
        self.raw = 0

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def topk(h: Handle, logits, V: int = None, vals=None, idx=None, k: int = K, stream=None):
    """logits [rows, ld] bf16 -> (vals fp32 [rows, 16], idx int32 [rows, 16])."""
    _need(_is16(logits) and logits.dim() == 2 and logits.stride(1) == 1, "logits: 2-D bf16, unit stride")
    rows, ld = logits.shape[0], logits.stride(0)
    V = logits.shape[1] if V is None else V
    dev = logits.device
    vals = torch.empty((rows, k), dtype=torch.float32, device=dev) if vals is None else vals
    idx = torch.empty((rows, k), dtype=torch.int32, device=dev) if idx is None else idx
    _check(h._lib.dflash2_topk(h.ptr, _ptr(logits), rows, V, ld, k, _ptr(vals), _ptr(idx),
                               _stream(stream)), "dflash2_topk")
    return vals, idx


def pair_scores_workspace(h: Handle, B: int, L: int, d: int) -> int:
    return int(h._lib.dflash2_pair_scores_workspace(h.ptr, B, L, d))


def pair_scores(h: Handle, cand_idx, cand_val, last_verified, hs, W_H, b_H, A, Bt, V: int = None,
                gate=None, S=None, workspace=None, stream=None):
    """-> (S fp32 [B, L, 16, 16], gate fp32 [B, L, 256]).

    workspace: device bytes (uint8 tensor) of at least pair_scores_workspace(h, B, L, d);
    allocated here by torch when None."""
    B, L, k = cand_idx.shape
    _need(k == K, "cand_idx: [B, L, 16]")
    d = hs.shape[-1]
    V = A.shape[0] if V is None else V
    dev = cand_idx.device
    for name, t in (("hs", hs), ("W_H", W_H), ("A", A), ("Bt", Bt)):
        _need(_is16(t) and t.is_contiguous(), f"{name}: contiguous bf16")
    gate = torch.empty((B, L, EMBED), dtype=torch.float32, device=dev) if gate is None else gate
    S = torch.empty((B, L, K, K), dtype=torch.float32, device=dev) if S is None else S
    if workspace is None:
        workspace = torch.empty(max(pair_scores_workspace(h, B, L, d), 256), dtype=torch.uint8, device=dev)
    _check(h._lib.dflash2_pair_scores(h.ptr, _ptr(cand_idx), _ptr(cand_val), _ptr(last_verified),
                                      _ptr(hs), _ptr(W_H), _ptr(b_H), _ptr(A), _ptr(Bt), B, L, d, V,
                                      _ptr(gate), _ptr(S), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)),
           "dflash2_pair_scores")
    return S, gate


def walk(h: Handle, S, cand_idx, temperature: float = 0.0, seed: int = 0, offset: int = 0,
         draft_tok=None, draft_slot=None, draft_q=None, want_q: bool = True, stream=None):
    """-> (draft_tok int32 [B, L], draft_slot int32 [B, L], draft_q fp32 [B, L, 16] or None)."""
    B, L = S.shape[0], S.shape[1]
    dev = S.device
    draft_tok = torch.empty((B, L), dtype=torch.int32, device=dev) if draft_tok is None else draft_tok
    draft_slot = torch.empty((B, L), dtype=torch.int32, device=dev) if draft_slot is None else draft_slot
    if draft_q is None and want_q:
        draft_q = torch.empty((B, L, K), dtype=torch.float32, device=dev)
    _check(h._lib.dflash2_walk(h.ptr, _ptr(S), _ptr(cand_idx), B, L, float(temperature), seed, offset,
                               _ptr(draft_tok), _ptr(draft_slot), _ptr(draft_q), _stream(stream)),
           "dflash2_walk")
    return draft_tok, draft_slot, draft_q


def walk_viterbi(h: Handle, S, cand_idx, draft_tok=None, draft_slot=None, score=None, want_score: bool = True,
                 stream=None):
    """Exact best path -> (draft_tok int32 [B, L], draft_slot int32 [B, L], score fp32 [B] or None)."""
    B, L = S.shape[0], S.shape[1]
    dev = S.device
    draft_tok = torch.empty((B, L), dtype=torch.int32, device=dev) if draft_tok is None else draft_tok
    draft_slot = torch.empty((B, L), dtype=torch.int32, device=dev) if draft_slot is None else draft_slot
    if score is None and want_score:
        score = torch.empty((B,), dtype=torch.float32, device=dev)
    _check(h._lib.dflash2_walk_viterbi(h.ptr, _ptr(S), _ptr(cand_idx), B, L, _ptr(draft_tok), _ptr(draft_slot),
                                       _ptr(score), _stream(stream)),
           "dflash2_walk_viterbi")
    return draft_tok, draft_slot, score


def selector_eval(h: Handle, gt, cand_idx, accept1=None, accept16=None, counts=None, stream=None):
    """Table 1 evaluation -> (accept1 int32 [B], accept16 int32 [B], counts int64 [L, 4])."""
    B, L = gt.shape
    dev = gt.device
    accept1 = torch.empty((B,), dtype=torch.int32, device=dev) if accept1 is None else accept1
    accept16 = torch.empty((B,), dtype=torch.int32, device=dev) if accept16 is None else accept16
    counts = torch.empty((L, 4), dtype=torch.int64, device=dev) if counts is None else counts
    _check(h._lib.dflash2_selector_eval(h.ptr, _ptr(gt), _ptr(cand_idx), B, L, _ptr(accept1), _ptr(accept16),
                                        _ptr(counts), _stream(stream)),
           "dflash2_selector_eval")
    return accept1, accept16, counts


def conv2tap_workspace(h: Handle, B: int, L: int, d: int) -> int:
    return int(h._lib.dflash2_conv2tap_workspace(h.ptr, B, L, d))


def conv2tap(h: Handle, x, x_prev, k0, k1, W_c, b_c=None, hs=None, y=None, y_fp32: bool = False,
             workspace=None, stream=None):
    """x [B, L, d] bf16 -> y [B, L, d] (bf16, or fp32 when y_fp32).

    workspace: device bytes (uint8 tensor) of at least conv2tap_workspace(h, B, L, d);
    allocated here by torch when None."""
    B, L, d = x.shape
    dev = x.device
    if y is None:
        y = torch.empty((B, L, d), dtype=torch.float32 if y_fp32 else torch.bfloat16, device=dev)
    y_is_fp32 = 1 if y.dtype == torch.float32 else 0
    if workspace is None:
        workspace = torch.empty(max(conv2tap_workspace(h, B, L, d), 256), dtype=torch.uint8, device=dev)
    _check(h._lib.dflash2_conv2tap(h.ptr, _ptr(x), _ptr(x_prev), _ptr(hs), _ptr(k0), _ptr(k1), _ptr(W_c),
                                   _ptr(b_c), B, L, d, _ptr(y), y_is_fp32, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "dflash2_conv2tap")
    return y


def gemm_conv2tap_workspace(h: Handle, B: int, L: int, d: int) -> int:
    return h._lib.dflash2_gemm_conv2tap_workspace(h.ptr, B, L, d)


def gemm_conv2tap(h: Handle, A, W, x_prev, hs, k0, k1, W_c, b_c=None, c_work=None, y=None, y_fp32: bool = False,
                  stream=None):
    """Conv fused into its producing GEMM: A [B, L, K] bf16, W [d, K] bf16 -> (y [B, L, d], c fp32 [B*L, 2d/16]).

    c_work: workspace of at least gemm_conv2tap_workspace(h, B, L, d) bytes (the correction, then
    per-row-tile counters); allocated when None."""
    B, L, Kd = A.shape
    d = W.shape[0]
    dev = A.device
    for name, t in (("A", A), ("W", W), ("x_prev", x_prev), ("hs", hs), ("W_c", W_c)):
        _need(_is16(t) and t.is_contiguous(), f"{name}: contiguous bf16")
    if c_work is None:
        c_work = torch.empty(((gemm_conv2tap_workspace(h, B, L, d) + 3) // 4,), dtype=torch.float32, device=dev)
    if y is None:
        y = torch.empty((B, L, d), dtype=torch.float32 if y_fp32 else torch.bfloat16, device=dev)
    y_is_fp32 = 1 if y.dtype == torch.float32 else 0
    _check(h._lib.dflash2_gemm_conv2tap(h.ptr, _ptr(A), _ptr(W), _ptr(x_prev), _ptr(hs), _ptr(k0), _ptr(k1),
                                        _ptr(W_c), _ptr(b_c), B, L, Kd, d, _ptr(c_work),
                                        c_work.numel() * c_work.element_size(), _ptr(y), y_is_fp32, _stream(stream)),
           "dflash2_gemm_conv2tap")
    n = 2 * (d // 16)
    return y, c_work.view(-1)[: B * L * n].view(B * L, n)


def verify_workspace(h: Handle, B: int, L: int, V: int) -> int:
    return int(h._lib.dflash2_verify_workspace(h.ptr, B, L, V))


def verify(h: Handle, target, draft_tok, draft_slot=None, draft_q=None, cand_idx=None,
           temperature: float = 0.0, seed: int = 0, offset: int = 0, V: int = None,
           accept_len=None, out_tok=None, workspace=None, stream=None):
    """target [B, L+1, V(ld)] bf16 -> (accept_len int32 [B], out_tok int32 [B, L+1]).

    workspace: device bytes (uint8 tensor) of at least verify_workspace(h, B, L, V);
    allocated here by torch when None."""
    B, L1 = target.shape[0], target.shape[1]
    ld = target.stride(1)
    V = target.shape[2] if V is None else V
    dev = target.device
    accept_len = torch.empty((B,), dtype=torch.int32, device=dev) if accept_len is None else accept_len
    out_tok = torch.empty((B, L1), dtype=torch.int32, device=dev) if out_tok is None else out_tok
    if workspace is None:
        workspace = torch.empty(max(verify_workspace(h, B, L1 - 1, V), 256), dtype=torch.uint8, device=dev)
    _check(h._lib.dflash2_verify(h.ptr, _ptr(target), ld, _ptr(draft_tok), _ptr(draft_slot), _ptr(draft_q),
                                 _ptr(cand_idx), B, L1 - 1, V, float(temperature), seed, offset,
                                 _ptr(accept_len), _ptr(out_tok), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)), "dflash2_verify")
    return accept_len, out_tok


def lmhead_topk_workspace(h: Handle, M: int, V: int, d: int) -> int:
    return int(h._lib.dflash2_lmhead_topk_workspace(h.ptr, M, V, d))


def lmhead_topk(h: Handle, hidden, W, vals=None, idx=None, workspace=None, stream=None):
    """hidden [M, d] bf16, W [V, d] bf16 -> (vals fp32 [M, 16], idx int32 [M, 16])."""
    M, d = hidden.shape
    V = W.shape[0]
    dev = hidden.device
    vals = torch.empty((M, K), dtype=torch.float32, device=dev) if vals is None else vals
    idx = torch.empty((M, K), dtype=torch.int32, device=dev) if idx is None else idx
    need = lmhead_topk_workspace(h, M, V, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _check(h._lib.dflash2_lmhead_topk(h.ptr, _ptr(hidden), _ptr(W), M, V, d, _ptr(vals), _ptr(idx),
                                      _ptr(workspace), workspace.numel(), _stream(stream)),
           "dflash2_lmhead_topk")
    return vals, idx


def lmhead_topk_gate(h: Handle, hidden, W, W_H, b_H=None, vals=None, idx=None, gate=None, workspace=None,
                     stream=None):
    """Fused LM head + top-16 + context gate -> (vals fp32 [M, 16], idx int32 [M, 16], gate fp32 [M, 256])."""
    for name, t in (("hidden", hidden), ("W", W), ("W_H", W_H)):
        _need(_is16(t) and t.is_contiguous(), f"{name}: contiguous bf16")
    M, d = hidden.shape
    V = W.shape[0]
    dev = hidden.device
    vals = torch.empty((M, K), dtype=torch.float32, device=dev) if vals is None else vals
    idx = torch.empty((M, K), dtype=torch.int32, device=dev) if idx is None else idx
    gate = torch.empty((M, EMBED), dtype=torch.float32, device=dev) if gate is None else gate
    if workspace is None:
        workspace = torch.empty(max(lmhead_topk_workspace(h, M, V, d), 256), dtype=torch.uint8, device=dev)
    _check(h._lib.dflash2_lmhead_topk_gate(h.ptr, _ptr(hidden), _ptr(W), _ptr(W_H), _ptr(b_H), M, V, d, _ptr(vals),
                                           _ptr(idx), _ptr(gate), _ptr(workspace), workspace.numel(),
                                           _stream(stream)), "dflash2_lmhead_topk_gate")
    return vals, idx, gate


def pair_scores_proj_workspace(h: Handle, B: int, L: int) -> int:
    return h._lib.dflash2_pair_scores_proj_workspace(h.ptr, B, L)


def pair_scores_proj(h: Handle, cand_idx, cand_val, last_verified, gate, E, W_A, W_B, P=None, S=None, stream=None):
    """Projection-form pair scores -> (S fp32 [B, L, 16, 16], P fp32 [B*L*16 + B, 512])."""
    B, L, k = cand_idx.shape
    _need(k == K, "cand_idx: [B, L, 16]")
    for name, t in (("E", E), ("W_A", W_A), ("W_B", W_B)):
        _need(_is16(t) and t.is_contiguous(), f"{name}: contiguous bf16")
    V, d = E.shape
    dev = cand_idx.device
    if P is None:
        P = torch.empty((B * L * K + B, 2 * EMBED), dtype=torch.float32, device=dev)
    S = torch.empty((B, L, K, K), dtype=torch.float32, device=dev) if S is None else S
    _check(h._lib.dflash2_pair_scores_proj(h.ptr, _ptr(cand_idx), _ptr(cand_val), _ptr(last_verified), _ptr(gate),
                                           _ptr(E), _ptr(W_A), _ptr(W_B), B, L, d, V, _ptr(P),
                                           P.numel() * P.element_size(), _ptr(S), _stream(stream)),
           "dflash2_pair_scores_proj")
    return S, P


def lmhead_topk_noalloc(h: Handle, hidden, W, vals=None, idx=None, stream=None):
    """lmhead_topk for callers that cannot allocate: the library's fixed
    device scratch replaces the workspace (calls sharing a device must not
    overlap on the GPU).  Outputs not passed in are allocated here, by torch."""
    M, d = hidden.shape
    V = W.shape[0]
    dev = hidden.device
    vals = torch.empty((M, K), dtype=torch.float32, device=dev) if vals is None else vals
    idx = torch.empty((M, K), dtype=torch.int32, device=dev) if idx is None else idx
    _check(h._lib.dflash2_lmhead_topk_noalloc(h.ptr, _ptr(hidden), _ptr(W), M, V, d, _ptr(vals), _ptr(idx),
                                              _stream(stream)), "dflash2_lmhead_topk_noalloc")
    return vals, idx


class KVCache:
    """A cache of keys and values in pages (the C struct dflash2_kv_cache, built once and passed to many calls).

    k, v: bf16 [num_pages, page_size, kv_heads, head_dim] with equal strides, head_dim (64 or 128)
    contiguous; a head-major pool [num_pages, kv_heads, page_size, head_dim] is passed as
    ``pool.transpose(1, 2)``.  block_table: int32 [B, max_pages], position j of sequence b is in page
    ``block_table[b, j // page_size]``; None: page b is the whole of sequence b."""

    def __init__(self, k, v, block_table=None):
        _need(_is16(k) and _is16(v) and k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride() and
              (k.stride(3) == 1 or k.shape[3] == 1), "k, v: bf16 [pages, page_size, heads, dim], equal strides, "
              "unit stride along dim")
        self.k, self.v, self.block_table = k, v, block_table
        pages, page, heads, dim = k.shape
        s = self.struct = _lib.KvCacheStruct()
        s.k, s.v = _ptr(k), _ptr(v)
        s.num_pages, s.page_size, s.heads, s.head_dim = pages, page, heads, dim
        s.page_stride, s.token_stride, s.head_stride = k.stride()[:3]
        if block_table is not None:
            _need(block_table.dtype == torch.int32 and block_table.dim() == 2 and
                  (block_table.stride(1) == 1 or block_table.shape[1] <= 1), "block_table: int32 [B, max_pages]")
            s.block_table = _ptr(block_table)
            s.max_pages, s.table_ld = block_table.shape[1], block_table.stride(0)
        else:
            s.max_pages = 1
        self.batch = pages if block_table is None else block_table.shape[0]
        self.capacity = page * s.max_pages
        self.heads, self.dim = heads, dim
        self.addr = ctypes.addressof(s)



def _raw_stream(h, stream):
    """The stream's handle; None: the current stream of the handle's device (which has to be the current one)."""
    return torch._C._cuda_getCurrentRawStream(h.device) if stream is None else stream.cuda_stream


def _new_on(stream, shape, dtype, dev):
    """A tensor of the allocator's pool for the call's stream (so that its memory, once freed, is not handed to
    another stream while the call still runs)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def tree_attention_workspace(h: Handle, B: int, T: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(h._lib.dflash2_tree_attention_workspace(h.ptr, B, T, heads, kv_heads, head_dim))


def tree_attention(h: Handle, q, cache: KVCache, cache_len, k_new=None, v_new=None, tree_mask=None,
                   scale: float = None, out=None, lse=None, workspace=None, stream=None):
    """Drafted tokens over a cache and over their own chain or tree -> (out bf16 [B, T, heads, dim], lse fp32 [B, T, heads]).

    q [B, T, heads, dim]; k_new, v_new [B, T, kv_heads, dim] (equal strides; None: the cache alone); tree_mask
    int64 [B, T, (T + 63) // 64], bit s % 64 of word s // 64 of node t set where t sees s (None: a chain).
    scale: 1 / sqrt(dim) when None.  workspace: device bytes of at least tree_attention_workspace(...)."""
    if out is None or lse is None or workspace is None:
        _need(q.dim() == 4 and q.is_cuda, "q: CUDA bf16 [B, T, heads, dim]")
        B, T, heads, dim = q.shape
        if out is None:
            out = _new_on(stream, q.shape, torch.bfloat16, q.device)
        if lse is None:
            lse = _new_on(stream, (B, T, heads), torch.float32, q.device)
        if workspace is None:
            workspace = _new_on(stream, (max(tree_attention_workspace(h, B, T, heads, cache.heads, dim), 256),),
                                torch.uint8, q.device)
    status = h._bind.tree_attention(h.raw, cache.addr, cache.batch, q, cache_len, k_new, v_new, tree_mask,
                                    cache.dim ** -0.5 if scale is None else scale, out, lse, workspace,
                                    _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_tree_attention")
    return out, lse


def prefix_attention_workspace(h: Handle, B: int, T: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(h._lib.dflash2_prefix_attention_workspace(h.ptr, B, T, heads, kv_heads, head_dim))


def prefix_attention(h: Handle, q, cache: KVCache, cache_len, prefix_len, prefix_start=None, k_new=None, v_new=None,
                     tree_mask=None, scale: float = None, out=None, lse=None, workspace=None, stream=None):
    """tree_attention for sequences that share their beginnings, which are read and multiplied once for a group ->
    (out bf16 [B, T, heads, dim], lse fp32 [B, T, heads]).

    prefix_len int32 [groups]: how many first positions the sequences prefix_start[g] .. prefix_start[g + 1] - 1 share;
    prefix_start int32 [groups + 1] (None: one group, the whole batch).  The other arguments are tree_attention's;
    workspace: device bytes of at least prefix_attention_workspace(...)."""
    if out is None or lse is None or workspace is None:
        _need(q.dim() == 4 and q.is_cuda, "q: CUDA bf16 [B, T, heads, dim]")
        B, T, heads, dim = q.shape
        if out is None:
            out = _new_on(stream, q.shape, torch.bfloat16, q.device)
        if lse is None:
            lse = _new_on(stream, (B, T, heads), torch.float32, q.device)
        if workspace is None:
            workspace = _new_on(stream, (max(prefix_attention_workspace(h, B, T, heads, cache.heads, dim), 256),),
                                torch.uint8, q.device)
    status = h._bind.prefix_attention(h.raw, h.device, cache.addr, cache.batch, q, cache_len, prefix_len, prefix_start,
                                      k_new, v_new, tree_mask, cache.dim ** -0.5 if scale is None else scale, out, lse,
                                      workspace, _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_prefix_attention")
    return out, lse


def cache_commit(h: Handle, k_new, v_new, cache: KVCache, cache_len, count=None, path=None, scores=None,
                 new_len=None, stream=None):
    """Appends the accepted nodes' keys and values to the cache -> new_len int32 [B].

    k_new, v_new [B, T, kv_heads, dim]; count int32 [B] accepted nodes (None: T); path int32 [B, T] their ids
    (None: 0, 1, ...); scores fp32 [B, kv_heads, ld]: the appended positions' entries become 0."""
    if new_len is None:
        new_len = _new_on(stream, (k_new.shape[0],), torch.int32, k_new.device)
    status = h._bind.cache_commit(h.raw, cache.addr, cache.batch, k_new, v_new, cache_len, count, path, scores, new_len,
                                  _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_cache_commit")
    return new_len


def cache_scores(h: Handle, q, lse, cache: KVCache, cache_len, scores, count=None, path=None, scale: float = None,
                 stream=None):
    """Adds to scores fp32 [B, kv_heads, ld] the attention weight that each cached position received from the
    accepted nodes (q and lse as in tree_attention, count and path as in cache_commit) -> scores."""
    status = h._bind.cache_scores(h.raw, cache.addr, cache.batch, q, lse, cache_len, scores, count, path,
                                  cache.dim ** -0.5 if scale is None else scale, _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_cache_scores")
    return scores


def cache_evict(h: Handle, scores, cache: KVCache, cache_len, dst: KVCache, keep: int, recent: int, kept=None,
                new_len=None, dst_scores=None, want_scores: bool = True, stream=None):
    """Keeps, per head, the last `recent` positions and the highest-scored others, `keep` in all, in dst ->
    (kept int32 [B, kv_heads, keep], new_len int32 [B], dst_scores fp32 [B, kv_heads, keep] or None).

    scores fp32 [B, kv_heads, ld]; dst's pages must be none of the source's."""
    if kept is None or new_len is None or (dst_scores is None and want_scores):
        B, shape = scores.shape[0], (scores.shape[0], cache.heads, max(keep, 0))
        if kept is None:
            kept = _new_on(stream, shape, torch.int32, scores.device)
        if new_len is None:
            new_len = _new_on(stream, (B,), torch.int32, scores.device)
        if dst_scores is None and want_scores:
            dst_scores = _new_on(stream, shape, torch.float32, scores.device)
    status = h._bind.cache_evict(h.raw, cache.addr, cache.batch, dst.addr, dst.batch, scores, cache_len, keep, recent, kept,
                                 new_len, dst_scores, _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_cache_evict")
    return kept, new_len, dst_scores


class Rope:
    """Rotary positions of one model: rates per pair, layout, and the factor of cos and sin.

    rotary_dim: rotated elements of a head, from its first one on.  interleaved: pairs are neighbours, not half the
    rotated part apart.  scaling, for longer contexts than trained on: None, or a dict with "kind" and its numbers:
    "linear" and "ntk": factor; "yarn": factor, original, fast (32), slow (1); "wavelength": factor, original, low, high
    (the formulas stand at dflash2_rope_scaling in include/dflash2.h)."""

    KINDS = {"linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}

    def __init__(self, rotary_dim, theta=10000.0, interleaved=False, scaling=None, device=None):
        s = _lib.RopeScalingStruct()
        if scaling is not None:
            given = dict(scaling)
            kind = given.pop("kind", None)
            _need(kind in self.KINDS, f"scaling: kind is one of {', '.join(self.KINDS)}")
            s.kind = self.KINDS[kind]
            if kind == "yarn":
                s.fast, s.slow = 32.0, 1.0
            takes = {"yarn": ("factor", "original", "fast", "slow"), "wavelength": ("factor", "original", "low", "high")}
            for name, value in given.items():
                _need(name in takes.get(kind, ("factor",)), f"scaling: {kind} takes no {name}")
                setattr(s, name, float(value))
        _need(0 < rotary_dim <= 512, "rotary_dim: 2 .. 512")
        turns = torch.empty(max(rotary_dim // 2, 1), dtype=torch.int64)
        factor = ctypes.c_float()
        _check(_lib.load().dflash2_rope_turns(rotary_dim, float(theta), ctypes.byref(s), ctypes.c_void_p(turns.data_ptr()),
                                              ctypes.byref(factor)), "dflash2_rope_turns")
        self.rotary_dim, self.interleaved, self.factor = rotary_dim, bool(interleaved), factor.value
        self.turns = turns.to(torch.device("cuda", torch.cuda.current_device()) if device is None else device)
        r = self.struct = _lib.RopeTableStruct()
        r.turns, r.rotary_dim, r.interleaved, r.factor = self.turns.data_ptr(), rotary_dim, self.interleaved, self.factor
        self.addr = ctypes.addressof(r)
        self.device = self.turns.device.index


def rope(h: Handle, x, rope: Rope, base=None, depth=None, inverse: bool = False, out=None, stream=None):
    """x [B, T, heads, dim] rotated by its positions base[b] + depth[b, t] -> out, bf16 of the same shape.

    base int32 [B] (None: 0), depth int32 [B, T] (None: t; a tree's nodes have their depths).  out may be x (drafted keys
    rotated in place keep the strides that they have to share with their values).
    inverse: by the negated angles, which is the gradient (and undoes the rotation, but for the scaling's factor)."""
    _need(rope.device == h.device, "rope: expected one on the handle's device")
    if out is None:
        out = _new_on(stream, x.shape, torch.bfloat16, x.device)
    status = h._bind.rope(h.raw, h.device, rope.addr, x, out, base, depth, inverse, _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_rope")
    return out


def cache_append(h: Handle, k_new, v_new, cache: KVCache, cache_len, rope: Rope = None, count=None, position=None, q=None,
                 q_out=None, scores=None, new_len=None, stream=None):
    """Appends new tokens' keys (rotated by `rope`) and values to the cache -> (new_len int32 [B], q_out or None).

    k_new, v_new [B, T, kv_heads, dim]; count int32 [B] tokens of each sequence (None: T); position int32 [B] of its first
    one (None: cache_len); q [B, T, heads, dim]: the tokens' queries, rotated to q_out, which may be q (rows past count are
    left alone; zeros where q_out is allocated here); scores as in cache_commit."""
    _need(rope is None or rope.device == h.device, "rope: expected one on the handle's device")
    if new_len is None:
        new_len = _new_on(stream, (k_new.shape[0],), torch.int32, k_new.device)
    if q is not None and q_out is None:
        q_out = _new_on(stream, q.shape, torch.bfloat16, q.device)
        if count is not None:
            with torch.cuda.stream(stream):
                q_out.zero_()
    status = h._bind.cache_append(h.raw, h.device, cache.addr, cache.batch, k_new, v_new, cache_len,
                                  0 if rope is None else rope.addr, count, position, q, q_out, scores, new_len,
                                  _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_cache_append")
    return new_len, q_out


def logits_adjust(h: Handle, logits, counts=None, tokens=None, tree_mask=None, repetition=None, frequency=None,
                  presence=None, bias=None, allowed=None, out=None, stream=None):
    """The target's logits [B, T, V] after a request's penalties, biases and allowed tokens -> out, bf16 [B, T, V].

    counts int32 [B, V] as token_counts keeps them; tokens int32 [B, T], the nodes' own, of which a node counts those it
    sees (tree_mask as in tree_attention; None: a chain); repetition, frequency, presence fp32 [B]; bias fp32 [B, V] or
    [1, V]; allowed int32 [B or 1, T or 1, (V + 31) // 32], a bit per token.  Rows of logits, out, counts and bias lie a
    multiple of 8 elements apart, which an odd V gets as a slice of a wider tensor.  out may be logits."""
    if out is None:
        _need(logits.dim() == 3, "logits: [B, T, V]")
        B, T, V = logits.shape
        out = _new_on(stream, (B, T, (V + 7) // 8 * 8), torch.bfloat16, logits.device)[..., :V]
    status = h._bind.logits_adjust(h.raw, h.device, logits, counts, tokens, tree_mask, repetition, frequency, presence,
                                   bias, allowed, out, _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_logits_adjust")
    return out


def token_counts(h: Handle, tokens, counts, count=None, path=None, prompt: bool = False, stream=None):
    """Adds tokens int32 [B, N] to counts int32 [B, V] -> counts: bits 0-30 how often each was emitted, or, with prompt,
    bit 31 (the sign): it occurs in the prompt.

    count int32 [B] (None: N) and path int32 [B, N] (None: 0, 1, ...) choose tokens as in cache_commit."""
    status = h._bind.token_counts(h.raw, h.device, tokens, counts, count, path, prompt, _raw_stream(h, stream))
    if status:
        _check(status, "dflash2_token_counts")
    return counts


def selftest_wait_timeout(h: Handle, limit_ns: int, words=None, stream=None):
    """Runs the library's bounded-wait self-test: one kernel whose two waits
    cannot be satisfied gives up after limit_ns each.  Returns the result word
    (bit 2 = the kernel reached its end; bits 0/1 = a wait was satisfied)."""
    if words is None:
        words = torch.zeros(2, dtype=torch.int32, device=torch.device("cuda", h.device))
    _check(h._lib.dflash2_selftest_wait_timeout(h.ptr, int(limit_ns), _ptr(words), _stream(stream)),
           "dflash2_selftest_wait_timeout")
    return words
