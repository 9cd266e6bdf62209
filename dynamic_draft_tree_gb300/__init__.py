"""GB300 dynamic draft-tree hot path: Python binding of the libdt C ABI.

Every function here has the name of the C entry point it calls and only
marshals arguments (torch CUDA tensors -> device pointers, the current CUDA
stream); all work runs in libdt's sm_103a kernels. See include/dt.h for the
semantics, layouts and error behaviour of each call.
"""
import ctypes
import struct

import torch

from ._lib import (lib, check, DtError, DtConfig, DtTreeView, DtPruneParams, DtPruneOut, DtTemplate,  # noqa
                   DtTreeMeta, EXPORTS, DT_OK, DT_ERR_ARG, DT_ERR_CUDA, DT_ERR_DEVICE,
                   DT_ERR_DEVICE_TIMEOUT, DT_BF16, DT_F32, DT_GREEDY, DT_SAMPLE, DT_VERIFY_PACKED,
                   DT_POLICY_CAST_WIDTH_DEPTH, DT_POLICY_CAST_VERIFY, DT_POLICY_GRAFT_CHECKPOINT, DT_POLICY_NONE,
                   DT_DEV_BAD_LOGITS, DT_DEV_BAD_TOKEN, DT_DEV_BAD_TREE, DT_DEV_TIMEOUT, DT_DEV_INTERNAL, DT_DEV_KV_FULL,
                   DT_DEV_BAD_PAGE, DT_SEEN_PROMPT, DT_F16, DtBlockPool, DtKvRows, DtAttnArgs, DtLogitsParams, DtPromptArgs, DtLogprobArgs, DtKvPages,
                   DT_FLAG_TEST_TIMEOUT, DT_FLAG_TEST_ARRIVED, DT_ANCHOR_ROOT, DT_ANCHOR_TAIL, LIB_PATH)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor required")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor required")
    return t.data_ptr()


def _stream(stream=None):
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


class Handle:
    """An open libdt handle (one draft tree in flight) and its configuration."""

    def __init__(self, B_max, V, K, W, D_max, P_max, dtype=DT_BF16, flags=0):
        self.cfg = DtConfig(B_max, V, K, W, D_max, P_max, dtype, flags)
        self.h = ctypes.c_void_p()
        check(lib.dt_create(ctypes.byref(self.cfg), ctypes.byref(self.h)))

    def close(self):
        if self.h:
            check(lib.dt_destroy(self.h))
            self.h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _DevArray:
    """Zero-copy view of a library-owned device array, for torch.as_tensor."""

    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (ptr, False), "version": 3, "strides": None}


def dt_create(B_max, V, K, W, D_max, P_max, dtype=DT_BF16, flags=0):
    return Handle(B_max, V, K, W, D_max, P_max, dtype, flags)


def dt_destroy(h):
    h.close()


def dt_get_tree(h):
    """The tree arrays as torch tensors viewing the handle's workspace (valid until the next call)."""
    v = DtTreeView()
    check(lib.dt_get_tree(h.h, ctypes.byref(v)))
    Bm, N, D, LW, W = h.cfg.B_max, v.N, v.D_max, v.LW, v.W

    def view(ptr, shape, ts):
        return torch.as_tensor(_DevArray(ptr, shape, ts), device="cuda")

    return dict(B=v.B, K=v.K, W=W, D_max=D, N=N, LW=LW, depth=v.depth,
                token=view(v.token, (Bm, N), "<i4"), parent=view(v.parent, (Bm, N), "<i4"),
                node_depth=view(v.node_depth, (Bm, N), "<i4"), logc=view(v.logc, (Bm, N), "<f4"),
                value=view(v.value, (Bm, N), "<f4"),
                layer_order=view(v.layer_order, (Bm, D + 1, LW), "<i4"),
                layer_count=view(v.layer_count, (Bm, D + 1), "<i4"),
                frontier=view(v.frontier, (Bm, W), "<i4"),
                frontier_count=view(v.frontier_count, (Bm,), "<i4"))


def dt_get_status(h, stream=None):
    """Synchronises the stream; returns the device status bits (0 = clean)."""
    bits = ctypes.c_int32(0)
    rc = lib.dt_get_status(h.h, _stream(stream), ctypes.byref(bits))
    if rc not in (DT_OK, DT_ERR_DEVICE, DT_ERR_DEVICE_TIMEOUT):
        check(rc)
    return bits.value


def dt_clear_status(h, stream=None):
    check(lib.dt_clear_status(h.h, _stream(stream)))


def dt_tree_reset(h, root_token, stream=None):
    check(lib.dt_tree_reset(h.h, root_token.numel(), _ptr(root_token), _stream(stream)))


def dt_select_frontier(h, width=None, stop=None, frontier_token=None, stream=None):
    wl = 0 if width is None else width.numel()
    check(lib.dt_select_frontier(h.h, _ptr(width), wl, _ptr(stop), _ptr(frontier_token), _stream(stream)))


def dt_expand_layer(h, logits, F, ld=None, stream=None):
    ld = logits.shape[-1] if ld is None else ld
    check(lib.dt_expand_layer(h.h, _ptr(logits), ld, F, _stream(stream)))


def dt_expand_prune_select(h, logits, F, policy, params=None, out=None, width=None, frontier_token=None, ld=None,
                           stream=None):
    """Expansion, then the policy's pruning (DT_POLICY_NONE: none), then the next frontier."""
    ld = logits.shape[-1] if ld is None else ld
    wl = 0 if width is None else width.numel()
    check(lib.dt_expand_prune_select(h.h, _ptr(logits), ld, F, policy,
                                     None if params is None else ctypes.byref(params),
                                     None if out is None else ctypes.byref(out), _ptr(width), wl,
                                     _ptr(frontier_token), _stream(stream)))


def dt_cast_prune(h, policy, params, out, stream=None):
    check(lib.dt_cast_prune(h.h, policy, ctypes.byref(params), ctypes.byref(out), _stream(stream)))


def dt_cast_prune_select(h, params, out, frontier_token=None, stream=None):
    """CAST width/depth pruning of the newest layer, then the next layer's frontier, in one launch."""
    check(lib.dt_cast_prune_select(h.h, ctypes.byref(params), ctypes.byref(out), _ptr(frontier_token),
                                   _stream(stream)))


def dt_cast_verify_rerank(h, params, out, selected, stream=None):
    """CAST verify count, then the rerank to that count (selected [B][m_cap]), in two launches."""
    check(lib.dt_cast_verify_rerank(h.h, ctypes.byref(params), ctypes.byref(out), _ptr(selected),
                                    _stream(stream)))


def dt_rerank(h, m, m_cap, selected, stream=None):
    ml = 0 if m is None else m.numel()
    check(lib.dt_rerank(h.h, _ptr(m), ml, m_cap, _ptr(selected), _stream(stream)))


def dt_graft_retrieve(h, M, template, R_cap, ret_token, ret_parent, ret_count, selected=None, m_cap=0,
                      ret_anchor=None, stream=None):
    """Retrieval envelope from M; a tail-anchored template needs ``selected`` / ``m_cap``."""
    check(lib.dt_graft_retrieve(h.h, _ptr(M), ctypes.byref(template.c), R_cap, _ptr(selected), m_cap,
                                _ptr(ret_token), _ptr(ret_parent), _ptr(ret_count), _ptr(ret_anchor),
                                _stream(stream)))


def dt_build_tree_meta(h, selected, m_cap, meta, pos_offset=None, ret_token=None, ret_parent=None,
                       ret_count=None, R_cap=0, ret_anchor=None, K_total=0, stream=None):
    check(lib.dt_build_tree_meta(h.h, _ptr(selected), m_cap, _ptr(ret_token), _ptr(ret_parent),
                                 _ptr(ret_count), _ptr(ret_anchor), R_cap, K_total, _ptr(pos_offset),
                                 ctypes.byref(meta.c), _stream(stream)))


def dt_expand_layer_sampled(h, logits, F, seed, round_, ld=None, stream=None):
    """dt_expand_layer with the children drawn from softmax(row) without replacement (Philox draws)."""
    ld = logits.shape[-1] if ld is None else ld
    check(lib.dt_expand_layer_sampled(h.h, _ptr(logits), ld, F, seed, round_, _stream(stream)))


def dt_verify_sampled(h, meta, logits, draft_rows, seed, round_, accept_len, accept_path, bonus, packed=False,
                      ld=None, ld_d=None, stream=None):
    """Verify of sampled drafts: draft_rows is the [D_max][B][W][V] buffer the layers were drawn from."""
    ld = logits.shape[-1] if ld is None else ld
    ld_d = draft_rows.shape[-1] if ld_d is None else ld_d
    check(lib.dt_verify_sampled(h.h, ctypes.byref(meta.c), _ptr(logits), ld, DT_VERIFY_PACKED if packed else 0,
                                _ptr(draft_rows), ld_d, seed, round_, _ptr(accept_len), _ptr(accept_path),
                                _ptr(bonus), _stream(stream)))


def dt_block_expand(h, logits, L, params=None, out=None, ld=None, stream=None):
    """Draft layers 1..L from a block drafter's rows [B][L][V] (one call; Graft gates with params)."""
    ld = logits.shape[-1] if ld is None else ld
    check(lib.dt_block_expand(h.h, _ptr(logits), ld, L, None if params is None else ctypes.byref(params),
                              None if out is None else ctypes.byref(out), _stream(stream)))


def dt_verify(h, meta, logits, mode, seed, round_, accept_len, accept_path, bonus, top8=None, ld=None,
              stream=None):
    ld = logits.shape[-1] if ld is None else ld
    check(lib.dt_verify(h.h, ctypes.byref(meta.c), _ptr(logits), ld, mode, seed, round_, _ptr(accept_len),
                        _ptr(accept_path), _ptr(bonus), _ptr(top8), _stream(stream)))


def dt_verify_rows(h, meta, logits, mode, with_top8=False, ld=None, stream=None):
    """Streaming half of dt_verify (one read of every used target row)."""
    ld = logits.shape[-1] if ld is None else ld
    check(lib.dt_verify_rows(h.h, ctypes.byref(meta.c), _ptr(logits), ld, mode, 1 if with_top8 else 0,
                             _stream(stream)))


def dt_verify_accept(h, meta, logits, mode, seed, round_, accept_len, accept_path, bonus, top8=None, ld=None,
                     stream=None):
    """Acceptance half of dt_verify (after dt_verify_rows)."""
    ld = logits.shape[-1] if ld is None else ld
    check(lib.dt_verify_accept(h.h, ctypes.byref(meta.c), _ptr(logits), ld, mode, seed, round_, _ptr(accept_len),
                               _ptr(accept_path), _ptr(bonus), _ptr(top8), _stream(stream)))


def dt_adj_update(h, M, meta, top8, stream=None):
    check(lib.dt_adj_update(h.h, _ptr(M), ctypes.byref(meta.c), _ptr(top8), _stream(stream)))


def dt_commit_kv(h, tmp_kv, cache, cache_len, accept_len, accept_path, row_off=None, P=None, stream=None):
    """Append the root's and the accepted positions' KV rows to each request's cache.

    tmp_kv [B][P][...] and cache [B][L_max][...] are device tensors whose trailing dimensions form
    one row (contiguous, a multiple of 16 bytes); cache_len [B] int32 is updated in place. With
    ``row_off`` ([B+1] int32 device, dt_tree_meta.row_off) tmp_kv is packed: [rows][...], the row of
    position i of request b being row_off[b] + i; P (positions per request of the tree) is then
    required."""
    packed = row_off is not None
    lead = 1 if packed else 2
    if tmp_kv.dim() < lead + 1 or cache.dim() < 3:
        raise ValueError("tmp_kv needs [B][positions][row...] ([rows][row...] packed), cache [B][L_max][row...]")
    esz = tmp_kv.element_size()
    row0 = tmp_kv[0] if packed else tmp_kv[0, 0]
    row_bytes = row0.numel() * esz
    if cache[0, 0].numel() * cache.element_size() != row_bytes:
        raise ValueError("tmp_kv and cache rows differ in size")
    if not row0.is_contiguous() or not cache[0, 0].is_contiguous():
        raise ValueError("KV rows must be contiguous")
    for t in (tmp_kv, cache):
        if not t.is_cuda:
            raise ValueError("device tensor required")
    if packed:
        if P is None:
            raise ValueError("P is required with row_off")
        pos_stride, req_stride = tmp_kv.stride(0) * esz, 0
    else:
        P = tmp_kv.shape[1]
        pos_stride, req_stride = tmp_kv.stride(1) * esz, tmp_kv.stride(0) * esz
    check(lib.dt_commit_kv(h.h, tmp_kv.data_ptr(), pos_stride, req_stride, P,
                           cache.data_ptr(), cache.stride(1) * cache.element_size(),
                           cache.stride(0) * cache.element_size(), cache.shape[1], row_bytes, _ptr(cache_len),
                           _ptr(accept_len), _ptr(accept_path), accept_path.shape[-1], _ptr(row_off),
                           _stream(stream)))


def dt_row_topk_static(logits, K, logp, ids, V=None, status=None, stream=None):
    """Row log-softmax top-K with no handle and no allocation: logits [rows][ld] (bf16 or fp32),
    logp [rows][K] fp32 and ids [rows][K] int32 caller-owned; status an int32 device word or None."""
    ld = logits.shape[-1]
    rows = logits.numel() // ld
    V = ld if V is None else V
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("logits must be bfloat16 or float32")
    if logp.dtype != torch.float32 or ids.dtype != torch.int32 or logp.numel() < rows * K or ids.numel() < rows * K:
        raise ValueError("logp must be float32 and ids int32, each with rows*K elements")
    dtype = DT_BF16 if logits.dtype == torch.bfloat16 else DT_F32
    check(lib.dt_row_topk_static(_ptr(logits), ld, rows, V, K, dtype, _ptr(logp), _ptr(ids), _ptr(status),
                                 _stream(stream)))


# The calls below run beside kernels of a few microseconds, so their marshalling is kept short: one look at
# the current device and stream a call, one condition a tensor, the argument struct packed in one go.
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_I32, _I64, _F32, _U8 = torch.int32, torch.int64, torch.float32, torch.uint8


def _packer(struct_type):
    """Packs the fields of a ctypes structure (integers, floats, pointers) with the same layout."""
    codes = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P"}
    s = struct.Struct("@" + "".join(codes[f[1]] for f in struct_type._fields_) + "0P")
    assert s.size == ctypes.sizeof(struct_type)
    return s.pack


_pack_kv_rows, _pack_attn, _pack_logits = _packer(DtKvRows), _packer(DtAttnArgs), _packer(DtLogitsParams)
_pack_prompt, _pack_logprobs, _pack_kv_pages = _packer(DtPromptArgs), _packer(DtLogprobArgs), _packer(DtKvPages)


def _refuse(t, dtype, dev, name, n):
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    if t.numel() < n:
        raise ValueError(f"{name} has fewer than {n} entries")
    raise ValueError(f"{name} must be contiguous")


def _dev(t, dtype, dev, name, n=1):
    """Pointer of a contiguous tensor on device `dev` with this dtype and at least n entries; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or t.numel() < n:
        _refuse(t, dtype, dev, name, n)
    return t.data_ptr()


def _strided(t, dtype, dev, st, name):
    """Pointer of a tensor on device `dev` with this dtype and a contiguous last dimension (st: its strides)."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    if st[-1] != 1:
        raise ValueError(f"{name} needs a contiguous last dimension")
    return t.data_ptr()


class BlockPool:
    """Pages of a KV cache and who owns them (dt_block_pool): device tensors, caller-owned.

    block_table [B][max_blocks], n_owned [B], free_list [n_blocks], free_count [1], all int32."""

    def __init__(self, block_table, n_owned, free_list, free_count, page):
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B][max_blocks]")
        self.B, self.max_blocks = block_table.shape
        self.page, self.n_blocks = page, free_list.numel()
        self.block_table, self.n_owned, self.free_list, self.free_count = block_table, n_owned, free_list, free_count
        self.device = _device()
        self.c = DtBlockPool(page, self.n_blocks, self.max_blocks,
                             _dev(block_table, _I32, self.device, "block_table"),
                             _dev(n_owned, _I32, self.device, "n_owned", self.B),
                             _dev(free_list, _I32, self.device, "free_list"),
                             _dev(free_count, _I32, self.device, "free_count"))
        self.ref = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, B, max_blocks, n_blocks, page, device="cuda"):
        """A pool whose blocks are all free: block 0 is granted first."""
        i32 = dict(dtype=_I32, device=device)
        return cls(torch.full((B, max_blocks), -1, **i32), torch.zeros((B,), **i32),
                   torch.arange(n_blocks - 1, -1, -1, **i32), torch.full((1,), n_blocks, **i32), page)


def _slots_args(B, dev, slots, slot_off, S):
    n_slots = slots.numel()
    if not (slots.dtype is _I64 and slots.get_device() == dev and slots.is_contiguous()):
        _dev(slots, _I64, dev, "slots")
    if slot_off is None:
        sh = slots.shape
        if len(sh) != 2 or sh[0] < B:
            raise ValueError("slots must be [B][S] without slot_off")
        return slots.data_ptr(), n_slots, sh[1], 0
    return slots.data_ptr(), n_slots, n_slots if S is None else S, _dev(slot_off, _I32, dev, "slot_off", B + 1)


def dt_kv_reserve(h, pool, seq_len, n_new, slots, n_extra=0, slot_off=None, S=None, stream=None):
    """Pages and slots (int64, [B][S], or packed by slot_off [B+1] with at most S a request) for the next
    n_new + n_extra tokens of every request."""
    B, dev = n_new.numel(), _device()
    if B > pool.B or pool.device != dev:
        raise ValueError("the pool holds fewer requests than n_new, or is on another device")
    sp, n_slots, S, so = _slots_args(B, dev, slots, slot_off, S)
    if not (seq_len.dtype is _I32 and n_new.dtype is _I32 and seq_len.get_device() == dev and n_new.get_device() == dev
            and seq_len.is_contiguous() and n_new.is_contiguous() and seq_len.numel() >= B):
        _dev(seq_len, _I32, dev, "seq_len", B)
        _dev(n_new, _I32, dev, "n_new")
    rc = lib.dt_kv_reserve(h.h, B, pool.ref, seq_len.data_ptr(), n_new.data_ptr(), n_extra, sp, n_slots, S, so,
                           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


def dt_kv_release(h, pool, keep_len, stream=None):
    """Gives back every request's blocks past keep_len tokens (0: all of them)."""
    B, dev = keep_len.numel(), _device()
    if B > pool.B or pool.device != dev:
        raise ValueError("the pool holds fewer requests than keep_len, or is on another device")
    rc = lib.dt_kv_release(h.h, B, pool.ref, _dev(keep_len, _I32, dev, "keep_len"),
                           _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


def dt_kv_fork(h, pool, refs, cache, src, dst, seq_len, length=None, shared_len=0, stream=None):
    """Requests dst continue requests src (int32, one entry a fork) behind their first ``length`` tokens (default seq_len, which is
    updated): whole pages shared, the last one's tokens copied in cache [planes][blocks][page][H][D], any strides but the
    last dimension's. refs [n_blocks] int32: owners of a block beyond its first, zero at the start."""
    n, dev, cs, sc = src.numel(), _device(), cache.shape, cache.stride()
    if pool.device != dev:
        raise ValueError("the pool is on another device")
    if len(cs) != 5 or cs[1] != pool.n_blocks or cs[2] != pool.page:
        raise ValueError("cache must be [planes][blocks][page][H][D] with the pool's blocks and page")
    if cache.get_device() != dev or sc[4] != 1:
        _strided(cache, cache.dtype, dev, sc, "cache")
    e = cache.element_size()
    kv = _pack_kv_pages(cache.data_ptr(), sc[0] * e, sc[1] * e, sc[2] * e, sc[3] * e, cs[0], cs[3], cs[4] * e)
    rc = lib.dt_kv_fork(h.h, pool.B, pool.ref, _dev(refs, _I32, dev, "refs", pool.n_blocks), kv, n, _dev(src, _I32, dev, "src"),
                        _dev(dst, _I32, dev, "dst", n), 0 if length is None else _dev(length, _I32, dev, "length", n),
                        _dev(seq_len, _I32, dev, "seq_len", pool.B), shared_len,
                        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


def dt_kv_release_shared(h, pool, refs, keep_len, stream=None):
    """Gives back every request's blocks past keep_len tokens (0: all of them) in a pool with forks."""
    B, dev = keep_len.numel(), _device()
    if B > pool.B or pool.device != dev:
        raise ValueError("the pool holds fewer requests than keep_len, or is on another device")
    rc = lib.dt_kv_release_shared(h.h, B, pool.ref, _dev(refs, _I32, dev, "refs", pool.n_blocks),
                                  _dev(keep_len, _I32, dev, "keep_len"), _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


def dt_commit_kv_paged(h, tmp, cache, slots, n_new, seq_len, len_out, path=None, row_off=None, n_extra=0,
                       slot_off=None, S=None, P=None, committed=None, stream=None):
    """KV rows into pages: tmp [planes][B][P][H][D] or, with row_off [B+1], [planes][rows][H][D] (P: positions a
    request, default all rows); cache [planes][blocks][page][H][D], any strides but the last dimension's (pages
    with the heads first are a transposed view); path [B][D_path] as written by dt_verify, or None (rows 0..n-1);
    committed [B] (optional) gets the number of tokens appended, 0 for a refused request."""
    B, dev = n_new.numel(), _device()
    ts, cs, st, sc = tmp.shape, cache.shape, tmp.stride(), cache.stride()
    if len(ts) != (5 if row_off is None else 4) or len(cs) != 5:
        raise ValueError("tmp needs [planes][B][P][H][D] ([planes][rows][H][D] packed), cache [planes][blocks][page][H][D]")
    H, D = ts[-2], ts[-1]
    if H != cs[3] or D != cs[4] or ts[0] != cs[0]:
        raise ValueError("tmp and cache differ in planes, heads or head size")
    if row_off is None:
        P, rows = ts[2], ts[1] * ts[2]
        one = P == 1 and ts[1] > 1  # the requests are the rows (a dimension of one has any stride)
        row = st[1] if one else st[2]
        if ts[1] < B or (ts[1] > 1 and not one and st[1] != P * row):
            raise ValueError("tmp [planes][B][P] needs B requests, P rows apart")
    else:
        rows, row = ts[1], st[1]
        P = rows if P is None else P
    dp = 0
    if path is not None:
        if path.dim() != 2 or path.shape[0] < B:
            raise ValueError("path must be [B][D_path]")
        dp = path.shape[1]
    e, dtype = tmp.element_size(), tmp.dtype
    if not (cache.dtype is dtype and tmp.get_device() == dev and cache.get_device() == dev and st[-1] == 1
            and sc[4] == 1):
        _strided(tmp, dtype, dev, st, "tmp")
        _strided(cache, dtype, dev, sc, "cache")
    if not (n_new.dtype is _I32 and seq_len.dtype is _I32 and len_out.dtype is _I32 and n_new.get_device() == dev
            and seq_len.get_device() == dev and len_out.get_device() == dev and n_new.is_contiguous()
            and seq_len.is_contiguous() and len_out.is_contiguous() and seq_len.numel() >= B and len_out.numel() >= B):
        for t, name in ((n_new, "n_new"), (seq_len, "seq_len"), (len_out, "len_out")):
            _dev(t, _I32, dev, name, B)
    kv = _pack_kv_rows(tmp.data_ptr(), st[0] * e, row * e, st[-2] * e, rows, cache.data_ptr(), sc[0] * e, sc[1] * e,
                       sc[2] * e, sc[3] * e, ts[0], H, D * e, cs[2], cs[1], 0 if committed is None else _dev(committed, _I32, dev, "committed", B))
    sp, n_slots, S, so = _slots_args(B, dev, slots, slot_off, S)
    rc = lib.dt_commit_kv_paged(h.h, B, kv, P, 0 if row_off is None else _dev(row_off, _I32, dev, "row_off", B + 1),
                                0 if path is None else _dev(path, _I32, dev, "path"), dp, n_new.data_ptr(), n_extra, sp,
                                n_slots, S, so, seq_len.data_ptr(), len_out.data_ptr(),
                                _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


def dt_tree_attention_workspace(h, B, P, H_q, H_kv, D, shared=False):
    """A workspace tensor for dt_tree_attention calls of at most these sizes (one call at a time)."""
    n = ctypes.c_int64(0)
    check(lib.dt_tree_attention_workspace(h.h, B, P, H_q, H_kv, D, 1 if shared else 0, ctypes.byref(n)))
    return torch.empty(n.value, dtype=_U8, device="cuda")


_ATTN_TYPES = {torch.bfloat16: DT_BF16, torch.float16: DT_F16}


def dt_tree_attention(h, q, k_new, v_new, k_pages, v_pages, block_table, seq_len, n_pos, out, workspace, mask=None,
                      row_off=None, P=None, shared_len=0, scale=None, stream=None):
    """Tree attention over pages: q and out [B][P][H_q][D], k_new and v_new [B][P][H_kv][D], or packed
    [rows][heads][D] with row_off [B+1] (P: positions a request, default the mask's or all rows); k_pages and
    v_pages [blocks][page][H_kv][D], any strides but the last dimension's; block_table [B][max_blocks]; mask
    [B][P][P] uint8 or None (a chain); scale defaults to D ** -0.5."""
    dtype, dev, B = q.dtype, _device(), n_pos.numel()
    code = _ATTN_TYPES.get(dtype)
    if code is None:
        raise ValueError("q must be bfloat16 or float16")
    qh, nh, ph, th = q.shape, k_new.shape, k_pages.shape, block_table.shape
    qs, os_, ks, vs, kp, vp_ = q.stride(), out.stride(), k_new.stride(), v_new.stride(), k_pages.stride(), v_pages.stride()
    if len(qh) != (4 if row_off is None else 3) or out.shape != qh or len(ph) != 4 or v_pages.shape != ph:
        raise ValueError("q and out need [B][P][H][D] ([rows][H][D] packed), pages [blocks][page][H_kv][D]")
    D = qh[-1]
    if v_new.shape != nh or len(nh) != len(qh) or nh[0] != qh[0] or nh[-3] != qh[-3] or nh[-1] != D or ph[2] != nh[-2] \
            or ph[3] != D:
        raise ValueError("k_new, v_new and the pages must match q's rows and one another's heads and head size")
    if len(th) != 2 or th[0] < B:
        raise ValueError("block_table must be [B][max_blocks]")
    at = -3  # dimension of the rows
    if row_off is None:
        P, rows = qh[1], qh[0] * qh[1]
        if qh[0] < B:
            raise ValueError("q holds fewer requests than n_pos")
        if qh[0] > 1:
            if P == 1:  # the requests are the rows (a dimension of one has any stride)
                at = 0
            elif not (qs[0] == P * qs[1] and os_[0] == P * os_[1] and ks[0] == P * ks[1] and vs[0] == P * vs[1]):
                raise ValueError("padded rows must be P rows apart")
    else:
        rows = qh[0]
        if P is None:
            P = mask.shape[-1] if mask is not None else min(rows, h.cfg.P_max)
    if mask is not None:
        mh = mask.shape
        if len(mh) != 3 or mh[0] < B or mh[1] != P or mh[2] != P:
            raise ValueError("mask must be [B][P][P]")
    if not (out.dtype is dtype and k_new.dtype is dtype and v_new.dtype is dtype and k_pages.dtype is dtype
            and v_pages.dtype is dtype):
        raise ValueError(f"q, k_new, v_new, k_pages, v_pages and out must all be {dtype}")
    if not (q.get_device() == dev and out.get_device() == dev and k_new.get_device() == dev and v_new.get_device() == dev
            and k_pages.get_device() == dev and v_pages.get_device() == dev):
        raise ValueError("q, k_new, v_new, k_pages, v_pages and out must be on the current CUDA device")
    if not (qs[-1] == 1 and os_[-1] == 1 and ks[-1] == 1 and vs[-1] == 1 and kp[3] == 1 and vp_[3] == 1):
        raise ValueError("q, k_new, v_new, k_pages, v_pages and out need a contiguous last dimension")
    if not (block_table.dtype is _I32 and seq_len.dtype is _I32 and n_pos.dtype is _I32 and workspace.dtype is _U8
            and block_table.get_device() == dev and seq_len.get_device() == dev and n_pos.get_device() == dev
            and workspace.get_device() == dev and block_table.is_contiguous() and seq_len.is_contiguous()
            and n_pos.is_contiguous() and workspace.is_contiguous() and seq_len.numel() >= B):
        for t, kind, name, n in ((block_table, _I32, "block_table", B), (seq_len, _I32, "seq_len", B),
                                 (n_pos, _I32, "n_pos", 1), (workspace, _U8, "workspace", 1)):
            _dev(t, kind, dev, name, n)
    a = _pack_attn(B, P, qh[-2], nh[-2], D, code, D ** -0.5 if scale is None else scale, shared_len, rows,
                   q.data_ptr(), qs[at], qs[-2], out.data_ptr(), os_[at], os_[-2], k_new.data_ptr(), v_new.data_ptr(),
                   ks[at], ks[-2], vs[at], vs[-2], k_pages.data_ptr(), v_pages.data_ptr(), kp[0], kp[1], kp[2], vp_[0],
                   vp_[1], vp_[2], ph[0], ph[1], block_table.data_ptr(), th[1], seq_len.data_ptr(), n_pos.data_ptr(),
                   0 if mask is None else _dev(mask, _U8, dev, "mask"),
                   0 if row_off is None else _dev(row_off, _I32, dev, "row_off", B + 1), workspace.data_ptr(),
                   workspace.numel())
    rc = lib.dt_tree_attention(h.h, a, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


def dt_prompt_attention_workspace(h, B, H_q, H_kv, D):
    """A workspace tensor for dt_prompt_attention calls of this head size (one call at a time)."""
    n = ctypes.c_int64(0)
    check(lib.dt_prompt_attention_workspace(h.h, B, H_q, H_kv, D, ctypes.byref(n)))
    return torch.empty(n.value, dtype=_U8, device="cuda")


def dt_prompt_attention(h, q, k_new, v_new, row_off, out, workspace, k_pages=None, v_pages=None, block_table=None,
                        seq_len=None, scale=None, stream=None):
    """Causal attention over packed prompts: q and out [rows][H_q][D], k_new and v_new [rows][H_kv][D], request b's rows
    row_off[b] .. row_off[b + 1] - 1 (row_off [B+1]); behind seq_len[b] cached tokens with k_pages and v_pages
    [blocks][page][H_kv][D], any strides but the last dimension's, block_table [B][max_blocks] and seq_len [B] (all or
    none); scale defaults to D ** -0.5."""
    dtype, dev, B = q.dtype, _device(), row_off.numel() - 1
    code = _ATTN_TYPES.get(dtype)
    if code is None:
        raise ValueError("q must be bfloat16 or float16")
    qh, nh = q.shape, k_new.shape
    qs, os_, ks, vs = q.stride(), out.stride(), k_new.stride(), v_new.stride()
    if len(qh) != 3 or out.shape != qh or len(nh) != 3 or v_new.shape != nh or nh[0] != qh[0] or nh[2] != qh[2]:
        raise ValueError("q and out need [rows][H_q][D], k_new and v_new [rows][H_kv][D]")
    if B < 1:
        raise ValueError("row_off must be [B+1]")
    rows, H, D = qh
    if not (out.dtype is dtype and k_new.dtype is dtype and v_new.dtype is dtype):
        raise ValueError(f"q, k_new, v_new and out must all be {dtype}")
    if not (q.get_device() == dev and out.get_device() == dev and k_new.get_device() == dev and v_new.get_device() == dev):
        raise ValueError("q, k_new, v_new and out must be on the current CUDA device")
    if not (qs[2] == 1 and os_[2] == 1 and ks[2] == 1 and vs[2] == 1):
        raise ValueError("q, k_new, v_new and out need a contiguous last dimension")
    if not (row_off.dtype is _I32 and workspace.dtype is _U8 and row_off.get_device() == dev
            and workspace.get_device() == dev and row_off.is_contiguous() and workspace.is_contiguous()):
        _dev(row_off, _I32, dev, "row_off")
        _dev(workspace, _U8, dev, "workspace")
    pages = (0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    if k_pages is not None or v_pages is not None or block_table is not None or seq_len is not None:
        if k_pages is None or v_pages is None or block_table is None or seq_len is None:
            raise ValueError("k_pages, v_pages, block_table and seq_len come together")
        ph, th, kp, vp_ = k_pages.shape, block_table.shape, k_pages.stride(), v_pages.stride()
        if len(ph) != 4 or v_pages.shape != ph or ph[2] != nh[1] or ph[3] != D:
            raise ValueError("pages must be [blocks][page][H_kv][D] with the heads and the head size of k_new")
        if len(th) != 2 or th[0] < B:
            raise ValueError("block_table must be [B][max_blocks]")
        if not (k_pages.dtype is dtype and v_pages.dtype is dtype and k_pages.get_device() == dev
                and v_pages.get_device() == dev and kp[3] == 1 and vp_[3] == 1):
            _strided(k_pages, dtype, dev, kp, "k_pages")
            _strided(v_pages, dtype, dev, vp_, "v_pages")
        pages = (k_pages.data_ptr(), v_pages.data_ptr(), kp[0], kp[1], kp[2], vp_[0], vp_[1], vp_[2], ph[0], ph[1],
                 _dev(block_table, _I32, dev, "block_table"), th[1], _dev(seq_len, _I32, dev, "seq_len", B))
    a = _pack_prompt(B, H, nh[1], D, code, D ** -0.5 if scale is None else scale, rows, q.data_ptr(), qs[0], qs[1],
                     out.data_ptr(), os_[0], os_[1], k_new.data_ptr(), v_new.data_ptr(), ks[0], ks[1], vs[0], vs[1],
                     row_off.data_ptr(), *pages, workspace.data_ptr(), workspace.numel())
    rc = lib.dt_prompt_attention(h.h, a, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


def dt_count_tokens(h, counts, tokens, n_new, path=None, row_off=None, n_extra=0, prompt=False, P=None, stream=None):
    """Adds tokens ([B][P], or packed by row_off) to the token history counts [B][V] (prompt: marks them)."""
    B, dev = n_new.numel(), _device()
    if counts.dim() != 2 or counts.shape[1] != h.cfg.V or counts.shape[0] < B:
        raise ValueError("counts must be [B][V]")
    if row_off is None:
        if tokens.dim() != 2 or tokens.shape[0] < B:
            raise ValueError("tokens must be [B][P] without row_off")
        P = tokens.shape[1]
    elif P is None:
        P = max(1, tokens.numel())
    if path is not None and (path.dim() != 2 or path.shape[0] < B):
        raise ValueError("path must be [B][D_path]")
    check(lib.dt_count_tokens(h.h, B, _dev(counts, _I32, dev, "counts"), _dev(tokens, _I32, dev, "tokens"), tokens.numel(), P,
                              _dev(row_off, _I32, dev, "row_off", B + 1), _dev(path, _I32, dev, "path"),
                              0 if path is None else path.shape[1], _dev(n_new, _I32, dev, "n_new"), n_extra,
                              1 if prompt else 0, _raw_stream(dev) if stream is None else stream.cuda_stream))


def dt_logits_process(h, logits, out, n_pos, tokens=None, mask=None, row_off=None, counts=None, repetition=None,
                      frequency=None, presence=None, bias_ids=None, bias_vals=None, allow=None, P=None, stream=None):
    """Penalties, biases and grammar masks on target rows: logits and out [B][P][V], or packed [rows][V] with
    row_off (rows may be further apart than V); out may be logits. allow: int32 words, rows as logits."""
    cfg = h.cfg
    dtype = torch.bfloat16 if cfg.dtype == DT_BF16 else _F32
    B, V, dev = n_pos.numel(), cfg.V, _device()
    ls, ls_, os_ = logits.shape, logits.stride(), out.stride()
    if len(ls) != (3 if row_off is None else 2) or out.shape != ls or ls[-1] != V:
        raise ValueError("logits and out need [B][P][V] ([rows][V] packed)")
    at = -2  # dimension of the rows
    if row_off is None:
        P, rows = ls[1], ls[0] * ls[1]
        if ls[0] < B:
            raise ValueError("logits holds fewer requests than n_pos")
        if ls[0] > 1:
            if P == 1:  # the requests are the rows (a dimension of one has any stride)
                at = 0
            elif not (ls_[0] == P * ls_[1] and os_[0] == P * os_[1]):
                raise ValueError("padded rows must be P rows apart")
    else:
        rows = ls[0]
        if P is None:
            P = mask.shape[-1] if mask is not None else tokens.shape[-1] if tokens is not None else min(rows, cfg.P_max)
    if mask is not None:
        mh = mask.shape
        if len(mh) != 3 or mh[0] < B or mh[1] != P or mh[2] != P:
            raise ValueError("mask must be [B][P][P]")
    if tokens is not None:
        th = tokens.shape
        if len(th) != 2 or th[0] < B or th[1] != P:
            raise ValueError("tokens must be [B][P]")
    if counts is not None:
        ch = counts.shape
        if len(ch) != 2 or ch[0] < B or ch[1] != V:
            raise ValueError("counts must be [B][V]")
    n_bias = words = 0
    if bias_ids is not None or bias_vals is not None:
        if bias_ids is None or bias_vals is None or bias_ids.dim() != 2 or bias_ids.shape[0] < B or \
                bias_vals.shape != bias_ids.shape:
            raise ValueError("bias_ids and bias_vals must be [B][n_bias] both")
        n_bias = bias_ids.shape[1]
    if allow is not None:
        words = allow.shape[-1]
        if allow.numel() < rows * words or words < (V + 31) // 32:
            raise ValueError("allow needs a row of ceil(V / 32) words for every row of logits")
    if not (logits.dtype is dtype and out.dtype is dtype and logits.get_device() == dev and out.get_device() == dev
            and ls_[-1] == 1 and os_[-1] == 1):
        _strided(logits, dtype, dev, ls_, "logits")
        _strided(out, dtype, dev, os_, "out")
    p = _pack_logits(P, _dev(n_pos, _I32, dev, "n_pos"), 0 if row_off is None else _dev(row_off, _I32, dev, "row_off", B + 1),
                     rows, 0 if tokens is None else _dev(tokens, _I32, dev, "tokens"),
                     0 if mask is None else _dev(mask, _U8, dev, "mask"),
                     0 if counts is None else _dev(counts, _I32, dev, "counts"),
                     0 if repetition is None else _dev(repetition, _F32, dev, "repetition", B),
                     0 if frequency is None else _dev(frequency, _F32, dev, "frequency", B),
                     0 if presence is None else _dev(presence, _F32, dev, "presence", B),
                     0 if bias_ids is None else _dev(bias_ids, _I32, dev, "bias_ids", 0),
                     0 if bias_vals is None else _dev(bias_vals, _F32, dev, "bias_vals", 0), n_bias,
                     0 if allow is None else _dev(allow, _I32, dev, "allow"), words)
    rc = lib.dt_logits_process(h.h, B, logits.data_ptr(), ls_[at], out.data_ptr(), os_[at], p,
                               _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


def dt_token_logprobs_workspace(h, entries, K=0):
    """A workspace tensor for dt_token_logprobs calls of at most so many entries and alternatives (one call at a time)."""
    n = ctypes.c_int64(0)
    check(lib.dt_token_logprobs_workspace(h.h, entries, K, ctypes.byref(n)))
    return torch.empty(n.value, dtype=_U8, device="cuda")


def dt_token_logprobs(h, logits, n_new, logp, workspace, tokens=None, last=None, shift=1, n_extra=0, path=None, row_off=None,
                      entropy=None, rank=None, top_ids=None, top_logp=None, P=None, stream=None):
    """Log probabilities of tokens under rows of logits: logits [B][P][V], or packed [rows][V] with row_off [B+1] (rows may be
    further apart than V). Outputs (float32, rank and top_ids int32, any of them None) [B][P], or [rows] packed, or with
    path [B][D_path] one entry a path position; top_ids and top_logp have a last dimension of K alternatives. tokens: laid
    out as the outputs, with path [B][P] (P: positions a request); last [B]: the token behind a request's last entry."""
    cfg = h.cfg
    dtype = torch.bfloat16 if cfg.dtype == DT_BF16 else _F32
    B, V, dev = n_new.numel(), cfg.V, _device()
    ls, ls_ = logits.shape, logits.stride()
    if len(ls) != (3 if row_off is None else 2) or ls[-1] != V:
        raise ValueError("logits need [B][P][V] ([rows][V] packed)")
    at = -2  # dimension of the rows
    if row_off is None:
        P, rows = ls[1], ls[0] * ls[1]
        if ls[0] < B:
            raise ValueError("logits holds fewer requests than n_new")
        if ls[0] > 1:
            if P == 1:  # the requests are the rows (a dimension of one has any stride)
                at = 0
            elif ls_[0] != P * ls_[1]:
                raise ValueError("padded rows must be P rows apart")
    else:
        rows = ls[0]
        if P is None:
            P = tokens.shape[1] if path is not None and tokens is not None and tokens.dim() == 2 else max(1, rows)
    dp = 0
    if path is not None:
        if path.dim() != 2 or path.shape[0] < B:
            raise ValueError("path must be [B][D_path]")
        dp = path.shape[1]
    if tokens is not None and (path is not None or row_off is None) and \
            (tokens.dim() != 2 or tokens.shape[0] < B or tokens.shape[1] != P):
        raise ValueError("tokens must be [B][P]")
    n_out = B * dp if path is not None else rows if row_off is not None else B * P
    K = 0
    if top_ids is not None or top_logp is not None:
        if top_ids is None or top_logp is None or top_ids.shape != top_logp.shape:
            raise ValueError("top_ids and top_logp come together, of one shape")
        K = top_ids.shape[-1]
    if not (logits.dtype is dtype and logits.get_device() == dev and ls_[-1] == 1):
        _strided(logits, dtype, dev, ls_, "logits")
    a = _pack_logprobs(B, P, rows, 0 if row_off is None else _dev(row_off, _I32, dev, "row_off", B + 1),
                       0 if path is None else _dev(path, _I32, dev, "path"), dp, _dev(n_new, _I32, dev, "n_new"), n_extra, shift,
                       0 if tokens is None else _dev(tokens, _I32, dev, "tokens"), 0 if tokens is None else tokens.numel(),
                       0 if last is None else _dev(last, _I32, dev, "last", B), n_out,
                       0 if logp is None else _dev(logp, _F32, dev, "logp", n_out),
                       0 if entropy is None else _dev(entropy, _F32, dev, "entropy", n_out),
                       0 if rank is None else _dev(rank, _I32, dev, "rank", n_out), K,
                       0 if K == 0 else _dev(top_ids, _I32, dev, "top_ids", n_out * K),
                       0 if K == 0 else _dev(top_logp, _F32, dev, "top_logp", n_out * K), _dev(workspace, _U8, dev, "workspace"),
                       workspace.numel())
    rc = lib.dt_token_logprobs(h.h, logits.data_ptr(), ls_[at], a, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        check(rc)


class Meta:
    """Caller-owned device arrays of a flattened verify tree (dt_tree_meta)."""

    def __init__(self, B, P, D_path, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.P, self.D_path = P, D_path
        self.tokens = torch.empty((B, P), **i32)
        self.parents = torch.empty((B, P), **i32)
        self.depth = torch.empty((B, P), **i32)
        self.node_id = torch.empty((B, P), **i32)
        self.mask = torch.empty((B, P, P), dtype=torch.uint8, device=device)
        self.position_ids = torch.empty((B, P), **i32)
        self.retrieve = torch.empty((B, P, D_path), **i32)
        self.n_leaves = torch.empty((B,), **i32)
        self.n_pos = torch.empty((B,), **i32)
        self.row_off = torch.empty((B + 1,), **i32)
        self.c = DtTreeMeta(P, D_path, *[_ptr(t) for t in (self.tokens, self.parents, self.depth, self.node_id,
                                                            self.mask, self.position_ids, self.retrieve,
                                                            self.n_leaves, self.n_pos, self.row_off)])

    def numpy(self):
        return {k: getattr(self, k).cpu().numpy() for k in
                ("tokens", "parents", "depth", "node_id", "mask", "position_ids", "retrieve", "n_leaves",
                 "n_pos", "row_off")}


def make_prune_params(S_T=None, S_D=None, L=512.0, n0=0, C1=0.0, C2=0.0, C3=0.0, R=3, width_cap=1, m_cap=1,
                      D_max=1, ckpt_layers=(), tau=(), k_draft=(), K_total=0, per_request=False):
    """dt_prune_params from device tables (float64 tensors [M_rows][N_cols]) and scalars."""
    p = DtPruneParams()
    p.S_T = _ptr(S_T)
    p.S_D = _ptr(S_D)
    if S_T is not None:
        p.M_rows, p.N_cols = S_T.shape
    p.L, p.n0, p.C1, p.C2, p.C3, p.R = L, n0, C1, C2, C3, R
    p.width_cap, p.m_cap, p.D_max = width_cap, m_cap, D_max
    p.n_ckpt = len(ckpt_layers)
    for i, (c, t, k) in enumerate(zip(ckpt_layers, tau, k_draft)):
        p.ckpt_layer[i], p.tau[i], p.k_draft[i] = c, t, k
    p.K_total = K_total
    p.per_request = 1 if per_request else 0
    return p


def make_prune_out(width=None, stop=None, m=None, stage=None):
    return DtPruneOut(_ptr(width), _ptr(stop), _ptr(m), _ptr(stage))


class Template:
    """Host-side retrieval template (parent, rank) in breadth-first order, hanging from the root or
    (anchor DT_ANCHOR_TAIL) from the deepest kept draft node."""

    def __init__(self, parent, rank, anchor=DT_ANCHOR_ROOT):
        self.n = len(parent)
        self.anchor = anchor
        self._p = (ctypes.c_int32 * max(1, self.n))(*parent)
        self._r = (ctypes.c_int32 * max(1, self.n))(*rank)
        self.c = DtTemplate(self.n, ctypes.cast(self._p, ctypes.c_void_p), ctypes.cast(self._r, ctypes.c_void_p),
                            anchor)
