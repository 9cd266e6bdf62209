"""ctypes binding of libdt.so: the same entry points as include/dt.h, argument marshalling only.

Tensors are torch CUDA tensors; their device pointers and the current CUDA
stream are handed to the C ABI. Every computation runs in the library's
kernels. Importing this module fails loudly when libdt.so is missing.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdt.so")

DT_OK, DT_ERR_ARG, DT_ERR_CUDA, DT_ERR_DEVICE, DT_ERR_DEVICE_TIMEOUT = 0, -1, -2, -3, -4
DT_BF16, DT_F32, DT_F16 = 0, 1, 2
DT_GREEDY, DT_SAMPLE = 0, 1
DT_VERIFY_PACKED = 2
DT_POLICY_CAST_WIDTH_DEPTH, DT_POLICY_CAST_VERIFY, DT_POLICY_GRAFT_CHECKPOINT, DT_POLICY_NONE = 0, 1, 2, 3
DT_DEV_BAD_LOGITS, DT_DEV_BAD_TOKEN, DT_DEV_BAD_TREE, DT_DEV_TIMEOUT, DT_DEV_INTERNAL = 1, 2, 4, 8, 16
DT_DEV_KV_FULL, DT_DEV_BAD_PAGE = 32, 64
DT_SEEN_PROMPT = 0x40000000
DT_FLAG_TEST_TIMEOUT, DT_FLAG_TEST_ARRIVED = 1, 2
DT_ANCHOR_ROOT, DT_ANCHOR_TAIL = 0, 1

EXPORTS = ["dt_last_error_string", "dt_create", "dt_destroy", "dt_get_tree", "dt_get_status",
           "dt_clear_status", "dt_tree_reset", "dt_select_frontier", "dt_expand_layer", "dt_cast_prune",
           "dt_rerank", "dt_graft_retrieve", "dt_build_tree_meta", "dt_verify", "dt_adj_update",
           "dt_row_topk_static", "dt_cast_prune_select",
           "dt_cast_verify_rerank", "dt_expand_prune_select", "dt_verify_rows", "dt_verify_accept",
           "dt_commit_kv", "dt_block_expand", "dt_expand_layer_sampled", "dt_verify_sampled",
           "dt_kv_reserve", "dt_kv_release", "dt_commit_kv_paged", "dt_tree_attention",
           "dt_tree_attention_workspace", "dt_count_tokens", "dt_logits_process", "dt_prompt_attention",
           "dt_prompt_attention_workspace", "dt_token_logprobs", "dt_token_logprobs_workspace",
           "dt_kv_fork", "dt_kv_release_shared"]

c_i32p = ctypes.c_void_p
vp = ctypes.c_void_p


class DtConfig(ctypes.Structure):
    _fields_ = [("B_max", ctypes.c_int32), ("V", ctypes.c_int32), ("K", ctypes.c_int32),
                ("W", ctypes.c_int32), ("D_max", ctypes.c_int32), ("P_max", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class DtTreeView(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("K", ctypes.c_int32), ("W", ctypes.c_int32),
                ("D_max", ctypes.c_int32), ("N", ctypes.c_int32), ("LW", ctypes.c_int32),
                ("depth", ctypes.c_int32), ("token", vp), ("parent", vp), ("node_depth", vp),
                ("logc", vp), ("value", vp), ("layer_order", vp), ("layer_count", vp),
                ("frontier", vp), ("frontier_count", vp)]


class DtPruneParams(ctypes.Structure):
    _fields_ = [("S_T", vp), ("S_D", vp), ("M_rows", ctypes.c_int32), ("N_cols", ctypes.c_int32),
                ("L", ctypes.c_double), ("n0", ctypes.c_int64), ("C1", ctypes.c_double),
                ("C2", ctypes.c_double), ("C3", ctypes.c_double), ("R", ctypes.c_int32),
                ("width_cap", ctypes.c_int32), ("m_cap", ctypes.c_int32), ("D_max", ctypes.c_int32),
                ("n_ckpt", ctypes.c_int32), ("ckpt_layer", ctypes.c_int32 * 16),
                ("tau", ctypes.c_double * 16), ("k_draft", ctypes.c_int32 * 16),
                ("K_total", ctypes.c_int32), ("per_request", ctypes.c_int32)]


class DtPruneOut(ctypes.Structure):
    _fields_ = [("width", vp), ("stop", vp), ("m", vp), ("stage", vp)]


class DtTemplate(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("parent", vp), ("rank", vp), ("anchor", ctypes.c_int32)]


class DtTreeMeta(ctypes.Structure):
    _fields_ = [("P", ctypes.c_int32), ("D_path", ctypes.c_int32), ("tokens", vp), ("parents", vp),
                ("depth", vp), ("node_id", vp), ("mask", vp), ("position_ids", vp),
                ("retrieve", vp), ("n_leaves", vp), ("n_pos", vp), ("row_off", vp)]


class DtBlockPool(ctypes.Structure):
    _fields_ = [("page", ctypes.c_int32), ("n_blocks", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("block_table", vp), ("n_owned", vp), ("free_list", vp), ("free_count", vp)]


class DtKvRows(ctypes.Structure):
    _fields_ = [("tmp", vp), ("tmp_plane", ctypes.c_int64), ("tmp_row", ctypes.c_int64),
                ("tmp_head", ctypes.c_int64), ("rows", ctypes.c_int64), ("cache", vp),
                ("cache_plane", ctypes.c_int64), ("cache_block", ctypes.c_int64), ("cache_tok", ctypes.c_int64),
                ("cache_head", ctypes.c_int64), ("planes", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_bytes", ctypes.c_int64), ("page", ctypes.c_int32), ("n_blocks", ctypes.c_int32), ("committed", vp)]


class DtKvPages(ctypes.Structure):
    _fields_ = [("cache", vp), ("cache_plane", ctypes.c_int64), ("cache_block", ctypes.c_int64),
                ("cache_tok", ctypes.c_int64), ("cache_head", ctypes.c_int64), ("planes", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_bytes", ctypes.c_int64)]


class DtAttnArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("P", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("shared_len", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("q", vp), ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("out", vp), ("o_row", ctypes.c_int64), ("o_head", ctypes.c_int64),
                ("k_new", vp), ("v_new", vp), ("kn_row", ctypes.c_int64), ("kn_head", ctypes.c_int64),
                ("vn_row", ctypes.c_int64), ("vn_head", ctypes.c_int64),
                ("k_pages", vp), ("v_pages", vp), ("k_block", ctypes.c_int64), ("k_tok", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_block", ctypes.c_int64), ("v_tok", ctypes.c_int64),
                ("v_head", ctypes.c_int64), ("n_blocks", ctypes.c_int32), ("page", ctypes.c_int32),
                ("block_table", vp), ("max_blocks", ctypes.c_int32), ("seq_len", vp), ("n_pos", vp), ("mask", vp),
                ("row_off", vp), ("workspace", vp), ("workspace_bytes", ctypes.c_int64)]


class DtPromptArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("rows", ctypes.c_int64),
                ("q", vp), ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("out", vp), ("o_row", ctypes.c_int64), ("o_head", ctypes.c_int64),
                ("k_new", vp), ("v_new", vp), ("kn_row", ctypes.c_int64), ("kn_head", ctypes.c_int64),
                ("vn_row", ctypes.c_int64), ("vn_head", ctypes.c_int64), ("row_off", vp),
                ("k_pages", vp), ("v_pages", vp), ("k_block", ctypes.c_int64), ("k_tok", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_block", ctypes.c_int64), ("v_tok", ctypes.c_int64),
                ("v_head", ctypes.c_int64), ("n_blocks", ctypes.c_int32), ("page", ctypes.c_int32),
                ("block_table", vp), ("max_blocks", ctypes.c_int32), ("seq_len", vp), ("workspace", vp),
                ("workspace_bytes", ctypes.c_int64)]


class DtLogprobArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("P", ctypes.c_int32), ("rows", ctypes.c_int64), ("row_off", vp), ("path", vp),
                ("D_path", ctypes.c_int32), ("n_new", vp), ("n_extra", ctypes.c_int32), ("shift", ctypes.c_int32),
                ("tokens", vp), ("n_tokens", ctypes.c_int64), ("last", vp), ("n_out", ctypes.c_int64), ("logp", vp),
                ("entropy", vp), ("rank", vp), ("K", ctypes.c_int32), ("top_ids", vp), ("top_logp", vp),
                ("workspace", vp), ("workspace_bytes", ctypes.c_int64)]


class DtLogitsParams(ctypes.Structure):
    _fields_ = [("P", ctypes.c_int32), ("n_pos", vp), ("row_off", vp), ("rows", ctypes.c_int64), ("tokens", vp),
                ("mask", vp), ("counts", vp), ("repetition", vp), ("frequency", vp), ("presence", vp),
                ("bias_ids", vp), ("bias_vals", vp), ("n_bias", ctypes.c_int32), ("allow", vp),
                ("allow_ld", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libdt.so not found at {LIB_PATH}: build it with __graft_entry__.build() "
                          "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    I = ctypes.c_int
    sig = {
        "dt_last_error_string": ([], ctypes.c_char_p),
        "dt_create": ([ctypes.POINTER(DtConfig), ctypes.POINTER(vp)], I),
        "dt_destroy": ([vp], I),
        "dt_get_tree": ([vp, ctypes.POINTER(DtTreeView)], I),
        "dt_get_status": ([vp, vp, ctypes.POINTER(ctypes.c_int32)], I),
        "dt_clear_status": ([vp, vp], I),
        "dt_tree_reset": ([vp, ctypes.c_int32, vp, vp], I),
        "dt_select_frontier": ([vp, vp, ctypes.c_int32, vp, vp, vp], I),
        "dt_expand_layer": ([vp, vp, ctypes.c_int64, ctypes.c_int32, vp], I),
        "dt_cast_prune": ([vp, ctypes.c_int32, ctypes.POINTER(DtPruneParams), ctypes.POINTER(DtPruneOut), vp], I),
        "dt_rerank": ([vp, vp, ctypes.c_int32, ctypes.c_int32, vp, vp], I),
        "dt_graft_retrieve": ([vp, vp, ctypes.POINTER(DtTemplate), ctypes.c_int32, vp, ctypes.c_int32,
                               vp, vp, vp, vp, vp], I),
        "dt_build_tree_meta": ([vp, vp, ctypes.c_int32, vp, vp, vp, vp, ctypes.c_int32, ctypes.c_int32, vp,
                                ctypes.POINTER(DtTreeMeta), vp], I),
        "dt_expand_layer_sampled": ([vp, vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint64, vp], I),
        "dt_verify_sampled": ([vp, ctypes.POINTER(DtTreeMeta), vp, ctypes.c_int64, ctypes.c_int32, vp, ctypes.c_int64,
                               ctypes.c_uint64, ctypes.c_uint64, vp, vp, vp, vp], I),
        "dt_block_expand": ([vp, vp, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(DtPruneParams),
                             ctypes.POINTER(DtPruneOut), vp], I),
        "dt_verify": ([vp, ctypes.POINTER(DtTreeMeta), vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64,
                       ctypes.c_uint64, vp, vp, vp, vp, vp], I),
        "dt_adj_update": ([vp, vp, ctypes.POINTER(DtTreeMeta), vp, vp], I),
        "dt_cast_prune_select": ([vp, ctypes.POINTER(DtPruneParams), ctypes.POINTER(DtPruneOut), vp, vp], I),
        "dt_expand_prune_select": ([vp, vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                    ctypes.POINTER(DtPruneParams), ctypes.POINTER(DtPruneOut), vp, ctypes.c_int32,
                                    vp, vp], I),
        "dt_verify_rows": ([vp, ctypes.POINTER(DtTreeMeta), vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, vp], I),
        "dt_verify_accept": ([vp, ctypes.POINTER(DtTreeMeta), vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64,
                              ctypes.c_uint64, vp, vp, vp, vp, vp], I),
        "dt_commit_kv": ([vp, vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, vp, ctypes.c_int64, ctypes.c_int64,
                          ctypes.c_int32, ctypes.c_int64, vp, vp, vp, ctypes.c_int32, vp, vp], I),
        "dt_cast_verify_rerank": ([vp, ctypes.POINTER(DtPruneParams), ctypes.POINTER(DtPruneOut), vp, vp], I),
        "dt_kv_reserve": ([vp, ctypes.c_int32, vp, vp, vp, ctypes.c_int32, vp,
                           ctypes.c_int64, ctypes.c_int32, vp, vp], I),
        "dt_kv_release": ([vp, ctypes.c_int32, vp, vp, vp], I),
        "dt_commit_kv_paged": ([vp, ctypes.c_int32, vp, ctypes.c_int32, vp, vp, ctypes.c_int32,
                                vp, ctypes.c_int32, vp, ctypes.c_int64, ctypes.c_int32, vp, vp, vp, vp], I),
        "dt_tree_attention": ([vp, vp, vp], I),
        "dt_tree_attention_workspace": ([vp] + [ctypes.c_int32] * 6 + [ctypes.POINTER(ctypes.c_int64)], I),
        "dt_prompt_attention": ([vp, vp, vp], I),
        "dt_prompt_attention_workspace": ([vp] + [ctypes.c_int32] * 4 + [ctypes.POINTER(ctypes.c_int64)], I),
        "dt_token_logprobs": ([vp, vp, ctypes.c_int64, vp, vp], I),
        "dt_token_logprobs_workspace": ([vp, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(ctypes.c_int64)], I),
        "dt_kv_fork": ([vp, ctypes.c_int32, vp, vp, vp, ctypes.c_int32, vp, vp, vp, vp, ctypes.c_int32, vp], I),
        "dt_kv_release_shared": ([vp, ctypes.c_int32, vp, vp, vp, vp], I),
        "dt_count_tokens": ([vp, ctypes.c_int32, vp, vp, ctypes.c_int64, ctypes.c_int32, vp, vp, ctypes.c_int32, vp, ctypes.c_int32,
                             ctypes.c_int32, vp], I),
        "dt_logits_process": ([vp, ctypes.c_int32, vp, ctypes.c_int64, vp, ctypes.c_int64,
                               vp, vp], I),
        "dt_row_topk_static": ([vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                vp, vp, vp, vp], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load()


class DtError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"libdt error {code}: {msg}")
        self.code = code


def check(rc):
    if rc != DT_OK:
        raise DtError(rc, lib.dt_last_error_string().decode(errors="replace"))
    return rc
