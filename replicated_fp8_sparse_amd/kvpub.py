"""Thin ctypes binding of libkvpub.so (include/kvpub.h).

Argument marshalling only: every step of the cache-store and the fence runs in
the library's HIP kernels.  Functions keep the C names and return the status
code; ``check()`` turns a non-zero status into ``KvpubError``.  Device
pointers and streams are plain integers (``tensor.data_ptr()``,
``torch.cuda.current_stream().cuda_stream``).

The library must have been built (``replicated_fp8_sparse_amd.build`` or
``__graft_entry__.build()``); loading fails loudly otherwise -- there is no
fallback path.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvpub.so")

KVPUB_OK = 0
KVPUB_ERR_INVALID_ARG = 1
KVPUB_ERR_OUT_OF_MEMORY = 2
KVPUB_ERR_UNSUPPORTED = 3
KVPUB_ERR_HIP = 4
KVPUB_ERR_CAPTURING = 5
KVPUB_ERR_FENCE_TIMEOUT = 6
KVPUB_ERR_IN_USE = 7

KVPUB_FLAG_FENCE_TIMEOUT = 0x1
KVPUB_FLAG_POISONED = 0x2

KVPUB_CONFIG_FENCE_RELEASE_ONLY = 0x1

SLOTS_PER_PAGE = 64
LATENT_DIM = 512
ROPE_DIM = 64
INDEXER_DIM = 128
MAIN_ROW_BYTES = 656
MAIN_PAGE_BYTES = 64 * 656
IDX_PAGE_BYTES = 64 * 128 + 64 * 4
IDX_SCALES_OFFSET = 64 * 128
MAX_REPLICAS = 8

BF16, FP16, FP32 = 0, 1, 2
ROTATE_PAIRS, ROTATE_HALVES = 0, 1
SCALING_NONE, SCALING_LINEAR, SCALING_GROWN, SCALING_RAMP, SCALING_BLEND = range(5)

# Every function include/kvpub.h declares.
EXPORTS = ("kvpub_config_init", "kvpub_create", "kvpub_create_static", "kvpub_store", "kvpub_gather", "kvpub_fence",
           "kvpub_fence_host_epoch",
           "kvpub_graph_create", "kvpub_graph_replay", "kvpub_graph_destroy",
           "kvpub_epoch_read", "kvpub_error_read", "kvpub_participant_signal",
           "kvpub_destroy", "kvpub_strerror", "kvpub_abi_version", "kvpub_vmm_create",
           "kvpub_vmm_grow", "kvpub_vmm_pages", "kvpub_vmm_destroy",
           "kvpub_attend_workspace", "kvpub_attend", "kvpub_attend_slots_workspace", "kvpub_attend_slots",
           "kvpub_attend_weights", "kvpub_evict_workspace", "kvpub_evict", "kvpub_attend_expanded",
           "kvpub_rotation_turns", "kvpub_rotate", "kvpub_store_rotated", "kvpub_heads_append",
           "kvpub_heads_attend_workspace", "kvpub_heads_attend")


class kvpub_config(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32),
                ("num_replicas", ctypes.c_uint32),
                ("num_layers", ctypes.c_uint32),
                ("block_size", ctypes.c_uint32),
                ("num_pages", ctypes.c_uint64),
                ("main_page_stride", ctypes.c_uint64),
                ("main_layer_stride", ctypes.c_uint64),
                ("idx_page_stride", ctypes.c_uint64),
                ("idx_layer_stride", ctypes.c_uint64),
                ("num_lanes", ctypes.c_uint32),
                ("num_participants", ctypes.c_uint32),
                ("fence_timeout_ns", ctypes.c_uint64),
                ("device", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class kvpub_layer_io(ctypes.Structure):
    _fields_ = [("latent", ctypes.c_void_p),
                ("rope", ctypes.c_void_p),
                ("indexer", ctypes.c_void_p),
                ("latent_row_stride", ctypes.c_int64),
                ("rope_row_stride", ctypes.c_int64),
                ("indexer_row_stride", ctypes.c_int64),
                ("slot_mapping", ctypes.c_void_p),
                ("num_tokens", ctypes.c_int64),
                ("layer", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class kvpub_queries(ctypes.Structure):
    _fields_ = [("q_latent", ctypes.c_void_p),
                ("q_rope", ctypes.c_void_p),
                ("q_latent_token_stride", ctypes.c_int64),
                ("q_latent_head_stride", ctypes.c_int64),
                ("q_rope_token_stride", ctypes.c_int64),
                ("q_rope_head_stride", ctypes.c_int64),
                ("num_tokens", ctypes.c_int64),
                ("num_heads", ctypes.c_uint32),
                ("scale", ctypes.c_float)]


class kvpub_pages(ctypes.Structure):
    _fields_ = [("kv_len", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p),
                ("page_table_stride", ctypes.c_int64),
                ("tree_mask", ctypes.c_void_p),
                ("tree_words", ctypes.c_uint32),
                ("num_seqs", ctypes.c_uint32),
                ("max_q_len", ctypes.c_uint32),
                ("max_kv_len", ctypes.c_uint32)]


class kvpub_evict_io(ctypes.Structure):
    _fields_ = [("weights_in", ctypes.c_void_p),
                ("weights_out", ctypes.c_void_p),
                ("weights_stride", ctypes.c_int64),
                ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p),
                ("page_table_stride", ctypes.c_int64),
                ("dst_table", ctypes.c_void_p),
                ("dst_table_stride", ctypes.c_int64),
                ("kept", ctypes.c_void_p),
                ("kept_stride", ctypes.c_int64),
                ("new_len", ctypes.c_void_p),
                ("num_seqs", ctypes.c_uint32),
                ("max_kv_len", ctypes.c_uint32),
                ("budget", ctypes.c_uint32),
                ("first", ctypes.c_uint32),
                ("last", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class kvpub_expanded_io(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q_nope", "q_rope", "k_nope", "k_rope", "v", "out", "lse")] +
                [(n, ctypes.c_int64) for n in (
                    "q_nope_token_stride", "q_nope_head_stride", "q_rope_token_stride", "q_rope_head_stride",
                    "k_nope_token_stride", "k_nope_head_stride", "k_rope_token_stride", "v_token_stride",
                    "v_head_stride", "out_token_stride", "out_head_stride", "lse_token_stride")] +
                [("q_start", ctypes.c_void_p),
                 ("k_start", ctypes.c_void_p),
                 ("num_tokens", ctypes.c_int64),
                 ("num_keys", ctypes.c_int64),
                 ("num_seqs", ctypes.c_uint32),
                 ("num_heads", ctypes.c_uint32),
                 ("max_q_len", ctypes.c_uint32),
                 ("causal", ctypes.c_uint32),
                 ("scale", ctypes.c_float),
                 ("reserved", ctypes.c_uint32)])


class kvpub_rotation(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p),
                ("dim", ctypes.c_uint32),
                ("start", ctypes.c_uint32),
                ("layout", ctypes.c_uint32),
                ("magnitude", ctypes.c_float)]


class kvpub_rotation_config(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_uint32),
                ("scaling", ctypes.c_uint32),
                ("base", ctypes.c_double),
                ("factor", ctypes.c_double),
                ("original", ctypes.c_double),
                ("low", ctypes.c_double),
                ("high", ctypes.c_double)]


class kvpub_rotate_io(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p),
                ("x_token_stride", ctypes.c_int64),
                ("x_head_stride", ctypes.c_int64),
                ("y_token_stride", ctypes.c_int64),
                ("y_head_stride", ctypes.c_int64),
                ("positions", ctypes.c_void_p),
                ("rotation", kvpub_rotation),
                ("num_tokens", ctypes.c_int64),
                ("num_heads", ctypes.c_uint32),
                ("head_dim", ctypes.c_uint32),
                ("type", ctypes.c_uint32),
                ("transpose", ctypes.c_uint32)]


class kvpub_heads(ctypes.Structure):
    _fields_ = [("bases", ctypes.c_void_p * MAX_REPLICAS),
                ("num_pages", ctypes.c_uint64),
                ("page_stride", ctypes.c_uint64),
                ("layer_stride", ctypes.c_uint64),
                ("num_replicas", ctypes.c_uint32),
                ("num_layers", ctypes.c_uint32),
                ("num_kv_heads", ctypes.c_uint32),
                ("head_dim", ctypes.c_uint32)]


class kvpub_heads_rows(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p),
                ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64),
                ("v_head_stride", ctypes.c_int64),
                ("num_tokens", ctypes.c_int64),
                ("type", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class kvpub_heads_queries(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p),
                ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p),
                ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64),
                ("out_token_stride", ctypes.c_int64),
                ("out_head_stride", ctypes.c_int64),
                ("lse_token_stride", ctypes.c_int64),
                ("num_tokens", ctypes.c_int64),
                ("num_heads", ctypes.c_uint32),
                ("type", ctypes.c_uint32),
                ("scale", ctypes.c_float),
                ("reserved", ctypes.c_uint32)]


class KvpubError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: kvpub status {status} ({strerror(status)})")


_lib = None


def load(path=LIB_PATH):
    """Load libkvpub.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with replicated_fp8_sparse_amd.build."
                          "build_library() (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    vp, u32, u64, i64, i32 = (ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64,
                              ctypes.c_int64, ctypes.c_int)
    cfgp = ctypes.POINTER(kvpub_config)
    rp, hp, hqp = ctypes.POINTER(kvpub_rotation), ctypes.POINTER(kvpub_heads), ctypes.POINTER(kvpub_heads_queries)
    qp, pp, ep = ctypes.POINTER(kvpub_queries), ctypes.POINTER(kvpub_pages), ctypes.POINTER(kvpub_evict_io)
    sig = {
        "kvpub_config_init": (None, [cfgp, u32, u32, u64]),
        "kvpub_create": (i32, [cfgp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp)]),
        "kvpub_create_static": (i32, [cfgp, ctypes.POINTER(vp), ctypes.POINTER(vp), vp, ctypes.POINTER(vp)]),
        "kvpub_store": (i32, [vp, u32, i64, vp, i64, vp, i64, vp, i64, vp, vp]),
        "kvpub_gather": (i32, [vp, u32, u32, i64, vp, vp, i64, vp, i64, vp, i64, vp]),
        "kvpub_fence": (i32, [vp, u32, vp]),
        "kvpub_fence_host_epoch": (i32, [vp, u32, vp]),
        "kvpub_graph_create": (i32, [vp, ctypes.POINTER(kvpub_layer_io), u32, u32, ctypes.POINTER(vp)]),
        "kvpub_graph_replay": (i32, [vp, vp]),
        "kvpub_graph_destroy": (i32, [vp]),
        "kvpub_epoch_read": (i32, [vp, u32, ctypes.POINTER(u64)]),
        "kvpub_error_read": (i32, [vp, ctypes.POINTER(u64), ctypes.POINTER(u32), i32]),
        "kvpub_participant_signal": (i32, [vp, u32, u32, ctypes.POINTER(ctypes.POINTER(u64))]),
        "kvpub_destroy": (i32, [vp]),
        "kvpub_strerror": (ctypes.c_char_p, [i32]),
        "kvpub_abi_version": (u32, []),
        "kvpub_vmm_create": (i32, [cfgp, u64, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp)]),
        "kvpub_vmm_grow": (i32, [vp, u64, vp]),
        "kvpub_vmm_pages": (i32, [vp, ctypes.POINTER(u64)]),
        "kvpub_vmm_destroy": (i32, [vp]),
        "kvpub_attend_workspace": (u64, [qp, pp]),
        "kvpub_attend": (i32, [vp, u32, u32, qp, pp, vp, i64, i64, vp, i64, vp, u64, vp]),
        "kvpub_attend_slots_workspace": (u64, [qp, u32]),
        "kvpub_attend_slots": (i32, [vp, u32, u32, qp, vp, i64, u32, vp, i64, i64, vp, i64, vp, u64, vp]),
        "kvpub_attend_weights": (i32, [vp, u32, u32, qp, pp, vp, i64, vp, vp, i64, vp]),
        "kvpub_evict_workspace": (u64, [ep]),
        "kvpub_evict": (i32, [vp, u32, ep, vp, u64, vp]),
        "kvpub_attend_expanded": (i32, [vp, ctypes.POINTER(kvpub_expanded_io), vp]),
        "kvpub_rotation_turns": (i32, [ctypes.POINTER(kvpub_rotation_config), ctypes.POINTER(u64)]),
        "kvpub_rotate": (i32, [vp, ctypes.POINTER(kvpub_rotate_io), vp]),
        "kvpub_store_rotated": (i32, [vp, u32, i64, vp, i64, vp, i64, vp, i64, vp, vp, rp, rp, vp]),
        "kvpub_heads_append": (i32, [vp, hp, u32, ctypes.POINTER(kvpub_heads_rows), pp, rp, vp, vp]),
        "kvpub_heads_attend_workspace": (u64, [hp, hqp, pp]),
        "kvpub_heads_attend": (i32, [vp, hp, u32, u32, hqp, pp, vp, u64, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def strerror(status):
    try:
        return load().kvpub_strerror(int(status)).decode()
    except ImportError:
        return "library not loaded"


def check(status, what="kvpub"):
    if status != KVPUB_OK:
        raise KvpubError(status, what)
    return status


# -- same names as the C ABI ------------------------------------------------

def kvpub_config_init(num_replicas, num_layers, num_pages):
    cfg = kvpub_config()
    load().kvpub_config_init(ctypes.byref(cfg), num_replicas, num_layers, num_pages)
    return cfg


def kvpub_create(cfg, main_bases, idx_bases):
    """Returns (status, ctx handle or None).  Bases are device addresses (ints)."""
    R = len(main_bases)
    mb = (ctypes.c_void_p * R)(*main_bases)
    ib = (ctypes.c_void_p * R)(*idx_bases)
    out = ctypes.c_void_p()
    st = load().kvpub_create(ctypes.byref(cfg), mb, ib, ctypes.byref(out))
    return st, (out.value if st == KVPUB_OK else None)


def kvpub_create_static(cfg, main_bases, idx_bases, stream=0):
    """Returns (status, ctx handle or None); the context's words live in the
    library's static per-GPU array (no allocation)."""
    R = len(main_bases)
    mb = (ctypes.c_void_p * R)(*main_bases)
    ib = (ctypes.c_void_p * R)(*idx_bases)
    out = ctypes.c_void_p()
    st = load().kvpub_create_static(ctypes.byref(cfg), mb, ib, stream, ctypes.byref(out))
    return st, (out.value if st == KVPUB_OK else None)


def kvpub_store(ctx, layer, num_tokens, latent, latent_row_stride, rope, rope_row_stride,
                indexer, indexer_row_stride, slot_mapping, stream=0):
    return load().kvpub_store(ctx, layer, num_tokens, latent, latent_row_stride, rope,
                              rope_row_stride, indexer, indexer_row_stride, slot_mapping,
                              stream)


def kvpub_gather(ctx, replica, layer, num_tokens, slot_mapping, latent_out, latent_row_stride,
                 rope_out, rope_row_stride, indexer_out, indexer_row_stride, stream=0):
    return load().kvpub_gather(ctx, replica, layer, num_tokens, slot_mapping, latent_out,
                               latent_row_stride, rope_out, rope_row_stride, indexer_out,
                               indexer_row_stride, stream)


def kvpub_fence(ctx, lane=0, stream=0):
    return load().kvpub_fence(ctx, lane, stream)


def kvpub_fence_host_epoch(ctx, lane=0, stream=0):
    return load().kvpub_fence_host_epoch(ctx, lane, stream)


def kvpub_graph_create(ctx, ios, lane=0):
    """ios: sequence of kvpub_layer_io.  Returns (status, graph handle or None)."""
    n = len(ios)
    arr = (kvpub_layer_io * n)(*ios)
    out = ctypes.c_void_p()
    st = load().kvpub_graph_create(ctx, arr, n, lane, ctypes.byref(out))
    return st, (out.value if st == KVPUB_OK else None)


def kvpub_graph_replay(graph, stream=0):
    return load().kvpub_graph_replay(graph, stream)


def kvpub_graph_destroy(graph):
    return load().kvpub_graph_destroy(graph)


def kvpub_epoch_read(ctx, lane=0):
    v = ctypes.c_uint64()
    st = load().kvpub_epoch_read(ctx, lane, ctypes.byref(v))
    return st, v.value


def kvpub_error_read(ctx, clear=False):
    """Returns (status, invalid_slots, flags)."""
    inv = ctypes.c_uint64()
    fl = ctypes.c_uint32()
    st = load().kvpub_error_read(ctx, ctypes.byref(inv), ctypes.byref(fl), 1 if clear else 0)
    return st, inv.value, fl.value


def kvpub_participant_signal(ctx, lane, p):
    """Returns (status, ctypes pointer to the host-coherent uint64 signal word)."""
    out = ctypes.POINTER(ctypes.c_uint64)()
    st = load().kvpub_participant_signal(ctx, lane, p, ctypes.byref(out))
    return st, (out if st == KVPUB_OK else None)


def kvpub_destroy(ctx):
    return load().kvpub_destroy(ctx)


def kvpub_abi_version():
    return load().kvpub_abi_version()


def kvpub_vmm_create(cfg, max_pages):
    """Returns (status, vmm handle or None, main base addresses, idx base addresses);
    cfg's layer strides are updated in place."""
    R = cfg.num_replicas
    mb = (ctypes.c_void_p * max(R, 1))()
    ib = (ctypes.c_void_p * max(R, 1))()
    out = ctypes.c_void_p()
    st = load().kvpub_vmm_create(ctypes.byref(cfg), max_pages, mb, ib, ctypes.byref(out))
    if st != KVPUB_OK:
        return st, None, [], []
    return st, out.value, [mb[r] for r in range(R)], [ib[r] for r in range(R)]


def kvpub_vmm_grow(vmm, num_pages, ctx=None):
    return load().kvpub_vmm_grow(vmm, num_pages, ctx)


def kvpub_vmm_pages(vmm):
    v = ctypes.c_uint64()
    st = load().kvpub_vmm_pages(vmm, ctypes.byref(v))
    return st, v.value


def kvpub_vmm_destroy(vmm):
    return load().kvpub_vmm_destroy(vmm)


def kvpub_strerror(status):
    return strerror(status)


def layer_io(latent, rope, indexer, slot_mapping, num_tokens, layer,
             latent_row_stride=LATENT_DIM, rope_row_stride=ROPE_DIM,
             indexer_row_stride=INDEXER_DIM):
    """Build a kvpub_layer_io from device addresses."""
    return kvpub_layer_io(latent, rope, indexer, latent_row_stride, rope_row_stride,
                          indexer_row_stride, slot_mapping, num_tokens, layer, 0)


# -- attention over the published cache ---------------------------------------
# Descriptors (None passes a null pointer) are built by queries(), pages(),
# evict_io() and expanded_io() below.

def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def kvpub_attend_workspace(q, pages):
    return load().kvpub_attend_workspace(_ref(q), _ref(pages))


def kvpub_attend(ctx, replica, layer, q, pages, out, out_token_stride, out_head_stride, lse, lse_token_stride,
                 workspace, workspace_bytes, stream=0):
    return load().kvpub_attend(ctx, replica, layer, _ref(q), _ref(pages), out, out_token_stride, out_head_stride,
                               lse, lse_token_stride, workspace, workspace_bytes, stream)


def kvpub_attend_slots_workspace(q, num_slots):
    return load().kvpub_attend_slots_workspace(_ref(q), num_slots)


def kvpub_attend_slots(ctx, replica, layer, q, slots, slots_stride, num_slots, out, out_token_stride,
                       out_head_stride, lse, lse_token_stride, workspace, workspace_bytes, stream=0):
    return load().kvpub_attend_slots(ctx, replica, layer, _ref(q), slots, slots_stride, num_slots, out,
                                     out_token_stride, out_head_stride, lse, lse_token_stride, workspace,
                                     workspace_bytes, stream)


def kvpub_attend_weights(ctx, replica, layer, q, pages, lse, lse_token_stride, weights_in, weights_out,
                         weights_stride, stream=0):
    return load().kvpub_attend_weights(ctx, replica, layer, _ref(q), _ref(pages), lse, lse_token_stride,
                                       weights_in, weights_out, weights_stride, stream)


def kvpub_evict_workspace(io):
    return load().kvpub_evict_workspace(_ref(io))


def kvpub_evict(ctx, layer, io, workspace, workspace_bytes, stream=0):
    return load().kvpub_evict(ctx, layer, _ref(io), workspace, workspace_bytes, stream)


def kvpub_attend_expanded(ctx, io, stream=0):
    return load().kvpub_attend_expanded(ctx, _ref(io), stream)


def queries(q_latent, q_rope, num_tokens, num_heads, scale, q_latent_token_stride=None,
            q_latent_head_stride=LATENT_DIM, q_rope_token_stride=None, q_rope_head_stride=ROPE_DIM):
    """Build a kvpub_queries from device addresses; strides default to dense [T, H, .]."""
    lt = num_heads * LATENT_DIM if q_latent_token_stride is None else q_latent_token_stride
    rt = num_heads * ROPE_DIM if q_rope_token_stride is None else q_rope_token_stride
    return kvpub_queries(q_latent, q_rope, lt, q_latent_head_stride, rt, q_rope_head_stride, num_tokens,
                         num_heads, scale)


def pages(kv_len, page_table, page_table_stride, num_seqs, max_kv_len, q_start=0, max_q_len=1, tree_mask=0,
          tree_words=0):
    """Build a kvpub_pages from device addresses."""
    return kvpub_pages(kv_len, q_start, page_table, page_table_stride, tree_mask, tree_words, num_seqs, max_q_len,
                       max_kv_len)


def evict_io(weights_in, weights_out, weights_stride, kv_len, page_table, page_table_stride, dst_table,
             dst_table_stride, kept, kept_stride, new_len, num_seqs, max_kv_len, budget, first=0, last=0):
    """Build a kvpub_evict_io from device addresses."""
    return kvpub_evict_io(weights_in, weights_out, weights_stride, kv_len, page_table, page_table_stride, dst_table,
                          dst_table_stride, kept, kept_stride, new_len, num_seqs, max_kv_len, budget, first, last, 0)


def expanded_io(q_nope, q_rope, k_nope, k_rope, v, out, lse, q_start, k_start, num_seqs, num_heads, num_tokens,
                num_keys, max_q_len, scale, k_head_stride=128, v_head_stride=128, causal=1):
    """Build a kvpub_expanded_io from device addresses: dense queries, outputs and
    RoPE rows, keys and values of the given head strides."""
    H = num_heads
    return kvpub_expanded_io(q_nope, q_rope, k_nope, k_rope, v, out, lse, H * 128, 128, H * 64, 64,
                             H * k_head_stride, k_head_stride, 64, H * v_head_stride, v_head_stride, H * 128, 128, H,
                             q_start, k_start, num_tokens, num_keys, num_seqs, H, max_q_len, causal, scale, 0)


# -- rotary positions and the cache of key and value heads ----------------------

def kvpub_rotation_turns(config):
    """Returns (status, turns as a numpy uint64 array or None): the table to copy to the device."""
    import numpy as np
    turns = np.zeros(max(config.dim, 8) // 2, dtype=np.uint64)
    st = load().kvpub_rotation_turns(ctypes.byref(config), turns.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)))
    return st, (turns if st == KVPUB_OK else None)


def kvpub_rotate(ctx, io, stream=0):
    return load().kvpub_rotate(ctx, _ref(io), stream)


def kvpub_store_rotated(ctx, layer, num_tokens, latent, latent_row_stride, rope, rope_row_stride, indexer,
                        indexer_row_stride, slot_mapping, positions, rope_rotation, indexer_rotation, stream=0):
    return load().kvpub_store_rotated(ctx, layer, num_tokens, latent, latent_row_stride, rope, rope_row_stride, indexer,
                                      indexer_row_stride, slot_mapping, positions, _ref(rope_rotation),
                                      _ref(indexer_rotation), stream)


def kvpub_heads_append(ctx, cache, layer, rows, pages, rotation=None, positions=None, stream=0):
    return load().kvpub_heads_append(ctx, _ref(cache), layer, _ref(rows), _ref(pages), _ref(rotation), positions, stream)


def kvpub_heads_attend_workspace(cache, q, pages):
    return load().kvpub_heads_attend_workspace(_ref(cache), _ref(q), _ref(pages))


def kvpub_heads_attend(ctx, cache, replica, layer, q, pages, workspace, workspace_bytes, stream=0):
    return load().kvpub_heads_attend(ctx, _ref(cache), replica, layer, _ref(q), _ref(pages), workspace, workspace_bytes,
                                     stream)


def rotation_config(dim, base=10000.0, scaling=SCALING_NONE, factor=1.0, original=1.0, low=1.0, high=32.0):
    return kvpub_rotation_config(dim, scaling, base, factor, original, low, high)


def rotation(turns, dim, start=0, layout=ROTATE_PAIRS, magnitude=1.0):
    """Build a kvpub_rotation; turns: the device address of its table."""
    return kvpub_rotation(turns, dim, start, layout, magnitude)


def rotate_io(x, y, positions, rotation, num_tokens, num_heads, head_dim, type, x_token_stride=None, x_head_stride=None,
              y_token_stride=None, y_head_stride=None, transpose=0):
    """Build a kvpub_rotate_io from device addresses; strides default to dense [T, H, head_dim]."""
    width = lambda s: head_dim if s is None else s
    dense = lambda s, head: num_heads * width(head) if s is None else s
    return kvpub_rotate_io(x, y, dense(x_token_stride, x_head_stride), width(x_head_stride),
                           dense(y_token_stride, y_head_stride), width(y_head_stride), positions, rotation, num_tokens,
                           num_heads, head_dim, type, transpose)


def heads_page_bytes(num_kv_heads, head_dim):
    """Bytes of a page of the cache of heads (KVPUB_HEADS_PAGE_BYTES)."""
    return (num_kv_heads * (128 * head_dim + 2) + 15) // 16 * 16


def heads(bases, num_pages, num_kv_heads, head_dim, num_layers=1, page_stride=None, layer_stride=None):
    """Build a kvpub_heads over replicas at these device addresses; strides default to dense pages and layers."""
    page = heads_page_bytes(num_kv_heads, head_dim) if page_stride is None else page_stride
    layer = num_pages * page if layer_stride is None else layer_stride
    return kvpub_heads((ctypes.c_void_p * MAX_REPLICAS)(*bases), num_pages, page, layer, len(bases), num_layers,
                       num_kv_heads, head_dim)


def heads_rows(k, v, num_tokens, type, k_token_stride, k_head_stride, v_token_stride, v_head_stride):
    """Build a kvpub_heads_rows from device addresses."""
    return kvpub_heads_rows(k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, num_tokens, type, 0)


def heads_queries(q, out, lse, num_tokens, num_heads, head_dim, scale, type, q_token_stride=None, q_head_stride=None,
                  out_token_stride=None, out_head_stride=None, lse_token_stride=None):
    """Build a kvpub_heads_queries from device addresses; strides default to dense [T, H, head_dim] and [T, H]."""
    qh = head_dim if q_head_stride is None else q_head_stride
    oh = head_dim if out_head_stride is None else out_head_stride
    return kvpub_heads_queries(q, out, lse, num_heads * qh if q_token_stride is None else q_token_stride, qh,
                               num_heads * oh if out_token_stride is None else out_token_stride, oh,
                               num_heads if lse_token_stride is None else lse_token_stride, num_tokens, num_heads, type,
                               scale, 0)
