"""ctypes binding of the C ABI (include/prefill.h, include/prefill_ops.h).

Argument marshalling only: every step of the prefill pass runs in the CUDA
library.  There is no fallback: if the library is missing or a call fails,
the binding raises.  PyTorch is used by callers for device memory and
streams; this module passes raw pointers and sizes.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libprefill_kv_shared.so")

PF_OK = 0
PF_E_ARG = -1
PF_E_KV_MAGIC = -2
PF_E_KV_SHAPE = -3
PF_E_KV_RANGE = -4
PF_E_CUDA = -5
PF_E_DEVICE_TIMEOUT = -6
PF_E_DEVICE_TOKEN = -7
PF_E_NOMEM = -8
PF_E_IO = -9

PF_OUT_EMBD = -1

PF_PRUNE_OFF = 0
PF_PRUNE_ON = 1
PF_PRUNE_OFF_PLAIN = 2

PF_W_F32 = 0
PF_W_Q4_0 = 2
PF_L_F32 = 0
PF_L_BF16 = 1
PF_FFN_GEGLU = 0
PF_FFN_SWIGLU = 1

# every symbol the headers declare
EXPORTS = (
    "prefill_create", "prefill_ubatch", "prefill_sync", "prefill_n_pos", "prefill_reset",
    "prefill_set_prune", "prefill_prune_active", "prefill_kv_image_bytes", "kv_save", "kv_load",
    "prefill_destroy", "prefill_last_error", "prefill_prune_predicate", "prefill_kv_header_check",
    "prefill_kv_image_bytes_for", "prefill_set_timing", "prefill_get_stats", "prefill_reset_stats",
    "pfop_linear_f32", "pfop_linear_resid", "pfop_linear_glu", "pfop_linear_ple", "pfop_linear_qkv",
    "pfop_attention", "pfop_rmsnorm", "pfop_embed", "pfop_kv_copy", "pfop_last_error", "pfop_linear_bench",
    "pfop_attention_split_noalloc", "pfop_attention_bench", "pfop_kv_copy_bench",
    "kv_save_file", "kv_load_file", "prefill_kv_file_check", "pfop_linear_row", "prefill_set_output",
    "pfop_linear_wait_test", "prefill_ubatch_seqs", "prefill_seq_n_pos", "prefill_seq_reset",
    "prefill_graph_capture", "prefill_graph_launch", "pfop_set_gemm_pairs", "pfop_qkv_row_order",
    "pfop_repack_q4", "pfop_attention_packed", "pfop_attention_tree", "pfop_attention_work_bytes",
    "pfop_attention_status", "pfop_logprobs", "pfop_attention_paged", "pfop_attention_paged_work_bytes",
    "pfop_attention_paged_status", "pfop_qk_norm_rope", "pfop_verify_draft", "pfop_verify_draft_work_bytes",
)


class PrefillError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"status {code}: {msg}")
        self.code = code


class ModelDesc(C.Structure):
    _fields_ = [
        ("n_layer", C.c_int32), ("n_layer_kv_from_start", C.c_int32), ("d_model", C.c_int32),
        ("n_head", C.c_int32), ("n_head_kv", C.c_int32), ("head_dim", C.c_int32),
        ("ffn_dim", C.c_int32), ("vocab", C.c_int32), ("ple_dim", C.c_int32),
        ("ffn_kind", C.c_int32), ("wtype", C.c_int32), ("rms_eps", C.c_float),
        ("rope_base", C.c_float), ("kv_src", C.POINTER(C.c_int32)), ("max_ctx", C.c_int32),
        ("ubatch_max", C.c_int32), ("prune_shared_enable", C.c_int32), ("n_seq_max", C.c_int32),
        ("embeddings", C.c_int32), ("embd_layer_inp", C.POINTER(C.c_int32)),
    ]


KC_GEMM, KC_ATTN, KC_NORM, KC_OTHER, KC_GEMM_ROW, KC_ATTN_ROW = 0, 1, 2, 3, 4, 5
KC_NAMES = ("gemm", "attention", "norm", "other", "gemm_row", "attention_row")
KC_COUNT = len(KC_NAMES)


class Stats(C.Structure):
    _fields_ = [("launches", C.c_int64 * KC_COUNT), ("flops", C.c_double * KC_COUNT),
                ("bytes", C.c_double * KC_COUNT), ("timed", C.c_int64 * KC_COUNT), ("ms", C.c_double * KC_COUNT)]


class LayerWeights(C.Structure):
    _fields_ = [(k, C.c_void_p) for k in ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate",
                                          "w_up", "w_down", "ple_gate", "ple_proj")]


class SeqRun(C.Structure):
    _fields_ = [("seq_id", C.c_int32), ("n_tokens", C.c_int32), ("is_last", C.c_int32)]


class AttnRun(C.Structure):
    _fields_ = [("n_rows", C.c_int32), ("pos0", C.c_int32), ("cell0", C.c_int32)]


class Weights(C.Structure):
    _fields_ = [("tok_embd", C.c_void_p), ("ple_embd", C.c_void_p), ("out_norm", C.c_void_p),
                ("layers", C.POINTER(LayerWeights))]


_lib = None


def load(path: str = LIB_PATH) -> C.CDLL:
    """Load the library (building it first if the sources are newer)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path) or os.environ.get("PREFILL_REBUILD"):
        from . import build as _b
        _b.build()
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not found: {path}")
    lib = C.CDLL(path)
    vp, i32, i64, f32, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
    sig = {
        "prefill_create": (C.c_int, [C.POINTER(ModelDesc), C.POINTER(Weights), vp, C.POINTER(vp)]),
        "prefill_ubatch": (C.c_int, [vp, vp, i32, i64, i32, vp]),
        "prefill_sync": (C.c_int, [vp]),
        "prefill_set_output": (C.c_int, [vp, i32, vp]),
        "prefill_ubatch_seqs": (C.c_int, [vp, vp, C.POINTER(SeqRun), i32, vp]),
        "prefill_seq_n_pos": (i64, [vp, i32]),
        "prefill_seq_reset": (C.c_int, [vp, i32]),
        "prefill_graph_capture": (C.c_int, [vp, vp, i32, i64, i32, vp]),
        "prefill_graph_launch": (C.c_int, [vp]),
        "prefill_n_pos": (i64, [vp]),
        "prefill_reset": (C.c_int, [vp]),
        "prefill_set_prune": (C.c_int, [vp, i32]),
        "prefill_prune_active": (C.c_int, [vp]),
        "prefill_kv_image_bytes": (i64, [vp, i64]),
        "kv_save": (C.c_int, [vp, vp, sz]),
        "kv_load": (C.c_int, [vp, vp, sz, i64]),
        "kv_save_file": (C.c_int, [vp, C.c_char_p]),
        "kv_load_file": (C.c_int, [vp, C.c_char_p, i64]),
        "prefill_kv_file_check": (C.c_int, [C.c_char_p, i32, i32, i64, C.POINTER(C.c_int64)]),
        "prefill_destroy": (None, [vp]),
        "prefill_last_error": (C.c_char_p, [vp]),
        "prefill_prune_predicate": (C.c_int, [C.POINTER(ModelDesc)]),
        "prefill_kv_header_check": (C.c_int, [vp, i32, i32, i64, i64, sz]),
        "prefill_kv_image_bytes_for": (i64, [i32, i64, i32]),
        "prefill_set_timing": (C.c_int, [vp, i32]),
        "prefill_get_stats": (C.c_int, [vp, C.POINTER(Stats)]),
        "prefill_reset_stats": (C.c_int, [vp]),
        "pfop_linear_f32": (C.c_int, [i32, vp, i32, i32, i32, vp, i32, i32, vp, vp]),
        "pfop_linear_resid": (C.c_int, [i32, vp, i32, i32, vp, i32, i32, vp, vp, vp]),
        "pfop_linear_glu": (C.c_int, [i32, vp, vp, i32, i32, i32, vp, i32, i32, vp, vp]),
        "pfop_linear_ple": (C.c_int, [i32, vp, i32, i32, vp, i32, i32, vp, i32, vp, vp]),
        "pfop_linear_qkv": (C.c_int, [i32, vp, vp, vp, i32, i32, i32, i32, f32, vp, i32, i32, i32, i32,
                                      vp, vp, vp, vp]),
        "pfop_attention": (C.c_int, [i32, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]),
        "pfop_rmsnorm": (C.c_int, [vp, i32, i32, i32, vp, f32, vp, vp, vp]),
        "pfop_embed": (C.c_int, [i32, vp, vp, i32, i32, i32, f32, vp, i32, vp, vp, vp]),
        "pfop_kv_copy": (C.c_int, [i32, vp, i64, vp, i64, i32, i64, vp, vp]),
        "pfop_last_error": (C.c_char_p, []),
        "pfop_attention_split_noalloc": (C.c_int, [vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]),
        "pfop_linear_bench": (C.c_int, [i32, vp, i32, i32, i32, i32, vp, i32, i32, vp, i32, i32,
                                        C.POINTER(C.c_float), vp]),
        "pfop_attention_bench": (C.c_int, [i32, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, i64, i32, i32,
                                           C.POINTER(C.c_float), vp]),
        "pfop_kv_copy_bench": (C.c_int, [i32, vp, i64, vp, i64, i32, i64, vp, i64, i32, i32,
                                         C.POINTER(C.c_float), vp]),
        "pfop_linear_row": (C.c_int, [i32, vp, i32, i32, i32, vp, vp, i32, C.POINTER(C.c_float), vp]),
        "pfop_linear_wait_test": (C.c_int, [i32, vp, i32, i32, i32, vp, i32, i32, vp, i32, vp]),
        "pfop_set_gemm_pairs": (C.c_int, [i32]),
        "pfop_qkv_row_order": (i32, [i32, i32, i32, i32, vp, i32]),
        "pfop_repack_q4": (i64, [vp, i32, i32, i32, vp, i64]),
        "pfop_attention_packed": (C.c_int, [vp, vp, vp, i64, i32, i32, i32, C.POINTER(AttnRun), i32, vp, vp, i64, vp]),
        "pfop_attention_tree": (C.c_int, [vp, vp, vp, i64, i32, i32, i32, C.POINTER(AttnRun), i32, vp, i32, vp, vp,
                                          i64, vp]),
        "pfop_attention_work_bytes": (i64, [i32, i32, i32, C.POINTER(AttnRun), i32]),
        "pfop_attention_status": (C.c_int, [vp, vp]),
        "pfop_logprobs": (C.c_int, [i32, vp, i64, i32, i32, vp, i32, vp, vp, vp, vp, vp]),
        # (the runs by address: a POINTER argument takes ctypes a third of a microsecond)
        "pfop_attention_paged": (C.c_int, [vp, vp, vp, i32, i32, i32, i32, i32, vp, i32, vp, i64, vp, i32, vp, vp, i64,
                                           vp]),
        "pfop_attention_paged_work_bytes": (i64, [i32, i32, i32, C.POINTER(AttnRun), i32]),
        "pfop_attention_paged_status": (C.c_int, [vp, vp]),
        "pfop_qk_norm_rope": (C.c_int, [i32, vp, i64, vp, i64, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, f32, f32,
                                        vp, vp, vp, i64, vp]),
        "pfop_verify_draft": (C.c_int, [i32, vp, i64, vp, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp]),
        "pfop_verify_draft_work_bytes": (i64, [i32, i32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(a) -> int | None:
    """Address of a numpy array, a torch tensor or an int; None stays None."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return a.data_ptr()


def _buffer(a, what: str, dtype: str | None = None, min_elems: int = 0) -> int | None:
    """Byte size of a numpy array or torch tensor handed to the library (None
    for a raw address), after checking what the library cannot see behind a
    pointer: contiguity, element type and element count."""
    if a is None or isinstance(a, int):
        return None
    if isinstance(a, np.ndarray):
        ok, n, dt, nbytes = a.flags["C_CONTIGUOUS"], a.size, str(a.dtype), a.nbytes
    else:
        ok, n, dt = a.is_contiguous(), a.numel(), str(a.dtype).replace("torch.", "")
        nbytes = n * a.element_size()
    if not ok:
        raise ValueError(f"{what}: buffer must be contiguous")
    if dtype is not None and dt != dtype:
        raise ValueError(f"{what}: element type must be {dtype}, got {dt}")
    if n < min_elems:
        raise ValueError(f"{what}: needs at least {min_elems} elements, got {n}")
    return nbytes


def _stream(stream) -> int | None:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def check_op(rc: int):
    if rc != PF_OK:
        raise PrefillError(rc, load().pfop_last_error().decode())


# ---------------------------------------------------------------------------
# model description from a config dict


def make_desc(cfg: dict, max_ctx: int, ubatch_max: int, prune: bool = True, n_seq_max: int = 1,
              embeddings: bool = False, layer_inp=None):
    """layer_inp: None, or n_layer + 1 flags requesting the hidden state
    entering each layer (the last one: the final hidden state)."""
    kv_src = (C.c_int32 * cfg["n_layer"])(*cfg["kv_src"])
    inp = None
    if layer_inp is not None:
        if len(layer_inp) != cfg["n_layer"] + 1:
            raise ValueError("layer_inp needs n_layer + 1 flags")
        inp = (C.c_int32 * (cfg["n_layer"] + 1))(*[1 if f else 0 for f in layer_inp])
    d = ModelDesc(
        n_layer=cfg["n_layer"], n_layer_kv_from_start=cfg["n_layer_kv_from_start"],
        d_model=cfg["d_model"], n_head=cfg["n_head"], n_head_kv=cfg["n_head_kv"],
        head_dim=cfg["head_dim"], ffn_dim=cfg["ffn_dim"], vocab=cfg["vocab"],
        ple_dim=cfg["ple_dim"], ffn_kind=PF_FFN_GEGLU if cfg["ffn"] == "geglu" else PF_FFN_SWIGLU,
        wtype=PF_W_Q4_0 if cfg["wtype"] == "q4_0" else PF_W_F32, rms_eps=cfg["rms_eps"],
        rope_base=cfg["rope_base"], kv_src=C.cast(kv_src, C.POINTER(C.c_int32)), max_ctx=max_ctx,
        ubatch_max=ubatch_max, prune_shared_enable=1 if prune else 0, n_seq_max=n_seq_max,
        embeddings=1 if embeddings else 0,
        embd_layer_inp=C.cast(inp, C.POINTER(C.c_int32)) if inp is not None else None)
    d._keep = (kv_src, inp)
    return d


def prune_predicate(cfg: dict, prune: bool = True, n_seq_max: int = 1, embeddings: bool = False,
                    layer_inp=None) -> bool:
    d = make_desc(cfg, 16, 16, prune, n_seq_max, embeddings, layer_inp)
    rc = load().prefill_prune_predicate(C.byref(d))
    if rc < 0:
        raise PrefillError(rc, "bad description")
    return bool(rc)


def kv_image_bytes_for(n_layers_written: int, n_pos: int, kv_dim: int) -> int:
    return int(load().prefill_kv_image_bytes_for(n_layers_written, n_pos, kv_dim))


def kv_file_check(path: str, n_layers_written: int, kv_dim: int, max_ctx: int) -> tuple[int, int]:
    """(status, positions) of a KV image file checked on the host only."""
    n = C.c_int64(-1)
    rc = load().prefill_kv_file_check(os.fsencode(path), n_layers_written, kv_dim, max_ctx, C.byref(n))
    return rc, n.value


def prefill_with_cache(ctx: "PrefillContext", tokens, ubatch: int, logits, path: str) -> int:
    """The PicoLM flow for a fixed prompt prefix (KV cache article, "usage"):
    if `path` holds a valid image of the prompt's first positions, restore it
    and prefill only the rest; otherwise prefill everything and save the
    cache to `path`.  Returns how many prompt positions came from the file.
    Whether the file was made from the same prefix is the caller's contract
    (the image stores no tokens)."""
    n = len(tokens)
    ctx.reset()
    start = 0
    if os.path.exists(path):
        rc, n_file = kv_file_check(path, ctx.n_layers_written, ctx.kv_dim, ctx.max_ctx)
        if rc == PF_OK and 0 < n_file < n and ctx.kv_load_file(path, n_file) == PF_OK:
            start = n_file
    for i in range(start, n, ubatch):
        ctx.ubatch(tokens[i:i + ubatch], i, i + ubatch >= n, logits)
    if start == 0:
        ctx.sync()
        ctx.kv_save_file(path)
    return start


def kv_header_check(header: bytes, n_layers_written: int, kv_dim: int, n_pos: int, max_ctx: int,
                    image_bytes: int) -> int:
    buf = (C.c_uint8 * 16).from_buffer_copy(header[:16].ljust(16, b"\0"))
    return int(load().prefill_kv_header_check(buf, n_layers_written, kv_dim, n_pos, max_ctx, image_bytes))


def qkv_row_order(Hq: int, Hkv: int, hd: int, with_kv: bool = True):
    """Stored row order of a Q|K|V projection (host only): the source row of
    each stored row in [Wq; Wk; Wv], -1 for padding."""
    import numpy as np
    cap = ((Hq + 2 * Hkv) * hd + 127) // 128 * 128
    out = np.empty(cap, dtype=np.int32)
    n = int(load().pfop_qkv_row_order(Hq, Hkv, hd, 1 if with_kv else 0, out.ctypes.data, cap))
    if n < 0:
        raise PrefillError(n, load().pfop_last_error().decode())
    return out[:n]


def repack_q4(w, bn: int):
    """A Q4_0 matrix [N][K/32][18] in the library's stored tile layout (host
    only), as bytes."""
    import numpy as np
    w = np.ascontiguousarray(w, dtype=np.uint8)
    N, K = w.shape[0], w.shape[1] * 32
    need = int(load().pfop_repack_q4(w.ctypes.data, N, K, bn, None, 0))
    if need < 0:
        raise PrefillError(need, load().pfop_last_error().decode())
    out = np.empty(need, dtype=np.uint8)
    rc = int(load().pfop_repack_q4(w.ctypes.data, N, K, bn, out.ctypes.data, need))
    if rc != need:
        raise PrefillError(rc, load().pfop_last_error().decode())
    return out


# ---------------------------------------------------------------------------
# several sequences in one call: attention and log probabilities


_torch = None


def _t():
    """torch, imported at first use (the library itself does not need it)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _on_device(t, what: str, dtype, shape, index: int) -> int:
    """Address of a contiguous tensor of the given type and shape on CUDA
    device `index`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{what}: element type must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)} does not fit {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{what}: must be on CUDA device {index}, is on {t.device}")
    raise ValueError(f"{what}: buffer must be contiguous")


def _call_on(index: int, stream, fn, *args):
    """fn(*args, stream) with CUDA device `index` current; stream None: the
    device's current torch stream, so that the call is ordered with the torch
    work around it."""
    c = (_torch or _t())._C
    if c._cuda_getDevice() != index:
        with _torch.cuda.device(index):
            return _call_on(index, stream, fn, *args)
    rc = fn(*args, c._cuda_getCurrentRawStream(index) if stream is None else _stream(stream))
    if rc != PF_OK:
        check_op(rc)


def _i32(x, what: str) -> int:
    """x as the int32 of a C argument (ctypes drops what does not fit)."""
    x = int(x)
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{what}: {x} does not fit 32 bits")
    return x


class AttnRuns:
    """The runs of an attention_packed / attention_tree / attention_paged call
    and the call's scratch: runs = [(n_rows, pos0, cell0), ...] (see
    pfop_attn_run; over pages cell0 is the run's first entry in the table), for
    n_head / n_head_kv heads of head_dim.  Kept by a program for as many
    calls as have these runs, and until the last of them is done; calls that
    use one AttnRuns share its scratch, so they must not overlap on the GPU
    (one stream, or events between them; graphs recorded with the same
    AttnRuns may not run at once).  Made outside a recording it may be used on
    any stream; made within one it belongs to that graph."""

    def __init__(self, runs, n_head: int, n_head_kv: int, head_dim: int, device=None):
        torch = _t()
        self._lib = load()
        self.shape = (_i32(n_head, "n_head"), _i32(n_head_kv, "n_head_kv"), _i32(head_dim, "head_dim"))
        runs = [(_i32(n, "n_rows"), _i32(p, "pos0"), _i32(c, "cell0")) for n, p, c in runs]
        self.n_runs = len(runs)
        self.n_rows = sum(r[0] for r in runs)
        self.runs = (AttnRun * max(1, len(runs)))(*[AttnRun(*r) for r in runs])
        self.runs_at = C.addressof(self.runs)
        with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
            self.device = torch.cuda.current_device()
            need = int(self._lib.pfop_attention_paged_work_bytes(*self.shape, self.runs, self.n_runs))
            if need < 0:
                check_op(need)
            self.work = torch.empty(need, dtype=torch.uint8, device="cuda")
            self.work[:4096].zero_()
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()  # a call may come on any stream
        self.work_at, self.work_bytes = self.work.data_ptr(), need

    def check(self, stream=None):
        """Wait for the stream (None: the current one) and raise if a call
        gave up a bounded wait, or met a page id outside its cache."""
        _call_on(self.device, stream, self._lib.pfop_attention_paged_status, self.work_at)

    def _fit(self, q, k, v, out):
        """The number of cells; raises where a buffer does not fit."""
        # (len() of a tensor takes as long as five of these checks)
        hq, hkv, hd = self.shape
        qs, ks, os, d, f16 = q.shape, k.shape, out.shape, self.device, _torch.float16
        if not (q.dtype is f16 and k.dtype is f16 and v.dtype is f16 and out.dtype is _torch.bfloat16
                and len(qs) == 3 and len(ks) == 3 and len(os) == 3 and v.shape == ks
                and qs[0] >= self.n_rows and qs[1] == hq and qs[2] == hd and ks[1] == hkv and ks[2] == hd
                and os[0] >= self.n_rows and os[1] == hq and os[2] == hd
                and q.get_device() == d and k.get_device() == d and v.get_device() == d and out.get_device() == d
                and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
            self._refuse(q, k, v, out)
        return ks[0]

    def _refuse(self, q, k, v, out):
        """Say which buffer does not fit."""
        hq, hkv, hd = self.shape
        for t, what in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
            if t.dim() != 3:
                raise ValueError(f"{what}: needs [rows or cells, heads, head_dim], got {tuple(t.shape)}")
        if len(q) < self.n_rows or len(out) < self.n_rows:
            raise ValueError(f"q and out: the runs have {self.n_rows} rows")
        _on_device(q, "q", _torch.float16, (len(q), hq, hd), self.device)
        _on_device(k, "k", _torch.float16, (len(k), hkv, hd), self.device)
        _on_device(v, "v", _torch.float16, (len(k), hkv, hd), self.device)
        _on_device(out, "out", _torch.bfloat16, (len(out), hq, hd), self.device)


def attention_packed(q, k, v, runs: AttnRuns, out, stream=None):
    """Causal attention of several sequences' rows (pfop_attention_packed):
    q [T, n_head, head_dim] and k, v [n_cells, n_head_kv, head_dim] float16,
    out [T, n_head, head_dim] bfloat16, all on the runs' device.  Enqueued on
    `stream` (None: the current torch stream)."""
    cells = runs._fit(q, k, v, out)
    _call_on(runs.device, stream, runs._lib.pfop_attention_packed, q.data_ptr(), k.data_ptr(), v.data_ptr(), cells,
             *runs.shape, runs.runs, runs.n_runs, out.data_ptr(), runs.work_at, runs.work_bytes)


def _mask_sizes(mask, runs):
    ms = mask.shape
    if len(ms) != 2 or ms[0] < runs.n_rows:
        raise ValueError(f"mask: needs [{runs.n_rows}, words]")
    if ms[1] > 4:
        raise ValueError(f"mask: at most 4 words a row, got {ms[1]}")


def attention_tree(q, k, v, runs: AttnRuns, mask, out, stream=None):
    """Attention of drafted token trees (pfop_attention_tree): as
    attention_packed, with mask [T, words] int64, bit j % 64 of word j / 64
    set where the row sees drafted token j of its run."""
    _mask_sizes(mask, runs)
    cells = runs._fit(q, k, v, out)
    m = _on_device(mask, "mask", _torch.int64, mask.shape, runs.device)
    _call_on(runs.device, stream, runs._lib.pfop_attention_tree, q.data_ptr(), k.data_ptr(), v.data_ptr(), cells,
             *runs.shape, runs.runs, runs.n_runs, m, mask.shape[1], out.data_ptr(), runs.work_at, runs.work_bytes)


def logprobs(logits, tokens=None, logp=None, entropy=None, top_id=None, top_logp=None, stream=None):
    """Log probabilities over the vocabulary (pfop_logprobs): logits [rows,
    vocab] float32 or bfloat16 (rows may be strided: a view of wider rows);
    tokens [rows] int32 with logp [rows] float32; entropy [rows] float32;
    top_id [rows, n] int32 with top_logp [rows, n] float32.  Outputs left
    None are skipped.  Enqueued on `stream` (None: the current torch
    stream)."""
    torch = _t()
    if logits.dtype is torch.float32:
        kind = PF_L_F32
    elif logits.dtype is torch.bfloat16:
        kind = PF_L_BF16
    else:
        raise ValueError(f"logits: element type must be float32 or bfloat16, got {logits.dtype}")
    shape, stride = logits.shape, logits.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError("logits: needs [rows, vocab] with dense rows")
    if (tokens is None) != (logp is None) or (top_id is None) != (top_logp is None):
        raise ValueError("tokens and logp, top_id and top_logp go together")
    rows, vocab = shape
    if rows >= 1 << 31 or vocab >= 1 << 31:
        raise ValueError(f"logits: {tuple(shape)} does not fit 32 bits")
    d = logits.get_device()
    if d < 0:
        raise ValueError(f"logits: must be on a CUDA device, is on {logits.device}")
    f32, i32, one = torch.float32, torch.int32, (rows,)
    n_top = 0 if top_id is None else _i32(top_id.shape[-1], "top_id")
    _call_on(d, stream, load().pfop_logprobs, kind, logits.data_ptr(), stride[0] if rows > 1 else vocab, rows,
             vocab, None if tokens is None else _on_device(tokens, "tokens", i32, one, d), n_top,
             None if logp is None else _on_device(logp, "logp", f32, one, d),
             None if entropy is None else _on_device(entropy, "entropy", f32, one, d),
             None if top_id is None else _on_device(top_id, "top_id", i32, (rows, n_top), d),
             None if top_logp is None else _on_device(top_logp, "top_logp", f32, (rows, n_top), d))


# ---------------------------------------------------------------------------
# a serving step over a paged cache


def attention_paged(q, k, v, runs: AttnRuns, pages, out, mask=None, stream=None):
    """Attention of new tokens over a paged cache (pfop_attention_paged): q
    [T, n_head, head_dim] and k, v [n_pages, page_size, n_head_kv, head_dim]
    float16, pages int32 (the runs' page ids: a run's cell0 counts from its
    first element, row by row where it has two dimensions), out [T, n_head,
    head_dim] bfloat16, mask as for attention_tree (None: causal), all on the
    runs' device.  Enqueued on `stream` (None: the current torch stream)."""
    ks = k.shape
    if len(ks) != 4:
        raise ValueError(f"k and v: need [pages, page size, heads, head_dim], got {tuple(ks)}")
    # (one expression: each of these takes a tenth of a microsecond, a call of one token 8 on the GPU)
    qs, os, d, f16 = q.shape, out.shape, runs.device, _torch.float16
    hq, hkv, hd = runs.shape
    if not (q.dtype is f16 and k.dtype is f16 and v.dtype is f16 and out.dtype is _torch.bfloat16
            and pages.dtype is _torch.int32 and len(qs) == 3 and len(os) == 3 and v.shape == ks
            and qs[0] >= runs.n_rows and qs[1] == hq and qs[2] == hd and ks[2] == hkv and ks[3] == hd
            and os[0] >= runs.n_rows and os[1] == hq and os[2] == hd and q.get_device() == d and k.get_device() == d
            and v.get_device() == d and out.get_device() == d and pages.get_device() == d and q.is_contiguous()
            and k.is_contiguous() and v.is_contiguous() and out.is_contiguous() and pages.is_contiguous()
            and ks[0] < 1 << 31 and ks[1] < 1 << 31):
        _i32(ks[0], "pages of k"), _i32(ks[1], "page size")
        _on_device(k, "k", f16, (*ks[:2], hkv, hd), d)
        _on_device(v, "v", f16, ks, d)
        _on_device(pages, "pages", _torch.int32, pages.shape, d)
        runs._refuse(q, k.view(-1, hkv, hd), v.view(-1, hkv, hd), out)
    m, words = None, 0
    if mask is not None:
        _mask_sizes(mask, runs)
        words = mask.shape[1]
        if words < 1:
            raise ValueError("mask: needs at least a word a row")
        m = _on_device(mask, "mask", _torch.int64, mask.shape, d)
    _call_on(d, stream, runs._lib.pfop_attention_paged, q.data_ptr(), k.data_ptr(), v.data_ptr(),
             ks[0], ks[1], hq, hkv, hd, runs.runs_at, runs.n_runs,
             pages.data_ptr(), pages.numel(), m, words, out.data_ptr(), runs.work_at, runs.work_bytes)


def _vector(t, what: str, dtype, n: int, index: int) -> int:
    """Address of a contiguous tensor of n elements (as _on_device, without
    making a shape to compare with)."""
    if t.dtype is dtype and t.numel() == n and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    return _on_device(t, what, dtype, (n,), index)


def _heads(t, what: str, dtype, index: int):
    """Refuse what is not [rows, heads, head_dim] with a row's heads dense (the
    rows may be parts of wider ones)."""
    if t.dtype is not dtype:
        raise ValueError(f"{what}: element type must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{what}: must be on CUDA device {index}, is on {t.device}")
    (_, h, d), (_, sh, se) = t.shape, t.stride()
    if se != 1 or (h > 1 and sh != d):
        raise ValueError(f"{what}: a row's heads must be dense")


def qk_norm_rope(q, pos, q_out, k=None, v=None, slots=None, k_cache=None, v_cache=None, q_gain=None, k_gain=None,
                 eps=1e-6, rope_base=10000.0, stream=None):
    """Norm and rotation of queries and keys, K and V into the cache
    (pfop_qk_norm_rope): q [T, n_head, head_dim], k, v [T, n_head_kv, head_dim]
    float32 or bfloat16 (rows may be strided: parts of one projection's rows);
    pos, slots [T] int32; q_out [T, n_head, head_dim] float16; k_cache, v_cache
    [cells, n_head_kv, head_dim] or [pages, page size, n_head_kv, head_dim]
    float16; gains [head_dim] float32 (None: no norm).  k None: queries only
    (k_gain is then not looked at).
    Enqueued on `stream` (None: the current torch stream)."""
    torch = _torch or _t()
    dt = q.dtype
    if dt is torch.float32:
        kind = PF_L_F32
    elif dt is torch.bfloat16:
        kind = PF_L_BF16
    else:
        raise ValueError(f"q: element type must be float32 or bfloat16, got {dt}")
    d = q.get_device()
    if d < 0:
        raise ValueError(f"q: must be on a CUDA device, is on {q.device}")
    # One expression a group of tensors: a step of one row takes 2 us on the
    # GPU, a tensor checked in a call of its own 0.6 us here.
    i32, f16, f32, qs = torch.int32, torch.float16, torch.float32, q.shape
    if len(qs) != 3:
        raise ValueError(f"q: needs [rows, heads, head_dim], got {tuple(qs)}")
    rows, hq, hd = qs
    q_ld, sh, se = q.stride()
    if not (se == 1 and (sh == hd or hq == 1) and pos.dtype is i32 and q_out.dtype is f16 and pos.numel() == rows
            and q_out.shape == qs and pos.get_device() == d and q_out.get_device() == d and pos.is_contiguous()
            and q_out.is_contiguous() and rows < 1 << 31 and hq < 1 << 31):
        _heads(q, "q", dt, d)
        _on_device(pos, "pos", i32, qs[:1], d)
        _on_device(q_out, "q_out", f16, qs, d)
        _i32(rows, "rows")
    qga = kga = ka = va = sa = kca = vca = None
    if q_gain is not None:
        qga = _vector(q_gain, "q_gain", f32, hd, d)
    k_ld = v_ld = hkv = cells = 0
    if k is not None:
        if v is None or slots is None or k_cache is None or v_cache is None:
            raise ValueError("k needs v, slots, k_cache and v_cache")
        ks, cs = k.shape, k_cache.shape
        if len(ks) != 3 or ks[0] != rows or ks[1] < 1 or ks[2] != hd or v.shape != ks:
            raise ValueError(f"k and v: shapes {tuple(ks)}, {tuple(v.shape)} do not fit q's {tuple(qs)}")
        hkv = ks[1]
        if len(cs) not in (3, 4) or cs[-2] != hkv or cs[-1] != hd:
            raise ValueError(f"k_cache: shape {tuple(cs)} does not fit {(hkv, hd)}")
        k_ld, sh, se = k.stride()
        v_ld, vsh, vse = v.stride()
        if not (se == 1 and vse == 1 and (hkv == 1 or (sh == hd and vsh == hd)) and k.dtype is dt and v.dtype is dt
                and k_cache.dtype is f16 and v_cache.dtype is f16 and slots.dtype is i32 and v_cache.shape == cs
                and slots.numel() == rows and k.get_device() == d and v.get_device() == d
                and k_cache.get_device() == d and v_cache.get_device() == d and slots.get_device() == d
                and k_cache.is_contiguous() and v_cache.is_contiguous() and slots.is_contiguous()):
            _heads(k, "k", dt, d)
            _heads(v, "v", dt, d)
            _on_device(k_cache, "k_cache", f16, cs, d)
            _on_device(v_cache, "v_cache", f16, cs, d)
            _on_device(slots, "slots", i32, qs[:1], d)
        ka, va, kca, vca, sa = k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), slots.data_ptr()
        cells = cs[0] if len(cs) == 3 else cs[0] * cs[1]
        if k_gain is not None:
            kga = _vector(k_gain, "k_gain", f32, hd, d)
    elif v is not None or slots is not None or k_cache is not None or v_cache is not None:
        raise ValueError("v, slots, k_cache and v_cache go with k")
    if rows < 2:  # (the stride of one row says nothing)
        q_ld, k_ld, v_ld = hq * hd, hkv * hd, hkv * hd
    _call_on(d, stream, (_lib or load()).pfop_qk_norm_rope, kind, q.data_ptr(), q_ld, ka, k_ld, va, v_ld, rows, hq, hkv,
             hd, pos.data_ptr(), sa, qga, kga, eps, rope_base, q_out.data_ptr(), kca, vca, cells)


class VerifyWork:
    """The scratch of verify_draft calls of up to `rows` rows, of any number of
    sequences (n_seq of them: checked only).  Kept until the last call with it
    is done; calls that share one must not overlap on the GPU.  It needs no
    clearing, but like any tensor it is the current stream's: a call on another
    stream comes after that one's work."""

    def __init__(self, rows: int, n_seq: int, device=None):
        torch = _t()
        lib, rows = load(), _i32(rows, "rows")
        need = int(lib.pfop_verify_draft_work_bytes(rows, _i32(n_seq, "n_seq")))
        if need < 0:
            check_op(need)
        need = int(lib.pfop_verify_draft_work_bytes(rows, 0))  # (fewer sequences, more draft rows)
        with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
            self.device = torch.cuda.current_device()
            self.work = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.work_at, self.work_bytes = self.work.data_ptr(), need


def _rows_of(t, what: str, dtype, shape, index: int) -> int:
    """The row stride of logits of this type and shape, their rows dense."""
    if t.shape != shape or t.dtype is not dtype or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: needs {list(shape)} of {dtype} with dense rows")
    if t.get_device() != index:
        raise ValueError(f"{what}: must be on CUDA device {index}, is on {t.device}")
    return t.stride(0) if shape[0] > 1 else shape[1]


def verify_draft(target, tokens, first, u, noise, n_accept, token, p_accept, work: VerifyWork, draft=None,
                 stream=None):
    """Drafted tokens accepted or refused, and the token that follows
    (pfop_verify_draft): target [rows, vocab] and draft [rows - sequences,
    vocab] float32 or bfloat16 (rows may be strided; draft None: drafts without
    a distribution); tokens [rows], first [sequences + 1] int32; u [rows],
    noise [sequences, vocab] float32; outputs n_accept, token [sequences] int32
    and p_accept [rows] float32 (None: not wanted).  Enqueued on `stream` (None:
    the current torch stream)."""
    torch = _torch or _t()
    dt = target.dtype
    if dt is torch.float32:
        kind = PF_L_F32
    elif dt is torch.bfloat16:
        kind = PF_L_BF16
    else:
        raise ValueError(f"target: element type must be float32 or bfloat16, got {dt}")
    ts, n, d, f32, i32 = target.shape, first.numel() - 1, work.device, torch.float32, torch.int32
    if len(ts) != 2:
        raise ValueError(f"target: needs [rows, vocab], got {tuple(ts)}")
    rows, vocab = ts
    if n < 0 or n > rows:
        raise ValueError(f"first: {n + 1} entries do not fit {rows} rows")
    t_ld, se = target.stride()
    ns = noise.shape
    if not ((se == 1 or vocab < 2) and target.get_device() == d and tokens.dtype is i32 and first.dtype is i32
            and u.dtype is f32 and noise.dtype is f32 and n_accept.dtype is i32 and token.dtype is i32 and len(ns) == 2
            and ns[0] == n and ns[1] == vocab and tokens.numel() == rows and u.numel() == rows
            and n_accept.numel() == n and token.numel() == n and tokens.get_device() == d and first.get_device() == d
            and u.get_device() == d and noise.get_device() == d and n_accept.get_device() == d
            and token.get_device() == d and tokens.is_contiguous() and first.is_contiguous() and u.is_contiguous()
            and noise.is_contiguous() and n_accept.is_contiguous() and token.is_contiguous()
            and rows < 1 << 31 and vocab < 1 << 31):
        _i32(rows, "rows"), _i32(vocab, "vocab")
        _rows_of(target, "target", dt, (rows, vocab), d)
        for t, what, dtype, size in ((tokens, "tokens", i32, (rows,)), (first, "first", i32, (n + 1,)),
                                     (u, "u", f32, (rows,)), (noise, "noise", f32, (n, vocab)),
                                     (n_accept, "n_accept", i32, (n,)), (token, "token", i32, (n,))):
            _on_device(t, what, dtype, size, d)
    da, d_ld = None, 0
    if draft is not None:
        d_ld = _rows_of(draft, "draft", dt, (rows - n, vocab), d)
        # (of no rows: an address that no row is read from, since none means drafts without a distribution)
        da = draft.data_ptr() if rows > n else target.data_ptr()
    pa = None
    if p_accept is not None:
        pa = _vector(p_accept, "p_accept", f32, rows, d)
    _call_on(d, stream, (_lib or load()).pfop_verify_draft, kind, target.data_ptr(), t_ld if rows > 1 else vocab, da,
             d_ld, rows, n, vocab, tokens.data_ptr(), first.data_ptr(), u.data_ptr(), noise.data_ptr(),
             n_accept.data_ptr(), token.data_ptr(), pa, work.work_at, work.work_bytes)


# ---------------------------------------------------------------------------
# a prefill context


class PrefillContext:
    """One sequence on the current CUDA device (see prefill.h)."""

    def __init__(self, weights, max_ctx: int, ubatch_max: int, prune: bool = True, stream=None,
                 n_seq_max: int = 1, embeddings: bool = False, layer_inp=None):
        lib = load()
        cfg = weights.cfg
        self.cfg = cfg
        self._desc = make_desc(cfg, max_ctx, ubatch_max, prune, n_seq_max, embeddings, layer_inp)
        keep = []

        def p(a):
            if a is None:
                return None
            a = np.ascontiguousarray(a)
            keep.append(a)
            return a.ctypes.data

        layers = (LayerWeights * cfg["n_layer"])()
        for il, lw in enumerate(weights.layers):
            for k in LayerWeights._fields_:
                setattr(layers[il], k[0], p(lw[k[0]]))
        w = Weights(tok_embd=p(weights.tok_embd), ple_embd=p(weights.ple_embd),
                    out_norm=p(weights.out_norm), layers=C.cast(layers, C.POINTER(LayerWeights)))
        h = C.c_void_p()
        rc = lib.prefill_create(C.byref(self._desc), C.byref(w), _stream(stream), C.byref(h))
        if rc != PF_OK:
            raise PrefillError(rc, lib.prefill_last_error(None).decode())
        self._h = h
        self._lib = lib
        self.vocab = cfg["vocab"]
        self.max_ctx = max_ctx
        self.n_layers_written = min(cfg["n_layer_kv_from_start"], cfg["n_layer"])
        self.kv_dim = cfg["n_head_kv"] * cfg["head_dim"]

    def _check(self, rc):
        if rc != PF_OK:
            raise PrefillError(rc, self._lib.prefill_last_error(self._h).decode())

    def ubatch(self, tokens, pos0: int, is_last: bool, logits=None):
        """tokens: numpy int32 (host) or an int32 device tensor; logits: fp32
        device tensor [vocab] (needed when is_last)."""
        if isinstance(tokens, np.ndarray):
            tokens = np.ascontiguousarray(tokens, dtype=np.int32)
            n = len(tokens)
        else:
            _buffer(tokens, "tokens", "int32")
            n = tokens.numel()
        if is_last:
            _buffer(logits, "logits", "float32", self.cfg["vocab"])
        self._check(self._lib.prefill_ubatch(self._h, _ptr(tokens), n, pos0, 1 if is_last else 0,
                                             _ptr(logits)))

    def set_output(self, which: int, dst):
        """Hidden-state output buffer: which = PF_OUT_EMBD (the embeddings
        output) or a layer index in [0, n_layer]; dst an fp32 device tensor
        with ubatch_max x d_model elements, or None."""
        if dst is not None:
            _buffer(dst, "dst", "float32")
        self._check(self._lib.prefill_set_output(self._h, which, _ptr(dst)))

    def ubatch_seqs(self, tokens, runs, logits=None):
        """Several sequences in one ubatch: runs = [(seq_id, n_tokens,
        is_last), ...] in the order of their tokens; tokens: numpy int32
        (host) or an int32 device tensor holding the runs' tokens one after
        another; logits: fp32 device tensor [number of is_last runs, vocab]."""
        arr = (SeqRun * len(runs))(*[SeqRun(int(q), int(n), 1 if last else 0) for q, n, last in runs])
        if isinstance(tokens, np.ndarray):
            tokens = np.ascontiguousarray(tokens, dtype=np.int32)
        else:
            _buffer(tokens, "tokens", "int32")
        n_last = sum(1 for r in runs if r[2])
        if n_last:
            _buffer(logits, "logits", "float32", n_last * self.cfg["vocab"])
        self._check(self._lib.prefill_ubatch_seqs(self._h, _ptr(tokens), arr, len(runs), _ptr(logits)))

    def graph_capture(self, tokens, pos0: int, is_last: bool, logits=None):
        """Record one ubatch (tokens: int32 device tensor) for graph_launch."""
        _buffer(tokens, "tokens", "int32")
        if is_last:
            _buffer(logits, "logits", "float32", self.cfg["vocab"])
        self._check(self._lib.prefill_graph_capture(self._h, _ptr(tokens), tokens.numel(), pos0,
                                                    1 if is_last else 0, _ptr(logits)))

    def graph_launch(self):
        self._check(self._lib.prefill_graph_launch(self._h))

    def seq_n_pos(self, seq_id: int) -> int:
        return int(self._lib.prefill_seq_n_pos(self._h, seq_id))

    def seq_reset(self, seq_id: int):
        self._check(self._lib.prefill_seq_reset(self._h, seq_id))

    def sync(self):
        self._check(self._lib.prefill_sync(self._h))

    def reset(self):
        self._check(self._lib.prefill_reset(self._h))

    @property
    def n_pos(self) -> int:
        return int(self._lib.prefill_n_pos(self._h))

    def set_prune(self, enable):
        """True / PF_PRUNE_ON, False / PF_PRUNE_OFF, or PF_PRUNE_OFF_PLAIN."""
        mode = enable if isinstance(enable, int) and not isinstance(enable, bool) else (1 if enable else 0)
        self._check(self._lib.prefill_set_prune(self._h, mode))

    @property
    def prune_active(self) -> bool:
        return bool(self._lib.prefill_prune_active(self._h))

    def kv_image_bytes(self, n_pos: int) -> int:
        return int(self._lib.prefill_kv_image_bytes(self._h, n_pos))

    def kv_save(self, dst, nbytes: int):
        size = _buffer(dst, "dst")
        if size is not None and nbytes > size:
            raise ValueError(f"dst: nbytes {nbytes} exceeds the buffer's {size} bytes")
        self._check(self._lib.kv_save(self._h, _ptr(dst), nbytes))

    def kv_load(self, src, nbytes: int, n_pos: int):
        size = _buffer(src, "src")
        if size is not None and nbytes > size:
            raise ValueError(f"src: nbytes {nbytes} exceeds the buffer's {size} bytes")
        self._check(self._lib.kv_load(self._h, _ptr(src), nbytes, n_pos))

    def kv_save_file(self, path: str):
        self._check(self._lib.kv_save_file(self._h, os.fsencode(path)))

    def kv_load_file(self, path: str, n_pos: int = -1) -> int:
        """Restore a KV image file; returns the status (0, or the refusal code,
        in which case the cache is unchanged and a full prefill is due)."""
        rc = self._lib.kv_load_file(self._h, os.fsencode(path), n_pos)
        if rc not in (PF_OK, PF_E_KV_MAGIC, PF_E_KV_SHAPE, PF_E_KV_RANGE, PF_E_IO):
            self._check(rc)
        return rc

    def set_timing(self, enable: bool):
        self._check(self._lib.prefill_set_timing(self._h, 1 if enable else 0))

    def stats(self) -> dict:
        st = Stats()
        self._check(self._lib.prefill_get_stats(self._h, C.byref(st)))
        return {name: dict(launches=st.launches[i], flops=st.flops[i], bytes=st.bytes[i],
                           timed=st.timed[i], ms=st.ms[i]) for i, name in enumerate(KC_NAMES)}

    def reset_stats(self):
        self._check(self._lib.prefill_reset_stats(self._h))

    def close(self):
        if getattr(self, "_h", None):
            self._lib.prefill_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
