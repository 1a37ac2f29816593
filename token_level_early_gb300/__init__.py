"""River-LLM token-level early-exit decode on GB300 (sm_103a).

Thin ctypes binding of librv.so (C ABI in include/rv.h).  Every step of the
decode path runs in the library's CUDA kernels; this module only marshals
arguments and raises RVError on a non-zero status.  There is no CPU fallback:
loading fails loudly when librv.so is missing.
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import concurrent.futures as _fut
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
LIB_PATH = os.path.join(_HERE, "librv.so")
_CSRC = os.path.join(_HERE, "csrc")
_BUILD = os.path.join(_ROOT, "_build")
SOURCES = ["api.cu", "decode_b1.cu", "attention.cu", "general.cu", "quant.cu", "noalloc.cu", "stream.cu", "gemm_tc.cu", "rows_mma.cu",
           "rope.cu", "kv8.cu", "kv8_attention.cu", "kv8_attention_e4m3.cu"]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"

RV_OK, RV_EINVAL, RV_ENOMEM, RV_ECUDA, RV_ECAPACITY, RV_ESTATE, RV_ETIMEOUT = 0, -1, -2, -3, -4, -5, -6
PROJ_Q, PROJ_K, PROJ_V, PROJ_O, PROJ_GATE, PROJ_UP, PROJ_DOWN = range(7)
DUMP_HIDDEN, DUMP_S, DUMP_LOGITS, DUMP_KV, DUMP_LENS = range(5)
EXPORTED = ("rv_last_error", "rv_load_model", "rv_quantize_river", "rv_export_river", "rv_prefill",
            "rv_decode_step", "rv_decode_step_dev", "rv_sync_status", "rv_kv_reset", "rv_set_debug",
            "rv_debug_dump", "rv_kv_bytes", "rv_param_bytes", "rv_free_model", "rv_time_kernel", "rv_greedy_head_noalloc", "rv_offload_backbone",
            "rv_set_option", "rv_debug_fail_alloc", "rv_decode_attention_plan",
            "rv_rope_init", "rv_rope", "rv_kv8_append", "rv_kv8_read", "rv_kv8_attention", "rv_kv8_attention_workspace",
            "rv_set_rope", "rv_kv_cache_bytes")
OPT_DECODE_ENGINE, ENGINE_CHAIN, ENGINE_PERSISTENT = 0, 0, 1
OPT_QUANTIZER, QUANT_RTN, QUANT_HQQ = 1, 0, 1
OPT_WAIT_LIMIT_US = 2
OPT_KV_CACHE, KV_16BIT, KV_INT8, KV_E4M3 = 3, 0, 1, 2
F16, BF16, F32 = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_BANDS, ROPE_RAMP = range(5)
KV8_INT8, KV8_E4M3 = 0, 1
TIME_GATEUP, TIME_O, TIME_LMHEAD, TIME_ATTN = 0, 1, 2, 3


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def build(verbose: bool = False) -> str:
    """Compile librv.so for sm_103a (one translation unit per source, in parallel)."""
    os.makedirs(_BUILD, exist_ok=True)
    flags = [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-O3",
             "--expt-relaxed-constexpr"]
    hdrs = [os.path.join(_CSRC, h) for h in os.listdir(_CSRC) if h.endswith(".cuh")]
    hdrs.append(os.path.join(_ROOT, "include", "rv.h"))
    newest_hdr = max(os.path.getmtime(h) for h in hdrs)

    def one(src):
        s = os.path.join(_CSRC, src)
        o = os.path.join(_BUILD, src.replace(".cu", ".o"))
        if os.path.exists(o) and os.path.getmtime(o) >= max(os.path.getmtime(s), newest_hdr):
            return o
        cmd = [nvcc(), *flags, "-c", s, "-o", o]
        if verbose:
            print(" ".join(cmd))
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return o

    with _fut.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(one, SOURCES))
    cmd = [nvcc(), ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-rpath,/usr/local/cuda/lib64", *objs,
           "-o", LIB_PATH]
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    return LIB_PATH


class RVConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("d_model", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("vocab", ctypes.c_int), ("tied_embed", ctypes.c_int), ("act_dtype", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("max_batch", ctypes.c_int), ("max_seq", ctypes.c_int)]


class Heads(ctypes.Structure):
    """rv_heads: a device tensor [B][T][heads][head_dim] (strides in elements); see also heads()."""
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int), ("heads", ctypes.c_int),
                ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("scaling", ctypes.c_int), ("original_max_position", ctypes.c_int), ("theta", ctypes.c_double),
                ("factor", ctypes.c_double), ("low_freq_factor", ctypes.c_double),
                ("high_freq_factor", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("attention_factor", ctypes.c_double)]


class RopePlan(ctypes.Structure):
    """rv_rope_plan, as rope_plan() fills it in."""
    _fields_ = [("head_dim", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("attention_factor", ctypes.c_float), ("turns", ctypes.c_uint64 * 128)]


class KV8(ctypes.Structure):
    """rv_kv8: an 8-bit K/V cache of one layer in the caller's device memory
    (k_codes .. v_tail are device pointers; layouts in include/rv.h)."""
    _fields_ = [("max_batch", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("max_seq", ctypes.c_int), ("block", ctypes.c_int), ("format", ctypes.c_int),
                ("act_dtype", ctypes.c_int), ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("k_tail", ctypes.c_void_p),
                ("v_tail", ctypes.c_void_p)]


class RVError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"rv error {code}: {msg}")
        self.code = code


_lib = None


def lib():
    """Load librv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first (token_level_early_gb300.build())")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    sig = {
        "rv_last_error": ([], ctypes.c_char_p),
        "rv_load_model": ([ctypes.POINTER(RVConfig), vp, vp, ctypes.POINTER(vp)], i32),
        "rv_quantize_river": ([vp, i32, i32], i32),
        "rv_export_river": ([vp, i32, i32, vp, vp, vp], i32),
        "rv_prefill": ([vp, vp, i32, i32, f32, i32, vp, vp], i32),
        "rv_decode_step": ([vp, vp, i32, f32, vp, vp, vp], i32),
        "rv_decode_step_dev": ([vp, vp, i32, f32, vp, vp, vp], i32),
        "rv_sync_status": ([vp], i32),
        "rv_kv_reset": ([vp, vp, i32], i32),
        "rv_set_debug": ([vp, i32], i32),
        "rv_debug_dump": ([vp, i32, vp, sz], i32),
        "rv_kv_bytes": ([vp], sz),
        "rv_param_bytes": ([vp, i32], sz),
        "rv_offload_backbone": ([vp, i32], i32),
        "rv_free_model": ([vp], None),
        "rv_time_kernel": ([vp, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_float),
                            ctypes.POINTER(ctypes.c_double)], i32),
        "rv_greedy_head_noalloc": ([vp, vp, vp, i32, i32, i32, f32, vp, vp, vp], i32),
        "rv_set_option": ([vp, i32, i32], i32),
        "rv_debug_fail_alloc": ([i32], i32),
        "rv_decode_attention_plan": ([i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32)], i32),
    }
    hp, kp, rp = ctypes.POINTER(Heads), ctypes.POINTER(KV8), ctypes.POINTER(RopePlan)
    sig.update({
        "rv_rope_init": ([ctypes.POINTER(RopeConfig), rp], i32),
        "rv_rope": ([rp, hp, hp, hp, hp, i32, i32, vp, vp, i32, vp], i32),
        "rv_kv8_append": ([kp, hp, hp, i32, i32, vp, vp, vp, vp], i32),
        "rv_kv8_read": ([kp, hp, hp, i32, i32, vp, vp, vp, vp], i32),
        "rv_kv8_attention": ([kp, hp, hp, i32, i32, f32, vp, vp, vp, vp, sz, vp], i32),
        "rv_kv8_attention_workspace": ([kp, i32, i32, i32], sz),
        "rv_set_rope": ([vp, ctypes.POINTER(RopeConfig)], i32),
        "rv_kv_cache_bytes": ([vp], sz),
    })
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def _check(rc: int):
    if rc != RV_OK:
        raise RVError(rc, lib().rv_last_error().decode(errors="replace"))


def _p(a):
    return None if a is None else a.ctypes.data


def greedy_head_noalloc(d_lm_head: int, d_final_norm: int, d_h: int, vocab: int, d_model: int, act_dtype: int,
                        rms_eps: float, d_next_id: int, d_logits: Optional[int] = None, stream: Optional[int] = None):
    """rv_greedy_head_noalloc on device pointers (see include/rv.h)."""
    _check(lib().rv_greedy_head_noalloc(d_lm_head, d_final_norm, d_h, vocab, d_model, act_dtype, float(rms_eps),
                                        d_next_id, d_logits, stream))


def decode_attention_plan(batch: int, n_kv_heads: int, n_sm: int, max_cluster: int, max_splits: int,
                          context: int):
    """rv_decode_attention_plan (host arithmetic, no GPU needed): returns
    (plan, splits), plan 0 = cluster plan, 1 = global-merge plan."""
    sp = ctypes.c_int(0)
    rc = lib().rv_decode_attention_plan(batch, n_kv_heads, n_sm, max_cluster, max_splits, context, ctypes.byref(sp))
    if rc < 0:
        _check(rc)
    return rc, sp.value


def debug_fail_alloc(after: int) -> None:
    """Test hook: the device allocation after the next `after` ones fails
    (once); after < 0 turns it off (rv_debug_fail_alloc)."""
    _check(lib().rv_debug_fail_alloc(int(after)))


_DTYPES = {"torch.float16": F16, "torch.bfloat16": BF16, "torch.float32": F32}


def heads(tensor) -> Heads:
    """Heads of a torch CUDA tensor [B][T][heads][head_dim] (any strides with a
    contiguous last dimension); the tensor must outlive the calls that use it."""
    if tensor.dim() != 4 or (tensor.shape[-1] > 1 and tensor.stride(-1) != 1):
        raise ValueError("a [B][T][heads][head_dim] tensor with a contiguous last dimension is needed")
    if str(tensor.dtype) not in _DTYPES:
        raise ValueError(f"unsupported dtype {tensor.dtype}")
    sb, st, sh, _ = tensor.stride()
    return Heads(tensor.data_ptr(), _DTYPES[str(tensor.dtype)], tensor.shape[2], sb, st, sh)


def rope_plan(head_dim: int, rotary_dim: Optional[int] = None, layout: int = ROPE_HALF, theta: float = 10000.0,
              scaling: int = ROPE_PLAIN, factor: float = 1.0, low_freq_factor: float = 1.0,
              high_freq_factor: float = 4.0, original_max_position: int = 0, beta_fast: float = 32.0,
              beta_slow: float = 1.0, attention_factor: float = 0.0) -> RopePlan:
    """rv_rope_init: the plan of a rotary configuration (host arithmetic, no GPU needed)."""
    cfg = RopeConfig(head_dim, head_dim if rotary_dim is None else rotary_dim, layout, scaling, original_max_position,
                     theta, factor, low_freq_factor, high_freq_factor, beta_fast, beta_slow, attention_factor)
    plan = RopePlan()
    _check(lib().rv_rope_init(ctypes.byref(cfg), ctypes.byref(plan)))
    return plan


def rope(plan: RopePlan, q_in: Heads, q_out: Heads, k_in: Optional[Heads], k_out: Optional[Heads], B: int, T: int,
         d_pos: Optional[int], d_count: Optional[int] = None, inverse: bool = False, stream: Optional[int] = None):
    """rv_rope: rotate query and key heads (inverse: the gradient's direction)."""
    _check(lib().rv_rope(plan, q_in, q_out, k_in, k_out, B, T, d_pos, d_count, inverse, stream))


def kv8_append(cache: KV8, k: Heads, v: Heads, B: int, T: int, d_pos: Optional[int], d_count: Optional[int] = None,
               d_err: Optional[int] = None, stream: Optional[int] = None):
    """rv_kv8_append: quantise new K/V into the cache."""
    _check(lib().rv_kv8_append(cache, k, v, B, T, d_pos, d_count, d_err, stream))


def kv8_read(cache: KV8, k_out: Optional[Heads], v_out: Optional[Heads], B: int, T: int, d_pos: Optional[int],
             d_count: Optional[int] = None, d_err: Optional[int] = None, stream: Optional[int] = None):
    """rv_kv8_read: read positions of the cache back as values."""
    _check(lib().rv_kv8_read(cache, k_out, v_out, B, T, d_pos, d_count, d_err, stream))


def kv8_attention_workspace(cache: KV8, B: int, T: int, n_heads: int) -> int:
    """rv_kv8_attention_workspace: bytes of workspace for kv8_attention."""
    n = lib().rv_kv8_attention_workspace(cache, B, T, n_heads)
    if n == 0 and lib().rv_last_error():
        raise RVError(RV_EINVAL, lib().rv_last_error().decode(errors="replace"))
    return int(n)


def kv8_attention(cache: KV8, q: Heads, out: Heads, B: int, T: int, scale: float, d_pos: Optional[int],
                  d_count: Optional[int], d_lse: Optional[int], workspace: Optional[int], workspace_bytes: int,
                  stream: Optional[int] = None):
    """rv_kv8_attention: attention of T new tokens per row over the cache."""
    _check(lib().rv_kv8_attention(cache, q, out, B, T, scale, d_pos, d_count, d_lse, workspace, workspace_bytes,
                                  stream))


def config_of(shape, max_batch: int, max_seq: int) -> RVConfig:
    return RVConfig(shape.n_layers, shape.d_model, shape.n_heads, shape.n_kv_heads, shape.head_dim, shape.ffn,
                    shape.vocab, shape.tied_embed, shape.act_dtype, shape.rms_eps, shape.rope_theta, max_batch,
                    max_seq)


class Model:
    """A backbone on the GPU with its river and KV cache (owns an rv_model)."""

    def __init__(self, shape, weights: Sequence[Optional[np.ndarray]], max_batch: int, max_seq: int,
                 stream: Optional[int] = None):
        self.shape = shape
        self.max_batch, self.max_seq = max_batch, max_seq
        ws = [None if w is None else np.ascontiguousarray(w, dtype=np.uint16) for w in weights]
        ptrs = (ctypes.c_void_p * len(ws))(*[_p(w) for w in ws])
        self._cfg = config_of(shape, max_batch, max_seq)
        h = ctypes.c_void_p()
        _check(lib().rv_load_model(ctypes.byref(self._cfg), ptrs, stream, ctypes.byref(h)))
        self._h = h
        self.group = None

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib().rv_free_model(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def proj_dims(self, proj: int):
        s = self.shape
        d, qd, kvd = s.d_model, s.n_heads * s.head_dim, s.n_kv_heads * s.head_dim
        return [(qd, d), (kvd, d), (kvd, d), (d, qd), (s.ffn, d), (s.ffn, d), (d, s.ffn)][proj]

    def quantize_river(self, group: int, entry_layer: int = 1):
        _check(lib().rv_quantize_river(self._h, group, entry_layer))
        self.group = group

    def export_river(self, layer: int, proj: int):
        N, K = self.proj_dims(proj)
        G = -(-K // self.group)
        q = np.zeros((N, K // 8), dtype=np.uint32)
        s = np.zeros((N, G), dtype=np.uint16)
        z = np.zeros((N, G), dtype=np.uint16)
        _check(lib().rv_export_river(self._h, layer, proj, _p(q), _p(s), _p(z)))
        return q, s, z

    def prefill(self, tokens: np.ndarray, tau: float, fixed_exit: int = -1):
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        B, T0 = t.shape
        nxt = np.zeros(B, dtype=np.int32)
        ex = np.zeros(B, dtype=np.int32)
        _check(lib().rv_prefill(self._h, _p(t), B, T0, float(tau), int(fixed_exit), _p(nxt), _p(ex)))
        return nxt, ex

    def decode_step(self, tokens, tau: float, forced=None):
        t = np.ascontiguousarray(tokens, dtype=np.int32).reshape(-1)
        B = t.size
        f = None if forced is None else np.ascontiguousarray(forced, dtype=np.int32).reshape(-1)
        nxt = np.zeros(B, dtype=np.int32)
        ex = np.zeros(B, dtype=np.int32)
        _check(lib().rv_decode_step(self._h, _p(t), B, float(tau), _p(f), _p(nxt), _p(ex)))
        return nxt, ex

    def decode_step_dev(self, d_tokens: int, B: int, tau: float, d_forced: Optional[int], d_next: int,
                        d_exit: int):
        _check(lib().rv_decode_step_dev(self._h, d_tokens, B, float(tau), d_forced, d_next, d_exit))

    def sync_status(self):
        _check(lib().rv_sync_status(self._h))

    def kv_reset(self, rows=None):
        if rows is None:
            _check(lib().rv_kv_reset(self._h, None, 0))
        else:
            r = np.ascontiguousarray(rows, dtype=np.int32)
            _check(lib().rv_kv_reset(self._h, _p(r), r.size))

    def set_option(self, option: int, value: int):
        _check(lib().rv_set_option(self._h, option, value))

    def set_engine(self, engine: int):
        self.set_option(OPT_DECODE_ENGINE, engine)

    def set_quantizer(self, method: int):
        """River quantizer of the next quantize_river: QUANT_RTN or QUANT_HQQ."""
        self.set_option(OPT_QUANTIZER, method)

    def set_kv_cache(self, kind: int):
        """KV_16BIT, KV_INT8 or KV_E4M3; forgets every cached position."""
        self.set_option(OPT_KV_CACHE, kind)

    def set_rope(self, config: Optional[RopeConfig]):
        """Rotary frequencies for long contexts (None: the model's own); forgets every cached position."""
        _check(lib().rv_set_rope(self._h, None if config is None else ctypes.byref(config)))

    def set_debug(self, enable: bool):
        _check(lib().rv_set_debug(self._h, 1 if enable else 0))

    def dump(self, what: int) -> np.ndarray:
        s, B = self.shape, self.max_batch
        if what == DUMP_HIDDEN:
            a = np.zeros((s.n_layers + 1, B, s.d_model), dtype=np.float32)
        elif what == DUMP_S:
            a = np.zeros((s.n_layers, B), dtype=np.float32)
        elif what == DUMP_LOGITS:
            a = np.zeros((B, s.vocab), dtype=np.float32)
        elif what == DUMP_KV:
            a = np.zeros((s.n_layers, 2, B, s.n_kv_heads, self.max_seq, s.head_dim), dtype=np.uint16)
        elif what == DUMP_LENS:
            a = np.zeros(B, dtype=np.int32)
        else:
            raise ValueError(what)
        _check(lib().rv_debug_dump(self._h, what, _p(a), a.nbytes))
        return a

    def time_kernel(self, kind: int, layer: int, river: bool, iters: int):
        """Mean device ms per launch and algorithmic bytes per launch of one GEMV kernel."""
        ms = ctypes.c_float(0)
        by = ctypes.c_double(0)
        _check(lib().rv_time_kernel(self._h, kind, layer, 1 if river else 0, iters, ctypes.byref(ms),
                                    ctypes.byref(by)))
        return float(ms.value), float(by.value)

    def kv_bytes(self) -> int:
        return int(lib().rv_kv_bytes(self._h))

    def kv_cache_bytes(self) -> int:
        """Device bytes of the K/V cache (kv_bytes: of its dump)."""
        return int(lib().rv_kv_cache_bytes(self._h))

    def offload_backbone(self, keep_layers: int) -> None:
        """Free backbone layers keep_layers+1..L on the device; exits are capped at keep_layers."""
        _check(lib().rv_offload_backbone(self._h, int(keep_layers)))

    def param_bytes(self, which: int) -> int:
        return int(lib().rv_param_bytes(self._h, which))
