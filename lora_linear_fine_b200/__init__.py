"""Python binding of the B200 fused LoRA-adapted linear layer (C ABI in
``include/lora_linear.h``).

The functions named like the C entry points (``lora_linear_fwd`` ...) take raw
device pointers (ints) and return the C status code; they only marshal
arguments.  ``forward`` / ``backward`` / ``LoRALinearFunction`` wrap them for
torch tensors (torch provides device memory and the stream).  Every step of the
computation runs in the library's CUDA kernels; there is no fallback: if the
library cannot be loaded, the first call raises ImportError.

The attention-input block (RMSNorm, then the q, k, v projections, q and k
rotated) is a sequence of calls on one stream:

    lora_linear_rmsnorm_fwd(X, g, M, d, eps, Xn, rstd, s)
    lora_linear_fwd_rope(desc_q, rope, Xn, Wq, Aq, Bq, Yq, Tq, ws, n, s)   # q, rotated
    lora_linear_fwd_rope(desc_k, rope, Xn, Wk, Ak, Bk, Yk, Tk, ws, n, s)   # k, rotated
    lora_linear_fwd(desc_v, Xn, Wv, Av, Bv, None, None, None, Yv, Tv, None, ws, n, s)
    lora_linear_bwd_rope(desc_q, rope, dYq, Xn, Wq, Aq, Bq, Tq, dXn, 0, dAq, dBq, ws, n, s)
    lora_linear_bwd_rope(desc_k, rope, dYk, Xn, Wk, Ak, Bk, Tk, dXn, 1, dAk, dBk, ws, n, s)
    lora_linear_bwd_rope(desc_v, None, dYv, Xn, Wv, Av, Bv, Tv, dXn, 1, dAv, dBv, ws, n, s)
    lora_linear_rmsnorm_bwd(X, g, rstd, dXn, M, d, dX, s)

with rope = make_rope_desc(pos, cos, sin, n_pos, head_dim) and dXn an fp32
[M x d] buffer that the q call writes and the k and v calls add to.

The rest of an attention block, as torch functions over a batch of packed
documents (``layer_norm`` in place of the RMSNorm, ``rotary`` for layouts that
the projections' epilogue does not cover, ``attention``):

    plan = AttentionPlan(starts, M)                 # once a batch, for all layers
    cos, sin = rotary_tables(n_pos, rot)            # once a model
    Xn, mean, rstd = layer_norm(X, g, b)
    q, k, v = (forward(Xn, W, A, B, s)[0] for W, A, B in ...)
    q, k = rotary(q, k, pos, cos, sin, head_dim)
    O, lse = attention(q, k, v, plan, heads, kv_heads)
    dq, dk, dv = attention_backward(dO, q, k, v, O, lse, plan, heads, kv_heads)
    dq, dk = rotary(dq, dk, pos, cos, sin, head_dim, inverse=True)
    dX, dg, db = layer_norm_backward(dXn, X, g, mean, rstd)

Like ``forward`` and ``backward`` they record nothing for autograd: outputs do
not require a gradient whatever the inputs do, and a training step calls the
backward functions itself or from the ``backward`` of an autograd.Function of
its own, as ``LoRALinearFunction`` does.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblora_linear.so")

ACT_IDENTITY, ACT_SILU, ACT_SWIGLU = 0, 1, 2
ACT_CODES = {"identity": ACT_IDENTITY, "silu": ACT_SILU, "swiglu": ACT_SWIGLU}

STATUS_NAMES = {
    0: "LORA_OK", 1: "LORA_ERR_INVALID_ARG", 2: "LORA_ERR_ALIGNMENT", 3: "LORA_ERR_UNSUPPORTED",
    4: "LORA_ERR_ARCH", 5: "LORA_ERR_WORKSPACE", 6: "LORA_ERR_CUDA", 7: "LORA_ERR_DEVICE_STATUS",
}

# Every symbol include/lora_linear.h declares.
EXPORTED = ("lora_linear_workspace_size", "lora_linear_workspace_init", "lora_linear_device_status",
            "lora_linear_fwd", "lora_linear_bwd", "lora_status_string", "lora_linear_abi_version",
            "lora_linear_launch_count", "lora_linear_fwd_noalloc", "lora_linear_noalloc_status",
            "lora_linear_timing_enable",
            "lora_linear_timing_read", "lora_linear_selftest_wait_timeout",
            "lora_linear_workspace_size_w4", "lora_linear_dequant_w4", "lora_linear_fwd_w4", "lora_linear_bwd_w4",
            "lora_linear_workspace_size_dropout", "lora_linear_fwd_dropout", "lora_linear_bwd_dropout",
            "lora_linear_w4_tiled_bytes", "lora_linear_w4_tile", "lora_linear_fwd_w4_tiled",
            "lora_linear_rmsnorm_fwd", "lora_linear_rmsnorm_bwd", "lora_linear_workspace_size_rope",
            "lora_linear_fwd_rope", "lora_linear_bwd_rope", "lora_linear_ce_workspace_size",
            "lora_linear_ce_fwd", "lora_linear_ce_bwd", "lora_linear_ce_fwd_bwd",
            "lora_linear_layernorm_fwd", "lora_linear_layernorm_workspace_size", "lora_linear_layernorm_bwd",
            "lora_linear_rotary_tables", "lora_linear_rotary", "lora_linear_attn_plan_size", "lora_linear_attn_plan",
            "lora_linear_attn_fwd", "lora_linear_attn_workspace_size", "lora_linear_attn_bwd")


class LoraLinearDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("d_in", ctypes.c_int64), ("d_out", ctypes.c_int64),
                ("r", ctypes.c_int64), ("s", ctypes.c_float), ("act", ctypes.c_int32)]


class LoraRopeDesc(ctypes.Structure):
    """Rotary tables: pos (int32 [M]), cos / sin (fp32 [n_pos x head_dim/2]) device pointers."""
    _fields_ = [("pos", ctypes.c_void_p), ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
                ("n_pos", ctypes.c_int64), ("head_dim", ctypes.c_int32)]


class LoraCeDesc(ctypes.Structure):
    """Output projection + cross-entropy: M tokens, hidden size d, vocabulary V."""
    _fields_ = [("M", ctypes.c_int64), ("d", ctypes.c_int64), ("V", ctypes.c_int64)]


class LoraRotaryTableDesc(ctypes.Structure):
    """Rotary tables of a (stretched) context; scaling is one of ROTARY_SCALINGS."""
    _fields_ = [("n_pos", ctypes.c_int64), ("rot", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("original", ctypes.c_double), ("amplitude", ctypes.c_double)]


class LoraRotaryDesc(ctypes.Structure):
    """Rotation of finished q and k: the first rot features of each head."""
    _fields_ = [("M", ctypes.c_int64), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32)]


class LoraAttnDesc(ctypes.Structure):
    """Attention over packed documents: M rows, n_docs documents."""
    _fields_ = [("M", ctypes.c_int64), ("n_docs", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("scale", ctypes.c_float), ("softcap", ctypes.c_float)]


class LoraError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m lora_linear_fine_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, u32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(ctypes.c_uint32)
    dp = ctypes.POINTER(LoraLinearDesc)
    lib.lora_linear_workspace_size.argtypes = [dp, i32]
    lib.lora_linear_workspace_size.restype = sz
    lib.lora_linear_workspace_init.argtypes = [vp, sz, vp]
    lib.lora_linear_workspace_init.restype = i32
    lib.lora_linear_device_status.argtypes = [vp, vp, u32p]
    lib.lora_linear_device_status.restype = i32
    lib.lora_linear_fwd.argtypes = [dp] + [vp] * 10 + [vp, sz, vp]
    lib.lora_linear_fwd.restype = i32
    lib.lora_linear_bwd.argtypes = [dp] + [vp] * 15 + [vp, sz, vp]
    lib.lora_linear_bwd.restype = i32
    lib.lora_status_string.argtypes = [i32]
    lib.lora_status_string.restype = ctypes.c_char_p
    lib.lora_linear_abi_version.argtypes = []
    lib.lora_linear_abi_version.restype = i32
    lib.lora_linear_launch_count.argtypes = []
    lib.lora_linear_launch_count.restype = ctypes.c_uint64
    lib.lora_linear_fwd_noalloc.argtypes = [dp] + [vp] * 10 + [vp]
    lib.lora_linear_fwd_noalloc.restype = i32
    lib.lora_linear_noalloc_status.argtypes = [vp, u32p]
    lib.lora_linear_noalloc_status.restype = i32
    lib.lora_linear_timing_enable.argtypes = [i32]
    lib.lora_linear_timing_enable.restype = i32
    dblp, u64p = ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_uint64)
    lib.lora_linear_timing_read.argtypes = [dblp, u64p, dblp, u64p]
    lib.lora_linear_timing_read.restype = i32
    lib.lora_linear_selftest_wait_timeout.argtypes = [vp, sz, i32, vp]
    lib.lora_linear_selftest_wait_timeout.restype = i32
    lib.lora_linear_workspace_size_w4.argtypes = [dp, i32]
    lib.lora_linear_workspace_size_w4.restype = sz
    lib.lora_linear_dequant_w4.argtypes = [vp, vp, ctypes.c_int64, ctypes.c_int64, vp, vp]
    lib.lora_linear_dequant_w4.restype = i32
    lib.lora_linear_fwd_w4.argtypes = [dp] + [vp] * 12 + [vp, sz, vp]
    lib.lora_linear_fwd_w4.restype = i32
    lib.lora_linear_bwd_w4.argtypes = [dp] + [vp] * 17 + [vp, sz, vp]
    lib.lora_linear_bwd_w4.restype = i32
    i64 = ctypes.c_int64
    lib.lora_linear_w4_tiled_bytes.argtypes = [i64, i64]
    lib.lora_linear_w4_tiled_bytes.restype = sz
    lib.lora_linear_w4_tile.argtypes = [vp, i64, i64, vp, vp]
    lib.lora_linear_w4_tile.restype = i32
    lib.lora_linear_fwd_w4_tiled.argtypes = [dp] + [vp] * 8 + [vp, sz, vp]
    lib.lora_linear_fwd_w4_tiled.restype = i32
    f32 = ctypes.c_float
    lib.lora_linear_workspace_size_dropout.argtypes = [dp, i32]
    lib.lora_linear_workspace_size_dropout.restype = sz
    lib.lora_linear_fwd_dropout.argtypes = [dp] + [vp] * 9 + [f32] + [vp] * 3 + [vp, sz, vp]
    lib.lora_linear_fwd_dropout.restype = i32
    lib.lora_linear_bwd_dropout.argtypes = [dp] + [vp] * 10 + [f32] + [vp] * 7 + [vp, sz, vp]
    lib.lora_linear_bwd_dropout.restype = i32
    rp = ctypes.POINTER(LoraRopeDesc)
    lib.lora_linear_rmsnorm_fwd.argtypes = [vp, vp, i64, i64, f32, vp, vp, vp]
    lib.lora_linear_rmsnorm_fwd.restype = i32
    lib.lora_linear_rmsnorm_bwd.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp]
    lib.lora_linear_rmsnorm_bwd.restype = i32
    lib.lora_linear_workspace_size_rope.argtypes = [dp, i32]
    lib.lora_linear_workspace_size_rope.restype = sz
    lib.lora_linear_fwd_rope.argtypes = [dp, rp] + [vp] * 6 + [vp, sz, vp]
    lib.lora_linear_fwd_rope.restype = i32
    lib.lora_linear_bwd_rope.argtypes = [dp, rp] + [vp] * 7 + [i32, vp, vp] + [vp, sz, vp]
    lib.lora_linear_bwd_rope.restype = i32
    cp = ctypes.POINTER(LoraCeDesc)
    lib.lora_linear_ce_workspace_size.argtypes = [cp, i32]
    lib.lora_linear_ce_workspace_size.restype = sz
    lib.lora_linear_ce_fwd.argtypes = [cp] + [vp] * 5 + [vp, sz, vp]
    lib.lora_linear_ce_fwd.restype = i32
    lib.lora_linear_ce_bwd.argtypes = [cp] + [vp] * 6 + [vp, sz, vp]
    lib.lora_linear_ce_bwd.restype = i32
    lib.lora_linear_ce_fwd_bwd.argtypes = [cp] + [vp] * 7 + [vp, sz, vp]
    lib.lora_linear_ce_fwd_bwd.restype = i32
    lib.lora_linear_layernorm_fwd.argtypes = [vp, vp, vp, i64, i64, f32, vp, vp, vp, vp]
    lib.lora_linear_layernorm_fwd.restype = i32
    lib.lora_linear_layernorm_workspace_size.argtypes = [i64, i64]
    lib.lora_linear_layernorm_workspace_size.restype = sz
    lib.lora_linear_layernorm_bwd.argtypes = [vp, i32, vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, sz, vp]
    lib.lora_linear_layernorm_bwd.restype = i32
    lib.lora_linear_rotary_tables.argtypes = [ctypes.POINTER(LoraRotaryTableDesc), vp, vp, vp]
    lib.lora_linear_rotary_tables.restype = i32
    lib.lora_linear_rotary.argtypes = [ctypes.POINTER(LoraRotaryDesc), rp, vp, vp, vp, vp, vp, sz, vp]
    lib.lora_linear_rotary.restype = i32
    lib.lora_linear_attn_plan_size.argtypes = [i64, i64]
    lib.lora_linear_attn_plan_size.restype = sz
    lib.lora_linear_attn_plan.argtypes = [vp, vp, i64, i64, i32, vp, sz, vp]
    lib.lora_linear_attn_plan.restype = i32
    ap = ctypes.POINTER(LoraAttnDesc)
    lib.lora_linear_attn_fwd.argtypes = [ap, vp, sz] + [vp] * 7
    lib.lora_linear_attn_fwd.restype = i32
    lib.lora_linear_attn_workspace_size.argtypes = [ap]
    lib.lora_linear_attn_workspace_size.restype = sz
    lib.lora_linear_attn_bwd.argtypes = [ap, vp, sz] + [vp] * 11 + [sz, vp]
    lib.lora_linear_attn_bwd.restype = i32
    return lib


class _LazyLib:
    """Loads the shared library on first use (so the build script can import
    this package before the library exists); a missing library raises."""

    _h = None

    def __getattr__(self, name):
        if _LazyLib._h is None:
            _LazyLib._h = _load()
        f = getattr(_LazyLib._h, name)
        setattr(self, name, f)
        return f


_lib = _LazyLib()


class _LazyTorch:
    """The torch functions' short way into the library (csrc/lora_torch.cpp),
    loaded on first use like it.  It is bound to one interpreter and one torch;
    where it is absent or does not load, every call declines (None), and the
    functions below go the long way into the same library."""

    def __getattr__(self, name):
        import importlib.util
        import warnings
        import torch  # noqa: F401  (the module is linked with torch's libraries)
        path = os.path.join(_PKG, "_lora_torch.so")
        try:
            spec = importlib.util.spec_from_file_location("_lora_torch", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
        except (ImportError, OSError) as e:
            warnings.warn(f"{path} cannot be loaded ({e}): small calls take some 6 us more; build it with "
                          "`python -m lora_linear_fine_b200.build`", RuntimeWarning, stacklevel=3)
            decline = lambda *args: None
            self.__dict__.update(dict.fromkeys(("layer_norm", "layer_norm_backward", "rotary_tables", "rotary", "attention",
                                                "attention_backward"), decline))
        else:
            self.__dict__.update({k: v for k, v in vars(module).items() if not k.startswith("__")})
        return self.__dict__[name]


_torch = _LazyTorch()


def _done(result, what):
    """The outputs of a call through _torch; a number is its status."""
    if type(result) is int:
        raise LoraError(result, what)
    return result


# ---------------------------------------------------------------------------
# 1:1 wrappers of the C entry points (pointers are ints or None)
# ---------------------------------------------------------------------------
def make_desc(M, d_in, d_out, r, s, act) -> LoraLinearDesc:
    if isinstance(act, str):
        act = ACT_CODES[act]
    return LoraLinearDesc(int(M), int(d_in), int(d_out), int(r), float(s), int(act))


def lora_linear_workspace_size(desc: LoraLinearDesc, for_backward: int) -> int:
    return int(_lib.lora_linear_workspace_size(ctypes.byref(desc), int(for_backward)))


def lora_linear_workspace_init(workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_workspace_init(workspace, workspace_bytes, stream))


def lora_linear_selftest_wait_timeout(workspace, workspace_bytes, limit_log2, stream) -> int:
    return int(_lib.lora_linear_selftest_wait_timeout(workspace, workspace_bytes, int(limit_log2), stream))


def lora_linear_device_status(workspace, stream):
    out = ctypes.c_uint32(0)
    st = int(_lib.lora_linear_device_status(workspace, stream, ctypes.byref(out)))
    return st, int(out.value)


def lora_linear_fwd(desc, X, W, A, B, W_up, A_up, B_up, Y, T_save, Z_save, workspace, workspace_bytes,
                    stream) -> int:
    return int(_lib.lora_linear_fwd(ctypes.byref(desc), X, W, A, B, W_up, A_up, B_up, Y, T_save, Z_save,
                                    workspace, workspace_bytes, stream))


def lora_linear_bwd(desc, dY, X, W, A, B, W_up, A_up, B_up, T_save, Z_save, dX, dA, dB, dA_up, dB_up,
                    workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_bwd(ctypes.byref(desc), dY, X, W, A, B, W_up, A_up, B_up, T_save, Z_save,
                                    dX, dA, dB, dA_up, dB_up, workspace, workspace_bytes, stream))


def lora_linear_fwd_noalloc(desc, X, W, A, B, W_up, A_up, B_up, Y, T_save, Z_save, stream) -> int:
    """The forward for callers that cannot allocate device memory: its scratch
    is a fixed 16 MiB device array inside the library (see the C header)."""
    return int(_lib.lora_linear_fwd_noalloc(ctypes.byref(desc), X, W, A, B, W_up, A_up, B_up, Y, T_save, Z_save,
                                            stream))


def lora_linear_noalloc_status(stream):
    """(status code, status word) of the no-alloc forward's scratch array on the
    current device; synchronises ``stream``."""
    out = ctypes.c_uint32(0)
    st = int(_lib.lora_linear_noalloc_status(stream, ctypes.byref(out)))
    return st, int(out.value)


NOALLOC_SCRATCH_BYTES = 16 << 20


# 4-bit frozen base weight ("w4g64": codes two per byte, low nibble first; one
# bf16 scale per row and 64 input features, group-major; W = bf16(scale * (code - 8)))
def lora_linear_workspace_size_w4(desc: LoraLinearDesc, for_backward: int) -> int:
    return int(_lib.lora_linear_workspace_size_w4(ctypes.byref(desc), int(for_backward)))


def lora_linear_dequant_w4(Wq, Ws, d_out, d_in, W, stream) -> int:
    return int(_lib.lora_linear_dequant_w4(Wq, Ws, int(d_out), int(d_in), W, stream))


def lora_linear_fwd_w4(desc, X, Wq, Ws, A, B, Wq_up, Ws_up, A_up, B_up, Y, T_save, Z_save, workspace,
                       workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_fwd_w4(ctypes.byref(desc), X, Wq, Ws, A, B, Wq_up, Ws_up, A_up, B_up, Y, T_save,
                                       Z_save, workspace, workspace_bytes, stream))


def lora_linear_w4_tiled_bytes(d_out, d_in) -> int:
    return int(_lib.lora_linear_w4_tiled_bytes(int(d_out), int(d_in)))


def lora_linear_w4_tile(Wq, d_out, d_in, Wt, stream) -> int:
    return int(_lib.lora_linear_w4_tile(Wq, int(d_out), int(d_in), Wt, stream))


def lora_linear_fwd_w4_tiled(desc, X, Wt, Ws, A, B, Y, T_save, Z_save, workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_fwd_w4_tiled(ctypes.byref(desc), X, Wt, Ws, A, B, Y, T_save, Z_save, workspace,
                                             workspace_bytes, stream))


def lora_linear_bwd_w4(desc, dY, X, Wq, Ws, A, B, Wq_up, Ws_up, A_up, B_up, T_save, Z_save, dX, dA, dB, dA_up,
                       dB_up, workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_bwd_w4(ctypes.byref(desc), dY, X, Wq, Ws, A, B, Wq_up, Ws_up, A_up, B_up, T_save,
                                       Z_save, dX, dA, dB, dA_up, dB_up, workspace, workspace_bytes, stream))


# RMSNorm prologue and rotary-embedding epilogue of the attention-input projections
def make_rope_desc(pos, cos, sin, n_pos, head_dim) -> LoraRopeDesc:
    return LoraRopeDesc(pos, cos, sin, int(n_pos), int(head_dim))


def lora_linear_rmsnorm_fwd(X, g, M, d, eps, Xn, rstd, stream) -> int:
    return int(_lib.lora_linear_rmsnorm_fwd(X, g, int(M), int(d), float(eps), Xn, rstd, stream))


def lora_linear_rmsnorm_bwd(X, g, rstd, dXn, M, d, dX, stream) -> int:
    """dXn: the fp32 sum of the projections' input gradients."""
    return int(_lib.lora_linear_rmsnorm_bwd(X, g, rstd, dXn, int(M), int(d), dX, stream))


def lora_linear_workspace_size_rope(desc: LoraLinearDesc, for_backward: int) -> int:
    return int(_lib.lora_linear_workspace_size_rope(ctypes.byref(desc), int(for_backward)))


def lora_linear_fwd_rope(desc, rope, X, W, A, B, Y, T_save, workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_fwd_rope(ctypes.byref(desc), ctypes.byref(rope), X, W, A, B, Y, T_save, workspace,
                                         workspace_bytes, stream))


def lora_linear_bwd_rope(desc, rope, dY, X, W, A, B, T_save, dXn, accumulate, dA, dB, workspace, workspace_bytes,
                         stream) -> int:
    """rope None: the projection is not rotated (v).  dXn: fp32, written
    (accumulate 0) or added to (accumulate 1)."""
    return int(_lib.lora_linear_bwd_rope(ctypes.byref(desc), None if rope is None else ctypes.byref(rope), dY, X, W,
                                         A, B, T_save, dXn, int(accumulate), dA, dB, workspace, workspace_bytes,
                                         stream))


# Output projection fused with the cross-entropy loss.
def make_ce_desc(M, d, V) -> LoraCeDesc:
    return LoraCeDesc(int(M), int(d), int(V))


def lora_linear_ce_workspace_size(desc, for_backward) -> int:
    return int(_lib.lora_linear_ce_workspace_size(ctypes.byref(desc), int(for_backward)))


def lora_linear_ce_fwd(desc, H, W, labels, loss, lse, workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_ce_fwd(ctypes.byref(desc), H, W, labels, loss, lse, workspace, workspace_bytes,
                                       stream))


def lora_linear_ce_bwd(desc, H, W, labels, lse, dloss, dH, workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_ce_bwd(ctypes.byref(desc), H, W, labels, lse, dloss, dH, workspace, workspace_bytes,
                                       stream))


def lora_linear_ce_fwd_bwd(desc, H, W, labels, dloss, loss, lse, dH, workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_ce_fwd_bwd(ctypes.byref(desc), H, W, labels, dloss, loss, lse, dH, workspace,
                                           workspace_bytes, stream))


def linear_cross_entropy(H, W, labels, workspace=None, stream=None):
    """(loss, lse): the mean cross-entropy of the logits H W^T against int32
    labels (below 0: ignored), for bf16 H [M x d] and W [V x d] on the current
    device.  lse [M] fp32 is the backward's input."""
    import torch
    M, d = H.shape
    V = W.shape[0]
    desc = make_ce_desc(M, d, V)
    ws = (workspace or Workspace(lora_linear_ce_workspace_size(desc, 0), H.device, stream)).ensure(
        lora_linear_ce_workspace_size(desc, 0), stream)
    loss = torch.empty((), dtype=torch.float32, device=H.device)
    lse = torch.empty(M, dtype=torch.float32, device=H.device)
    _check(lora_linear_ce_fwd(desc, _ptr(H), W.data_ptr(), _ptr(labels), loss.data_ptr(), _ptr(lse),
                              ws.buf.data_ptr(), ws.nbytes, _stream_handle(stream)), "lora_linear_ce_fwd")
    return loss, lse


def linear_cross_entropy_backward(H, W, labels, lse, dloss, workspace=None, stream=None):
    """dH (bf16 [M x d]) = dloss * d(loss)/dH; dloss a 0-d fp32 device tensor."""
    import torch
    M, d = H.shape
    V = W.shape[0]
    desc = make_ce_desc(M, d, V)
    ws = (workspace or Workspace(lora_linear_ce_workspace_size(desc, 1), H.device, stream)).ensure(
        lora_linear_ce_workspace_size(desc, 1), stream)
    dH = torch.empty((M, d), dtype=torch.bfloat16, device=H.device)
    _check(lora_linear_ce_bwd(desc, _ptr(H), W.data_ptr(), _ptr(labels), _ptr(lse), dloss.data_ptr(), _ptr(dH),
                              ws.buf.data_ptr(), ws.nbytes, _stream_handle(stream)), "lora_linear_ce_bwd")
    return dH


def lora_linear_timing_enable(enable: int) -> int:
    return int(_lib.lora_linear_timing_enable(int(enable)))


def lora_linear_timing_read():
    """(status, fwd_gemm_ms, fwd_launches, bwd_gemm_ms, bwd_launches) since the last read."""
    fm, bm = ctypes.c_double(0), ctypes.c_double(0)
    fl, bl = ctypes.c_uint64(0), ctypes.c_uint64(0)
    st = int(_lib.lora_linear_timing_read(ctypes.byref(fm), ctypes.byref(fl), ctypes.byref(bm), ctypes.byref(bl)))
    return st, fm.value, int(fl.value), bm.value, int(bl.value)


def status_string(status: int) -> str:
    s = _lib.lora_status_string(int(status))
    return s.decode() if s else "?"


def lora_linear_abi_version() -> int:
    return int(_lib.lora_linear_abi_version())


def lora_linear_launch_count() -> int:
    return int(_lib.lora_linear_launch_count())


# ---------------------------------------------------------------------------
# torch-tensor convenience layer (device memory + stream only)
# ---------------------------------------------------------------------------
def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(st: int, what: str):
    if st != 0:
        raise LoraError(st, what)


class Workspace:
    """A device workspace (torch uint8 tensor) whose status word is zeroed once."""

    def __init__(self, nbytes: int, device=None, stream=None):
        import torch
        self.nbytes = max(int(nbytes), 256)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        _check(lora_linear_workspace_init(self.buf.data_ptr(), self.nbytes, _stream_handle(stream)),
               "lora_linear_workspace_init")

    def ensure(self, nbytes: int, stream=None):
        if nbytes > self.nbytes:
            self.__init__(nbytes, self.buf.device, stream)
        return self

    def status(self, stream=None):
        st, word = lora_linear_device_status(self.buf.data_ptr(), _stream_handle(stream))
        return word


def forward(X, W, A, B, s, act="identity", W_up=None, A_up=None, B_up=None, save=True, workspace=None,
            stream=None):
    """Y (and the saved T, Z for the backward) for bf16 tensors on the current device."""
    import torch
    M, d_in = X.shape
    d_out = W.shape[0]
    r = 0 if A is None else A.shape[0]
    act_code = ACT_CODES[act] if isinstance(act, str) else act
    desc = make_desc(M, d_in, d_out, r, s, act_code)
    np_ = 2 if act_code == ACT_SWIGLU else 1
    Y = torch.empty((M, d_out), dtype=torch.bfloat16, device=X.device)
    T = torch.empty((np_, M, r), dtype=torch.float32, device=X.device) if (save and r > 0) else None
    Z = (torch.empty((np_, M, d_out), dtype=torch.float32, device=X.device)
         if (save and act_code != ACT_IDENTITY) else None)
    need = lora_linear_workspace_size(desc, 0)
    ws = (workspace or Workspace(need, X.device, stream)).ensure(need, stream)
    _check(lora_linear_fwd(desc, _ptr(X), _ptr(W), _ptr(A), _ptr(B), _ptr(W_up), _ptr(A_up), _ptr(B_up),
                           _ptr(Y), _ptr(T), _ptr(Z), ws.buf.data_ptr(), ws.nbytes, _stream_handle(stream)),
           "lora_linear_fwd")
    return Y, T, Z


def backward(dY, X, W, A, B, s, act="identity", W_up=None, A_up=None, B_up=None, T_save=None, Z_save=None,
             workspace=None, stream=None):
    """dX, dA, dB (and dA_up, dB_up for swiglu)."""
    import torch
    M, d_in = X.shape
    d_out = W.shape[0]
    r = 0 if A is None else A.shape[0]
    act_code = ACT_CODES[act] if isinstance(act, str) else act
    desc = make_desc(M, d_in, d_out, r, s, act_code)
    dX = torch.empty((M, d_in), dtype=torch.bfloat16, device=X.device)
    dA = torch.empty((r, d_in), dtype=torch.float32, device=X.device) if r > 0 else None
    dB = torch.empty((d_out, r), dtype=torch.float32, device=X.device) if r > 0 else None
    sw = act_code == ACT_SWIGLU
    dA_up = torch.empty_like(dA) if (sw and r > 0) else None
    dB_up = torch.empty_like(dB) if (sw and r > 0) else None
    need = lora_linear_workspace_size(desc, 1)
    ws = (workspace or Workspace(need, X.device, stream)).ensure(need, stream)
    _check(lora_linear_bwd(desc, _ptr(dY), _ptr(X), _ptr(W), _ptr(A), _ptr(B), _ptr(W_up), _ptr(A_up),
                           _ptr(B_up), _ptr(T_save), _ptr(Z_save), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(dA_up),
                           _ptr(dB_up), ws.buf.data_ptr(), ws.nbytes, _stream_handle(stream)),
           "lora_linear_bwd")
    return dX, dA, dB, dA_up, dB_up


def _make_autograd():
    import torch

    class LoRALinearFunction(torch.autograd.Function):
        """y = act(x W^T + s (x A^T) B^T) with W frozen; grads for x, A, B.

        A and B are bf16 parameters; their gradients come back from the kernels
        in fp32 and are cast to the parameter dtype by autograd's contract."""

        @staticmethod
        def forward(ctx, X, W, A, B, s, act):
            Y, T, Z = forward(X, W, A, B, s, act)
            ctx.save_for_backward(X, W, A, B, T, Z)
            ctx.s, ctx.act = s, act
            return Y

        @staticmethod
        def backward(ctx, dY):
            X, W, A, B, T, Z = ctx.saved_tensors
            dX, dA, dB, _, _ = backward(dY.contiguous(), X, W, A, B, ctx.s, ctx.act, T_save=T, Z_save=Z)
            return dX, None, dA.to(A.dtype), dB.to(B.dtype), None, None

    return LoRALinearFunction


try:  # torch is optional for the 1:1 C wrappers
    LoRALinearFunction = _make_autograd()
except Exception:  # pragma: no cover
    LoRALinearFunction = None


# dropout on the adapter branch's input (mask: [M x d_in/8] bytes, bit j of byte b keeps element 8b + j)
def lora_linear_workspace_size_dropout(desc: LoraLinearDesc, for_backward: int) -> int:
    return int(_lib.lora_linear_workspace_size_dropout(ctypes.byref(desc), int(for_backward)))


def lora_linear_fwd_dropout(desc, X, W, A, B, W_up, A_up, B_up, mask, mask_up, p_drop, Y, T_save, Z_save,
                            workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_fwd_dropout(ctypes.byref(desc), X, W, A, B, W_up, A_up, B_up, mask, mask_up,
                                            float(p_drop), Y, T_save, Z_save, workspace, workspace_bytes, stream))


def lora_linear_bwd_dropout(desc, dY, X, W, A, B, W_up, A_up, B_up, mask, mask_up, p_drop, T_save, Z_save, dX, dA,
                            dB, dA_up, dB_up, workspace, workspace_bytes, stream) -> int:
    return int(_lib.lora_linear_bwd_dropout(ctypes.byref(desc), dY, X, W, A, B, W_up, A_up, B_up, mask, mask_up,
                                            float(p_drop), T_save, Z_save, dX, dA, dB, dA_up, dB_up, workspace,
                                            workspace_bytes, stream))


def linear_cross_entropy_fwd_bwd(H, W, labels, dloss, workspace=None, stream=None):
    """(loss, lse, dH) in one call, for a loss that is the step's final scalar
    (dloss: its upstream factor, a 0-d fp32 device tensor): the same results
    as linear_cross_entropy followed by linear_cross_entropy_backward, without
    recomputing the logits."""
    import torch
    M, d = H.shape
    V = W.shape[0]
    desc = make_ce_desc(M, d, V)
    ws = (workspace or Workspace(lora_linear_ce_workspace_size(desc, 2), H.device, stream)).ensure(
        lora_linear_ce_workspace_size(desc, 2), stream)
    loss = torch.empty((), dtype=torch.float32, device=H.device)
    lse = torch.empty(M, dtype=torch.float32, device=H.device)
    dH = torch.empty((M, d), dtype=torch.bfloat16, device=H.device)
    _check(lora_linear_ce_fwd_bwd(desc, _ptr(H), W.data_ptr(), _ptr(labels), dloss.data_ptr(), loss.data_ptr(),
                                  _ptr(lse), _ptr(dH), ws.buf.data_ptr(), ws.nbytes, _stream_handle(stream)),
           "lora_linear_ce_fwd_bwd")
    return loss, lse, dH


# ---------------------------------------------------------------------------
# layer norm, rotary positions, attention over packed documents
# ---------------------------------------------------------------------------
ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "wavelength": 3, "ramp": 4}
ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}


def lora_linear_layernorm_fwd(X, g, b, M, d, eps, Y, mean, rstd, stream) -> int:
    return int(_lib.lora_linear_layernorm_fwd(X, g, b, int(M), int(d), float(eps), Y, mean, rstd, stream))


def lora_linear_layernorm_workspace_size(M, d) -> int:
    return int(_lib.lora_linear_layernorm_workspace_size(int(M), int(d)))


def lora_linear_layernorm_bwd(dY, dy_f32, X, g, mean, rstd, M, d, dX, dg, db, workspace, workspace_bytes,
                              stream) -> int:
    return int(_lib.lora_linear_layernorm_bwd(dY, int(dy_f32), X, g, mean, rstd, int(M), int(d), dX, dg, db, workspace,
                                              workspace_bytes, stream))


def make_rotary_table_desc(n_pos, rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192,
                           amplitude=1.0) -> LoraRotaryTableDesc:
    return LoraRotaryTableDesc(int(n_pos), int(rot), ROTARY_SCALINGS.get(scaling, scaling), float(base),
                               float(factor), float(low), float(high), float(original), float(amplitude))


def lora_linear_rotary_tables(desc, cos, sin, stream) -> int:
    return int(_lib.lora_linear_rotary_tables(ctypes.byref(desc), cos, sin, stream))


def make_rotary_desc(M, heads, kv_heads, head_dim, rot, layout="half", inverse=False) -> LoraRotaryDesc:
    return LoraRotaryDesc(int(M), int(heads), int(kv_heads), int(head_dim), int(rot),
                          ROTARY_LAYOUTS.get(layout, layout), int(inverse))


def lora_linear_rotary(desc, rope, Q, K, Yq, Yk, workspace, workspace_bytes, stream) -> int:
    """rope: make_rope_desc(pos, cos, sin, n_pos, head_dim), tables of rot / 2 columns."""
    return int(_lib.lora_linear_rotary(ctypes.byref(desc), ctypes.byref(rope), Q, K, Yq, Yk, workspace,
                                       workspace_bytes, stream))


def lora_linear_attn_plan_size(M, n_docs) -> int:
    return int(_lib.lora_linear_attn_plan_size(int(M), int(n_docs)))


def lora_linear_attn_plan(starts, prefix_len, M, n_docs, causal, plan, plan_bytes, stream) -> int:
    return int(_lib.lora_linear_attn_plan(starts, prefix_len, int(M), int(n_docs), int(causal), plan, plan_bytes,
                                          stream))


def make_attn_desc(M, n_docs, heads, kv_heads, head_dim, causal=True, scale=None, softcap=0.0) -> LoraAttnDesc:
    """scale None: 1 / sqrt(head_dim)."""
    return LoraAttnDesc(int(M), int(n_docs), int(heads), int(kv_heads), int(head_dim), int(causal),
                        float(head_dim) ** -0.5 if scale is None else float(scale), float(softcap))


def lora_linear_attn_fwd(desc, plan, plan_bytes, Q, K, V, slopes, O, lse, stream) -> int:
    return int(_lib.lora_linear_attn_fwd(ctypes.byref(desc), plan, plan_bytes, Q, K, V, slopes, O, lse, stream))


def lora_linear_attn_workspace_size(desc) -> int:
    return int(_lib.lora_linear_attn_workspace_size(ctypes.byref(desc)))


def lora_linear_attn_bwd(desc, plan, plan_bytes, dO, Q, K, V, O, lse, slopes, dQ, dK, dV, workspace, workspace_bytes,
                         stream) -> int:
    return int(_lib.lora_linear_attn_bwd(ctypes.byref(desc), plan, plan_bytes, dO, Q, K, V, O, lse, slopes, dQ, dK, dV,
                                         workspace, workspace_bytes, stream))


def _refuse(what):
    raise LoraError(1, what)


def _tensors(device, *named):
    """Checks (name, tensor or None, dtype, shape): device, type, shape, density.  A dimension of None is any."""
    for name, t, dtype, shape in named:
        if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
            continue
        if t.device != device:
            _refuse(f"{name} is on {t.device}, not {device}")
        if t.dtype != dtype:
            _refuse(f"{name} is {t.dtype}, not {dtype}")
        if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
            _refuse(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if not t.is_contiguous():
            _refuse(f"{name} is not contiguous")


class _On:
    """The device of a call's tensors and its stream (None: that device's
    current stream) as the current ones, so that outputs belong to the stream
    that writes them; the inputs are recorded on a stream of the caller's."""

    def __init__(self, device, stream, *inputs):
        import torch
        if device.type != "cuda":
            _refuse(f"the tensors are on {device}, not on a CUDA device")
        if stream is None:
            self._ctx = torch.cuda.device(device)
            return
        if stream.device != device:
            _refuse(f"the stream is on {stream.device}, not {device}")
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        self._ctx = torch.cuda.stream(stream)

    def __enter__(self):
        self._ctx.__enter__()
        return _stream_handle()

    def __exit__(self, *exc):
        return self._ctx.__exit__(*exc)


def _call(run, device, stream, *inputs):
    """run(stream handle) with the device and the stream of a call as the current ones."""
    import torch
    if stream is None and device.type == "cuda" and torch.cuda.current_device() == device.index:
        return run(torch._C._cuda_getCurrentRawStream(device.index))      # they are
    with _On(device, stream, *inputs) as st:
        return run(st)


def _workspace(workspace, nbytes, device, stream):
    """The workspace of a call, which `stream` (None: the current one) works in."""
    if workspace is None:
        return Workspace(nbytes, device)
    if workspace.buf.device != device:
        _refuse(f"the workspace is on {workspace.buf.device}, not {device}")
    workspace.ensure(nbytes)
    if stream is not None:
        workspace.buf.record_stream(stream)
    return workspace


def layer_norm(X, g, b=None, eps=1e-5, stream=None):
    """(Y, mean, rstd): the layer norm of each row of X (bf16 [M x d]) with
    scale g and shift b (bf16 [d]; b may be None); mean, rstd fp32 [M] are the
    backward's inputs.  Not recorded for autograd: layer_norm_backward gives the
    gradients."""
    import torch
    if stream is None and (out := _torch.layer_norm(X, g, b, eps)) is not None:
        return _done(out, "lora_linear_layernorm_fwd")
    if X.dim() != 2:
        _refuse(f"X has shape {tuple(X.shape)}")
    M, d = X.shape
    bf16, device = torch.bfloat16, X.device
    _tensors(device, ("X", X, bf16, X.shape), ("g", g, bf16, (d,)), ("b", b, bf16, (d,)))

    def run(st):
        Y = torch.empty_like(X)
        mean = torch.empty(M, dtype=torch.float32, device=device)
        rstd = torch.empty_like(mean)
        _check(_lib.lora_linear_layernorm_fwd(X.data_ptr(), g.data_ptr(), _ptr(b), M, d, eps, Y.data_ptr(),
                                              mean.data_ptr(), rstd.data_ptr(), st), "lora_linear_layernorm_fwd")
        return Y, mean, rstd
    return _call(run, device, stream, X, g, b)


def layer_norm_backward(dY, X, g, mean, rstd, bias=True, workspace=None, stream=None):
    """(dX, dg, db) for dY bf16 or fp32 [M x d]; dg, db fp32 [d] (db None
    without ``bias``)."""
    import torch
    if stream is None and workspace is not None and (
            out := _torch.layer_norm_backward(dY, X, g, mean, rstd, bias, workspace.buf)) is not None:
        return _done(out, "lora_linear_layernorm_bwd")
    if X.dim() != 2:
        _refuse(f"X has shape {tuple(X.shape)}")
    M, d = X.shape
    bf16, f32, device = torch.bfloat16, torch.float32, X.device
    if dY.dtype not in (bf16, f32):
        _refuse(f"dY is {dY.dtype}, not bfloat16 or float32")
    _tensors(device, ("dY", dY, dY.dtype, X.shape), ("X", X, bf16, X.shape), ("g", g, bf16, (d,)),
             ("mean", mean, f32, (M,)), ("rstd", rstd, f32, (M,)))

    def run(st):
        dX = torch.empty_like(X)
        dg = torch.empty(d, dtype=f32, device=device)
        db = torch.empty_like(dg) if bias else None
        ws = _workspace(workspace, lora_linear_layernorm_workspace_size(M, d), device, stream)
        _check(_lib.lora_linear_layernorm_bwd(dY.data_ptr(), dY.dtype == f32, X.data_ptr(), g.data_ptr(),
                                              mean.data_ptr(), rstd.data_ptr(), M, d, dX.data_ptr(), dg.data_ptr(),
                                              _ptr(db), ws.buf.data_ptr(), ws.nbytes, st), "lora_linear_layernorm_bwd")
        return dX, dg, db
    return _call(run, device, stream, dY, X, g, mean, rstd)


def rotary_tables(n_pos, rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192,
                  amplitude=1.0, device=None, stream=None):
    """(cos, sin) fp32 [n_pos x rot/2] on ``device`` (default: the current one)
    under a scaling of ROTARY_SCALINGS; low and high are numbers of turns over
    the ``original`` context ("wavelength", "ramp")."""
    import torch
    if scaling not in ROTARY_SCALINGS:
        _refuse(f"scaling {scaling!r} is none of {sorted(ROTARY_SCALINGS)}")
    if n_pos < 0 or rot < 0:
        _refuse(f"n_pos {n_pos}, rot {rot}")
    if device is None and stream is None and torch.cuda.is_initialized() and (
            out := _torch.rotary_tables(n_pos, rot, base, ROTARY_SCALINGS[scaling], factor, low, high, original,
                                        amplitude)) is not None:
        return _done(out, "lora_linear_rotary_tables")
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device()) if stream is None else stream.device
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    desc = make_rotary_table_desc(n_pos, rot, base, scaling, factor, low, high, original, amplitude)

    def run(st):
        cos = torch.empty((n_pos, rot // 2), dtype=torch.float32, device=device)
        sin = torch.empty_like(cos)
        _check(lora_linear_rotary_tables(desc, cos.data_ptr(), sin.data_ptr(), st), "lora_linear_rotary_tables")
        return cos, sin
    return _call(run, device, stream)


def rotary(Q, K, pos, cos, sin, head_dim, layout="half", inverse=False, inplace=False, workspace=None, stream=None):
    """(Yq, Yk): the heads of Q [M x heads * head_dim] and K (bf16; K may be
    None) turned at the int32 positions pos [M] by the tables cos, sin
    [n_pos x rot/2]; the first rot features of each head take part.
    ``inverse`` turns back: the gradients of Q and K from those of Yq and Yk (not
    recorded for autograd).  A position outside the tables leaves its token
    unturned and sets bit 2 of the workspace's status(): pass a workspace to be
    able to read it."""
    import torch
    if stream is None and workspace is not None and not inplace and layout in ROTARY_LAYOUTS and (
            out := _torch.rotary(Q, K, pos, cos, sin, head_dim, ROTARY_LAYOUTS[layout], inverse, workspace.buf)) is not None:
        return _done(out, "lora_linear_rotary")
    if layout not in ROTARY_LAYOUTS:
        _refuse(f"layout {layout!r} is none of {sorted(ROTARY_LAYOUTS)}")
    if Q.dim() != 2 or cos.dim() != 2:
        _refuse(f"Q has shape {tuple(Q.shape)}, cos {tuple(cos.shape)}")
    (M, q_cols), (n_pos, half) = Q.shape, cos.shape
    if head_dim <= 0 or q_cols % head_dim != 0:
        _refuse(f"{q_cols} features are no heads of {head_dim}")
    if K is not None and (K.dim() != 2 or K.shape[1] % head_dim != 0):
        _refuse(f"K's features are no heads of {head_dim}")
    k_cols = 0 if K is None else K.shape[1]
    bf16, f32, device = torch.bfloat16, torch.float32, Q.device
    _tensors(device, ("Q", Q, bf16, Q.shape), ("K", K, bf16, (M, k_cols)), ("pos", pos, torch.int32, (M,)),
             ("cos", cos, f32, cos.shape), ("sin", sin, f32, cos.shape))
    if inplace and K is not None and M > 0 and (Q.data_ptr() < K.data_ptr() + 2 * K.numel() and
                                                K.data_ptr() < Q.data_ptr() + 2 * Q.numel()):
        _refuse("Q and K overlap: in place each would be turned twice")

    def run(st):
        Yq = Q if inplace else torch.empty_like(Q)
        Yk = K if inplace or K is None else torch.empty_like(K)
        ws = _workspace(workspace, 256, device, stream)
        desc = LoraRotaryDesc(M, q_cols // head_dim, k_cols // head_dim, head_dim, 2 * half, ROTARY_LAYOUTS[layout],
                              bool(inverse))
        rope = LoraRopeDesc(pos.data_ptr(), cos.data_ptr(), sin.data_ptr(), n_pos, head_dim)
        _check(_lib.lora_linear_rotary(desc, rope, Q.data_ptr(), _ptr(K), Yq.data_ptr(), _ptr(Yk), ws.buf.data_ptr(),
                                       ws.nbytes, st), "lora_linear_rotary")
        return Yq, Yk
    return _call(run, device, stream, Q, K, pos, cos, sin)


class AttentionPlan:
    """The documents of a batch of M rows as tiles, for ``attention`` and
    ``attention_backward`` of every layer: starts (int32 [n_docs + 1], on the
    GPU) holds the documents' first rows and the end of the last one.  Without
    ``causal`` a row sees its whole document, with it the rows up to itself and
    the first prefix_len (int32 [n_docs]) rows of its document.  The offsets are
    checked on the GPU: status() is 2 if they were not valid, and attention on
    such a plan computes nothing, so that its outputs hold whatever their memory
    held.  A batch whose offsets are not known to be good reads status() (which
    waits for the stream) before it uses them."""

    def __init__(self, starts, M, prefix_len=None, causal=True, stream=None):
        import torch
        if starts.dim() != 1 or starts.numel() < 1:
            _refuse(f"starts has shape {tuple(starts.shape)}")
        n = starts.numel() - 1
        _tensors(starts.device, ("starts", starts, torch.int32, (n + 1,)), ("prefix_len", prefix_len, torch.int32, (n,)))
        self.M, self.n_docs, self.causal, self.nbytes = int(M), n, bool(causal), lora_linear_attn_plan_size(M, n)
        if self.nbytes <= 0:
            _refuse(f"{M} rows in {n} documents")

        def run(st):
            buf = torch.empty(self.nbytes, dtype=torch.uint8, device=starts.device)
            _check(_lib.lora_linear_attn_plan(starts.data_ptr(), _ptr(prefix_len), self.M, n, self.causal,
                                              buf.data_ptr(), self.nbytes, st), "lora_linear_attn_plan")
            return buf
        self.buf = _call(run, starts.device, stream, starts, prefix_len)

    def status(self, stream=None):
        import torch
        with torch.cuda.device(self.buf.device):
            return lora_linear_device_status(self.buf.data_ptr(), _stream_handle(stream))[1]


def _attention_args(Q, K, V, plan, heads, kv_heads, scale, softcap, slopes):
    import torch
    if Q.dim() != 2 or heads <= 0 or kv_heads <= 0 or Q.shape[1] % heads != 0:
        _refuse(f"Q has shape {tuple(Q.shape)} for {heads} heads")
    M, cols = Q.shape
    D, bf16 = cols // heads, torch.bfloat16
    if M != plan.M:
        _refuse(f"{M} rows with a plan of {plan.M}")
    kv = (M, kv_heads * D)
    _tensors(Q.device, ("Q", Q, bf16, Q.shape), ("K", K, bf16, kv), ("V", V, bf16, kv),
             ("slopes", slopes, torch.float32, (heads,)), ("the plan", plan.buf, torch.uint8, (plan.nbytes,)))
    return LoraAttnDesc(M, plan.n_docs, heads, kv_heads, D, plan.causal, D ** -0.5 if scale is None else scale, softcap)


def attention(Q, K, V, plan, heads, kv_heads, scale=None, softcap=0.0, slopes=None, stream=None):
    """(O, lse): attention of Q (bf16 [M x heads * head_dim]) over K, V (bf16
    [M x kv_heads * head_dim]) within the plan's documents; scale None is
    1 / sqrt(head_dim), softcap caps the scores by a tanh, slopes (fp32
    [heads]) subtract slope * |i - j|.  lse fp32 [M x heads] is the backward's
    input.  Not recorded for autograd: attention_backward gives the gradients.
    With a plan whose status() is not 0 the outputs are not written."""
    import torch
    if stream is None and (out := _torch.attention(Q, K, V, plan.buf, plan.M, plan.n_docs, plan.causal, heads, kv_heads,
                                                   scale, softcap, slopes)) is not None:
        return _done(out, "lora_linear_attn_fwd")
    desc = _attention_args(Q, K, V, plan, heads, kv_heads, scale, softcap, slopes)
    device = Q.device

    def run(st):
        O = torch.empty_like(Q)
        lse = torch.empty((plan.M, heads), dtype=torch.float32, device=device)
        _check(_lib.lora_linear_attn_fwd(desc, plan.buf.data_ptr(), plan.nbytes, Q.data_ptr(), K.data_ptr(),
                                         V.data_ptr(), _ptr(slopes), O.data_ptr(), lse.data_ptr(), st),
               "lora_linear_attn_fwd")
        return O, lse
    return _call(run, device, stream, Q, K, V, slopes, plan.buf)


def attention_backward(dO, Q, K, V, O, lse, plan, heads, kv_heads, scale=None, softcap=0.0, slopes=None,
                       workspace=None, stream=None):
    """(dQ, dK, dV) of ``attention`` for its O and lse; not written with a plan
    whose status() is not 0."""
    import torch
    if stream is None and workspace is not None and (
            out := _torch.attention_backward(dO, Q, K, V, O, lse, plan.buf, plan.M, plan.n_docs, plan.causal, heads,
                                             kv_heads, scale, softcap, slopes, workspace.buf)) is not None:
        return _done(out, "lora_linear_attn_bwd")
    desc = _attention_args(Q, K, V, plan, heads, kv_heads, scale, softcap, slopes)
    device = Q.device
    _tensors(device, ("dO", dO, torch.bfloat16, Q.shape), ("O", O, torch.bfloat16, Q.shape),
             ("lse", lse, torch.float32, (plan.M, heads)))

    def run(st):
        dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
        ws = _workspace(workspace, _lib.lora_linear_attn_workspace_size(desc), device, stream)
        _check(_lib.lora_linear_attn_bwd(desc, plan.buf.data_ptr(), plan.nbytes, dO.data_ptr(), Q.data_ptr(),
                                         K.data_ptr(), V.data_ptr(), O.data_ptr(), lse.data_ptr(), _ptr(slopes),
                                         dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), ws.buf.data_ptr(), ws.nbytes, st),
               "lora_linear_attn_bwd")
        return dQ, dK, dV
    return _call(run, device, stream, dO, Q, K, V, O, lse, slopes, plan.buf)
