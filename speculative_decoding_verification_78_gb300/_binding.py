"""ctypes binding of libspec_verify.so: the C entry points under the same names.

Argument marshalling only: every step of the verify path runs in the library's CUDA kernels.
torch is used for device memory and streams. There is no fallback: when the library is
missing, every call raises.
"""

from __future__ import annotations

import ctypes
import functools
import inspect
import os
import threading

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libspec_verify.so")
# the same kernels compiled with SPEC_CHECKED: computed indices range-checked (SPEC_ERR_CHECK)
CHECKED_LIB_PATH = os.path.join(PKG, "libspec_verify_checked.so")

SPEC_F32, SPEC_BF16, SPEC_F16 = 0, 1, 2
SPEC_OK = 0
SPEC_ERR_NULL, SPEC_ERR_SHAPE, SPEC_ERR_TEMP, SPEC_ERR_DTYPE = -1, -2, -3, -4
SPEC_ERR_WORKSPACE, SPEC_ERR_ALIGN, SPEC_ERR_LAUNCH = -5, -6, -7
SPEC_ERR_NONFINITE, SPEC_ERR_TOKEN, SPEC_ERR_PARENT, SPEC_ERR_CHECK = -20, -21, -22, -24
SPEC_ERR_TIMEOUT = -23
SPEC_ERR_LENGTH, SPEC_ERR_PAGE, SPEC_ERR_POSITION, SPEC_ERR_PATH = -25, -26, -27, -28
SPEC_MAX_V, SPEC_MAX_GAMMA, SPEC_MAX_NODES = 1 << 20, 255, 1024
SPEC_LMHEAD_MAX_V = 1 << 19

# every symbol include/spec_verify.h declares
EXPORTS = ("spec_workspace_bytes", "spec_workspace_init", "spec_verify_chain",
           "spec_verify_tree", "spec_verify_tree_sample", "spec_lmhead_workspace_bytes",
           "spec_verify_chain_lmhead", "spec_probs", "spec_status_string",
           "spec_last_cuda_error", "spec_cuda_error_string",
           "spec_launch_shape", "spec_verify_chain_static", "spec_sample", "spec_topk",
           "spec_tree_mask", "spec_selftest_bounded_wait", "spec_kv_append",
           "spec_kv_attention_workspace_bytes", "spec_kv_attention", "spec_kv_commit")
SPEC_MAX_TOPK = 16
SPEC_STATIC_SCRATCH_BYTES = 4 << 20
SPEC_CALL_CHAIN, SPEC_CALL_TREE, SPEC_CALL_PROBS = 0, 1, 2

_lock = threading.Lock()
_lib = None
_checked_lib = None


class SpecKVCache(ctypes.Structure):
    """spec_kv_cache_t: one layer's paged 8-bit cache as the library sees it."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class SpecError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {spec_status_string(code)} ({code})"
        if code == SPEC_ERR_LAUNCH:
            ce = spec_last_cuda_error()
            if ce:
                msg += f"; CUDA error {ce}: {spec_cuda_error_string(ce)}"
        super().__init__(msg)


def load_library(checked: bool = False):
    """Loads libspec_verify.so (built in-tree by __graft_entry__.build()), or with
    checked=True its checked build libspec_verify_checked.so."""
    global _lib, _checked_lib
    with _lock:
        if (_checked_lib if checked else _lib) is not None:
            return _checked_lib if checked else _lib
        path = CHECKED_LIB_PATH if checked else LIB_PATH
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build the CUDA library first "
                              "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.spec_workspace_bytes.argtypes = [i32, i32, i32, i32]
        lib.spec_workspace_bytes.restype = sz
        lib.spec_workspace_init.argtypes = [vp, sz, vp]
        lib.spec_workspace_init.restype = i32
        lib.spec_verify_chain.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, f32, vp, vp, vp,
                                          vp, sz, vp]
        lib.spec_verify_chain.restype = i32
        lib.spec_verify_tree.argtypes = [vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz,
                                         vp]
        lib.spec_verify_tree.restype = i32
        lib.spec_verify_tree_sample.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, f32,
                                                vp, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_tree_sample.restype = i32
        lib.spec_lmhead_workspace_bytes.argtypes = [i32, i32, i32]
        lib.spec_lmhead_workspace_bytes.restype = sz
        lib.spec_verify_chain_lmhead.argtypes = [vp, vp, i32, vp, vp, i32, vp, vp, i32, i32, i32,
                                                 f32, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_chain_lmhead.restype = i32
        lib.spec_probs.argtypes = [vp, i32, i32, i32, f32, vp, vp, vp, sz, vp]
        lib.spec_probs.restype = i32
        lib.spec_status_string.argtypes = [i32]
        lib.spec_status_string.restype = ctypes.c_char_p
        lib.spec_last_cuda_error.argtypes = []
        lib.spec_last_cuda_error.restype = i32
        lib.spec_cuda_error_string.argtypes = [i32]
        lib.spec_cuda_error_string.restype = ctypes.c_char_p
        lib.spec_launch_shape.argtypes = [i32, i32, i32, i32, i32, f32, vp, vp, vp]
        lib.spec_launch_shape.restype = i32
        lib.spec_verify_chain_static.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, f32, vp, vp,
                                                 vp, vp]
        lib.spec_verify_chain_static.restype = i32
        lib.spec_sample.argtypes = [vp, i32, i32, i32, f32, vp, vp, vp, vp, sz, vp]
        lib.spec_sample.restype = i32
        lib.spec_topk.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]
        lib.spec_topk.restype = i32
        lib.spec_tree_mask.argtypes = [vp, i32, i32, vp, vp, vp]
        lib.spec_tree_mask.restype = i32
        lib.spec_selftest_bounded_wait.argtypes = [vp, ctypes.c_double, vp]
        lib.spec_selftest_bounded_wait.restype = i32
        i64, cache = ctypes.c_int64, ctypes.POINTER(SpecKVCache)
        lib.spec_kv_append.argtypes = [cache, vp, i32, vp, vp, i32, i32, vp, i64, vp, i64, vp, i64,
                                       i32, vp, i32, vp, i32, i32, i32, vp, vp, vp, vp]
        lib.spec_kv_append.restype = i32
        lib.spec_kv_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        lib.spec_kv_attention_workspace_bytes.restype = sz
        lib.spec_kv_attention.argtypes = [cache, vp, i32, vp, vp, i32, i32, vp, i64, i32, i32, f32,
                                          vp, vp, vp, vp, vp, sz, vp]
        lib.spec_kv_attention.restype = i32
        lib.spec_kv_commit.argtypes = [cache, i32, vp, i32, vp, i32, i32, vp, vp, vp, vp, vp]
        lib.spec_kv_commit.restype = i32
        if checked:
            _checked_lib = lib
        else:
            _lib = lib
        return lib


# ------------------------------------------------------------------ marshalling helpers

def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a torch.Tensor, got {type(t)}")
    if t.numel() and not t.is_cuda:
        raise ValueError("device tensor expected (the library takes device pointers)")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else None


def dtype_flag(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype in (torch.bfloat16, torch.int16) or str(t.dtype) == "torch.uint16":
        return SPEC_BF16
    raise TypeError(f"logits must be float32 or bfloat16 (got {t.dtype})")


def _stream(stream):
    if stream is None:
        # the raw handle of torch.cuda.current_stream(), without building the Stream object (several
        # microseconds of a call)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _expect(t, name, numel, dtypes):
    """Raises ValueError / TypeError unless tensor t (when given) holds `numel` elements of one
    of `dtypes`: the library reads and writes exactly that many elements behind each pointer."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements ({tuple(t.shape)}), expected {numel}")


def _chain_shape_check(target_logits, draft_logits, draft_tokens, uniforms, temperature,
                       accept_len, out_tokens, status):
    """(B, gamma, V) of a chain call, after checking every operand against them: the draft
    logits [B, gamma, V] of the target's dtype, int32 tokens [B, gamma], fp32 uniforms
    [B, gamma+1], int32 outputs [B] and [B, gamma+1] and status [1]. NULL (None) operands are
    left to the library's own checks."""
    if not isinstance(target_logits, torch.Tensor) or target_logits.dim() != 3:
        raise ValueError("target_logits must be a [B, gamma+1, V] tensor")
    B, g1, V = target_logits.shape
    gamma = g1 - 1
    if gamma < 0:
        raise ValueError("target_logits must have gamma+1 >= 1 positions")
    dtype_flag(target_logits)
    if draft_logits is not None:
        if draft_logits.dtype != target_logits.dtype:
            raise TypeError(f"draft_logits dtype {draft_logits.dtype} differs from "
                            f"target_logits dtype {target_logits.dtype}")
        _expect(draft_logits, "draft_logits", B * gamma * V, (target_logits.dtype,))
    _expect(draft_tokens, "draft_tokens", B * gamma, (torch.int32,))
    _expect(uniforms, "uniforms", B * (gamma + 1), (torch.float32,))
    _expect(accept_len, "accept_len", B, (torch.int32,))
    _expect(out_tokens, "out_tokens", B * (gamma + 1), (torch.int32,))
    _expect(status, "status", 1, (torch.int32,))
    return B, gamma, V


# ------------------------------------------------------------------ the C entry points

def spec_workspace_bytes(B: int, rows_per_b: int, V: int, dtype: int) -> int:
    return int(load_library().spec_workspace_bytes(B, rows_per_b, V, dtype))


def spec_workspace_init(workspace: torch.Tensor, stream=None) -> int:
    return load_library().spec_workspace_init(_ptr(workspace), _nbytes(workspace), _stream(stream))


def spec_verify_chain(target_logits, draft_logits, draft_tokens, uniforms, temperature,
                      accept_len, out_tokens, status, workspace, stream=None) -> int:
    """target_logits [B, gamma+1, V], draft_logits [B, gamma, V] (fp32 or bf16), draft_tokens
    [B, gamma] int32, uniforms [B, gamma+1] fp32; outputs accept_len [B], out_tokens
    [B, gamma+1] int32; status [1] int32; workspace uint8 (scratch, no initialisation).
    Raises ValueError / TypeError when an operand's size or dtype does not match (B, gamma, V)."""
    B, gamma, V = _chain_shape_check(target_logits, draft_logits, draft_tokens, uniforms,
                                     temperature, accept_len, out_tokens, status)
    return load_library().spec_verify_chain(
        _ptr(target_logits), _ptr(draft_logits), dtype_flag(target_logits), _ptr(draft_tokens),
        _ptr(uniforms), B, gamma, V, float(temperature), _ptr(accept_len), _ptr(out_tokens),
        _ptr(status), _ptr(workspace), _nbytes(workspace), _stream(stream))


def spec_verify_chain_static(target_logits, draft_logits, draft_tokens, uniforms, temperature,
                             accept_len, out_tokens, status, stream=None) -> int:
    """spec_verify_chain with the library's static scratch instead of a workspace (same
    operand checks)."""
    B, gamma, V = _chain_shape_check(target_logits, draft_logits, draft_tokens, uniforms,
                                     temperature, accept_len, out_tokens, status)
    return load_library().spec_verify_chain_static(
        _ptr(target_logits), _ptr(draft_logits), dtype_flag(target_logits), _ptr(draft_tokens),
        _ptr(uniforms), B, gamma, V, float(temperature), _ptr(accept_len), _ptr(out_tokens),
        _ptr(status), _stream(stream))


def spec_verify_tree(target_logits, parents, node_tokens, accept_len, path_nodes, out_tokens,
                     status, workspace, stream=None) -> int:
    """target_logits [B, N, V]; parents, node_tokens [B, N] int32; outputs accept_len [B],
    path_nodes [B, N], out_tokens [B, N] int32."""
    B, N, V = target_logits.shape
    return load_library().spec_verify_tree(
        _ptr(target_logits), dtype_flag(target_logits), _ptr(parents), _ptr(node_tokens), B, N,
        V, _ptr(accept_len), _ptr(path_nodes), _ptr(out_tokens), _ptr(status), _ptr(workspace),
        _nbytes(workspace), _stream(stream))


def spec_verify_tree_sample(target_logits, draft_logits, parents, node_tokens, uniforms,
                            temperature, accept_len, path_nodes, out_tokens, status, workspace,
                            stream=None) -> int:
    """target_logits, draft_logits [B, N, V]; parents, node_tokens [B, N] int32; uniforms [B, N]
    fp32 ([b, 0] the final draw, [b, i] node i's test); outputs as spec_verify_tree."""
    B, N, V = target_logits.shape
    if draft_logits is not None and (draft_logits.dtype != target_logits.dtype or
                                     tuple(draft_logits.shape) != (B, N, V)):
        raise ValueError("draft_logits must match target_logits in dtype and shape")
    _expect(uniforms, "uniforms", B * N, (torch.float32,))
    _expect(parents, "parents", B * N, (torch.int32,))
    _expect(node_tokens, "node_tokens", B * N, (torch.int32,))
    return load_library().spec_verify_tree_sample(
        _ptr(target_logits), _ptr(draft_logits), dtype_flag(target_logits), _ptr(parents),
        _ptr(node_tokens), _ptr(uniforms), B, N, V, float(temperature), _ptr(accept_len),
        _ptr(path_nodes), _ptr(out_tokens), _ptr(status), _ptr(workspace), _nbytes(workspace),
        _stream(stream))


def spec_lmhead_workspace_bytes(B: int, gamma: int, V: int) -> int:
    return int(load_library().spec_lmhead_workspace_bytes(B, gamma, V))


def spec_verify_chain_lmhead(hidden_t, head_t, hidden_d, head_d, draft_tokens, uniforms,
                             temperature, logits_t, logits_d, accept_len, out_tokens, status,
                             workspace, stream=None) -> int:
    """hidden_t [B*(gamma+1), Ht], head_t [V, Ht], hidden_d [B*gamma, Hd], head_d [V, Hd] (bf16);
    draft_tokens [B, gamma] int32, uniforms [B, gamma+1] fp32; logits_t / logits_d bf16 outputs;
    accept_len [B], out_tokens [B, gamma+1] int32; status [1]; workspace uint8."""
    B, gamma = draft_tokens.shape
    V, Ht = head_t.shape
    Hd = head_d.shape[1]
    _expect(head_t, "head_t", V * Ht, (torch.bfloat16,))
    _expect(head_d, "head_d", V * Hd, (torch.bfloat16,))
    _expect(hidden_t, "hidden_t", B * (gamma + 1) * Ht, (torch.bfloat16,))
    _expect(hidden_d, "hidden_d", B * gamma * Hd, (torch.bfloat16,))
    _expect(logits_t, "logits_t", B * (gamma + 1) * V, (torch.bfloat16,))
    _expect(logits_d, "logits_d", B * gamma * V, (torch.bfloat16,))
    _expect(draft_tokens, "draft_tokens", B * gamma, (torch.int32,))
    _expect(uniforms, "uniforms", B * (gamma + 1), (torch.float32,))
    return load_library().spec_verify_chain_lmhead(
        _ptr(hidden_t), _ptr(head_t), Ht, _ptr(hidden_d), _ptr(head_d), Hd, _ptr(draft_tokens),
        _ptr(uniforms), B, gamma, V, float(temperature), _ptr(logits_t), _ptr(logits_d),
        _ptr(accept_len), _ptr(out_tokens), _ptr(status), _ptr(workspace), _nbytes(workspace),
        _stream(stream))


def spec_probs(logits, temperature, out_probs, status, workspace, stream=None) -> int:
    """logits [..., V] -> out_probs [..., V] fp32."""
    V = logits.shape[-1]
    rows = logits.numel() // V if V else 0
    return load_library().spec_probs(
        _ptr(logits), dtype_flag(logits), rows, V, float(temperature), _ptr(out_probs),
        _ptr(status), _ptr(workspace), _nbytes(workspace), _stream(stream))


def spec_launch_shape(kind: int, B: int, rows_per_b: int, V: int, dtype: int,
                      temperature: float = 1.0):
    """(kernels, grid, cluster) of a call of this shape on the current device."""
    k, g, c = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    rc = load_library().spec_launch_shape(kind, B, rows_per_b, V, dtype, float(temperature),
                                          ctypes.byref(k), ctypes.byref(g), ctypes.byref(c))
    if rc != SPEC_OK:
        raise SpecError(rc, "spec_launch_shape")
    return k.value, g.value, c.value


def spec_sample(logits, temperature, uniforms, out_tokens, status, workspace, stream=None) -> int:
    """logits [rows, V] -> out_tokens [rows] int32 (uniforms [rows] fp32)."""
    V = logits.shape[-1]
    rows = logits.numel() // V if V else 0
    return load_library().spec_sample(
        _ptr(logits), dtype_flag(logits), rows, V, float(temperature), _ptr(uniforms),
        _ptr(out_tokens), _ptr(status), _ptr(workspace), _nbytes(workspace), _stream(stream))


def spec_topk(logits, k, out_idx, status, workspace, stream=None) -> int:
    """logits [rows, V] -> out_idx [rows, k] int32."""
    V = logits.shape[-1]
    rows = logits.numel() // V if V else 0
    return load_library().spec_topk(_ptr(logits), dtype_flag(logits), rows, V, int(k),
                                    _ptr(out_idx), _ptr(status), _ptr(workspace),
                                    _nbytes(workspace), _stream(stream))


def spec_tree_mask(parents, mask_words, status, stream=None) -> int:
    """parents [B, N] int32 -> mask_words [B, N, ceil(N/32)] (int32 tensor holding the bits)."""
    B, N = parents.shape
    return load_library().spec_tree_mask(_ptr(parents), B, N, _ptr(mask_words), _ptr(status),
                                         _stream(stream))


def spec_status_string(code: int) -> str:
    try:
        return load_library().spec_status_string(int(code)).decode()
    except ImportError:
        return f"status {code}"


def spec_last_cuda_error() -> int:
    """The cudaError_t behind this thread's last SPEC_ERR_LAUNCH (0 if none)."""
    try:
        return int(load_library().spec_last_cuda_error())
    except ImportError:
        return 0


def spec_cuda_error_string(cuda_error: int) -> str:
    return load_library().spec_cuda_error_string(int(cuda_error)).decode()


def spec_selftest_bounded_wait(status, limit_seconds: float, stream=None) -> int:
    """The bounded-wait self-check (see include/spec_verify.h): returns the SPEC_* code of the
    call; the kernel writes SPEC_ERR_TIMEOUT into status[0] when its waits give up."""
    _expect(status, "status", 1, (torch.int32,))
    return int(load_library().spec_selftest_bounded_wait(_ptr(status), float(limit_seconds),
                                                         _stream(stream)))


# ------------------------------------------------------------------ the paged 8-bit KV cache

_E4M3 = torch.float8_e4m3fn
_KV_DTYPES = {torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}


class KVCache:
    """The paged 8-bit KV cache of one or several layers: k, v [layers, num_pages, kv_heads,
    page_size, head_dim] float8_e4m3fn (or uint8) and k_scale, v_scale [layers, num_pages,
    kv_heads] fp32, all contiguous CUDA tensors that the caller owns; without the layers axis they
    are one layer. Layers share page numbers (one page table serves them all)."""

    def __init__(self, k, v, k_scale, v_scale):
        if not isinstance(k, torch.Tensor) or k.dim() not in (4, 5):
            raise ValueError("k must be a [layers, num_pages, kv_heads, page_size, head_dim] "
                             "tensor (or one layer of it)")
        for t, name, shape in ((v, "v", k.shape), (k_scale, "k_scale", k.shape[:-2]),
                               (v_scale, "v_scale", k.shape[:-2])):
            if not isinstance(t, torch.Tensor) or t.shape != shape:
                raise ValueError(f"{name} must be a {list(shape)} tensor beside k {list(k.shape)}")
        if k.dim() == 4:
            k, v, k_scale, v_scale = (t[None] for t in (k, v, k_scale, v_scale))
        self.layers, self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        for t, name in ((k, "k"), (v, "v")):
            _expect(t, name, k.numel(), (_E4M3, torch.uint8))
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _expect(t, name, self.layers * self.num_pages * self.kv_heads, (torch.float32,))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        ptrs = [_ptr(t).value if t.numel() else 0 for t in (k, v, k_scale, v_scale)]
        page = self.num_pages * self.kv_heads
        steps = [page * self.page_size * self.head_dim] * 2 + [page * 4] * 2
        # (pointers to) the spec_kv_cache_t of each layer
        self._structs = [ctypes.pointer(SpecKVCache(*(p + i * s for p, s in zip(ptrs, steps)),
                                                    self.num_pages, self.page_size, self.kv_heads,
                                                    self.head_dim))
                         for i in range(self.layers)]

    def struct(self, layer=0):
        """A pointer to the spec_kv_cache_t of one layer."""
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of a cache of {self.layers}")
        return self._structs[layer]


def _kv_dtype(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a [B, N, heads, head_dim] tensor")
    flag = _KV_DTYPES.get(t.dtype)
    if flag is None:
        raise TypeError(f"{name} must be bfloat16 or float16 (got {t.dtype})")
    return flag


def _tokens(t, name, B, N, heads, D, dtype):
    """(pointer, token stride) of a [B, N, heads, D] operand whose heads and dims are contiguous
    and whose tokens lie evenly apart."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name}: expected a {dtype} tensor")
    if t.shape != (B, N, heads, D):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(B, N, heads, D)}")
    if not t.numel():
        return None, heads * D
    if not t.is_cuda:
        raise ValueError("device tensor expected (the library takes device pointers)")
    sb, sn, sh, sd = t.stride()
    step = sn if N > 1 else sb if B > 1 else heads * D
    if sd != 1 or (heads > 1 and sh != D) or (B > 1 and N > 1 and sb != N * sn):
        raise ValueError(f"{name}: heads and dims must be contiguous and tokens evenly apart "
                         f"(strides {t.stride()})")
    return t.data_ptr(), step


def _operand(t, name, numel, dtype):
    """The pointer of a contiguous device tensor of `numel` elements of `dtype` (None stays None):
    _expect and _ptr in one pass."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != numel:
        _expect(t, name, numel, (dtype,))
    if not t.is_contiguous() or not t.is_cuda:
        return _ptr(t)   # raises, or an empty tensor
    return t.data_ptr() or None


_I32, _F32 = torch.int32, torch.float32


def _kv_shared(page_table, seq_lens, new_lens, mask, status, B, N):
    """Checks what every KV call takes; returns (pages_per_seq, the five pointers)."""
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or \
            page_table.shape[0] != B:
        raise ValueError(f"page_table must be a [{B}, pages] tensor")
    return (page_table.shape[1], _operand(page_table, "page_table", page_table.numel(), _I32),
            _operand(seq_lens, "seq_lens", B, _I32), _operand(new_lens, "new_lens", B, _I32),
            _operand(mask, "mask", B * N * ((N + 31) // 32), _I32),
            _operand(status, "status", 1, _I32))


def spec_kv_append(cache, layer, page_table, seq_lens, new_lens, k, v, q, q_out, rope, interleaved,
                   positions, mask_words, status, stream=None) -> int:
    """k, v [B, N, kv_heads, D] and q, q_out [B, N, q_heads, D] (bf16 or fp16; q None: no queries);
    page_table [B, pages], seq_lens [B], new_lens [B] or None, positions [B, N] or None int32;
    rope [rows, rope_dim] fp32 or None; mask_words [B, N, ceil(N/32)] int32 or None."""
    flag = _kv_dtype(k, "k")
    B, N = k.shape[:2]
    D, dtype = cache.head_dim, k.dtype
    pps, table, lens, news, mask, st = _kv_shared(page_table, seq_lens, new_lens, mask_words, status,
                                                  B, N)
    kp, ks = _tokens(k, "k", B, N, cache.kv_heads, D, dtype)
    vp, vs = _tokens(v, "v", B, N, cache.kv_heads, D, dtype)
    heads, qp, qs, qo = 0, None, D, None
    if q is not None:
        heads = q.shape[2] if q.dim() == 4 else -1
        qp, qs = _tokens(q, "q", B, N, heads, D, dtype)
        qo = _operand(q_out, "q_out", q.numel(), dtype)
    rows = width = 0
    rp = None
    if rope is not None:
        if not isinstance(rope, torch.Tensor) or rope.dim() != 2:
            raise ValueError("rope must be a [rows, rope_dim] tensor")
        rows, width = rope.shape
        rp = _operand(rope, "rope", rows * width, _F32)
    pos = _operand(positions, "positions", B * N, _I32)
    return load_library().spec_kv_append(
        cache.struct(layer), table, pps, lens, news, B, N, kp, ks, vp, vs, qp, qs, heads, qo, flag,
        rp, rows, width, int(bool(interleaved)), pos, mask, st, _stream(stream))


def spec_kv_attention_workspace_bytes(B: int, N: int, q_heads: int, kv_heads: int,
                                      head_dim: int) -> int:
    return int(load_library().spec_kv_attention_workspace_bytes(B, N, q_heads, kv_heads, head_dim))


def spec_kv_attention(cache, layer, page_table, seq_lens, new_lens, q, scale, mask_words, out, lse,
                      status, workspace, stream=None) -> int:
    """q, out [B, N, q_heads, D] (bf16 or fp16); lse [B, N, q_heads] fp32 or None; workspace uint8
    (scratch); the others as for spec_kv_append."""
    flag = _kv_dtype(q, "q")
    B, N, heads, D = q.shape
    if D != cache.head_dim:
        raise ValueError(f"q: head_dim {D}, the cache's is {cache.head_dim}")
    pps, table, lens, news, mask, st = _kv_shared(page_table, seq_lens, new_lens, mask_words, status,
                                                  B, N)
    qp, qs = _tokens(q, "q", B, N, heads, D, q.dtype)
    return load_library().spec_kv_attention(
        cache.struct(layer), table, pps, lens, news, B, N, qp, qs, heads, flag, float(scale), mask,
        _operand(out, "out", q.numel(), q.dtype), _operand(lse, "lse", B * N * heads, _F32), st,
        _ptr(workspace), _nbytes(workspace), _stream(stream))


def spec_kv_commit(cache, page_table, seq_lens, path_nodes, accept_len, out_lens, status,
                   stream=None) -> int:
    """path_nodes [B, N], accept_len [B] (as spec_verify_tree returns them), out_lens [B] int32:
    every layer of the cache."""
    if not isinstance(path_nodes, torch.Tensor) or path_nodes.dim() != 2:
        raise ValueError("path_nodes must be a [B, N] tensor")
    B, N = path_nodes.shape
    pps, table, lens, _, _, st = _kv_shared(page_table, seq_lens, None, None, status, B, N)
    return load_library().spec_kv_commit(
        cache.struct(0), cache.layers, table, pps, lens, B, N,
        _operand(path_nodes, "path_nodes", B * N, _I32),
        _operand(accept_len, "accept_len", B, _I32), _operand(out_lens, "out_lens", B, _I32), st,
        _stream(stream))


# ------------------------------------------------------------------ conveniences (allocation)

def _torch_stream(stream):
    """The torch stream of what `stream` may be: one of torch's, or a cudaStream_t."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream)   # 0 and 1: the legacy default stream
    return torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()


def _allocates(call):
    """A wrapper that allocates does so on the stream it is given: there an initial value is in place
    before the call starts, and what the wrapper drops when it returns (a workspace) is not handed out
    again before the call has ended. What it returns may be used, and dropped, on the stream that is
    current in the caller."""
    at = list(inspect.signature(call).parameters).index("stream")

    @functools.wraps(call)
    def on_its_stream(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return call(*args, **kw)
        here = torch.cuda.current_stream()
        with torch.cuda.stream(_torch_stream(stream)):
            out = call(*args, **kw)
        for t in out:
            if t is not None and t.is_cuda:
                t.record_stream(here)
        return out

    return on_its_stream


def new_workspace(B: int, rows_per_b: int, V: int, dtype: int, device=None) -> torch.Tensor:
    """A workspace tensor large enough for the given call shape (scratch; never needs zeroing)."""
    n = spec_workspace_bytes(B, rows_per_b, V, dtype)
    if n == 0:
        raise SpecError(SPEC_ERR_SHAPE, "spec_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def check(code: int, where: str) -> None:
    if code != SPEC_OK:
        raise SpecError(code, where)


@_allocates
def verify_chain(target_logits, draft_logits, draft_tokens, uniforms, temperature,
                 workspace=None, stream=None):
    """Allocates the outputs and runs spec_verify_chain. Returns (accept_len, out_tokens,
    status) device tensors."""
    B, g1, V = target_logits.shape
    dev = target_logits.device
    if workspace is None:
        workspace = new_workspace(B, 2 * (g1 - 1) + 1, V, dtype_flag(target_logits), dev)
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    out = torch.empty((B, g1), dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    check(spec_verify_chain(target_logits, draft_logits, draft_tokens, uniforms, temperature,
                            acc, out, st, workspace, stream), "spec_verify_chain")
    return acc, out, st


@_allocates
def verify_tree(target_logits, parents, node_tokens, workspace=None, stream=None):
    """Allocates the outputs and runs spec_verify_tree. Returns (accept_len, path_nodes,
    out_tokens, status) device tensors."""
    B, N, V = target_logits.shape
    dev = target_logits.device
    if workspace is None:
        workspace = new_workspace(B, N, V, dtype_flag(target_logits), dev)
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    path = torch.empty((B, N), dtype=torch.int32, device=dev)
    out = torch.empty((B, N), dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    check(spec_verify_tree(target_logits, parents, node_tokens, acc, path, out, st, workspace,
                           stream), "spec_verify_tree")
    return acc, path, out, st


@_allocates
def verify_tree_sample(target_logits, draft_logits, parents, node_tokens, uniforms, temperature,
                       workspace=None, stream=None):
    """Allocates the outputs and runs spec_verify_tree_sample. Returns (accept_len, path_nodes,
    out_tokens, status) device tensors."""
    B, N, V = target_logits.shape
    dev = target_logits.device
    if workspace is None:
        workspace = new_workspace(B, 2 * N, V, dtype_flag(target_logits), dev)
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    path = torch.empty((B, N), dtype=torch.int32, device=dev)
    out = torch.empty((B, N), dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    check(spec_verify_tree_sample(target_logits, draft_logits, parents, node_tokens, uniforms,
                                  temperature, acc, path, out, st, workspace, stream),
          "spec_verify_tree_sample")
    return acc, path, out, st


@_allocates
def verify_chain_lmhead(hidden_t, head_t, hidden_d, head_d, draft_tokens, uniforms,
                        temperature, workspace=None, stream=None):
    """Allocates the outputs and runs spec_verify_chain_lmhead. Returns (accept_len, out_tokens,
    status, logits_t, logits_d) device tensors."""
    B, gamma = draft_tokens.shape
    V = head_t.shape[0]
    dev = hidden_t.device
    if workspace is None:
        n = spec_lmhead_workspace_bytes(B, gamma, V)
        if n == 0:
            raise SpecError(SPEC_ERR_SHAPE, "spec_lmhead_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    lt = torch.empty((B * (gamma + 1), V), dtype=torch.bfloat16, device=dev)
    ld = torch.empty((B * gamma, V), dtype=torch.bfloat16, device=dev)
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    out = torch.empty((B, gamma + 1), dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    check(spec_verify_chain_lmhead(hidden_t, head_t, hidden_d, head_d, draft_tokens, uniforms,
                                   temperature, lt, ld, acc, out, st, workspace, stream),
          "spec_verify_chain_lmhead")
    return acc, out, st, lt, ld


@_allocates
def probs(logits, temperature, workspace=None, stream=None):
    """Allocates the output and runs spec_probs. Returns (probs fp32, status)."""
    V = logits.shape[-1]
    rows = logits.numel() // V
    dev = logits.device
    if workspace is None:
        workspace = new_workspace(rows, 1, V, dtype_flag(logits), dev)
    out = torch.empty(logits.shape, dtype=torch.float32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    check(spec_probs(logits, temperature, out, st, workspace, stream), "spec_probs")
    return out, st


@_allocates
def sample(logits, temperature, uniforms=None, workspace=None, stream=None):
    """Allocates the output and runs spec_sample. Returns (tokens [rows] int32, status)."""
    V = logits.shape[-1]
    rows = logits.numel() // V
    dev = logits.device
    if workspace is None:
        workspace = new_workspace(rows, 1, V, dtype_flag(logits), dev)
    out = torch.empty(rows, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    check(spec_sample(logits, temperature, uniforms, out, st, workspace, stream), "spec_sample")
    return out, st


@_allocates
def topk(logits, k, workspace=None, stream=None):
    """Allocates the output and runs spec_topk. Returns (indices [rows, k] int32, status)."""
    V = logits.shape[-1]
    rows = logits.numel() // V
    dev = logits.device
    if workspace is None:
        workspace = new_workspace(rows, k, V, dtype_flag(logits), dev)
    out = torch.empty((rows, k), dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    check(spec_topk(logits, k, out, st, workspace, stream), "spec_topk")
    return out, st


@_allocates
def tree_mask(parents, stream=None):
    """Allocates the output and runs spec_tree_mask. Returns (mask words [B, N, W] int32 holding
    the uint32 bit patterns, status)."""
    B, N = parents.shape
    W = (N + 31) // 32
    out = torch.empty((B, N, W), dtype=torch.int32, device=parents.device)
    st = torch.zeros(1, dtype=torch.int32, device=parents.device)
    check(spec_tree_mask(parents, out, st, stream), "spec_tree_mask")
    return out, st


def new_kv_cache(num_pages, kv_heads, head_dim, page_size=64, layers=1, device=None) -> KVCache:
    """An empty paged 8-bit KV cache (its pages need no initial contents)."""
    shape = (layers, num_pages, kv_heads, page_size, head_dim)
    k, v = (torch.empty(shape, dtype=torch.uint8, device=device or "cuda").view(_E4M3)
            for _ in range(2))
    ks, vs = (torch.ones(shape[:3], dtype=torch.float32, device=k.device) for _ in range(2))
    return KVCache(k, v, ks, vs)


def new_attention_workspace(B, N, q_heads, kv_heads, head_dim, device=None) -> torch.Tensor:
    """A workspace for kv_attention calls of this shape (scratch; never needs zeroing)."""
    n = spec_kv_attention_workspace_bytes(B, N, q_heads, kv_heads, head_dim)
    if n == 0:
        raise SpecError(SPEC_ERR_SHAPE, "spec_kv_attention_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


@_allocates
def kv_append(cache, page_table, seq_lens, k, v, q=None, rope=None, layer=0, interleaved=False,
              positions=None, mask=None, new_lens=None, q_out=None, status=None, stream=None):
    """Appends the new tokens' keys (rotated) and values to one layer of the cache and rotates the
    queries (spec_kv_append). Returns (q_out, status); q_out is None without q."""
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=seq_lens.device)
    check(spec_kv_append(cache, layer, page_table, seq_lens, new_lens, k, v, q, q_out, rope,
                         interleaved, positions, mask, status, stream), "spec_kv_append")
    return q_out, status


@_allocates
def kv_attention(cache, page_table, seq_lens, q, scale=None, mask=None, layer=0, new_lens=None,
                 out=None, workspace=None, status=None, return_lse=False, stream=None):
    """Attention of the new tokens over one layer of the cache, which already holds them
    (spec_kv_attention). scale: 1 / sqrt(head_dim) by default. Returns (out, lse, status); lse is
    None unless return_lse."""
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    B, N, heads, D = q.shape
    lse = torch.empty((B, N, heads), dtype=torch.float32, device=q.device) if return_lse else None
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=q.device)
    if workspace is None:
        workspace = new_attention_workspace(B, N, heads, cache.kv_heads, D, q.device)
    if scale is None:
        scale = D ** -0.5
    check(spec_kv_attention(cache, layer, page_table, seq_lens, new_lens, q, scale, mask, out, lse,
                            status, workspace, stream), "spec_kv_attention")
    return out, lse, status


@_allocates
def kv_commit(cache, page_table, seq_lens, path_nodes, accept_len, out_lens=None, status=None,
              stream=None):
    """Keeps the accepted paths of verified trees in every layer of the cache (spec_kv_commit).
    Returns (the sequences' new lengths, status)."""
    if out_lens is None:
        out_lens = torch.empty_like(seq_lens)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=seq_lens.device)
    check(spec_kv_commit(cache, page_table, seq_lens, path_nodes, accept_len, out_lens, status,
                         stream), "spec_kv_commit")
    return out_lens, status
