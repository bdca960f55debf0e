"""ctypes binding of libskinny (include/skinny.h): argument marshalling only.

Every computation runs in the CUDA kernels of libskinny.so.  There is no CPU
or PyTorch fallback: if the library is missing or fails to load, importing the
package raises.  PyTorch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libskinny.so")

STATUS = {
    0: "SK_OK",
    1: "SK_ERR_INVALID_ARG",
    2: "SK_ERR_UNSUPPORTED_SHAPE",
    3: "SK_ERR_MISALIGNED",
    4: "SK_ERR_NOT_INITIALIZED",
    5: "SK_ERR_CUDA",
    6: "SK_ERR_TIMEOUT",
    7: "SK_ERR_WORKSPACE",
}
SK_OK = 0
SK_ERR_INVALID_ARG, SK_ERR_UNSUPPORTED_SHAPE, SK_ERR_MISALIGNED = 1, 2, 3
SK_ERR_NOT_INITIALIZED, SK_ERR_CUDA, SK_ERR_TIMEOUT, SK_ERR_WORKSPACE = 4, 5, 6, 7


class SkinnyError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.sk_status_string(status).decode()} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(LIB_PATH)
    p, i, f, ll, d = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_double
    sig = {
        "sk_init": ([ctypes.c_size_t], i),
        "sk_shutdown": ([], i),
        "sk_stream_workspace": ([p, ctypes.c_size_t], i),
        "nvfp4_gemm": ([p, p, p, f, p, i, i, i, p], i),
        "nvfp4_gemm_f16out": ([p, p, p, f, p, i, i, i, p], i),
        "fp8_gemm": ([p, p, p, p, i, i, i, p], i),
        "fp8_gemm_f16out": ([p, p, p, p, i, i, i, p], i),
        "lm_head_argmax": ([p, p, p, f, p, p, i, i, i, p], i),
        "lm_head_verify": ([p, p, p, f, p, p, p, p, i, i, i, p], i),
        "fp8_quantize": ([p, p, p, i, i, p], i),
        "lm_head_sample": ([p, p, p, f, p, p, f, i, f, p, i, i, i, p], i),
        "nvfp4_quantize": ([p, p, p, p, i, i, p], i),
        "sk_status_string": ([i], ctypes.c_char_p),
        "sk_last_device_error": ([p], i),
        "sk_set_pdl": ([i], i),
        "sk_set_variant": ([i], i),
        "sk_version": ([], i),
        "sk_inject_wait_timeout": ([i], None),
        "nvfp4_gemm_noalloc": ([p, p, p, f, p, i, i, i, p], i),
        "kv4_append": ([p, ll, p, ll, p, p, f, f, p, p, i, i, i, i, i, p], i),
        "kv4_attention": ([p, ll, p, p, p, f, f, f, p, p, p, p, i, i, i, i, i, i, i, i, p], i),
        "kv4_evict": ([p, p, p, p, p, p, p, p, i, i, i, i, i, i, i, i, i, p], i),
        "rope_frequencies": ([p, i, i, d, d, d, d, d], i),
        "qk_norm_rope": ([p, ll, p, ll, p, p, p, p, d, d, p, ll, p, ll, i, i, i, i, i, i, p], i),
        "kv4_append_rope": ([p, ll, p, ll, p, ll, p, p, p, p, p, d, d, p, ll, p, f, f, i, i, i, i, i, i, i, i, p], i),
        "kv4_window_attention": ([p, ll, p, p, p, f, f, f, i, i, p, p, i, i, i, i, i, i, i, i, p], i),
        "kv4_chunk_attention": ([p, ll, p, p, p, p, f, f, f, i, i, p, p, i, i, i, i, i, i, i, i, p], i),
        "token_logprobs": ([p, i, ll, p, f, i, p, p, p, p, p, i, i, p], i),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


lib = _load()

# Names declared in include/skinny.h (the tests check that each is exported).
EXPORTS = ("sk_init", "sk_shutdown", "sk_stream_workspace", "nvfp4_gemm", "nvfp4_gemm_f16out", "fp8_gemm",
           "fp8_gemm_f16out", "lm_head_argmax", "lm_head_verify", "lm_head_sample", "fp8_quantize",
           "nvfp4_quantize", "kv4_append", "kv4_attention", "kv4_evict", "rope_frequencies", "qk_norm_rope",
           "kv4_append_rope", "kv4_window_attention", "kv4_chunk_attention", "token_logprobs",
           "sk_status_string", "sk_last_device_error",
           "sk_set_pdl", "sk_set_variant", "sk_inject_wait_timeout", "nvfp4_gemm_noalloc", "sk_version")


def _check(status: int, what: str) -> None:
    if status != SK_OK:
        raise SkinnyError(status, what)


def status_string(status: int) -> str:
    return lib.sk_status_string(int(status)).decode()


def init(workspace_bytes: int = 0) -> None:
    """sk_init on the current CUDA device (call once per device, before graph capture)."""
    _check(lib.sk_init(int(workspace_bytes)), "sk_init")


def shutdown() -> None:
    _check(lib.sk_shutdown(), "sk_shutdown")


def stream_workspace(stream, workspace_bytes: int = 64 << 20) -> None:
    """sk_stream_workspace: a workspace of its own for `stream` (a torch CUDA
    stream) on the current device; 0 bytes removes it."""
    _check(lib.sk_stream_workspace(_stream_ptr(stream), int(workspace_bytes)), "sk_stream_workspace")


def set_pdl(enable: bool) -> bool:
    return bool(lib.sk_set_pdl(1 if enable else 0))


VARIANT_AUTO, VARIANT_TENSOR, VARIANT_SIMT = 0, 1, 2


def set_variant(variant: int) -> int:
    """Kernel variant (VARIANT_AUTO, VARIANT_TENSOR or VARIANT_SIMT); returns the previous one."""
    prev = int(lib.sk_set_variant(int(variant)))
    if prev < 0:
        raise ValueError(f"unknown kernel variant {variant}")
    return prev


def _stream_ptr(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream))


def last_device_error(stream=None) -> int:
    """Synchronise `stream`; return the status of the device error word (and clear it)."""
    return int(lib.sk_last_device_error(_stream_ptr(stream)))


def _dims(x, codes, nv: bool):
    import torch

    if x.dtype != torch.float16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError("x must be a 2-D CUDA float16 tensor [M][K]")
    if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_cuda:
        raise TypeError("W_codes must be a 2-D CUDA uint8 tensor")
    for t in (x, codes):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    M, K = x.shape
    N = codes.shape[0]
    if codes.shape[1] != (K // 2 if nv else K):
        raise ValueError(f"W_codes has shape {tuple(codes.shape)}, expected [N][{K // 2 if nv else K}]")
    return int(M), int(N), int(K)


def nvfp4_gemm(x, W_codes, W_scales, W_gscale: float, y=None, f16_out: bool = False, stream=None):
    """y[M][N] = x . dequant(W)^T for NVFP4 weights (FP32 output, or FP16 with f16_out)."""
    import torch

    M, N, K = _dims(x, W_codes, True)
    if W_scales.dtype != torch.uint8 or tuple(W_scales.shape) != (N, K // 16) or not W_scales.is_contiguous():
        raise ValueError("W_scales must be a contiguous uint8 tensor [N][K/16]")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16 if f16_out else torch.float32, device=x.device)
    fn = lib.nvfp4_gemm_f16out if f16_out else lib.nvfp4_gemm
    _check(fn(x.data_ptr(), W_codes.data_ptr(), W_scales.data_ptr(), float(W_gscale), y.data_ptr(),
              M, N, K, _stream_ptr(stream)), "nvfp4_gemm")
    return y


def fp8_gemm(x, W_codes, W_scales, y=None, f16_out: bool = False, stream=None):
    """y[M][N] = x . dequant(W)^T for FP8-E4M3 weights with 128x128 FP32 block scales."""
    import torch

    M, N, K = _dims(x, W_codes, False)
    if W_scales.dtype != torch.float32 or tuple(W_scales.shape) != ((N + 127) // 128, (K + 127) // 128) \
            or not W_scales.is_contiguous():
        raise ValueError("W_scales must be a contiguous float32 tensor [ceil(N/128)][ceil(K/128)]")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16 if f16_out else torch.float32, device=x.device)
    fn = lib.fp8_gemm_f16out if f16_out else lib.fp8_gemm
    _check(fn(x.data_ptr(), W_codes.data_ptr(), W_scales.data_ptr(), y.data_ptr(), M, N, K,
              _stream_ptr(stream)), "fp8_gemm")
    return y


def lm_head_argmax(x, W_codes, W_scales, W_gscale: float, logits=None, argmax=None,
                   want_logits: bool = True, stream=None):
    """NVFP4 vocabulary projection with the fused per-row argmax.

    Returns (logits or None, argmax int32 [M])."""
    import torch

    M, N, K = _dims(x, W_codes, True)
    if W_scales.dtype != torch.uint8 or tuple(W_scales.shape) != (N, K // 16) or not W_scales.is_contiguous():
        raise ValueError("W_scales must be a contiguous uint8 tensor [N][K/16]")
    if logits is None and want_logits:
        logits = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if argmax is None:
        argmax = torch.empty((M,), dtype=torch.int32, device=x.device)
    _check(lib.lm_head_argmax(x.data_ptr(), W_codes.data_ptr(), W_scales.data_ptr(), float(W_gscale),
                              logits.data_ptr() if logits is not None else None, argmax.data_ptr(),
                              M, N, K, _stream_ptr(stream)), "lm_head_argmax")
    return logits, argmax


def lm_head_verify(x, W_codes, W_scales, W_gscale: float, draft, logits=None, argmax=None, accept=None,
                   want_logits: bool = True, stream=None):
    """lm_head_argmax plus the greedy verification of a speculative round:
    draft is int32 [M - 1] on the device (ignored when M == 1).

    Returns (logits or None, argmax int32 [M], accept int32 [2] = (accepted drafts, bonus token))."""
    import torch

    M, N, K = _dims(x, W_codes, True)
    if W_scales.dtype != torch.uint8 or tuple(W_scales.shape) != (N, K // 16) or not W_scales.is_contiguous():
        raise ValueError("W_scales must be a contiguous uint8 tensor [N][K/16]")
    if M > 1 and (draft is None or draft.dtype != torch.int32 or not draft.is_cuda or draft.numel() < M - 1
                  or not draft.is_contiguous()):
        raise ValueError("draft must be a contiguous CUDA int32 tensor of at least M - 1 tokens")
    if logits is None and want_logits:
        logits = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if argmax is None:
        argmax = torch.empty((M,), dtype=torch.int32, device=x.device)
    if accept is None:
        accept = torch.empty((2,), dtype=torch.int32, device=x.device)
    _check(lib.lm_head_verify(x.data_ptr(), W_codes.data_ptr(), W_scales.data_ptr(), float(W_gscale),
                              logits.data_ptr() if logits is not None else None, argmax.data_ptr(),
                              draft.data_ptr() if (draft is not None and M > 1) else None, accept.data_ptr(),
                              M, N, K, _stream_ptr(stream)), "lm_head_verify")
    return logits, argmax, accept


def _weights_f16(w):
    import torch

    if w.dtype != torch.float16 or w.dim() != 2 or not w.is_cuda or not w.is_contiguous():
        raise TypeError("w must be a contiguous 2-D CUDA float16 tensor [N][K]")
    return int(w.shape[0]), int(w.shape[1])


def fp8_quantize(w, stream=None):
    """FP16 [N][K] -> (codes uint8 [N][K], scales float32 [ceil(N/128)][ceil(K/128)])."""
    import torch

    N, K = _weights_f16(w)
    codes = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    scales = torch.empty(((N + 127) // 128, (K + 127) // 128), dtype=torch.float32, device=w.device)
    _check(lib.fp8_quantize(w.data_ptr(), codes.data_ptr(), scales.data_ptr(), N, K, _stream_ptr(stream)),
           "fp8_quantize")
    return codes, scales


def nvfp4_quantize(w, stream=None):
    """FP16 [N][K] -> (codes uint8 [N][K/2], scales uint8 [N][K/16], tensor scale float32 [1], on the device)."""
    import torch

    N, K = _weights_f16(w)
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device=w.device)
    gscale = torch.empty((1,), dtype=torch.float32, device=w.device)
    _check(lib.nvfp4_quantize(w.data_ptr(), codes.data_ptr(), scales.data_ptr(), gscale.data_ptr(), N, K,
                              _stream_ptr(stream)), "nvfp4_quantize")
    return codes, scales, gscale


def lm_head_sample(x, W_codes, W_scales, W_gscale: float, u, temperature: float, top_k: int, top_p: float,
                   logits=None, token=None, stream=None):
    """NVFP4 vocabulary projection with a sampled pick per row (temperature /
    top-k / top-p; u is a float32 CUDA tensor of M uniforms in [0, 1)).

    Returns (logits float32 [M][N], token int32 [M])."""
    import torch

    M, N, K = _dims(x, W_codes, True)
    if W_scales.dtype != torch.uint8 or tuple(W_scales.shape) != (N, K // 16) or not W_scales.is_contiguous():
        raise ValueError("W_scales must be a contiguous uint8 tensor [N][K/16]")
    if u.dtype != torch.float32 or not u.is_cuda or u.numel() < M or not u.is_contiguous():
        raise ValueError("u must be a contiguous CUDA float32 tensor of at least M uniforms")
    if logits is None:
        logits = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if token is None:
        token = torch.empty((M,), dtype=torch.int32, device=x.device)
    _check(lib.lm_head_sample(x.data_ptr(), W_codes.data_ptr(), W_scales.data_ptr(), float(W_gscale),
                              logits.data_ptr(), u.data_ptr(), float(temperature), int(top_k), float(top_p),
                              token.data_ptr(), M, N, K, _stream_ptr(stream)), "lm_head_sample")
    return logits, token


# ------------------------------------------- key/value cache in 4 bits ------

def kv4_cache(pages: int, kv_heads: int, head_dim: int, page_size: int, device="cuda"):
    """An empty cache: uint8 [pages][kv_heads][page_size / 16][18 * head_dim] (include/skinny.h has the record)."""
    import torch

    if page_size % 16 or head_dim not in (64, 128, 256):
        raise ValueError("page_size must be a multiple of 16 and head_dim 64, 128 or 256")
    return torch.zeros((pages, kv_heads, page_size // 16, 18 * head_dim), dtype=torch.uint8, device=device)


def _cache_dims(cache):
    """(pages, kv_heads, head_dim, page_size) of a cache."""
    shape = cache.shape
    if cache.dtype is not _torch().uint8 or len(shape) != 4 or not cache.is_cuda or not cache.is_contiguous():
        raise TypeError("cache must be a contiguous 4-D CUDA uint8 tensor [pages][kv_heads][page_size/16][18 head_dim]")
    pages, heads, recs, rec = shape
    if rec % 18:
        raise ValueError(f"cache records of {rec} bytes: expected 18 * head_dim")
    return pages, heads, rec // 18, recs * 16


def _need(t, dtype, shape, what):
    """`t` as a contiguous CUDA tensor of this type and shape, or an error naming it."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA {dtype} tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _rows_f16(t, heads, dim, what):
    """Strided rows [T][heads][dim] of FP16: (rows, elements from row to row)."""
    shape = t.shape
    if t.dtype is not _torch().float16 or len(shape) != 3 or shape[1] != heads or shape[2] != dim or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA float16 tensor [T][{heads}][{dim}]")
    row, head, one = t.stride()
    if one != 1 or (head != dim and heads > 1):
        raise ValueError(f"{what}: heads and components must be contiguous (only the row stride is free)")
    n = shape[0]
    return n, row if n > 1 else heads * dim            # a single row has no stride to keep to


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch

        _TORCH = torch
    return _TORCH


def _raw_stream(stream, device):
    """The cudaStream_t of `stream`, or of the current stream of the tensors' device.  Asked for as a number:
    building torch's stream object takes longer (2.9 us of a call's 11 us) than the launch itself."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    number = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(device).cuda_stream if number is None else number(device)


def _new(shape, dtype, device, stream):
    """An output's memory, from the pool of the stream that will write it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def kv4_append(k, v, slots, cache, k_scale: float, v_scale: float, k_held=None, v_held=None, stream=None) -> None:
    """Write keys and values (FP16 [T][kv_heads][head_dim], row stride free) to the cache's slots
    (int32 [T], page * page_size + offset; negative: skipped).

    k_held and v_held (FP16 [T][kv_heads][head_dim], both or neither) get the values the cache then stands for."""
    torch = _torch()
    pages, heads, dim, page = _cache_dims(cache)
    n, ks = _rows_f16(k, heads, dim, "k")
    nv, vs = _rows_f16(v, heads, dim, "v")
    if n != nv:
        raise ValueError("k and v have different numbers of tokens")
    sp = _need(slots, torch.int32, (n,), "slots")
    hk = None if k_held is None else _need(k_held, torch.float16, (n, heads, dim), "k_held")
    hv = None if v_held is None else _need(v_held, torch.float16, (n, heads, dim), "v_held")
    _check(lib.kv4_append(k.data_ptr(), ks, v.data_ptr(), vs, sp, cache.data_ptr(), k_scale, v_scale, hk, hv,
                          n, pages, heads, dim, page, _raw_stream(stream, cache.get_device())), "kv4_append")


def kv4_attention(q, cache, table, lens, k_scale: float, v_scale: float, scale: float, rows: int = 1, out=None,
                  lse=None, acc=None, acc_out=None, stream=None):
    """Attention of `rows` query rows per sequence (q FP16 [seqs * rows][q_heads][head_dim], row stride free)
    over the cache's pages (table int32 [seqs][width]) up to lens (int32 [seqs]).

    acc_out (float32 [seqs][kv_heads][width * page_size], may be acc) gets acc plus the weight each position
    received; acc may be None (zeros).  Returns (out FP16, lse float32 [seqs * rows][q_heads])."""
    torch = _torch()
    pages, heads, dim, page = _cache_dims(cache)
    if q.dim() != 3:
        raise ValueError("q must be a CUDA float16 tensor [seqs * rows][q_heads][head_dim]")
    hq = q.shape[1]
    n, qs = _rows_f16(q, hq, dim, "q")
    if table.dim() != 2:
        raise ValueError("table must be a contiguous CUDA int32 tensor [seqs][width]")
    seqs, width = table.shape
    if seqs * rows != n:
        raise ValueError(f"q has {n} rows, expected {seqs} sequences x {rows}")
    tp = _need(table, torch.int32, (seqs, width), "table")
    lp = _need(lens, torch.int32, (seqs,), "lens")
    if out is None:
        out = _new((n, hq, dim), torch.float16, q.device, stream)
    if lse is None:
        lse = _new((n, hq), torch.float32, q.device, stream)
    ap = None if acc is None else _need(acc, torch.float32, (seqs, heads, width * page), "acc")
    op = None if acc_out is None else _need(acc_out, torch.float32, (seqs, heads, width * page), "acc_out")
    _check(lib.kv4_attention(q.data_ptr(), qs, cache.data_ptr(), tp, lp, k_scale, v_scale, scale,
                             _need(out, torch.float16, (n, hq, dim), "out"), _need(lse, torch.float32, (n, hq), "lse"),
                             ap, op, seqs, rows, hq, heads, dim, pages, page, width,
                             _raw_stream(stream, cache.get_device())),
           "kv4_attention")
    return out, lse


ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "turns": 3, "index": 4}


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original: float = 0.0, low: float = 1.0, high: float = 32.0, device="cuda"):
    """The frequencies of rot_dim / 2 pairs as fractions of a turn per position in units of 2^-64 (int64 holding the
    u64 of include/skinny.h), lengthened for longer contexts by one of ROPE_SCALINGS."""
    torch = _torch()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALINGS)}")
    freqs = torch.empty((max(0, rot_dim) // 2,), dtype=torch.int64)
    room = freqs if freqs.numel() else torch.empty((1,), dtype=torch.int64)      # an empty tensor has no address
    _check(lib.rope_frequencies(room.data_ptr(), rot_dim, ROPE_SCALINGS[scaling], base, factor, original, low, high),
           "rope_frequencies")
    return freqs.to(device)


def _rope_args(q, positions, freqs, q_weight, k_weight, dim):
    """Pointers of what both rotating calls take, and the rotated components of a head."""
    torch = _torch()
    rot = 0 if freqs is None else 2 * freqs.numel()
    fp = None if rot == 0 else _need(freqs, torch.int64, (rot // 2,), "freqs")
    pp = None if positions is None else _need(positions, torch.int32, (q.shape[0],), "positions")
    qw = None if q_weight is None else _need(q_weight, torch.float32, (dim,), "q_weight")
    kw = None if k_weight is None else _need(k_weight, torch.float32, (dim,), "k_weight")
    return pp, fp, qw, kw, rot


def qk_norm_rope(q, k, positions, freqs, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 amplitude: float = 1.0, q_out=None, k_out=None, stream=None):
    """Norm of every query and key head (FP16 [T][heads][head_dim], row stride free; weights float32 [head_dim], or
    neither) and its rotation by positions (int32 [T]) under freqs (rope_frequencies; None: no rotation).

    q_out and k_out may be q and k themselves.  Returns (q_out, k_out)."""
    torch = _torch()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be CUDA float16 tensors [T][heads][head_dim]")
    hq, dim = q.shape[1:]
    heads = k.shape[1]
    n, qs = _rows_f16(q, hq, dim, "q")
    nk, ks = _rows_f16(k, heads, dim, "k")
    if n != nk:
        raise ValueError("q and k have different numbers of tokens")
    pp, fp, qw, kw, rot = _rope_args(q, positions, freqs, q_weight, k_weight, dim)
    if q_out is None:
        q_out = _new((n, hq, dim), torch.float16, q.device, stream)
    if k_out is None:
        k_out = _new((n, heads, dim), torch.float16, q.device, stream)
    nq, qos = _rows_f16(q_out, hq, dim, "q_out")
    no, kos = _rows_f16(k_out, heads, dim, "k_out")
    if nq != n or no != n:
        raise ValueError("q_out and k_out must have as many tokens as q and k")
    _check(lib.qk_norm_rope(q.data_ptr(), qs, k.data_ptr(), ks, pp, fp, qw, kw, eps, amplitude, q_out.data_ptr(), qos,
                            k_out.data_ptr(), kos, n, hq, heads, dim, rot, int(interleaved),
                            _raw_stream(stream, q.get_device())), "qk_norm_rope")
    return q_out, k_out


def kv4_append_rope(q, k, v, slots, positions, freqs, cache, k_scale: float, v_scale: float, q_weight=None, k_weight=None,
                    eps: float = 1e-6, interleaved: bool = False, amplitude: float = 1.0, q_out=None, stream=None):
    """qk_norm_rope with the keys and the values (FP16 [T][kv_heads][head_dim]) written to the cache's slots (kv4_append).

    Returns q_out (FP16 [T][q_heads][head_dim], may be q itself)."""
    torch = _torch()
    pages, heads, dim, page = _cache_dims(cache)
    if q.dim() != 3:
        raise ValueError("q must be a CUDA float16 tensor [T][q_heads][head_dim]")
    hq = q.shape[1]
    n, qs = _rows_f16(q, hq, dim, "q")
    nk, ks = _rows_f16(k, heads, dim, "k")
    nv, vs = _rows_f16(v, heads, dim, "v")
    if n != nk or n != nv:
        raise ValueError("q, k and v have different numbers of tokens")
    pp, fp, qw, kw, rot = _rope_args(q, positions, freqs, q_weight, k_weight, dim)
    sp = _need(slots, torch.int32, (n,), "slots")
    if q_out is None:
        q_out = _new((n, hq, dim), torch.float16, q.device, stream)
    no, qos = _rows_f16(q_out, hq, dim, "q_out")
    if no != n:
        raise ValueError("q_out must have as many tokens as q")
    _check(lib.kv4_append_rope(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, sp, pp, fp, qw, kw, eps, amplitude,
                               q_out.data_ptr(), qos, cache.data_ptr(), k_scale, v_scale, n, pages, hq, heads, dim, page,
                               rot, int(interleaved), _raw_stream(stream, cache.get_device())), "kv4_append_rope")
    return q_out


def kv4_window_attention(q, cache, table, lens, k_scale: float, v_scale: float, scale: float, window: int, sinks: int = 0,
                         rows: int = 1, out=None, lse=None, stream=None):
    """kv4_attention where a row sees only the last `window` positions up to its own and the first `sinks` ones.

    Returns (out FP16, lse float32 [seqs * rows][q_heads])."""
    torch = _torch()
    pages, heads, dim, page = _cache_dims(cache)
    if q.dim() != 3:
        raise ValueError("q must be a CUDA float16 tensor [seqs * rows][q_heads][head_dim]")
    hq = q.shape[1]
    n, qs = _rows_f16(q, hq, dim, "q")
    if table.dim() != 2:
        raise ValueError("table must be a contiguous CUDA int32 tensor [seqs][width]")
    seqs, width = table.shape
    if seqs * rows != n:
        raise ValueError(f"q has {n} rows, expected {seqs} sequences x {rows}")
    if out is None:
        out = _new((n, hq, dim), torch.float16, q.device, stream)
    if lse is None:
        lse = _new((n, hq), torch.float32, q.device, stream)
    _check(lib.kv4_window_attention(q.data_ptr(), qs, cache.data_ptr(), _need(table, torch.int32, (seqs, width), "table"),
                                    _need(lens, torch.int32, (seqs,), "lens"), k_scale, v_scale, scale, window, sinks,
                                    _need(out, torch.float16, (n, hq, dim), "out"),
                                    _need(lse, torch.float32, (n, hq), "lse"), seqs, rows, hq, heads, dim, pages, page,
                                    width, _raw_stream(stream, cache.get_device())), "kv4_window_attention")
    return out, lse


def kv4_chunk_attention(q, cache, table, lens, starts, k_scale: float, v_scale: float, scale: float, window: int = 0,
                        sinks: int = 0, out=None, lse=None, stream=None):
    """Attention of chunks of new tokens (q FP16 [rows][q_heads][head_dim], row stride free; sequence b's rows are
    starts[b] .. starts[b + 1] - 1, int32 [seqs + 1], its last positions) over the cache's pages up to lens.

    With window > 0 a row sees only the last `window` positions up to its own and the first `sinks` ones.
    Returns (out FP16, lse float32 [rows][q_heads]); rows of no sequence are not written."""
    torch = _torch()
    pages, heads, dim, page = _cache_dims(cache)
    if q.dim() != 3:
        raise ValueError("q must be a CUDA float16 tensor [rows][q_heads][head_dim]")
    hq = q.shape[1]
    n, qs = _rows_f16(q, hq, dim, "q")
    if table.dim() != 2:
        raise ValueError("table must be a contiguous CUDA int32 tensor [seqs][width]")
    seqs, width = table.shape
    i32 = torch.int32
    if out is None:
        out = _new((n, hq, dim), torch.float16, q.device, stream)
    if lse is None:
        lse = _new((n, hq), torch.float32, q.device, stream)
    _check(lib.kv4_chunk_attention(q.data_ptr(), qs, cache.data_ptr(), _need(table, i32, (seqs, width), "table"),
                                   _need(lens, i32, (seqs,), "lens"), _need(starts, i32, (seqs + 1,), "starts"), k_scale,
                                   v_scale, scale, window, sinks, _need(out, torch.float16, (n, hq, dim), "out"),
                                   _need(lse, torch.float32, (n, hq), "lse"), n, seqs, hq, heads, dim, pages, page, width,
                                   _raw_stream(stream, cache.get_device())), "kv4_chunk_attention")
    return out, lse


def kv4_evict(cache, table, lens, acc, dst_table, budget: int, recent: int, kept=None, new_lens=None, acc_out=None,
              stream=None):
    """Keep at most `budget` positions per sequence and kv head (the last `recent` and the largest of
    acc, float32 [seqs][kv_heads][width * page_size]) and copy them, in order, to the pages of dst_table.

    Returns (new_lens int32 [seqs], kept int32 [seqs][kv_heads][budget], acc_out float32
    [seqs][kv_heads][dst_width * page_size])."""
    torch = _torch()
    pages, heads, dim, page = _cache_dims(cache)
    if table.dim() != 2 or dst_table.dim() != 2:
        raise ValueError("table and dst_table must be contiguous CUDA int32 tensors [seqs][width]")
    seqs, width = table.shape
    dwidth = dst_table.shape[1]
    if new_lens is None:
        new_lens = _new((seqs,), torch.int32, cache.device, stream)
    if kept is None:
        kept = _new((seqs, heads, budget), torch.int32, cache.device, stream)
    if acc_out is None:
        acc_out = _new((seqs, heads, dwidth * page), torch.float32, cache.device, stream)
    i32, f32 = torch.int32, torch.float32
    _check(lib.kv4_evict(cache.data_ptr(), _need(table, i32, (seqs, width), "table"), _need(lens, i32, (seqs,), "lens"),
                         _need(acc, f32, (seqs, heads, width * page), "acc"),
                         _need(dst_table, i32, (seqs, dwidth), "dst_table"),
                         _need(kept, i32, (seqs, heads, budget), "kept"), _need(new_lens, i32, (seqs,), "new_lens"),
                         _need(acc_out, f32, (seqs, heads, dwidth * page), "acc_out"), seqs, budget, recent, heads, dim,
                         pages, page, width, dwidth, _raw_stream(stream, cache.get_device())), "kv4_evict")
    return new_lens, kept, acc_out


def token_logprobs(logits, tokens=None, top_n: int = 0, temperature: float = 1.0, logprob=None, rank=None,
                   entropy=None, top_ids=None, top_logprobs=None, stream=None):
    """Log probability and rank of `tokens` (int32 [M], or None) under softmax(logits / temperature), the rows'
    entropy and their top_n alternatives; logits float32 or float16 [M][N], row stride free.

    Returns (logprob float32 [M], rank int32 [M], entropy float32 [M], top_ids int32 [M][top_n],
    top_logprobs float32 [M][top_n]); logprob and rank are None without tokens."""
    torch = _torch()
    f32, i32 = torch.float32, torch.int32
    if logits.dim() != 2 or logits.dtype not in (f32, torch.float16) or not logits.is_cuda:
        raise TypeError("logits must be a 2-D CUDA float32 or float16 tensor [M][N]")
    M, N = logits.shape
    stride, one = logits.stride()
    if N > 1 and one != 1:
        raise ValueError("logits: the entries of a row must be contiguous (only the row stride is free)")
    dev = logits.device
    tp = lp = rp = None
    if tokens is not None:
        tp = _need(tokens, i32, (M,), "tokens")
        if logprob is None:
            logprob = _new((M,), f32, dev, stream)
        if rank is None:
            rank = _new((M,), i32, dev, stream)
        lp, rp = _need(logprob, f32, (M,), "logprob"), _need(rank, i32, (M,), "rank")
    else:
        logprob = rank = None
    if entropy is None:
        entropy = _new((M,), f32, dev, stream)
    if top_ids is None:
        top_ids = _new((M, top_n), i32, dev, stream)
    if top_logprobs is None:
        top_logprobs = _new((M, top_n), f32, dev, stream)
    _check(lib.token_logprobs(logits.data_ptr(), 0 if logits.dtype == f32 else 1, stride if M > 1 else max(stride, N),
                              tp, temperature, top_n, lp, rp, _need(entropy, f32, (M,), "entropy"),
                              _need(top_ids, i32, (M, top_n), "top_ids"),
                              _need(top_logprobs, f32, (M, top_n), "top_logprobs"), M, N,
                              _raw_stream(stream, logits.get_device())),
           "token_logprobs")
    return logprob, rank, entropy, top_ids, top_logprobs
