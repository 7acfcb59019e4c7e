"""Python binding of libcsa.so -- the DeepSeek-V4 CSA/HCA hot path on B200.

Argument marshalling only: every step runs in the CUDA kernels of libcsa.so
(declared in include/csa.h).  Functions carry the C ABI names and take torch
tensors that already live on the current CUDA device; outputs are allocated
here when not supplied, scratch memory is a torch uint8 workspace sized by the
library's *_workspace_bytes() query, and work is enqueued on torch's current
stream.  A non-zero status from the library raises CsaError.  There is no CPU
path: importing works without a GPU, but every call needs the CUDA library.
"""
import ctypes
import os

import torch

__all__ = [
    "CsaError", "lib", "csa_compress", "csa_indexer_topk", "csa_sparse_attn", "hca_attn", "csa_decode",
    "hca_decode", "csa_check_status", "csa_status_string", "csa_version", "LIB_PATH", "csa_decode_append",
    "hca_decode_append", "csa_mxfp4_quantize", "csa_mxfp8_quantize", "csa_decode_fp8", "csa_peak_mma",
    "csa_decode_search", "csa_topk_merge", "csa_decode_attend", "csa_attn_combine", "rope_inv_freq",
    "csa_qk_norm_rope", "csa_qk_norm_rope_backward", "csa_paged_append", "csa_tree_attn",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcsa.so")

_lib = None


class CsaError(RuntimeError):
    def __init__(self, code, what):
        super().__init__("%s failed: %s (status %d)" % (what, csa_status_string(code), code))
        self.code = code


def lib():
    """The loaded libcsa.so. Raises if the CUDA library has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libcsa.so not found at %s; build it with "
                               "`python -m long_context_compressed_gated_b200.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        sig = {
            "csa_status_string": ([I], ctypes.c_char_p),
            "csa_last_cuda_error": ([], I),
            "csa_version": ([], I),
            "csa_check_status": ([P, P], I),
            "csa_debug_inject": ([I], I),
            "csa_decode_append": ([P, P, P, P, P, P, P, I, I64, I, I, I, I, P, P, P, P, P, P, P, P, P, P], I),
            "hca_decode_append": ([P, P, P, P, P, I, I64, I, I, I, P, P, P, P, P, P, P, P], I),
            "csa_mxfp4_quantize": ([P, I64, I, I, P, P, P], I),
            "csa_mxfp8_quantize": ([P, I64, I, P, P, P], I),
            "csa_peak_mma": ([I, I64, I, P, SZ, P, P], I),
            "csa_compress": ([P, P, P, P, I64, I, I, P, P, P], I),
            "csa_indexer_topk_workspace_bytes": ([I64, I64, I, I, I], SZ),
            "csa_indexer_topk": ([P, P, P, P, P, I64, I64, I64, I, I, I, I, P, P, P, SZ, P], I),
            "csa_sparse_attn_workspace_bytes": ([I64, I, I, I, I], SZ),
            "csa_sparse_attn": ([P, P, P, P, P, P, I64, I64, I64, I, I, I, I, F, P, I, P, P, SZ, P], I),
            "hca_attn_workspace_bytes": ([I64, I, I, I], SZ),
            "hca_attn": ([P, P, P, P, P, I64, I64, I64, I, I, I, I, F, P, I, P, P, SZ, P], I),
            "csa_decode_workspace_bytes": ([I, I64, I, I, I, I, I, I], SZ),
            "csa_decode": ([P, P, P, P, P, P, P, P, P, P, P, I, I64, I, I, I, I, I, I, I, F, P, I, P, P, P, P, SZ,
                            P], I),
            "csa_decode_fp8": ([P, P, P, P, P, P, P, P, P, P, P, P, P, I, I64, I, I, I, I, I, I, I, F, P, I, P, P, P,
                                P, SZ, P], I),
            "hca_decode_workspace_bytes": ([I, I64, I, I, I], SZ),
            "csa_decode_search_workspace_bytes": ([I, I64, I], SZ),
            "csa_decode_search": ([P, P, P, P, P, P, I, I64, I64, I, I, I, I, P, P, SZ, P], I),
            "csa_topk_merge_workspace_bytes": ([I, I], SZ),
            "csa_topk_merge": ([P, I, I, I, P, P, P, P, SZ, P], I),
            "csa_decode_attend": ([P, P, P, P, I64, P, P, P, I, I64, I, I, I, I, I, F, P, I, P, P, SZ, P], I),
            "csa_attn_combine": ([P, P, I, I, I, I, P, I, P, P], I),
            "csa_qk_norm_rope": ([P, I64, P, I64, P, P, F, P, I64, P, I, I, I, I64, I, I, I, I, P, P, I, P], I),
            "csa_qk_norm_rope_backward_workspace_bytes": ([I64, I, I, I], SZ),
            "csa_qk_norm_rope_backward": ([P, I64, P, I64, P, P, F, P, I64, P, I, I, I, P, P, I64, I, I, I, I, I, P, I64,
                                           P, I64, P, P, P, SZ, P], I),
            "csa_paged_append": ([P, I64, P, I64, P, F, P, P, P, P, I, I, I, P, I64, I, I, I, I, I64, I, P, P, P, SZ,
                                  P], I),
            "csa_tree_attn_workspace_bytes": ([I, I64, I, I, I, I, I], SZ),
            "csa_tree_attn": ([P, P, P, P, P, P, P, P, I64, I, I, I, I, I, I64, I, I, F, P, I, P, P, SZ, P], I),
            "hca_decode": ([P, P, P, P, P, P, I, I64, I, I, I, I, F, P, I, P, P, SZ, P], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def csa_status_string(code):
    return lib().csa_status_string(int(code)).decode()


def csa_version():
    return lib().csa_version()


_ODTYPE = {torch.bfloat16: 0, torch.float32: 1}  # csa_dtype_t


def _out(O, like, shape, out_dtype, name="O"):
    """Output tensor of the given dtype (bf16 or fp32): allocated when O is None."""
    if out_dtype not in _ODTYPE:
        raise TypeError("%s dtype must be torch.bfloat16 or torch.float32" % name)
    if O is None:
        return torch.empty(shape, dtype=out_dtype, device=like.device)
    return _dev(O, out_dtype, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


# torch's own accessor of the current stream's handle by device number, where it has one: the
# public one builds a Stream object, over a microsecond a call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev=None):
    """The current stream's handle, of the current device (whose number may be given)."""
    if dev is None:
        dev = torch.cuda.current_device()
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _dev(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims, got %d" % (name, ndim, t.dim()))
    return t


def _check(code, what):
    if code != 0:
        raise CsaError(code, what)


def _workspace(nbytes, device, workspace=None):
    if workspace is not None:
        if workspace.numel() < nbytes:
            raise ValueError("workspace too small: %d < %d bytes" % (workspace.numel(), nbytes))
        return workspace
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    ws[:4].zero_()  # status word
    return ws


def csa_check_status(workspace):
    """Synchronise the current stream, return and clear the device status word."""
    return lib().csa_check_status(_ptr(workspace), _stream())


def csa_peak_mma(kind, iters, ctas=None, workspace=None):
    """Enqueue the tensor-pipe peak loop (kind 0 = bf16, 1 = MXFP4) on the current
    stream; returns (flops of the launch, workspace).  ctas defaults to the SM count."""
    dev = torch.device("cuda", torch.cuda.current_device())
    if ctas is None:
        ctas = torch.cuda.get_device_properties(dev).multi_processor_count
    ws = _workspace(256, dev, workspace)
    fl = ctypes.c_double(0.0)
    _check(lib().csa_peak_mma(int(kind), int(iters), int(ctas), _ptr(ws), ws.numel(), ctypes.byref(fl), _stream()),
           "csa_peak_mma")
    return fl.value, ws


MX_OCP, MX_INDEXER = 0, 1


def csa_mxfp4_quantize(x, mode=MX_OCP, codes=None, scales=None):
    """bf16 [..., n] (n % 32 == 0) -> MXFP4 (codes uint8 [..., n/2], scales uint8
    [..., n/32]).  mode MX_INDEXER keeps the scale bytes in 125..128."""
    _dev(x, torch.bfloat16, "x")
    n = x.shape[-1]
    rows = x.numel() // n if n else 0
    lead = tuple(x.shape[:-1])
    codes = torch.empty(lead + (n // 2,), dtype=torch.uint8, device=x.device) if codes is None else \
        _dev(codes, torch.uint8, "codes")
    scales = torch.empty(lead + (n // 32,), dtype=torch.uint8, device=x.device) if scales is None else \
        _dev(scales, torch.uint8, "scales")
    _check(lib().csa_mxfp4_quantize(_ptr(x), rows, n, int(mode), _ptr(codes), _ptr(scales), _stream()),
           "csa_mxfp4_quantize")
    return codes, scales


def csa_mxfp8_quantize(x, codes=None, scales=None):
    """bf16 [..., n] (n % 32 == 0) -> MXFP8 (E4M3 codes uint8 [..., n], E8M0 scales
    uint8 [..., n/32]): the FP8 form of the compressed K/V cache."""
    _dev(x, torch.bfloat16, "x")
    n = x.shape[-1]
    rows = x.numel() // n if n else 0
    lead = tuple(x.shape[:-1])
    codes = torch.empty(lead + (n,), dtype=torch.uint8, device=x.device) if codes is None else \
        _dev(codes, torch.uint8, "codes")
    scales = torch.empty(lead + (n // 32,), dtype=torch.uint8, device=x.device) if scales is None else \
        _dev(scales, torch.uint8, "scales")
    _check(lib().csa_mxfp8_quantize(_ptr(x), rows, n, _ptr(codes), _ptr(scales), _stream()), "csa_mxfp8_quantize")
    return codes, scales


def csa_compress(K, V, Z, B, m, Kc=None, Vc=None):
    """Gated pooling of every complete block of m tokens. K,V,Z [T,d] bf16, B [m,d] f32.
    Returns (Kc, Vc) [T//m, d] bf16."""
    _dev(K, torch.bfloat16, "K", 2), _dev(V, torch.bfloat16, "V", 2), _dev(Z, torch.bfloat16, "Z", 2)
    _dev(B, torch.float32, "B", 2)
    T, d = K.shape
    nb = T // m
    Kc = torch.empty(nb, d, dtype=torch.bfloat16, device=K.device) if Kc is None else _dev(Kc, torch.bfloat16, "Kc")
    Vc = torch.empty(nb, d, dtype=torch.bfloat16, device=K.device) if Vc is None else _dev(Vc, torch.bfloat16, "Vc")
    _check(lib().csa_compress(_ptr(K), _ptr(V), _ptr(Z), _ptr(B), T, d, m, _ptr(Kc), _ptr(Vc), _stream()),
           "csa_compress")
    return Kc, Vc


def csa_indexer_topk(qI_codes, qI_scales, w_codes, kI_codes, kI_scales, m, k, t0=0, idx=None, scores=None,
                     want_scores=True, workspace=None):
    """MXFP4 lightning indexer + causal top-k. Returns (idx [T,k] int32, scores [T,k] f32 or None, workspace)."""
    _dev(qI_codes, torch.uint8, "qI_codes", 3), _dev(qI_scales, torch.uint8, "qI_scales", 3)
    _dev(w_codes, torch.uint8, "w_codes", 2), _dev(kI_codes, torch.uint8, "kI_codes", 2)
    _dev(kI_scales, torch.uint8, "kI_scales", 2)
    T, HI, half = qI_codes.shape
    dI = half * 2
    Nc = kI_codes.shape[0]
    dev = qI_codes.device
    idx = torch.empty(T, k, dtype=torch.int32, device=dev) if idx is None else _dev(idx, torch.int32, "idx")
    if want_scores and scores is None:
        scores = torch.empty(T, k, dtype=torch.float32, device=dev)
    elif scores is not None:
        _dev(scores, torch.float32, "scores")
    ws = _workspace(lib().csa_indexer_topk_workspace_bytes(T, Nc, HI, dI, k), dev, workspace)
    _check(lib().csa_indexer_topk(_ptr(qI_codes), _ptr(qI_scales), _ptr(w_codes), _ptr(kI_codes), _ptr(kI_scales),
                                  T, t0, Nc, HI, dI, m, k, _ptr(idx), _ptr(scores), _ptr(ws), ws.numel(),
                                  _stream()), "csa_indexer_topk")
    return idx, scores, ws


def csa_sparse_attn(Q, Kc, Vc, idx, Kraw, Vraw, W, scale, t0=0, O=None, lse=None, want_lse=True, workspace=None,
                    out_dtype=torch.bfloat16):
    """CSA attention over the selected entries plus the raw window. Returns (O, lse, workspace).
    out_dtype: torch.bfloat16 (default) or torch.float32 for O."""
    _dev(Q, torch.bfloat16, "Q", 3), _dev(Kc, torch.bfloat16, "Kc", 2), _dev(Vc, torch.bfloat16, "Vc", 2)
    _dev(idx, torch.int32, "idx", 2), _dev(Kraw, torch.bfloat16, "Kraw", 2), _dev(Vraw, torch.bfloat16, "Vraw", 2)
    T, H, d = Q.shape
    k = idx.shape[1]
    dev = Q.device
    O = _out(O, Q, Q.shape, out_dtype)
    if want_lse and lse is None:
        lse = torch.empty(T, H, dtype=torch.float32, device=dev)
    ws = _workspace(lib().csa_sparse_attn_workspace_bytes(T, H, d, k, W), dev, workspace)
    _check(lib().csa_sparse_attn(_ptr(Q), _ptr(Kc), _ptr(Vc), _ptr(idx), _ptr(Kraw), _ptr(Vraw), T, t0,
                                 Kc.shape[0], H, d, k, W, float(scale), _ptr(O), _ODTYPE[out_dtype], _ptr(lse),
                                 _ptr(ws), ws.numel(), _stream()), "csa_sparse_attn")
    return O, lse, ws


def hca_attn(Q, Kc, Vc, Kraw, Vraw, m, W, scale, t0=0, O=None, lse=None, want_lse=True, workspace=None,
             out_dtype=torch.bfloat16):
    """HCA attention over every visible compressed entry plus the raw window. Returns (O, lse, workspace).
    out_dtype: torch.bfloat16 (default) or torch.float32 for O."""
    _dev(Q, torch.bfloat16, "Q", 3), _dev(Kc, torch.bfloat16, "Kc", 2), _dev(Vc, torch.bfloat16, "Vc", 2)
    _dev(Kraw, torch.bfloat16, "Kraw", 2), _dev(Vraw, torch.bfloat16, "Vraw", 2)
    T, H, d = Q.shape
    dev = Q.device
    O = _out(O, Q, Q.shape, out_dtype)
    if want_lse and lse is None:
        lse = torch.empty(T, H, dtype=torch.float32, device=dev)
    ws = _workspace(lib().hca_attn_workspace_bytes(T, H, d, W), dev, workspace)
    _check(lib().hca_attn(_ptr(Q), _ptr(Kc), _ptr(Vc), _ptr(Kraw), _ptr(Vraw), T, t0, Kc.shape[0], H, d, m, W,
                          float(scale), _ptr(O), _ODTYPE[out_dtype], _ptr(lse), _ptr(ws), ws.numel(), _stream()),
           "hca_attn")
    return O, lse, ws


def csa_decode(q, qI_codes, qI_scales, w_codes, Kc, Vc, kI_codes, kI_scales, Kwin, Vwin, pos, m, k, scale,
               O=None, lse=None, idx=None, scores=None, want_lse=True, want_sel=True, workspace=None,
               out_dtype=torch.bfloat16):
    """One new token per sequence against its compressed cache (indexer, top-k,
    sparse + window attention). pos: list of absolute positions (host).
    Returns (O [B,H,d], lse, idx [B,k], scores [B,k], workspace)."""
    _dev(q, torch.bfloat16, "q", 3), _dev(qI_codes, torch.uint8, "qI_codes", 3)
    _dev(qI_scales, torch.uint8, "qI_scales", 3), _dev(w_codes, torch.uint8, "w_codes", 2)
    _dev(Kc, torch.bfloat16, "Kc", 3), _dev(Vc, torch.bfloat16, "Vc", 3)
    _dev(kI_codes, torch.uint8, "kI_codes", 3), _dev(kI_scales, torch.uint8, "kI_scales", 3)
    _dev(Kwin, torch.bfloat16, "Kwin", 3), _dev(Vwin, torch.bfloat16, "Vwin", 3)
    B, H, d = q.shape
    HI, dI = qI_codes.shape[1], qI_codes.shape[2] * 2
    Ncap = Kc.shape[1]
    W = Kwin.shape[1]
    dev = q.device
    O = _out(O, q, q.shape, out_dtype)
    if want_lse and lse is None:
        lse = torch.empty(B, H, dtype=torch.float32, device=dev)
    if want_sel:
        idx = torch.empty(B, k, dtype=torch.int32, device=dev) if idx is None else idx
        scores = torch.empty(B, k, dtype=torch.float32, device=dev) if scores is None else scores
    posa = (ctypes.c_int64 * B)(*[int(p) for p in pos])
    ws = _workspace(lib().csa_decode_workspace_bytes(B, Ncap, H, d, HI, dI, k, W), dev, workspace)
    _check(lib().csa_decode(_ptr(q), _ptr(qI_codes), _ptr(qI_scales), _ptr(w_codes), _ptr(Kc), _ptr(Vc),
                            _ptr(kI_codes), _ptr(kI_scales), _ptr(Kwin), _ptr(Vwin), posa, B, Ncap, H, d, HI, dI,
                            m, k, W, float(scale), _ptr(O), _ODTYPE[out_dtype], _ptr(lse), _ptr(idx),
                            _ptr(scores), _ptr(ws), ws.numel(), _stream()), "csa_decode")
    return O, lse, idx, scores, ws


def csa_decode_fp8(q, qI_codes, qI_scales, w_codes, Kc_codes, Kc_scales, Vc_codes, Vc_scales, kI_codes, kI_scales,
                   Kwin, Vwin, pos, m, k, scale, O=None, lse=None, idx=None, scores=None, want_lse=True,
                   want_sel=True, workspace=None, out_dtype=torch.bfloat16):
    """csa_decode over an MXFP8 compressed cache: Kc/Vc codes [B,Ncap,d] uint8 (E4M3)
    and scales [B,Ncap,d/32] uint8 (E8M0).  Returns (O, lse, idx, scores, workspace)."""
    _dev(q, torch.bfloat16, "q", 3), _dev(qI_codes, torch.uint8, "qI_codes", 3)
    _dev(qI_scales, torch.uint8, "qI_scales", 3), _dev(w_codes, torch.uint8, "w_codes", 2)
    for t, n in ((Kc_codes, "Kc_codes"), (Kc_scales, "Kc_scales"), (Vc_codes, "Vc_codes"), (Vc_scales, "Vc_scales"),
                 (kI_codes, "kI_codes"), (kI_scales, "kI_scales")):
        _dev(t, torch.uint8, n, 3)
    _dev(Kwin, torch.bfloat16, "Kwin", 3), _dev(Vwin, torch.bfloat16, "Vwin", 3)
    B, H, d = q.shape
    HI, dI = qI_codes.shape[1], qI_codes.shape[2] * 2
    Ncap = Kc_codes.shape[1]
    W = Kwin.shape[1]
    dev = q.device
    O = _out(O, q, q.shape, out_dtype)
    if want_lse and lse is None:
        lse = torch.empty(B, H, dtype=torch.float32, device=dev)
    if want_sel:
        idx = torch.empty(B, k, dtype=torch.int32, device=dev) if idx is None else idx
        scores = torch.empty(B, k, dtype=torch.float32, device=dev) if scores is None else scores
    posa = (ctypes.c_int64 * B)(*[int(p) for p in pos])
    ws = _workspace(lib().csa_decode_workspace_bytes(B, Ncap, H, d, HI, dI, k, W), dev, workspace)
    _check(lib().csa_decode_fp8(_ptr(q), _ptr(qI_codes), _ptr(qI_scales), _ptr(w_codes), _ptr(Kc_codes),
                                _ptr(Kc_scales), _ptr(Vc_codes), _ptr(Vc_scales), _ptr(kI_codes), _ptr(kI_scales),
                                _ptr(Kwin), _ptr(Vwin), posa, B, Ncap, H, d, HI, dI, m, k, W, float(scale), _ptr(O),
                                _ODTYPE[out_dtype], _ptr(lse), _ptr(idx), _ptr(scores), _ptr(ws), ws.numel(),
                                _stream()), "csa_decode_fp8")
    return O, lse, idx, scores, ws


def hca_decode(q, Kc, Vc, Kwin, Vwin, pos, m, scale, O=None, lse=None, want_lse=True, workspace=None,
               out_dtype=torch.bfloat16):
    """HCA decode: one token per sequence, dense over its visible cache + window."""
    _dev(q, torch.bfloat16, "q", 3), _dev(Kc, torch.bfloat16, "Kc", 3), _dev(Vc, torch.bfloat16, "Vc", 3)
    _dev(Kwin, torch.bfloat16, "Kwin", 3), _dev(Vwin, torch.bfloat16, "Vwin", 3)
    B, H, d = q.shape
    Ncap, W = Kc.shape[1], Kwin.shape[1]
    dev = q.device
    O = _out(O, q, q.shape, out_dtype)
    if want_lse and lse is None:
        lse = torch.empty(B, H, dtype=torch.float32, device=dev)
    posa = (ctypes.c_int64 * B)(*[int(p) for p in pos])
    ws = _workspace(lib().hca_decode_workspace_bytes(B, Ncap, H, d, W), dev, workspace)
    _check(lib().hca_decode(_ptr(q), _ptr(Kc), _ptr(Vc), _ptr(Kwin), _ptr(Vwin), posa, B, Ncap, H, d, m, W,
                            float(scale), _ptr(O), _ODTYPE[out_dtype], _ptr(lse), _ptr(ws), ws.numel(), _stream()),
           "hca_decode")
    return O, lse, ws


def csa_decode_append(K_new, V_new, Z_new, B, pos, Kwin, Vwin, Kblk, Vblk, Zblk, Kc, Vc, kI_codes_new=None,
                      kI_scales_new=None, kI_codes=None, kI_scales=None):
    """Append one token per sequence to the decode state (window, block staging,
    and on block completion the compressed entry and its indexer key), in place.
    K_new/V_new/Z_new [Bseq,d] bf16; B [m,d] f32; pos: host positions of the new
    tokens; Kwin/Vwin [Bseq,W,d]; Kblk/Vblk/Zblk [Bseq,m,d]; Kc/Vc [Bseq,Ncap,d];
    kI_* (all or none): the completed entry's MXFP4 key [Bseq,dI/2]/[Bseq,dI/32]
    and the cache's key tensors [Bseq,Ncap,dI/2]/[Bseq,Ncap,dI/32]."""
    for t, n in ((K_new, "K_new"), (V_new, "V_new"), (Z_new, "Z_new"), (Kwin, "Kwin"), (Vwin, "Vwin"),
                 (Kblk, "Kblk"), (Vblk, "Vblk"), (Zblk, "Zblk"), (Kc, "Kc"), (Vc, "Vc")):
        _dev(t, torch.bfloat16, n)
    _dev(B, torch.float32, "B", 2)
    nb, d = K_new.shape
    m = Kblk.shape[1]
    W = Kwin.shape[1]
    Ncap = Kc.shape[1]
    posa = (ctypes.c_int64 * nb)(*[int(p) for p in pos])
    dI = 0
    if kI_codes is not None:
        for t, n in ((kI_codes_new, "kI_codes_new"), (kI_scales_new, "kI_scales_new"), (kI_codes, "kI_codes"),
                     (kI_scales, "kI_scales")):
            _dev(t, torch.uint8, n)
        dI = kI_codes.shape[-1] * 2
    _check(lib().csa_decode_append(_ptr(K_new), _ptr(V_new), _ptr(Z_new), _ptr(B), _ptr(kI_codes_new),
                                   _ptr(kI_scales_new), posa, nb, Ncap, d, dI, m, W, _ptr(Kwin), _ptr(Vwin),
                                   _ptr(Kblk), _ptr(Vblk), _ptr(Zblk), _ptr(Kc), _ptr(Vc), _ptr(kI_codes),
                                   _ptr(kI_scales), _stream()), "csa_decode_append")


def hca_decode_append(K_new, V_new, Z_new, B, pos, Kwin, Vwin, Kblk, Vblk, Zblk, Kc, Vc):
    """csa_decode_append without indexer keys (the HCA layer's cache, ratio m')."""
    csa_decode_append(K_new, V_new, Z_new, B, pos, Kwin, Vwin, Kblk, Vblk, Zblk, Kc, Vc)


def csa_decode_search(qI_codes, qI_scales, w_codes, kI_codes, kI_scales, pos, m, k, j_base=0, keys=None,
                      workspace=None):
    """The k best entries of a cache slice (global indices j_base + local) as exact
    uint64 keys [B, k] (torch.int64 storage; 0 = none).  Returns (keys, workspace)."""
    B, HI, half = qI_codes.shape
    dI = half * 2
    Nloc = kI_codes.shape[1]
    dev = qI_codes.device
    keys = torch.empty(B, k, dtype=torch.int64, device=dev) if keys is None else _dev(keys, torch.int64, "keys")
    posa = (ctypes.c_int64 * B)(*[int(p) for p in pos])
    ws = _workspace(lib().csa_decode_search_workspace_bytes(B, Nloc, k), dev, workspace)
    _check(lib().csa_decode_search(_ptr(qI_codes), _ptr(qI_scales), _ptr(w_codes), _ptr(kI_codes), _ptr(kI_scales),
                                   posa, B, Nloc, int(j_base), HI, dI, m, k, _ptr(keys), _ptr(ws), ws.numel(),
                                   _stream()), "csa_decode_search")
    return keys, ws


def csa_topk_merge(keys, k, idx=None, scores=None, workspace=None):
    """keys [B, L, k] (int64 storage of the uint64 keys) -> (idx [B,k], scores [B,k])."""
    _dev(keys, torch.int64, "keys", 3)
    B, L, kk = keys.shape
    assert kk == k
    dev = keys.device
    idx = torch.empty(B, k, dtype=torch.int32, device=dev) if idx is None else idx
    scores = torch.empty(B, k, dtype=torch.float32, device=dev) if scores is None else scores
    ws = _workspace(lib().csa_topk_merge_workspace_bytes(B, L), dev, workspace)
    _check(lib().csa_topk_merge(_ptr(keys), B, L, k, _ptr(idx), _ptr(scores), None, _ptr(ws), ws.numel(), _stream()),
           "csa_topk_merge")
    return idx, scores


def csa_decode_attend(q, Kc, Vc, idx, Kwin, Vwin, pos, m, W, scale, j_base=0, O=None, lse=None,
                      out_dtype=torch.float32, workspace=None):
    """Attention over the selected entries inside a cache slice [B, Nloc, d] (+ the
    window when W > 0).  Returns (O, lse) for merging with csa_attn_combine."""
    B, H, d = q.shape
    Nloc = Kc.shape[1]
    k = idx.shape[1]
    dev = q.device
    O = _out(O, q, q.shape, out_dtype)
    lse = torch.empty(B, H, dtype=torch.float32, device=dev) if lse is None else lse
    posa = (ctypes.c_int64 * B)(*[int(p) for p in pos])
    ws = _workspace(lib().csa_decode_workspace_bytes(B, Nloc, H, d, 16, 128, k, W), dev, workspace)
    _check(lib().csa_decode_attend(_ptr(q), _ptr(Kc), _ptr(Vc), _ptr(idx), int(j_base), _ptr(Kwin) if W else None,
                                   _ptr(Vwin) if W else None, posa, B, Nloc, H, d, m, k, W, float(scale), _ptr(O),
                                   _ODTYPE[out_dtype], _ptr(lse), _ptr(ws), ws.numel(), _stream()),
           "csa_decode_attend")
    return O, lse


def csa_attn_combine(O_parts, lse_parts, out_dtype=torch.bfloat16, O=None, lse=None):
    """O_parts [L, B, H, d] f32, lse_parts [L, B, H] f32 -> (O [B, H, d], lse [B, H])."""
    _dev(O_parts, torch.float32, "O_parts", 4), _dev(lse_parts, torch.float32, "lse_parts", 3)
    L, B, H, d = O_parts.shape
    O = _out(O, O_parts, (B, H, d), out_dtype)
    lse = torch.empty(B, H, dtype=torch.float32, device=O_parts.device) if lse is None else lse
    _check(lib().csa_attn_combine(_ptr(O_parts), _ptr(lse_parts), L, B, H, d, _ptr(O), _ODTYPE[out_dtype], _ptr(lse),
                                  _stream()), "csa_attn_combine")
    return O, lse


# ---------------------------------------------------------------- norm, position rotation, paged cache
ROPE_HALVES, ROPE_PAIRS = 0, 1


def rope_inv_freq(rot_dim, base=10000.0):
    """base^(-2p/rot_dim) for p < rot_dim/2: radians per position of the rotated
    channel pairs, as a float64 CPU tensor (any other float64 CPU tensor of that
    length, a stretched or scaled one say, serves as well)."""
    return float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)


def _device(t, name):
    """The device number of a call: its first tensor's, which is the current one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError("%s must be on the current CUDA device (cuda:%d), got %s" %
                         (name, torch.cuda.current_device(), t.device))
    return dev


def _on(t, dev, name):
    """t is on the call's device, too."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.get_device() != dev:
        raise ValueError("%s must be on the current CUDA device (cuda:%d), got %s" % (name, dev, t.device))


def _like(x, dtype):
    """A dense tensor of the shape of x, whose rows are dense (_rows), on its device."""
    return torch.empty_like(x) if x.dtype == dtype else torch.empty_like(x, dtype=dtype)


def _dense(t, dtype, ndim, name, dev):
    """A contiguous tensor of the call: its shape."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, dev, name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    shape = t.shape
    if len(shape) != ndim:
        raise ValueError("%s must have %d dims, got %d" % (name, ndim, len(shape)))
    return shape


def _given(t, dtype, shape, name, dev):
    """A tensor of a known shape, an output that the caller supplies above all."""
    if _dense(t, dtype, len(shape), name, dev) != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def _vector(t, n, dtype, name, dev):
    """n elements, or None: the address."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, dev, name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must have %d elements in one dense dim, got %s" % (name, n, tuple(t.shape)))
    return t.data_ptr()


def _scratch(workspace, dev, bytes_needed):
    """The caller's workspace (its size is checked by the library), or a new one of
    bytes_needed() bytes with a clear status word."""
    if workspace is not None:
        _dense(workspace, torch.uint8, 1, "workspace", dev)
        return workspace
    return _workspace(bytes_needed(), torch.device("cuda", dev))


def _rows(t, dtypes, name, dev):
    """Token rows [T, heads, d], each row dense: (elements from row to row, T, heads, d)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, dev, name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be one of %s, got %s" % (name, tuple(dtypes), t.dtype))
    shape = t.shape
    if len(shape) != 3:
        raise ValueError("%s must have 3 dims, got %d" % (name, len(shape)))
    T, heads, d = shape
    rs, hs, cs = t.stride()
    if (cs != 1 and d > 1 or hs != d and heads > 1) and t.numel():
        raise ValueError("%s must have dense [heads, d] rows" % name)
    return (rs if T > 1 else heads * d), T, heads, d


def _freq(inv_freq):
    """(host pointer, rot_dim) of the rotation's frequencies; None: no rotation."""
    if inv_freq is None:
        return None, 0
    if inv_freq.dtype != torch.float64 or inv_freq.is_cuda or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous 1-D float64 CPU tensor")
    return inv_freq.data_ptr(), 2 * inv_freq.numel()


def _qk_sides(q, k):
    """(device number, type, tokens, query heads, key heads, head dim, row strides of q and k)"""
    if q is None and k is None:
        raise ValueError("q or k must be given")
    qs = H = ks = Hk = 0
    if q is not None:
        dev, dtype = _device(q, "q"), q.dtype
        qs, T, H, d = _rows(q, _ODTYPE, "q", dev)
    if k is not None:
        if q is None:
            dev, dtype = _device(k, "k"), k.dtype
        ks, Tk, Hk, dk = _rows(k, _ODTYPE, "k", dev)
        if q is None:
            T, d = Tk, dk
        elif k.dtype != dtype or Tk != T or dk != d:
            raise ValueError("q and k must agree in type, tokens and head dim")
    return dev, dtype, T, H, Hk, d, qs, ks


def csa_qk_norm_rope(q, k, inv_freq, wq=None, wk=None, eps=1e-6, pos=None, t0=0, rot_start=0, rot_style=ROPE_HALVES,
                     yq=None, yk=None, out_dtype=None):
    """Per-head RMS norm (weights wq/wk [d] f32; None: no norm) and position
    rotation of queries q [T,H,d] and keys k [T,Hk,d] (bf16 or fp32; views of a
    packed projection are fine; either may be None).  inv_freq [rot/2] float64 on
    the CPU (None: no rotation), turning channels rot_start .. rot_start + rot.
    pos [T] int64 positions on the device, or None: t0, t0 + 1, ...
    Returns (yq, yk) of out_dtype (default: the inputs' type), which autograd does
    not follow: gradients come from csa_qk_norm_rope_backward."""
    dev, dtype, T, H, Hk, d, qs, ks = _qk_sides(q, k)
    ot = dtype if out_dtype is None else out_dtype
    wqp, wkp = _vector(wq, d, torch.float32, "wq", dev), _vector(wk, d, torch.float32, "wk", dev)
    pp = _vector(pos, T, torch.int64, "pos", dev)
    fp, rot = _freq(inv_freq)
    if ot not in _ODTYPE:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    if q is not None:
        yq = _like(q, ot) if yq is None else _given(yq, ot, q.shape, "yq", dev)
    if k is not None:
        yk = _like(k, ot) if yk is None else _given(yk, ot, k.shape, "yk", dev)
    if q is None and yq is not None or k is None and yk is not None:
        raise ValueError("an output without its input")
    _check(lib().csa_qk_norm_rope(_ptr(q), qs, _ptr(k), ks, wqp, wkp, eps, pp, t0, fp, rot_start, rot, rot_style, T, H,
                                  Hk, d, _ODTYPE[dtype], _ptr(yq), _ptr(yk), _ODTYPE[ot], _stream(dev)),
           "csa_qk_norm_rope")
    return yq, yk


def csa_qk_norm_rope_backward(q, k, dyq, dyk, inv_freq, wq=None, wk=None, eps=1e-6, pos=None, t0=0, rot_start=0,
                              rot_style=ROPE_HALVES, dq=None, dk=None, dwq=None, dwk=None, workspace=None):
    """Gradients of csa_qk_norm_rope from dyq/dyk (the types and shapes of yq/yk):
    dq/dk of q's type (given ones may be views of a packed gradient), dwq/dwk [d]
    f32.  Returns (dq, dk, dwq, dwk, workspace), None where there is no input."""
    dev, dtype, T, H, Hk, d, qs, ks = _qk_sides(q, k)
    wqp, wkp = _vector(wq, d, torch.float32, "wq", dev), _vector(wk, d, torch.float32, "wk", dev)
    pp = _vector(pos, T, torch.int64, "pos", dev)
    fp, rot = _freq(inv_freq)
    dy = dyq if q is not None else dyk
    if dy is None or dy.dtype not in _ODTYPE:
        raise TypeError("the gradients must be torch.bfloat16 or torch.float32")
    yt = dy.dtype
    sides = []
    for x, dy, dx, w, dw, heads, n in ((q, dyq, dq, wq, dwq, H, "q"), (k, dyk, dk, wk, dwk, Hk, "k")):
        if x is None:
            if dy is not None or dx is not None or dw is not None:
                raise ValueError("gradients of %s without %s" % (n, n))
            sides.append((None, 0, None, None))
            continue
        shape = (T, heads, d)
        _given(dy, yt, shape, "dy", dev)
        if dx is None:
            dx, stride = _like(x, dtype), heads * d
        else:
            stride, *got = _rows(dx, (dtype,), "dx", dev)
            if tuple(got) != shape:
                raise ValueError("d%s must have shape %s" % (n, shape))
        if w is None:
            if dw is not None:
                raise ValueError("dw%s without w%s" % (n, n))
            sides.append((dx, stride, None, None))
        else:
            if dw is None:
                dw = torch.empty_like(w)
                dwp = dw.data_ptr()
            else:
                dwp = _vector(dw, d, torch.float32, "dw", dev)
            if heads == 0:  # the library leaves the side out
                dw.zero_()
                dwp = None
            sides.append((dx, stride, dw, dwp))
    (dq, dqs, dwq, dwqp), (dk, dks, dwk, dwkp) = sides
    L = lib()
    ws = _scratch(workspace, dev, lambda: L.csa_qk_norm_rope_backward_workspace_bytes(T, H, Hk, d))
    _check(L.csa_qk_norm_rope_backward(_ptr(q), qs, _ptr(k), ks, wqp if H else None, wkp if Hk else None, eps, pp, t0,
                                       fp, rot_start, rot, rot_style, _ptr(dyq), _ptr(dyk), T, H, Hk, d,
                                       _ODTYPE[dtype], _ODTYPE[yt], _ptr(dq), dqs, _ptr(dk), dks, dwqp, dwkp,
                                       ws.data_ptr(), ws.numel(), _stream(dev)), "csa_qk_norm_rope_backward")
    return dq, dk, dwq, dwk, ws


_BF16 = (torch.bfloat16,)


def _paged(Kpages, Vpages, dev):
    """(pages, key heads, rows a page, d) of a paged cache."""
    shape = _dense(Kpages, torch.bfloat16, 4, "Kpages", dev)
    if _dense(Vpages, torch.bfloat16, 4, "Vpages", dev) != shape:
        raise ValueError("Kpages and Vpages must have the same shape")
    return shape


def csa_paged_append(k, v, Kpages, Vpages, block_table, seq, pos, inv_freq, slot=None, wk=None, eps=1e-6, rot_start=0,
                     rot_style=ROPE_HALVES, workspace=None):
    """Write the tokens' keys (normed by wk [d] f32 unless None, rotated to pos) and
    values into a paged cache, in place: k, v [T,Hk,d] bf16 (views of a packed
    projection are fine); Kpages/Vpages [n_pages,Hk,page,d] bf16; block_table
    [B,max_pages] int32; seq [T] int32; pos, slot [T] int64 on the device (slot
    None: pos; a negative slot skips its token).  Returns the workspace, whose
    status word reports numbers outside their tables."""
    dev = _device(k, "k")
    n_pages, Hk, page, d = _paged(Kpages, Vpages, dev)
    B, max_pages = _dense(block_table, torch.int32, 2, "block_table", dev)
    ks, T, kh, kd = _rows(k, _BF16, "k", dev)
    vs, Tv, vh, vd = _rows(v, _BF16, "v", dev)
    if Tv != T or kh != Hk or vh != Hk or kd != d or vd != d:
        raise ValueError("k and v must be [T, %d, %d]" % (Hk, d))
    wp = _vector(wk, d, torch.float32, "wk", dev)
    pp, sp = _vector(pos, T, torch.int64, "pos", dev), _vector(slot, T, torch.int64, "slot", dev)
    bp = _vector(seq, T, torch.int32, "seq", dev)
    fp, rot = _freq(inv_freq)
    ws = _scratch(workspace, dev, lambda: 256)
    _check(lib().csa_paged_append(k.data_ptr(), ks, v.data_ptr(), vs, wp, eps, pp, sp, bp, fp, rot_start, rot,
                                  rot_style, block_table.data_ptr(), T, Hk, d, B, max_pages, n_pages, page,
                                  Kpages.data_ptr(), Vpages.data_ptr(), ws.data_ptr(), ws.numel(), _stream(dev)),
           "csa_paged_append")
    return ws


def csa_tree_attn(q, Kpages, Vpages, block_table, seq_lens, q_start, mask, scale, W=-1, pos=None, O=None, lse=None,
                  want_lse=True, workspace=None, out_dtype=torch.bfloat16):
    """Attention of drafted tokens (or of one token a sequence) over a paged cache:
    q [R,H,d] bf16, the rows q_start[b] .. q_start[b+1] of it the nodes of sequence
    b, whose cache rows follow its seq_lens[b] committed ones; mask [R] int64
    (storage of the uint64 bits): the drafted rows of its own sequence that a row
    sees; W >= 0: committed rows s > pos[r] - W only.  Returns (O, lse, workspace)."""
    dev = _device(q, "q")
    n_pages, Hk, page, d = _paged(Kpages, Vpages, dev)
    B, max_pages = _dense(block_table, torch.int32, 2, "block_table", dev)
    shape = _dense(q, torch.bfloat16, 3, "q", dev)
    R, H, dq = shape
    if dq != d:
        raise ValueError("q must have head dim %d, got %d" % (d, dq))
    lp, sp = _vector(seq_lens, B, torch.int32, "seq_lens", dev), _vector(q_start, B + 1, torch.int32, "q_start", dev)
    mp, pp = _vector(mask, R, torch.int64, "mask", dev), _vector(pos, R, torch.int64, "pos", dev)
    if out_dtype not in _ODTYPE:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    O = _like(q, out_dtype) if O is None else _given(O, out_dtype, shape, "O", dev)
    if lse is not None:
        _given(lse, torch.float32, (R, H), "lse", dev)
    elif want_lse:
        lse = q.new_empty((R, H), dtype=torch.float32)
    L = lib()
    ws = _scratch(workspace, dev, lambda: L.csa_tree_attn_workspace_bytes(B, R, H, Hk, d, page, max_pages))
    _check(L.csa_tree_attn(q.data_ptr(), Kpages.data_ptr(), Vpages.data_ptr(), block_table.data_ptr(), lp, sp, mp, pp,
                           R, B, H, Hk, d, page, n_pages, max_pages, W, scale, O.data_ptr(), _ODTYPE[out_dtype],
                           _ptr(lse), ws.data_ptr(), ws.numel(), _stream(dev)), "csa_tree_attn")
    return O, lse, ws
