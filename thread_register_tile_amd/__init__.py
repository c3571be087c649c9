"""Python binding of libtrt.so, the MI355X register-tile GEMM library.

Argument marshalling only: every step of the computation runs in the HIP
kernels of libtrt.so.  PyTorch provides device memory and the current
stream; nothing here computes on tensors.  If the library is not built, every
call raises -- there is no fallback path.

    import thread_register_tile_amd as trt
    C = trt.gemm(A, B)                          # C = A @ B
    C = trt.gemm(A, B, bias=b, relu=True, residual=R)
    C = trt.gemm(At, B, opA="T")                # A stored transposed
    y = trt.layernorm(x, gamma, beta)
    dx, dgamma, dbeta = trt.layernorm_bwd(dy, x, gamma)
    loss, lse = trt.linear_xent(x, W, target)   # cross entropy of x @ W.T
    dx, dW = trt.linear_xent_bwd(x, W, target, lse, dloss)
    r, h = trt.block_norm(r0, y, gate)          # r = r0 + gate N(y), h = N(r)
    grads = trt.block_norm_bwd(dh, dr, r, y, gate)
    q, scale = trt.act8_pack(x)                 # x in 8 bits, a scale to 32 columns
    x = trt.act8_unpack(q, scale, torch.bfloat16)
    dW = trt.act8_weight_grad(dy, q, scale)     # dy.T @ x
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtrt.so")

# status codes (include/trt.h)
OK, ERR_SIZE, ERR_STRIDE, ERR_NULL, ERR_ALIGN, ERR_OVERLAP, ERR_DTYPE, \
    ERR_UNSUPPORTED, ERR_HIP, ERR_ARG = range(10)
STATUS_NAMES = {OK: "TRT_OK", ERR_SIZE: "TRT_ERR_SIZE", ERR_STRIDE: "TRT_ERR_STRIDE",
                ERR_NULL: "TRT_ERR_NULL", ERR_ALIGN: "TRT_ERR_ALIGN",
                ERR_OVERLAP: "TRT_ERR_OVERLAP", ERR_DTYPE: "TRT_ERR_DTYPE",
                ERR_UNSUPPORTED: "TRT_ERR_UNSUPPORTED", ERR_HIP: "TRT_ERR_HIP",
                ERR_ARG: "TRT_ERR_ARG"}

F16, BF16, F32 = 1, 2, 3
OP_N, OP_T = 0, 1

MAP_C_OWNER = 0
MAP_LDS_SLOT_A = 1
MAP_LDS_SLOT_B = 2
MAP_COPY_KCONTIG_A = 3
MAP_COPY_MNCONTIG_A = 4
MAP_COPY_KCONTIG_B = 5
MAP_COPY_MNCONTIG_B = 6
MAP_DMA_KC_SLOT_A = 7
MAP_DMA_KC_SLOT_B = 8
MAP_DMA_MN_SLOT_A = 9
MAP_DMA_MN_SLOT_B = 10


class TrtError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("relu", ctypes.c_int32),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("row_scale", ctypes.c_void_p)]


class Block(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("rows_per_gate", ctypes.c_int64),
                ("post_gamma", ctypes.c_void_p), ("post_beta", ctypes.c_void_p),
                ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float), ("post", ctypes.c_int32), ("rms", ctypes.c_int32),
                ("gate_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32)]


class Saved(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scale", ctypes.c_void_p),
                ("lds", ctypes.c_int64)]


class BlockGrads(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("post_gamma", ctypes.c_void_p),
                ("post_beta", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p)]


class TileDesc(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("bk", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded libtrt.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m thread_register_tile_amd.build` (no fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
        gemm_args = [i64, i64, i64, vp, i64, i32, vp, i64, i32, vp, i64, i32, i32,
                     ctypes.POINTER(Epilogue)]
        L.trt_gemm.argtypes = gemm_args + [vp]
        L.trt_gemm.restype = i32
        L.trt_gemm_tiled.argtypes = gemm_args + [ctypes.POINTER(TileDesc), vp]
        L.trt_gemm_tiled.restype = i32
        L.trt_validate.argtypes = gemm_args + [ctypes.POINTER(TileDesc)]
        L.trt_validate.restype = i32
        L.trt_gemm_ws.argtypes = gemm_args + [vp, i64, vp]
        L.trt_gemm_ws.restype = i32
        L.trt_gemm_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32]
        L.trt_gemm_workspace_size.restype = i64
        L.trt_gemm_noalloc.argtypes = gemm_args + [vp]
        L.trt_gemm_noalloc.restype = i32
        L.trt_tile_count.argtypes = []
        L.trt_tile_count.restype = i32
        L.trt_tile_at.argtypes = [i32, ctypes.POINTER(TileDesc), ctypes.POINTER(i32),
                                  ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.trt_tile_at.restype = i32
        L.trt_layout_dump.argtypes = [i32, ctypes.POINTER(TileDesc), vp, vp, i64, vp]
        L.trt_layout_dump.restype = i32
        L.trt_layout_dump_host.argtypes = [i32, ctypes.POINTER(TileDesc), vp, vp, i64]
        L.trt_layout_dump_host.restype = i32
        L.trt_layout_size.argtypes = [i32, ctypes.POINTER(TileDesc)]
        L.trt_layout_size.restype = i64
        L.trt_layout_rank.argtypes = [ctypes.POINTER(TileDesc), ctypes.POINTER(i32),
                                      ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.trt_layout_rank.restype = i32
        L.trt_mfma_probe.argtypes = [i32, i32, vp, vp, vp, vp]
        L.trt_mfma_probe.restype = i32
        L.trt_hbm_read_probe.argtypes = [vp, i64, vp, i64, vp]
        L.trt_hbm_read_probe.restype = i32
        L.trt_mfma_loop_probe.argtypes = [i32, vp, i32, vp, i64, vp]
        L.trt_mfma_loop_probe.restype = i32
        L.trt_clock_probe.argtypes = [i64, vp, i64, vp]
        L.trt_clock_probe.restype = i32
        u32p = ctypes.POINTER(ctypes.c_uint32)
        L.trt_gf2_rank.argtypes = [i32, i32, u32p]
        L.trt_gf2_rank.restype = i32
        L.trt_gf2_compose.argtypes = [i32, i32, u32p, i32, i32, u32p, u32p]
        L.trt_gf2_compose.restype = i32
        L.trt_gf2_product.argtypes = [i32, i32, u32p, i32, i32, u32p, u32p]
        L.trt_gf2_product.restype = i32
        L.trt_gf2_sublayout.argtypes = [i32, i32, u32p, ctypes.c_uint32, ctypes.c_uint32, u32p,
                                        ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.trt_gf2_sublayout.restype = i32
        L.trt_gf2_invert_and_compose.argtypes = [i32, i32, u32p, i32, u32p, u32p]
        L.trt_gf2_invert_and_compose.restype = i32
        L.trt_block_reduce.argtypes = [vp, i64, i64, i32, i32, vp, vp]
        L.trt_block_reduce.restype = i32
        i32p = ctypes.POINTER(i32)
        L.trt_regtile_thread_shape.argtypes = [i32, i32, i32, i32p, i32p]
        L.trt_regtile_thread_shape.restype = i32
        L.trt_regtile_owner.argtypes = [i32, i32, i32, i32, vp, vp, i64]
        L.trt_regtile_owner.restype = i32
        L.trt_gemm_regtile.argtypes = gemm_args + [i32, i32, i32, vp]
        L.trt_gemm_regtile.restype = i32
        L.trt_choose_tile.argtypes = [i64, i64, i32, ctypes.POINTER(TileDesc)]
        L.trt_choose_tile.restype = i32
        f32 = ctypes.c_float
        L.trt_layernorm.argtypes = [i64, i64, vp, i64, vp, vp, f32, vp, i64, i32, i32, vp]
        L.trt_layernorm.restype = i32
        L.trt_layernorm_bwd_workspace_size.argtypes = [i64, i64, i32]
        L.trt_layernorm_bwd_workspace_size.restype = i64
        L.trt_layernorm_bwd.argtypes = [i64, i64, vp, i64, vp, i64, vp, f32, vp, i64, vp, vp, i32,
                                        i32, vp, i64, vp]
        L.trt_layernorm_bwd.restype = i32
        L.trt_linear_xent_workspace_size.argtypes = [i64, i64, i64]
        L.trt_linear_xent_workspace_size.restype = i64
        L.trt_linear_xent.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp, i32, vp, i64,
                                      vp]
        L.trt_linear_xent.restype = i32
        L.trt_linear_xent_bwd_workspace_size.argtypes = [i64, i64, i64, i64]
        L.trt_linear_xent_bwd_workspace_size.restype = i64
        L.trt_linear_xent_bwd.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64, vp,
                                          i64, vp, i64, vp, i64, i32, i32, i64, vp, i64, vp]
        L.trt_linear_xent_bwd.restype = i32
        L.trt_act8_pack.argtypes = [i64, i64, vp, i64, vp, i64, vp, i64, i32, vp]
        L.trt_act8_pack.restype = i32
        L.trt_act8_unpack.argtypes = [i64, i64, vp, i64, vp, i64, vp, i64, i32, vp]
        L.trt_act8_unpack.restype = i32
        L.trt_act8_weight_grad_workspace_size.argtypes = [i64, i64, i64, vp, i64]
        L.trt_act8_weight_grad_workspace_size.restype = i64
        L.trt_act8_weight_grad.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32,
                                           i32, vp, i64, vp]
        L.trt_act8_weight_grad.restype = i32
        L.trt_block_norm.argtypes = [i64, i64, vp, i64, vp, i64, ctypes.POINTER(Block), vp, i64, vp, i64,
                                     i32, vp]
        L.trt_block_norm.restype = i32
        L.trt_block_norm_bwd_workspace_size.argtypes = [i64, i64, i64, i32]
        L.trt_block_norm_bwd_workspace_size.restype = i64
        L.trt_block_norm_bwd.argtypes = [i64, i64, vp, i64, vp, i64, ctypes.POINTER(Saved),
                                         ctypes.POINTER(Saved), ctypes.POINTER(Block), vp, i64, vp, i64,
                                         ctypes.POINTER(BlockGrads), i32, vp, i64, vp]
        L.trt_block_norm_bwd.restype = i32
        L.trt_abi_version.argtypes = []
        L.trt_abi_version.restype = i32
        L.trt_last_error.argtypes = []
        L.trt_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def last_error() -> str:
    return lib().trt_last_error().decode()


def abi_version() -> int:
    return lib().trt_abi_version()


def _check(status):
    if status != OK:
        raise TrtError(status, last_error())


def _tile(tile):
    if tile is None:
        return None
    return ctypes.byref(TileDesc(*tile))


def _epi(bias_ptr, relu, res_ptr, ldr, scale_ptr=0):
    if not bias_ptr and not relu and not res_ptr and not scale_ptr:
        return None
    return ctypes.byref(Epilogue(bias_ptr or None, int(bool(relu)), res_ptr or None, ldr,
                                 scale_ptr or None))


# ---- raw entry points (pointers and sizes, as in include/trt.h) --------------

def gemm_raw(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype, out_dtype,
             bias=0, relu=False, residual=0, ldr=0, scale=0, tile=None, stream=0):
    """trt_gemm_tiled on raw device addresses (ints).  Raises TrtError."""
    _check(lib().trt_gemm_tiled(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype,
                                out_dtype, _epi(bias, relu, residual, ldr, scale),
                                _tile(tile), stream or None))


def gemm_ws_raw(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype, out_dtype,
                bias=0, relu=False, residual=0, ldr=0, scale=0, workspace=0, workspace_bytes=0,
                stream=0):
    """trt_gemm_ws on raw device addresses (ints).  Raises TrtError."""
    _check(lib().trt_gemm_ws(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype, out_dtype,
                             _epi(bias, relu, residual, ldr, scale), workspace or None,
                             workspace_bytes, stream or None))


NOALLOC_SCRATCH_BYTES = 16777216   # TRT_NOALLOC_SCRATCH_BYTES


def gemm_noalloc_raw(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype, out_dtype,
                     bias=0, relu=False, residual=0, ldr=0, scale=0, stream=0):
    """trt_gemm_noalloc on raw device addresses (ints).  Raises TrtError."""
    _check(lib().trt_gemm_noalloc(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype,
                                  out_dtype, _epi(bias, relu, residual, ldr, scale),
                                  stream or None))


def workspace_size(M, N, K, opA=OP_N, opB=OP_N, in_dtype=F16) -> int:
    """trt_gemm_workspace_size: bytes of workspace trt_gemm_ws uses (0: none)."""
    n = lib().trt_gemm_workspace_size(M, N, K, opA, opB, in_dtype)
    if n < 0:
        raise TrtError(ERR_ARG, last_error())
    return n


def validate_raw(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype, out_dtype,
                 bias=0, relu=False, residual=0, ldr=0, scale=0, tile=None) -> int:
    """trt_validate: the status a call would return, without any GPU work."""
    return lib().trt_validate(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype,
                              out_dtype, _epi(bias, relu, residual, ldr, scale), _tile(tile))


def choose_tile(M, N, in_dtype=F16):
    """trt_choose_tile: the (BM, BN, BK) tile trt_gemm uses for an M x N output."""
    t = TileDesc()
    _check(lib().trt_choose_tile(M, N, in_dtype, ctypes.byref(t)))
    return (t.bm, t.bn, t.bk)


def tiles():
    """Compiled tiles: [(bm, bn, bk, waves_m, waves_n, regs_per_lane, frag), ...]
    where frag is the edge (16 or 32) of the matrix-core fragments."""
    out = []
    for i in range(lib().trt_tile_count()):
        t = TileDesc()
        wm, wn, regs, fr = (ctypes.c_int32() for _ in range(4))
        _check(lib().trt_tile_at(i, ctypes.byref(t), ctypes.byref(wm), ctypes.byref(wn),
                                 ctypes.byref(regs), ctypes.byref(fr)))
        out.append((t.bm, t.bn, t.bk, wm.value, wn.value, regs.value, fr.value))
    return out


def layout_size(map_id, tile) -> int:
    return lib().trt_layout_size(map_id, _tile(tile))


def layout_rank(tile):
    r, i, o = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().trt_layout_rank(_tile(tile), ctypes.byref(r), ctypes.byref(i), ctypes.byref(o)))
    return r.value, i.value, o.value


def layout_dump_host(map_id, tile):
    """Evaluate a layout map on the host: returns (rows, cols) numpy int32."""
    import numpy as np
    n = layout_size(map_id, tile)
    if n < 0:
        raise TrtError(ERR_ARG, "unknown map or tile")
    rows = np.empty(n, dtype=np.int32)
    cols = np.empty(n, dtype=np.int32)
    _check(lib().trt_layout_dump_host(map_id, _tile(tile), rows.ctypes.data,
                                      cols.ctypes.data, n))
    return rows, cols


# ---- torch-facing helpers (device memory and the current stream) ----------------

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


_DT = {}


def _code_of(dtype):
    code = _DT.get(dtype)
    if code is None:
        torch = _torch()
        _DT.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
        if dtype not in _DT:
            raise TrtError(ERR_DTYPE, f"unsupported dtype {dtype}")
        code = _DT[dtype]
    return code


def _dtype_code(t):
    return _code_of(t.dtype)


def _stream(device):
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


def _ld(t, name):
    """Leading dimension of a 2-D tensor whose inner stride is 1."""
    if t.dim() != 2:
        raise TrtError(ERR_ARG, f"{name} must be 2-D")
    if t.stride(1) != 1 and t.size(1) > 1:
        raise TrtError(ERR_STRIDE, f"{name} must have unit inner stride")
    return max(t.stride(0), 1)


def _gemm_call(A, B, opA, opB, bias, relu, residual, row_scale, out, out_dtype, M, N, K):
    """Shapes, dtypes and raw pointers of a GEMM on torch tensors; allocates
    `out` if it is not given.  Returns (out, positional args, keyword args)
    for gemm_raw / gemm_regtile_raw."""
    torch = _torch()
    opa = OP_T if opA in ("T", OP_T, True) else OP_N
    opb = OP_T if opB in ("T", OP_T, True) else OP_N
    M_ = A.size(1) if opa else A.size(0)
    K_ = A.size(0) if opa else A.size(1)
    N_ = B.size(0) if opb else B.size(1)
    KB = B.size(1) if opb else B.size(0)
    if KB != K_:
        raise TrtError(ERR_SIZE, f"inner dimensions differ: {K_} vs {KB}")
    M, N, K = M or M_, N or N_, K or K_
    dt = _dtype_code(A)
    if _dtype_code(B) != dt:
        raise TrtError(ERR_DTYPE, "A and B dtypes differ")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or A.dtype, device=A.device)
    odt = _dtype_code(out)
    for name, t, need in (("bias", bias, N), ("row_scale", row_scale, M)):
        if t is None:
            continue
        if t.dtype != out.dtype:
            raise TrtError(ERR_DTYPE, f"{name} must have the output dtype {out.dtype}")
        if not t.is_contiguous() or t.numel() < need:
            raise TrtError(ERR_SIZE, f"{name} must be contiguous with at least {need} elements")
    ldr = 0
    if residual is not None:
        if residual.dtype != out.dtype:
            raise TrtError(ERR_DTYPE, f"residual must have the output dtype {out.dtype}")
        if residual.dim() != 2 or residual.size(0) < M or residual.size(1) < N:
            raise TrtError(ERR_SIZE, f"residual must be at least [{M}, {N}]")
        ldr = _ld(residual, "residual")
    args = (M, N, K, A.data_ptr(), _ld(A, "A"), opa, B.data_ptr(), _ld(B, "B"), opb,
            out.data_ptr(), _ld(out, "out"), dt, odt)
    kw = dict(bias=bias.data_ptr() if bias is not None else 0, relu=relu,
              residual=residual.data_ptr() if residual is not None else 0, ldr=ldr,
              scale=row_scale.data_ptr() if row_scale is not None else 0,
              stream=_stream(A.device))
    return out, args, kw


def gemm(A, B, *, opA="N", opB="N", bias=None, relu=False, residual=None, row_scale=None,
         out=None, out_dtype=None, tile=None, M=None, N=None, K=None):
    """C = relu((A.B) * row_scale[:, None] + bias) + residual on the GPU, in one kernel.

    A is [M, K] (opA="N") or its transpose stored as [K, M] (opA="T"); B is
    [K, N] (opB="N") or stored as [N, K] (opB="T"); A and B share one dtype,
    float16, bfloat16 or float32.  Tensors may be
    row-padded views (unit inner stride, any row stride).  bias is [N],
    row_scale [M], residual [M, N], all of the output dtype: out's dtype if
    out is given, else out_dtype (a torch dtype: float16, bfloat16 or
    float32), else A's dtype.  out, if given, is written; otherwise a new
    [M, N] tensor is returned.  Runs on torch's current stream; no
    synchronisation.
    """
    out, args, kw = _gemm_call(A, B, opA, opB, bias, relu, residual, row_scale, out, out_dtype,
                               M, N, K)
    gemm_raw(*args, tile=tile, **kw)
    return out


def gemm_regtile(A, B, *, lm, ln, max_threads=None, opA="N", opB="N", bias=None, relu=False,
                 residual=None, row_scale=None, out=None, out_dtype=None):
    """gemm() computed on vector lanes with a register tile of logical shape
    (lm, ln) and the thread shape regtile_thread_shape(lm, ln, max_threads)
    (trt_gemm_regtile).  Same arguments and result as gemm()."""
    out, args, kw = _gemm_call(A, B, opA, opB, bias, relu, residual, row_scale, out, out_dtype,
                               None, None, None)
    gemm_regtile_raw(*args, lm, ln, max_threads or REGTILE_MAX_THREADS, **kw)
    return out


def layout_dump(map_id, tile, device="cuda"):
    """Evaluate a layout map with the kernels' device functions; returns
    (rows, cols) as int32 tensors on `device`."""
    torch = _torch()
    n = layout_size(map_id, tile)
    if n < 0:
        raise TrtError(ERR_ARG, "unknown map or tile")
    rows = torch.empty(n, dtype=torch.int32, device=device)
    cols = torch.empty(n, dtype=torch.int32, device=device)
    _check(lib().trt_layout_dump(map_id, _tile(tile), rows.data_ptr(), cols.data_ptr(), n,
                                 _stream(rows.device)))
    return rows, cols


def mfma_probe(a_regs, b_regs, dtype=F16, shape=16):
    """Run one matrix-core instruction (shape 16: 16x16x32, 32: 32x32x16):
    a_regs, b_regs are [64, 8] 16-bit tensors (lane-major operand registers);
    returns [64, 4] (shape 16) or [64, 16] (shape 32) fp32."""
    torch = _torch()
    c = torch.empty((64, 4 if shape == 16 else 16), dtype=torch.float32, device=a_regs.device)
    a = a_regs.contiguous()
    b = b_regs.contiguous()
    _check(lib().trt_mfma_probe(dtype, shape, a.data_ptr(), b.data_ptr(), c.data_ptr(),
                                _stream(a.device)))
    return c


READ_PROBE_SINK_BYTES = 32768   # TRT_READ_PROBE_SINK_BYTES


def hbm_read_probe_raw(x, nbytes, sink, sink_bytes, stream=0):
    """trt_hbm_read_probe on raw device addresses; raises TrtError on error."""
    _check(lib().trt_hbm_read_probe(x, nbytes, sink, sink_bytes, stream))


def hbm_read_probe(x, sink=None):
    """Stream-read the bytes of device tensor x once (a bandwidth yardstick);
    returns the [2048, 16]-byte digest tensor (uint8), whose XOR over rows is
    the XOR of x's 16-byte words."""
    torch = _torch()
    if sink is None:
        sink = torch.empty(READ_PROBE_SINK_BYTES, dtype=torch.uint8, device=x.device)
    hbm_read_probe_raw(x.data_ptr(), x.numel() * x.element_size(), sink.data_ptr(),
                       sink.numel() * sink.element_size(), _stream(x.device))
    return sink.view(-1, 16)


MFMA_PROBE_OPERAND_BYTES = 16384   # TRT_MFMA_PROBE_OPERAND_BYTES
MFMA_PROBE_SINK_BYTES = 4194304    # TRT_MFMA_PROBE_SINK_BYTES


def mfma_loop_probe_raw(dtype, operands, iters, sink, sink_bytes, stream=0):
    """trt_mfma_loop_probe on raw device addresses; raises TrtError on error."""
    _check(lib().trt_mfma_loop_probe(dtype, operands, iters, sink, sink_bytes, stream))


def mfma_loop_probe(operands, iters, dtype=F16, sink=None):
    """Run the matrix-core yardstick on a device tensor of 16 KiB of operand
    data; returns the [256*256, 16] fp32 sums (one row per thread)."""
    torch = _torch()
    if sink is None:
        sink = torch.empty(MFMA_PROBE_SINK_BYTES // 4, dtype=torch.float32,
                           device=operands.device)
    mfma_loop_probe_raw(dtype, operands.data_ptr(), iters, sink.data_ptr(),
                        sink.numel() * sink.element_size(), _stream(operands.device))
    return sink.view(-1, 16)


def mfma_loop_probe_flops(iters, dtype=F16):
    """FLOPs of one trt_mfma_loop_probe launch."""
    if dtype == F32:
        return 256 * 4 * iters * 32 * (2 * 16 * 16 * 4)
    return 256 * 4 * iters * 64 * (2 * 16 * 16 * 32)


CLOCK_PROBE_SINK_BYTES = 4096     # TRT_CLOCK_PROBE_SINK_BYTES


def clock_probe_raw(ticks, sink, sink_bytes, stream=0):
    """trt_clock_probe on a raw device address; raises TrtError on error."""
    _check(lib().trt_clock_probe(ticks, sink, sink_bytes, stream))


def clock_probe(ticks, device="cuda", sink=None):
    """Run the clock yardstick once on the current stream; returns the device
    tensor of [256, 2] int64 (shader cycles, real-time ticks) per workgroup."""
    torch = _torch()
    if sink is None:
        sink = torch.empty(CLOCK_PROBE_SINK_BYTES // 8, dtype=torch.int64, device=device)
    clock_probe_raw(ticks, sink.data_ptr(), sink.numel() * sink.element_size(),
                    _stream(sink.device))
    return sink.view(-1, 2)


# ---- the GF(2) layout algebra (host only; maps as lists of column words) -------

def _u32(cols):
    arr = (ctypes.c_uint32 * max(len(cols), 1))(*[int(c) for c in cols])
    return arr


def gf2_rank(cols, nout):
    r = lib().trt_gf2_rank(len(cols), nout, _u32(cols))
    if r < 0:
        raise TrtError(ERR_ARG, last_error())
    return r


def gf2_compose(outer, outer_nout, inner, inner_nout):
    """outer o inner (outer has inner_nout input bits)."""
    out = (ctypes.c_uint32 * max(len(inner), 1))()
    _check(lib().trt_gf2_compose(len(outer), outer_nout, _u32(outer), len(inner), inner_nout,
                                 _u32(inner), out))
    return list(out)[:len(inner)]


def gf2_product(a, a_nout, b, b_nout):
    out = (ctypes.c_uint32 * max(len(a) + len(b), 1))()
    _check(lib().trt_gf2_product(len(a), a_nout, _u32(a), len(b), b_nout, _u32(b), out))
    return list(out)[:len(a) + len(b)]


def gf2_sublayout(cols, nout, in_mask, out_mask):
    """Returns (columns, nin, nout) of the restricted, projected map."""
    out = (ctypes.c_uint32 * 32)()
    ni, no = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().trt_gf2_sublayout(len(cols), nout, _u32(cols), in_mask, out_mask, out,
                                   ctypes.byref(ni), ctypes.byref(no)))
    return list(out)[:ni.value], ni.value, no.value


def gf2_invert_and_compose(R, S, t_bits):
    """Q with S(Q(x)) == R(x); raises TrtError (ERR_ARG) when R leaves S's image."""
    out = (ctypes.c_uint32 * max(len(R), 1))()
    _check(lib().trt_gf2_invert_and_compose(len(R), t_bits, _u32(R), len(S), _u32(S), out))
    return list(out)[:len(R)]


# ---- the rank-1 block reduction ---------------------------------------------------

# ---- register tiles of any logical shape -------------------------------------

REGTILE_MAX_THREADS = 64     # one wavefront per tile
REGTILE_MAX_REGS = 8         # registers per axis


def regtile_thread_shape(lm, ln, max_threads=REGTILE_MAX_THREADS):
    """trt_regtile_thread_shape: the physical thread shape (tm, tn) the
    deterministic policy picks for a logical (lm, ln) tile."""
    tm, tn = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().trt_regtile_thread_shape(lm, ln, max_threads, ctypes.byref(tm),
                                          ctypes.byref(tn)))
    return tm.value, tn.value


def regtile_owner(lm, ln, tm, tn):
    """trt_regtile_owner: (rows, cols) int32 arrays indexed by
    thread * registers_per_thread + register."""
    import numpy as np
    n = lm * ln
    rows = np.empty(max(n, 1), dtype=np.int32)
    cols = np.empty(max(n, 1), dtype=np.int32)
    _check(lib().trt_regtile_owner(lm, ln, tm, tn, rows.ctypes.data, cols.ctypes.data, n))
    return rows[:n], cols[:n]


def gemm_regtile_raw(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype, out_dtype, lm, ln,
                     max_threads=REGTILE_MAX_THREADS, bias=0, relu=False, residual=0, ldr=0,
                     scale=0, stream=0):
    """trt_gemm_regtile on raw device addresses (ints).  Raises TrtError."""
    _check(lib().trt_gemm_regtile(M, N, K, A, lda, opA, B, ldb, opB, C, ldc, in_dtype,
                                  out_dtype, _epi(bias, relu, residual, ldr, scale), lm, ln,
                                  max_threads, stream or None))


REDUCE_SUM, REDUCE_MAX, REDUCE_MIN = 0, 1, 2


def block_reduce_raw(x, n, block, dtype, op, out, stream=0):
    """trt_block_reduce on raw device addresses; raises TrtError on error."""
    _check(lib().trt_block_reduce(x, n, block, dtype, op, out, stream or None))


def block_reduce(x, block, op=REDUCE_SUM, out=None):
    """out[b] = op over each block of `block` consecutive elements of the 1-D
    device tensor x (float16, bfloat16 or float32); returns float32 [nblocks]."""
    torch = _torch()
    n = x.numel()
    nb = -(-n // block)
    if out is None:
        out = torch.empty(nb, dtype=torch.float32, device=x.device)
    block_reduce_raw(x.data_ptr(), n, block, _dtype_code(x), op, out.data_ptr(), _stream(x.device))
    return out


# ---- the layer norm and its gradients ---------------------------------------------

def _device(first, **others):
    """The CUDA device that every tensor given lives on."""
    dev = first.device
    if dev.type != "cuda":
        raise TrtError(ERR_ARG, "tensors must be on a GPU")
    for name, t in others.items():
        if t is not None and t.device != dev:
            raise TrtError(ERR_ARG, f"{name} is on {t.device}, not on {dev}")
    return dev


def _place(first, *others):
    """_device for calls of many small tensors: the device that all of them live on."""
    index = first.get_device()
    if index < 0:
        raise TrtError(ERR_ARG, "tensors must be on a GPU")
    for t in others:
        if t is not None and t.get_device() != index:
            raise TrtError(ERR_ARG, f"a tensor is on {t.device}, not on {first.device}")
    return first.device


def _on(dev, status_of):
    """status_of(stream) with dev current (a launch goes to the current device)."""
    torch = _torch()
    # (the handle itself, where torch gives it: making a Stream object of it takes
    # 1.7 us of a call's 10)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    stream = (raw(dev.index) if raw else _stream(dev)) or None
    if torch.cuda.current_device() == dev.index:
        return _check(status_of(stream))
    with torch.cuda.device(dev):
        _check(status_of(stream))


def _rows(t, name):
    """(rows, cols, leading dimension) of a tensor read as rows of its last
    dimension, without a copy."""
    if t.dim() == 0:
        raise TrtError(ERR_ARG, f"{name} must have at least one dimension")
    if t.dim() != 2:
        try:
            t = t.view(-1, t.size(-1))
        except RuntimeError:
            raise TrtError(ERR_STRIDE, f"{name} does not view as rows of its last dimension") from None
    (rows, cols), (ld, inner) = t.shape, t.stride()
    if cols > 1 and inner != 1:
        raise TrtError(ERR_STRIDE, f"{name} must have unit inner stride")
    if rows > 1 and ld < 1:
        raise TrtError(ERR_STRIDE, f"{name}: rows must have a positive stride")
    return rows, cols, ld if rows > 1 else max(cols, 1)


def _ld_as(t, name, like, ld):
    """The leading dimension of t, of `like`'s shape, whose own is ld."""
    return ld if t.stride() == like.stride() else _rows(t, name)[2]


def _vector(t, name, n, dtype):
    """Address of a contiguous vector of n elements of dtype, or None."""
    if t is None:
        return None
    if t.dim() != 1 or t.size(0) != n or not t.is_contiguous():
        raise TrtError(ERR_SIZE, f"{name} must be contiguous with {n} elements")
    if t.dtype != dtype:
        raise TrtError(ERR_DTYPE, f"{name} must be {dtype}")
    return t.data_ptr()


def _like(out, t, name):
    """out, or a new contiguous tensor of t's shape and dtype."""
    torch = _torch()
    if out is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    if out.shape != t.shape or out.dtype != t.dtype:
        raise TrtError(ERR_SIZE, f"{name} must be {list(t.shape)} of {t.dtype}")
    return out


def _new(t, dtype=None):
    """A new contiguous tensor of t's shape, of dtype or t's."""
    empty_like = _torch().empty_like
    if t.is_contiguous():
        return empty_like(t, dtype=dtype) if dtype else empty_like(t)
    return empty_like(t, dtype=dtype, memory_format=_torch().contiguous_format)


def _workspace(ws, need, like):
    """ws, or a new workspace of need bytes on like's device."""
    if ws is None:
        return like.new_empty(need, dtype=_torch().uint8)
    if not ws.is_contiguous():
        raise TrtError(ERR_STRIDE, "the workspace must be contiguous")
    return ws


def layernorm(x, gamma=None, beta=None, *, eps=1e-5, out=None):
    """The layer norm of every row of x (its last dimension), times gamma plus
    beta (ones and zeros where None): trt_layernorm.  x: float16, bfloat16 or
    float32, rows of unit inner stride; gamma and beta: one dtype, x's or
    float32.  out, if given, has x's shape and dtype and may not overlap the
    inputs; otherwise a new tensor is returned.  Runs on torch's current
    stream; no synchronisation, and nothing recorded for autograd: the result
    never requires a gradient.
    """
    rows, cols, ldx = _rows(x, "x")
    param = next((t.dtype for t in (gamma, beta) if t is not None), x.dtype)
    pdt = next((_dtype_code(t) for t in (gamma, beta) if t is not None), _dtype_code(x))
    g, b = _vector(gamma, "gamma", cols, param), _vector(beta, "beta", cols, param)
    ldy = max(cols, 1) if out is None else _rows(out, "out")[2]
    out = _like(out, x, "out")
    dev = _device(x, gamma=gamma, beta=beta, out=out)
    _on(dev, lambda s: lib().trt_layernorm(rows, cols, x.data_ptr(), ldx, g, b, eps,
                                           out.data_ptr(), ldy,
                                           _dtype_code(x), pdt, s))
    return out


def layernorm_bwd_workspace_size(rows, cols, dtype=F16) -> int:
    """trt_layernorm_bwd_workspace_size: bytes of workspace of the backward pass."""
    n = lib().trt_layernorm_bwd_workspace_size(rows, cols, dtype)
    if n < 0:
        raise TrtError(ERR_ARG, last_error())
    return n


def layernorm_bwd(dy, x, gamma=None, *, eps=1e-5, params=True, dx=None, dgamma=None, dbeta=None,
                  workspace=None):
    """The gradients of layernorm at x for dy: (dx, dgamma, dbeta), by
    trt_layernorm_bwd.  dy has x's shape and dtype; eps is the forward pass's.
    dgamma and dbeta have gamma's dtype (float32 without a gamma, unless the
    dgamma or dbeta given says otherwise); with params=False neither is
    computed and both are None.  dx, dgamma, dbeta and workspace (a uint8
    tensor of layernorm_bwd_workspace_size(...) bytes) are written if given,
    else allocated.  Runs on torch's current stream; no synchronisation.
    """
    torch = _torch()
    rows, cols, ldx = _rows(x, "x")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise TrtError(ERR_SIZE, f"dy must be {list(x.shape)} of {x.dtype}")
    param = next((t for t in (gamma, dgamma, dbeta) if t is not None), None)
    pdtype = torch.float32 if param is None else param.dtype
    pdt = F32 if param is None else _dtype_code(param)
    lddx = max(cols, 1) if dx is None else _rows(dx, "dx")[2]
    dx = _like(dx, x, "dx")
    if params:
        need = layernorm_bwd_workspace_size(rows, cols, _dtype_code(x))
        if dgamma is None:
            dgamma = x.new_empty(cols, dtype=pdtype)
        if dbeta is None:
            dbeta = torch.empty_like(dgamma)
        workspace = _workspace(workspace, need, x)
    else:
        dgamma = dbeta = workspace = None
    g, dg, db = (_vector(t, name, cols, pdtype) for t, name in
                 ((gamma, "gamma"), (dgamma, "dgamma"), (dbeta, "dbeta")))
    dev = _device(x, dy=dy, gamma=gamma, dx=dx, dgamma=dgamma, dbeta=dbeta, workspace=workspace)
    ws, wsb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    _on(dev, lambda s: lib().trt_layernorm_bwd(rows, cols, dy.data_ptr(), _rows(dy, "dy")[2],
                                               x.data_ptr(), ldx, g, eps, dx.data_ptr(),
                                               lddx, dg, db, _dtype_code(x), pdt,
                                               ws, wsb, s))
    return dx, dgamma, dbeta


# ---- the linear cross entropy and its gradients -------------------------------------

def _xent_inputs(x, w, target):
    """(tokens, vocab, width, ldx, ldw) of a head's input, weight and targets."""
    torch = _torch()
    tokens, width, ldx = _rows(x, "x")
    if w.dim() != 2 or w.size(1) != width:
        raise TrtError(ERR_SIZE, f"w must be [vocab, {width}]")
    vocab, _, ldw = _rows(w, "w")
    if w.dtype != x.dtype:
        raise TrtError(ERR_DTYPE, "x and w dtypes differ")
    if target.dtype != torch.int64:
        raise TrtError(ERR_DTYPE, "target must be int64")
    if target.shape != x.shape[:-1] or not target.is_contiguous():
        raise TrtError(ERR_SIZE, f"target must be contiguous of shape {list(x.shape[:-1])}")
    return tokens, vocab, width, ldx, ldw


def _per_token(t, name, shape):
    """(address, increment) of a float32 value for each token; a tensor of one
    element, or one expanded from it, stands for all tokens."""
    torch = _torch()
    if t is None:
        return None, 0
    if t.dtype != torch.float32:
        raise TrtError(ERR_DTYPE, f"{name} must be float32")
    if t.numel() == 1:
        return t.data_ptr(), 0
    if t.shape != shape:
        raise TrtError(ERR_SIZE, f"{name} must have shape {list(shape)} or one element")
    if all(st == 0 for st, n in zip(t.stride(), t.shape) if n > 1):
        return t.data_ptr(), 0
    if t.dim() == 1:
        return t.data_ptr(), t.stride(0)
    if not t.is_contiguous():
        raise TrtError(ERR_STRIDE, f"{name} must be contiguous or one-dimensional")
    return t.data_ptr(), 1


def _tokens_out(t, name, like):
    """t, or a new float32 tensor of like's shape."""
    torch = _torch()
    if t is None:
        return torch.empty_like(like, dtype=torch.float32)
    if t.shape != like.shape or t.dtype != torch.float32 or not t.is_contiguous():
        raise TrtError(ERR_SIZE, f"{name} must be contiguous float32 of shape {list(like.shape)}")
    return t




def linear_xent_workspace_size(tokens, vocab, width) -> int:
    """trt_linear_xent_workspace_size: bytes of workspace of the forward pass."""
    n = lib().trt_linear_xent_workspace_size(tokens, vocab, width)
    if n < 0:
        raise TrtError(ERR_ARG, last_error())
    return n


def linear_xent(x, w, target, *, ignore_index=-100, loss=None, lse=None, workspace=None):
    """The softmax cross entropy of the logits x @ w.T, which are not stored:
    (loss, lse) per token, float32, by trt_linear_xent.  x: [..., width] and w:
    [vocab, width], float16 or bfloat16; target: int64 of x's leading shape.
    Tokens whose target is ignore_index have loss and lse 0.  loss, lse and
    workspace (a uint8 tensor of linear_xent_workspace_size(...) bytes) are
    written if given, else allocated.  Runs on torch's current stream; no
    synchronisation, and nothing recorded for autograd: the results never
    require a gradient (linear_xent_bwd gives them).
    """
    tokens, vocab, width, ldx, ldw = _xent_inputs(x, w, target)
    workspace = _workspace(workspace, linear_xent_workspace_size(tokens, vocab, width), x)
    loss, lse = _tokens_out(loss, "loss", target), _tokens_out(lse, "lse", target)
    dev = _device(x, w=w, target=target, loss=loss, lse=lse, workspace=workspace)
    _on(dev, lambda s: lib().trt_linear_xent(tokens, vocab, width, x.data_ptr(), ldx, w.data_ptr(), ldw,
                                             target.data_ptr(), ignore_index, loss.data_ptr(),
                                             lse.data_ptr(), _dtype_code(x), workspace.data_ptr(),
                                             workspace.nbytes, s))
    return loss, lse


def linear_xent_bwd_workspace_size(tokens, vocab, width, piece=0) -> int:
    """trt_linear_xent_bwd_workspace_size: bytes of workspace of the backward pass."""
    n = lib().trt_linear_xent_bwd_workspace_size(tokens, vocab, width, piece)
    if n < 0:
        raise TrtError(ERR_ARG, last_error())
    return n


def linear_xent_bwd(x, w, target, lse, dloss, dlse=None, *, ignore_index=-100, need_dx=True,
                    need_dw=True, out_dtype=None, piece=0, dx=None, dw=None, workspace=None):
    """The gradients (dx, dw) of linear_xent for the upstream gradients dloss
    and dlse (None: zero), by trt_linear_xent_bwd.  x, w, target and lse are the
    forward pass's; dloss and dlse: float32 per token, or one element for all.
    dx and dw have out_dtype (default: x's dtype, or the dtype of the one
    given); the one not needed is None.  piece: vocabulary entries at a time
    (0: the library's choice).  dx, dw and workspace (a uint8 tensor of
    linear_xent_bwd_workspace_size(...) bytes) are written if given, else
    allocated.  Runs on torch's current stream; no synchronisation.
    """
    torch = _torch()
    tokens, vocab, width, ldx, ldw = _xent_inputs(x, w, target)
    if lse.shape != target.shape or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise TrtError(ERR_SIZE, f"lse must be contiguous float32 of shape {list(target.shape)}")
    (dl, dl_inc), (de, de_inc) = _per_token(dloss, "dloss", target.shape), _per_token(dlse, "dlse", target.shape)
    if dl is None:
        raise TrtError(ERR_NULL, "dloss must be given")
    given = next((t.dtype for t in (dx, dw) if t is not None), x.dtype)
    odt = out_dtype or given

    def output(t, like, need, name):
        if not need:
            return None, 0
        if t is None:
            t = torch.empty_like(like, dtype=odt, memory_format=torch.contiguous_format)
        elif t.shape != like.shape or t.dtype != odt:
            raise TrtError(ERR_SIZE, f"{name} must be {list(like.shape)} of {odt}")
        return t, _rows(t, name)[2]

    (dx, lddx), (dw, lddw) = output(dx, x, need_dx, "dx"), output(dw, w, need_dw, "dw")
    out = next((t for t in (dx, dw) if t is not None), x)
    workspace = _workspace(workspace, linear_xent_bwd_workspace_size(tokens, vocab, width, piece), x)
    dev = _device(x, w=w, target=target, lse=lse, dloss=dloss, dlse=dlse, dx=dx, dw=dw, workspace=workspace)
    _on(dev, lambda s: lib().trt_linear_xent_bwd(
        tokens, vocab, width, x.data_ptr(), ldx, w.data_ptr(), ldw, target.data_ptr(), ignore_index,
        lse.data_ptr(), dl, dl_inc, de, de_inc, None if dx is None else dx.data_ptr(), lddx,
        None if dw is None else dw.data_ptr(), lddw, _dtype_code(x), _dtype_code(out), piece,
        workspace.data_ptr(), workspace.nbytes, s))
    return dx, dw


# ---- activations saved in 8 bits, and a weight gradient from them --------------------

ACT8_BLOCK = 32     # columns to a scale


def _act8(q, scale, name=""):
    """(rows, cols, ldq, lds) of 8-bit rows and their scales."""
    torch = _torch()
    if q.dtype != torch.int8 or scale.dtype != torch.uint8:
        raise TrtError(ERR_DTYPE, f"{name}q must be int8 and {name}scale uint8")
    rows, cols, ldq = _rows(q, f"{name}q")
    want = (*q.shape[:-1], -(-cols // ACT8_BLOCK))
    if scale.shape != want:
        raise TrtError(ERR_SIZE, f"{name}scale must be {list(want)}")
    return rows, cols, ldq, _rows(scale, f"{name}scale")[2]


def act8_pack(x, *, q=None, scale=None):
    """x's rows (its last dimension) in 8 bits: (q, scale), by trt_act8_pack.
    x: float16, bfloat16 or float32, rows of unit inner stride; q: int8 of x's
    shape; scale: uint8 of x's leading shape, one for every ACT8_BLOCK columns.
    An element stands for q * 2^(scale - 133); a block that holds an infinity
    or a NaN is NaN throughout.  q and scale are written if given, else
    allocated.  Runs on torch's current stream; no synchronisation.
    """
    torch = _torch()
    rows, cols, ldx = _rows(x, "x")
    ldq, lds = max(cols, 1), max(-(-cols // ACT8_BLOCK), 1)
    given = q is not None or scale is not None
    if q is None:
        q = _new(x, torch.int8)
    elif q.shape != x.shape:
        raise TrtError(ERR_SIZE, f"q must be {list(x.shape)}")
    if scale is None:
        scale = x.new_empty((*x.shape[:-1], -(-cols // ACT8_BLOCK)), dtype=torch.uint8)
    if given:
        _, _, ldq, lds = _act8(q, scale)
    dev = _place(x, q, scale)
    _on(dev, lambda s: lib().trt_act8_pack(rows, cols, x.data_ptr(), ldx, q.data_ptr(), ldq, scale.data_ptr(), lds,
                                           _dtype_code(x), s))
    return q, scale


def act8_unpack(q, scale, dtype, *, out=None):
    """What act8_pack's rows stand for, rounded to dtype (exact in bfloat16 and
    float32, and in float16 for rows that were float16): trt_act8_unpack.  out,
    if given, has q's shape and dtype; otherwise a new tensor is returned.  Runs
    on torch's current stream; no synchronisation.
    """
    rows, cols, ldq, lds = _act8(q, scale)
    if out is None:
        out, ldx = _new(q, dtype), max(cols, 1)
    elif out.shape != q.shape or out.dtype != dtype:
        raise TrtError(ERR_SIZE, f"out must be {list(q.shape)} of {dtype}")
    else:
        ldx = _rows(out, "out")[2]
    dev = _place(q, scale, out)
    _on(dev, lambda s: lib().trt_act8_unpack(rows, cols, q.data_ptr(), ldq, scale.data_ptr(), lds, out.data_ptr(),
                                             ldx, _code_of(dtype), s))
    return out


def act8_weight_grad_workspace_size(tokens, outputs, inputs, dy_ptr=0, lddy=None) -> int:
    """trt_act8_weight_grad_workspace_size: bytes of workspace for a dy at
    address dy_ptr with rows lddy elements apart (contiguous where None)."""
    n = lib().trt_act8_weight_grad_workspace_size(tokens, outputs, inputs, dy_ptr or None,
                                                  outputs if lddy is None else lddy)
    if n < 0:
        raise TrtError(ERR_ARG, last_error())
    return n


def act8_weight_grad(dy, q, scale, *, out_dtype=None, dw=None, workspace=None):
    """The weight gradient dy.T @ x of a linear layer whose input x [..., inputs]
    was saved by act8_pack: trt_act8_weight_grad.  dy: [..., outputs], float16 or
    bfloat16, q's leading shape; dw: [outputs, inputs] of out_dtype (default:
    dy's, or that of the dw given).  dw and workspace (a uint8 tensor of
    act8_weight_grad_workspace_size(...) bytes) are written if given, else
    allocated.  Runs on torch's current stream; no synchronisation.
    """
    tokens, inputs, ldq, lds = _act8(q, scale)
    _, outputs, lddy = _rows(dy, "dy")
    if dy.shape[:-1] != q.shape[:-1]:
        raise TrtError(ERR_SIZE, f"dy must have q's leading shape {list(q.shape[:-1])}")
    if dw is None:
        dw, lddw = dy.new_empty((outputs, inputs), dtype=out_dtype or dy.dtype), max(inputs, 1)
    elif dw.dim() != 2 or dw.shape != (outputs, inputs) or dw.dtype != (out_dtype or dw.dtype):
        raise TrtError(ERR_SIZE, f"dw must be [{outputs}, {inputs}] of {out_dtype or dw.dtype}")
    else:
        lddw = _rows(dw, "dw")[2]
    at = dy.data_ptr()
    workspace = _workspace(workspace, act8_weight_grad_workspace_size(tokens, outputs, inputs, at, lddy), dy)
    dev = _place(dy, q, scale, dw, workspace)
    _on(dev, lambda s: lib().trt_act8_weight_grad(tokens, outputs, inputs, at, lddy, q.data_ptr(), ldq,
                                                  scale.data_ptr(), lds, dw.data_ptr(), lddw, _dtype_code(dy),
                                                  _dtype_code(dw), workspace.data_ptr(), workspace.nbytes, s))
    return dw


# ---- the norms around a block with its gate and residual, and their gradients ---------

def _gate_span(gate, shape, rows, cols, rows_per_gate):
    """The rows that each row of a gate covers: the gate [cols] is for all rows;
    one of x's leading sizes, from some point on 1 (and x's last), broadcasts
    over what follows; with rows_per_gate it is [ceil(rows / that), cols]."""
    if rows_per_gate is not None:
        if rows_per_gate < 1 or gate.dim() != 2 or gate.shape != (-(-rows // rows_per_gate), cols):
            raise TrtError(ERR_SIZE, f"gate must be [{-(-rows // max(rows_per_gate, 1))}, {cols}] for rows_per_gate {rows_per_gate}")
        return rows_per_gate
    if gate.dim() == 1 and gate.size(0) == cols:
        return rows
    span, at = 1, gate.dim() - 2
    while at >= 0 and gate.size(at) == 1:
        span *= shape[at] if gate.dim() == len(shape) else 1
        at -= 1
    if gate.dim() != len(shape) or gate.size(-1) != cols or gate.shape[:at + 1] != shape[:at + 1]:
        raise TrtError(ERR_SIZE, f"gate {list(gate.shape)} does not cover rows of {list(shape)}: [{cols}], or leading "
                                 "sizes followed by ones, or rows_per_gate given")
    return span


def _block(x, rows, cols, gate, post, post_gamma, post_beta, gamma, beta, alpha, rms, eps, rows_per_gate, none):
    """(Block, gate's span or 0, parameters' dtype) for rows of x; none: the
    parameters' dtype where none is given."""
    param = none
    for t in (post_gamma, post_beta, gamma, beta):
        if t is not None:
            param = t.dtype
            break
    span = at = ldg = 0
    gate_code = F32
    if gate is not None:
        span = _gate_span(gate, x.shape, rows, cols, rows_per_gate)
        at, ldg, gate_code = gate.data_ptr(), cols if gate.is_contiguous() else _rows(gate, "gate")[2], _code_of(gate.dtype)
    elif rows_per_gate is not None:
        raise TrtError(ERR_ARG, "rows_per_gate without a gate")
    return Block(at or None, ldg, span, _vector(post_gamma, "post_gamma", cols, param),
                 _vector(post_beta, "post_beta", cols, param), _vector(gamma, "gamma", cols, param),
                 _vector(beta, "beta", cols, param), alpha, eps, bool(post), bool(rms), gate_code,
                 _code_of(param)), span, param


def block_norm(r, y, gate=None, *, post=True, post_gamma=None, post_beta=None, gamma=None, beta=None,
               alpha=1.0, rms=False, eps=1e-5, rows_per_gate=None, need_h=True, r_out=None, h=None):
    """The end of a block and the start of the next: (r_out, h) of
        u = norm(y) * post_gamma + post_beta   (u = y without post)
        r_out = alpha * r + gate * u
        h = norm(r_out) * gamma + beta
    by trt_block_norm.  r, the residual stream, and y, the block's output, have
    one shape and dtype; the norms are layer norms, or root mean square norms
    with rms.  gate (ones where None): [cols] for every row, y's shape, y's
    leading sizes followed by ones ([batch, 1, cols] for [batch, tokens, cols]),
    or [ceil(rows / rows_per_gate), cols] with rows_per_gate; y's dtype or
    float32.  post_gamma, post_beta, gamma, beta: [cols] of one dtype, y's or
    float32; ones and zeros where None.  Without need_h no norm follows and h is
    None.  r_out and h are written if given, else allocated.  Runs on torch's
    current stream; no synchronisation, and nothing recorded for autograd
    (block_norm_bwd gives the gradients).
    """
    if y.shape != r.shape or y.dtype != r.dtype:
        raise TrtError(ERR_SIZE, f"y must be {list(r.shape)} of {r.dtype}")
    if h is not None and not need_h:
        raise TrtError(ERR_ARG, "h given without need_h")
    rows, cols, ldr = _rows(r, "r")
    ldy, ldro = _ld_as(y, "y", r, ldr), max(cols, 1)
    ldh = ldro
    block, _, _ = _block(r, rows, cols, gate, post, post_gamma, post_beta, gamma, beta, alpha, rms, eps, rows_per_gate, r.dtype)
    if r_out is None:
        r_out = _new(r)
    else:
        ldro = _rows(_like(r_out, r, "r_out"), "r_out")[2]
    if not need_h:
        h_at = None
    elif h is None:
        h = _new(r)
        h_at = h.data_ptr()
    else:
        ldh, h_at = _rows(_like(h, r, "h"), "h")[2], h.data_ptr()
    dev = _place(r, y, gate, post_gamma, post_beta, gamma, beta, r_out, h)
    _on(dev, lambda s: lib().trt_block_norm(rows, cols, r.data_ptr(), ldr, y.data_ptr(), ldy, block, r_out.data_ptr(),
                                            ldro, h_at, ldh, _dtype_code(r), s))
    return r_out, h


def block_norm_bwd_workspace_size(rows, cols, rows_per_gate=0, dtype=F16) -> int:
    """trt_block_norm_bwd_workspace_size: bytes of workspace of the backward
    pass (rows_per_gate 0: no gate)."""
    n = lib().trt_block_norm_bwd_workspace_size(rows, cols, rows_per_gate, dtype)
    if n < 0:
        raise TrtError(ERR_ARG, last_error())
    return n


def _saved(t, name, up, ld):
    """(Saved, its two tensors) of rows like up's, or of 8-bit ones as (q, scale)."""
    if isinstance(t, (tuple, list)):
        q, scale = t
        _, _, ldq, lds = _act8(q, scale, f"{name}'s ")
        if q.shape != up.shape:
            raise TrtError(ERR_SIZE, f"{name}'s q must be {list(up.shape)}")
        return Saved(q.data_ptr(), ldq, scale.data_ptr(), lds), q, scale
    if t.shape != up.shape or t.dtype != up.dtype:
        raise TrtError(ERR_SIZE, f"{name} must be {list(up.shape)} of {up.dtype}, or act8_pack's (q, scale) of that shape")
    return Saved(t.data_ptr(), _ld_as(t, name, up, ld), None, 0), t, None


def block_norm_bwd(dh, dr_out, r_out, y, gate=None, *, post=True, post_gamma=None, post_beta=None, gamma=None,
                   alpha=1.0, rms=False, eps=1e-5, rows_per_gate=None, params=True, dr=None, dy=None, workspace=None):
    """The gradients of block_norm for dh and dr_out, those of its results:
    (dr, dy, dgate, dpost_gamma, dpost_beta, dgamma, dbeta), by
    trt_block_norm_bwd.  Either of dh and dr_out may be None (zero); r_out is
    the forward pass's result, y its input, both tensors or both the (q, scale) of
    act8_pack, taken as the values that they stand for; r_out may be None without
    dh.  The other arguments are the forward pass's (the gradients do not
    depend on beta).  dgate is None without a gate, dpost_gamma and dpost_beta
    without post, dgamma and dbeta without dh, all five with params=False; they
    have their operand's shape and dtype (the parameters' one dtype, float32
    where none is given).  dr, dy and workspace (a uint8 tensor of
    block_norm_bwd_workspace_size(...) bytes) are written if given, else
    allocated.  Runs on torch's current stream; no synchronisation.
    """
    torch = _torch()
    up = dr_out if dh is None else dh
    if up is None:
        raise TrtError(ERR_NULL, "dh or dr_out must be given")
    rows, cols, ld = _rows(up, "dr_out" if dh is None else "dh")
    if dr_out is not None and (dr_out.shape != up.shape or dr_out.dtype != up.dtype):
        raise TrtError(ERR_SIZE, f"dr_out must be {list(up.shape)} of {up.dtype}")
    if dh is not None and r_out is None:
        raise TrtError(ERR_NULL, "dh needs r_out")
    block, span, param = _block(up, rows, cols, gate, post, post_gamma, post_beta, gamma, None, alpha, rms, eps, rows_per_gate,
                                torch.float32)
    code = _dtype_code(up)
    sy, y0, y1 = _saved(y, "y", up, ld)
    sr = r0 = r1 = None
    if dh is not None:
        sr, r0, r1 = _saved(r_out, "r_out", up, ld)
    lddr = lddy = max(cols, 1)
    if dr is None:
        dr = _new(up)
    else:
        lddr = _rows(_like(dr, up, "dr"), "dr")[2]
    if dy is None:
        dy = _new(up)
    else:
        lddy = _rows(_like(dy, up, "dy"), "dy")[2]
    dgate = dpg = dpb = dg = db = None
    if params:
        if gate is not None:
            dgate = _new(gate)
        made = 2 * bool(post) + 2 * (dh is not None)
        if made:
            made = up.new_empty((made, cols), dtype=param).unbind()
            if post:
                dpg, dpb = made[:2]
            if dh is not None:
                dg, db = made[-2:]
        need = lib().trt_block_norm_bwd_workspace_size(rows, cols, span, code)
        if need < 0:
            raise TrtError(ERR_ARG, last_error())
        workspace = _workspace(workspace, need, up)
        ws, wsb = workspace.data_ptr(), workspace.nbytes
    else:
        workspace, ws, wsb = None, None, 0
    grads = BlockGrads(*((None, 0) if dgate is None else (dgate.data_ptr(), cols)),
                       *(None if t is None else t.data_ptr() for t in (dpg, dpb, dg, db)))
    dev = _place(up, dr_out, gate, post_gamma, post_beta, gamma, dr, dy, workspace, y0, y1, r0, r1)
    dh_at, lddh = (None, 0) if dh is None else (dh.data_ptr(), ld)
    dr_at, lddro = (None, 0) if dr_out is None else (dr_out.data_ptr(), _ld_as(dr_out, "dr_out", up, ld))
    _on(dev, lambda s: lib().trt_block_norm_bwd(rows, cols, dh_at, lddh, dr_at, lddro, sr, sy, block, dr.data_ptr(), lddr,
                                                dy.data_ptr(), lddy, grads, code, ws, wsb, s))
    return dr, dy, dgate, dpg, dpb, dg, db
