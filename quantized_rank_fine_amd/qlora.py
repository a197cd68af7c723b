"""Thin Python binding of libqlora (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: it turns torch tensors into device pointers, takes the
current HIP stream, calls the library and raises on a non-OK status.  Every
step of the hot path runs in the HIP kernels of ``libqlora.so``; if the
library is missing the import fails loudly.
"""

import ctypes
import os
import re

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqlora.so")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "qlora.h")

F32, BF16 = 0, 1
LAB_GROUP = 16                        # QLORA_LAB_GROUP: 16-entry scale groups
MAX_TOP = 64                          # QLORA_MAX_TOP
NOALLOC_SCRATCH_BYTES = 32 << 20      # QLORA_NOALLOC_SCRATCH_BYTES
CB_NF4, CB_UNIFORM4, CB_INT4, CB_INT3, CB_TERNARY = 0, 1, 2, 3, 4   # qlora_codebook
STATUS = {0: "ok", 1: "null pointer", 2: "invalid shape", 3: "pointer not 16-byte aligned",
          4: "invalid dtype", 5: "workspace too small", 6: "HIP runtime error",
          7: "invalid value"}
KERNELS = ("quantize", "xa_rowdot", "fwd_gemm", "dy_pass", "dx_gemm", "da_pass", "reduce",
           "fwd_smallm", "token_logp", "pref_loss", "policy_loss", "dropout", "muon",
           "ep_bwd", "token_top", "distill")
PREF_SIGMOID, PREF_SQUARED, PREF_HINGE = 0, 1, 2                     # qlora_pref_kind
EP_NONE, EP_RELU, EP_GELU, EP_GELU_TANH, EP_SILU = 0, 1, 2, 3, 4      # qlora_ep_act
OBJ_NLL, OBJ_CLIP = 0, 1                                             # qlora_objective


class QloraError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} (status {status})")


class qlora_nf4(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_int64), ("out", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("qscale", ctypes.c_void_p),
                ("gscale", ctypes.c_void_p), ("codebook", ctypes.c_int32),
                ("block", ctypes.c_int32)]


class qlora_lora(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("dropout_p", ctypes.c_float),
                ("keep", ctypes.c_void_p)]


class qlora_epilogue(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("bias", ctypes.c_void_p), ("mul", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("Z", ctypes.c_void_p)]


class qlora_adam_state(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("theta_bf16", ctypes.c_void_p)]


class qlora_adam_hparams(ctypes.Structure):
    _fields_ = [("step", ctypes.c_int64), ("lr", ctypes.c_float), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
                ("weight_decay", ctypes.c_float)]


class qlora_pref(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("beta", ctypes.c_float), ("margin", ctypes.c_float),
                ("smoothing", ctypes.c_float), ("average", ctypes.c_int32)]


class qlora_policy(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("clip_lo", ctypes.c_float),
                ("clip_hi", ctypes.c_float), ("clip_dual", ctypes.c_float),
                ("kl_coef", ctypes.c_float), ("ent_coef", ctypes.c_float)]


class qlora_muon_mat(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("theta", ctypes.c_void_p),
                ("theta_bf16", ctypes.c_void_p), ("update", ctypes.c_void_p),
                ("scale", ctypes.c_float)]


class qlora_muon_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("nesterov", ctypes.c_int32),
                ("steps", ctypes.c_int32), ("eps", ctypes.c_double),
                ("coef", ctypes.c_double * 3)]


_lib = None


def lib():
    """Load libqlora.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "(or python quantized_rank_fine_amd/build.py)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    pnf4 = ctypes.POINTER(qlora_nf4)
    L.qlora_quantize.argtypes = [vp, pnf4, vp]
    L.qlora_linear_fwd.argtypes = [pnf4, vp, i64, ctypes.c_int, vp, vp, i32, ctypes.c_int, vp, vp,
                                   vp, sz, vp]
    L.qlora_linear_fwd_noalloc.argtypes = [pnf4, vp, i64, ctypes.c_int, vp, vp, i32,
                                           ctypes.c_int, vp, vp, vp]
    L.qlora_linear_fwd_noalloc.restype = ctypes.c_int
    L.qlora_linear_bwd.argtypes = [pnf4, vp, vp, i64, ctypes.c_int, vp, vp, i32, ctypes.c_int, vp,
                                   vp, vp, vp, vp, sz, vp]
    plora = ctypes.POINTER(qlora_lora)
    L.qlora_linear_fwd_lora.argtypes = [pnf4, vp, i64, ctypes.c_int, vp, vp, i32, ctypes.c_int,
                                        plora, vp, vp, vp, sz, vp]
    L.qlora_linear_bwd_lora.argtypes = [pnf4, vp, vp, i64, ctypes.c_int, vp, vp, i32,
                                        ctypes.c_int, plora, vp, vp, vp, vp, vp, sz, vp]
    L.qlora_linear_fwd_ep.argtypes = [pnf4, vp, i64, ctypes.c_int, vp, vp, i32, ctypes.c_int,
                                      plora, ctypes.POINTER(qlora_epilogue), vp, vp, vp, sz, vp]
    L.qlora_ep_bwd.argtypes = [vp, vp, vp, i64, i64, ctypes.c_int, i32, vp, vp, vp, vp, sz, vp]
    L.qlora_ep_bwd_workspace_bytes.argtypes = [i64, i64, ctypes.c_int]
    L.qlora_ep_bwd_workspace_bytes.restype = sz
    pst, php = ctypes.POINTER(qlora_adam_state), ctypes.POINTER(qlora_adam_hparams)
    L.qlora_linear_bwd_adam.argtypes = [pnf4, vp, vp, i64, ctypes.c_int, vp, vp, i32,
                                        ctypes.c_int, plora, vp, vp, pst, pst, php, vp, vp, vp,
                                        sz, vp]
    L.qlora_linear_fwd_group.argtypes = [i32, ctypes.POINTER(pnf4), ctypes.POINTER(vp), i64,
                                         ctypes.c_int, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                         i32, ctypes.c_int, ctypes.POINTER(vp),
                                         ctypes.POINTER(vp), vp, sz, vp]
    L.qlora_linear_fwd_group.restype = ctypes.c_int
    L.qlora_fwd_group_workspace_bytes.argtypes = [i32, i64, ctypes.POINTER(i64),
                                                  ctypes.POINTER(i64), i32, ctypes.c_int]
    L.qlora_fwd_group_workspace_bytes.restype = sz
    L.qlora_merge.argtypes = [pnf4, vp, vp, i32, ctypes.c_int, vp, ctypes.c_int, vp]
    f32 = ctypes.c_float
    L.qlora_adam_step.argtypes = [vp, vp, vp, vp, i64, i64, f32, f32, f32, f32, f32, vp, vp]
    L.qlora_loftq_init.argtypes = [vp, pnf4, vp, i32, i32, i32, vp, vp, ctypes.c_int, vp, sz, vp]
    L.qlora_loftq_workspace_bytes.argtypes = [i64, i64, i32]
    L.qlora_loftq_workspace_bytes.restype = sz
    ci, u64 = ctypes.c_int, ctypes.c_uint64
    L.qlora_token_logp_fwd.argtypes = [vp, i64, i64, i64, ci, vp, f32, vp, vp, vp, vp, sz, vp]
    L.qlora_token_logp_bwd.argtypes = [vp, i64, i64, i64, ci, vp, f32, vp, vp, vp, vp, vp, i64,
                                       vp]
    L.qlora_pref_loss.argtypes = [vp, vp, vp, vp, i64, i64, ctypes.POINTER(qlora_pref), vp, vp,
                                  vp, vp, sz, vp]
    ppol = ctypes.POINTER(qlora_policy)
    L.qlora_policy_loss.argtypes = [vp, vp, i64, vp, vp, vp, vp, ppol, vp, vp, vp, vp, sz, vp]
    L.qlora_policy_logits.argtypes = [vp, i64, i64, i64, ci, vp, f32, vp, vp, vp, vp, ppol, vp,
                                      vp, vp, i64, vp, sz, vp]
    L.qlora_dropout.argtypes = [vp, i64, vp, i64, i64, i64, ci, f32, u64, u64, vp, i64, vp]
    pmat = ctypes.POINTER(qlora_muon_mat)
    L.qlora_muon_step.argtypes = [i32, pmat, ctypes.POINTER(qlora_muon_hparams), vp, sz, vp]
    L.qlora_muon_workspace_bytes.argtypes = [i32, pmat]
    L.qlora_muon_workspace_bytes.restype = sz
    L.qlora_token_top.argtypes = [vp, i64, i64, i64, ci, vp, f32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.qlora_distill_logits.argtypes = [vp, i64, i64, i64, ci, f32, vp, i32, vp, vp, i32, vp, vp,
                                       vp, i64, vp, sz, vp]
    for f in (L.qlora_token_top_workspace_bytes, L.qlora_distill_workspace_bytes):
        f.argtypes = [i64, i64, ci, i32]
        f.restype = sz
    for f in (L.qlora_token_logp_fwd, L.qlora_token_logp_bwd, L.qlora_pref_loss,
              L.qlora_policy_loss, L.qlora_policy_logits, L.qlora_dropout, L.qlora_muon_step,
              L.qlora_linear_fwd_ep, L.qlora_ep_bwd, L.qlora_token_top, L.qlora_distill_logits):
        f.restype = ctypes.c_int
    L.qlora_token_logp_workspace_bytes.argtypes = [i64, i64, ci]
    L.qlora_policy_logits_workspace_bytes.argtypes = [i64, i64, ci]
    L.qlora_pref_workspace_bytes.argtypes = [i64, i64]
    L.qlora_policy_workspace_bytes.argtypes = [i64]
    for f in (L.qlora_token_logp_workspace_bytes, L.qlora_policy_logits_workspace_bytes,
              L.qlora_pref_workspace_bytes, L.qlora_policy_workspace_bytes):
        f.restype = sz
    for f in (L.qlora_quantize, L.qlora_linear_fwd, L.qlora_linear_bwd, L.qlora_merge,
              L.qlora_adam_step, L.qlora_loftq_init, L.qlora_linear_fwd_lora,
              L.qlora_linear_bwd_lora, L.qlora_linear_bwd_adam):
        f.restype = ctypes.c_int
    for f in (L.qlora_fwd_workspace_bytes, L.qlora_bwd_workspace_bytes):
        f.argtypes = [i64, i64, i64, i32, ctypes.c_int]
        f.restype = sz
    L.qlora_status_string.argtypes = [ctypes.c_int]
    L.qlora_status_string.restype = ctypes.c_char_p
    L.qlora_levels.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.qlora_levels.restype = None
    L.qlora_thresholds.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.qlora_thresholds.restype = None
    for f in (L.qlora_codebook_levels, L.qlora_codebook_thresholds):
        f.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_float)]
        f.restype = ctypes.c_int
    L.qlora_timing_enable.argtypes = [ctypes.c_int]
    L.qlora_timing_enable.restype = ctypes.c_int
    L.qlora_timing_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                    ctypes.POINTER(ctypes.c_int64)]
    L.qlora_timing_read.restype = ctypes.c_int
    L.qlora_timing_reset.argtypes = []
    L.qlora_timing_reset.restype = None
    L.qlora_kernel_name.argtypes = [ctypes.c_int]
    L.qlora_kernel_name.restype = ctypes.c_char_p
    _lib = L
    return L


def header_functions():
    """Names of the functions include/qlora.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(qlora_[a-z0-9_]+)\s*\(",
                       text, flags=re.M)
    inline = set(re.findall(r"static\s+inline\s+\w+\s+(qlora_[a-z0-9_]+)\s*\(", text))
    return sorted(set(names) - inline)


# ------------------------------------------------------------------ helpers

def _ptr(t):
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


_current_raw = None      # (device index -> stream handle, current device), once initialised


def _stream_getters():
    import torch
    torch.cuda.current_stream()          # initialises the runtime, or says that there is none
    # torch.cuda.current_stream().cuda_stream without the Stream object (0.2 us, not 2.7),
    # where this torch has the two calls for it
    handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if handle is None or device is None:
        return lambda d: torch.cuda.current_stream(d).cuda_stream, torch.cuda.current_device
    return handle, device


def _stream(stream):
    global _current_raw
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _current_raw is None:
        _current_raw = _stream_getters()
    handle, device = _current_raw
    return handle(device())


def _check(status, where):
    if status != 0:
        raise QloraError(status, where)


def nf4_struct(n_in, n_out, codes, qscale, gscale, codebook=CB_NF4, block=0):
    """qlora_nf4 describing caller-owned buffers (tensors or raw pointers)."""
    return qlora_nf4(int(n_in), int(n_out), _ptr(codes), _ptr(qscale), _ptr(gscale),
                     int(codebook), int(block))


class NF4Weight:
    """Caller-owned device buffers of one quantized (in, out) weight, the
    codebook its codes index and its scale format: block 64 (int8 block
    scales, double-quantized) or LAB_GROUP (one fp32 scale per 16 entries)."""

    def __init__(self, n_in, n_out, device="cuda", codebook=CB_NF4, block=64):
        import torch
        n = n_in * n_out
        self.n_in, self.n_out = n_in, n_out
        self.codebook = codebook
        self.block = block
        self.codes = torch.empty(n // 2, dtype=torch.uint8, device=device)
        if block == LAB_GROUP:
            self.qscale = None
            self.gscale = torch.empty(n // LAB_GROUP, dtype=torch.float32, device=device)
        else:
            self.qscale = torch.empty(n // 64, dtype=torch.int8, device=device)
            self.gscale = torch.empty((n // 64 + 255) // 256, dtype=torch.float32, device=device)

    def struct(self):
        return nf4_struct(self.n_in, self.n_out, self.codes, self.qscale, self.gscale,
                          self.codebook, 0 if self.block == 64 else self.block)


# ------------------------------------------------------------- entry points

def qlora_quantize(W0, wq, stream=None):
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    _check(lib().qlora_quantize(_ptr(W0), ctypes.byref(s), _stream(stream)), "qlora_quantize")


def qlora_merge(wq, A, B, r, adt, W, wdt, stream=None):
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    _check(lib().qlora_merge(ctypes.byref(s), _ptr(A), _ptr(B), int(r), int(adt), _ptr(W),
                             int(wdt), _stream(stream)), "qlora_merge")


def qlora_adam_step(theta, grad, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8,
                    weight_decay=0.0, theta_bf16=None, n=None, stream=None):
    n = theta.numel() if n is None else int(n)
    _check(lib().qlora_adam_step(_ptr(theta), _ptr(grad), _ptr(m), _ptr(v), n, int(step),
                                 float(lr), float(beta1), float(beta2), float(eps),
                                 float(weight_decay), _ptr(theta_bf16), _stream(stream)),
           "qlora_adam_step")


MUON_MAX_MATS = 4096                  # QLORA_MUON_MAX_MATS
MUON_COEF = (3.4445, -4.7750, 2.0315)


def muon_mat(rows, cols, grad, m=None, theta=None, theta_bf16=None, update=None, scale=1.0):
    """qlora_muon_mat: one matrix of qlora_muon_step (tensors or raw pointers)."""
    return qlora_muon_mat(int(rows), int(cols), _ptr(grad), _ptr(m), _ptr(theta),
                          _ptr(theta_bf16), _ptr(update), float(scale))


def muon_mats(mats):
    """The host array of a call's matrices; may be kept as long as their buffers are."""
    mats = list(mats)
    return (qlora_muon_mat * len(mats))(*mats)


def qlora_muon_workspace_bytes(mats):
    return int(lib().qlora_muon_workspace_bytes(len(mats), mats))


def qlora_muon_step(mats, lr, ws, ws_bytes, momentum=0.95, nesterov=True, weight_decay=0.0,
                    eps=1e-7, steps=5, coef=MUON_COEF, stream=None):
    """One orthogonalised step of the matrices of `mats` (from muon_mats)."""
    hp = qlora_muon_hparams(float(lr), float(momentum), float(weight_decay), int(bool(nesterov)),
                            int(steps), float(eps), (ctypes.c_double * 3)(*coef))
    _check(lib().qlora_muon_step(len(mats), mats, ctypes.byref(hp), _ptr(ws), int(ws_bytes),
                                 _stream(stream)), "qlora_muon_step")


def qlora_loftq_workspace_bytes(n_in, n_out, k):
    return int(lib().qlora_loftq_workspace_bytes(int(n_in), int(n_out), int(k)))


def qlora_loftq_init(W0, wq, omega, k, r, iters, A, B, adt, ws, ws_bytes, stream=None):
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    _check(lib().qlora_loftq_init(_ptr(W0), ctypes.byref(s), _ptr(omega), int(k), int(r),
                                  int(iters), _ptr(A), _ptr(B), int(adt), _ptr(ws),
                                  int(ws_bytes), _stream(stream)), "qlora_loftq_init")


def qlora_fwd_workspace_bytes(M, n_in, n_out, r, act=BF16):
    return int(lib().qlora_fwd_workspace_bytes(M, n_in, n_out, r, int(act)))


def qlora_bwd_workspace_bytes(M, n_in, n_out, r, act=BF16):
    return int(lib().qlora_bwd_workspace_bytes(M, n_in, n_out, r, int(act)))


def qlora_linear_fwd(wq, X, M, act, A, B, r, adt, Y, XA, ws, ws_bytes, stream=None):
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    _check(lib().qlora_linear_fwd(ctypes.byref(s), _ptr(X), int(M), int(act), _ptr(A), _ptr(B),
                                  int(r), int(adt), _ptr(Y), _ptr(XA), _ptr(ws), int(ws_bytes),
                                  _stream(stream)), "qlora_linear_fwd")


def qlora_linear_fwd_noalloc(wq, X, M, act, A, B, r, adt, Y, XA, stream=None):
    """qlora_linear_fwd with the library's device-resident scratch (no
    workspace argument; nothing is allocated)."""
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    _check(lib().qlora_linear_fwd_noalloc(ctypes.byref(s), _ptr(X), int(M), int(act), _ptr(A),
                                          _ptr(B), int(r), int(adt), _ptr(Y), _ptr(XA),
                                          _stream(stream)), "qlora_linear_fwd_noalloc")


def qlora_linear_bwd(wq, X, dY, M, act, A, B, r, adt, XA, dX, dA, dB, ws, ws_bytes,
                     stream=None):
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    _check(lib().qlora_linear_bwd(ctypes.byref(s), _ptr(X), _ptr(dY), int(M), int(act), _ptr(A),
                                  _ptr(B), int(r), int(adt), _ptr(XA), _ptr(dX), _ptr(dA),
                                  _ptr(dB), _ptr(ws), int(ws_bytes), _stream(stream)),
           "qlora_linear_bwd")


def _lora(scale, dropout_p, keep):
    return qlora_lora(float(scale), float(dropout_p), _ptr(keep))


def qlora_linear_fwd_lora(wq, X, M, act, A, B, r, adt, scale, dropout_p, keep, Y, XA, ws,
                          ws_bytes, stream=None):
    """qlora_linear_fwd with the alpha/r factor `scale` and dropout on X.A
    (`keep`: [M, r] uint8 device mask or None, `dropout_p` its probability)."""
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    o = _lora(scale, dropout_p, keep)
    _check(lib().qlora_linear_fwd_lora(ctypes.byref(s), _ptr(X), int(M), int(act), _ptr(A),
                                       _ptr(B), int(r), int(adt), ctypes.byref(o), _ptr(Y),
                                       _ptr(XA), _ptr(ws), int(ws_bytes), _stream(stream)),
           "qlora_linear_fwd_lora")


def qlora_linear_bwd_lora(wq, X, dY, M, act, A, B, r, adt, scale, dropout_p, keep, XA, dX, dA,
                          dB, ws, ws_bytes, stream=None):
    """qlora_linear_bwd with the same adapter options as the forward."""
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    o = _lora(scale, dropout_p, keep)
    _check(lib().qlora_linear_bwd_lora(ctypes.byref(s), _ptr(X), _ptr(dY), int(M), int(act),
                                       _ptr(A), _ptr(B), int(r), int(adt), ctypes.byref(o),
                                       _ptr(XA), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws),
                                       int(ws_bytes), _stream(stream)),
           "qlora_linear_bwd_lora")


def epilogue_struct(act=EP_NONE, bias=None, mul=None, residual=None, Z=None):
    """qlora_epilogue: the elementwise end of qlora_linear_fwd_ep (device tensors
    or None; Z receives the value before the activation)."""
    return qlora_epilogue(int(act), _ptr(bias), _ptr(mul), _ptr(residual), _ptr(Z))


def qlora_linear_fwd_ep(wq, X, M, act, A, B, r, adt, scale, dropout_p, keep, ep, Y, XA, ws,
                        ws_bytes, stream=None):
    """qlora_linear_fwd_lora with the elementwise end `ep` (from epilogue_struct):
    Y = residual + act(Z) mul, Z = the linear + bias."""
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    o = _lora(scale, dropout_p, keep)
    _check(lib().qlora_linear_fwd_ep(ctypes.byref(s), _ptr(X), int(M), int(act), _ptr(A),
                                     _ptr(B), int(r), int(adt), ctypes.byref(o),
                                     ctypes.byref(ep), _ptr(Y), _ptr(XA), _ptr(ws),
                                     int(ws_bytes), _stream(stream)), "qlora_linear_fwd_ep")


def qlora_ep_bwd_workspace_bytes(M, n_out, act=BF16):
    return int(lib().qlora_ep_bwd_workspace_bytes(int(M), int(n_out), int(act)))


def qlora_ep_bwd(Z, mul, dY, M, n_out, act, ep_act, dZ, dmul, dbias, ws, ws_bytes, stream=None):
    """The gradient of the elementwise end: dZ (qlora_linear_bwd's dY), dmul and
    dbias, each of which may be None."""
    _check(lib().qlora_ep_bwd(_ptr(Z), _ptr(mul), _ptr(dY), int(M), int(n_out), int(act),
                              int(ep_act), _ptr(dZ), _ptr(dmul), _ptr(dbias), _ptr(ws),
                              int(ws_bytes), _stream(stream)), "qlora_ep_bwd")


def qlora_linear_bwd_adam(wq, X, dY, M, act, A, B, r, adt, XA, dX, state_A, state_B, step, lr,
                          ws, ws_bytes, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
                          lora=None, dA=None, dB=None, stream=None):
    """The backward with one Adam step of A and B fused into its last launch.
    state_A / state_B: (theta, m, v, theta_bf16 or None) device tensors;
    lora: None or (scale, dropout_p, keep)."""
    s = wq.struct() if isinstance(wq, NF4Weight) else wq
    sa = qlora_adam_state(*[_ptr(t) for t in state_A])
    sb = qlora_adam_state(*[_ptr(t) for t in state_B])
    hp = qlora_adam_hparams(int(step), float(lr), float(beta1), float(beta2), float(eps),
                            float(weight_decay))
    o = _lora(*lora) if lora is not None else None
    _check(lib().qlora_linear_bwd_adam(ctypes.byref(s), _ptr(X), _ptr(dY), int(M), int(act),
                                       _ptr(A), _ptr(B), int(r), int(adt),
                                       ctypes.byref(o) if o is not None else None, _ptr(XA),
                                       _ptr(dX), ctypes.byref(sa), ctypes.byref(sb),
                                       ctypes.byref(hp), _ptr(dA), _ptr(dB), _ptr(ws),
                                       int(ws_bytes), _stream(stream)),
           "qlora_linear_bwd_adam")


def qlora_fwd_group_workspace_bytes(M, ins, outs, r, act=None):
    n = len(ins)
    act = BF16 if act is None else act
    return int(lib().qlora_fwd_group_workspace_bytes(n, int(M), (ctypes.c_int64 * n)(*ins),
                                                     (ctypes.c_int64 * n)(*outs), int(r),
                                                     int(act)))


def qlora_linear_fwd_group(wqs, Xs, M, act, As, Bs, r, adt, Ys, XAs, ws, ws_bytes, stream=None):
    """Forward of up to 4 independent few-token linears in one pair of
    launches (lists of the per-linear weights and tensors)."""
    n = len(wqs)
    structs = [w.struct() if isinstance(w, NF4Weight) else w for w in wqs]
    pw = (ctypes.POINTER(qlora_nf4) * n)(*[ctypes.pointer(st) for st in structs])
    arr = lambda ts: (ctypes.c_void_p * n)(*[_ptr(t) for t in ts])
    _check(lib().qlora_linear_fwd_group(n, pw, arr(Xs), int(M), int(act), arr(As), arr(Bs),
                                        int(r), int(adt), arr(Ys), arr(XAs), _ptr(ws),
                                        int(ws_bytes), _stream(stream)),
           "qlora_linear_fwd_group")


def pref_struct(kind, beta, margin=0.0, smoothing=0.0, average=False):
    """qlora_pref: the objective of qlora_pref_loss."""
    return qlora_pref(int(kind), float(beta), float(margin), float(smoothing), int(average))


def policy_struct(kind, clip_lo=0.2, clip_hi=0.2, clip_dual=0.0, kl_coef=0.0, ent_coef=0.0):
    """qlora_policy: the objective of qlora_policy_loss and qlora_policy_logits."""
    return qlora_policy(int(kind), float(clip_lo), float(clip_hi), float(clip_dual),
                        float(kl_coef), float(ent_coef))


def qlora_token_logp_workspace_bytes(T, V, dt):
    return int(lib().qlora_token_logp_workspace_bytes(int(T), int(V), int(dt)))


def qlora_token_logp_fwd(logits, ld, T, V, dt, labels, scale, logp, stats, entropy, ws, ws_bytes,
                         stream=None):
    """Log-probability of each row's label (int64), the row's (m, z) and, if
    `entropy` is not None, its entropy."""
    _check(lib().qlora_token_logp_fwd(_ptr(logits), int(ld), int(T), int(V), int(dt),
                                      _ptr(labels), float(scale), _ptr(logp), _ptr(stats),
                                      _ptr(entropy), _ptr(ws), int(ws_bytes), _stream(stream)),
           "qlora_token_logp_fwd")


def qlora_token_logp_bwd(logits, ld, T, V, dt, labels, scale, stats, entropy, g, g_entropy,
                         dlogits, ldd, stream=None):
    """The logits' gradient (dlogits may be logits) from that of the
    log-probabilities and, unless both are None, of the entropies."""
    _check(lib().qlora_token_logp_bwd(_ptr(logits), int(ld), int(T), int(V), int(dt),
                                      _ptr(labels), float(scale), _ptr(stats), _ptr(entropy),
                                      _ptr(g), _ptr(g_entropy), _ptr(dlogits), int(ldd),
                                      _stream(stream)), "qlora_token_logp_bwd")


def qlora_token_top_workspace_bytes(T, V, dt, k):
    return int(lib().qlora_token_top_workspace_bytes(int(T), int(V), int(dt), int(k)))


def qlora_token_top(logits, ld, T, V, dt, labels, scale, k, ids, top, logp, entropy, ws, ws_bytes,
                    stream=None):
    """The k most likely words of each row (ids int32, top their log p), the
    labels' log p and the entropy; labels, logp and entropy may be None."""
    _check(lib().qlora_token_top(_ptr(logits), int(ld), int(T), int(V), int(dt), _ptr(labels),
                                 float(scale), int(k), _ptr(ids), _ptr(top), _ptr(logp),
                                 _ptr(entropy), _ptr(ws), int(ws_bytes), _stream(stream)),
           "qlora_token_top")


def qlora_distill_workspace_bytes(T, V, dt, k):
    return int(lib().qlora_distill_workspace_bytes(int(T), int(V), int(dt), int(k)))


def qlora_distill_logits(logits, ld, T, V, dt, scale, weight, k, ids, teacher, normalize, loss, kl,
                         dlogits, ldd, ws, ws_bytes, stream=None):
    """Divergence from a teacher's k alternatives a row (ids int32, teacher their
    log p, as qlora_token_top gives them) and the logits' gradient (dlogits may
    be logits); weight may be None."""
    _check(lib().qlora_distill_logits(_ptr(logits), int(ld), int(T), int(V), int(dt),
                                      float(scale), _ptr(weight), int(k), _ptr(ids),
                                      _ptr(teacher), int(bool(normalize)), _ptr(loss), _ptr(kl),
                                      _ptr(dlogits), int(ldd), _ptr(ws), int(ws_bytes),
                                      _stream(stream)), "qlora_distill_logits")


def qlora_pref_workspace_bytes(P, T):
    return int(lib().qlora_pref_workspace_bytes(int(P), int(T)))


def qlora_pref_loss(logp, ref, mask, cu, P, T, pref, loss, rewards, dlogp, ws, ws_bytes,
                    stream=None):
    """Loss of P pairs of answers and its gradient by token; `pref` from
    pref_struct; ref and mask may be None."""
    _check(lib().qlora_pref_loss(_ptr(logp), _ptr(ref), _ptr(mask), _ptr(cu), int(P), int(T),
                                 ctypes.byref(pref), _ptr(loss), _ptr(rewards), _ptr(dlogp),
                                 _ptr(ws), int(ws_bytes), _stream(stream)), "qlora_pref_loss")


def qlora_policy_workspace_bytes(T):
    return int(lib().qlora_policy_workspace_bytes(int(T)))


def qlora_policy_loss(logp, entropy, T, weight, adv, old, ref, policy, out, dlogp, dentropy, ws,
                      ws_bytes, stream=None):
    """Policy objective over tokens: out[4], dlogp and, if wanted, dentropy;
    `policy` from policy_struct; entropy, weight, adv, old, ref may be None."""
    _check(lib().qlora_policy_loss(_ptr(logp), _ptr(entropy), int(T), _ptr(weight), _ptr(adv),
                                   _ptr(old), _ptr(ref), ctypes.byref(policy), _ptr(out),
                                   _ptr(dlogp), _ptr(dentropy), _ptr(ws), int(ws_bytes),
                                   _stream(stream)), "qlora_policy_loss")


def qlora_policy_logits_workspace_bytes(T, V, dt):
    return int(lib().qlora_policy_logits_workspace_bytes(int(T), int(V), int(dt)))


def qlora_policy_logits(logits, ld, T, V, dt, labels, scale, weight, adv, old, ref, policy, out,
                        logp, dlogits, ldd, ws, ws_bytes, stream=None):
    """The same objective from the logits to their gradient (dlogits may be
    logits); logp may be None."""
    _check(lib().qlora_policy_logits(_ptr(logits), int(ld), int(T), int(V), int(dt),
                                     _ptr(labels), float(scale), _ptr(weight), _ptr(adv),
                                     _ptr(old), _ptr(ref), ctypes.byref(policy), _ptr(out),
                                     _ptr(logp), _ptr(dlogits), int(ldd), _ptr(ws),
                                     int(ws_bytes), _stream(stream)), "qlora_policy_logits")


def qlora_dropout(x, ldx, residual, ldr, rows, cols, dt, p, seed, counter, y, ldy, stream=None):
    """y = residual + keep * x / (1 - p) with the mask of (seed, counter);
    residual may be None.  The backward is the same call on the gradient."""
    _check(lib().qlora_dropout(_ptr(x), int(ldx), _ptr(residual), int(ldr), int(rows), int(cols),
                               int(dt), float(p), int(seed), int(counter), _ptr(y), int(ldy),
                               _stream(stream)), "qlora_dropout")


def qlora_levels():
    buf = (ctypes.c_float * 16)()
    lib().qlora_levels(buf)
    return list(buf)


def qlora_thresholds():
    buf = (ctypes.c_float * 15)()
    lib().qlora_thresholds(buf)
    return list(buf)


def qlora_codebook_levels(codebook):
    buf = (ctypes.c_float * 16)()
    _check(0 if lib().qlora_codebook_levels(int(codebook), buf) == 0 else 4,
           "qlora_codebook_levels")
    return list(buf)


def qlora_codebook_thresholds(codebook):
    buf = (ctypes.c_float * 15)()
    _check(0 if lib().qlora_codebook_thresholds(int(codebook), buf) == 0 else 4,
           "qlora_codebook_thresholds")
    return list(buf)


def qlora_status_string(status):
    return lib().qlora_status_string(int(status)).decode()


def qlora_timing_enable(kinds=None):
    """Time the given kernel kinds (indices into KERNELS); None = all."""
    if kinds is None:
        mask = (1 << len(KERNELS)) - 1
    else:
        mask = 0
        for k in kinds:
            mask |= 1 << (KERNELS.index(k) if isinstance(k, str) else int(k))
    return lib().qlora_timing_enable(mask)


def qlora_timing_disable():
    return lib().qlora_timing_enable(0)


def qlora_timing_read(kind):
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    rc = lib().qlora_timing_read(int(kind), ctypes.byref(ms), ctypes.byref(n))
    if rc != 0:
        raise RuntimeError(f"qlora_timing_read failed ({rc})")
    return ms.value, n.value


def qlora_timing_reset():
    lib().qlora_timing_reset()


def qlora_kernel_name(kind):
    return lib().qlora_kernel_name(int(kind)).decode()
