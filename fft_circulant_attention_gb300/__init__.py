"""Python binding of libcat, the GB300 CAT library (include/cat.h): the
forward pass and its backward pass.

CAT (circular-convolutional attention), from the notes page "CAT:
Circular-Convolutional Attention for Sub-Quadratic Transformers", section
方法详解: per batch b and head h, z = X·W_A[:, h], z* = softmax over the N
tokens, and O_h = circ(z*)·V_h = IFFT(FFT(z*) ⊙ FFT(V_h)).

This module only marshals arguments (tensor -> device pointer, stream ->
handle, status -> exception; the operator plans' calls do it natively).  Every step of the computation runs in the
CUDA kernels of ``libcat.so``; there is no other implementation behind it,
and importing it fails loudly when the library has not been built.

The functions carry the C names: ``cat_plan_create``, ``cat_forward``,
``cat_forward_zstar``, ``cat_forward_host``, ``cat_forward_fused``,
``cat_project``, ``cat_forward_noalloc``, ``cat_backward``,
``cat_backward_dz``, ``cat_plan_create_2d``, ``cat2d_forward``, ``cat2d_scores``,
``cat_plan_query``,
``cat_plan_sync``,
``cat_plan_timing``, ``cat_plan_stage_times``, ``cat_plan_pass_times``,
``cat_plan_describe``, ``cat_plan_set_stream``, ``cat_plan_destroy`` and
``cat_status_string``.  ``Plan`` (1-D) and ``Plan2D`` (token grid) wrap them
for convenience.  The operators around a CAT layer in a training step are
``cat_plan_create_attn``, ``cat_attn_forward``, ``cat_attn_backward``
(softmax attention over packed sequences, ``AttnPlan``),
``cat_plan_create_layernorm``, ``cat_layernorm_forward``,
``cat_layernorm_backward`` (``LayerNormPlan``), ``cat_plan_create_clip``,
``cat_grad_norm`` and ``cat_grad_clip`` (``ClipPlan``); those at its ends and
between its layers are ``cat_plan_create_embed``, ``cat_embed_forward``,
``cat_embed_backward`` (``EmbedPlan``), ``cat_plan_create_resnorm``,
``cat_resnorm_forward``, ``cat_resnorm_backward`` (``ResNormPlan``),
``cat_plan_create_xent``, ``cat_xent_forward`` and ``cat_xent_backward``
(``XentPlan``).
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcat.so")

CAT_F32, CAT_BF16 = 0, 1
CAT_I32, CAT_I64 = 2, 3
CAT_OK = 0
STATUS = {
    0: "CAT_OK", -1: "CAT_ERR_INVALID_ARG", -2: "CAT_ERR_UNSUPPORTED_N",
    -3: "CAT_ERR_MISALIGNED", -4: "CAT_ERR_PLAN_MISMATCH", -5: "CAT_ERR_ALLOC",
    -6: "CAT_ERR_CUDA", -7: "CAT_ERR_DEVICE_STATUS", -8: "CAT_ERR_ALIAS",
    -9: "CAT_ERR_TOO_LARGE",
}
for _code, _name in STATUS.items():
    globals()[_name] = _code

# Every symbol include/cat.h declares, with (restype, argtypes).
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_F = ctypes.c_float
SIGNATURES = {
    "cat_plan_create": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _I, _P]),
    "cat_plan_destroy": (_I, [_P]),
    "cat_plan_set_stream": (_I, [_P, _P]),
    "cat_forward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I]),
    "cat_forward_zstar": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I]),
    "cat_forward_fused": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I]),
    "cat_project": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I]),
    "cat_forward_host": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I]),
    "cat_plan_sync": (_I, [_P]),
    "cat_plan_describe": (_I, [_P, ctypes.c_char_p, _I]),
    "cat_plan_timing": (_I, [_P, _I]),
    "cat_plan_stage_times": (_I, [_P, ctypes.POINTER(ctypes.c_float), _I,
                                  ctypes.POINTER(_I)]),
    "cat_plan_pass_times": (_I, [_P, ctypes.POINTER(ctypes.c_float), _I,
                                 ctypes.POINTER(_I)]),
    "cat_forward_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "cat_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I]),
    "cat_backward_dz": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I]),
    "cat_plan_create_2d": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _I, _I, _P]),
    "cat_plan_query": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t), ctypes.c_char_p,
                            _I]),
    "cat2d_forward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I]),
    "cat2d_scores": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I]),
    "cat_probe_dft32": (_I, [_P, _P, _I, _I, _I, _P]),
    "cat_plan_create_attn": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _I, _I, _I, _F, _P]),
    "cat_attn_forward": (_I, [_P] * 7 + [_I, _I] + [_L] * 3),
    "cat_attn_backward": (_I, [_P] * 11 + [_I, _I] + [_L] * 6),
    "cat_plan_create_layernorm": (_I, [ctypes.POINTER(_P), _I, _I, _I, _F, _P]),
    "cat_layernorm_forward": (_I, [_P] * 7 + [_I]),
    "cat_layernorm_backward": (_I, [_P] * 9 + [_I]),
    "cat_plan_create_clip": (_I, [ctypes.POINTER(_P), _I, _P, _P, _P]),
    "cat_grad_norm": (_I, [_P, _P, _P]),
    "cat_grad_clip": (_I, [_P, _P, _P, _F, _P]),
    "cat_plan_create_embed": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _F, _P]),
    "cat_embed_forward": (_I, [_P, _P, _I, _P, _P, _I]),
    "cat_embed_backward": (_I, [_P, _P, _I, _P, _P, _I, _I]),
    "cat_plan_create_resnorm": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _F, _F, _P]),
    "cat_resnorm_forward": (_I, [_P, _P, _P, _P, _I] + [_P] * 7 + [_I]),
    "cat_resnorm_backward": (_I, [_P, _P, _P, _P, _I] + [_P] * 13 + [_I]),
    "cat_plan_create_xent": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _I, _P]),
    "cat_xent_forward": (_I, [_P, _P, _P, _P, _I, _P, _P, _I]),
    "cat_xent_backward": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _P, _P, _I]),
    "cat_status_string": (ctypes.c_char_p, [_I]),
}

_LIB = None


class CatError(RuntimeError):
    """A libcat call returned a non-zero status."""

    def __init__(self, status, where=""):
        self.status = status
        super().__init__("%s%s (%d)" % (where + ": " if where else "",
                                        STATUS.get(status, "CAT_ERR_UNKNOWN"), status))


def lib():
    """The loaded libcat.so (ctypes.CDLL).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libcat.so is missing at %s: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _ptr(x):
    """Device or host address of a tensor / numpy array / int (None -> 0)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):
        return x.ctypes.data
    raise TypeError("cannot take the address of %r" % type(x))


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st, where):
    if st != CAT_OK:
        raise CatError(st, where)


def dtype_code(dtype):
    """CAT_F32 / CAT_BF16 from a code, a name or a torch dtype."""
    if isinstance(dtype, int):
        return dtype
    name = str(dtype).replace("torch.", "")
    if name in ("float32", "f32", "float"):
        return CAT_F32
    if name in ("bfloat16", "bf16"):
        return CAT_BF16
    raise ValueError("unsupported dtype %r" % (dtype,))


def cat_probe_dft32(x, y, nsig, mode, rounds, stream=None):
    """Measurement probe: one DFT-32 stage `rounds` times on `nsig` signals
    (mode 0 FP32 pipe, 1 / 2 tensor cores with 2 / 3 bf16 terms)."""
    _check(lib().cat_probe_dft32(_ptr(x), _ptr(y), nsig, mode, rounds, _stream(stream)),
           "cat_probe_dft32")


def cat_status_string(status):
    return lib().cat_status_string(status).decode()


def cat_plan_create(B, N, D, H, dtype, stream=None):
    """Create a plan; returns its handle (an int).  Raises CatError."""
    h = ctypes.c_void_p()
    _check(lib().cat_plan_create(ctypes.byref(h), B, N, D, H, dtype_code(dtype),
                                 _stream(stream)), "cat_plan_create")
    return h.value


def cat_plan_query(B, N, D, H, dtype):
    """(device workspace bytes, description) of the plan cat_plan_create would
    build for this shape, computed on the host without a device."""
    nbytes = ctypes.c_size_t(0)
    buf = ctypes.create_string_buffer(512)
    _check(lib().cat_plan_query(B, N, D, H, dtype_code(dtype), ctypes.byref(nbytes), buf, 512),
           "cat_plan_query")
    return nbytes.value, buf.value.decode()


def cat_plan_destroy(plan):
    _check(lib().cat_plan_destroy(plan), "cat_plan_destroy")


def cat_plan_set_stream(plan, stream):
    _check(lib().cat_plan_set_stream(plan, _stream(stream)), "cat_plan_set_stream")


def cat_forward(plan, X, W_A, V, O, B, N, D, H, dtype):
    _check(lib().cat_forward(plan, _ptr(X), _ptr(W_A), _ptr(V), _ptr(O), B, N, D, H,
                             dtype_code(dtype)), "cat_forward")


def cat_forward_zstar(plan, X, W_A, zstar, B, N, D, H, dtype):
    _check(lib().cat_forward_zstar(plan, _ptr(X), _ptr(W_A), _ptr(zstar), B, N, D, H,
                                   dtype_code(dtype)), "cat_forward_zstar")


def cat_forward_host(plan, X, W_A, V, O, B, N, D, H, dtype):
    _check(lib().cat_forward_host(plan, _ptr(X), _ptr(W_A), _ptr(V), _ptr(O), B, N, D, H,
                                  dtype_code(dtype)), "cat_forward_host")


def cat_forward_fused(plan, X, W_V, W_A, V, O, B, N, D, H, dtype):
    _check(lib().cat_forward_fused(plan, _ptr(X), _ptr(W_V), _ptr(W_A), _ptr(V), _ptr(O), B, N, D,
                                   H, dtype_code(dtype)), "cat_forward_fused")


def cat_project(plan, X, W_V, W_A, V, zstar, B, N, D, H, dtype):
    _check(lib().cat_project(plan, _ptr(X), _ptr(W_V), _ptr(W_A), _ptr(V), _ptr(zstar), B, N, D,
                             H, dtype_code(dtype)), "cat_project")


def cat_forward_noalloc(X, W_A, V, O, B, N, D, H, dtype, stream=None):
    """The forward without a plan or any allocation (fixed device workspace;
    B·H·N and N bounded).  Enqueued on `stream` (default: the legacy default
    stream)."""
    _check(lib().cat_forward_noalloc(_ptr(X), _ptr(W_A), _ptr(V), _ptr(O), B, N, D, H,
                                     dtype_code(dtype), _stream(stream)), "cat_forward_noalloc")


def cat_backward(plan, X, W_A, V, dO, dX, dW_A, dV, B, N, D, H, dtype):
    _check(lib().cat_backward(plan, _ptr(X), _ptr(W_A), _ptr(V), _ptr(dO), _ptr(dX), _ptr(dW_A),
                              _ptr(dV), B, N, D, H, dtype_code(dtype)), "cat_backward")


def cat_backward_dz(plan, X, W_A, V, dO, dzstar, dz, B, N, D, H, dtype):
    _check(lib().cat_backward_dz(plan, _ptr(X), _ptr(W_A), _ptr(V), _ptr(dO), _ptr(dzstar),
                                 _ptr(dz), B, N, D, H, dtype_code(dtype)), "cat_backward_dz")


def cat_plan_create_2d(B, h, w, D, H, dtype, stream=None):
    """Create a 2-D (h x w token grid) plan; returns its handle."""
    hd = ctypes.c_void_p()
    _check(lib().cat_plan_create_2d(ctypes.byref(hd), B, h, w, D, H, dtype_code(dtype),
                                    _stream(stream)), "cat_plan_create_2d")
    return hd.value


def cat2d_forward(plan, Q, K, V, O, B, h, w, D, H, dtype):
    _check(lib().cat2d_forward(plan, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), B, h, w, D, H,
                               dtype_code(dtype)), "cat2d_forward")


def cat2d_scores(plan, Q, K, a, B, h, w, D, H, dtype):
    _check(lib().cat2d_scores(plan, _ptr(Q), _ptr(K), _ptr(a), B, h, w, D, H,
                              dtype_code(dtype)), "cat2d_scores")


def cat_plan_create_attn(max_tokens, max_seqs, Hq, Hkv, dh, dtype, causal=True, scale=0.0,
                         stream=None):
    """Create a softmax-attention plan (packed sequences); returns its handle."""
    h = ctypes.c_void_p()
    _check(lib().cat_plan_create_attn(ctypes.byref(h), max_tokens, max_seqs, Hq, Hkv, dh,
                                      dtype_code(dtype), int(causal), scale, _stream(stream)),
           "cat_plan_create_attn")
    return h.value


def cat_attn_forward(plan, Q, K, V, O, lse, cu_seqlens, T, S, ldq, ldk, ldv):
    _check(lib().cat_attn_forward(plan, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse),
                                  _ptr(cu_seqlens), T, S, ldq, ldk, ldv), "cat_attn_forward")


def cat_attn_backward(plan, Q, K, V, O, lse, dO, dQ, dK, dV, cu_seqlens, T, S, ldq, ldk, ldv,
                      lddq, lddk, lddv):
    _check(lib().cat_attn_backward(plan, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), _ptr(dO),
                                   _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(cu_seqlens), T, S, ldq, ldk,
                                   ldv, lddq, lddk, lddv), "cat_attn_backward")


def cat_plan_create_layernorm(max_rows, D, dtype, eps=1e-5, stream=None):
    """Create a layer-norm plan; returns its handle."""
    h = ctypes.c_void_p()
    _check(lib().cat_plan_create_layernorm(ctypes.byref(h), max_rows, D, dtype_code(dtype), eps,
                                           _stream(stream)), "cat_plan_create_layernorm")
    return h.value


def cat_layernorm_forward(plan, X, gamma, beta, Y, mean, rstd, rows):
    _check(lib().cat_layernorm_forward(plan, _ptr(X), _ptr(gamma), _ptr(beta), _ptr(Y),
                                       _ptr(mean), _ptr(rstd), rows), "cat_layernorm_forward")


def cat_layernorm_backward(plan, X, gamma, mean, rstd, dY, dX, dgamma, dbeta, rows):
    _check(lib().cat_layernorm_backward(plan, _ptr(X), _ptr(gamma), _ptr(mean), _ptr(rstd),
                                        _ptr(dY), _ptr(dX), _ptr(dgamma), _ptr(dbeta), rows),
           "cat_layernorm_backward")


def cat_plan_create_clip(sizes, dtypes, stream=None):
    """Create a gradient-clipping plan for tensors of these sizes and dtypes;
    returns its handle."""
    n = len(sizes)
    if len(dtypes) != n:
        raise ValueError("sizes and dtypes differ in length")
    h = ctypes.c_void_p()
    _check(lib().cat_plan_create_clip(ctypes.byref(h), n, (_L * n)(*sizes),
                                      (_I * n)(*[dtype_code(d) for d in dtypes]),
                                      _stream(stream)), "cat_plan_create_clip")
    return h.value


def _addresses(tensors):
    return (_P * len(tensors))(*[_ptr(t) for t in tensors])


def cat_grad_norm(plan, grads, norm):
    _check(lib().cat_grad_norm(plan, _addresses(grads), _ptr(norm)), "cat_grad_norm")


def cat_grad_clip(plan, grads, outs, max_norm, norm):
    a = _addresses(grads)
    _check(lib().cat_grad_clip(plan, a, a if outs is grads else _addresses(outs), max_norm,
                               _ptr(norm)), "cat_grad_clip")


def id_code(dtype):
    """CAT_I32 / CAT_I64 from a code or a torch dtype."""
    if isinstance(dtype, int):
        return dtype
    name = str(dtype).replace("torch.", "")
    if name in ("int32", "int64"):
        return CAT_I32 if name == "int32" else CAT_I64
    raise ValueError("ids must be int32 or int64, not %r" % (dtype,))


def cat_plan_create_embed(max_tokens, V, D, dtype, scale=1.0, stream=None):
    """Create an embedding plan; returns its handle."""
    h = ctypes.c_void_p()
    _check(lib().cat_plan_create_embed(ctypes.byref(h), max_tokens, V, D, dtype_code(dtype),
                                       scale, _stream(stream)), "cat_plan_create_embed")
    return h.value


def cat_embed_forward(plan, ids, id_type, W, Y, T):
    _check(lib().cat_embed_forward(plan, _ptr(ids), id_code(id_type), _ptr(W), _ptr(Y), T),
           "cat_embed_forward")


def cat_embed_backward(plan, ids, id_type, dY, dW, accumulate, T):
    _check(lib().cat_embed_backward(plan, _ptr(ids), id_code(id_type), _ptr(dY), _ptr(dW),
                                    int(accumulate), T), "cat_embed_backward")


def cat_plan_create_resnorm(max_rows, D, dtype, post=False, eps=1e-5, scale=1.0, stream=None):
    """Create a plan for the residual stream between two blocks; returns its handle."""
    h = ctypes.c_void_p()
    _check(lib().cat_plan_create_resnorm(ctypes.byref(h), max_rows, D, dtype_code(dtype),
                                         int(post), eps, scale, _stream(stream)),
           "cat_plan_create_resnorm")
    return h.value


def cat_resnorm_forward(plan, R, B, gate, gate_rows, post_gamma, post_beta, gamma, beta, H, Y,
                        stats, rows):
    _check(lib().cat_resnorm_forward(plan, _ptr(R), _ptr(B), _ptr(gate), int(gate_rows),
                                     _ptr(post_gamma), _ptr(post_beta), _ptr(gamma), _ptr(beta),
                                     _ptr(H), _ptr(Y), _ptr(stats), rows), "cat_resnorm_forward")


def cat_resnorm_backward(plan, H, B, gate, gate_rows, post_gamma, post_beta, gamma, stats, dH, dY,
                         dR, dB, dgate, dpost_gamma, dpost_beta, dgamma, dbeta, rows):
    _check(lib().cat_resnorm_backward(plan, _ptr(H), _ptr(B), _ptr(gate), int(gate_rows),
                                      _ptr(post_gamma), _ptr(post_beta), _ptr(gamma), _ptr(stats),
                                      _ptr(dH), _ptr(dY), _ptr(dR), _ptr(dB), _ptr(dgate),
                                      _ptr(dpost_gamma), _ptr(dpost_beta), _ptr(dgamma),
                                      _ptr(dbeta), rows), "cat_resnorm_backward")


def cat_plan_create_xent(max_tokens, V, D, dtype, grad=True, stream=None):
    """Create a cross entropy plan; returns its handle."""
    h = ctypes.c_void_p()
    _check(lib().cat_plan_create_xent(ctypes.byref(h), max_tokens, V, D, dtype_code(dtype),
                                      int(grad), _stream(stream)), "cat_plan_create_xent")
    return h.value


def cat_xent_forward(plan, X, W, targets, id_type, loss, lse, T):
    _check(lib().cat_xent_forward(plan, _ptr(X), _ptr(W), _ptr(targets), id_code(id_type),
                                  _ptr(loss), _ptr(lse), T), "cat_xent_forward")


def cat_xent_backward(plan, X, W, targets, id_type, lse, dloss, dloss_each, dX, dW, T):
    _check(lib().cat_xent_backward(plan, _ptr(X), _ptr(W), _ptr(targets), id_code(id_type),
                                   _ptr(lse), _ptr(dloss), int(dloss_each), _ptr(dX), _ptr(dW),
                                   T), "cat_xent_backward")


def cat_plan_sync(plan):
    _check(lib().cat_plan_sync(plan), "cat_plan_sync")


def cat_plan_timing(plan, max_calls):
    _check(lib().cat_plan_timing(plan, max_calls), "cat_plan_timing")


def cat_plan_stage_times(plan):
    """(ms per stage [score, softmax/spectrum, circulant product], calls)."""
    ms = (ctypes.c_float * 3)()
    n = ctypes.c_int(0)
    _check(lib().cat_plan_stage_times(plan, ms, 3, ctypes.byref(n)), "cat_plan_stage_times")
    return [float(v) for v in ms], n.value


def cat_plan_pass_times(plan):
    """(ms of passes A, B, C summed over recorded chunks, launches of each)."""
    ms = (ctypes.c_float * 3)()
    n = ctypes.c_int(0)
    _check(lib().cat_plan_pass_times(plan, ms, 3, ctypes.byref(n)), "cat_plan_pass_times")
    return [float(v) for v in ms], n.value


def cat_plan_describe(plan):
    buf = ctypes.create_string_buffer(512)
    _check(lib().cat_plan_describe(plan, buf, 512), "cat_plan_describe")
    return buf.value.decode()


class Plan:
    """Owns one libcat plan for a fixed (B, N, D, H, dtype).

    ``forward(X, W_A, V, O=None)`` takes CUDA tensors of the plan's dtype
    (X, V, O: [B, N, D]; W_A: [D, H]) and enqueues the forward on the plan's
    stream (torch's current stream when the plan was made, unless given).
    """

    def __init__(self, B, N, D, H, dtype, stream=None):
        import torch
        self.B, self.N, self.D, self.H = B, N, D, H
        self.dtype = dtype_code(dtype)
        self.torch_dtype = torch.bfloat16 if self.dtype == CAT_BF16 else torch.float32
        if stream is None and torch.cuda.is_available():
            stream = torch.cuda.current_stream()
        self.handle = cat_plan_create(B, N, D, H, self.dtype, stream)

    def _shape(self):
        return (self.B, self.N, self.D, self.H, self.dtype)

    def forward(self, X, W_A, V, O=None):
        import torch
        if O is None:
            O = torch.empty_like(V)
        for t in (X, W_A, V, O):
            if not t.is_contiguous() or t.dtype != self.torch_dtype:
                raise ValueError("tensors must be contiguous %s" % self.torch_dtype)
        cat_forward(self.handle, X, W_A, V, O, *self._shape())
        return O

    def forward_fused(self, X, W_V, W_A, V=None, O=None):
        """V = X·W_V and the scores from one pass over X (tensor cores), then
        the forward; returns (V, O)."""
        import torch
        V = torch.empty_like(X) if V is None else V
        O = torch.empty_like(X) if O is None else O
        for t in (X, W_V, W_A, V, O):
            if not t.is_contiguous() or t.dtype != self.torch_dtype:
                raise ValueError("tensors must be contiguous %s" % self.torch_dtype)
        cat_forward_fused(self.handle, X, W_V, W_A, V, O, *self._shape())
        return V, O

    def project(self, X, W_V, W_A):
        """The fused projection alone: returns (V, z*)."""
        import torch
        V = torch.empty_like(X)
        zs = torch.empty((self.B, self.H, self.N), dtype=torch.float32, device=X.device)
        cat_project(self.handle, X, W_V, W_A, V, zs, *self._shape())
        return V, zs

    def zstar(self, X, W_A, out=None):
        import torch
        if out is None:
            out = torch.empty((self.B, self.H, self.N), dtype=torch.float32, device=X.device)
        cat_forward_zstar(self.handle, X, W_A, out, *self._shape())
        return out

    def backward(self, X, W_A, V, dO, dX=None, dW_A=None, dV=None):
        """Gradients (dX, dW_A, dV) for the upstream gradient dO = dL/dO."""
        import torch
        dX = torch.empty_like(X) if dX is None else dX
        dW_A = torch.empty_like(W_A) if dW_A is None else dW_A
        dV = torch.empty_like(V) if dV is None else dV
        for t in (X, W_A, V, dO, dX, dW_A, dV):
            if not t.is_contiguous() or t.dtype != self.torch_dtype:
                raise ValueError("tensors must be contiguous %s" % self.torch_dtype)
        cat_backward(self.handle, X, W_A, V, dO, dX, dW_A, dV, *self._shape())
        return dX, dW_A, dV

    def backward_dz(self, X, W_A, V, dO):
        """(dL/dz*, dL/dz), each fp32 [B, H, N]."""
        import torch
        shape = (self.B, self.H, self.N)
        dzs = torch.empty(shape, dtype=torch.float32, device=X.device)
        dz = torch.empty(shape, dtype=torch.float32, device=X.device)
        cat_backward_dz(self.handle, X, W_A, V, dO, dzs, dz, *self._shape())
        return dzs, dz

    def forward_host(self, X, W_A, V, O):
        cat_forward_host(self.handle, X, W_A, V, O, *self._shape())
        return O

    def sync(self):
        cat_plan_sync(self.handle)

    def describe(self):
        return cat_plan_describe(self.handle)

    def timing(self, max_calls):
        cat_plan_timing(self.handle, max_calls)

    def stage_times(self):
        return cat_plan_stage_times(self.handle)

    def pass_times(self):
        return cat_plan_pass_times(self.handle)

    def close(self):
        if self.handle:
            cat_plan_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Plan2D:
    """Owns one 2-D circulant-attention plan for a fixed (B, h, w, D, H, dtype):
    ``forward(Q, K, V, O=None)`` with CUDA tensors [B, h·w, D] of the plan's
    dtype; ``scores(Q, K)`` returns the fp32 scores a [B, H, h·w]."""

    def __init__(self, B, h, w, D, H, dtype, stream=None):
        import torch
        self.B, self.h, self.w, self.D, self.H = B, h, w, D, H
        self.dtype = dtype_code(dtype)
        self.torch_dtype = torch.bfloat16 if self.dtype == CAT_BF16 else torch.float32
        if stream is None and torch.cuda.is_available():
            stream = torch.cuda.current_stream()
        self.handle = cat_plan_create_2d(B, h, w, D, H, self.dtype, stream)

    def _shape(self):
        return (self.B, self.h, self.w, self.D, self.H, self.dtype)

    def forward(self, Q, K, V, O=None):
        import torch
        if O is None:
            O = torch.empty_like(V)
        for t in (Q, K, V, O):
            if not t.is_contiguous() or t.dtype != self.torch_dtype:
                raise ValueError("tensors must be contiguous %s" % self.torch_dtype)
        cat2d_forward(self.handle, Q, K, V, O, *self._shape())
        return O

    def scores(self, Q, K):
        import torch
        a = torch.empty((self.B, self.H, self.h * self.w), dtype=torch.float32, device=Q.device)
        cat2d_scores(self.handle, Q, K, a, *self._shape())
        return a

    def sync(self):
        cat_plan_sync(self.handle)

    def describe(self):
        return cat_plan_describe(self.handle)

    def close(self):
        if self.handle:
            cat_plan_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_MARSHAL = None


def _marshal():
    """The native marshalling of the operator plans' calls (csrc/marshal.cpp),
    built for the running torch.  Raises if it has not been built."""
    global _MARSHAL
    if _MARSHAL is None:
        import importlib.machinery
        import importlib.util

        from .build import marshal_path
        path = marshal_path()
        if not os.path.exists(path):
            raise RuntimeError(
                "%s is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` "
                "(needs torch's headers and a C++ compiler)" % path)
        loader = importlib.machinery.ExtensionFileLoader("_marshal", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
        loader.exec_module(m)
        _MARSHAL = m
    return _MARSHAL


class _OpPlan:
    """What the operator plans share.  With a stream given, every call runs on
    it, and outputs that the call allocates belong to it; without one, all is
    on torch's current stream at the call."""

    handle = None

    def _open(self, device, stream):
        import torch
        if device is None:
            device = torch.cuda.current_device() if torch.cuda.is_available() else 0
        self.device = torch.device("cuda", device) if isinstance(device, int) else \
            torch.device(device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._fixed = stream is not None
        self._on = _stream(stream) if self._fixed else None
        if self._fixed:
            self._under = torch.cuda.stream
            self._own = stream if hasattr(stream, "cuda_stream") else \
                torch.cuda.ExternalStream(self._on, self.device) if self._on else \
                torch.cuda.default_stream(self.device)
        self._current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
        self._index = self.device.index

    def _native(self, names, dims=(0, 0, 0), dtype=CAT_F32):
        """What the native calls need: the plan, its shape, the C functions."""
        fns = [ctypes.cast(getattr(lib(), n), _P).value for n in names]
        self._names = names
        self._args = _marshal().make(*fns, self.handle, *dims, dtype, self._index)

    def _use(self):
        """Point the plan at the stream this call runs on."""
        s = self._current(self._index)
        if s != self._on:
            cat_plan_set_stream(self.handle, s)
            self._on = s

    def _call(self, which, fn, *tensors):
        """The outputs of a native call on the plan's stream, or its error."""
        if self._fixed:
            with self._under(self._own):
                r = fn(self._args, *tensors)
        else:
            self._use()
            r = fn(self._args, *tensors)
        if r.__class__ is int:
            raise CatError(r, self._names[which])
        return r

    def sync(self):
        cat_plan_sync(self.handle)

    def describe(self):
        return cat_plan_describe(self.handle)

    def close(self):
        if self.handle:
            self._args = None                 # (a later call is refused)
            cat_plan_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _on_device(device):
    import contextlib

    import torch
    return torch.cuda.device(device) if torch.cuda.is_available() else contextlib.nullcontext()


class AttnPlan(_OpPlan):
    """Softmax attention over packed sequences: up to ``max_tokens`` rows and
    ``max_seqs`` sequences a call, ``Hq`` query heads over ``Hkv`` key heads of
    width ``dh``.

    ``forward(Q, K, V, cu_seqlens)`` -> (O, lse) and ``backward(Q, K, V, O,
    lse, dO, cu_seqlens)`` -> (dQ, dK, dV); Q, O, dO [T, Hq, dh], K, V
    [T, Hkv, dh], lse fp32 [Hq, T], cu_seqlens int32 [S + 1] on the device.
    Q, K, V (and dQ, dK, dV where given) may be column ranges of wider rows.
    Rows that no sequence holds (padding) are not written: in outputs that the
    call allocates they are undefined, so pass zeroed ones (``O=``, ``dQ=`` ..)
    where a later product runs over them.  ``scale``: positive, or None for
    1/sqrt(dh).
    """

    def __init__(self, max_tokens, max_seqs, Hq, Hkv, dh, dtype, causal=True, scale=None,
                 stream=None, device=None):
        if scale is not None and not scale > 0:      # (0 is the C interface's 1/sqrt(dh))
            raise ValueError("scale must be positive, or None for 1/sqrt(dh)")
        self.Hq, self.Hkv, self.dh = Hq, Hkv, dh
        self.dtype = dtype_code(dtype)
        self._open(device, stream)
        with _on_device(self.device):
            self.handle = cat_plan_create_attn(max_tokens, max_seqs, Hq, Hkv, dh, self.dtype,
                                               causal, 0.0 if scale is None else scale, self._on)
        self._native(("cat_attn_forward", "cat_attn_backward"), (Hq, Hkv, dh), self.dtype)
        self._fwd, self._bwd = _marshal().attn_forward, _marshal().attn_backward

    def forward(self, Q, K, V, cu_seqlens, O=None, lse=None):
        return self._call(0, self._fwd, Q, K, V, cu_seqlens, O, lse)

    def backward(self, Q, K, V, O, lse, dO, cu_seqlens, dQ=None, dK=None, dV=None):
        return self._call(1, self._bwd, Q, K, V, O, lse, dO, cu_seqlens, dQ, dK, dV)


class LayerNormPlan(_OpPlan):
    """Layer norm over the last dimension (``D``) of up to ``max_rows`` rows.

    ``forward(X, gamma=None, beta=None)`` -> (Y, mean, rstd) and ``backward(X,
    gamma, mean, rstd, dY)`` -> (dX, dgamma, dbeta); X, Y, dY, dX [..., D],
    mean and rstd fp32 [...].
    """

    def __init__(self, max_rows, D, dtype, eps=1e-5, stream=None, device=None):
        self.D = D
        self.dtype = dtype_code(dtype)
        self._open(device, stream)
        with _on_device(self.device):
            self.handle = cat_plan_create_layernorm(max_rows, D, self.dtype, eps, self._on)
        self._native(("cat_layernorm_forward", "cat_layernorm_backward"), (D, 0, 0), self.dtype)
        self._fwd, self._bwd = _marshal().ln_forward, _marshal().ln_backward

    def forward(self, X, gamma=None, beta=None, Y=None, mean=None, rstd=None):
        return self._call(0, self._fwd, X, gamma, beta, Y, mean, rstd)

    def backward(self, X, gamma, mean, rstd, dY, dX=None, dgamma=None, dbeta=None):
        return self._call(1, self._bwd, X, gamma, mean, rstd, dY, dX, dgamma, dbeta)


class ClipPlan(_OpPlan):
    """The global norm of a list of gradients of these ``sizes`` (elements) and
    ``dtypes``, and clipping by it.

    ``norm(grads)`` -> fp32 scalar tensor; ``clip(grads, max_norm, out=None)``
    scales the gradients in place (or into ``out``) by max_norm / norm where
    the norm is larger, and returns the norm before clipping.
    """

    def __init__(self, sizes, dtypes, stream=None, device=None):
        self.sizes = [int(n) for n in sizes]
        self.dtypes = [dtype_code(d) for d in dtypes]
        self._open(device, stream)
        with _on_device(self.device):
            self.handle = cat_plan_create_clip(self.sizes, self.dtypes, self._on)
        self._native(("cat_grad_norm", "cat_grad_clip"))
        _marshal().set_list(self._args, self.sizes, self.dtypes)
        self._clip = _marshal().clip

    def norm(self, grads, norm=None):
        return self._call(0, self._clip, grads, None, None, norm)

    def clip(self, grads, max_norm, out=None, norm=None):
        return self._call(1, self._clip, grads, out, float(max_norm), norm)


class EmbedPlan(_OpPlan):
    """Rows of a table W [V, D] looked up by token, for up to ``max_tokens``
    tokens a call.

    ``forward(ids, W)`` -> Y [..., D] = scale·W[ids], zeros where an id is
    negative; ``backward(ids, dY)`` -> dW [V, D], the sum of the rows of each
    id's tokens times scale.  With ``accumulate=True`` the sums are added to the
    ``dW`` given (the gradient of output weights tied to the table, say), and
    rows of other ids keep their values.  ids: int32 or int64 of any shape.
    """

    def __init__(self, max_tokens, V, D, dtype, scale=1.0, stream=None, device=None):
        self.V, self.D = V, D
        self.dtype = dtype_code(dtype)
        self._open(device, stream)
        with _on_device(self.device):
            self.handle = cat_plan_create_embed(max_tokens, V, D, self.dtype, scale, self._on)
        self._native(("cat_embed_forward", "cat_embed_backward"), (V, D, 0), self.dtype)
        self._fwd, self._bwd = _marshal().embed_forward, _marshal().embed_backward

    def forward(self, ids, W, Y=None):
        return self._call(0, self._fwd, ids, W, Y)

    def backward(self, ids, dY, dW=None, accumulate=False):
        return self._call(1, self._bwd, ids, dY, dW, accumulate)


class ResNormPlan(_OpPlan):
    """The residual stream between two blocks: up to ``max_rows`` rows of D.

    ``forward(R, B, gate, gamma, beta, post_gamma, post_beta)`` -> (H, Y, stats):
    H = R + scale·gate·u with u = LN(B)·post_gamma + post_beta (``post=True``) or
    u = B, and Y = LN(H)·gamma + beta.  gate: None, [D], or the shape of B; every
    norm weight may be None.  ``backward(H, B, gate, gamma, post_gamma,
    post_beta, stats, dH, dY)`` -> (dR, dB, dgate, dgamma, dbeta, dpost_gamma,
    dpost_beta), None where there is no gate or no norm behind the block; dH may
    be None.  stats: fp32 [2 or 4, ...], mean and rstd of H, and of B.
    """

    def __init__(self, max_rows, D, dtype, eps=1e-5, scale=1.0, post=False, stream=None,
                 device=None):
        self.D, self.post = D, bool(post)
        self.dtype = dtype_code(dtype)
        self._open(device, stream)
        with _on_device(self.device):
            self.handle = cat_plan_create_resnorm(max_rows, D, self.dtype, self.post, eps, scale,
                                                  self._on)
        self._native(("cat_resnorm_forward", "cat_resnorm_backward"), (D, int(self.post), 0),
                     self.dtype)
        self._fwd, self._bwd = _marshal().resnorm_forward, _marshal().resnorm_backward

    def forward(self, R, B, gate=None, gamma=None, beta=None, post_gamma=None, post_beta=None,
                H=None, Y=None, stats=None):
        return self._call(0, self._fwd, R, B, gate, gamma, beta, post_gamma, post_beta, H, Y,
                          stats)

    def backward(self, H, B, gate, gamma, post_gamma, post_beta, stats, dH, dY, dR=None, dB=None,
                 dgate=None, dgamma=None, dbeta=None, dpost_gamma=None, dpost_beta=None):
        return self._call(1, self._bwd, H, B, gate, gamma, post_gamma, post_beta, stats, dH, dY,
                          dR, dB, dgate, dgamma, dbeta, dpost_gamma, dpost_beta)


class XentPlan(_OpPlan):
    """Softmax cross entropy over a vocabulary of V from hidden states of width
    D, for up to ``max_tokens`` tokens a call, without keeping the logits.

    ``forward(X, W, targets)`` -> (loss, lse), fp32 [...]; X [..., D], W [V, D],
    targets int32 or int64 [...], negative where a token has none (loss and lse
    are 0 there).  ``backward(X, W, targets, lse, dloss)`` -> (dX, dW); dloss:
    fp32, one value or the shape of targets.  ``dX=False`` or ``dW=False``: not
    wanted (None).  ``grad=False``: a plan for the forward alone, with far less
    workspace.
    """

    def __init__(self, max_tokens, V, D, dtype, grad=True, stream=None, device=None):
        self.V, self.D = V, D
        self.dtype = dtype_code(dtype)
        self._open(device, stream)
        with _on_device(self.device):
            self.handle = cat_plan_create_xent(max_tokens, V, D, self.dtype, grad, self._on)
        self._native(("cat_xent_forward", "cat_xent_backward"), (V, D, 0), self.dtype)
        self._fwd, self._bwd = _marshal().xent_forward, _marshal().xent_backward

    def forward(self, X, W, targets, loss=None, lse=None):
        return self._call(0, self._fwd, X, W, targets, loss, lse)

    def backward(self, X, W, targets, lse, dloss, dX=None, dW=None):
        return self._call(1, self._bwd, X, W, targets, lse, dloss, dX, dW)


__all__ = ["EmbedPlan", "ResNormPlan", "XentPlan", "cat_plan_create_embed", "cat_embed_forward",
           "cat_embed_backward", "cat_plan_create_resnorm", "cat_resnorm_forward",
           "cat_resnorm_backward", "cat_plan_create_xent", "cat_xent_forward",
           "cat_xent_backward", "id_code", "CAT_I32", "CAT_I64", "AttnPlan", "LayerNormPlan",
           "ClipPlan", "cat_plan_create_attn", "cat_attn_forward", "cat_attn_backward",
           "cat_plan_create_layernorm", "cat_layernorm_forward", "cat_layernorm_backward",
           "cat_plan_create_clip", "cat_grad_norm", "cat_grad_clip",
           "CatError", "Plan", "Plan2D", "lib", "dtype_code", "cat_plan_create", "cat_plan_destroy",
           "cat_plan_set_stream", "cat_forward", "cat_forward_zstar", "cat_forward_host",
           "cat_plan_sync", "cat_plan_describe", "cat_plan_timing", "cat_plan_stage_times",
           "cat_plan_pass_times", "cat_forward_noalloc", "cat_backward", "cat_backward_dz",
           "cat_plan_create_2d", "cat2d_forward", "cat2d_scores", "cat_plan_query",
           "cat_status_string", "CAT_F32", "CAT_BF16",
           "SIGNATURES", "LIB_PATH"]
