"""Python binding of libfq: the C ABI calls with torch tensors for device memory.

Every step of the operator runs in libfq's CUDA kernels; this module only checks
tensor placement, allocates outputs with torch, and passes pointers and the current
CUDA stream. There is no CPU implementation here.

stream= takes another torch.cuda.Stream than the current one, for the kernels and for the
outputs and workspaces that a call allocates: as with any tensor of another stream's memory,
a caller who uses an output on the current stream lets that wait for `stream`, and calls
record_stream on it before dropping it.
"""

import ctypes

import torch

from . import _lib

_DT = {torch.bfloat16: _lib.FQ_BF16, torch.float16: _lib.FQ_FP16}
_OUT_DT = {**_DT, torch.float32: _lib.FQ_FP32}
_INT_OUT = {"int32": _lib.FQ_OUT_INT32, "int8": _lib.FQ_OUT_INT8}  # else INT4


def _stream_ptr(stream=None):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _raw_stream(stream, device):
    """The stream's handle as a number (the current one of `device` unless given)."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device)


def _fits(t, dtype, device):
    """Whether t is a contiguous tensor of this type on this CUDA device: the checks of a call
    that is in order. (A call that is not goes through the ones below, which say what is
    wrong.)"""
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.is_contiguous()


def _empty(like, shape, dtype, stream):
    """An output or a workspace, on the device of `like`, that a call on `stream` (None: the
    current one) writes. It is taken from that stream's memory: memory that another stream freed
    may still be read by what is queued there."""
    if stream is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _check_input(name, t, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libfq has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")


def _check_device(x, **others):
    """x on the current CUDA device (the plan was made, and its kernels launch, there) and
    every other tensor beside it."""
    cur = torch.cuda.current_device()
    if x.device.index != cur:
        raise ValueError(f"x is on {x.device} but the current CUDA device is cuda:{cur}; "
                         "call torch.cuda.set_device first")
    for name, t in others.items():
        if t is not None and t.device != x.device:
            raise ValueError(f"{name} must be on {x.device}, got {t.device}")


def _check_output(name, t, nbytes, device, dtype=None):
    """A caller-supplied output: on `device`, contiguous, exactly `nbytes` bytes (the
    kernel writes all of them, so a smaller buffer would be overrun), and of `dtype` when
    the values are numbers rather than packed codes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    have = t.numel() * t.element_size()
    if have != nbytes:
        raise ValueError(f"{name} must hold {nbytes} bytes, got {have}")


def _scale_bytes(K, M, N):
    return K * (-(-M * N // 64)) * 2


class FlatQuant:
    """A plan for one shape [K, M, N] and input dtype (the handle of fq_create)."""

    def __init__(self, K, M, N, dtype=torch.bfloat16, kernel="auto"):
        lib = _lib.load()
        if dtype not in _DT:
            raise ValueError("dtype must be torch.bfloat16 or torch.float16")
        self.K, self.M, self.N, self.dtype = int(K), int(M), int(N), dtype
        h = ctypes.c_void_p()
        _lib.check(lib.fq_create(ctypes.byref(h), self.K, self.M, self.N, _DT[dtype]),
                   "fq_create")
        self._h = h
        self._lib = lib
        self.set_kernel(kernel)

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.fq_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_kernel(self, kernel):
        code = {"auto": _lib.FQ_KERNEL_AUTO, "general": _lib.FQ_KERNEL_GENERAL,
                "tcgen05": _lib.FQ_KERNEL_TCGEN05}[kernel]
        _lib.check(self._lib.fq_set_kernel(self._h, code), "fq_set_kernel")
        self.kernel = kernel

    def set_intermediate_rounding(self, enable):
        """Round x' = x . P2 to the input dtype before the left product (see
        fq_set_intermediate_rounding); runs the general kernel."""
        _lib.check(self._lib.fq_set_intermediate_rounding(self._h, int(bool(enable))),
                   "fq_set_intermediate_rounding")
        self.intermediate_rounding = bool(enable)

    def debug_arm_stall(self, wait_limit_s):
        """Test hook: the next tensor-core launch issues no x loads and every bounded wait in
        it gives up after wait_limit_s seconds (see fq_debug_arm_stall)."""
        _lib.check(self._lib.fq_debug_arm_stall(self._h, float(wait_limit_s)), "fq_debug_arm_stall")

    @property
    def last_kernel(self):
        return {0: "auto", 1: "general", 2: "tcgen05"}[self._lib.fq_last_kernel(self._h)]

    @property
    def last_launch_count(self):
        return self._lib.fq_last_launch_count(self._h)

    def device_status(self):
        v = ctypes.c_uint32(0)
        st = self._lib.fq_device_status(self._h, ctypes.byref(v))
        if st not in (_lib.FQ_OK, _lib.FQ_ERR_DEVICE_TIMEOUT):
            _lib.check(st, "fq_device_status")
        return int(v.value)

    def _inputs(self, x, P1, P2, allow_no_p2=False):
        dev = torch.cuda.current_device() if isinstance(x, torch.Tensor) and x.is_cuda else -1
        if (dev >= 0 and _fits(x, self.dtype, dev) and _fits(P1, self.dtype, dev) and _fits(P2, self.dtype, dev)
                and x.shape == (self.K, self.M, self.N) and P1.shape == (self.M, self.M)
                and P2.shape == (self.N, self.N)):
            return P2
        _check_input("x", x, self.dtype)
        _check_input("P1", P1, self.dtype)
        if tuple(x.shape) != (self.K, self.M, self.N):
            raise ValueError(f"x must have shape {(self.K, self.M, self.N)}, got {tuple(x.shape)}")
        if tuple(P1.shape) != (self.M, self.M):
            raise ValueError("P1 must be [M, M]")
        if P2 is not None and P2.numel() == 0 and allow_no_p2:
            P2 = None
        if P2 is None:
            if not allow_no_p2:
                raise ValueError("P2 is required in per-token mode")
        else:
            _check_input("P2", P2, self.dtype)
            if tuple(P2.shape) != (self.N, self.N):
                raise ValueError("P2 must be [N, N]")
        _check_device(x, P1=P1, P2=P2)
        return P2

    def quantize_per_token(self, x, P1, P2, clip_ratio=1.0, out_dtype="int4",
                           out=None, quant_scale=None, stream=None):
        """Per-token INT4 or INT8 quantization of P1 . (x . P2). Returns (out, quantScale):
        out is uint8 [K, M*N/2] for "int4", int32 [K, M, N/8] for "int32" or int8 [K, M*N]
        for "int8" (the activations of int8_matmul)."""
        self._inputs(x, P1, P2)
        K, M, N = self.K, self.M, self.N
        if out is None:
            if out_dtype == "int8":
                out = _empty(x, (K, M * N), torch.int8, stream)
            elif out_dtype == "int32":
                out = _empty(x, (K, M, N // 8), torch.int32, stream)
            else:
                out = _empty(x, (K, M * N // 2), torch.uint8, stream)
        else:
            _check_output("out", out, K * M * N // (1 if out_dtype == "int8" else 2), x.device)
        if quant_scale is None:
            quant_scale = _empty(x, (K,), torch.float32, stream)
        else:
            _check_output("quant_scale", quant_scale, 4 * K, x.device, torch.float32)
        st = self._lib.fq_quantize_per_token(
            self._h, x.data_ptr(), P1.data_ptr(), P2.data_ptr(), float(clip_ratio),
            _INT_OUT.get(out_dtype, _lib.FQ_OUT_INT4), out.data_ptr(), quant_scale.data_ptr(),
            _raw_stream(stream, x.get_device()))
        if st != _lib.FQ_OK:
            _lib.check(st, "fq_quantize_per_token")
        return out, quant_scale

    def quantize_mx(self, x, P1, P2, dst_type_max=0.0, out=None, scales=None, stream=None):
        """Per-group E2M1 + E8M0 quantization of P1 . (x . P2) (P2 None skips the right
        multiply). Returns (out uint8 [K, M*N/2], scales uint8 [K, ceilDiv(M*N,64), 2])."""
        P2 = self._inputs(x, P1, P2, allow_no_p2=True)
        K, M, N = self.K, self.M, self.N
        if out is None:
            out = _empty(x, (K, M * N // 2), torch.uint8, stream)
        else:
            _check_output("out", out, K * M * N // 2, x.device)
        if scales is None:
            scales = _empty(x, (K, -(-M * N // 64), 2), torch.uint8, stream)
        else:
            _check_output("scales", scales, _scale_bytes(K, M, N), x.device)
        _lib.check(self._lib.fq_quantize_mx(
            self._h, _ptr(x), _ptr(P1), _ptr(P2), float(dst_type_max), _ptr(out),
            _ptr(scales), _stream_ptr(stream)), "fq_quantize_mx")
        return out, scales

    def debug_rotate(self, x, P1, P2, out=None, stream=None):
        """x'' = P1 . (x . P2) as float32 [K, M, N] (test hook)."""
        P2 = self._inputs(x, P1, P2, allow_no_p2=True)
        if out is None:
            out = _empty(x, (self.K, self.M, self.N), torch.float32, stream)
        else:
            _check_output("out", out, 4 * self.K * self.M * self.N, x.device, torch.float32)
        _lib.check(self._lib.fq_debug_rotate(self._h, _ptr(x), _ptr(P1), _ptr(P2), _ptr(out),
                                             _stream_ptr(stream)), "fq_debug_rotate")
        return out


def quantize_per_token(x, P1, P2, clip_ratio=1.0, out_dtype="int4", kernel="auto"):
    K, M, N = x.shape
    return FlatQuant(K, M, N, x.dtype, kernel).quantize_per_token(x, P1, P2, clip_ratio, out_dtype)


def quantize_mx(x, P1, P2, dst_type_max=0.0, kernel="auto"):
    K, M, N = x.shape
    return FlatQuant(K, M, N, x.dtype, kernel).quantize_mx(x, P1, P2, dst_type_max)


def quantize_mx_static(x, P1, P2, dst_type_max=0.0, out=None, scales=None, stream=None):
    """Per-group quantization through fq_quantize_mx_static: no handle, and the library
    allocates nothing (its scratch is a static device array). Outputs are allocated here
    by torch unless passed in."""
    lib = _lib.load()
    if x.dtype not in _DT:
        raise ValueError("x must be bfloat16 or float16")
    for name, t in (("x", x), ("P1", P1)):
        _check_input(name, t, x.dtype)
    if P2 is not None and P2.numel() == 0:
        P2 = None
    if P2 is not None:
        _check_input("P2", P2, x.dtype)
    if x.dim() != 3:
        raise ValueError("x must be [K, M, N]")
    K, M, N = x.shape
    if tuple(P1.shape) != (M, M):
        raise ValueError("P1 must be [M, M]")
    if P2 is not None and tuple(P2.shape) != (N, N):
        raise ValueError("P2 must be [N, N]")
    _check_device(x, P1=P1, P2=P2)
    if out is None:
        out = _empty(x, (K, M * N // 2), torch.uint8, stream)
    else:
        _check_output("out", out, K * M * N // 2, x.device)
    if scales is None:
        scales = _empty(x, (K, -(-M * N // 64), 2), torch.uint8, stream)
    else:
        _check_output("scales", scales, _scale_bytes(K, M, N), x.device)
    _lib.check(lib.fq_quantize_mx_static(K, M, N, _DT[x.dtype], _ptr(x), _ptr(P1), _ptr(P2),
                                         float(dst_type_max), _ptr(out), _ptr(scales),
                                         _stream_ptr(stream)), "fq_quantize_mx_static")
    return out, scales


def int8_matmul(a, a_scale, w, w_scale, out_dtype=torch.bfloat16, out=None, status=None, stream=None):
    """C [T, O] = (a . w^T) * a_scale[:, None] * w_scale[None, :] for int8 a [T, L] and w [O, L]
    with float32 scales (see fq_int8_matmul): a and a_scale as quantize_per_token gives them
    with out_dtype="int8", w and w_scale alike for the weights' rows. out_dtype bfloat16,
    float16 or float32. status: an int32 tensor of one element, ORed with a nonzero code if a
    bounded wait inside the kernel gives up (the output is then undefined); without it
    int8_device_status() tells."""
    lib = _lib.load()
    dev = torch.cuda.current_device() if isinstance(a, torch.Tensor) and a.is_cuda else -1
    if not (dev >= 0 and _fits(a, torch.int8, dev) and _fits(a_scale, torch.float32, dev) and _fits(w, torch.int8, dev)
            and _fits(w_scale, torch.float32, dev)):
        for name, t, dt in (("a", a, torch.int8), ("a_scale", a_scale, torch.float32), ("w", w, torch.int8),
                            ("w_scale", w_scale, torch.float32)):
            _check_input(name, t, dt)
        _check_device(a, a_scale=a_scale, w=w, w_scale=w_scale)
    if (a.dim(), a_scale.dim(), w.dim(), w_scale.dim()) != (2, 1, 2, 1):
        raise ValueError("a and w must have two dimensions, a_scale and w_scale one")
    if out_dtype not in _OUT_DT:
        raise ValueError("out_dtype must be torch.bfloat16, torch.float16 or torch.float32")
    T, L = a.shape
    O, Lw = w.shape
    if Lw != L:
        raise ValueError(f"w must have rows of {L} codes, got {Lw}")
    if a_scale.numel() != T or w_scale.numel() != O:
        raise ValueError("a_scale and w_scale must have one scale per row of a and of w")
    if out is None:
        out = _empty(a, (T, O), out_dtype, stream)
    else:
        _check_output("out", out, T * O * out_dtype.itemsize, a.device, out_dtype)
    if status is not None:
        _check_output("status", status, 4, a.device, torch.int32)
    st = lib.fq_int8_matmul(T, O, L, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                            _OUT_DT[out_dtype], out.data_ptr(), status.data_ptr() if status is not None else None,
                            _raw_stream(stream, dev))
    if st != _lib.FQ_OK:
        _lib.check(st, "fq_int8_matmul")
    return out


def int8_device_status():
    """Reads and clears the current device's status word of int8_matmul calls without one of their
    own: 0, or the bits of bounded waits that gave up since. Synchronizes the device."""
    v = ctypes.c_uint32(0)
    st = _lib.load().fq_int8_device_status(ctypes.byref(v))
    if st not in (_lib.FQ_OK, _lib.FQ_ERR_DEVICE_TIMEOUT):
        _lib.check(st, "fq_int8_device_status")
    return int(v.value)


class KVCache:
    """A paged key / value cache in 8 bits: E4M3 codes [num_pages, kv_heads, page_size, head_dim]
    (`k`, `v`) and one E8M0 byte for each page and head, [num_pages, kv_heads] (`k_scale`,
    `v_scale`); see fq_kv_cache. page_size 16, 32, 64 or 128, head_dim 64 or 128.

    The batch of a call is given by three int32 CUDA tensors, which the kernels read on the
    device: cu_new [B + 1] (rows cu_new[b] .. cu_new[b + 1] - 1 of the token arrays are sequence
    b's new tokens), seq_lens [B] (lengths with the new tokens) and page_table [B, W].
    """

    def __init__(self, num_pages, page_size, kv_heads, head_dim, device=None):
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        shape = (int(num_pages), int(kv_heads), int(page_size), int(head_dim))
        codes = [torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.full(shape[:2], 87, dtype=torch.uint8, device=dev) for _ in range(2)]
        self._attach(*codes, *scales)

    @classmethod
    def from_buffers(cls, k, v, k_scale, v_scale):
        """A cache over the caller's own tensors (k, v float8_e4m3fn, the scales uint8)."""
        self = cls.__new__(cls)
        self._attach(k, v, k_scale, v_scale)
        return self

    def _attach(self, k, v, k_scale, v_scale):
        for name, t, dt in (("k", k, torch.float8_e4m3fn), ("v", v, torch.float8_e4m3fn),
                            ("k_scale", k_scale, torch.uint8), ("v_scale", v_scale, torch.uint8)):
            _check_input(name, t, dt)
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must both be [num_pages, kv_heads, page_size, head_dim]")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.shape != k.shape[:2]:
                raise ValueError(f"{name} must be [num_pages, kv_heads]")
        for name, t in (("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if t.device != k.device:
                raise ValueError(f"{name} must be on {k.device}, got {t.device}")
        if k.shape[2] not in (16, 32, 64, 128):
            raise ValueError(f"page_size must be 16, 32, 64 or 128, got {k.shape[2]}")
        if k.shape[3] not in (64, 128):
            raise ValueError(f"head_dim must be 64 or 128, got {k.shape[3]}")
        self._tensors = (k, v, k_scale, v_scale)
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self._device = k.get_device()
        self._status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._status_ptr = self._status.data_ptr()
        self._lib = _lib.load()
        self._desc = _lib.KvCacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                      self.num_pages, self.kv_heads, self.page_size, self.head_dim)
        self._desc_ref = ctypes.byref(self._desc)
        self._workspace_bytes = {}  # by the sizes that decide it

    k = property(lambda self: self._tensors[0], doc="E4M3 codes of the keys")
    v = property(lambda self: self._tensors[1], doc="E4M3 codes of the values")
    k_scale = property(lambda self: self._tensors[2], doc="E8M0 bytes of the keys")
    v_scale = property(lambda self: self._tensors[3], doc="E8M0 bytes of the values")

    def device_status(self):
        """Reads and clears the cache's status word: 0, or the bits that calls on this cache have
        set since (FQ_KV_BAD_BATCH: a batch's contents were out of range), on whatever stream.
        Synchronizes the device."""
        torch.cuda.synchronize(self._device)
        v = int(self._status.item())
        if v:
            self._status.bitwise_and_(~v)
            torch.cuda.synchronize(self._device)  # a later call on another stream comes after it
        return v

    def _batch_desc(self, cu_new, seq_lens, page_table):
        dev = self._device
        if not (_fits(cu_new, torch.int32, dev) and _fits(seq_lens, torch.int32, dev)
                and _fits(page_table, torch.int32, dev)):
            for name, t in (("cu_new", cu_new), ("seq_lens", seq_lens), ("page_table", page_table)):
                _check_input(name, t, torch.int32)
            _check_device(self.k, cu_new=cu_new, seq_lens=seq_lens, page_table=page_table)
        B = seq_lens.numel()
        if seq_lens.dim() != 1 or cu_new.dim() != 1 or cu_new.numel() != B + 1:
            raise ValueError("seq_lens must be [B] and cu_new [B + 1]")
        if page_table.dim() != 2 or page_table.shape[0] != B:
            raise ValueError("page_table must be [B, W]")
        return _lib.KvBatchDesc(cu_new.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), B,
                                page_table.shape[1])

    def _tokens(self, name, t, T, heads, dtype):
        """A token array [T, heads, head_dim]: heads contiguous, any distance between tokens."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.get_device() != self._device:
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor (libfq has no CPU path)")
            raise ValueError(f"{name} must be on {self.k.device}, got {t.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
        D = self.head_dim
        shape = t.shape
        if len(shape) != 3 or shape[0] != T or shape[2] != D or (heads is not None and shape[1] != heads):
            raise ValueError(f"{name} must be [{T}, {'heads' if heads is None else heads}, {D}], got {tuple(shape)}")
        s0, s1, s2 = t.stride()
        if s2 != 1 or (shape[1] > 1 and s1 != D):
            raise ValueError(f"the heads of one token of {name} must be contiguous")
        return s0 if T > 1 else shape[1] * D

    def _check_current(self):
        """The cache on the current CUDA device, where its kernels are launched."""
        cur = torch.cuda.current_device()
        if self._device != cur:
            raise ValueError(f"the cache is on {self.k.device} but the current CUDA device is cuda:{cur}; "
                             "call torch.cuda.set_device first")

    def append(self, k, v, cu_new, seq_lens, page_table, q=None, inv_freq=None, interleaved=False, q_out=None,
               stream=None):
        """Appends k and v [T, kv_heads, head_dim] (bfloat16 or float16) to the cache. With
        inv_freq (float32 [rot / 2]) keys, and q [T, q_heads, head_dim] if given, are rotated by
        their positions first (see fq_kv_append). Returns the rotated queries, or None."""
        if not isinstance(k, torch.Tensor) or k.dtype not in _DT:
            raise ValueError("k must be a bfloat16 or float16 tensor")
        self._check_current()
        T = k.shape[0] if k.dim() else 0
        ks = self._tokens("k", k, T, self.kv_heads, k.dtype)
        vs = self._tokens("v", v, T, self.kv_heads, k.dtype)
        batch = self._batch_desc(cu_new, seq_lens, page_table)
        rot, freq, qs, hq, q_ptr, out_ptr = 0, None, 0, 0, None, None
        if inv_freq is not None:
            if not _fits(inv_freq, torch.float32, self._device):
                _check_input("inv_freq", inv_freq, torch.float32)
                _check_device(self.k, inv_freq=inv_freq)
            rot, freq = 2 * inv_freq.numel(), inv_freq.data_ptr()
        if q is not None:
            qs = self._tokens("q", q, T, None, k.dtype)
            hq = q.shape[1]
            if q_out is None:
                q_out = _empty(q, (T, hq, self.head_dim), q.dtype, stream)
            else:
                _check_output("q_out", q_out, T * hq * self.head_dim * 2, q.device, q.dtype)
            q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out needs q")
        st = self._lib.fq_kv_append(
            self._desc_ref, ctypes.byref(batch), T, _DT[k.dtype], k.data_ptr(), ks, v.data_ptr(), vs, freq,
            rot, 1 if interleaved else 0, q_ptr, qs, hq, out_ptr, self._status_ptr, _raw_stream(stream, self._device))
        if st != _lib.FQ_OK:
            _lib.check(st, "fq_kv_append")
        return q_out

    def attention(self, q, cu_new, seq_lens, page_table, max_q_len, max_seq_len=None, scale=None, causal=True,
                  out=None, lse=None, return_lse=False, stream=None):
        """softmax(scale q k^T) v over the cache for the new tokens' queries q [T, q_heads,
        head_dim] (see fq_kv_attention). max_q_len and max_seq_len bound the batch's new tokens
        and lengths (max_seq_len: the page table's capacity unless given); scale: head_dim ** -0.5
        unless given. Returns out, or (out, lse [T, q_heads] float32) with return_lse."""
        if not isinstance(q, torch.Tensor) or q.dtype not in _DT:
            raise ValueError("q must be a bfloat16 or float16 tensor")
        self._check_current()
        T = q.shape[0] if q.dim() else 0
        qs = self._tokens("q", q, T, None, q.dtype)
        hq, D = q.shape[1], self.head_dim
        batch = self._batch_desc(cu_new, seq_lens, page_table)
        max_q_len = int(max_q_len)  # (of a tensor its value: the sizes below are a key)
        max_seq_len = batch.table_width * self.page_size if max_seq_len is None else int(max_seq_len)
        if out is None:
            out = _empty(q, (T, hq, D), q.dtype, stream)
        else:
            _check_output("out", out, T * hq * D * 2, q.device, q.dtype)
        if lse is not None:
            _check_output("lse", lse, T * hq * 4, q.device, torch.float32)
        elif return_lse:
            lse = _empty(q, (T, hq), torch.float32, stream)
        sizes = (T, hq, batch.num_seqs, batch.table_width, max_q_len, max_seq_len)
        need = self._workspace_bytes.get(sizes)
        if need is None:
            n = ctypes.c_int64(0)
            _lib.check(self._lib.fq_kv_attention_workspace(self._desc_ref, ctypes.byref(batch), T, hq,
                                                           max_q_len, max_seq_len, ctypes.byref(n)),
                       "fq_kv_attention_workspace")
            if len(self._workspace_bytes) >= 4096:
                self._workspace_bytes.clear()
            need = self._workspace_bytes[sizes] = n.value
        ws = _empty(q, (need,), torch.uint8, stream) if need else None
        st = self._lib.fq_kv_attention(
            self._desc_ref, ctypes.byref(batch), T, _DT[q.dtype], q.data_ptr(), qs, hq, max_q_len,
            max_seq_len, float(scale if scale is not None else D ** -0.5), 1 if causal else 0, out.data_ptr(),
            lse.data_ptr() if lse is not None else None, ws.data_ptr() if ws is not None else None, need,
            self._status_ptr, _raw_stream(stream, self._device))
        if st != _lib.FQ_OK:
            _lib.check(st, "fq_kv_attention")
        return (out, lse) if return_lse else out


def debug_rotate(x, P1, P2, kernel="auto"):
    K, M, N = x.shape
    return FlatQuant(K, M, N, x.dtype, kernel).debug_rotate(x, P1, P2)


class HostPipeline:
    """End-to-end use from host memory. The tokens are processed in `chunks` equal slices:
    the host-to-device copy of slice c + 1, the operator on slice c and the device-to-host
    copy of slice c - 1 run on three streams at once (the copy engines work in both
    directions together), so a step costs about its larger transfer instead of the sum.
    Device buffers, streams and the per-slice handle are allocated once, in the
    constructor. With chunks = 1, or when K is not a multiple of `chunks`, everything runs
    on the caller's stream in one slice."""

    def __init__(self, fq: FlatQuant, mode, out_dtype="int4", device=None, chunks=8):
        self.fq = fq
        self.mode = mode
        self.out_dtype = out_dtype
        dev = device or torch.device("cuda", torch.cuda.current_device())
        K, M, N = fq.K, fq.M, fq.N
        self.x = torch.empty((K, M, N), dtype=fq.dtype, device=dev)
        self.P1 = torch.empty((M, M), dtype=fq.dtype, device=dev)
        self.P2 = torch.empty((N, N), dtype=fq.dtype, device=dev)
        if mode == "per_token":
            if out_dtype == "int8":
                self.out = torch.empty((K, M * N), dtype=torch.int8, device=dev)
            elif out_dtype == "int32":
                self.out = torch.empty((K, M, N // 8), dtype=torch.int32, device=dev)
            else:
                self.out = torch.empty((K, M * N // 2), dtype=torch.uint8, device=dev)
            self.scale = torch.empty((K,), dtype=torch.float32, device=dev)
        else:
            self.out = torch.empty((K, M * N // 2), dtype=torch.uint8, device=dev)
            self.scale = torch.empty((K, -(-M * N // 64), 2), dtype=torch.uint8, device=dev)
        self.chunks = chunks if chunks >= 1 and K % chunks == 0 else 1
        self.kc = K // self.chunks
        if self.chunks > 1:
            self.fq_c = FlatQuant(self.kc, M, N, fq.dtype, kernel=getattr(fq, "kernel", "auto"))
            self.s_in = torch.cuda.Stream(dev)
            self.s_out = torch.cuda.Stream(dev)

    def host_outputs(self):
        """Pinned host buffers shaped like the outputs."""
        return (torch.empty_like(self.out, device="cpu").pin_memory(),
                torch.empty_like(self.scale, device="cpu").pin_memory())

    def h2d_bytes(self):
        return sum(t.numel() * t.element_size() for t in (self.x, self.P1, self.P2))

    def d2h_bytes(self):
        return sum(t.numel() * t.element_size() for t in (self.out, self.scale))

    def _launch(self, fq, x, out, scale, clip_ratio, dst_type_max, s):
        if self.mode == "per_token":
            fq.quantize_per_token(x, self.P1, self.P2, clip_ratio, self.out_dtype,
                                  out=out, quant_scale=scale, stream=s)
        else:
            fq.quantize_mx(x, self.P1, self.P2, dst_type_max, out=out, scales=scale, stream=s)

    def run(self, x_host, P1_host, P2_host, out_host, scale_host, clip_ratio=1.0,
            dst_type_max=0.0, stream=None):
        s = stream if stream is not None else torch.cuda.current_stream()
        if self.chunks == 1:
            with torch.cuda.stream(s):
                self.x.copy_(x_host, non_blocking=True)
                self.P1.copy_(P1_host, non_blocking=True)
                self.P2.copy_(P2_host, non_blocking=True)
                self._launch(self.fq, self.x, self.out, self.scale, clip_ratio, dst_type_max, s)
                out_host.copy_(self.out, non_blocking=True)
                scale_host.copy_(self.scale, non_blocking=True)
            return out_host, scale_host
        # the side streams start after everything queued on the caller's stream so far
        # (the previous step included), and the caller's stream ends after the last copy out
        start = torch.cuda.Event()
        start.record(s)
        self.s_in.wait_event(start)
        self.s_out.wait_event(start)
        with torch.cuda.stream(self.s_in):
            self.P1.copy_(P1_host, non_blocking=True)
            self.P2.copy_(P2_host, non_blocking=True)
        for c in range(self.chunks):
            sl = slice(c * self.kc, (c + 1) * self.kc)
            with torch.cuda.stream(self.s_in):
                self.x[sl].copy_(x_host[sl], non_blocking=True)
                landed = torch.cuda.Event()
                landed.record(self.s_in)
            s.wait_event(landed)
            with torch.cuda.stream(s):
                self._launch(self.fq_c, self.x[sl], self.out[sl], self.scale[sl], clip_ratio,
                             dst_type_max, s)
                done = torch.cuda.Event()
                done.record(s)
            self.s_out.wait_event(done)
            with torch.cuda.stream(self.s_out):
                out_host[sl].copy_(self.out[sl], non_blocking=True)
                scale_host[sl].copy_(self.scale[sl], non_blocking=True)
        end = torch.cuda.Event()
        end.record(self.s_out)
        s.wait_event(end)
        return out_host, scale_host
