"""Serving operators over a paged key/value cache (include/dg.h).

Argument checks and marshalling (in C++, csrc/dg_serving_py.cpp: the calls are
short); the work is in libdg.so.  Tensors may be views with any token and head
stride as long as the components of a head are contiguous.  Every call is
asynchronous on `stream` (default: the current stream of the tensors' device),
keeps the memory of what it was passed until it has run there,
allocates nothing but a workspace the caller did not bring, and can be captured
into a CUDA graph.  Nothing is recorded for a backward pass: tensors that
require a gradient are refused unless gradients are off.  The argument
objects note the addresses of their tensors, so they cannot be changed after
they were made; the tensors' contents may.  A tensor that got other memory or
another shape since (resized, moved, transposed in place) is refused.  A copy
notes its own tensors; copy.deepcopy copies the tensors too.  Errors that only
the device finds go to the call's status word, or to serving_status().

    cache = PagedKV(k_pages, v_pages)                   # [n_pages, Hkv, page, hd]
    batch = PagedBatch(cu_q, kv_lens, page_table)       # device int32
    paged_append(cache, batch, k, v, rope=rope, norm=norm, q=q, q_out=q)
    paged_attention(cache, batch, q, out)
"""
from __future__ import annotations

import ctypes
import math
import os

NATIVE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_serving.so")
_I32, _I64, _F, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class _Heads(ctypes.Structure):
    _fields_ = [("data", _P), ("token_stride", _I64), ("head_stride", _I64)]


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", _P), ("rot_dim", _I32), ("interleaved", _I32), ("amplitude", _F)]


class _HeadNorm(ctypes.Structure):
    _fields_ = [("enabled", _I32), ("eps", _F), ("q_gain", _P), ("k_gain", _P)]


class _PagedKV(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("dtype", _I32), ("n_pages", _I32), ("n_kv_heads", _I32), ("page_size", _I32),
                ("head_dim", _I32)]


class _PagedBatch(ctypes.Structure):
    _fields_ = [("n_seqs", _I32), ("n_tokens", _I32), ("cu_q", _P), ("kv_lens", _P), ("page_table", _P),
                ("table_stride", _I64), ("max_pages", _I32), ("prefix_pages", _P), ("prefix_len", _I32)]


def signatures():
    """ctypes signatures of the operators' entry points (see lib()); struct
    arguments go as addresses."""
    return {
        "dg_qk_norm_rope": ([_I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P], _I32),
        "dg_paged_append": ([_P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P], _I32),
        "dg_paged_attention_workspace": ([_I32, _I32, _I32, _I32], ctypes.c_size_t),
        "dg_paged_attention": ([_P, _P, _I32, _P, _F, _I32, _P, _P, _P, ctypes.c_size_t, _P, _P], _I32),
        "dg_serving_status": ([_P], _I32),
        "dg_test_paged_walk": ([_P, _P, _I32, _I32, _I32, _P, _P, _I32, _P], _I32),
    }


_NAMES = ("dg_qk_norm_rope", "dg_paged_append", "dg_paged_attention", "dg_paged_attention_workspace")
_bound = None


def _native():
    """The compiled side of this module (csrc/dg_serving_py.cpp), bound to libdg.so."""
    global _bound
    if _bound is None:
        import torch  # noqa: F401  (the module links against it)

        import block_text_diffusion_b200 as package
        L = package.lib()
        if not os.path.exists(NATIVE_PATH):
            raise RuntimeError(f"{NATIVE_PATH} is missing: build it with `python -m block_text_diffusion_b200.build`")
        from . import build
        if build.binding_built_for() != build.binding_key():
            raise RuntimeError(f"{NATIVE_PATH} was built for another torch or Python ({build.binding_built_for().strip()}): "
                               "build it with `python -m block_text_diffusion_b200.build`")
        from . import _serving
        _serving.bind(*[ctypes.cast(getattr(L, n), _P).value for n in _NAMES], package.DGError)
        _bound = _serving
    return _bound


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _tensor(t, name, dtype, dim, device=None, contiguous=False):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-D {dtype} tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _dtype_code(dtype):
    import torch
    _need(dtype in (torch.float32, torch.bfloat16), f"dtype must be float32 or bfloat16, got {dtype}")
    return 1 if dtype == torch.bfloat16 else 0


class _Fixed:
    """What a call reads was noted when the object was made, so nothing is reassigned later."""

    def __setattr__(self, name, value):
        if "_fixed" in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} is fixed: make another {type(self).__name__}")
        self.__dict__[name] = value

    def __reduce__(self):   # a copy notes the addresses of its own tensors
        return type(self), self._args


class Rope(_Fixed):
    """Position rotation: pair j of a head turns by position * inv_freq[j].

    inv_freq: float64 device tensor [rot_dim / 2] (see rope_frequencies); the
    first rot_dim components rotate, the rest pass.  interleaved False pairs
    (j, j + rot_dim / 2), True pairs (2j, 2j + 1).  amplitude multiplies the
    rotated components (long-context scalings use it)."""

    def __init__(self, inv_freq, interleaved=False, amplitude=1.0):
        import torch
        _tensor(inv_freq, "inv_freq", torch.float64, 1, contiguous=True)
        _need(inv_freq.is_cuda, "inv_freq must be on a GPU")
        self.inv_freq, self.index = inv_freq, inv_freq.get_device()
        self.rot_dim = 2 * inv_freq.numel()
        self._args = (inv_freq, interleaved, amplitude)
        self._c = _Rope(inv_freq.data_ptr(), self.rot_dim, int(bool(interleaved)), float(amplitude))
        self._at = ctypes.addressof(self._c)
        self._fixed = True


class HeadNorm(_Fixed):
    """RMSNorm of each head: x / sqrt(mean(x^2) + eps) * gain (gains [head_dim], None: ones)."""

    def __init__(self, eps=1e-6, q_gain=None, k_gain=None):
        _need(eps >= 0.0, "eps must not be negative")
        self.q_gain, self.k_gain = q_gain, k_gain
        self._args = (eps, q_gain, k_gain)
        self._c = _HeadNorm(1, float(eps), None if q_gain is None else q_gain.data_ptr(),
                            None if k_gain is None else k_gain.data_ptr())
        self._at = ctypes.addressof(self._c)
        self._fixed = True


def rope_frequencies(rot_dim, theta=10000.0, scaling="none", factor=1.0, original_len=None, beta_fast=32.0,
                     beta_slow=1.0):
    """(inv_freq, amplitude): radians per position of the rot_dim / 2 pairs, as
    a list of floats for torch.tensor(..., dtype=torch.float64), and the
    multiplier of the rotated components.

    scaling "none":   w_j = theta^(-2j / rot_dim).
    scaling "linear": w_j / factor (positions interpolated).
    scaling "ntk":    theta * factor^(rot_dim / (rot_dim - 2)): the slowest pair
                      stretches by `factor`, the fastest hardly at all.
    scaling "yarn":   (Peng et al. 2023) pairs that turn more than beta_fast
                      times over original_len stay, those below beta_slow turns
                      are interpolated, a ramp between; amplitude
                      0.1 ln(factor) + 1."""
    _need(rot_dim >= 2 and rot_dim % 2 == 0, "rot_dim must be even and positive")
    _need(theta > 0.0 and factor >= 1.0, "theta must be positive and factor at least 1")
    _need(scaling in ("none", "linear", "ntk", "yarn"), f"unknown scaling {scaling!r}")
    n = rot_dim // 2
    if scaling == "ntk":
        _need(rot_dim > 2, "ntk scaling needs rot_dim > 2")
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    w = [theta ** (-2.0 * j / rot_dim) for j in range(n)]
    if scaling == "linear":
        return [x / factor for x in w], 1.0
    if scaling != "yarn" or factor == 1.0:
        return w, 1.0
    _need(original_len is not None and original_len > 0, "yarn scaling needs original_len")
    _need(theta > 1.0 and beta_fast > beta_slow > 0.0, "yarn scaling needs theta > 1 and beta_fast > beta_slow > 0")

    def pair_of(turns):   # the (fractional) pair that makes this many turns over original_len
        return rot_dim * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))

    lo = max(math.floor(pair_of(beta_fast)), 0)
    hi = min(math.ceil(pair_of(beta_slow)), rot_dim - 1)
    out = []
    for j, x in enumerate(w):
        ramp = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)   # 0: as it is, 1: interpolated
        out.append(x * (1.0 - ramp) + x / factor * ramp)
    return out, 0.1 * math.log(factor) + 1.0


class PagedKV(_Fixed):
    """A paged cache: keys and values [n_pages, n_kv_heads, page_size, head_dim],
    contiguous, page_size a power of two from 16 to 256."""

    def __init__(self, k, v):
        import torch
        _need(isinstance(k, torch.Tensor) and k.is_cuda, "k must be a tensor on a GPU")
        code = _dtype_code(k.dtype)
        _tensor(k, "k", k.dtype, 4, contiguous=True)
        _tensor(v, "v", k.dtype, 4, k.device, contiguous=True)
        _need(k.shape == v.shape and k.numel() > 0, "k and v must have one shape, not empty")
        page = k.shape[2]
        _need(16 <= page <= 256 and page & (page - 1) == 0, "page_size must be a power of two from 16 to 256")
        self.k, self.v, self.dtype, self.device, self.index = k, v, k.dtype, k.device, k.get_device()
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self._args = (k, v)
        self._c = _PagedKV(k.data_ptr(), v.data_ptr(), code, self.n_pages, self.n_kv_heads, page, self.head_dim)
        self._at = ctypes.addressof(self._c)
        self._fixed = True

    @classmethod
    def empty(cls, n_pages, n_kv_heads, page_size, head_dim, dtype, device="cuda"):
        """A cache of uninitialised pages."""
        import torch
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device))


class PagedBatch(_Fixed):
    """A ragged batch over a paged cache: sequence b has the token rows
    cu_q[b] .. cu_q[b+1] - 1 as its newest tokens and kv_lens[b] tokens of its
    own in the cache, those included, in the pages page_table[b].  prefix_len
    tokens in prefix_pages come before every sequence.  All tensors int32 on
    the GPU, read there at each call (a captured call sees later contents)."""

    def __init__(self, cu_q, kv_lens, page_table, prefix_pages=None, prefix_len=0):
        import torch
        i32 = torch.int32
        _tensor(cu_q, "cu_q", i32, 1, contiguous=True)
        _need(cu_q.is_cuda and cu_q.numel() >= 1, "cu_q must be on a GPU, with one entry more than sequences")
        n = cu_q.numel() - 1
        _tensor(kv_lens, "kv_lens", i32, 1, cu_q.device, contiguous=True)
        _need(kv_lens.numel() == n, f"kv_lens must have {n} entries")
        _tensor(page_table, "page_table", i32, 2, cu_q.device)
        _need(page_table.shape[0] == n, f"page_table must have {n} rows")
        _need(page_table.stride(1) == 1 or page_table.shape[1] <= 1, "the entries of a page_table row must be contiguous")
        _need(n <= 1 or page_table.stride(0) >= page_table.shape[1], "page_table rows overlap")
        _need(0 <= prefix_len < 1 << 31, "prefix_len must lie in [0, 2^31)")
        _need(prefix_len == 0 or prefix_pages is not None, "prefix_len without prefix_pages")
        if prefix_pages is not None:
            _tensor(prefix_pages, "prefix_pages", i32, 1, cu_q.device, contiguous=True)
        self.cu_q, self.kv_lens, self.page_table, self.prefix_pages = cu_q, kv_lens, page_table, prefix_pages
        self.n_seqs, self.prefix_len, self.index = n, int(prefix_len), cu_q.get_device()
        # what dg_paged_batch needs, and the tensors it comes from (each call checks that they did not move)
        self._args = (cu_q, kv_lens, page_table, prefix_pages, prefix_len)
        self._words = (self.index, n, cu_q.data_ptr(), kv_lens.data_ptr(), page_table.data_ptr(),
                       max(page_table.stride(0), page_table.shape[1]), page_table.shape[1],
                       prefix_pages.data_ptr() if prefix_len else 0, int(prefix_len),
                       prefix_pages.numel() if prefix_len else 0, cu_q, kv_lens, page_table, prefix_pages)
        self._fixed = True


def qk_norm_rope(q, k, positions, q_out, k_out, rope=None, norm=None, stream=None):
    """RMSNorm of each query and key head and the position rotation, one pass.

    q [T, Hq, hd] -> q_out, k [T, Hkv, hd] -> k_out (a pair may be None;
    outputs may be the inputs), positions int32 [T] (None without rope)."""
    _native().qk_norm_rope(q, k, positions, q_out, k_out, rope, norm, stream)


def paged_append(cache, batch, k, v, rope=None, norm=None, q=None, q_out=None, status=None, stream=None):
    """The batch's new tokens into the cache's pages: k [T, Hkv, hd] normalised
    and rotated at its position, v as it is; with q [T, Hq, hd] the same tokens'
    queries, normalised and rotated, into q_out (which may be q).

    status: int32 [1] device tensor, zero before; becomes 5 (DG_ERR_STATE) if a
    token had no valid slot (it is not stored).  None: see serving_status."""
    _native().paged_append(cache, batch, k, v, rope, norm, q, q_out, status, stream)


def paged_attention_workspace(n_tokens, n_heads, head_dim, with_prefix=False):
    """Bytes of workspace paged_attention needs for that many token rows."""
    from . import DGError, lib
    # (ctypes would take what does not fit an int32 modulo 2^32)
    fits = all(0 <= x < 1 << 31 for x in (n_tokens, n_heads, head_dim))
    n = int(lib().dg_paged_attention_workspace(n_tokens, n_heads, head_dim, int(bool(with_prefix)))) if fits else 0
    if n == 0:
        raise DGError(1, "dg_paged_attention_workspace")
    return n


def paged_attention(cache, batch, q, out, scale=None, causal=True, lse=None, workspace=None, status=None,
                    stream=None):
    """Attention of q [T, Hq, hd] over the cache into out (which may be q).

    Every query sees the batch's whole prefix and its sequence's own tokens: all
    of them, or (causal) those up to its own.  scale defaults to 1 / sqrt(hd).
    lse: float32 [T, Hq], receives ln(sum(exp(scores))).  A query that sees no
    key gets zeros and -inf.  workspace: uint8 tensor of at least
    paged_attention_workspace(...) bytes (None: allocated for the call); two
    calls that may overlap need two.  status: int32 [1], zero before; becomes 5
    (DG_ERR_STATE) if a page id or length was out of range, 4 (DG_ERR_TIMEOUT) if
    a wait ran out.  None: see serving_status."""
    call = _native().paged_attention
    if workspace is None:
        import torch

        from . import DGError
        n = call(cache, batch, q, out, scale, causal, lse, None, status, stream)
        if n == 0:
            raise DGError(1, "dg_paged_attention_workspace")
        if stream is not None and stream.device != cache.device:
            raise ValueError(f"stream must be one of {cache.device}")
        # allocated on the call's stream: freed, the memory goes back to that stream's pool
        with torch.cuda.stream(torch.cuda.current_stream(cache.device) if stream is None else stream):
            workspace = torch.empty(n, dtype=torch.uint8, device=cache.device)
    call(cache, batch, q, out, scale, causal, lse, workspace, status, stream)


def serving_status(stream=None):
    """Waits for `stream` (default: the current one) and raises DGError for the
    first error that calls without a status tensor met on its device since this
    was last asked (a token without a slot, a page id or length out of range, a
    wait that ran out).  The outputs of such a call are not to be used."""
    import torch

    from . import _check, _stream, lib
    with torch.cuda.device(torch.cuda.current_device() if stream is None else stream.device):
        _check(lib().dg_serving_status(_stream(stream)), "device status")
