"""EntropyCache denoising step on GB300: Python binding of the C ABI (include/entropycache.h).

Argument marshalling only: every stage of the step runs in the library's CUDA kernels.
PyTorch supplies device memory and streams. The library must be built in-tree first
(`python -m entropy_gated_kv_gb300.build`); importing the binding does not build it and
nothing here falls back to a CPU implementation.

Stages (EntropyCache, gist.science zh summary §2.2):
  entropy_decode     (a) softmax + greedy decode + Shannon entropy per candidate row
  select_recompute   (b)+(c) commit, max-entropy gate vs tau, decode history, recompute set
  kv_scatter         (c) fresh K/V rows of the recompute set into the cache
  partial_attention  (d) bidirectional attention of the recompute rows over all L rows
  step               all of the above for one denoising step over n layers

The same stages over other caches: kv_scatter_quant / kv_gather_quant write and read a QuantCache
(8-bit rows), partial_attention_quant attends to it, prefix_attention attends to a prefix that
the batch shares and to each sequence's own cache.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from . import _capi as C
from ._capi import EcError  # noqa: F401

__all__ = [
    "Params",
    "DecodeState",
    "lib",
    "workspace",
    "entropy_decode",
    "entropy_decode_workspace_size",
    "entropy_decode_noalloc",
    "select_recompute",
    "candidates",
    "kv_scatter",
    "partial_attention",
    "partial_attention_workspace_size",
    "QuantCache",
    "kv_scatter_quant",
    "kv_gather_quant",
    "partial_attention_quant",
    "partial_attention_quant_workspace_size",
    "prefix_attention",
    "prefix_attention_workspace_size",
    "step",
    "step_workspace_size",
    "LayerWeights",
    "rope_table",
    "layer_forward",
    "layer_forward_workspace_size",
    "read_device_error",
    "EcError",
]


def lib() -> ctypes.CDLL:
    return C.load()


def _vp(t: torch.Tensor | None) -> ctypes.c_void_p | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("EntropyCache kernels take CUDA tensors (there is no CPU path)")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream: torch.cuda.Stream | None) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(d) -> int:
    if d in ("bf16", torch.bfloat16, C.EC_BF16):
        return C.EC_BF16
    if d in ("f32", torch.float32, C.EC_F32):
        return C.EC_F32
    raise ValueError(f"unsupported logits dtype {d!r}")


class _Kept:
    """Room for what Params keeps beside its fields: __dict__ holds the fields, and nothing else."""

    __slots__ = ("_kept",)


@dataclass
class Params(_Kept):
    """Step shape and knobs (ec_params)."""

    B: int
    L: int
    Hq: int
    Hkv: int
    D: int
    V: int
    C_max: int
    k: int
    n_dec: int = 1
    tau: float = 1.0
    logits_dtype: object = "bf16"
    conf_threshold: float = 0.0  # > 0: commit only candidates at least this confident (at least one)
    scope_lo: int = 0  # the gate's scope [scope_lo, scope_hi) for block-by-block decoding;
    scope_hi: int = 0  # both 0: the whole sequence

    def c(self) -> C.EcParams:
        return C.EcParams(self.B, self.L, self.Hq, self.Hkv, self.D, self.V, self.C_max, self.k, self.n_dec,
                          float(self.tau), _dtype_code(self.logits_dtype), float(self.conf_threshold),
                          int(self.scope_lo), int(self.scope_hi))

    def ref(self):
        """byref(c()), made once and again after a field has changed."""
        fields, kept = tuple(self.__dict__.values()), getattr(self, "_kept", None)
        if kept is None or kept[0] != fields:
            kept = self._kept = (fields, ctypes.byref(self.c()))
        return kept[1]

    def __getstate__(self):  # copies and pickles hold the fields only
        return dict(self.__dict__)


class DecodeState:
    """Per-sequence decode state (ec_state) as CUDA tensors."""

    FIELDS = ("tokens", "mask", "ring", "ring_head", "ring_count", "dec_pos", "E", "flag", "idx", "R", "dev_err")

    def __init__(self, p: Params, device="cuda"):
        B, L, k = p.B, p.L, p.k
        z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
        self.tokens = z(B, L)
        self.mask = z(B, L, dt=torch.uint8)
        self.ring = z(B, k)
        self.ring_head = z(B)
        self.ring_count = z(B)
        self.dec_pos = z(B, p.n_dec)
        self.E = z(B, dt=torch.float32)
        self.flag = z(B, dt=torch.uint8)
        self.idx = z(B, L)
        self.R = z(B)
        self.dev_err = z(1)

    @classmethod
    def from_arrays(cls, p: Params, device="cuda", **arrays) -> "DecodeState":
        st = cls(p, device)
        for name, a in arrays.items():
            getattr(st, name).copy_(torch.as_tensor(a).to(getattr(st, name).dtype))
        return st

    def c(self) -> C.EcState:
        return C.EcState(*[_vp(getattr(self, f)) for f in self.FIELDS])

    def clone(self) -> "DecodeState":
        other = object.__new__(DecodeState)
        for f in self.FIELDS:
            setattr(other, f, getattr(self, f).clone())
        return other


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Scratch buffer for an entry point's workspace (the library needs no initial contents)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def entropy_decode_workspace_size(n_rows: int, V: int, dtype) -> int:
    return int(lib().ec_entropy_decode_workspace_size(n_rows, V, _dtype_code(dtype)))


def entropy_decode(logits: torch.Tensor, V: int | None = None, ws: torch.Tensor | None = None,
                   out: tuple | None = None, stream=None):
    """(a) ids int32, entropy fp32, log_conf fp32 for each row of logits [n_rows, row_stride]."""
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [n_rows, row_stride] with unit inner stride")
    n, V = logits.shape[0], (V if V is not None else logits.shape[1])
    code = _dtype_code(logits.dtype)
    if out is None:
        out = (torch.empty(n, dtype=torch.int32, device=logits.device),
               torch.empty(n, dtype=torch.float32, device=logits.device),
               torch.empty(n, dtype=torch.float32, device=logits.device))
    if ws is None:
        ws = workspace(entropy_decode_workspace_size(n, V, code), logits.device)
    st = lib().ec_entropy_decode(_vp(logits), logits.stride(0), n, V, code, _vp(out[0]), _vp(out[1]), _vp(out[2]),
                                 _vp(ws), ws.numel(), _stream(stream))
    C.check(st, "ec_entropy_decode")
    return out


def entropy_decode_noalloc(logits: torch.Tensor, V: int | None = None, out: tuple | None = None, stream=None):
    """(a) like entropy_decode, but with no workspace: for callers that cannot allocate device
    memory. The scratch is a 1 MiB array owned by the library; calls that overlap on the GPU
    race, and the first call on a device must come before any stream capture."""
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [n_rows, row_stride] with unit inner stride")
    n, V = logits.shape[0], (V if V is not None else logits.shape[1])
    code = _dtype_code(logits.dtype)
    if out is None:
        out = (torch.empty(n, dtype=torch.int32, device=logits.device),
               torch.empty(n, dtype=torch.float32, device=logits.device),
               torch.empty(n, dtype=torch.float32, device=logits.device))
    st = lib().ec_entropy_decode_noalloc(_vp(logits), logits.stride(0), n, V, code, _vp(out[0]), _vp(out[1]),
                                         _vp(out[2]), _stream(stream))
    C.check(st, "ec_entropy_decode_noalloc")
    return out


def lm_head_entropy_workspace_size(n_rows: int) -> int:
    return int(lib().ec_lm_head_entropy_workspace_size(n_rows))


def lm_head_entropy(hidden: torch.Tensor, weight: torch.Tensor, ws: torch.Tensor | None = None,
                    out: tuple | None = None, stream=None):
    """(a) from the hidden states: ids, entropy, log_conf of logits = hidden @ weight.T, which
    are computed on the tensor cores and never stored. hidden [n_rows, d_model] and weight
    [V, d_model]: contiguous CUDA bf16."""
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise ValueError("hidden and weight must be bf16")
    if hidden.dim() != 2 or weight.dim() != 2 or hidden.shape[1] != weight.shape[1]:
        raise ValueError("hidden [n_rows, d_model] and weight [V, d_model]")
    if not (hidden.is_contiguous() and weight.is_contiguous()):
        raise ValueError("hidden and weight must be contiguous")
    n, d = hidden.shape
    V = weight.shape[0]
    if out is None:
        out = (torch.empty(n, dtype=torch.int32, device=hidden.device),
               torch.empty(n, dtype=torch.float32, device=hidden.device),
               torch.empty(n, dtype=torch.float32, device=hidden.device))
    if ws is None:
        ws = workspace(lm_head_entropy_workspace_size(n), hidden.device)
    st = lib().ec_lm_head_entropy(_vp(hidden), _vp(weight), n, d, V, _vp(out[0]), _vp(out[1]), _vp(out[2]), _vp(ws),
                                  ws.numel(), _stream(stream))
    C.check(st, "ec_lm_head_entropy")
    return out


def select_recompute(p: Params, state: DecodeState, cand_pos, cand_count, ids, entropy, log_conf, stream=None):
    """(b)+(c) commit, gate, history push and recompute set; updates `state` in place."""
    pc, sc = p.c(), state.c()
    st = lib().ec_select_recompute(ctypes.byref(pc), ctypes.byref(sc), _vp(cand_pos), _vp(cand_count), _vp(ids),
                                   _vp(entropy), _vp(log_conf), _stream(stream))
    C.check(st, "ec_select_recompute")


def candidates(p: Params, state: DecodeState, mode: str, start: int, width: int, cand_pos=None, cand_count=None,
               stream=None):
    """Candidates of a block-wise ("block") or sliding-window ("sliding") decoding step: the
    masked positions of the window, built on the device from state.mask. Returns
    (cand_pos int32 [B, C_max], cand_count int32 [B])."""
    code = {"block": C.EC_CAND_BLOCK, "sliding": C.EC_CAND_SLIDING}[mode]
    dev = state.mask.device
    if cand_pos is None:
        cand_pos = torch.empty(p.B, p.C_max, dtype=torch.int32, device=dev)
    if cand_count is None:
        cand_count = torch.empty(p.B, dtype=torch.int32, device=dev)
    pc, sc = p.c(), state.c()
    st = lib().ec_candidates(ctypes.byref(pc), ctypes.byref(sc), code, int(start), int(width), _vp(cand_pos),
                             _vp(cand_count), _stream(stream))
    C.check(st, "ec_candidates")
    return cand_pos, cand_count


def kv_scatter(p: Params, k_cache, v_cache, k_new, v_new, idx, R, src_by_position: bool = False,
               dev_err=None, stream=None):
    """(c) k_cache[b, idx[b, r]] = k_new[b, r or idx[b, r]] (same for v) for r < R[b]."""
    pc = p.c()
    st = lib().ec_kv_scatter(ctypes.byref(pc), _vp(k_cache), _vp(v_cache), _vp(k_new), _vp(v_new),
                             int(bool(src_by_position)), _vp(idx), _vp(R), _vp(dev_err), _stream(stream))
    C.check(st, "ec_kv_scatter")


def partial_attention_workspace_size(p: Params) -> int:
    pc = p.c()
    return int(lib().ec_partial_attention_workspace_size(ctypes.byref(pc)))


def partial_attention(p: Params, q, k_cache, v_cache, R, out, scale: float | None = None,
                      ws: torch.Tensor | None = None, dev_err=None, stream=None):
    """(d) out[b, r, h] = softmax(scale q k^T) v over all L keys, for r < R[b]."""
    pc = p.c()
    if ws is None:
        ws = workspace(partial_attention_workspace_size(p), q.device)
    sc = (1.0 / math.sqrt(p.D)) if scale is None else float(scale)
    st = lib().ec_partial_attention(ctypes.byref(pc), _vp(q), _vp(k_cache), _vp(v_cache), _vp(R), sc, _vp(out),
                                    _vp(ws), ws.numel(), _vp(dev_err), _stream(stream))
    C.check(st, "ec_partial_attention")
    return out


def dense_attention(p: Params, q, k_cache, v_cache, out, scale: float | None = None, dev_err=None, stream=None):
    """(d) for a step known to be full: out[b, r, h] = softmax(scale q k^T) v over all L keys for
    every position r (q in position order), two query tiles per CTA with a softmax warpgroup
    each; D = 128."""
    pc = p.c()
    sc = (1.0 / math.sqrt(p.D)) if scale is None else float(scale)
    st = lib().ec_dense_attention(ctypes.byref(pc), _vp(q), _vp(k_cache), _vp(v_cache), sc, _vp(out), _vp(dev_err),
                                  _stream(stream))
    C.check(st, "ec_dense_attention")
    return out


# ---- 8-bit caches and shared prefixes ------------------------------------------------------------


def _checked(t, name: str, dtype, shape: tuple, index: int) -> int:
    """Address of t, a contiguous tensor of that type and shape on CUDA device `index`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}: EntropyCache kernels take CUDA tensors, all of one device")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cuda_index(t, name: str) -> int:
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} is on {t.device}: EntropyCache kernels take CUDA tensors (there is no CPU path)")
    return i


class _Cache:
    """The checked C view (ec_kv) of an 8-bit cache."""

    __slots__ = ("c", "ref", "shape", "exp_shape", "index", "at")

    def __init__(self, k, v, k_exp, v_exp):
        self.shape, self.index = tuple(k.shape), _cuda_index(k, "k")
        if len(self.shape) != 4:
            raise ValueError(f"a cache is [B, L, Hkv, D], got {list(self.shape)}")
        kv = [_checked(t, n, torch.float8_e4m3fn, self.shape, self.index) for t, n in ((k, "k"), (v, "v"))]
        if k_exp is None or v_exp is None:
            raise ValueError("an 8-bit cache has exponent bytes k_exp and v_exp")
        B, L, H, _ = self.shape
        self.exp_shape = (B, H, -(-L // 16) * 16)
        ep = [_checked(e, n, torch.uint8, self.exp_shape, self.index) for e, n in ((k_exp, "k_exp"), (v_exp, "v_exp"))]
        self.at = (*kv, *ep)
        self.c = C.EcKv(C.EC_E4M3, L, *self.at)
        self.ref = ctypes.byref(self.c)

    def holds(self, k, v, k_exp, v_exp) -> bool:
        """Whether the view is still that of these tensors. Addresses alone do not tell: one that was
        resized, restrided or given other data in place may lie where it lay."""
        return (self.at == (k.data_ptr(), v.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr())
                and k.shape == self.shape and v.shape == self.shape
                and k_exp.shape == self.exp_shape and v_exp.shape == self.exp_shape
                and k.is_contiguous() and v.is_contiguous() and k_exp.is_contiguous() and v_exp.is_contiguous()
                and k.dtype is v.dtype is torch.float8_e4m3fn and k_exp.dtype is v_exp.dtype is torch.uint8)


class QuantCache:
    """One layer's K/V cache in 8 bits (ec_kv, EC_E4M3): k, v float8_e4m3fn [B, L, Hkv, D] and
    k_exp, v_exp uint8 [B, Hkv, S], S = L rounded up to a multiple of 16. The row of position j
    and head h stands for k[b, j, h] * 2^(k_exp[b, h, j] - 127). A tensor may be exchanged for another one or
    changed in place; every call checks what the cache holds then."""

    __slots__ = ("k", "v", "k_exp", "v_exp", "_c")

    def __init__(self, k, v, k_exp, v_exp):
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.view()

    def __setattr__(self, name, value):
        object.__setattr__(self, "_c", None)
        object.__setattr__(self, name, value)

    def view(self) -> _Cache:
        """The checked C view; made and checked again when a tensor is not what it was."""
        c, k, v, ke, ve = self._c, self.k, self.v, self.k_exp, self.v_exp
        if c is None or not c.holds(k, v, ke, ve):
            c = _Cache(k, v, ke, ve)
            object.__setattr__(self, "_c", c)
        return c

    @classmethod
    def empty(cls, B: int, L: int, Hkv: int, D: int, device="cuda") -> "QuantCache":
        """A cache of zero rows."""
        S = -(-L // 16) * 16
        z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=device)  # noqa: E731
        codes = [z(B, L, Hkv, D).view(torch.float8_e4m3fn) for _ in range(2)]
        return cls(*codes, *(z(B, Hkv, S).fill_(17) for _ in range(2)))


def _kv(cache, shape: tuple, index: int, what: str):
    """byref of the ec_kv of `cache`, a QuantCache or a pair of bf16 tensors, of that shape ([.., L, Hkv, D])."""
    if isinstance(cache, QuantCache):
        view = cache.view()
        _expect(view, shape, what)
        if view.index != index:
            raise ValueError(f"{what} is on cuda:{view.index}, the other tensors on cuda:{index}")
        return view.ref
    k, v = cache
    kp = _checked(k, what, torch.bfloat16, shape, index)
    return ctypes.byref(C.EcKv(C.EC_BF16, shape[-3], kp, _checked(v, what, torch.bfloat16, shape, index), None, None))


def _prefix_shape(prefix, p: Params) -> tuple:
    if isinstance(prefix, QuantCache):
        return (1, prefix.k.shape[1], p.Hkv, p.D)
    k = prefix[0]  # [Lp, Hkv, D], or one sequence of a batch's layout
    n = k.dim()
    if n != 3 and n != 4:
        raise ValueError(f"a prefix is [Lp, Hkv, D], got {list(k.shape)}")
    return (k.shape[0], p.Hkv, p.D) if n == 3 else (1, k.shape[1], p.Hkv, p.D)


def _launch(index: int, stream, call):
    """call(stream handle) with CUDA device `index` and the caller's `stream` (None: the device's
    current one) current, so that what the call allocates belongs to the stream it launches on."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if torch._C._cuda_getDevice() == index:
        return call(torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return call(torch._C._cuda_getCurrentRawStream(index))


def _opt(t, name, dtype, shape, index):
    return None if t is None else _checked(t, name, dtype, shape, index)


def _expect(view: _Cache, shape: tuple, what: str):
    if view.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(view.shape)}")


def kv_scatter_quant(p: Params, cache: QuantCache, k_new, v_new, idx, R, src_by_position: bool = False, dev_err=None,
                     stream=None):
    """(c) the refresh of an 8-bit cache: cache[b, idx[b, r]] = the row k_new[b, r or idx[b, r]],
    quantised (same for v), for r < R[b]. k_new, v_new bf16 [B, L, Hkv, D]; idx [B, L] (strictly
    ascending per sequence unless src_by_position) and R [B] int32. See ec_kv_scatter_quant."""
    view, shape = cache.view(), (p.B, p.L, p.Hkv, p.D)
    i = view.index
    _expect(view, shape, "cache")
    kp = _checked(k_new, "k_new", torch.bfloat16, shape, i)
    vp = _checked(v_new, "v_new", torch.bfloat16, shape, i)
    ip = _checked(idx, "idx", torch.int32, shape[:2], i)
    rp = _checked(R, "R", torch.int32, shape[:1], i)
    ep = _opt(dev_err, "dev_err", torch.int32, (1,), i)
    by_pos = 1 if src_by_position else 0
    f = lib().ec_kv_scatter_quant
    if stream is None and torch._C._cuda_getDevice() == i:
        st = f(p.ref(), view.ref, kp, vp, by_pos, ip, rp, ep, torch._C._cuda_getCurrentRawStream(i))
    else:
        st = _launch(i, stream, lambda s: f(p.ref(), view.ref, kp, vp, by_pos, ip, rp, ep, s))
    C.check(st, "ec_kv_scatter_quant")


def kv_gather_quant(p: Params, cache: QuantCache, idx, R, out: tuple | None = None, dev_err=None, stream=None):
    """Rows of an 8-bit cache back as bf16: (k, v) with k[b, r] = cache row idx[b, r] for r < R[b]
    (idx None: row r). out: two bf16 tensors [B, L, Hkv, D], by default new ones whose other rows
    are zeros. See ec_kv_gather_quant."""
    view, shape = cache.view(), (p.B, p.L, p.Hkv, p.D)
    i = view.index
    _expect(view, shape, "cache")
    ip = _opt(idx, "idx", torch.int32, shape[:2], i)
    rp = _checked(R, "R", torch.int32, shape[:1], i)
    ep = _opt(dev_err, "dev_err", torch.int32, (1,), i)

    def call(s):
        k, v = out if out is not None else (torch.zeros(shape, dtype=torch.bfloat16, device=R.device) for _ in range(2))
        kp = _checked(k, "out[0]", torch.bfloat16, shape, i)
        vp = _checked(v, "out[1]", torch.bfloat16, shape, i)
        C.check(lib().ec_kv_gather_quant(p.ref(), view.ref, ip, rp, kp, vp, ep, s), "ec_kv_gather_quant")
        return k, v

    return _launch(i, stream, call)


def partial_attention_quant_workspace_size(p: Params) -> int:
    return int(lib().ec_partial_attention_quant_workspace_size(p.ref()))


def prefix_attention_workspace_size(p: Params) -> int:
    return int(lib().ec_prefix_attention_workspace_size(p.ref()))


def _attend(p: Params, q, prefix, cache, R, out, kv_len, scale, ws, dev_err, stream):
    i, shape, own = q.get_device(), (p.B, p.L, p.Hq, p.D), (p.B, p.L, p.Hkv, p.D)
    if i < 0:
        _cuda_index(q, "q")
    what = "ec_partial_attention_quant" if prefix is None else "ec_prefix_attention"
    own_kv = _kv(cache, own, i, "cache")
    kv = (own_kv,) if prefix is None else (_kv(prefix, _prefix_shape(prefix, p), i, "prefix"), own_kv)
    qp = _checked(q, "q", torch.bfloat16, shape, i)
    op = _checked(out, "out", torch.bfloat16, shape, i)
    rp = _checked(R, "R", torch.int32, shape[:1], i)
    lp = _opt(kv_len, "kv_len", torch.int32, shape[:1], i)
    ep = _opt(dev_err, "dev_err", torch.int32, (1,), i)
    if ws is not None and (ws.get_device() != i or not ws.is_contiguous()):
        raise ValueError(f"ws must be a contiguous tensor on {q.device}")
    sc = (1.0 / math.sqrt(p.D)) if scale is None else float(scale)

    f = getattr(lib(), what)
    if ws is not None and stream is None and torch._C._cuda_getDevice() == i:
        st = f(p.ref(), qp, *kv, rp, lp, sc, op, ws.data_ptr(), ws.nbytes, ep, torch._C._cuda_getCurrentRawStream(i))
    else:
        def call(s):
            w = ws
            if w is None:
                size = int(getattr(lib(), what + "_workspace_size")(p.ref()))
                w = torch.empty(max(256, size), dtype=torch.uint8, device=q.device)
            return f(p.ref(), qp, *kv, rp, lp, sc, op, w.data_ptr(), w.nbytes, ep, s)

        st = _launch(i, stream, call)
    C.check(st, what)
    return out


def partial_attention_quant(p: Params, q, cache: QuantCache, R, out, kv_len=None, scale: float | None = None,
                            ws: torch.Tensor | None = None, dev_err=None, stream=None):
    """(d) against an 8-bit cache: out[b, r, h] = softmax(scale q k^T) v over the first kv_len[b]
    keys (None: the scope's), for r < R[b]; zeros without a key. q, out bf16 [B, L, Hq, D]; R,
    kv_len int32 [B]; scale > 0. See ec_partial_attention_quant."""
    if not isinstance(cache, QuantCache):
        raise ValueError("cache must be a QuantCache")
    return _attend(p, q, None, cache, R, out, kv_len, scale, ws, dev_err, stream)


def prefix_attention(p: Params, q, prefix, cache, R, out, kv_len=None, scale: float | None = None,
                     ws: torch.Tensor | None = None, dev_err=None, stream=None):
    """(d) for a batch behind one prefix: attention over the prefix's keys, which every sequence
    sees, and the first kv_len[b] keys of the sequence's own cache. prefix: (k, v) bf16
    [Lp, Hkv, D], or a QuantCache of one sequence; cache: (k, v) bf16 [B, L, Hkv, D], or a
    QuantCache. The rest as partial_attention_quant. See ec_prefix_attention."""
    return _attend(p, q, prefix, cache, R, out, kv_len, scale, ws, dev_err, stream)


@dataclass
class LayerWeights:
    """Weights of one LLaMA-style layer for layer_forward (ec_layer): CUDA bf16 tensors wq
    [Hq D, d], wk and wv [Hkv D, d], wo [d, Hq D], wg and wu [d_ff, d], wd [d, d_ff], gamma1 and
    gamma2 [d]; rope_cos and rope_sin fp32 [L, D / 2] (rope_table)."""

    wq: torch.Tensor
    wk: torch.Tensor
    wv: torch.Tensor
    wo: torch.Tensor
    wg: torch.Tensor
    wu: torch.Tensor
    wd: torch.Tensor
    gamma1: torch.Tensor
    gamma2: torch.Tensor
    rope_cos: torch.Tensor
    rope_sin: torch.Tensor
    eps: float = 1e-5

    @property
    def d_ff(self) -> int:
        return int(self.wg.shape[0])

    def c(self) -> C.EcLayer:
        return C.EcLayer(self.d_ff, float(self.eps), *[_vp(getattr(self, n)) for n in
                                                      ("wq", "wk", "wv", "wo", "wg", "wu", "wd", "gamma1", "gamma2",
                                                       "rope_cos", "rope_sin")])


def rope_table(L: int, D: int, theta: float, device="cuda", stream=None):
    """RoPE cos / sin tables fp32 [L, D / 2] of the angles pos * theta^(-2i / D), built on the
    device in double precision (ec_rope_table)."""
    cs = torch.empty(L, D // 2, dtype=torch.float32, device=device)
    sn = torch.empty(L, D // 2, dtype=torch.float32, device=device)
    st = lib().ec_rope_table(int(L), int(D), float(theta), _vp(cs), _vp(sn), _stream(stream))
    C.check(st, "ec_rope_table")
    return cs, sn


def layer_forward_workspace_size(p: Params, d_ff: int) -> int:
    pc = p.c()
    return int(lib().ec_layer_forward_workspace_size(ctypes.byref(pc), int(d_ff)))


def layer_forward(p: Params, w: LayerWeights, idx, R, x_src, k_cache, v_cache, y=None, ws=None, dev_err=None,
                  stream=None):
    """The partial (R < L) or full forward of one layer for the recompute rows idx[b, :R[b]]
    (ec_layer_forward): refreshes k_cache / v_cache at those positions and returns y [B, L, d]
    (rows in recompute order, the first R[b] written)."""
    B, L, d = x_src.shape
    if y is None:
        y = torch.empty(B, L, d, dtype=torch.bfloat16, device=x_src.device)
    if ws is None:
        ws = workspace(layer_forward_workspace_size(p, w.d_ff), x_src.device)
    pc, wc = p.c(), w.c()
    st = lib().ec_layer_forward(ctypes.byref(pc), ctypes.byref(wc), _vp(idx), _vp(R), _vp(x_src), _vp(k_cache),
                                _vp(v_cache), _vp(y), _vp(ws), ws.numel(), _vp(dev_err), _stream(stream))
    C.check(st, "ec_layer_forward")
    return y


def step_workspace_size(p: Params) -> int:
    pc = p.c()
    return int(lib().ec_step_workspace_size(ctypes.byref(pc)))


def _ptr_array(ts) -> ctypes.Array:
    arr = (ctypes.c_void_p * max(1, len(ts)))()
    for i, t in enumerate(ts):
        arr[i] = t.data_ptr()
    return arr


def step(p: Params, state: DecodeState, logits, cand_pos, cand_count, layers: list[dict],
         scale: float | None = None, ws: torch.Tensor | None = None, stream=None):
    """One denoising step: (a)(b)(c) once, then scatter + attention for each layer.

    layers: dicts with k_cache, v_cache, k_src, v_src, q_src and out (CUDA bf16 tensors).
    """
    pc, sc = p.c(), state.c()
    if ws is None:
        ws = workspace(step_workspace_size(p), logits.device)
    names = ("k_cache", "v_cache", "k_src", "v_src", "q_src", "out")
    arrs = [_ptr_array([lay[n] for lay in layers]) for n in names]
    sc_ = (1.0 / math.sqrt(p.D)) if scale is None else float(scale)
    st = lib().ec_step(ctypes.byref(pc), ctypes.byref(sc), _vp(logits), _vp(cand_pos), _vp(cand_count), len(layers),
                       *arrs, sc_, _vp(ws), ws.numel(), _stream(stream))
    C.check(st, "ec_step")


def read_floor(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> None:
    """A plain read of the whole buffer in the decode's launch shape (ec_read_floor): the floor
    for the decode's read of the same bytes. A measurement aid."""
    st = lib().ec_read_floor(_vp(buf), buf.numel() * buf.element_size(), _vp(sink), _stream(stream))
    C.check(st, "ec_read_floor")


def selftest_bounded_wait(dev_err: torch.Tensor, limit_ns: int, stream=None) -> None:
    """Runs the library's bounded wait on a barrier nothing completes; afterwards dev_err
    holds EC_DEVERR_TIMEOUT (read it with read_device_error)."""
    st = lib().ec_selftest_bounded_wait(_vp(dev_err), int(limit_ns), _stream(stream))
    C.check(st, "ec_selftest_bounded_wait")


def read_device_error(dev_err: torch.Tensor, stream=None) -> tuple[int, int]:
    """Synchronises the stream and returns (status, device error word)."""
    w = ctypes.c_int32(0)
    st = lib().ec_read_device_error(_vp(dev_err), ctypes.byref(w), _stream(stream))
    return int(st), int(w.value)
