"""w12_weight_streaming_amd -- lossless 12-bit weight streaming for the
verification pass of greedy speculative decoding on MI355X (gfx950).

Thin ctypes binding over libw12.so (C ABI in include/w12.h), with the same
names as the C entry points: w12_pack, w12_decode, w12_check, w12_gemm,
w12_head_argmax, tree_accept, and for the pass's KV cache and sampling
requests w12_kv_append, w12_kv_attention, w12_kv_commit and
tree_accept_sampled; for its recurrent layers w12_delta_append,
w12_delta_rule and w12_delta_commit, and w12_norm between products. Every
step of the path runs in the library's HIP kernels; this module only checks
tensor dtypes/devices, passes device pointers and the current HIP stream, and
keeps zero-filled workspaces.
There is no CPU fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
import weakref
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw12.so")

W12_OK, W12_EINVAL, W12_ENOSPC, W12_EHIP, W12_ECORRUPT = 0, -1, -2, -3, -4
W12_Y_F32, W12_Y_BF16 = 0, 1
W12_KV_E4M3, W12_KV_INT8 = 0, 1
MFMA_MIN_ROWS = 5  # rows from which w12_gemm multiplies on the matrix cores (fewer: VALU path)
MAX_ROWS = 512

_lib = None


class W12Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().w12_strerror(status).decode()}")


class W12Matrix(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("records", ctypes.c_void_p), ("e_top", ctypes.c_void_p),
                ("esc_off", ctypes.c_void_p), ("esc", ctypes.c_void_p)]


class W12Cert8(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("qexp", ctypes.c_void_p), ("cbound", ctypes.c_void_p)]


class W12KvCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("kvtype", "layers", "num_pages", "kv_heads", "page_tokens", "head_dim",
                                              "slots", "recent_rows", "max_pages")] + \
               [(n, ctypes.c_void_p) for n in ("pages", "scales", "recent", "page_table", "len")]


class W12DeltaCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("layers", "slots", "step_rows", "key_heads", "value_heads", "key_dim",
                                              "value_dim", "conv_width")] + \
               [(n, ctypes.c_void_p) for n in ("state", "conv", "raw", "kv", "gates", "delta")]


def lib() -> ctypes.CDLL:
    """The loaded libw12.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m w12_weight_streaming_amd.build`"
                " (hipcc, gfx950). There is no fallback path.")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        mp = ctypes.POINTER(W12Matrix)
        kp = ctypes.POINTER(W12KvCache)
        dp = ctypes.POINTER(W12DeltaCache)
        sig = {
            "w12_strerror": (ctypes.c_char_p, [ctypes.c_int]),
            "w12_abi_version": (ctypes.c_int, []),
            "w12_num_blocks": (i64, [i64, i64]),
            "w12_pack_plan": (ctypes.c_int, [vp, i64, i64, vp, vp, vp]),
            "w12_pack": (ctypes.c_int, [vp, i64, i64, vp, vp, vp, vp, i64, vp]),
            "w12_decode": (ctypes.c_int, [mp, vp, vp]),
            "w12_check": (ctypes.c_int, [mp, vp, vp, vp]),
            "w12_gemm_workspace": (ctypes.c_int, [i64, i64, i64, ctypes.POINTER(sz)]),
            "w12_gemm": (ctypes.c_int, [mp, vp, i64, vp, ctypes.c_int, vp, sz, vp]),
            "w12_head_argmax_workspace": (ctypes.c_int, [i64, i64, i64, ctypes.POINTER(sz)]),
            "w12_head_argmax": (ctypes.c_int, [mp, vp, i64, vp, vp, vp, sz, vp]),
            "w12_gemm_qpass": (ctypes.c_int, [mp, vp, i64, vp, ctypes.c_int, vp, sz, vp]),
            "w12_gemm_noalloc": (ctypes.c_int, [mp, vp, i64, vp, ctypes.c_int, vp]),
            "w12_cert8_pack": (ctypes.c_int, [vp, i64, i64, vp, vp, vp, vp, vp]),
            "w12_head_argmax_certified_workspace": (ctypes.c_int, [i64, i64, i64, ctypes.POINTER(sz)]),
            "w12_head_argmax_certified": (ctypes.c_int, [mp, ctypes.POINTER(W12Cert8), vp, i64, vp, vp, vp, vp,
                                                         sz, vp]),
            "w12_head_argmax_qpass": (ctypes.c_int, [mp, vp, i64, vp, vp, vp, sz, vp]),
            "tree_accept": (ctypes.c_int, [i32, vp, i32, vp, vp, vp, vp, vp, vp, vp]),
            "w12_tree_build_workspace": (ctypes.c_int, [i32, i32, ctypes.POINTER(sz)]),
            "w12_tree_build": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, i32, vp, sz, vp, vp, vp, vp,
                                              vp, vp]),
            "w12_kv_append": (ctypes.c_int, [kp, i32, i32, vp, vp, i32, vp, vp, ctypes.c_int, i32, vp, i32, i32, i32,
                                             vp, vp]),
            "w12_kv_attention_workspace": (ctypes.c_int, [kp, i32, i32, i32, ctypes.POINTER(sz)]),
            "w12_kv_attention": (ctypes.c_int, [kp, i32, i32, vp, vp, i32, vp, vp, i32, ctypes.c_float, vp, vp, sz,
                                                vp]),
            "w12_kv_commit": (ctypes.c_int, [kp, i32, vp, vp, i32, vp, vp, vp, vp]),
            "tree_accept_sampled_workspace": (ctypes.c_int, [i32, i32, i32, ctypes.POINTER(sz)]),
            "tree_accept_sampled": (ctypes.c_int, [i32, vp, i32, vp, vp, vp, ctypes.c_int, i32, vp, vp, vp, vp, vp, vp,
                                                   vp, vp, sz, vp]),
            "w12_delta_append": (ctypes.c_int, [dp, i32, i32, vp, vp, i32, vp, vp, i64, vp, i64, ctypes.c_int, vp, vp, vp,
                                                vp, vp, vp]),
            "w12_delta_rule": (ctypes.c_int, [dp, i32, i32, vp, vp, i32, vp, vp, ctypes.c_float, i32, vp, vp]),
            "w12_delta_commit": (ctypes.c_int, [dp, i32, vp, vp, i32, vp, vp, vp, vp]),
            "w12_norm": (ctypes.c_int, [i64, i32, i32, vp, ctypes.c_int, i64, vp, vp, ctypes.c_int, i64, ctypes.c_float,
                                        vp, ctypes.c_int, vp, ctypes.c_float, vp, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return ["w12_strerror", "w12_abi_version", "w12_num_blocks", "w12_pack_plan", "w12_pack",
            "w12_decode", "w12_check", "w12_gemm_workspace", "w12_gemm",
            "w12_head_argmax_workspace", "w12_head_argmax", "w12_gemm_qpass",
            "w12_head_argmax_qpass", "tree_accept", "w12_tree_build_workspace", "w12_tree_build",
            "w12_gemm_noalloc", "w12_cert8_pack", "w12_head_argmax_certified_workspace",
            "w12_head_argmax_certified", "w12_kv_append", "w12_kv_attention_workspace",
            "w12_kv_attention", "w12_kv_commit", "tree_accept_sampled_workspace",
            "tree_accept_sampled", "w12_delta_append", "w12_delta_rule", "w12_delta_commit", "w12_norm"]


def _ok(status: int, what: str):
    if status != W12_OK:
        raise W12Error(status, what)


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t: torch.Tensor, dtype, name: str, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {t.dim()})")


@dataclass
class PackedW12:
    """Device-resident W12 matrix: the five buffers of include/w12.h."""
    n: int
    k: int
    records: torch.Tensor   # uint8 [n*k*3/2]
    e_top: torch.Tensor     # uint8 [n]
    esc_off: torch.Tensor   # int32 view of u32 [n*k/1024 + 1]
    esc: torch.Tensor       # int32 view of u32 [n_esc] (at least 1 element)
    n_esc: int

    def desc(self) -> W12Matrix:
        return W12Matrix(self.n, self.k, self.records.data_ptr(), self.e_top.data_ptr(),
                         self.esc_off.data_ptr(), self.esc.data_ptr())

    @property
    def device(self):
        return self.records.device

    def nbytes(self) -> int:
        """Packed bytes: records + e_top + esc_off + escape entries."""
        return (self.records.numel() + self.e_top.numel() + 4 * self.esc_off.numel()
                + 4 * self.n_esc)


# ------------------------------------------------------------------ workspaces

_ws_kept = threading.local()  # .cache: this host thread's workspaces
_zero_filled = weakref.WeakValueDictionary()  # address -> workspace that the products and heads expect zero-filled


def workspace(nbytes: int, device: torch.device, tag: str = "gemm") -> torch.Tensor:
    """Zero-filled device workspace of the products and heads, grown on demand
    and kept per (host thread, device, stream, tag): a call of theirs may be
    several launches, and another thread's on the same stream may come between
    them. Those calls leave it zero-filled; w12_kv_attention and
    tree_accept_sampled would not, and refuse it."""
    cache = _ws_kept.__dict__.setdefault("cache", {})
    key = (device.index, torch.cuda.current_stream(device).cuda_stream, tag)
    ws = cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = cache[key] = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        if tag in ("gemm", "head", "cert"):  # what the calls without ws= take
            _zero_filled[ws.data_ptr()] = ws
    return ws


# ------------------------------------------------------------------ entry points

def w12_pack(w: torch.Tensor, check: bool = True) -> PackedW12:
    """Pack bf16 weights [n, k] (on the GPU) into W12; with check=True run the
    load-time bit-for-bit check and raise if any weight fails to restore."""
    _need(w, torch.bfloat16, "w", 2)
    n, k = w.shape
    dev = w.device
    s = _stream(dev)
    L = lib()
    nb = L.w12_num_blocks(n, k)
    if nb < 0:
        raise W12Error(W12_EINVAL, f"w12_pack: shape {n}x{k}")
    e_top = torch.empty(n, dtype=torch.uint8, device=dev)
    esc_off = torch.empty(nb + 1, dtype=torch.int32, device=dev)
    _ok(L.w12_pack_plan(_ptr(w), n, k, _ptr(e_top), _ptr(esc_off), s), "w12_pack_plan")
    n_esc = int(esc_off[-1].item()) & 0xFFFFFFFF
    records = torch.empty(n * k * 3 // 2, dtype=torch.uint8, device=dev)
    esc = torch.empty(max(n_esc, 1), dtype=torch.int32, device=dev)
    _ok(L.w12_pack(_ptr(w), n, k, _ptr(e_top), _ptr(esc_off), _ptr(records), _ptr(esc),
                   n_esc, s), "w12_pack")
    pw = PackedW12(n, k, records, e_top, esc_off, esc, n_esc)
    if check:
        bad = w12_check(pw, w)
        if bad:
            raise W12Error(W12_ECORRUPT, f"w12_pack load-time check: {bad} weights differ")
    return pw


def w12_require_exact(pw: PackedW12, ref: torch.Tensor) -> None:
    """The load-time refusal: raise W12Error(W12_ECORRUPT) unless every
    weight of pw restores bit-for-bit to ref."""
    bad = w12_check(pw, ref)
    if bad:
        raise W12Error(W12_ECORRUPT, f"w12_check: {bad} weights differ")


def w12_decode(pw: PackedW12) -> torch.Tensor:
    out = torch.empty(pw.n, pw.k, dtype=torch.bfloat16, device=pw.device)
    d = pw.desc()
    _ok(lib().w12_decode(ctypes.byref(d), _ptr(out), _stream(pw.device)), "w12_decode")
    return out


def w12_check(pw: PackedW12, ref: torch.Tensor) -> int:
    """Number of weights whose restore differs from ref (0 = bit-exact)."""
    _need(ref, torch.bfloat16, "ref", 2)
    if tuple(ref.shape) != (pw.n, pw.k):
        raise ValueError("ref shape does not match the packed matrix")
    cnt = torch.zeros(1, dtype=torch.int64, device=pw.device)
    d = pw.desc()
    _ok(lib().w12_check(ctypes.byref(d), _ptr(ref), _ptr(cnt), _stream(pw.device)), "w12_check")
    return int(cnt.item())


def gemm_workspace_bytes(n: int, k: int, m: int) -> int:
    out = ctypes.c_size_t(0)
    _ok(lib().w12_gemm_workspace(n, k, m, ctypes.byref(out)), "w12_gemm_workspace")
    return out.value


def w12_gemm(pw: PackedW12, x: torch.Tensor, out: torch.Tensor | None = None,
             out_dtype=torch.float32, ws: torch.Tensor | None = None,
             qpass: bool = False) -> torch.Tensor:
    """y[m, n] = x[m, :] . W[n, :] with W streamed from W12 (fp32 accumulate).
    qpass=True runs w12_gemm_qpass (8-bit view, midpoint low nibbles)."""
    _need(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    if k != pw.k:
        raise ValueError(f"x has k={k}, matrix has k={pw.k}")
    if out is None:
        out = torch.empty(m, pw.n, dtype=out_dtype, device=x.device)
    if out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (m, pw.n):
        raise ValueError("out must be [m, n] float32 or bfloat16")
    _need(out, out.dtype, "out", 2)
    yt = W12_Y_F32 if out.dtype == torch.float32 else W12_Y_BF16
    need = gemm_workspace_bytes(pw.n, pw.k, m)
    if ws is None:
        ws = workspace(need, x.device)
    d = pw.desc()
    fn, name = (lib().w12_gemm_qpass, "w12_gemm_qpass") if qpass else (lib().w12_gemm, "w12_gemm")
    _ok(fn(ctypes.byref(d), _ptr(x), m, _ptr(out), yt, _ptr(ws), ws.numel(), _stream(x.device)), name)
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20


def w12_gemm_noalloc(pw: PackedW12, x: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """w12_gemm with the library's own static scratch as workspace: no
    device allocation in the call (out is the caller's). Calls that overlap
    on one device race."""
    _need(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    if k != pw.k:
        raise ValueError(f"x has k={k}, matrix has k={pw.k}")
    if out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (m, pw.n):
        raise ValueError("out must be [m, n] float32 or bfloat16")
    _need(out, out.dtype, "out", 2)
    yt = W12_Y_F32 if out.dtype == torch.float32 else W12_Y_BF16
    d = pw.desc()
    _ok(lib().w12_gemm_noalloc(ctypes.byref(d), _ptr(x), m, _ptr(out), yt, _stream(x.device)),
        "w12_gemm_noalloc")
    return out


def w12_head_argmax(pw: PackedW12, x: torch.Tensor, ws: torch.Tensor | None = None,
                    with_max: bool = True, qpass: bool = False):
    """Greedy token per row: (idx int32 [m], max logit float32 [m] or None).
    qpass=True runs w12_head_argmax_qpass (8-bit view, midpoint low nibbles)."""
    _need(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    if k != pw.k:
        raise ValueError(f"x has k={k}, head has k={pw.k}")
    idx = torch.empty(m, dtype=torch.int32, device=x.device)
    mx = torch.empty(m, dtype=torch.float32, device=x.device) if with_max else None
    need = ctypes.c_size_t(0)
    _ok(lib().w12_head_argmax_workspace(pw.n, pw.k, m, ctypes.byref(need)),
        "w12_head_argmax_workspace")
    if ws is None:
        ws = workspace(need.value, x.device, "head")
    d = pw.desc()
    fn, name = ((lib().w12_head_argmax_qpass, "w12_head_argmax_qpass") if qpass
                else (lib().w12_head_argmax, "w12_head_argmax"))
    _ok(fn(ctypes.byref(d), _ptr(x), m, _ptr(idx), _ptr(mx), _ptr(ws), ws.numel(),
           _stream(x.device)), name)
    return idx, mx


@dataclass
class Cert8Head:
    """Device-resident INT8 copy of an LM head for the certified argmax."""
    n: int
    k: int
    q: torch.Tensor        # int8 [n*k], 8 KB records
    qexp: torch.Tensor     # uint8 [n*k/32] block scale codes
    cbound: torch.Tensor   # float32 [n] per-row bound constants

    def desc(self) -> W12Cert8:
        return W12Cert8(self.n, self.k, self.q.data_ptr(), self.qexp.data_ptr(), self.cbound.data_ptr())

    def nbytes(self) -> int:
        return self.q.numel() + self.qexp.numel() + 4 * self.cbound.numel()


def w12_cert8_pack(w: torch.Tensor, pw: PackedW12) -> Cert8Head:
    """INT8 copy of the bf16 head w [n, k], using the window tops of its
    W12 pack pw (the weights W12 escapes are left to its escape list)."""
    _need(w, torch.bfloat16, "w", 2)
    n, k = w.shape
    if (n, k) != (pw.n, pw.k):
        raise ValueError("w and its W12 pack differ in shape")
    dev = w.device
    q = torch.empty(n * k, dtype=torch.int8, device=dev)
    qexp = torch.empty(n * k // 32, dtype=torch.uint8, device=dev)
    cb = torch.empty(n, dtype=torch.float32, device=dev)
    _ok(lib().w12_cert8_pack(_ptr(w), n, k, _ptr(pw.e_top), _ptr(q), _ptr(qexp), _ptr(cb), _stream(dev)),
        "w12_cert8_pack")
    return Cert8Head(n, k, q, qexp, cb)


def w12_head_argmax_certified(pw: PackedW12, cert: Cert8Head, x: torch.Tensor, ws: torch.Tensor | None = None,
                              with_max: bool = True):
    """Certified head argmax of 1 <= m <= 64 rows: (idx int32 [m], max
    logit float32 [m] or None, rescored vocabulary rows int32 [m])."""
    _need(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    if k != pw.k or (cert.n, cert.k) != (pw.n, pw.k):
        raise ValueError("x, the head and its INT8 copy must agree in shape")
    dev = x.device
    idx = torch.empty(m, dtype=torch.int32, device=dev)
    mx = torch.empty(m, dtype=torch.float32, device=dev) if with_max else None
    cnt = torch.empty(m, dtype=torch.int32, device=dev)
    need = ctypes.c_size_t(0)
    _ok(lib().w12_head_argmax_certified_workspace(pw.n, pw.k, m, ctypes.byref(need)),
        "w12_head_argmax_certified_workspace")
    if ws is None:
        ws = workspace(need.value, dev, "cert")
    d, c = pw.desc(), cert.desc()
    _ok(lib().w12_head_argmax_certified(ctypes.byref(d), ctypes.byref(c), _ptr(x), m, _ptr(idx), _ptr(mx),
                                        _ptr(cnt), _ptr(ws), ws.numel(), _stream(dev)),
        "w12_head_argmax_certified")
    return idx, mx, cnt


def tree_accept(node_off: torch.Tensor, parent: torch.Tensor, token: torch.Tensor,
                argmax: torch.Tensor):
    """Greedy tree acceptance; returns (accept_len [T], path [sum n], bonus [T])."""
    for t, nm in ((node_off, "node_off"), (parent, "parent"), (token, "token"),
                  (argmax, "argmax")):
        _need(t, torch.int32, nm, 1)
    T = node_off.numel() - 1
    total = parent.numel()
    if T < 0 or token.numel() != total or argmax.numel() != total:
        raise ValueError("tree_accept: inconsistent array sizes")
    dev = parent.device
    acc = torch.empty(max(T, 0), dtype=torch.int32, device=dev)
    path = torch.empty(total, dtype=torch.int32, device=dev)
    bonus = torch.empty(max(T, 0), dtype=torch.int32, device=dev)
    _ok(lib().tree_accept(T, _ptr(node_off), total, _ptr(parent), _ptr(token), _ptr(argmax),
                          _ptr(acc), _ptr(path), _ptr(bonus), _stream(dev)), "tree_accept")
    return acc, path, bonus


def w12_tree_build(lp: torch.Tensor, tok: torch.Tensor, depth: torch.Tensor, root: torch.Tensor,
                   budget: int, ws: torch.Tensor | None = None):
    """Best-first draft trees of R requests under one shared row budget.

    lp [R, D, K, K] fp32 edge scores, tok [R, D, K] int32, depth [R] int32,
    root [R] int32 (device tensors). Returns (node_off [R+1], parent, token,
    node_depth, score), the row arrays trimmed to node_off[R] rows."""
    _need(lp, torch.float32, "lp", 4)
    _need(tok, torch.int32, "tok", 3)
    _need(depth, torch.int32, "depth", 1)
    _need(root, torch.int32, "root", 1)
    R, D, K, K2 = lp.shape
    if K2 != K or tuple(tok.shape) != (R, D, K) or depth.numel() != R or root.numel() != R:
        raise ValueError("w12_tree_build: inconsistent shapes")
    dev = lp.device
    need = ctypes.c_size_t(0)
    _ok(lib().w12_tree_build_workspace(R, budget, ctypes.byref(need)), "w12_tree_build_workspace")
    if ws is None:
        ws = torch.empty(max(int(need.value), 16), dtype=torch.uint8, device=dev)
    node_off = torch.empty(R + 1, dtype=torch.int32, device=dev)
    parent = torch.empty(budget, dtype=torch.int32, device=dev)
    token = torch.empty(budget, dtype=torch.int32, device=dev)
    ndepth = torch.empty(budget, dtype=torch.int32, device=dev)
    score = torch.empty(budget, dtype=torch.float32, device=dev)
    _ok(lib().w12_tree_build(R, D, K, _ptr(lp), _ptr(tok), _ptr(depth), _ptr(root), budget, _ptr(ws),
                             ws.numel(), _ptr(node_off), _ptr(parent), _ptr(token), _ptr(ndepth),
                             _ptr(score), _stream(dev)), "w12_tree_build")
    n = int(node_off[-1].item())
    return node_off, parent[:n], token[:n], ndepth[:n], score[:n]


# ------------------------------------------------------------------ KV cache of the verify pass

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _get(t, dtype, name: str, ndim: int | None, index: int | None, entries: int | None = None) -> int:
    """Checks a tensor argument (on GPU `index`, if given, with that many
    entries, if given) and returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous() and (ndim is None or t.dim() == ndim)
            and t.get_device() >= 0):
        _need(t, dtype, name, ndim)
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index} (got {t.device})")
    if entries is not None and t.numel() != entries:
        raise ValueError(f"{name} must have {entries} entries (got {t.numel()})")
    return t.data_ptr()


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # a tensor on a GPU has made it ready


def _run(index: int, what: str, *args) -> None:
    """Calls an entry point with the current stream of GPU `index`, that GPU
    being the current one meanwhile."""
    fn = getattr(_lib or lib(), what)
    if _device_now() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != W12_OK:
        raise W12Error(status, what)


def _scratch(ws, index: int) -> tuple[int, int]:
    """Address and bytes of a workspace whose content is ignored and left as
    it comes: never one that a later product takes for zero-filled."""
    at = _get(ws, getattr(ws, "dtype", None), "ws", None, index)
    if ws.untyped_storage().data_ptr() in _zero_filled:
        raise ValueError("ws is a zero-filled workspace of the products or heads, which this call would leave dirty")
    return at, ws.numel() * ws.element_size()


@dataclass(frozen=True, eq=False)  # the description holds the arrays' addresses
class KvCache:
    """Device-resident KV cache: the arrays of include/w12.h. pages is
    [layers, num_pages, kv_heads, 2, page_tokens * head_dim] float8_e4m3fn or
    int8, scales its fp32 [layers, num_pages, kv_heads, 2], recent
    [layers, slots, kv_heads, 2, recent_rows * head_dim] bfloat16, page_table
    [slots, max_pages] int32, length [slots] int32. The arrays stay the same;
    their contents may be written at any time (a new sequence: its row of the
    page table, its length 0)."""
    pages: torch.Tensor
    scales: torch.Tensor
    recent: torch.Tensor
    page_table: torch.Tensor
    length: torch.Tensor
    head_dim: int

    def __post_init__(self):
        if not isinstance(self.pages, torch.Tensor) or self.pages.dtype not in (torch.float8_e4m3fn, torch.int8):
            raise TypeError("pages must be a float8_e4m3fn or int8 tensor")
        pages, scales, recent, table, length, dim = (self.pages, self.scales, self.recent, self.page_table, self.length,
                                                     self.head_dim)
        at = _get(pages, pages.dtype, "pages", 5, None)
        index = pages.get_device()
        ats = (at, _get(scales, _F32, "scales", 4, index), _get(recent, _BF16, "recent", 5, index),
               _get(table, _I32, "page_table", 2, index), _get(length, _I32, "length", 1, index))
        layers, num_pages, kv, two, page = pages.shape
        slots, blocks = table.shape
        rows = recent.shape
        if (two != 2 or dim < 1 or page % dim or scales.shape != (layers, num_pages, kv, 2) or length.shape[0] != slots
                or rows[0] != layers or rows[1] != slots or rows[2] != kv or rows[3] != 2 or rows[4] % dim):
            raise ValueError("the cache's arrays differ in shape")
        desc = W12KvCache(W12_KV_INT8 if pages.dtype is torch.int8 else W12_KV_E4M3, layers, num_pages, kv,
                                page // dim, dim, slots, rows[4] // dim, blocks, *ats)
        for name, value in (("index", index), ("kv_heads", kv), ("_desc", desc), ("_ref", ctypes.byref(desc))):
            object.__setattr__(self, name, value)

    @property
    def device(self):
        return self.pages.device

    def desc(self) -> W12KvCache:
        return self._desc

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.pages, self.scales, self.recent, self.page_table, self.length))


def kv_cache(layers: int, kv_heads: int, head_dim: int, num_pages: int, slots: int, max_pages: int,
             page_tokens: int = 64, step_rows: int = MAX_ROWS, int8: bool = False, device="cuda") -> KvCache:
    """An empty KV cache for steps of up to step_rows rows per sequence."""
    rows = -(-(page_tokens - 1 + step_rows) // 32) * 32
    dt = torch.int8 if int8 else torch.float8_e4m3fn
    return KvCache(
        torch.zeros(layers, num_pages, kv_heads, 2, page_tokens * head_dim, dtype=torch.uint8, device=device).view(dt),
        torch.ones(layers, num_pages, kv_heads, 2, dtype=torch.float32, device=device),
        torch.zeros(layers, slots, kv_heads, 2, rows * head_dim, dtype=torch.bfloat16, device=device),
        torch.zeros(slots, max_pages, dtype=torch.int32, device=device),
        torch.zeros(slots, dtype=torch.int32, device=device), head_dim)


def w12_kv_append(cache: KvCache, layer: int, qkv: torch.Tensor, row_off: torch.Tensor, rope: torch.Tensor,
                  q_heads: int, slot: torch.Tensor | None = None, parent: torch.Tensor | None = None,
                  interleaved: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotates q and k of qkv [rows, (q_heads + 2 kv_heads) * head_dim] (fp32
    or bf16) and appends k, v as the step's rows. rope [positions, rot_dim]
    fp32 holds cosines, then sines. Returns q [rows, q_heads, head_dim] bf16."""
    if not isinstance(qkv, torch.Tensor) or qkv.dtype not in (_F32, _BF16):
        raise TypeError("qkv must be a float32 or bfloat16 tensor")
    index, dim = cache.index, cache.head_dim
    at_x, at_rope = _get(qkv, qkv.dtype, "qkv", 2, index), _get(rope, _F32, "rope", 2, index)
    rows, width = qkv.shape
    if width != (q_heads + 2 * cache.kv_heads) * dim:
        raise ValueError(f"qkv has {width} columns, {q_heads} + 2 * {cache.kv_heads} heads of "
                         f"{dim} need {(q_heads + 2 * cache.kv_heads) * dim}")
    at_off = _get(row_off, _I32, "row_off", 1, index)
    seqs = row_off.shape[0] - 1
    if out is None:
        out = torch.empty(rows, q_heads, dim, dtype=_BF16, device=qkv.device)
    elif out.numel() < rows * q_heads * dim:
        raise ValueError("out must hold [rows, q_heads, head_dim]")
    positions, rot = rope.shape
    _run(index, "w12_kv_append", cache._ref, layer, seqs, 0 if slot is None else _get(slot, _I32, "slot", 1, index, seqs),
         at_off, rows, 0 if parent is None else _get(parent, _I32, "parent", 1, index, rows), at_x,
         W12_Y_F32 if qkv.dtype is _F32 else W12_Y_BF16, q_heads, at_rope, positions, rot, 1 if interleaved else 0,
         _get(out, _BF16, "out", None, index))
    return out


_kv_ws: dict = {}  # workspace bytes of w12_kv_attention by device and sizes


def _attention_workspace_bytes(cache: KvCache, seqs: int, rows: int, q_heads: int) -> int:
    key = (cache.index, cache.head_dim, cache.kv_heads, seqs, rows, q_heads)
    need = _kv_ws.get(key)
    if need is None:
        out = ctypes.c_size_t(0)
        with torch.cuda.device(cache.index):
            _ok(lib().w12_kv_attention_workspace(cache._ref, seqs, rows, q_heads, ctypes.byref(out)),
                "w12_kv_attention_workspace")
        need = _kv_ws[key] = out.value
    return need


def w12_kv_attention(cache: KvCache, layer: int, q: torch.Tensor, row_off: torch.Tensor,
                     slot: torch.Tensor | None = None, parent: torch.Tensor | None = None, scale: float | None = None,
                     out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the step's rows q [rows, q_heads, head_dim] bf16 over the
    cache; returns [rows, q_heads * head_dim] bf16. scale defaults to
    head_dim ** -0.5. ws: a workspace of the caller's, of one call at a time
    (its content is ignored, and is not zeros afterwards); without one the call
    allocates its own: it makes two launches, and those of another host thread
    on the same stream, or of a captured graph's replay, may come between them."""
    index = cache.index
    at_q = _get(q, _BF16, "q", 3, index)
    rows, q_heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError(f"q has head_dim {dim}, the cache {cache.head_dim}")
    at_off = _get(row_off, _I32, "row_off", 1, index)
    seqs = row_off.shape[0] - 1
    if out is None:
        out = torch.empty(rows, q_heads * dim, dtype=_BF16, device=q.device)
    elif out.numel() < rows * q_heads * dim:
        raise ValueError("out must hold [rows, q_heads * head_dim]")
    need = _attention_workspace_bytes(cache, seqs, rows, q_heads)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        scratch = ws.data_ptr(), need
    else:
        scratch = _scratch(ws, index)
    _run(index, "w12_kv_attention", cache._ref, layer, seqs,
         0 if slot is None else _get(slot, _I32, "slot", 1, index, seqs), at_off, rows,
         0 if parent is None else _get(parent, _I32, "parent", 1, index, rows), at_q, q_heads,
         dim ** -0.5 if scale is None else scale, _get(out, _BF16, "out", None, index),
         *scratch)
    return out


def w12_kv_commit(cache: KvCache, row_off: torch.Tensor, accept_len: torch.Tensor, path: torch.Tensor | None = None,
                  slot: torch.Tensor | None = None, length_out: torch.Tensor | None = None,
                  rows: int | None = None) -> torch.Tensor:
    """Keeps the accepted rows of the step (tree_accept's accept_len and
    path; path None: each sequence's first accept_len + 1 rows) in every
    layer. rows: how many the step had, known from path if there is one (at
    most 512 otherwise). Writes the new lengths into length_out [slots] (the cache's own by
    default) and returns it."""
    index = cache.index
    at_off = _get(row_off, _I32, "row_off", 1, index)
    seqs = row_off.shape[0] - 1
    at_path = 0
    if path is not None:
        at_path, rows = _get(path, _I32, "path", 1, index, rows), path.shape[0]
    elif rows is None:
        rows = MAX_ROWS
    if length_out is None:
        length_out = cache.length
    _run(index, "w12_kv_commit", cache._ref, seqs, 0 if slot is None else _get(slot, _I32, "slot", 1, index, seqs), at_off,
         rows, _get(accept_len, _I32, "accept_len", 1, index, seqs), at_path,
         _get(length_out, _I32, "length_out", 1, index, cache._desc.slots))
    return length_out


def tree_accept_sampled(node_off: torch.Tensor, parent: torch.Tensor, token: torch.Tensor, logits: torch.Tensor,
                        u_accept: torch.Tensor, u_bonus: torch.Tensor, temperature: torch.Tensor | None = None,
                        draft: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Tree acceptance of sampling requests: logits [nodes, vocab] fp32 or
    bf16 (a row per node), random numbers u_accept [nodes] and u_bonus
    [trees], temperature [trees] or None (1), draft [nodes, vocab] fp32 or
    None (chosen drafts); ws as w12_kv_attention's. Returns (accept_len, path,
    bonus) as tree_accept."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (_F32, _BF16):
        raise TypeError("logits must be a float32 or bfloat16 tensor")
    at_x = _get(logits, logits.dtype, "logits", 2, None)
    index, dev = logits.get_device(), logits.device
    at_off = _get(node_off, _I32, "node_off", 1, index)
    total, vocab = logits.shape
    T = node_off.shape[0] - 1
    if T < 1:
        raise ValueError("tree_accept_sampled: no trees")
    at = (_get(parent, _I32, "parent", 1, index, total), _get(token, _I32, "token", 1, index, total))
    at_u = (_get(u_accept, _F32, "u_accept", 1, index, total), _get(u_bonus, _F32, "u_bonus", 1, index, T))
    at_temp = 0 if temperature is None else _get(temperature, _F32, "temperature", 1, index, T)
    at_draft = 0 if draft is None else _get(draft, _F32, "draft", 2, index)
    if draft is not None and draft.shape != logits.shape:
        raise ValueError("draft and logits differ in shape")
    if ws is None:
        need = ctypes.c_size_t(0)
        _ok((_lib or lib()).tree_accept_sampled_workspace(T, total, vocab, ctypes.byref(need)),
            "tree_accept_sampled_workspace")
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        scratch = ws.data_ptr(), need.value
    else:
        scratch = _scratch(ws, index)
    # one allocation for the three outputs (bonus and accept_len first: T entries each)
    out = torch.empty(2 * T + total, dtype=_I32, device=dev)
    base = out.data_ptr()
    _run(index, "tree_accept_sampled", T, at_off, total, *at, at_x, W12_Y_F32 if logits.dtype is _F32 else W12_Y_BF16,
         vocab, at_temp, at_draft, *at_u, base, base + 8 * T, base + 4 * T, *scratch)
    return out[:T], out[2 * T:], out[T:2 * T]


# ------------------------------------------------------------------ recurrent layers of the verify pass

@dataclass(frozen=True, eq=False, init=False)  # the description holds the arrays' addresses
class DeltaCache:
    """Device-resident state of the recurrent layers: the arrays of
    include/w12.h. state is [layers, slots, value_heads, key_dim, value_dim]
    float32, conv [layers, slots, conv_width - 1, channels] bfloat16; of one
    step at a time raw [layers, step_rows, channels] bfloat16, kv [layers,
    step_rows, key_heads * key_dim + value_heads * value_dim] bfloat16, gates
    [layers, step_rows, 2, value_heads] float32, delta [layers, step_rows,
    value_heads, value_dim] float32. The arrays stay the same; their contents
    may be written at any time (a new sequence: its slot of state and conv
    zeroed)."""
    state: torch.Tensor
    conv: torch.Tensor
    raw: torch.Tensor
    kv: torch.Tensor
    gates: torch.Tensor
    delta: torch.Tensor
    key_heads: int

    def __init__(self, state, conv, raw, kv, gates, delta, key_heads):
        hk = key_heads
        try:  # all at once: programs describe their state again where they switch between steps' arrays
            index = state.get_device()
            layers, slots, hv, kd, vd = state.shape
            rows, width = raw.shape[1], conv.shape[2]
            kv_width = hk * kd + hv * vd
            channels = kv_width + hk * kd
            good = (index >= 0 and state.dtype is _F32 and gates.dtype is _F32 and delta.dtype is _F32
                    and conv.dtype is _BF16 and raw.dtype is _BF16 and kv.dtype is _BF16
                    and conv.shape == (layers, slots, width, channels) and raw.shape == (layers, rows, channels)
                    and kv.shape == (layers, rows, kv_width) and gates.shape == (layers, rows, 2, hv)
                    and delta.shape == (layers, rows, hv, vd)
                    and state.is_contiguous() and conv.is_contiguous() and raw.is_contiguous() and kv.is_contiguous()
                    and gates.is_contiguous() and delta.is_contiguous() and conv.get_device() == index
                    and raw.get_device() == index and kv.get_device() == index and gates.get_device() == index
                    and delta.get_device() == index)
        except (AttributeError, TypeError, ValueError, IndexError):
            good = False
        if not good:
            _get(state, _F32, "state", 5, None)
            for t, dtype, name, ndim in ((conv, _BF16, "conv", 4), (raw, _BF16, "raw", 3), (kv, _BF16, "kv", 3),
                                         (gates, _F32, "gates", 4), (delta, _F32, "delta", 4)):
                _get(t, dtype, name, ndim, state.get_device())
            raise ValueError("the recurrent state's arrays differ in shape")
        desc = W12DeltaCache(layers, slots, rows, hk, hv, kd, vd, width + 1, state.data_ptr(), conv.data_ptr(),
                             raw.data_ptr(), kv.data_ptr(), gates.data_ptr(), delta.data_ptr())
        self.__dict__.update(state=state, conv=conv, raw=raw, kv=kv, gates=gates, delta=delta, key_heads=hk, index=index,
                             value_heads=hv, key_dim=kd, value_dim=vd, channels=channels, conv_width=width + 1,
                             step_rows=rows, _desc=desc, _ref=ctypes.byref(desc))

    @property
    def device(self):
        return self.state.device

    def desc(self) -> W12DeltaCache:
        return self._desc

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.state, self.conv, self.raw, self.kv, self.gates, self.delta))


def delta_cache(layers: int, slots: int, key_heads: int, value_heads: int, key_dim: int, value_dim: int,
                conv_width: int = 4, step_rows: int = MAX_ROWS, device="cuda") -> DeltaCache:
    """Recurrent layers' state of `slots` fresh sequences, for steps of up to step_rows rows in all."""
    kv_width = key_heads * key_dim + value_heads * value_dim
    channels = kv_width + key_heads * key_dim
    f, b = dict(dtype=torch.float32, device=device), dict(dtype=torch.bfloat16, device=device)
    return DeltaCache(torch.zeros(layers, slots, value_heads, key_dim, value_dim, **f),
                      torch.zeros(layers, slots, conv_width - 1, channels, **b),
                      torch.zeros(layers, step_rows, channels, **b), torch.zeros(layers, step_rows, kv_width, **b),
                      torch.zeros(layers, step_rows, 2, value_heads, **f),
                      torch.zeros(layers, step_rows, value_heads, value_dim, **f), key_heads)


def _rows_of(t, name: str, columns: int, index: int) -> tuple[int, int, int]:
    """Address, row stride and type of a [rows, columns] fp32 or bf16 tensor
    on GPU `index` whose rows lie apart (columns of a wider product)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype, shape = t.dtype, t.shape
    if dtype is not _F32 and dtype is not _BF16:
        raise TypeError(f"{name} must be a float32 or bfloat16 tensor (got {dtype})")
    if len(shape) != 2 or shape[1] != columns:
        raise ValueError(f"{name} must be [rows, {columns}] (got {tuple(shape)})")
    if index < 0 or t.get_device() != index:
        raise ValueError(f"{name} must be on {'a GPU' if index < 0 else f'cuda:{index}'} (got {t.device})")
    step, unit = t.stride()
    if shape[0] == 1:
        step = -(-columns // 8) * 8  # one row: any stride
    elif step < columns:
        raise ValueError(f"{name}'s rows must lie apart (strides {t.stride()})")
    if unit != 1 and columns > 1:
        raise ValueError(f"{name}'s rows must be contiguous (strides {t.stride()})")
    return t.data_ptr(), step, W12_Y_F32 if dtype is _F32 else W12_Y_BF16


def w12_delta_append(cache: DeltaCache, layer: int, qkv: torch.Tensor, ba: torch.Tensor, row_off: torch.Tensor,
                     conv_weight: torch.Tensor, a_log: torch.Tensor, dt_bias: torch.Tensor,
                     conv_bias: torch.Tensor | None = None, slot: torch.Tensor | None = None,
                     parent: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Convolution, SiLU, normalised heads and gates of the step's rows, staged
    for w12_delta_rule and w12_delta_commit. qkv [rows, channels] and ba [rows,
    2 * value_heads] (b, then a), both fp32 or both bf16, may be columns of one
    product; conv_weight [channels, conv_width], conv_bias [channels], a_log
    and dt_bias [value_heads] fp32. Returns q [rows, key_heads, key_dim] bf16."""
    index, hv, hk, kd = cache.index, cache.value_heads, cache.key_heads, cache.key_dim
    at_x, step_x, kind = _rows_of(qkv, "qkv", cache.channels, index)
    at_b, step_b, kind_b = _rows_of(ba, "ba", 2 * hv, index)
    rows = qkv.shape[0]
    if kind_b != kind or ba.shape[0] != rows:
        raise ValueError("qkv and ba differ in type or rows")
    at_off = _get(row_off, _I32, "row_off", 1, index)
    seqs = row_off.shape[0] - 1
    at_w = _get(conv_weight, _F32, "conv_weight", 2, index)
    if conv_weight.shape != (cache.channels, cache.conv_width):
        raise ValueError(f"conv_weight must be [{cache.channels}, {cache.conv_width}]")
    at_c = 0 if conv_bias is None else _get(conv_bias, _F32, "conv_bias", 1, index, cache.channels)
    at_a, at_d = _get(a_log, _F32, "a_log", 1, index, hv), _get(dt_bias, _F32, "dt_bias", 1, index, hv)
    if out is None:
        out = torch.empty(rows, hk, kd, dtype=_BF16, device=qkv.device)
    at_out = _get(out, _BF16, "out", None, index)
    if out.numel() < rows * hk * kd:
        raise ValueError("out must hold [rows, key_heads, key_dim]")
    _run(index, "w12_delta_append", cache._ref, layer, seqs,
         0 if slot is None else _get(slot, _I32, "slot", 1, index, seqs), at_off, rows,
         0 if parent is None else _get(parent, _I32, "parent", 1, index, rows), at_x, step_x, at_b, step_b, kind, at_w,
         at_c, at_a, at_d, at_out)
    return out


def w12_delta_rule(cache: DeltaCache, layer: int, q: torch.Tensor, row_off: torch.Tensor,
                   slot: torch.Tensor | None = None, parent: torch.Tensor | None = None, scale: float | None = None,
                   keep: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gated delta rule over the step's staged rows, q [rows, key_heads,
    key_dim] bf16; returns [rows, value_heads * value_dim] bf16. scale defaults
    to key_dim ** -0.5. keep (chains only: prompts, plain decoding): every row
    joins the state and the window, and w12_delta_commit is not called. A step of
    single rows and long sequences is faster as two calls (include/w12.h)."""
    index = cache.index
    at_q = _get(q, _BF16, "q", 3, index)
    rows, hk, kd = q.shape
    if hk != cache.key_heads or kd != cache.key_dim:
        raise ValueError(f"q has {hk} heads of {kd}, the state {cache.key_heads} of {cache.key_dim}")
    if keep and parent is not None:
        raise ValueError("keep is for chains: the rows of a tree are kept by w12_delta_commit")
    at_off = _get(row_off, _I32, "row_off", 1, index)
    seqs = row_off.shape[0] - 1
    wide = cache.value_heads * cache.value_dim
    if out is None:
        out = torch.empty(rows, wide, dtype=_BF16, device=q.device)
    at_out = _get(out, _BF16, "out", None, index)
    if out.numel() < rows * wide:
        raise ValueError("out must hold [rows, value_heads * value_dim]")
    _run(index, "w12_delta_rule", cache._ref, layer, seqs,
         0 if slot is None else _get(slot, _I32, "slot", 1, index, seqs), at_off, rows,
         0 if parent is None else _get(parent, _I32, "parent", 1, index, rows), at_q,
         kd ** -0.5 if scale is None else scale, 1 if keep else 0, at_out)
    return out


def w12_delta_commit(cache: DeltaCache, row_off: torch.Tensor, accept_len: torch.Tensor,
                     path: torch.Tensor | None = None, slot: torch.Tensor | None = None,
                     rows: int | None = None) -> torch.Tensor:
    """Keeps the accepted rows of the step (tree_accept's accept_len and path;
    path None: each sequence's first accept_len + 1 rows) in every layer. rows:
    how many the step had, known from path if there is one (otherwise at most
    512 and what the staging holds). Returns the rows kept of each sequence
    [seqs] int32, -1 where it was refused."""
    index = cache.index
    at_off = _get(row_off, _I32, "row_off", 1, index)
    seqs = row_off.shape[0] - 1
    at_path = 0
    if path is not None:
        at_path, rows = _get(path, _I32, "path", 1, index, rows), path.shape[0]
    elif rows is None:
        rows = min(MAX_ROWS, cache.step_rows)
    kept = torch.empty(max(seqs, 0), dtype=_I32, device=cache.device)
    _run(index, "w12_delta_commit", cache._ref, seqs, 0 if slot is None else _get(slot, _I32, "slot", 1, index, seqs),
         at_off, rows, _get(accept_len, _I32, "accept_len", 1, index, seqs), at_path, kept.data_ptr())
    return kept


# ------------------------------------------------------------------ norms between products

def w12_norm(y: torch.Tensor | None, weight: torch.Tensor | None = None, post_weight: torch.Tensor | None = None,
             gate: torch.Tensor | None = None, h: torch.Tensor | None = None, scale: float = 1.0, groups: int = 1,
             eps: float = 1e-6, out: torch.Tensor | None = None) -> torch.Tensor:
    """Norm of a block's output y (post_weight), its gate (SiLU), the residual
    h += scale * that, in place, and the norm before the next block (weight);
    each part but one of y and h may be absent. y and gate [rows, groups *
    width] fp32 or bf16 may be columns of wider products, h [rows, groups *
    width] fp32 or bf16, the weights [width] fp32. Returns bf16 [rows, groups *
    width]."""
    first = y if y is not None else h
    if not isinstance(first, torch.Tensor) or first.dim() != 2:
        raise TypeError("w12_norm needs y or h, [rows, groups * width]")
    index, (rows, wide) = first.get_device(), first.shape
    if groups < 1 or wide % groups:
        raise ValueError(f"{wide} columns are not {groups} groups")
    if y is None and (post_weight is not None or gate is not None):
        raise ValueError("without y there is no post_weight and no gate")
    width = wide // groups
    none = (0, wide, W12_Y_F32)
    at_y = none if y is None else _rows_of(y, "y", wide, index)
    at_g = none if gate is None else _rows_of(gate, "gate", wide, index)
    at_h, kind_h = 0, W12_Y_F32
    if h is not None:
        if not isinstance(h, torch.Tensor) or h.dtype not in (_F32, _BF16):
            raise TypeError("h must be a float32 or bfloat16 tensor")
        at_h, kind_h = _get(h, h.dtype, "h", 2, index), W12_Y_F32 if h.dtype is _F32 else W12_Y_BF16
    if (gate is not None and gate.shape[0] != rows) or (h is not None and h is not first and h.shape != first.shape):
        raise ValueError("y, gate and h differ in shape")
    at_p = 0 if post_weight is None else _get(post_weight, _F32, "post_weight", 1, index, width)
    at_w = 0 if weight is None else _get(weight, _F32, "weight", 1, index, width)
    if out is None:
        out = torch.empty(rows, wide, dtype=_BF16, device=first.device)
    at_out = _get(out, _BF16, "out", None, index)
    if out.numel() < rows * wide:
        raise ValueError("out must hold [rows, groups * width]")
    _run(index, "w12_norm", rows, groups, width, at_y[0], at_y[2], at_y[1], at_p, at_g[0], at_g[2], at_g[1], scale, at_h,
         kind_h, at_w, eps, at_out)
    return out
