"""Python binding of libmoeq over torch device tensors.

torch provides device memory and the current HIP stream; each function below
validates shapes, passes raw pointers to the C ABI and returns the tensors
the library filled.  No arithmetic of the method happens here.

The functions record nothing for autograd: what they return does not require
grad, whatever their inputs do.  Gradients are calls of their own
(grouped_gemm with trans, grouped_wgrad, route_scored_grad, combine_grad,
block_norm_grad), for an autograd.Function of the caller's to make.
"""

import ctypes
import functools
from ctypes import c_void_p

import numpy as np
import torch

from . import _lib
from ._lib import MoeqError, check, lib  # noqa: F401

GATE, UP, DOWN = 0, 1, 2


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t, dtype, shape, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------- encoding

def quantize_rtn(w, bits, G):
    """Asymmetric RTN of an fp16 block [N, K]: (codes u8 [N,K], scales fp16
    [N,K/G], zeros u8 [N,K/G])."""
    N, K = w.shape
    _need(w, torch.float16, (N, K), "w")
    codes = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    scales = torch.empty((N, K // G), dtype=torch.float16, device=w.device)
    zeros = torch.empty((N, K // G), dtype=torch.uint8, device=w.device)
    check(lib().moeq_quantize_rtn(_ptr(w), N, K, G, bits, _ptr(codes), _ptr(scales), _ptr(zeros),
                                  _stream()), "moeq_quantize_rtn")
    return codes, scales, zeros


def build_lut(w, codes4, scales, zeros, q, G):
    """16-slot fp16 LUT [N, K/G, 16] of a block committed to q bit-planes."""
    N, K = w.shape
    _need(w, torch.float16, (N, K), "w")
    _need(codes4, torch.uint8, (N, K), "codes4")
    _need(scales, torch.float16, (N, K // G), "scales")
    _need(zeros, torch.uint8, (N, K // G), "zeros")
    lut = torch.empty((N, K // G, 16), dtype=torch.float16, device=w.device)
    check(lib().moeq_build_lut(_ptr(w), _ptr(codes4), _ptr(scales), _ptr(zeros), N, K, G, q,
                               _ptr(lut), _stream()), "moeq_build_lut")
    return lut


def fit_lowrank(w, codes, scales, zeros, G, omega, r, power_iters=2):
    """Rank-r compensator factors (U fp16 [N, r], V fp16 [r, K]) of the mean
    RTN residual of the blocks w [n, N, K] (or one block [N, K]); omega
    fp32 [K, l] is the Gaussian test matrix (see moeq_fit_lowrank)."""
    if w.dim() == 2:
        w, codes, scales, zeros = (t.unsqueeze(0) for t in (w, codes, scales, zeros))
    n_mat, N, K = w.shape
    l = omega.shape[1]
    _need(w, torch.float16, (n_mat, N, K), "w")
    _need(codes, torch.uint8, (n_mat, N, K), "codes")
    _need(scales, torch.float16, (n_mat, N, K // G), "scales")
    _need(zeros, torch.uint8, (n_mat, N, K // G), "zeros")
    _need(omega, torch.float32, (K, l), "omega")
    n = ctypes.c_size_t(0)
    check(lib().moeq_fit_lowrank_workspace_size(N, K, r, l, ctypes.byref(n)), "moeq_fit_lowrank_workspace_size")
    ws = torch.empty((max(1, n.value),), dtype=torch.uint8, device=w.device)
    U = torch.empty((N, r), dtype=torch.float16, device=w.device)
    V = torch.empty((r, K), dtype=torch.float16, device=w.device)
    check(lib().moeq_fit_lowrank(_ptr(w), _ptr(codes), _ptr(scales), _ptr(zeros), n_mat, N, K, G, _ptr(omega), l, r,
                                 power_iters, _ptr(U), _ptr(V), _ptr(ws), n.value, _stream()), "moeq_fit_lowrank")
    return U, V


# ---------------------------------------------------------------- layer

def _ptr_array(tensors):
    arr = (ctypes.c_void_p * len(tensors))()
    for i, t in enumerate(tensors):
        arr[i] = t.data_ptr() if t is not None else 0
    return arr


class PackedLayer:
    """A packed quantized layer: one device buffer plus the library handle.

    blocks: list over b = e*3 + blk of dicts with
      INT:      codes u8 [N,K], scales fp16 [N,K/G], zeros u8 [N,K/G]
      bitplane: codes (4-bit parent codes) u8 [N,K], lut fp16 [N,K/G,16]
    factors: list over b of (U [N,r], V [r,K]) fp16 or None (r = 0)
    shared: list over group*3+blk of (Us, Vs) or None (rs = 0)
    """

    def __init__(self, E, H, I, G, fmt, bits, blocks, factors=None, shared=None, share=0,
                 device=None):
        device = device or torch.device("cuda", torch.cuda.current_device())
        self.E, self.H, self.I, self.G = E, H, I, G
        self.fmt = fmt
        self.bits = np.asarray(bits, dtype=np.uint8).reshape(E * 3).copy()
        nb = 3 * E
        assert len(blocks) == nb
        fmt_id = _lib.FMT_INT if fmt == "int" else _lib.FMT_BITPLANE
        self._keep = []
        codes = _ptr_array([b["codes"] for b in blocks])
        if fmt == "int":
            scales = _ptr_array([b["scales"] for b in blocks])
            zeros = _ptr_array([b["zeros"] for b in blocks])
            luts = None
        else:
            scales = zeros = None
            luts = _ptr_array([b["lut"] for b in blocks])
        r = 0
        U = V = None
        if factors is not None and factors[0] is not None:
            r = factors[0][0].shape[1]
            U = _ptr_array([f[0] for f in factors])
            V = _ptr_array([f[1] for f in factors])
        rs = 0
        Us = Vs = None
        if shared is not None and shared[0] is not None:
            rs = shared[0][0].shape[1]
            Us = _ptr_array([f[0] for f in shared])
            Vs = _ptr_array([f[1] for f in shared])
        self.r, self.rs, self.share = r, rs, share
        bits_arr = (ctypes.c_uint8 * nb)(*[int(b) for b in self.bits])
        cast = lambda a: ctypes.cast(a, _lib.c_vpp) if a is not None else None
        d = _lib.LayerDesc(E, H, I, G, fmt_id, ctypes.cast(bits_arr, _lib.c_u8p), cast(codes),
                           cast(scales), cast(zeros), cast(luts), r, cast(U), cast(V), rs, share,
                           cast(Us), cast(Vs))
        self._desc_keep = (bits_arr, codes, scales, zeros, luts, U, V, Us, Vs)
        nbytes = ctypes.c_size_t(0)
        check(lib().moeq_pack_size(ctypes.byref(d), ctypes.byref(nbytes)), "moeq_pack_size")
        self.buf = torch.empty(nbytes.value, dtype=torch.uint8, device=device)
        handle = ctypes.c_void_p(0)
        check(lib().moeq_pack(ctypes.byref(d), _ptr(self.buf), nbytes.value, _stream(),
                              ctypes.byref(handle)), "moeq_pack")
        self.handle = handle
        self.nbytes = nbytes.value

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib._lib is not None:
            _lib._lib.moeq_layer_destroy(h)
            self.handle = None

    def block_bytes(self, e, blk):
        out = ctypes.c_size_t(0)
        check(lib().moeq_layer_block_bytes(self.handle, e, blk, ctypes.byref(out)), "block_bytes")
        return out.value

    def shared_bytes(self, g, blk):
        out = ctypes.c_size_t(0)
        check(lib().moeq_layer_shared_bytes(self.handle, g, blk, ctypes.byref(out)), "shared_bytes")
        return out.value

    def block_shape(self, blk):
        return (self.I, self.H) if blk in (GATE, UP) else (self.H, self.I)

    def debug_unpack(self, e, blk):
        N, K = self.block_shape(blk)
        out = torch.empty((N, K), dtype=torch.uint8, device=self.buf.device)
        check(lib().moeq_debug_unpack(self.handle, e, blk, _ptr(out), _stream()), "moeq_debug_unpack")
        return out

    def commit_bits(self, e, blk, q, lut):
        """Commit bit-plane count q of block (e, blk) with its LUT [N, K/G, 16]
        (see moeq_commit_bits); stream-ordered on the current stream."""
        N, K = self.block_shape(blk)
        _need(lut, torch.float16, (N, K // self.G, 16), "lut")
        check(lib().moeq_commit_bits(self.handle, e, blk, q, _ptr(lut), _stream()), "moeq_commit_bits")

    def committed_bits(self, e, blk):
        q = ctypes.c_int32(0)
        check(lib().moeq_committed_bits(self.handle, e, blk, ctypes.byref(q)), "moeq_committed_bits")
        return q.value

    def plane_release(self, e, blk, host, stream=None):
        """Copy the planes above the committed q to the pinned host tensor
        `host` (uint8, plane p at offset p * plane_bytes) on `stream`
        (default: the current stream) and mark them released."""
        s = ctypes.c_void_p((stream or torch.cuda.current_stream()).cuda_stream)
        check(lib().moeq_plane_release(self.handle, e, blk, _ptr(host), host.numel(), s), "moeq_plane_release")

    def plane_reload(self, e, blk, q, host, stream=None):
        """Copy planes back from `host` until q planes are resident (see
        moeq_plane_reload)."""
        s = ctypes.c_void_p((stream or torch.cuda.current_stream()).cuda_stream)
        check(lib().moeq_plane_reload(self.handle, e, blk, q, _ptr(host), host.numel(), s), "moeq_plane_reload")

    def plane_event(self, e, blk):
        """The hipEvent_t (as an integer) of the block's last release or reload copy."""
        ev = c_void_p(0)
        check(lib().moeq_plane_event(self.handle, e, blk, ctypes.byref(ev)), "moeq_plane_event")
        return ev.value

    def resident_planes(self, e, blk):
        n = ctypes.c_int32(0)
        check(lib().moeq_resident_planes(self.handle, e, blk, ctypes.byref(n)), "moeq_resident_planes")
        return n.value

    def set_desired_bits(self, e, blk, d):
        check(lib().moeq_set_desired_bits(self.handle, e, blk, d), "moeq_set_desired_bits")

    def desired_bits(self, e, blk):
        d = ctypes.c_int32(0)
        check(lib().moeq_desired_bits(self.handle, e, blk, ctypes.byref(d)), "moeq_desired_bits")
        return d.value

    def plane_region(self, e, blk, plane):
        """(device address, bytes) of bit-plane `plane` (0 = most significant)."""
        ptr, n = c_void_p(0), ctypes.c_size_t(0)
        check(lib().moeq_plane_region(self.handle, e, blk, plane, ctypes.byref(ptr), ctypes.byref(n)),
              "moeq_plane_region")
        return ptr.value, n.value


def quantize_block(w, fmt, bits, G):
    """Quantize one fp16 block with the library's kernels into the pack input
    dict (INT: codes/scales/zeros; bit-plane: 4-bit parent codes + LUT)."""
    if fmt == "int":
        c, s, z = quantize_rtn(w, bits, G)
        return dict(codes=c, scales=s, zeros=z)
    c, s, z = quantize_rtn(w, 4, G)
    return dict(codes=c, lut=build_lut(w, c, s, z, bits, G))


# -------------------------------------------------------------- routing

class RoutingOut:
    """Tensors of one routing, each with its own memory and version counter (an
    autograd.Function may save some of them and the caller write others)."""

    def __init__(self, T, E, k, device):
        self.T, self.E, self.k = T, E, k
        self.ws_bytes = _route_workspace_size(T, E, k)
        P = T * k
        # (sizes as numbers, after the first by new_empty: 1.2 us each on the host,
        # torch.empty of tuples 1.7)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        new = self.offsets.new_empty
        self.ids = new(T, k)
        self.sorted_pairs = new(P)
        self.pair_pos = new(P)
        self.gates = new(T, k, dtype=torch.float32)
        if self.ws_bytes:
            self.ws   # (made here, on the stream of the first call)
        self.c = _lib.Routing(self.ids.data_ptr(), self.gates.data_ptr(), self.offsets.data_ptr(),
                              self.sorted_pairs.data_ptr(), self.pair_pos.data_ptr())

    @functools.cached_property
    def ws(self):
        """Workspace of the call; where it needs none, a byte, made when asked for."""
        return self.offsets.new_empty((max(1, self.ws_bytes),), dtype=torch.uint8)

    def ws_addr(self):
        return self.ws.data_ptr() if self.ws_bytes else None


@functools.lru_cache(maxsize=1024)
def _route_workspace_size(T, E, k):
    n = ctypes.c_size_t(0)
    check(lib().moeq_route_workspace_size(T, E, k, ctypes.byref(n)), "moeq_route_workspace_size")
    return n.value


def route(logits, k, out=None):
    """Top-k routing and counting sort of fp32 logits [T, E] (see moeq_route)."""
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    if out is None:
        out = RoutingOut(T, E, k, logits.device)
    check(lib().moeq_route(_ptr(logits), T, E, k, ctypes.byref(out.c), out.ws_addr(), out.ws_bytes, _stream()),
          "moeq_route")
    return out


def route_mass(routing, edges=()):
    """Per-expert routing mass and (with edges) bucket index (see moeq_route_mass)."""
    E = routing.E
    mass = torch.empty((E,), dtype=torch.float32, device=routing.ids.device)
    bucket = torch.empty((E,), dtype=torch.int32, device=routing.ids.device) if len(edges) else None
    ed = (ctypes.c_float * max(1, len(edges)))(*[float(v) for v in edges])
    check(lib().moeq_route_mass(ctypes.byref(routing.c), routing.T, E, routing.k,
                                ctypes.cast(ed, c_void_p) if len(edges) else None, len(edges),
                                _ptr(mass), _ptr(bucket), _stream()), "moeq_route_mass")
    return mass, bucket


def plan_reductions(q, bytes_tbl, g, mu, eta, eps, target):
    """Greedy bit-plane release plan (see moeq_plan_reductions); host arrays.
    Returns (planned q, block of each action in order, released bytes, damage)."""
    q = np.ascontiguousarray(q, dtype=np.int32).copy()
    n = q.shape[0]
    bt = np.ascontiguousarray(bytes_tbl, dtype=np.float64).reshape(n, 3)
    gg = np.ascontiguousarray(g, dtype=np.float64).reshape(n, 3)
    mu = np.ascontiguousarray(mu, dtype=np.float64).reshape(n)
    eta = np.ascontiguousarray(eta, dtype=np.float64).reshape(n)
    cap = int(2 * n) + 1
    order = np.zeros(cap, dtype=np.int32)
    rel, dmg, na = ctypes.c_double(0), ctypes.c_double(0), ctypes.c_int32(0)
    dp = ctypes.POINTER(ctypes.c_double)
    ip = ctypes.POINTER(ctypes.c_int32)
    check(lib().moeq_plan_reductions(n, q.ctypes.data_as(ip), bt.ctypes.data_as(dp), gg.ctypes.data_as(dp),
                                     mu.ctypes.data_as(dp), eta.ctypes.data_as(dp), float(eps), float(target),
                                     order.ctypes.data_as(ip), cap, ctypes.byref(rel), ctypes.byref(dmg),
                                     ctypes.byref(na)), "moeq_plan_reductions")
    return q, order[:na.value].tolist(), rel.value, dmg.value


# ------------------------------------------------------------ expert FFN

class FfnWorkspace:
    """Workspace of moeq_expert_ffn, or (forward=True) of moeq_moe_forward."""

    def __init__(self, layer, T, k, path=0, split_k=0, forward=False):
        self.opts = _lib.FfnOptions(path, split_k)
        n = ctypes.c_size_t(0)
        size_fn = lib().moeq_forward_workspace_size if forward else lib().moeq_ffn_workspace_size
        check(size_fn(layer.handle, T, k, ctypes.byref(self.opts), ctypes.byref(n)), "workspace_size")
        self.nbytes = n.value
        self.buf = torch.empty(max(256, n.value), dtype=torch.uint8, device=layer.buf.device)


def expert_ffn(layer, x, routing, n_comp, out=None, out_dtype=torch.float16, ws=None, path=0,
               split_k=0):
    """Routed expert FFN y [T, H] (see moeq_expert_ffn)."""
    T = routing.T
    k = routing.k
    _need(x, torch.float16, (T, layer.H), "x")
    if out is None:
        out = torch.empty((T, layer.H), dtype=out_dtype, device=x.device)
    ydt = _lib.F32 if out.dtype == torch.float32 else _lib.F16
    _need(out, out.dtype, (T, layer.H), "out")
    if ws is None:
        ws = FfnWorkspace(layer, T, k, path, split_k)
    check(lib().moeq_expert_ffn(layer.handle, _ptr(x), T, k, ctypes.byref(routing.c), n_comp,
                                _ptr(out), ydt, _ptr(ws.buf), ws.buf.numel(), ctypes.byref(ws.opts),
                                _stream()), "moeq_expert_ffn")
    return out


def moe_forward(layer, logits, x, k, n_comp, routing=None, out=None, out_dtype=torch.float16, ws=None,
                path=0, split_k=0):
    """Routing and the expert FFN in one call (see moeq_moe_forward).
    Returns (y [T, H], routing)."""
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    _need(x, torch.float16, (T, layer.H), "x")
    if routing is None:
        routing = RoutingOut(T, E, k, x.device)
    if out is None:
        out = torch.empty((T, layer.H), dtype=out_dtype, device=x.device)
    ydt = _lib.F32 if out.dtype == torch.float32 else _lib.F16
    _need(out, out.dtype, (T, layer.H), "out")
    if ws is None:
        ws = FfnWorkspace(layer, T, k, path, split_k, forward=True)
    check(lib().moeq_moe_forward(layer.handle, _ptr(logits), _ptr(x), T, k, n_comp, ctypes.byref(routing.c),
                                 _ptr(out), ydt, _ptr(ws.buf), ws.buf.numel(), ctypes.byref(ws.opts), _stream()),
          "moeq_moe_forward")
    return out, routing


# --------------------------------- expert matrices in 16 or 8 bits

_DTYPE = {torch.float16: _lib.F16, torch.bfloat16: _lib.BF16, torch.float32: _lib.F32}
_16BIT = (torch.float16, torch.bfloat16)


def _like(t, dtypes, ndim, dev, name):
    """Checks a strided operand: on device index `dev`, one of `dtypes`,
    `ndim` dimensions, the last one contiguous."""
    try:
        if t.dtype in dtypes and t.dim() == ndim and t.get_device() == dev >= 0 and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device than the other tensors")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {tuple(dtypes)}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def _sizes(**sizes):
    """Refuses sizes that the library's 32-bit arguments would cut off."""
    for name, v in sizes.items():
        if v > 0x7fffffff:
            raise ValueError(f"{name}={v} is beyond 32 bits")


def _ld(t):
    """Elements between the rows of t (its row length when there is one row)."""
    return t.stride(-2) if t.shape[-2] > 1 else t.shape[-1]


def _flat(t, n, dtype, dev, name):
    _like(t, (dtype,), 1, dev, name)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} elements, got {t.shape[0]}")


def _groups(T, E, offsets, pairs, k, dev):
    """moeq_groups of sorted rows, and their count."""
    if offsets is None:
        if E != 1:
            raise ValueError("offsets are needed with more than one expert")
    else:
        _flat(offsets, E + 1, torch.int32, dev, "offsets")
    P = T
    if pairs is not None:
        _like(pairs, (torch.int32,), 1, dev, "pairs")
        P = pairs.shape[0]
    if T > 0x7fffffff or P > 0x7fffffff or E > 0x7fffffff or k > 0x7fffffff:
        _sizes(T=T, P=P, E=E, k=k)
    return _lib.Groups(offsets.data_ptr() if offsets is not None else None,
                       pairs.data_ptr() if pairs is not None else None, E, P, T, k), P


def _out(out, shape, dtype, dtypes, dev, like, name="out"):
    """The caller's output tensor, or a new one."""
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _like(out, dtypes, len(shape), dev, name)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(out.shape)}")
    _written(out)
    return out


def _written(t):
    """Counts a write of the library into t, as torch's own operations do: a
    backward pass that saved t before reports it instead of using it."""
    torch.autograd.graph.increment_version(t)


_FUNCS = {}


def _launch(name, dev, *args):
    """Calls entry point `name` on the current stream of device `dev`."""
    f = _FUNCS.get(name)
    if f is None:
        f = _FUNCS[name] = getattr(lib(), name)
    if torch._C._cuda_getDevice() == dev:
        st = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        check(st, name)


def grouped_gemm(x, w, offsets, pairs=None, k=1, trans=False, out=None, out_dtype=None):
    """Products of expert-sorted rows with their expert's matrix (see
    moeq_grouped_gemm): out[r] = x[pairs[r] // k] @ w[e].T, or @ w[e] with
    trans, for the rows offsets[e] <= r < offsets[e + 1] of every expert e.

    x fp16 or bf16 [T, K]; w of the same type [E, N, K] ([E, K, N] with
    trans); offsets int32 [E + 1]; pairs int32 [P] or None (out[r] from
    x[r]).  Returns [P, N] of out_dtype (x's type, or float32); rows outside
    the offsets are left as they were (undefined in a new tensor).  out may
    not overlap the inputs.  No autograd: the gradients are this call with trans
    and grouped_wgrad."""
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    _like(x, _16BIT, 2, dev, "x")
    _like(w, (x.dtype,), 3, dev, "w")
    T, K = x.shape
    E, N, Kw = w.shape if not trans else (w.shape[0], w.shape[2], w.shape[1])
    if Kw != K:
        raise ValueError(f"x has {K} columns, w {Kw}")
    if N > 0x7fffffff or K > 0x7fffffff:
        _sizes(N=N, K=K)
    g, P = _groups(T, E, offsets, pairs, k, dev)
    out = _out(out, (P, N), out_dtype or x.dtype, (x.dtype, torch.float32), dev, x)
    _launch("moeq_grouped_gemm", dev, g, x.data_ptr(), _ld(x), w.data_ptr(), _ld(w), w.stride(0), int(trans), N, K,
            _DTYPE[x.dtype], out.data_ptr(), _ld(out), _DTYPE[out.dtype])
    return out


def grouped_wgrad(dy, x, offsets, pairs=None, k=1, out=None, out_dtype=torch.float32):
    """Gradient of the experts' matrices (see moeq_grouped_wgrad): out[e] =
    sum over e's sorted rows r of the outer product of dy[r] and
    x[pairs[r] // k].  dy [P, N] and x [T, K] of one 16-bit type; returns
    [E, N, K] of out_dtype (float32 or that type).  out may not overlap the
    inputs."""
    dev = dy.get_device() if isinstance(dy, torch.Tensor) else -1
    _like(dy, _16BIT, 2, dev, "dy")
    _like(x, (dy.dtype,), 2, dev, "x")
    N, (T, K) = dy.shape[1], x.shape
    E = offsets.shape[0] - 1 if offsets is not None else 1
    g, P = _groups(T, E, offsets, pairs, k, dev)
    if P != dy.shape[0]:
        raise ValueError(f"dy has {dy.shape[0]} rows for {P} sorted rows")
    if N > 0x7fffffff or K > 0x7fffffff:
        _sizes(N=N, K=K)
    out = _out(out, (E, N, K), out_dtype, (dy.dtype, torch.float32), dev, dy)
    _launch("moeq_grouped_wgrad", dev, g, dy.data_ptr(), _ld(dy), x.data_ptr(), _ld(x), N, K, _DTYPE[dy.dtype],
            out.data_ptr(), _ld(out), out.stride(0), _DTYPE[out.dtype])
    return out


def quantize_i8(x):
    """8-bit codes int8 [rows, cols] and fp32 scales [rows] of the rows of x
    (fp16, bf16 or fp32; see moeq_quantize_i8).  A matrix per expert goes in
    as [E, N, K] and gives [E, N, K] and [E, N]."""
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    if isinstance(x, torch.Tensor) and x.dim() == 3:
        q, s = quantize_i8(x.reshape(-1, x.shape[-1]))
        return q.view(x.shape), s.view(x.shape[:2])
    _like(x, _DTYPE, 2, dev, "x")
    _sizes(rows=x.shape[0], cols=x.shape[1])
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    s = torch.empty((x.shape[0],), dtype=torch.float32, device=x.device)
    _launch("moeq_quantize_i8", dev, x.data_ptr(), _ld(x), x.shape[0], x.shape[1], _DTYPE[x.dtype], q.data_ptr(),
            x.shape[1], s.data_ptr())
    return q, s


def _i8_weights(x, wq, sw, dev):
    """(E, N, row and matrix strides) of 8-bit matrices [N, K] or [E, N, K]."""
    _like(wq, (torch.int8,), 3 if isinstance(wq, torch.Tensor) and wq.dim() == 3 else 2, dev, "wq")
    E = wq.shape[0] if wq.dim() == 3 else 1
    N = wq.shape[-2]
    if wq.shape[-1] != x.shape[1]:
        raise ValueError(f"x has {x.shape[1]} columns, wq {wq.shape[-1]}")
    if N > 0x7fffffff or x.shape[1] > 0x7fffffff:
        _sizes(N=N, K=x.shape[1])
    _like(sw, (torch.float32,), wq.dim() - 1, dev, "sw")
    if sw.shape != wq.shape[:-1] or not sw.is_contiguous():
        raise ValueError(f"sw must be contiguous of shape {tuple(wq.shape[:-1])}, got {tuple(sw.shape)}")
    return E, N, _ld(wq), wq.stride(0) if wq.dim() == 3 else 0


def gemm_i8(xq, sx, wq, sw, offsets=None, pairs=None, k=1, out=None, out_dtype=torch.float16):
    """Products of 8-bit codes with their scales (see moeq_gemm_i8): rows xq
    int8 [T, K] with sx fp32 [T]; one matrix wq int8 [N, K] with sw [N], or
    one per expert [E, N, K] with sw [E, N] and the sorted rows of
    grouped_gemm.  Returns [P, N]; out may not overlap the inputs."""
    dev = xq.get_device() if isinstance(xq, torch.Tensor) else -1
    _like(xq, (torch.int8,), 2, dev, "xq")
    T, K = xq.shape
    _flat(sx, T, torch.float32, dev, "sx")
    E, N, ldw, stride_w = _i8_weights(xq, wq, sw, dev)
    g, P = _groups(T, E, offsets, pairs, k, dev)
    out = _out(out, (P, N), out_dtype, _DTYPE, dev, xq)
    _launch("moeq_gemm_i8", dev, g, xq.data_ptr(), _ld(xq), sx.data_ptr(), wq.data_ptr(), ldw, stride_w, sw.data_ptr(),
            N, K, out.data_ptr(), _ld(out), _DTYPE[out.dtype])
    return out


def linear_i8(x, wq, sw, offsets=None, pairs=None, k=1, out=None, out_dtype=None, ws=None):
    """gemm_i8 of the rows x (fp16, bf16 or fp32 [T, K]) coded as by
    quantize_i8 (see moeq_linear_i8).  ws: uint8 workspace tensor, or None
    for one of the call's own; neither it nor out may overlap the inputs.
    Returns [P, N] of out_dtype (x's type).  No autograd, and no gradient of
    its own."""
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    _like(x, _DTYPE, 2, dev, "x")
    T, K = x.shape
    E, N, ldw, stride_w = _i8_weights(x, wq, sw, dev)
    g, P = _groups(T, E, offsets, pairs, k, dev)
    out = _out(out, (P, N), out_dtype or x.dtype, _DTYPE, dev, x)
    if ws is None:
        ws = x.new_empty((linear_i8_workspace_size(T, K),), dtype=torch.uint8)
    else:
        _like(ws, (torch.uint8,), 1, dev, "ws")
    _launch("moeq_linear_i8", dev, g, x.data_ptr(), _ld(x), _DTYPE[x.dtype], wq.data_ptr(), ldw, stride_w, sw.data_ptr(),
            N, K, out.data_ptr(), _ld(out), _DTYPE[out.dtype], ws.data_ptr(), ws.numel())
    return out


@functools.lru_cache(maxsize=1024)
def linear_i8_workspace_size(T, K):
    _sizes(T=T, K=K)
    n = ctypes.c_size_t(0)
    check(lib().moeq_linear_i8_workspace_size(T, K, ctypes.byref(n)), "moeq_linear_i8_workspace_size")
    return n.value


# ------------------------------ routing by scores, rows back to tokens

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


def _name(names, value, what):
    v = names.get(value)
    if v is None:
        raise ValueError(f"{what} must be one of {tuple(names)}, got {value!r}")
    return v


def route_scored(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max", renorm=True,
                 scale=1.0, out=None):
    """Routing of logits [T, E] (fp16, bf16 or fp32) by their scores (see
    moeq_scoring, moeq_route_scored): the k experts with the largest score +
    bias, ties to the lower id, with gates scale * score, divided by the k
    scores' sum with renorm; and the counting sort of route.

    score: "softmax" (over all E) or "sigmoid".  bias: fp32 [E] or None, for
    the choice only.  groups > 1: the experts stand in that many groups of
    consecutive ones, and only the top_groups best groups (default: all) are
    chosen from, by their largest choice (group_score "max") or the sum of
    their two largest ("top2").  A logit of -infinity takes its expert out.
    Returns a RoutingOut (out, if given).  No autograd: the logits' gradient is
    route_scored_grad."""
    dev = logits.get_device() if isinstance(logits, torch.Tensor) else -1
    _like(logits, _DTYPE, 2, dev, "logits")
    T, E = logits.shape
    if bias is not None:
        _flat(bias, E, torch.float32, dev, "bias")
    top_groups = groups if top_groups is None else top_groups
    if T > 0x7fffffff or k > 0x7fffffff or groups > 0x7fffffff or top_groups > 0x7fffffff:
        _sizes(T=T, k=k, groups=groups, top_groups=top_groups)
    d = _lib.Scoring(_name(_SCORES, score, "score"), bool(renorm), scale, _addr(bias), groups, top_groups,
                     _name(_GROUP_SCORES, group_score, "group_score"))
    if out is None:
        out = RoutingOut(T, E, k, logits.device)
    elif (out.T, out.E, out.k) != (T, E, k) or out.ids.get_device() != dev:
        raise ValueError(f"out is a routing of {(out.T, out.E, out.k)}, not of {(T, E, k)} on the logits' device")
    else:
        for t in (out.ids, out.gates, out.offsets, out.sorted_pairs, out.pair_pos):
            _written(t)
    _launch("moeq_route_scored", dev, d, logits.data_ptr(), _ld(logits), _DTYPE[logits.dtype], T, E, k, out.c,
            out.ws_addr(), out.ws_bytes)
    return out


def route_scored_grad(logits, ids, d_gates, score="softmax", renorm=True, scale=1.0, out=None):
    """Gradient of the logits [T, E] from that of the gates (d_gates fp32
    [T, k]) of route_scored's experts ids [T, k] (see moeq_route_scored_grad).
    Returns [T, E] of the logits' type; out may be the logits (in place)."""
    dev = logits.get_device() if isinstance(logits, torch.Tensor) else -1
    _like(logits, _DTYPE, 2, dev, "logits")
    T, E = logits.shape
    _like(ids, (torch.int32,), 2, dev, "ids")
    k = ids.shape[1]
    _dense(ids, (T, k), torch.int32, dev, "ids")
    _dense(d_gates, (T, k), torch.float32, dev, "d_gates")
    if T > 0x7fffffff or E > 0x7fffffff or k > 0x7fffffff:
        _sizes(T=T, E=E, k=k)
    d = _lib.Scoring(_name(_SCORES, score, "score"), bool(renorm), scale, None, 1, 1, 0)
    out = _out(out, (T, E), logits.dtype, (logits.dtype,), dev, logits)
    _launch("moeq_route_scored_grad", dev, d, logits.data_ptr(), _ld(logits), _DTYPE[logits.dtype], T, E, k,
            ids.data_ptr(), d_gates.data_ptr(), out.data_ptr(), _ld(out))
    return out


def _pairs_of(pair_pos, gates, k, dev):
    """(tokens, pairs per token) of the positions pair_pos [T * k]."""
    _like(pair_pos, (torch.int32,), 1, dev, "pair_pos")
    if gates is not None:
        _like(gates, (torch.float32,), 2, dev, "gates")
        if not gates.is_contiguous():
            raise ValueError("gates must be contiguous")
        if k is not None and k != gates.shape[1]:
            raise ValueError(f"k={k} beside gates of shape {tuple(gates.shape)}")
        T, k = gates.shape
    elif k is None or k < 1:
        raise ValueError(f"without gates k must be given and positive, got {k}")
    else:
        T = pair_pos.shape[0] // k
    if T * k != pair_pos.shape[0]:
        raise ValueError(f"pair_pos has {pair_pos.shape[0]} positions, not {k} for each of {T} tokens")
    return T, k


def _beside(dtype):
    """Types of a token's rows beside expert-sorted rows of `dtype`."""
    return tuple(_DTYPE) if dtype == torch.float32 else (dtype, torch.float32)


def combine(rows, pair_pos, gates=None, k=None, base=None, out=None, out_dtype=None):
    """The experts' rows back to their tokens (see moeq_combine): out[t] =
    base[t] + the sum over j < k of gates[t, j] * rows[pair_pos[t * k + j]].

    rows [P, N] fp16, bf16 or fp32 in expert order; pair_pos int32 [T * k] (of
    a routing; a position outside [0, P) adds nothing); gates fp32 [T, k], or
    None (ones) with k given; base [T, N] of out's type or None.  Returns
    [T, N] of out_dtype (base's or the rows' type, or float32; any of the three
    for fp32 rows).  out may be base (in place), and may overlap nothing else.
    No autograd: the gradients are combine_grad."""
    dev = rows.get_device() if isinstance(rows, torch.Tensor) else -1
    _like(rows, _DTYPE, 2, dev, "rows")
    P, N = rows.shape
    T, k = _pairs_of(pair_pos, gates, k, dev)
    out = _out(out, (T, N), out_dtype or (rows.dtype if base is None else base.dtype), _beside(rows.dtype), dev, rows)
    if base is not None:
        _like(base, (out.dtype,), 2, dev, "base")
        if base.shape != out.shape:
            raise ValueError(f"base must have shape {tuple(out.shape)}, got {tuple(base.shape)}")
    if P > 0x7fffffff or T > 0x7fffffff or N > 0x7fffffff:
        _sizes(P=P, T=T, N=N)
    _launch("moeq_combine", dev, rows.data_ptr(), _ld(rows), P, _DTYPE[rows.dtype], pair_pos.data_ptr(), _addr(gates), T, k,
            N, _addr(base), _ld(base) if base is not None else 0, out.data_ptr(), _ld(out), _DTYPE[out.dtype])
    return out


def combine_grad(dy, pair_pos, gates=None, rows=None, k=None, out=None, out_dtype=None):
    """Gradients of combine's inputs from that of its output, dy [T, N] (see
    moeq_combine_grad): (d_rows, d_gates) with d_rows[pair_pos[p]] = gates[p] *
    dy[p // k] and d_gates[p] = dy[p // k] . rows[pair_pos[p]].

    rows [P, N] as combine took them, or None: P = T * k (or out's rows), and
    d_gates is None, as it is without gates.  d_rows has the rows' type (out_dtype, or dy's,
    without rows); rows of it that no pair points at are left as they were
    (undefined in a new tensor).  No position may occur twice.  The gradient of
    base is dy.  out may not overlap the inputs."""
    dev = dy.get_device() if isinstance(dy, torch.Tensor) else -1
    _like(dy, _DTYPE, 2, dev, "dy")
    T, k = _pairs_of(pair_pos, gates, k, dev)
    N = dy.shape[1]
    if dy.shape[0] != T:
        raise ValueError(f"dy has {dy.shape[0]} rows for {T} tokens")
    dtype = rows.dtype if rows is not None else out_dtype or (out.dtype if out is not None else dy.dtype)
    if rows is not None:
        _like(rows, _DTYPE, 2, dev, "rows")
        if rows.shape[1] != N:
            raise ValueError(f"rows have {rows.shape[1]} columns, dy {N}")
        if out_dtype not in (None, dtype):
            raise TypeError(f"d_rows has the rows' type {dtype}, not {out_dtype}")
    if dtype not in _DTYPE or dy.dtype not in _beside(dtype):
        raise TypeError(f"dy of {dy.dtype} beside rows of {dtype}")
    P = rows.shape[0] if rows is not None else T * k if out is None else out.shape[0]
    out = _out(out, (P, N), dtype, (dtype,), dev, dy)
    d_gates = torch.empty_like(gates) if rows is not None and gates is not None else None
    if P > 0x7fffffff or T > 0x7fffffff or N > 0x7fffffff:
        _sizes(P=P, T=T, N=N)
    _launch("moeq_combine_grad", dev, dy.data_ptr(), _ld(dy), _DTYPE[dy.dtype], pair_pos.data_ptr(), _addr(gates), T, k, N,
            _addr(rows), _ld(rows) if rows is not None else 0, P, _DTYPE[dtype], out.data_ptr(), _ld(out), _addr(d_gates))
    return out, d_gates


# ------------------------------------------------- adapters of requests

def adapters(x, a, b, ids, y, scale=None, ranks=None, out=None, ws=None):
    """Low-rank adapters of the rows' requests beside a projection y of the
    rows x (see moeq_adapters): out[r] = y[r] + scale[i] * b[i] @ (a[i] @ x[r])
    for i = ids[r], and y[r] where ids[r] is no adapter (-1, say).

    x fp16 or bf16 [T, K]; a [n, R, K] and b [n, N, R] of the same type; ids
    int32 [T]; y [T, N] of that type or float32 (linear_i8 or grouped_gemm of
    the same x, or the expert layer's); scale fp32 [n] or None (ones); ranks
    int32 [n] or None (R): how much of R counts, finite in b.  Returns [T, N] of
    y's type; out may be y (in place).  ws: uint8 workspace tensor, or None for
    one of the call's own; neither it nor out may overlap the other inputs.  No
    autograd, and no gradient of its own."""
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    _like(x, _16BIT, 2, dev, "x")
    dtype, (T, K) = x.dtype, x.shape
    _like(a, (dtype,), 3, dev, "a")
    _like(b, (dtype,), 3, dev, "b")
    (n, R, Ka), N = a.shape, b.shape[1]
    if Ka != K or b.shape[0] != n or b.shape[2] != R:
        raise ValueError(f"a of {tuple(a.shape)} and b of {tuple(b.shape)} are no adapters for {K} columns")
    _flat(ids, T, torch.int32, dev, "ids")
    _like(y, (dtype, torch.float32), 2, dev, "y")
    if y.shape[0] != T or y.shape[1] != N:
        raise ValueError(f"y must have shape {(T, N)}, got {tuple(y.shape)}")
    if scale is not None:
        _flat(scale, n, torch.float32, dev, "scale")
    if ranks is not None:
        _flat(ranks, n, torch.int32, dev, "ranks")
    out = _out(out, (T, N), y.dtype, (y.dtype,), dev, y)
    if ws is None:
        ws = x.new_empty((adapters_workspace_size(T, R, K),), dtype=torch.uint8)
    else:
        _like(ws, (torch.uint8,), 1, dev, "ws")
    if n > 0x7fffffff or N > 0x7fffffff:
        _sizes(n=n, N=N)
    s = _lib.AdaptersSet(a.data_ptr(), b.data_ptr(), _ld(a), a.stride(0), _ld(b), b.stride(0), _addr(scale), _addr(ranks), n, R,
                         N, K, _DTYPE[dtype])
    _launch("moeq_adapters", dev, s, x.data_ptr(), _ld(x), ids.data_ptr(), T, y.data_ptr(), _ld(y), out.data_ptr(), _ld(out),
            _DTYPE[y.dtype], ws.data_ptr(), ws.numel())
    return out


@functools.lru_cache(maxsize=1024)
def adapters_workspace_size(T, R, K):
    _sizes(T=T, R=R, K=K)
    n = ctypes.c_size_t(0)
    check(lib().moeq_adapters_workspace_size(T, R, K, ctypes.byref(n)), "moeq_adapters_workspace_size")
    return n.value


# ------------------------------------------------ norms around a block

def _dense(t, shape, dtype, dev, name):
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0 and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device than the other tensors")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _addr(t):
    return t.data_ptr() if t is not None else None


def _norm(res, dtype, y, w_pre, w_post, gate, alpha, eps, post_norm, dev):
    """moeq_norm of the checked operands."""
    T, H = res.shape
    if dtype not in _DTYPE:
        raise TypeError(f"{dtype} is not a type of the norms")
    if T > 0x7fffffff or H > 0x7fffffff:
        _sizes(T=T, H=H)
    vec = (H,)
    if y is not None:
        _dense(y, res.shape, dtype, dev, "y")
    if w_pre is not None:
        _dense(w_pre, vec, dtype, dev, "w_pre")
    if w_post is not None:
        _dense(w_post, vec, dtype, dev, "w_post")
    per_token = gate is not None and gate.dim() == 2
    if gate is not None:
        _dense(gate, res.shape if per_token else vec, dtype, dev, "gate")
    return _lib.Norm(T, H, _DTYPE[dtype], _DTYPE[res.dtype], _addr(w_pre), _addr(w_post), _addr(gate), per_token,
                     bool(post_norm), alpha, eps)


def _res(res, name):
    """Device index of a residual [T, H]."""
    if not isinstance(res, torch.Tensor) or not res.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if res.dim() != 2 or res.dtype not in _DTYPE:
        raise TypeError(f"{name} must be [T, H] of fp16, bf16 or fp32, got {tuple(res.shape)} {res.dtype}")
    if not res.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return res.get_device()


def block_norm(residual, y=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=1e-6, post_norm=True,
               res_out=None, n_out=None):
    """The norms between two blocks (see moeq_block_norm): returns (r', n)
    with r' = alpha * residual + gate * (w_post * y / rms(y)) (y itself in
    place of its norm without post_norm) and n = w_pre * r' / rms(r').

    residual [T, H] (y's type or float32); y [T, H] fp16, bf16 or fp32, or
    None (r' is the residual itself, n of w_pre's type); w_pre, w_post [H],
    gate [H] or [T, H] of y's type, or None (ones).  res_out may be the
    residual and n_out may be y (in place); no other operands may overlap.  The
    low-bit expert layer takes fp16 only: beside it, y and n are fp16 (the
    residual may be float32).  No autograd: the gradients are
    block_norm_grad."""
    dev = _res(residual, "residual")
    dtype = y.dtype if y is not None else w_pre.dtype if w_pre is not None else residual.dtype
    d = _norm(residual, dtype, y, w_pre, w_post, gate, alpha, eps, post_norm, dev)
    if y is None:
        if res_out is not None:
            raise ValueError("res_out is not written without y")
        r = residual
    elif res_out is None:
        r = torch.empty_like(residual)
    else:
        r = res_out
        _dense(r, residual.shape, residual.dtype, dev, "res_out")
        _written(r)
    if n_out is None:
        n = torch.empty_like(residual if y is None else y, dtype=dtype)
    else:
        n = n_out
        _dense(n, residual.shape, dtype, dev, "n_out")
        _written(n)
    _launch("moeq_block_norm", dev, d, residual.data_ptr(), _addr(y), r.data_ptr(), n.data_ptr())
    return r, n


def block_norm_grad(res, d_n, y=None, d_res=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=1e-6,
                    post_norm=True, ws=None):
    """Gradients of block_norm's inputs (see moeq_block_norm_grad) from those
    of its outputs r' (d_res, or None) and n (d_n); res is the r' that it
    returned.  Returns a dict: d_residual, and d_y, d_w_pre, d_w_post (fp32),
    d_gate (fp32 [H], or [T, H] of the gate's type) for the inputs given.
    ws: uint8 workspace tensor, or None for one of the call's own."""
    dev = _res(res, "res")
    if not isinstance(d_n, torch.Tensor):
        raise TypeError("d_n must be a CUDA tensor")
    d = _norm(res, d_n.dtype, y, w_pre, w_post, gate, alpha, eps, post_norm, dev)
    T, H = res.shape
    _dense(d_n, res.shape, d_n.dtype, dev, "d_n")
    if d_res is not None:
        _dense(d_res, res.shape, res.dtype, dev, "d_res")
    out = {"d_residual": torch.empty_like(res)}
    if y is not None:
        out["d_y"] = torch.empty_like(y)
    if w_pre is not None:
        out["d_w_pre"] = torch.empty((H,), dtype=torch.float32, device=res.device)
    if w_post is not None:
        out["d_w_post"] = torch.empty((H,), dtype=torch.float32, device=res.device)
    if gate is not None:
        out["d_gate"] = torch.empty(gate.shape, dtype=gate.dtype if gate.dim() == 2 else torch.float32, device=res.device)
    if ws is None:
        ws = res.new_empty((block_norm_grad_workspace_size(T, H),), dtype=torch.uint8)
    else:
        _like(ws, (torch.uint8,), 1, dev, "ws")
    _launch("moeq_block_norm_grad", dev, d, res.data_ptr(), _addr(y), _addr(d_res), d_n.data_ptr(),
            _addr(out["d_residual"]), _addr(out.get("d_y")), _addr(out.get("d_w_pre")), _addr(out.get("d_w_post")),
            _addr(out.get("d_gate")), ws.data_ptr(), ws.numel())
    return out


@functools.lru_cache(maxsize=1024)
def block_norm_grad_workspace_size(T, H):
    _sizes(T=T, H=H)
    n = ctypes.c_size_t(0)
    check(lib().moeq_block_norm_grad_workspace_size(T, H, ctypes.byref(n)), "moeq_block_norm_grad_workspace_size")
    return n.value


# ------------------------------------------------------------ profiling

def profile_enable(on=True):
    check(lib().moeq_profile_enable(1 if on else 0), "moeq_profile_enable")


def profile_read(max_kernels=64):
    names = (ctypes.c_char_p * max_kernels)()
    launches = (ctypes.c_int32 * max_kernels)()
    ms = (ctypes.c_double * max_kernels)()
    n = ctypes.c_int32(0)
    check(lib().moeq_profile_read(max_kernels, names, launches, ms, ctypes.byref(n)), "moeq_profile_read")
    return {names[i].decode(): (int(launches[i]), float(ms[i])) for i in range(min(n.value, max_kernels))}
