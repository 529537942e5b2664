"""ctypes binding of libspc (include/spc.h): argument marshalling only.

Each function here has the name of the C entry point it wraps, takes torch
tensors that already live on the GPU, allocates the outputs and the workspace
with torch (device memory is all torch provides) and passes raw pointers and
the current HIP stream to the library.  Every step of the computation runs in
the library's HIP kernels; there is no CPU or PyTorch fallback, and a missing
``libspc.so`` raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspc.so")

SPC_OK, SPC_ERR_ARG, SPC_ERR_UNSUPPORTED, SPC_ERR_CAPACITY, SPC_ERR_COORD, SPC_ERR_WORKSPACE, SPC_ERR_HIP = range(7)
COORD_OUT_OF_RANGE, COORD_DUPLICATE = 1, 2
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_STATUS = {1: "SPC_ERR_ARG", 2: "SPC_ERR_UNSUPPORTED", 3: "SPC_ERR_CAPACITY", 4: "SPC_ERR_COORD",
           5: "SPC_ERR_WORKSPACE", 6: "SPC_ERR_HIP"}

EXPORTS = ("spc_out_shape", "spc_kmap_workspace", "spc_build_kmap", "spc_build_kmap_async", "spc_subm_conv_fwd",
           "spc_sparse_conv_fwd", "spc_sparse_inverse_conv_fwd", "spc_conv_fwd_fused", "spc_transpose_weight",
           "spc_conv_fwd_wt", "spc_conv_fwd_dev_rows", "spc_conv_bwd_input",
           "spc_conv_bwd_filter_workspace",
           "spc_conv_bwd_filter", "spc_conv_bwd_filter_noalloc", "spc_sparse_maxpool_fwd", "spc_sparse_maxpool_bwd",
           "spc_point_to_voxel_workspace", "spc_point_to_voxel", "spc_gather_by_voxel_id", "spc_dropout_fwd",
           "spc_dropout_bwd", "spc_group_norm_workspace", "spc_group_norm_fwd", "spc_group_norm_bwd",
           "spc_linear_recurrence_workspace", "spc_linear_recurrence_fwd", "spc_linear_recurrence_bwd",
           "spc_linear_recurrence_step", "spc_layer_norm_workspace", "spc_layer_norm_fwd", "spc_layer_norm_bwd",
           "spc_rotary", "spc_attention_workspace", "spc_attention_fwd", "spc_attention_bwd", "spc_calibrate_mfma",
           "spc_last_error", "spc_version")


class SpcError(RuntimeError):
    def __init__(self, status: int, func: str, msg: str):
        super().__init__(f"{func}: {_STATUS.get(status, status)}: {msg}")
        self.status = status


class Geom(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("shape", ctypes.c_int32 * 3), ("ksize", ctypes.c_int32 * 3),
                ("stride", ctypes.c_int32 * 3), ("pad", ctypes.c_int32 * 3), ("dil", ctypes.c_int32 * 3),
                ("subm", ctypes.c_int32), ("table", ctypes.c_int32)]


class _DropArg(ctypes.Structure):
    _fields_ = [("rng", ctypes.c_void_p), ("layer", ctypes.c_uint32), ("p", ctypes.c_float)]


class _AttnArg(ctypes.Structure):
    _fields_ = [("n_q", ctypes.c_int64), ("n_kv", ctypes.c_int64), ("n_seg", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("scale", ctypes.c_float), ("q_ptr", ctypes.c_void_p), ("kv_ptr", ctypes.c_void_p),
                ("q_order", ctypes.c_void_p), ("kv_order", ctypes.c_void_p)]


TABLES = {"hash": 0, "grid": 1}   # SPC_TABLE_HASH, SPC_TABLE_GRID


def _t3(v) -> tuple:
    if isinstance(v, int):
        return (v, v, v)
    v = tuple(int(a) for a in v)
    if len(v) != 3:
        raise ValueError("expected an int or 3 ints")
    return v


def make_geom(batch: int, shape, ksize, stride=1, pad=0, dil=1, subm: bool = True, table: str = "hash") -> Geom:
    a = lambda v: (ctypes.c_int32 * 3)(*_t3(v))
    if table not in TABLES:
        raise ValueError(f"table must be one of {tuple(TABLES)}, got {table!r}")
    return Geom(int(batch), a(shape), a(ksize), a(stride), a(pad), a(dil), 1 if subm else 0, TABLES[table])


_lib = None
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """The loaded libspc.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m sparse_convolution_hash_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    GP, DP, AP = ctypes.POINTER(Geom), ctypes.POINTER(_DropArg), ctypes.POINTER(_AttnArg)
    sig = {
        "spc_out_shape": [GP, ctypes.POINTER(_I32)],
        "spc_kmap_workspace": [GP, _I64, ctypes.POINTER(_SZ)],
        "spc_build_kmap": [GP, _P, _I64, _P, _I64, ctypes.POINTER(_I64), _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P,
                           _SZ, _P],
        "spc_build_kmap_async": [GP, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _SZ, _P],
        "spc_subm_conv_fwd": [_I32, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P],
        "spc_sparse_conv_fwd": [_I32, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _I64, _P, _P],
        "spc_sparse_inverse_conv_fwd": [_I32, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _I64, _P, _P],
        "spc_conv_fwd_fused": [_I32, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _I64, _P, _I32, _P, _P],
        "spc_transpose_weight": [_I32, _P, _I32, _I32, _I32, _P, _P],
        "spc_conv_fwd_wt": [_I32, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _I32, _P, _I64, _P, _I32, _P, _P],
        "spc_conv_fwd_dev_rows": [_I32, _P, _I64, _I32, _P, _I32, _I32, _I32, _P, _P, _P, _I64, _P, _P, _I32, _P,
                                  _P],
        "spc_conv_bwd_input": [_I32, _P, _I64, _I32, _P, _I32, _I32, _P, _I32, _P, _I64, _P, _P],
        "spc_conv_bwd_filter_workspace": [_I64, _I64, _I32, _I32, _I32, _I32, ctypes.POINTER(_SZ)],
        "spc_conv_bwd_filter": [_I32, _P, _I64, _I32, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P],
        "spc_conv_bwd_filter_noalloc": [_I32, _P, _I64, _I32, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P],
        "spc_sparse_maxpool_fwd": [_I32, _P, _I64, _I32, _P, _I32, _I64, _P, _P, _P],
        "spc_sparse_maxpool_bwd": [_I32, _P, _I64, _I32, _P, _P, _I32, _I64, _P, _P],
        "spc_point_to_voxel_workspace": [_I64, _I32, _I64, _I32, ctypes.POINTER(_SZ)],
        "spc_point_to_voxel": [_P, _I64, _I32, _P, _P, _I64, _I32, _I32, _P, _P, _P, _P,
                               ctypes.POINTER(ctypes.c_int64), _P, _SZ, _P],
        "spc_gather_by_voxel_id": [_I32, _P, _I64, _I32, _P, _I64, _P, _P],
        "spc_dropout_fwd": [_I32, _P, _I64, _P, DP, _P, _P],
        "spc_dropout_bwd": [_I32, _P, _I64, DP, _P, _P],
        "spc_group_norm_workspace": [_I64, _I32, _I32, _I64, ctypes.POINTER(_SZ)],
        "spc_group_norm_fwd": [_I32, _P, _I64, _I32, _I32, _P, _I64, _P, _P, ctypes.c_float, _I32, DP, _P, _P, _P, _SZ,
                               _P],
        "spc_group_norm_bwd": [_I32, _P, _P, _I64, _I32, _I32, _P, _I64, _P, _P, _P, _I32, DP, _P, _P, _P, _P, _SZ, _P],
        "spc_linear_recurrence_workspace": [_I32, _I64, _I32, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)],
        "spc_linear_recurrence_fwd": [_I32, _P, _P, _I64, _I64, _I32, _P, _I64, _P, _I32, _P, _P, _P, _P, _P, _SZ, _P],
        "spc_linear_recurrence_bwd": [_I32, _P, _P, _P, _I64, _I64, _I32, _P, _I64, _P, _I32, _P, _P, _P, _P, _P, _I64,
                                      _P, _P, _SZ, _P],
        "spc_linear_recurrence_step": [_I32, _P, _P, _I64, _I64, _I32, _P, _P, _P, _P],
        "spc_layer_norm_workspace": [_I64, _I32, ctypes.POINTER(_SZ)],
        "spc_layer_norm_fwd": [_I32, _P, _P, _I64, _I32, _P, _P, ctypes.c_float, _P, _P, _P, _P],
        "spc_layer_norm_bwd": [_I32, _P, _P, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ, _P],
        "spc_rotary": [_I32, _P, _I64, _I64, _I32, _I32, _P, _I64, _I32, _P, _P, _I32, _P, _I64, _P],
        "spc_attention_workspace": [_I32, AP, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)],
        "spc_attention_fwd": [_I32, AP, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _SZ, _P],
        "spc_attention_bwd": [_I32, AP, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _P,
                              _I64, _P, _SZ, _P],
        "spc_calibrate_mfma": [_I32, _I32, _I32, _P, ctypes.POINTER(ctypes.c_double), _P],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    for name in ("spc_last_error", "spc_version"):
        f = getattr(L, name)
        f.argtypes = []
        f.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(status: int, func: str):
    if status != SPC_OK:
        raise SpcError(status, func, lib().spc_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev: torch.device):
    """The current stream's handle on `dev` (torch's raw accessor when it has
    one: a Stream object per call costs host time on every launch)."""
    if _raw_stream is not None:
        return _raw_stream(dev.index if dev.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(dev).cuda_stream


def _call(dev: torch.device, f, *args) -> int:
    """f(*args, stream) on the current stream of `dev`, which need not be the
    current device."""
    if dev.index == torch.cuda.current_device():
        return f(*args, _stream(dev))
    with torch.cuda.device(dev):
        return f(*args, _stream(dev))


def _need(t: torch.Tensor, name: str, dtype=None, dev=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _scratch(workspace, need: int, like: torch.Tensor, least: int = 0):
    """The caller's workspace where it holds ``need`` bytes, else a new one of
    them (``least`` at least; none for 0) on the device of ``like``."""
    if workspace is not None:
        _need(workspace, "workspace", None, like.device)
        if workspace.numel() >= need:
            return workspace
    need = max(need, least)
    return like.new_empty((need,), dtype=torch.uint8) if need else None


def version() -> str:
    return lib().spc_version().decode()


def out_shape(batch, shape, ksize, stride=1, pad=0, dil=1, subm=False) -> tuple:
    g = make_geom(batch, shape, ksize, stride, pad, dil, subm)
    o = (ctypes.c_int32 * 3)()
    _check(lib().spc_out_shape(ctypes.byref(g), o), "spc_out_shape")
    return tuple(o)


def kmap_workspace(g: Geom, n_in: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().spc_kmap_workspace(ctypes.byref(g), int(n_in), ctypes.byref(b)), "spc_kmap_workspace")
    return b.value


@functools.lru_cache(maxsize=256)
def _kmap_plan(batch, shape, ksize, stride, pad, dil, subm, n_in, table):
    """(Geom, K, workspace bytes) of a kernel-map call; the Geom is shared and
    never modified."""
    g = make_geom(batch, shape, ksize, stride, pad, dil, subm, table)
    return g, int(g.ksize[0] * g.ksize[1] * g.ksize[2]), kmap_workspace(g, n_in)


def strided_out_bound(n_in: int, batch: int, shape, ksize, stride=1, pad=0, dil=1) -> int:
    """Upper bound of a strided map's output-site count that follows from the
    geometry alone (the role of spconv's ``out_inds_num_limit``): along an
    axis the offsets k*dil, k < ksize, reach an exact multiple of the stride at
    most ceil(ksize / (stride / gcd(stride, dil))) times, so an input feeds at
    most the product of those over the axes; and never more than the output
    grid holds."""
    import math
    ks, st, dl = _t3(ksize), _t3(stride), _t3(dil)
    per = 1
    for k, s, d in zip(ks, st, dl):
        per *= -(-k // (s // math.gcd(s, d)))
    vol = int(batch)
    for o in out_shape(batch, shape, ksize, stride, pad, dil, subm=False):
        vol *= max(o, 0)
    return int(min(int(n_in) * per, vol))


def build_kmap(coords: torch.Tensor, batch: int, shape: Sequence[int], ksize, stride=1, pad=0, dil=1,
               subm: bool = True, pairs: bool = True, with_nbr_in: bool = True, orders: bool = False,
               out_cap: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
               table: str = "hash", count_first: bool = False, device_count: bool = False) -> dict:
    """Kernel map of int32 [N, 4] (b, z, y, x) coordinates (spc_build_kmap).

    Returns a dict with ``nbr`` [n_out, K] (submanifold neighbour map or the
    strided output-side map, row-major), ``n_out``, ``coord_err`` (device
    int32 [1]) and, as requested, ``out_coords`` [n_out, 4], ``nbr_in`` [N, K],
    the CSR pair lists ``pair_ptr`` [K+1], ``pair_in`` / ``pair_out`` (first
    pair_ptr[K] entries valid) and the processing orders ``order`` (rows of
    nbr) and ``order_in`` (rows of nbr_in).  A strided call without
    ``out_cap`` sizes its outputs by ``strided_out_bound`` (one library call,
    which returns the count M; the result views hold M rows), or with
    ``count_first`` asks the library for M first and allocates exactly (two
    calls).  ``table`` picks the input table: ``"hash"`` (default) or
    ``"grid"`` (occupancy bitmap + index grid over the whole input grid, 4.125
    bytes of workspace per cell); the results are the same.

    ``device_count`` calls spc_build_kmap_async instead, which never waits:
    the result then holds ``n_out_dev`` (device int32 [1], the row count M in
    stream order), ``n_cap`` (the row capacity, out_cap or the bound) and
    ``n_out`` = None; ``nbr``, ``out_coords`` and ``order`` span n_cap rows,
    of which the first M are valid.  Bad coordinates then show only in
    ``coord_err``, and M > n_cap means the map holds no rows.
    """
    _need(coords, "coords", torch.int32)
    if coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be [N, 4]")
    dev = coords.device
    n = coords.shape[0]
    key = lambda v: v if isinstance(v, int) else tuple(v)
    g, K, ws_bytes = _kmap_plan(int(batch), key(shape), key(ksize), key(stride), key(pad), key(dil), bool(subm), n,
                                table)
    stream = _stream(dev)
    n_out = ctypes.c_int64(0)
    if not subm and out_cap is None and not count_first:
        out_cap = strided_out_bound(n, batch, shape, ksize, stride, pad, dil)
    if device_count and out_cap is None and not subm:
        raise ValueError("device_count needs out_cap (count_first waits for the count)")
    if not subm and out_cap is None:
        ws = _scratch(workspace, ws_bytes, coords, 256)
        st = lib().spc_build_kmap(ctypes.byref(g), coords.data_ptr(), n, None, 0, ctypes.byref(n_out), None, None,
                                  None, None, None, 0, None, None, None, ws.data_ptr(), ws.numel(), stream)
        _check(st, "spc_build_kmap")
        out_cap = n_out.value
        workspace = ws
    cap = n if subm else int(out_cap)
    # every int32 output in one allocation (each part starts 256-byte aligned)
    # and the workspace in a second one, which the results do not keep alive;
    # the library gets raw addresses, and the result views are made afterwards
    parts = [("err", 4), ("nbr", max(K * cap, 4))]
    if device_count:
        parts.append(("nout", 4))
    if not subm:
        parts.append(("out_coords", max(cap, 1) * 4))
    want_nbr_in = not subm and (with_nbr_in or orders)
    if want_nbr_in:
        parts.append(("nbr_in", max(n * K, 4)))
    if orders:
        parts.append(("order", max(cap, 4)))
        if not subm:
            parts.append(("order_in", max(n, 4)))
    if pairs:
        parts += [("pp", K + 1), ("pi", max(K * n, 4)), ("po", max(K * n, 4))]
    sizes = []
    for _, v in parts:
        sizes += [v, (-v) % 64]
    workspace = _scratch(workspace, ws_bytes, coords, 256)
    buf = torch.empty(sum(sizes), dtype=torch.int32, device=dev)
    base, addr, o = buf.data_ptr(), {}, 0
    for i, (name, _) in enumerate(parts):
        addr[name] = base + 4 * o
        o += sizes[2 * i] + sizes[2 * i + 1]
    a = addr.get
    if device_count:
        st = lib().spc_build_kmap_async(ctypes.byref(g), coords.data_ptr(), n, a("out_coords"), cap, a("nout"),
                                        a("nbr"), a("nbr_in"), a("pp"), a("pi"), a("po"),
                                        max(K * n, 0) if pairs else 0, a("order"), a("order_in"), a("err"),
                                        workspace.data_ptr(), workspace.numel(), stream)
        _check(st, "spc_build_kmap_async")
        m = cap
    else:
        st = lib().spc_build_kmap(ctypes.byref(g), coords.data_ptr(), n, a("out_coords"), cap, ctypes.byref(n_out),
                                  a("nbr"), a("nbr_in"), a("pp"), a("pi"), a("po"), max(K * n, 0) if pairs else 0,
                                  a("order"), a("order_in"), a("err"), workspace.data_ptr(), workspace.numel(), stream)
        _check(st, "spc_build_kmap")
        m = int(n_out.value)
    views = dict(zip((name for name, _ in parts), buf.split_with_sizes(sizes)[0::2]))
    res = {"coord_err": views["err"][:1], "n_out": None if device_count else m, "nbr": views["nbr"][:K * m].view(m, K)}
    if device_count:
        res["n_out_dev"], res["n_cap"] = views["nout"][:1], cap
    if not subm:
        res["out_coords"] = views["out_coords"][:4 * m].view(m, 4)
    if want_nbr_in:
        res["nbr_in"] = views["nbr_in"][:n * K].view(n, K)
    if orders:
        res["order"] = views["order"][:m]
        if not subm:
            res["order_in"] = views["order_in"][:n]
    if pairs:
        res["pair_ptr"], res["pair_in"], res["pair_out"] = views["pp"], views["pi"], views["po"]
    return res


def _conv_checks(x, weight, bias, dev):
    _need(x, "input", dev=dev)
    _need(weight, "weight", x.dtype, dev)
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if weight.dim() != 3:
        raise ValueError("weight must be [K, Cin, Cout]")
    if bias is not None:
        _need(bias, "bias", torch.float32, dev)


def _pretranspose(dtype, cin: int, flag) -> bool:
    """Whether a forward hands the kernel pre-transposed weights: for fp32
    and for contractions of more than 64 16-bit channels, where staging W's
    own layout would transpose every offset's weights once per tile (shorter
    16-bit contractions read W's own layout with transposing LDS reads)."""
    if flag is not None:
        return bool(flag)
    return dtype == torch.float32 or cin > 64


def transpose_weight(weight: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """weight [K, cin, cout] -> [K, cout, cin] on the device (spc_transpose_weight)."""
    _need(weight, "weight")
    if weight.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {weight.dtype}")
    if weight.dim() != 3:
        raise ValueError("weight must be [K, Cin, Cout]")
    K, cin, cout = weight.shape
    if out is None:
        out = torch.empty((K, cout, cin), dtype=weight.dtype, device=weight.device)
    else:
        _need(out, "out", weight.dtype, weight.device)
        if tuple(out.shape) != (K, cout, cin):
            raise ValueError(f"out must be [{K}, {cout}, {cin}], got {tuple(out.shape)}")
    st = lib().spc_transpose_weight(_DTYPES[weight.dtype], _ptr(weight), K, cin, cout, _ptr(out),
                                    _stream(weight.device))
    _check(st, "spc_transpose_weight")
    return out


def conv_fwd_wt(feats: torch.Tensor, weight_t: torch.Tensor, bias: Optional[torch.Tensor],
                map_: Optional[torch.Tensor], n_rows: int, map_is_subm: bool = False,
                order: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                relu: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Forward with pre-transposed weights weight_t [K, Cout, Cin] (spc_conv_fwd_wt);
    otherwise as conv_fwd_fused."""
    dev = feats.device
    _conv_checks(feats, weight_t, bias, dev)
    for t, nm in ((map_, "map"), (order, "order")):
        if t is not None:
            _need(t, nm, torch.int32, dev)
    K, cout, cin = weight_t.shape
    if residual is not None:
        _need(residual, "residual", feats.dtype, dev)
        if tuple(residual.shape) != (n_rows, cout):
            raise ValueError(f"residual must be [{n_rows}, {cout}], got {tuple(residual.shape)}")
    if out is None:
        out = torch.empty((n_rows, cout), dtype=feats.dtype, device=dev)
    st = lib().spc_conv_fwd_wt(_DTYPES[feats.dtype], _ptr(feats), feats.shape[0], cin, _ptr(weight_t), K, cout,
                               _ptr(bias), _ptr(map_), 1 if map_is_subm else 0, _ptr(order), int(n_rows),
                               _ptr(residual), 1 if relu else 0, _ptr(out), _stream(dev))
    _check(st, "spc_conv_fwd_wt")
    return out


def conv_fwd_dev_rows(feats: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                      map_: torch.Tensor, n_rows_dev: torch.Tensor, row_cap: int,
                      order: Optional[torch.Tensor] = None, weight_t: bool = False,
                      residual: Optional[torch.Tensor] = None, relu: bool = False,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Forward over the rows of a strided map built with device_count
    (spc_conv_fwd_dev_rows): out [row_cap, Cout], of which the first
    n_rows_dev rows are written.  ``weight`` is [K, Cin, Cout], or [K, Cout,
    Cin] from transpose_weight when ``weight_t``."""
    dev = feats.device
    _conv_checks(feats, weight, bias, dev)
    _need(map_, "map", torch.int32, dev)
    _need(n_rows_dev, "n_rows_dev", torch.int32, dev)
    if order is not None:
        _need(order, "order", torch.int32, dev)
    K = weight.shape[0]
    cin, cout = (weight.shape[2], weight.shape[1]) if weight_t else (weight.shape[1], weight.shape[2])
    if residual is not None:
        _need(residual, "residual", feats.dtype, dev)
        if tuple(residual.shape) != (row_cap, cout):
            raise ValueError(f"residual must be [{row_cap}, {cout}], got {tuple(residual.shape)}")
    if out is None:
        out = torch.empty((row_cap, cout), dtype=feats.dtype, device=dev)
    st = lib().spc_conv_fwd_dev_rows(_DTYPES[feats.dtype], _ptr(feats), feats.shape[0], cin, _ptr(weight),
                                     1 if weight_t else 0, K, cout, _ptr(bias), _ptr(map_), _ptr(order),
                                     int(row_cap), _ptr(n_rows_dev), _ptr(residual), 1 if relu else 0, _ptr(out),
                                     _stream(dev))
    _check(st, "spc_conv_fwd_dev_rows")
    return out


def subm_conv_fwd(feats: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                  nbr: Optional[torch.Tensor], order: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, pretranspose: Optional[bool] = None) -> torch.Tensor:
    """out[c] = bias + sum_k feats[nbr[c, k]] @ W[k] (spc_subm_conv_fwd, or
    spc_transpose_weight + spc_conv_fwd_wt when `pretranspose`, by default
    for fp32 and Cin > 64: the same result bit for bit)."""
    dev = feats.device
    _conv_checks(feats, weight, bias, dev)
    K, cin, cout = weight.shape
    n = feats.shape[0]
    for t, nm in ((nbr, "nbr"), (order, "order")):
        if t is not None:
            _need(t, nm, torch.int32, dev)
    if _pretranspose(feats.dtype, cin, pretranspose):
        if K > 1 and nbr is None:
            raise ValueError("nbr is required for K > 1")
        return conv_fwd_wt(feats, transpose_weight(weight), bias, nbr if K > 1 else None, n, K > 1,
                           order if K > 1 else None, out=out)
    if out is None:
        out = torch.empty((n, cout), dtype=feats.dtype, device=dev)
    st = lib().spc_subm_conv_fwd(_DTYPES[feats.dtype], _ptr(feats), n, cin, _ptr(weight), K, cout, _ptr(bias),
                                 _ptr(nbr), _ptr(order), _ptr(out), _stream(dev))
    _check(st, "spc_subm_conv_fwd")
    return out


def sparse_conv_fwd(feats: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                    nbr_out: torch.Tensor, n_out: int, order: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, pretranspose: Optional[bool] = None) -> torch.Tensor:
    """Strided forward over the n_out output rows of a strided kernel map
    (spc_sparse_conv_fwd; `pretranspose` as for subm_conv_fwd)."""
    dev = feats.device
    _conv_checks(feats, weight, bias, dev)
    _need(nbr_out, "nbr_out", torch.int32, dev)
    if order is not None:
        _need(order, "order", torch.int32, dev)
    K, cin, cout = weight.shape
    if _pretranspose(feats.dtype, cin, pretranspose):
        return conv_fwd_wt(feats, transpose_weight(weight), bias, nbr_out, n_out, False, order, out=out)
    if out is None:
        out = torch.empty((n_out, cout), dtype=feats.dtype, device=dev)
    st = lib().spc_sparse_conv_fwd(_DTYPES[feats.dtype], _ptr(feats), feats.shape[0], cin, _ptr(weight), K, cout,
                                   _ptr(bias), _ptr(nbr_out), _ptr(order), int(n_out), _ptr(out), _stream(dev))
    _check(st, "spc_sparse_conv_fwd")
    return out


def sparse_inverse_conv_fwd(feats: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                            nbr_in: torch.Tensor, n_fine: int, order_in: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None,
                            pretranspose: Optional[bool] = None) -> torch.Tensor:
    """Inverse (upsampling) forward onto the input sites of a strided kernel map
    (spc_sparse_inverse_conv_fwd): feats [n_coarse, cin] -> [n_fine, cout];
    `pretranspose` as for subm_conv_fwd."""
    dev = feats.device
    _conv_checks(feats, weight, bias, dev)
    _need(nbr_in, "nbr_in", torch.int32, dev)
    if order_in is not None:
        _need(order_in, "order_in", torch.int32, dev)
    K, cin, cout = weight.shape
    if _pretranspose(feats.dtype, cin, pretranspose):
        return conv_fwd_wt(feats, transpose_weight(weight), bias, nbr_in, n_fine, False, order_in, out=out)
    if out is None:
        out = torch.empty((n_fine, cout), dtype=feats.dtype, device=dev)
    st = lib().spc_sparse_inverse_conv_fwd(_DTYPES[feats.dtype], _ptr(feats), feats.shape[0], cin, _ptr(weight), K,
                                           cout, _ptr(bias), _ptr(nbr_in), _ptr(order_in), int(n_fine), _ptr(out),
                                           _stream(dev))
    _check(st, "spc_sparse_inverse_conv_fwd")
    return out


def conv_fwd_fused(feats: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                   map_: Optional[torch.Tensor], n_rows: int, order: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, relu: bool = False,
                   out: Optional[torch.Tensor] = None, pretranspose: Optional[bool] = None) -> torch.Tensor:
    """Forward over any map with the fused bias + residual + ReLU epilogue
    (spc_conv_fwd_fused); ``out`` may be ``residual`` itself; `pretranspose`
    as for subm_conv_fwd."""
    dev = feats.device
    _conv_checks(feats, weight, bias, dev)
    for t, nm in ((map_, "map"), (order, "order")):
        if t is not None:
            _need(t, nm, torch.int32, dev)
    K, cin, cout = weight.shape
    if residual is not None:
        _need(residual, "residual", feats.dtype, dev)
        if tuple(residual.shape) != (n_rows, cout):
            raise ValueError(f"residual must be [{n_rows}, {cout}], got {tuple(residual.shape)}")
    if _pretranspose(feats.dtype, cin, pretranspose):
        return conv_fwd_wt(feats, transpose_weight(weight), bias, map_, n_rows, False, order, residual, relu, out)
    if out is None:
        out = torch.empty((n_rows, cout), dtype=feats.dtype, device=dev)
    st = lib().spc_conv_fwd_fused(_DTYPES[feats.dtype], _ptr(feats), feats.shape[0], cin, _ptr(weight), K, cout,
                                  _ptr(bias), _ptr(map_), _ptr(order), int(n_rows), _ptr(residual),
                                  1 if relu else 0, _ptr(out), _stream(dev))
    _check(st, "spc_conv_fwd_fused")
    return out


def conv_bwd_input(dout: torch.Tensor, weight: torch.Tensor, map_: Optional[torch.Tensor], map_is_subm: bool,
                   n_in: int, order: Optional[torch.Tensor] = None,
                   din: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the input features (spc_conv_bwd_input)."""
    dev = dout.device
    _conv_checks(dout, weight, None, dev)
    for t, nm in ((map_, "map"), (order, "order")):
        if t is not None:
            _need(t, nm, torch.int32, dev)
    K, cin, cout = weight.shape
    if din is None:
        din = torch.empty((n_in, cin), dtype=dout.dtype, device=dev)
    st = lib().spc_conv_bwd_input(_DTYPES[dout.dtype], _ptr(dout), dout.shape[0], cout, _ptr(weight), K, cin,
                                  _ptr(map_), 1 if map_is_subm else 0, _ptr(order), int(n_in), _ptr(din),
                                  _stream(dev))
    _check(st, "spc_conv_bwd_input")
    return din


@functools.lru_cache(maxsize=256)
def conv_bwd_filter_workspace(n_in, n_out, cin, cout, K, want_dbias) -> int:
    b = ctypes.c_size_t()
    _check(lib().spc_conv_bwd_filter_workspace(int(n_in), int(n_out), int(cin), int(cout), int(K),
                                               1 if want_dbias else 0, ctypes.byref(b)),
           "spc_conv_bwd_filter_workspace")
    return b.value


def conv_bwd_filter(feats: torch.Tensor, dout: torch.Tensor, K: int, pair_ptr: Optional[torch.Tensor],
                    pair_in: Optional[torch.Tensor], pair_out: Optional[torch.Tensor], want_dbias: bool = False,
                    workspace: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None):
    """Weight (and optionally bias) gradient from CSR pair lists (spc_conv_bwd_filter).

    Returns ``(dw [K, Cin, Cout] fp32, dbias [Cout] fp32 or None)``."""
    dev = feats.device
    _need(feats, "feats", dev=dev)
    _need(dout, "dout", feats.dtype, dev)
    for t, nm in ((pair_ptr, "pair_ptr"), (pair_in, "pair_in"), (pair_out, "pair_out")):
        if t is not None:
            _need(t, nm, torch.int32, dev)
    cin, cout = feats.shape[1], dout.shape[1]
    ws = conv_bwd_filter_workspace(feats.shape[0], dout.shape[0], cin, cout, int(K), bool(want_dbias))
    workspace = _scratch(workspace, ws, feats, 256)
    if dw is None:
        dw = torch.empty((K, cin, cout), dtype=torch.float32, device=dev)
    db = torch.empty(cout, dtype=torch.float32, device=dev) if want_dbias else None
    st = lib().spc_conv_bwd_filter(_DTYPES[feats.dtype], _ptr(feats), feats.shape[0], cin, _ptr(dout),
                                   dout.shape[0], cout, int(K), _ptr(pair_ptr), _ptr(pair_in), _ptr(pair_out),
                                   _ptr(dw), _ptr(db), _ptr(workspace), workspace.numel(), _stream(dev))
    _check(st, "spc_conv_bwd_filter")
    return dw, db


def conv_bwd_filter_noalloc(feats: torch.Tensor, dout: torch.Tensor, K: int, pair_ptr: Optional[torch.Tensor],
                            pair_in: Optional[torch.Tensor], pair_out: Optional[torch.Tensor], dw: torch.Tensor,
                            dbias: Optional[torch.Tensor] = None) -> None:
    """spc_conv_bwd_filter_noalloc: the weight (and optionally bias) gradient
    into the caller's ``dw`` [K, Cin, Cout] fp32 (and ``dbias`` [Cout] fp32),
    with the library's static scratch instead of a workspace; neither the
    binding nor the library allocates anything."""
    dev = feats.device
    _need(feats, "feats", dev=dev)
    _need(dout, "dout", feats.dtype, dev)
    for t, nm in ((pair_ptr, "pair_ptr"), (pair_in, "pair_in"), (pair_out, "pair_out")):
        if t is not None:
            _need(t, nm, torch.int32, dev)
    cin, cout = feats.shape[1], dout.shape[1]
    _need(dw, "dw", torch.float32, dev)
    if tuple(dw.shape) != (int(K), cin, cout):
        raise ValueError(f"dw must be [{K}, {cin}, {cout}], got {tuple(dw.shape)}")
    if dbias is not None:
        _need(dbias, "dbias", torch.float32, dev)
        if tuple(dbias.shape) != (cout,):
            raise ValueError(f"dbias must be [{cout}], got {tuple(dbias.shape)}")
    st = lib().spc_conv_bwd_filter_noalloc(_DTYPES[feats.dtype], _ptr(feats), feats.shape[0], cin, _ptr(dout),
                                           dout.shape[0], cout, int(K), _ptr(pair_ptr), _ptr(pair_in),
                                           _ptr(pair_out), _ptr(dw), _ptr(dbias), _stream(dev))
    _check(st, "spc_conv_bwd_filter_noalloc")


def sparse_maxpool_fwd(feats: torch.Tensor, nbr_out: torch.Tensor, n_out: int, want_argk: bool = True,
                       out: Optional[torch.Tensor] = None, argk: Optional[torch.Tensor] = None):
    """Channel-wise max over each output's map row (spc_sparse_maxpool_fwd):
    returns ``(out [n_out, C], argk uint8 [n_out, C] or None)``."""
    dev = feats.device
    _need(feats, "feats", feats.dtype, dev)
    _need(nbr_out, "nbr_out", torch.int32, dev)
    C = feats.shape[1]
    K = nbr_out.shape[1] if nbr_out.dim() == 2 else 0
    if out is None:
        out = torch.empty((n_out, C), dtype=feats.dtype, device=dev)
    if want_argk and argk is None:
        argk = torch.empty((n_out, C), dtype=torch.uint8, device=dev)
    st = lib().spc_sparse_maxpool_fwd(_DTYPES[feats.dtype], _ptr(feats), feats.shape[0], C, _ptr(nbr_out), K,
                                      int(n_out), _ptr(out), _ptr(argk if want_argk else None), _stream(dev))
    _check(st, "spc_sparse_maxpool_fwd")
    return out, (argk if want_argk else None)


def sparse_maxpool_bwd(dout: torch.Tensor, argk: torch.Tensor, nbr_in: torch.Tensor, n_in: int,
                       din: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the pooled features routed to the winning inputs (spc_sparse_maxpool_bwd)."""
    dev = dout.device
    _need(dout, "dout", dout.dtype, dev)
    _need(argk, "argk", torch.uint8, dev)
    _need(nbr_in, "nbr_in", torch.int32, dev)
    C = dout.shape[1]
    K = nbr_in.shape[1] if nbr_in.dim() == 2 else 0
    if din is None:
        din = torch.empty((n_in, C), dtype=dout.dtype, device=dev)
    st = lib().spc_sparse_maxpool_bwd(_DTYPES[dout.dtype], _ptr(dout), dout.shape[0], C, _ptr(argk), _ptr(nbr_in),
                                      K, int(n_in), _ptr(din), _stream(dev))
    _check(st, "spc_sparse_maxpool_bwd")
    return din


def point_to_voxel(points: torch.Tensor, vsize_xyz, coors_range_xyz, max_num_voxels: int,
                   max_num_points_per_voxel: int, empty_mean: bool = True, with_id: bool = False):
    """Voxelise a point cloud [N, F] fp32 (spc_point_to_voxel), like spconv's
    PointToVoxel: returns (voxels [V, P, F], coords [V, 3] ZYX, num_points [V])
    and, with ``with_id``, the per-point voxel ids [N] as a fourth item."""
    dev = points.device
    _need(points, "points", torch.float32, dev)
    if points.dim() != 2:
        raise ValueError("points must be [N, F]")
    n, F = points.shape
    vs = (ctypes.c_float * 3)(*[float(v) for v in vsize_xyz])
    rg = (ctypes.c_float * 6)(*[float(v) for v in coors_range_xyz])
    b = ctypes.c_size_t()
    _check(lib().spc_point_to_voxel_workspace(n, F, int(max_num_voxels), int(max_num_points_per_voxel),
                                              ctypes.byref(b)), "spc_point_to_voxel_workspace")
    ws = torch.empty(max(int(b.value), 16), dtype=torch.uint8, device=dev)
    voxels = torch.empty((max_num_voxels, max_num_points_per_voxel, F), dtype=torch.float32, device=dev)
    coords = torch.empty((max_num_voxels, 3), dtype=torch.int32, device=dev)
    num = torch.empty((max_num_voxels,), dtype=torch.int32, device=dev)
    pcid = torch.empty((n,), dtype=torch.int32, device=dev) if with_id else None
    nv = ctypes.c_int64()
    st = lib().spc_point_to_voxel(_ptr(points), n, F, vs, rg, int(max_num_voxels), int(max_num_points_per_voxel),
                                  1 if empty_mean else 0, _ptr(voxels), _ptr(coords), _ptr(num), _ptr(pcid),
                                  ctypes.byref(nv), _ptr(ws), ws.numel(), _stream(dev))
    _check(st, "spc_point_to_voxel")
    V = nv.value
    res = (voxels[:V], coords[:V], num[:V])
    return res + (pcid,) if with_id else res


def gather_by_voxel_id(seg_features: torch.Tensor, pc_voxel_id: torch.Tensor,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Per-point features from per-voxel ones, zeros for id -1 (spc_gather_by_voxel_id)."""
    dev = seg_features.device
    _need(seg_features, "seg_features", seg_features.dtype, dev)
    _need(pc_voxel_id, "pc_voxel_id", torch.int32, dev)
    C = seg_features.shape[1]
    if out is None:
        out = torch.empty((pc_voxel_id.shape[0], C), dtype=seg_features.dtype, device=dev)
    st = lib().spc_gather_by_voxel_id(_DTYPES[seg_features.dtype], _ptr(seg_features), seg_features.shape[0], C,
                                      _ptr(pc_voxel_id), pc_voxel_id.shape[0], _ptr(out), _stream(dev))
    _check(st, "spc_gather_by_voxel_id")
    return out


ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2}   # SPC_ACT_*


class Dropout:
    """Dropout of one call (spc_dropout): ``rng`` int64 [2] on the GPU holds
    {seed, offset}, ``p`` the probability, ``layer`` tells the calls of one
    step apart.  The mask is a function of these alone and is drawn again by
    the backward; advance ``rng`` on the device between steps.  All three may
    be set again, for the calls that follow."""

    def __init__(self, rng: torch.Tensor, p: float, layer: int = 0):
        self._arg = _DropArg()
        self.rng, self.p, self.layer = rng, p, layer

    def __reduce__(self):   # a copy has a descriptor of its own
        return type(self), (self._rng, self._p, self.layer)

    @property
    def rng(self) -> torch.Tensor:
        return self._rng

    @rng.setter
    def rng(self, rng: torch.Tensor):
        _need(rng, "rng", torch.int64)
        if rng.shape != (2,):
            raise ValueError(f"rng must be [2] {{seed, offset}}, got {tuple(rng.shape)}")
        self._rng = rng

    @property
    def p(self) -> float:
        return self._p

    @p.setter
    def p(self, p: float):
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p={p} is outside [0, 1]")
        self._p = self._arg.p = float(p)

    @property
    def layer(self) -> int:
        return self._arg.layer

    @layer.setter
    def layer(self, layer: int):
        if not 0 <= layer < 1 << 32:
            raise ValueError(f"layer={layer} is not a 32-bit number")
        self._arg.layer = int(layer)


def _drop_arg(dropout, dev):
    if dropout is None:
        return None
    if not isinstance(dropout, Dropout):
        raise TypeError("dropout must be a Dropout")
    if dropout._rng.device != dev:
        raise ValueError(f"rng is on {dropout._rng.device}, expected {dev}")
    dropout._arg.rng = dropout._rng.data_ptr()   # where the tensor is now
    return ctypes.byref(dropout._arg)


def _need_like(t, name, dtype, dev, shape):
    _need(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")


def _rows_checks(x, name="input"):
    _need(x, name)
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"{name} must be [N, C]")


def _n_seg(seg_ptr, dev) -> int:
    if seg_ptr is None:
        return 1
    _need(seg_ptr, "seg_ptr", torch.int32, dev)
    if seg_ptr.dim() != 1 or seg_ptr.numel() < 2:
        raise ValueError("seg_ptr must be [n_seg + 1]")
    return seg_ptr.numel() - 1


def dropout_fwd(x: torch.Tensor, dropout: Dropout, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + dropout(x), any shape (spc_dropout_fwd); ``out`` may be x or
    residual."""
    _need(x, "input")
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    dev = x.device
    if dropout is None:
        raise TypeError("dropout must be a Dropout")
    if residual is not None:
        _need_like(residual, "residual", x.dtype, dev, x.shape)
    if out is None:
        out = torch.empty_like(x)
    else:
        _need_like(out, "out", x.dtype, dev, x.shape)
    st = lib().spc_dropout_fwd(_DTYPES[x.dtype], _ptr(x), x.numel(), _ptr(residual), _drop_arg(dropout, dev), _ptr(out),
                               _stream(dev))
    _check(st, "spc_dropout_fwd")
    return out


def dropout_bwd(dout: torch.Tensor, dropout: Dropout, din: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of dropout_fwd's x (spc_dropout_bwd): the same mask, drawn
    again.  ``din`` may be dout."""
    _need(dout, "dout")
    if dout.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dout.dtype}")
    dev = dout.device
    if dropout is None:
        raise TypeError("dropout must be a Dropout")
    if din is None:
        din = torch.empty_like(dout)
    else:
        _need_like(din, "din", dout.dtype, dev, dout.shape)
    st = lib().spc_dropout_bwd(_DTYPES[dout.dtype], _ptr(dout), dout.numel(), _drop_arg(dropout, dev), _ptr(din),
                               _stream(dev))
    _check(st, "spc_dropout_bwd")
    return din


@functools.lru_cache(maxsize=256)
def group_norm_workspace(n: int, C: int, groups: int, n_seg: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().spc_group_norm_workspace(n, C, groups, n_seg, ctypes.byref(b)), "spc_group_norm_workspace")
    return b.value


def _norm_checks(x, groups, seg_ptr, gamma, beta, act, workspace):
    _rows_checks(x)
    dev, (n, C) = x.device, x.shape
    n_seg = _n_seg(seg_ptr, dev)
    for t, nm in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            _need_like(t, nm, torch.float32, dev, (C,))
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {tuple(ACTIVATIONS)}, got {act!r}")
    workspace = _scratch(workspace, group_norm_workspace(n, C, int(groups), n_seg), x)
    return dev, n, C, n_seg, workspace, 0 if workspace is None else workspace.numel()


def group_norm_fwd(x: torch.Tensor, groups: int, seg_ptr: Optional[torch.Tensor] = None,
                   gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   act: str = "none", dropout: Optional[Dropout] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """dropout(act(group norm of x [N, C])) over the samples of seg_ptr int32
    [S + 1] (None: one sample) (spc_group_norm_fwd).  gamma, beta fp32 [C].
    Returns ``(y, stats fp32 [S, groups, 2])``, stats for group_norm_bwd;
    ``out`` may be x."""
    dev, n, C, n_seg, workspace, ws_bytes = _norm_checks(x, groups, seg_ptr, gamma, beta, act, workspace)
    if out is None:
        out = torch.empty_like(x)
    else:
        _need_like(out, "out", x.dtype, dev, x.shape)
    stats = x.new_empty((n_seg, groups, 2), dtype=torch.float32)
    st = lib().spc_group_norm_fwd(_DTYPES[x.dtype], _ptr(x), n, C, int(groups), _ptr(seg_ptr), n_seg, _ptr(gamma),
                                  _ptr(beta), eps, ACTIVATIONS[act], _drop_arg(dropout, dev), _ptr(out), _ptr(stats),
                                  _ptr(workspace), ws_bytes, _stream(dev))
    _check(st, "spc_group_norm_fwd")
    return out, stats


def group_norm_bwd(dout: torch.Tensor, x: torch.Tensor, groups: int, seg_ptr: Optional[torch.Tensor],
                   gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], stats: torch.Tensor,
                   act: str = "none", dropout: Optional[Dropout] = None, want_affine: bool = True,
                   dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of group_norm_fwd (spc_group_norm_bwd) from its x and stats:
    ``(dx, dgamma, dbeta)``, the last two fp32 [C] or None; ``dx`` may be dout."""
    dev, n, C, n_seg, workspace, ws_bytes = _norm_checks(x, groups, seg_ptr, gamma, beta, act, workspace)
    _need_like(dout, "dout", x.dtype, dev, x.shape)
    _need_like(stats, "stats", torch.float32, dev, (n_seg, groups, 2))
    if dx is None:
        dx = torch.empty_like(x)
    else:
        _need_like(dx, "dx", x.dtype, dev, x.shape)
    dgamma = dbeta = None
    if want_affine:
        dgamma, dbeta = x.new_empty((C,), dtype=torch.float32), x.new_empty((C,), dtype=torch.float32)
    st = lib().spc_group_norm_bwd(_DTYPES[x.dtype], _ptr(dout), _ptr(x), n, C, int(groups), _ptr(seg_ptr), n_seg,
                                  _ptr(gamma), _ptr(beta), _ptr(stats), ACTIVATIONS[act], _drop_arg(dropout, dev),
                                  _ptr(dx), _ptr(dgamma), _ptr(dbeta), _ptr(workspace), ws_bytes, _stream(dev))
    _check(st, "spc_group_norm_bwd")
    return dx, dgamma, dbeta


@functools.lru_cache(maxsize=256)
def linear_recurrence_workspace(dtype: torch.dtype, n: int, C: int, n_seg: int) -> tuple:
    """(workspace bytes, carry bytes) of the recurrence calls."""
    w, c = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().spc_linear_recurrence_workspace(_DTYPES[dtype], n, C, n_seg, ctypes.byref(w), ctypes.byref(c)),
           "spc_linear_recurrence_workspace")
    return w.value, c.value


def _gate_x(gate, x, names=("gate", "x")):
    """Checks a pair of [N, C] row views (which may be column slices of one
    tensor) and returns their common row stride."""
    for t, nm in ((gate, names[0]), (x, names[1])):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{nm} must be a CUDA (HIP) tensor")
        if t.dtype not in _DTYPES:
            raise TypeError(f"unsupported dtype {t.dtype}")
        if t.dim() != 2:
            raise ValueError(f"{nm} must be [N, C]")
    if gate.shape != x.shape or gate.dtype != x.dtype or gate.device != x.device:
        raise ValueError(f"{names[0]} and {names[1]} must agree in dtype, shape and device")
    n, C = x.shape
    (lg, cg), (lx, cx) = gate.stride(), x.stride()
    if C > 1 and (cg != 1 or cx != 1):
        raise ValueError(f"the channels of {names[0]} and {names[1]} must be contiguous")
    if n <= 1:
        return C
    if lg != lx:
        raise ValueError(f"{names[0]} and {names[1]} must have one row stride")
    return lx


def _lr_checks(gate, x, seg_ptr, h0, order, workspace):
    ld = _gate_x(gate, x)
    dev, (n, C) = x.device, x.shape
    n_seg = _n_seg(seg_ptr, dev)
    if h0 is not None:
        _need_like(h0, "h0", torch.float32, dev, (n_seg, C))
    if order is not None:
        _need_like(order, "order", torch.int32, dev, (n,))
    ws, carry = linear_recurrence_workspace(x.dtype, n, C, n_seg)
    return dev, n, C, n_seg, ld, _scratch(workspace, ws, x), carry


def linear_recurrence_fwd(gate: torch.Tensor, x: torch.Tensor, seg_ptr: Optional[torch.Tensor] = None,
                          h0: Optional[torch.Tensor] = None, order: Optional[torch.Tensor] = None,
                          reverse: bool = False, want_carry: bool = False, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None):
    """h_t = sigmoid(gate_t) h_{t-1} + sigmoid(-gate_t) x_t along the rows of
    each sample (spc_linear_recurrence_fwd): gate, x [N, C], or column slices
    of one wider tensor; h0 fp32 [S, C].  Returns ``(out [N, C], h_last fp32
    [S, C], carry or None)``; carry is for linear_recurrence_bwd."""
    dev, n, C, n_seg, ld, workspace, carry_bytes = _lr_checks(gate, x, seg_ptr, h0, order, workspace)
    if out is None:
        out = x.new_empty((n, C))
    else:
        _need_like(out, "out", x.dtype, dev, (n, C))
    h_last = x.new_empty((n_seg, C), dtype=torch.float32)
    carry = x.new_empty((max(carry_bytes // 4, 4),), dtype=torch.float32) if want_carry else None
    st = lib().spc_linear_recurrence_fwd(_DTYPES[x.dtype], _ptr(gate), _ptr(x), ld, n, C, _ptr(seg_ptr), n_seg,
                                         _ptr(order), 1 if reverse else 0, _ptr(h0), _ptr(out), _ptr(h_last),
                                         _ptr(carry), _ptr(workspace), workspace.numel(), _stream(dev))
    _check(st, "spc_linear_recurrence_fwd")
    return out, h_last, carry


def linear_recurrence_bwd(dout: torch.Tensor, gate: torch.Tensor, x: torch.Tensor, seg_ptr: Optional[torch.Tensor],
                          carry: torch.Tensor, h0: Optional[torch.Tensor] = None,
                          dh_last: Optional[torch.Tensor] = None, order: Optional[torch.Tensor] = None,
                          reverse: bool = False, want_dh0: bool = False, dgate: Optional[torch.Tensor] = None,
                          dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of linear_recurrence_fwd (spc_linear_recurrence_bwd) from its
    arguments and carry: ``(dgate [N, C], dx [N, C], dh0 fp32 [S, C] or None)``.
    ``dgate`` and ``dx`` may be given as column slices of one tensor."""
    dev, n, C, n_seg, ld, workspace, carry_bytes = _lr_checks(gate, x, seg_ptr, h0, order, workspace)
    _need_like(dout, "dout", x.dtype, dev, (n, C))
    _need_like(carry, "carry", torch.float32, dev, (max(carry_bytes // 4, 4),))
    if dh_last is not None:
        _need_like(dh_last, "dh_last", torch.float32, dev, (n_seg, C))
    if (dgate is None) != (dx is None):
        raise ValueError("dgate and dx: give both or neither")
    if dgate is None:
        dgate, dx = x.new_empty((n, C)), x.new_empty((n, C))
        ldg = C
    else:
        ldg = _gate_x(dgate, dx, ("dgate", "dx"))
        if dx.dtype != x.dtype or dx.shape != x.shape or dx.device != dev:
            raise ValueError("dgate and dx must agree with x in dtype, shape and device")
    dh0 = x.new_empty((n_seg, C), dtype=torch.float32) if want_dh0 else None
    st = lib().spc_linear_recurrence_bwd(_DTYPES[x.dtype], _ptr(dout), _ptr(gate), _ptr(x), ld, n, C, _ptr(seg_ptr),
                                         n_seg, _ptr(order), 1 if reverse else 0, _ptr(h0), _ptr(carry), _ptr(dh_last),
                                         _ptr(dgate), _ptr(dx), ldg, _ptr(dh0), _ptr(workspace), workspace.numel(),
                                         _stream(dev))
    _check(st, "spc_linear_recurrence_bwd")
    return dgate, dx, dh0


def linear_recurrence_step(gate: torch.Tensor, x: torch.Tensor, state: torch.Tensor,
                           new_state: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One step of N running sequences (spc_linear_recurrence_step): state
    fp32 [N, C] is replaced in place, or left and the new one written to
    ``new_state``; returns the new state in gate's dtype."""
    ld = _gate_x(gate, x)
    dev, (n, C) = x.device, x.shape
    _need_like(state, "state", torch.float32, dev, (n, C))
    if new_state is None:
        new_state = state
    else:
        _need_like(new_state, "new_state", torch.float32, dev, (n, C))
    if out is None:
        out = x.new_empty((n, C))
    else:
        _need_like(out, "out", x.dtype, dev, (n, C))
    st = lib().spc_linear_recurrence_step(_DTYPES[x.dtype], _ptr(gate), _ptr(x), ld, n, C, _ptr(state), _ptr(new_state),
                                          _ptr(out), _stream(dev))
    _check(st, "spc_linear_recurrence_step")
    return out


@functools.lru_cache(maxsize=256)
def layer_norm_workspace(n: int, C: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().spc_layer_norm_workspace(n, C, ctypes.byref(b)), "spc_layer_norm_workspace")
    return b.value


def layer_norm_fwd(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   total: Optional[torch.Tensor] = None):
    """Layer norm of x [N, C], or of x + residual, over the channels
    (spc_layer_norm_fwd); gamma, beta fp32 [C].  Returns ``(y, stats fp32
    [N, 2], total)``: total is x + residual as stored, None without a residual.
    ``out`` may be x, ``total`` x or residual."""
    _rows_checks(x)
    dev, (n, C) = x.device, x.shape
    for t, nm in ((gamma, "gamma"), (beta, "beta")):
        if t is not None:
            _need_like(t, nm, torch.float32, dev, (C,))
    if residual is not None:
        _need_like(residual, "residual", x.dtype, dev, x.shape)
        if total is None:
            total = torch.empty_like(x)
        else:
            _need_like(total, "total", x.dtype, dev, x.shape)
    elif total is not None:
        raise ValueError("total goes with a residual")
    if out is None:
        out = torch.empty_like(x)
    else:
        _need_like(out, "out", x.dtype, dev, x.shape)
    stats = x.new_empty((n, 2), dtype=torch.float32)
    st = _call(dev, lib().spc_layer_norm_fwd, _DTYPES[x.dtype], _ptr(x), _ptr(residual), n, C, _ptr(gamma), _ptr(beta), eps,
               _ptr(out), _ptr(total), _ptr(stats))
    _check(st, "spc_layer_norm_fwd")
    return out, stats, total


def layer_norm_bwd(dout: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor], stats: torch.Tensor,
                   dtotal: Optional[torch.Tensor] = None, want_affine: bool = True, dx: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of layer_norm_fwd (spc_layer_norm_bwd): x is what was normed
    (the forward's total with a residual), ``dtotal`` the gradient that reaches
    it past the norm.  Returns ``(dx, dgamma, dbeta)``, the last two fp32 [C] or
    None; dx is the gradient of x and residual alike and may be dout or dtotal."""
    _rows_checks(x)
    dev, (n, C) = x.device, x.shape
    if gamma is not None:
        _need_like(gamma, "gamma", torch.float32, dev, (C,))
    _need_like(dout, "dout", x.dtype, dev, x.shape)
    _need_like(stats, "stats", torch.float32, dev, (n, 2))
    if dtotal is not None:
        _need_like(dtotal, "dtotal", x.dtype, dev, x.shape)
    if dx is None:
        dx = torch.empty_like(x)
    else:
        _need_like(dx, "dx", x.dtype, dev, x.shape)
    dgamma = dbeta = None
    if want_affine:
        dgamma, dbeta = x.new_empty((C,), dtype=torch.float32), x.new_empty((C,), dtype=torch.float32)
    workspace = _scratch(workspace, layer_norm_workspace(n, C) if want_affine else 0, x)
    st = _call(dev, lib().spc_layer_norm_bwd, _DTYPES[x.dtype], _ptr(dout), _ptr(x), n, C, _ptr(gamma), _ptr(stats),
               _ptr(dtotal), _ptr(dx), _ptr(dgamma), _ptr(dbeta), _ptr(workspace), 0 if workspace is None else workspace.numel())
    _check(st, "spc_layer_norm_bwd")
    return dx, dgamma, dbeta


def _heads(t, name, dtype=None, dev=None, shape=None):
    """Checks a [N, H, D] view whose heads lie side by side within a row (a
    column slice of a wider tensor is one) and returns its row stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"unsupported dtype {t.dtype} of {name}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [N, heads, head_dim]")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
    n, H, D = t.shape
    ln, lh, ld = t.stride()
    if (D > 1 and ld != 1) or (H > 1 and lh != D):
        raise ValueError(f"the heads of {name} must lie side by side in a row")
    return ln if n > 1 else H * D


@functools.lru_cache(maxsize=256)
def _axis_pairs(pairs: tuple):
    return (ctypes.c_int32 * len(pairs))(*pairs)


def rotary(x: torch.Tensor, pos: torch.Tensor, freq: torch.Tensor, pairs: Sequence[int], inverse: bool = False,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotary positions of several axes (spc_rotary): x [N, heads, head_dim],
    or a column slice of a wider tensor; pos int32 [N, axes], which may be
    columns of the voxels' coordinates; freq fp32, one for each rotated pair;
    pairs: the pairs of each axis.  ``inverse`` rotates back, which is the
    gradient; ``out`` may be x."""
    ldx = _heads(x, "input")
    dev, (n, H, D) = x.device, x.shape
    pairs = tuple(int(v) for v in pairs)
    if not isinstance(pos, torch.Tensor) or not pos.is_cuda:
        raise TypeError("pos must be a CUDA (HIP) tensor")
    if pos.dtype != torch.int32:
        raise TypeError(f"pos must be {torch.int32}, got {pos.dtype}")
    if pos.device != dev:
        raise ValueError(f"pos is on {pos.device}, expected {dev}")
    if pos.dim() != 2 or pos.shape != (n, len(pairs)) or (pos.shape[1] > 1 and pos.stride(1) != 1):
        raise ValueError(f"pos must be [N, {len(pairs)}] with its axes side by side")
    _need(freq, "freq", torch.float32, dev)
    if freq.shape != (sum(pairs),):
        raise ValueError(f"freq must be [{sum(pairs)}], got {tuple(freq.shape)}")
    if out is None:
        out = x.new_empty((n, H, D))
    ldo = _heads(out, "out", x.dtype, dev, x.shape)
    if out is not x and n and out.data_ptr() == x.data_ptr() and out.stride() != x.stride():
        raise ValueError("out may be x itself, not another view of it")
    st = _call(dev, lib().spc_rotary, _DTYPES[x.dtype], _ptr(x), ldx, n, H, D, _ptr(pos),
               pos.stride(0) if n > 1 else len(pairs), len(pairs), _axis_pairs(pairs), _ptr(freq), 1 if inverse else 0,
               _ptr(out), ldo)
    _check(st, "spc_rotary")
    return out


@functools.lru_cache(maxsize=256)
def attention_workspace(dtype: torch.dtype, n_q: int, n_kv: int, n_seg: int, heads: int, kv_heads: int, head_dim: int) -> tuple:
    """(workspace bytes of attention_fwd, of attention_bwd)."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    a = _AttnArg(n_q, n_kv, n_seg, heads, kv_heads, head_dim, 0, 1.0)
    _check(lib().spc_attention_workspace(_DTYPES[dtype], ctypes.byref(a), ctypes.byref(f), ctypes.byref(b)),
           "spc_attention_workspace")
    return f.value, b.value


def _attn_checks(q, k, v, seg_ptr, order, kv_ptr, kv_order, causal, scale):
    """(descriptor, row strides of q, k, v, workspace bytes)."""
    ldq = _heads(q, "q")
    dev, (n, H, D) = q.device, q.shape
    ldk = _heads(k, "k", q.dtype, dev)
    m, Hk, _ = k.shape
    ldv = _heads(v, "v", q.dtype, dev, k.shape)
    if k.shape[2] != D:
        raise ValueError(f"q has head_dim {D}, k {k.shape[2]}")
    n_seg = _n_seg(seg_ptr, dev)
    if kv_ptr is None and kv_order is None and seg_ptr is not None or order is not None and kv_ptr is None and kv_order is None:
        if n != m:
            raise ValueError(f"{n} queries and {m} keys: kv_ptr or kv_order must say how the keys are laid out")
    if kv_ptr is None and kv_order is None:          # the rows attend to themselves
        kv_ptr, kv_order = seg_ptr, order
    else:
        if kv_ptr is None and seg_ptr is not None:
            raise ValueError("kv_order without kv_ptr: give both")
        if kv_ptr is not None and _n_seg(kv_ptr, dev) != n_seg:
            raise ValueError(f"seg_ptr has {n_seg} samples, kv_ptr {_n_seg(kv_ptr, dev)}")
    if order is not None:
        _need_like(order, "order", torch.int32, dev, (n,))
    if kv_order is not None:
        _need_like(kv_order, "kv_order", torch.int32, dev, (m,))
    a = _AttnArg(n, m, n_seg, H, Hk, D, 1 if causal else 0, max(D, 1) ** -0.5 if scale is None else scale, _ptr(seg_ptr), _ptr(kv_ptr),
                 _ptr(order), _ptr(kv_order))
    return a, (ldq, ldk, ldv), attention_workspace(q.dtype, n, m, n_seg, H, Hk, D)


def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seg_ptr: Optional[torch.Tensor] = None,
                  order: Optional[torch.Tensor] = None, kv_ptr: Optional[torch.Tensor] = None,
                  kv_order: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None,
                  want_stats: bool = False, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of each sample's queries to its keys (spc_attention_fwd): q
    [Nq, heads, D], k and v [Nkv, kv_heads, D], each of which may be a column
    slice of one product.  seg_ptr and order lay out the queries and, where
    neither kv_ptr nor kv_order is given, the keys; scale defaults to D^-1/2.
    Returns ``(out [Nq, heads, D], stats or None)``; stats are for
    attention_bwd: ``(ml fp32 [heads, Nq, 2], rest)``, from which the log of each
    row's sum follows, and what rounding left of out ([Nq, heads, D], fp16's
    times 2^11; None for fp32)."""
    a, (ldq, ldk, ldv), (need, _) = _attn_checks(q, k, v, seg_ptr, order, kv_ptr, kv_order, causal, scale)
    dev, (n, H, D) = q.device, q.shape
    if out is None:
        out = q.new_empty((n, H, D))
    ldo = _heads(out, "out", q.dtype, dev, q.shape)
    ml = rest = None
    if want_stats:
        ml = q.new_empty((H, n, 2), dtype=torch.float32)
        rest = q.new_empty((n, H, D)) if q.dtype != torch.float32 else None
    workspace = _scratch(workspace, need, q)
    st = _call(dev, lib().spc_attention_fwd, _DTYPES[q.dtype], ctypes.byref(a), _ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv,
               _ptr(out), ldo, _ptr(ml), _ptr(rest), _ptr(workspace), 0 if workspace is None else workspace.numel())
    _check(st, "spc_attention_fwd")
    return out, (ml, rest) if want_stats else None


def attention_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                  stats: tuple, seg_ptr: Optional[torch.Tensor] = None, order: Optional[torch.Tensor] = None,
                  kv_ptr: Optional[torch.Tensor] = None, kv_order: Optional[torch.Tensor] = None, causal: bool = False,
                  scale: Optional[float] = None, dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                  dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of attention_fwd (spc_attention_bwd) from its arguments, out
    and stats: ``(dq, dk, dv)``, which may be given as column slices of one
    tensor."""
    a, (ldq, ldk, ldv), (_, need) = _attn_checks(q, k, v, seg_ptr, order, kv_ptr, kv_order, causal, scale)
    dev, (n, H, D) = q.device, q.shape
    lddo, ldo = _heads(dout, "dout", q.dtype, dev, q.shape), _heads(out, "out", q.dtype, dev, q.shape)
    if not isinstance(stats, tuple) or len(stats) != 2:
        raise TypeError("stats must be what attention_fwd(..., want_stats=True) returned")
    ml, rest = stats
    _need_like(ml, "stats[0]", torch.float32, dev, (H, n, 2))
    if rest is not None:
        _need_like(rest, "stats[1]", q.dtype, dev, (n, H, D))
    dq = q.new_empty(q.shape) if dq is None else dq
    dk = k.new_empty(k.shape) if dk is None else dk
    dv = v.new_empty(v.shape) if dv is None else dv
    lddq, lddk, lddv = (_heads(t, nm, q.dtype, dev, like.shape) for t, nm, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)))
    workspace = _scratch(workspace, need, q)
    st = _call(dev, lib().spc_attention_bwd, _DTYPES[q.dtype], ctypes.byref(a), _ptr(dout), lddo, _ptr(q), ldq, _ptr(k), ldk,
               _ptr(v), ldv, _ptr(out), ldo, _ptr(ml), _ptr(rest), _ptr(dq), lddq, _ptr(dk), lddk, _ptr(dv), lddv,
               _ptr(workspace), 0 if workspace is None else workspace.numel())
    _check(st, "spc_attention_bwd")
    return dq, dk, dv


def calibrate_mfma(shape: int, blocks: int, iters: int, sink: torch.Tensor) -> float:
    """Launches the MFMA rate probe (spc_calibrate_mfma) on the current stream
    and returns the FLOP it executes; the caller times it."""
    _need(sink, "sink", torch.float32)
    if sink.numel() < blocks * 256:
        raise ValueError("sink needs blocks * 256 floats")
    f = ctypes.c_double(0.0)
    _check(lib().spc_calibrate_mfma(int(shape), int(blocks), int(iters), _ptr(sink), ctypes.byref(f),
                                    _stream(sink.device)), "spc_calibrate_mfma")
    return f.value
