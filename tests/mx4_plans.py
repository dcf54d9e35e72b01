"""Which compiled kernel a call of given sizes runs, from the library's own plans (host code; without a GPU they
count 256 CUs, an MI355X's)."""
import ctypes

from decode_gemv_thinkbit_amd import qlinear as ql


class _Gemv(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("tiles", "parts")]


class _Gemm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("tiles", "parts", "tile")]


class _Moe(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("xp", "split", "gate_waves", "down_waves")]
                + [(n, ctypes.c_bool) for n in ("one", "small", "join", "wide")]
                + [(n, ctypes.c_int64) for n in ("hidden_bytes", "product_bytes")])


def _call(symbol, result, kind, *sizes):
    fn = getattr(ql.lib(), symbol)
    fn.restype, fn.argtypes = result, [kind] * len(sizes)
    return fn(*sizes)


def gemv(M, N, K):
    """(16-row tiles a workgroup, token pieces, K ends inside a pair of chunks, K split)"""
    p = _call("_ZN2ql13mx4_gemv_planEiii", _Gemv, ctypes.c_int, M, N, K)
    return p.tiles, 1 if M <= 2 else 2 if M <= 4 else 4 if M <= 8 else 8, K % 256 != 0, p.parts > 1


def gemm(M, N, K):
    """("skinny", tiles of W, tiles of X, K ends inside a pair, K split) or ("tile", outputs, K ends inside a pair)"""
    p = _call("_ZN2ql13mx4_gemm_planEiii", _Gemm, ctypes.c_int, M, N, K)
    if p.tiles:
        return "skinny", p.tiles, 1 if M <= 16 else 2 if M <= 32 else 4, K % 256 != 0, p.parts > 1
    return "tile", ("256x256", "128x128", "64x128", "64x64")[p.tile], K % 256 != 0


def moe_plan(T, k, E, H, I):
    return _call("_ZN2ql8moe_planElllll", _Moe, ctypes.c_int64, T, k, E, H, I)


def moe(T, k, E, H, I):
    """(the gate and up kernel: token pieces, waves, a task shared by four, up to 64 pairs, H ends inside a pair),
    (the down kernel: kind, waves, waves to a task, I ends inside a pair)"""
    p = moe_plan(T, k, E, H, I)
    kind = "one" if p.one else "few" if p.small else "wide" if p.wide else "many"
    return ((p.xp, p.gate_waves, p.join, p.small, H % 256 != 0),
            (kind, p.down_waves, p.down_waves // k if p.one else p.split, I % 256 != 0))
