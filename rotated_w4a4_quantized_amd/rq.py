"""Thin ctypes binding of librq (include/rq.h): argument marshalling only.

Every computation runs inside librq's gfx950 kernels (or, for the offline
weight pack, in librq's host code).  This module converts numpy / torch
arguments into the C structs and raw pointers of the C ABI, passes the
current HIP stream, and raises RQError on any non-OK status.  There is no
fallback: if librq.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librq.so")

RQ_OK = 0
RQ_F32, RQ_BF16, RQ_I32, RQ_I8 = 0, 1, 2, 3
RQ_ROT_RPBH, RQ_ROT_DENSE, RQ_ROT_TRDQ = 0, 1, 2
RQ_Q_INT4_SYM, RQ_Q_LLOYDMAX, RQ_Q_INT4_ASYM, RQ_Q_MXFP4 = 0, 1, 2, 3
RQ_ENGINE_AUTO, RQ_ENGINE_FP6, RQ_ENGINE_INT8 = 0, 1, 2
ENGINES = {"auto": RQ_ENGINE_AUTO, "fp6": RQ_ENGINE_FP6, "int8": RQ_ENGINE_INT8}
RQ_WEIGHT_MAGIC = 0x31575152
STATUS_NAMES = {0: "RQ_OK", -1: "RQ_ERR_NULL", -2: "RQ_ERR_SHAPE", -3: "RQ_ERR_DTYPE",
                -4: "RQ_ERR_ALIGN", -5: "RQ_ERR_FORMAT", -6: "RQ_ERR_UNSUPPORTED",
                -7: "RQ_ERR_HIP"}


class RQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class c_rotation(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("K", ctypes.c_int32), ("block", ctypes.c_int32),
                ("r", ctypes.c_int32), ("sign", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("R", ctypes.c_void_p), ("smooth", ctypes.c_void_p), ("R2", ctypes.c_void_p)]


class c_quant(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("a_bits", ctypes.c_int32), ("w_bits", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("a_levels", ctypes.c_float * 16),
                ("w_levels", ctypes.c_float * 16)]


class c_weight_header(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("format", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
                ("r", ctypes.c_int32), ("b_div", ctypes.c_int32), ("a_bits", ctypes.c_int32),
                ("w_bits", ctypes.c_int32), ("row_bytes", ctypes.c_int32),
                ("scale_offset", ctypes.c_int64), ("codes_offset", ctypes.c_int64),
                ("total_bytes", ctypes.c_int64), ("a_levels", ctypes.c_float * 16),
                ("w_levels", ctypes.c_float * 16), ("wsum_offset", ctypes.c_int64),
                ("mma_offset", ctypes.c_int64), ("mma_stages", ctypes.c_int32),
                ("mma_ntiles", ctypes.c_int32), ("i8_offset", ctypes.c_int64),
                ("mxs_offset", ctypes.c_int64), ("reserved", ctypes.c_uint8 * 24)]


assert ctypes.sizeof(c_weight_header) == 256


class c_set_header(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("groups", ctypes.c_int32), ("steps", ctypes.c_int32),
                ("member_offset", ctypes.c_int64 * 64), ("step_group", ctypes.c_int32 * 1024),
                ("reserved", ctypes.c_uint8 * (4864 - 16 - 8 * 64 - 4 * 1024))]


assert ctypes.sizeof(c_set_header) == 4864

class c_kv_cache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page", ctypes.c_int32), ("batch", ctypes.c_int32), ("table_ld", ctypes.c_int32),
                ("pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("pos", ctypes.c_void_p)]


class c_qk_norm(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("table_rows", ctypes.c_int32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p)]


class c_norm(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class c_modulation(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("reserved", ctypes.c_int32), ("ld", ctypes.c_int64),
                ("per", ctypes.c_int64), ("index", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("shift", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class c_states(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("keys", ctypes.c_int64), ("k_ld", ctypes.c_int64),
                ("v_ld", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("mask_ld", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("mask", ctypes.c_void_p)]


# every symbol include/rq.h declares
EXPORTS = ("rq_version", "rq_last_error", "rq_lloydmax_gaussian", "rq_packed_weight_bytes",
           "rq_pack_weights", "rq_rotate_quant_workspace_bytes", "rq_codes_mma_bytes",
           "rq_rotate_quant", "rq_w4a4_linear", "rq_w4a4_linear_engine",
           "rq_rotate_quant_noalloc", "rq_activation_bytes", "rq_weight_set_bytes",
           "rq_pack_weight_set", "rq_weight_set_member", "rq_qk_norm_rope",
           "rq_paged_attention_workspace_bytes", "rq_paged_attention",
           "rq_cache_evict_workspace_bytes", "rq_cache_evict", "rq_block_norm",
           "rq_cross_attention_workspace_bytes", "rq_cross_attention",
           "rq_prefix_attention_workspace_bytes", "rq_prefix_attention")

_lib = None


def load() -> ctypes.CDLL:
    """Load librq.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FileNotFoundError(
            f"{LIB_PATH} is missing: build it with `python -m rotated_w4a4_quantized_amd.build` "
            "(there is no fallback path)")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.rq_version.restype = I32
    L.rq_last_error.restype = ctypes.c_char_p
    L.rq_lloydmax_gaussian.argtypes = [I32, P]
    L.rq_packed_weight_bytes.argtypes = [P, P, I32, ctypes.POINTER(SZ)]
    L.rq_pack_weights.argtypes = [P, P, P, I32, I32, P, SZ]
    L.rq_rotate_quant_workspace_bytes.argtypes = [P, P, I64, ctypes.POINTER(SZ)]
    L.rq_codes_mma_bytes.argtypes = [P, I64, ctypes.POINTER(SZ)]
    L.rq_rotate_quant.argtypes = [P, P, P, I32, I64, P, P, P, P, P, SZ, P]
    L.rq_w4a4_linear.argtypes = [P, P, P, P, P, P, I64, P, P, I32, P]
    L.rq_w4a4_linear_engine.argtypes = [P, P, P, P, P, P, I64, P, P, I32, I32, P]
    L.rq_rotate_quant_noalloc.argtypes = [P, P, P, I32, I64, P, P, P, P, P]
    L.rq_activation_bytes.argtypes = [P, P, I64, ctypes.POINTER(SZ), ctypes.POINTER(SZ),
                                      ctypes.POINTER(SZ)]
    L.rq_weight_set_bytes.argtypes = [P, I32, P, I32, ctypes.POINTER(SZ)]
    L.rq_pack_weight_set.argtypes = [P, I32, P, I32, P, P, I32, I32, P, SZ]
    L.rq_weight_set_member.argtypes = [P, I32, ctypes.POINTER(I32), ctypes.POINTER(P),
                                       ctypes.POINTER(I64)]
    L.rq_qk_norm_rope.argtypes = [P, P, I32, I64, I64, P, P, I64, P, I64, P, P, P, P]
    L.rq_paged_attention_workspace_bytes.argtypes = [P, I32, I64, I32, ctypes.POINTER(SZ)]
    L.rq_paged_attention.argtypes = [P, P, I32, I64, I32, ctypes.c_float, P, I64, P, I64, P, I64,
                                     P, I32, P, P, SZ, P]
    L.rq_cache_evict_workspace_bytes.argtypes = [P, I32, I64, ctypes.POINTER(SZ)]
    L.rq_cache_evict.argtypes = [P, P, I64, I32, I32, I32, P, P, P, P, SZ, P]
    F = ctypes.c_float
    L.rq_block_norm.argtypes = [P, P, P, I32, P, I32, I64, P, I32, I64, I64, F, F, P, I64, P, I64, P]
    L.rq_cross_attention_workspace_bytes.argtypes = [P, I64, I32, I32, ctypes.POINTER(SZ)]
    L.rq_cross_attention.argtypes = [P, P, I32, I64, I64, I64, I32, F, P, P, I64, I64, P, P, SZ, P]
    L.rq_prefix_attention_workspace_bytes.argtypes = [P, I32, I32, I64, I64, ctypes.POINTER(SZ)]
    L.rq_prefix_attention.argtypes = [P, P, I64, P, I32, I64, I32, F, P, I64, P, I64, P, I64, P, P, SZ, P]
    for name in ("rq_lloydmax_gaussian", "rq_packed_weight_bytes", "rq_pack_weights",
                 "rq_rotate_quant_workspace_bytes", "rq_codes_mma_bytes", "rq_rotate_quant",
                 "rq_w4a4_linear", "rq_w4a4_linear_engine", "rq_rotate_quant_noalloc",
                 "rq_activation_bytes", "rq_weight_set_bytes", "rq_pack_weight_set",
                 "rq_weight_set_member", "rq_qk_norm_rope", "rq_paged_attention_workspace_bytes",
                 "rq_paged_attention", "rq_cache_evict_workspace_bytes", "rq_cache_evict"):
        getattr(L, name).restype = I32
    _lib = L
    return L


def _check(status: int):
    if status != RQ_OK:
        raise RQError(status, load().rq_last_error().decode())


def _np_ptr(a: Optional[np.ndarray]):
    if a is None:
        return None
    assert a.flags["C_CONTIGUOUS"]
    return ctypes.c_void_p(a.ctypes.data)


def _t_ptr(t):
    if t is None:
        return None
    assert t.is_contiguous(), "device buffers must be contiguous"
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, index=None):
    if stream is None:
        import torch
        # (the address alone: torch.cuda.current_stream() builds a Stream object
        # around it, which costs as much as a launch; index: the current device, where known)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index))
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


# ---------------------------------------------------------------------------
# descriptors
# ---------------------------------------------------------------------------

@dataclass
class Rotation:
    """Host description of a rotation (numpy arrays)."""
    kind: int
    K: int
    block: int = 0
    r: int = 0
    sign: Optional[np.ndarray] = None
    perm: Optional[np.ndarray] = None
    R: Optional[np.ndarray] = None
    smooth: Optional[np.ndarray] = None
    R2: Optional[np.ndarray] = None

    @staticmethod
    def rpbh(sign, perm, block):
        sign = np.ascontiguousarray(sign, np.int8)
        perm = np.ascontiguousarray(perm, np.int32)
        return Rotation(RQ_ROT_RPBH, int(sign.size), int(block), 0, sign, perm, None)

    @staticmethod
    def dense(R, r):
        R = np.ascontiguousarray(R, np.float32)
        return Rotation(RQ_ROT_DENSE, int(R.shape[0]), 0, int(r), None, None, R)

    @staticmethod
    def trdq(smooth, R1, perm, R2, block):
        """TR-DQ: smoothing multiplier [K], block rotations R1, R2 [K/b][b][b],
        zigzag permutation [K] (a gather)."""
        smooth = np.ascontiguousarray(smooth, np.float32)
        return Rotation(RQ_ROT_TRDQ, int(smooth.size), int(block), 0, None,
                        np.ascontiguousarray(perm, np.int32), np.ascontiguousarray(R1, np.float32),
                        smooth, np.ascontiguousarray(R2, np.float32))

    def c_host(self) -> c_rotation:
        ptr = (lambda a: None if a is None else a.ctypes.data)
        return c_rotation(self.kind, self.K, self.block, self.r, ptr(self.sign), ptr(self.perm),
                          ptr(self.R), ptr(self.smooth), ptr(self.R2))

    def to_device(self, device="cuda") -> "DeviceRotation":
        import torch
        d = DeviceRotation(self)
        for name in ("sign", "perm", "R", "smooth", "R2"):
            a = getattr(self, name)
            if a is not None:
                setattr(d, name, torch.from_numpy(a).to(device))
        return d


@dataclass
class DeviceRotation:
    host: Rotation
    sign: object = None
    perm: object = None
    R: object = None
    smooth: object = None
    R2: object = None

    def c_dev(self) -> c_rotation:
        h = self.host
        ptr = (lambda t: None if t is None else t.data_ptr())
        return c_rotation(h.kind, h.K, h.block, h.r, ptr(self.sign), ptr(self.perm), ptr(self.R),
                          ptr(self.smooth), ptr(self.R2))


@dataclass
class Quant:
    kind: int = RQ_Q_INT4_SYM
    a_bits: int = 4
    w_bits: int = 4
    a_levels: Optional[np.ndarray] = None
    w_levels: Optional[np.ndarray] = None

    @staticmethod
    def int4():
        return Quant(RQ_Q_INT4_SYM, 4, 4)

    @staticmethod
    def int4_asym():
        """Asymmetric per-token INT4 activations (zero point), INT4 weights."""
        return Quant(RQ_Q_INT4_ASYM, 4, 4)

    @staticmethod
    def integer(a_bits, w_bits, asym=False):
        """Integer activations of a_bits (4, 6 or 8, zero point if asym) and
        symmetric weights of w_bits (W4A4, W4A8, W8A8, W6A6); 6- and 8-bit
        codes are stored one per byte."""
        return Quant(RQ_Q_INT4_ASYM if asym else RQ_Q_INT4_SYM, a_bits, w_bits)

    @staticmethod
    def mxfp4():
        """MXFP4: E2M1 elements, one E8M0 scale per 32 coordinates."""
        return Quant(RQ_Q_MXFP4, 4, 4)

    @property
    def scale_rows(self) -> int:
        """Rows of the fp32 scale output per token set: 2 (s, z) for INT4_ASYM."""
        return 2 if self.kind == RQ_Q_INT4_ASYM else 1

    @staticmethod
    def lloydmax(a_levels, w_levels):
        a = np.ascontiguousarray(a_levels, np.float32)
        w = np.ascontiguousarray(w_levels, np.float32)
        return Quant(RQ_Q_LLOYDMAX, 4, int(np.log2(w.size)), a, w)

    def c(self) -> c_quant:
        q = c_quant(self.kind, self.a_bits, self.w_bits, 0)
        if self.a_levels is not None:
            for i, v in enumerate(self.a_levels):
                q.a_levels[i] = float(v)
        if self.w_levels is not None:
            for i, v in enumerate(self.w_levels):
                q.w_levels[i] = float(v)
        return q


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def version() -> int:
    return load().rq_version()


def lloydmax_gaussian(L: int) -> np.ndarray:
    out = np.zeros(L, np.float32)
    _check(load().rq_lloydmax_gaussian(L, _np_ptr(out)))
    return out


def packed_weight_bytes(rot: Rotation, q: Quant, N: int) -> int:
    n = ctypes.c_size_t(0)
    cr, cq = rot.c_host(), q.c()
    _check(load().rq_packed_weight_bytes(ctypes.byref(cr), ctypes.byref(cq), N, ctypes.byref(n)))
    return n.value


@dataclass
class PackedWeights:
    blob: np.ndarray                      # uint8, host
    header: c_weight_header = field(default=None)

    @property
    def N(self):
        return self.header.N

    @property
    def K(self):
        return self.header.K

    def scales(self) -> np.ndarray:
        h = self.header
        return self.blob[h.scale_offset:h.scale_offset + 4 * h.N].view(np.float32)

    def codes(self) -> np.ndarray:
        h = self.header
        return self.blob[h.codes_offset:h.codes_offset + h.N * h.row_bytes].reshape(h.N, h.row_bytes)

    def wsum(self) -> np.ndarray:
        """INT4: per-channel sums of the quantized weight codes (int32 [N])."""
        h = self.header
        return self.blob[h.wsum_offset:h.wsum_offset + 4 * h.N].view(np.int32)

    def mx_scales(self) -> np.ndarray:
        """MXFP4: the E8M0 codes, uint8 [N][K/32]."""
        h = self.header
        return self.blob[h.scale_offset:h.scale_offset + h.N * (h.K // 32)].reshape(h.N, h.K // 32)

    def i8_codes(self) -> np.ndarray:
        """INT with 8-bit activations: the int8 weight codes [N][K], read back
        from the blob's fragment order [N/32][K/32][64 lanes][16 bytes] (lane
        l: row 32 tile + l % 32, coordinates 32 kb + 16 (l / 32) .. + 15)."""
        h = self.header
        tiles = -(-h.N // 32)
        raw = self.blob[h.i8_offset:h.i8_offset + tiles * 32 * h.K].view(np.int8)
        v = raw.reshape(tiles, h.K // 32, 2, 32, 16).transpose(0, 3, 1, 2, 4).reshape(tiles * 32, h.K)
        return v[:h.N]

    def mma_tiles(self) -> np.ndarray:
        """INT4: the GEMM's FP6 fragments, uint8 [ntiles][stages][3][64][16]."""
        h = self.header
        n = h.mma_ntiles * h.mma_stages * 3 * 1024
        return self.blob[h.mma_offset:h.mma_offset + n].reshape(h.mma_ntiles, h.mma_stages, 3, 64, 16)

    def to_device(self, device="cuda") -> "DeviceWeights":
        import torch
        return DeviceWeights(self.header, torch.from_numpy(self.blob).to(device))


@dataclass
class DeviceWeights:
    header: c_weight_header
    blob: object                          # torch uint8 tensor on the GPU

    @property
    def N(self):
        return self.header.N


def pack_weights(rot: Rotation, q: Quant, W: np.ndarray) -> PackedWeights:
    """Offline fold + quantize + pack (librq host code)."""
    if W.dtype == np.float32:
        wdt = RQ_F32
    elif W.dtype == np.uint16:
        wdt = RQ_BF16
    else:
        raise TypeError("W must be float32 or bf16 bit patterns (uint16)")
    W = np.ascontiguousarray(W)
    N = int(W.shape[0])
    nbytes = packed_weight_bytes(rot, q, N)
    blob = np.zeros(nbytes, np.uint8)
    cr, cq = rot.c_host(), q.c()
    _check(load().rq_pack_weights(ctypes.byref(cr), ctypes.byref(cq), _np_ptr(W), wdt, N,
                                  _np_ptr(blob), nbytes))
    hdr = c_weight_header.from_buffer_copy(blob[:256].tobytes())
    return PackedWeights(blob, hdr)


class WeightSet:
    """A time-step set (host blob): per group the weights folded with that
    group's rotation, and the step -> group table."""

    def __init__(self, blob: np.ndarray):
        self.blob = blob
        self.device_blob = None

    def member(self, step: int):
        """(group, header, byte offset) of the blob that step uses."""
        g = ctypes.c_int32(0)
        h = ctypes.c_void_p(0)
        off = ctypes.c_int64(0)
        _check(load().rq_weight_set_member(_np_ptr(self.blob), step, ctypes.byref(g),
                                           ctypes.byref(h), ctypes.byref(off)))
        hdr = c_weight_header.from_buffer_copy(self.blob[off.value:off.value + 256].tobytes())
        return g.value, hdr, off.value

    def to_device(self, device="cuda"):
        import torch
        self.device_blob = torch.from_numpy(self.blob).to(device)
        return self

    def device_member(self, step: int) -> "DeviceWeights":
        """The DeviceWeights of the step's member: a view into the device set."""
        g, hdr, off = self.member(step)
        return DeviceWeights(hdr, self.device_blob[off:off + hdr.total_bytes])


def pack_weight_set(rots, step_group, q: Quant, W: np.ndarray) -> WeightSet:
    """Offline packing of a time-step set (rq_pack_weight_set)."""
    W = np.ascontiguousarray(W, np.float32)
    N = int(W.shape[0])
    arr = (c_rotation * len(rots))(*[r.c_host() for r in rots])
    cq = q.c()
    n = ctypes.c_size_t(0)
    _check(load().rq_weight_set_bytes(arr, len(rots), ctypes.byref(cq), N, ctypes.byref(n)))
    blob = np.zeros(n.value, np.uint8)
    sg = np.ascontiguousarray(step_group, np.int32)
    _check(load().rq_pack_weight_set(arr, len(rots), _np_ptr(sg), sg.size, ctypes.byref(cq),
                                     _np_ptr(W), RQ_F32, N, _np_ptr(blob), n.value))
    return WeightSet(blob)


def rotate_quant_workspace_bytes(rot: Rotation, q: Quant, T: int) -> int:
    n = ctypes.c_size_t(0)
    cr, cq = rot.c_host(), q.c()
    _check(load().rq_rotate_quant_workspace_bytes(ctypes.byref(cr), ctypes.byref(cq), T,
                                                  ctypes.byref(n)))
    return n.value


def activation_bytes(rot: Rotation, q: Quant, T: int):
    """(codes, scale, codes_mma) byte counts of the activation buffers."""
    c, sc, m = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
    cr, cq = rot.c_host(), q.c()
    _check(load().rq_activation_bytes(ctypes.byref(cr), ctypes.byref(cq), T, ctypes.byref(c),
                                      ctypes.byref(sc), ctypes.byref(m)))
    return c.value, sc.value, m.value


def dtype_code(t) -> int:
    import torch
    return {torch.float32: RQ_F32, torch.bfloat16: RQ_BF16, torch.int16: RQ_BF16,
            torch.uint16: RQ_BF16, torch.int32: RQ_I32}[t.dtype]


def codes_mma_bytes(rot: Rotation, T: int) -> int:
    n = ctypes.c_size_t(0)
    cr = rot.c_host()
    _check(load().rq_codes_mma_bytes(ctypes.byref(cr), T, ctypes.byref(n)))
    return n.value


def rotate_quant(drot: DeviceRotation, q: Quant, X, codes, scale, top=None, workspace=None,
                 stream=None, codes_mma=None):
    """Launch the activation kernels on `stream` (default: torch's current).
    codes and/or codes_mma (the GEMM's matrix-core layout of this format:
    FP6 fragments for INT 4-bit, int8 fragments for INT 8-bit, tiled codes
    and scales for MXFP4, bf16 level fragments for Lloyd-Max) receive the
    codes; scale holds T floats, or 2T (s then z) for INT4_ASYM."""
    cr, cq = drot.c_dev(), q.c()
    T = int(X.shape[0])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    # (MXFP4: scale is a uint8 tensor of E8M0 codes, passed as a pointer)
    _check(load().rq_rotate_quant(ctypes.byref(cr), ctypes.byref(cq), _t_ptr(X), dtype_code(X), T,
                                  _t_ptr(codes), _t_ptr(scale), _t_ptr(top), _t_ptr(codes_mma),
                                  _t_ptr(workspace), ws_bytes, _stream(stream)))


def rotate_quant_noalloc(drot: DeviceRotation, q: Quant, X, codes, scale, top=None, stream=None,
                         codes_mma=None):
    """rq_rotate_quant_noalloc: rotate_quant without a workspace (the library's
    per-device scratch serves DENSE)."""
    cr, cq = drot.c_dev(), q.c()
    T = int(X.shape[0])
    _check(load().rq_rotate_quant_noalloc(ctypes.byref(cr), ctypes.byref(cq), _t_ptr(X),
                                          dtype_code(X), T, _t_ptr(codes), _t_ptr(scale),
                                          _t_ptr(top), _t_ptr(codes_mma), _stream(stream)))


def w4a4_linear(dw: DeviceWeights, codes, scale, Y, top=None, bias=None, T=None, stream=None,
                codes_mma=None, engine="auto"):
    """Launch the low-bit GEMM; Y dtype picks the output (f32, bf16, raw int32).
    When codes_mma is given it is read instead of codes (which may be None).
    engine: "auto" (rq_w4a4_linear), or "fp6" / "int8" (rq_w4a4_linear_engine)."""
    if T is None:
        if codes is None:
            raise ValueError("T must be given when codes is None")
        T = int(codes.shape[0])
    args = (ctypes.byref(dw.header), _t_ptr(dw.blob), _t_ptr(codes), _t_ptr(scale), _t_ptr(top),
            _t_ptr(codes_mma), T, _t_ptr(bias), _t_ptr(Y), dtype_code(Y))
    if engine == "auto":
        _check(load().rq_w4a4_linear(*args, _stream(stream)))
    else:
        _check(load().rq_w4a4_linear_engine(*args, ENGINES[engine], _stream(stream)))


# ---------------------------------------------------------------------------
# attention around the linears
# ---------------------------------------------------------------------------

def _io_dtype(t) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return RQ_BF16
    if t.dtype is torch.float32:
        return RQ_F32
    raise TypeError(f"expected a float32 or bfloat16 tensor, got {t.dtype}")


def _rows(t, n, width, name):
    """Address and row stride of a 2-D (or [n][heads][D]) tensor of n rows of
    width elements, each row contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        have = shape[1]
        ok = have >= width and (stride[1] == 1 or width == 1)
    elif len(shape) == 3:
        have = shape[1] * shape[2]
        ok = have == width and stride[2] == 1 and (stride[1] == shape[2] or shape[1] == 1)
    else:
        ok = False
    if not ok:
        raise ValueError(f"{name} must be rows of {width} contiguous elements")
    if shape[0] != n:
        raise ValueError(f"{name} must have {n} rows, got {shape[0]}")
    # (a single row has no stride to keep to, nor an end beyond its width)
    return t.data_ptr(), stride[0] if n > 1 else width


def _vector(t, n, dtype, name):
    """Address of a contiguous tensor of n elements (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements")
    return t.data_ptr()


def _workspace(t):
    """Address and bytes of a workspace (None: none).  A view that repeats or
    skips elements has other memory than its element count says."""
    if t is None:
        return None, 0
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _on_device(index, *tensors):
    """Refuse buffers that are not all on the current GPU (index: the first
    one's get_device(), -1 for host memory)."""
    import torch
    if index < 0 or index != torch.cuda.current_device():
        raise ValueError(f"the buffers are on device {index}, which is not the current GPU")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a buffer is on device {t.get_device()}, not on {index}")


class KVCache:
    """A paged key-value cache over the caller's tensors: k, v [pages][heads]
    [page][D] (bfloat16, or int8 with fp32 k_scale, v_scale [pages][heads]
    [page]), table int32 [batch][pages of a sequence] and, for eviction,
    weight fp32 and pos int32 [batch][heads][pages of a sequence * page].
    The tensors are held; replacing one needs a new KVCache."""

    def __init__(self, k, v, table, k_scale=None, v_scale=None, weight=None, pos=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [pages][heads][page][D] tensors of one shape and type")
        if k.dtype not in (torch.bfloat16, torch.int8):
            raise TypeError(f"the cache must be bfloat16 or int8, got {k.dtype}")
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("k and v must be contiguous")
        if table.dim() != 2 or table.dtype is not torch.int32 or not table.is_contiguous():
            raise ValueError("table must be a contiguous int32 [batch][pages] tensor")
        i8 = k.dtype is torch.int8
        if i8 and (k_scale is None or v_scale is None):
            raise ValueError("an int8 cache needs k_scale and v_scale")
        if not i8 and (k_scale is not None or v_scale is not None):
            raise ValueError("a bfloat16 cache has no scales")
        pages, heads, page, D = k.shape
        self.k, self.v, self.table, self.k_scale, self.v_scale = k, v, table, k_scale, v_scale
        self.weight, self.pos = weight, pos
        self.heads, self.head_dim, self.page, self.batch = heads, D, page, table.shape[0]
        self.slots = table.shape[1] * page
        for name, t in (("v", v), ("table", table), ("k_scale", k_scale), ("v_scale", v_scale),
                        ("weight", weight), ("pos", pos)):
            if t is not None and t.device != k.device:
                raise ValueError(f"{name} is on {t.device}, not on {k.device}")
        n = self.batch * heads * self.slots
        self.c = c_kv_cache(
            RQ_I8 if i8 else RQ_BF16, heads, D, page, self.batch, table.shape[1], pages,
            k.data_ptr(), v.data_ptr(),
            _vector(k_scale, pages * heads * page, torch.float32, "k_scale"),
            _vector(v_scale, pages * heads * page, torch.float32, "v_scale"), table.data_ptr(),
            _vector(weight, n, torch.float32, "weight"), _vector(pos, n, torch.int32, "pos"))
        self._ref = ctypes.byref(self.c)

    @staticmethod
    def alloc(batch, heads, head_dim, max_len, page=64, int8=False, track=False, device="cuda"):
        """An empty cache of its own pages, laid out sequence by sequence."""
        import torch
        per = -(-max_len // page)
        shape = (max(1, batch * per), heads, page, head_dim)
        new = lambda dt, *s: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
        kind = torch.int8 if int8 else torch.bfloat16
        table = torch.arange(batch * per, dtype=torch.int32, device=device).reshape(batch, per)
        meta = (batch, heads, per * page)
        return KVCache(new(kind, *shape), new(kind, *shape), table,
                       new(torch.float32, *shape[:3]) if int8 else None,
                       new(torch.float32, *shape[:3]) if int8 else None,
                       new(torch.float32, *meta) if track else None,
                       new(torch.int32, *meta) if track else None)


class QKNorm:
    """Head norm and position rotation: heads, weights fp32 [D] (None: ones),
    cos and sin fp32 [rows][rot_dim / 2] (None: no rotation)."""

    def __init__(self, q_heads, kv_heads, head_dim, q_weight=None, k_weight=None, cos=None,
                 sin=None, eps=1e-6, interleaved=False):
        import torch
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.q_weight, self.k_weight, self.cos, self.sin = q_weight, k_weight, cos, sin
        rows = half = 0
        if cos is not None or sin is not None:
            if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape:
                raise ValueError("cos and sin must be [rows][rot_dim / 2] tensors of one shape")
            rows, half = cos.shape
        held = [t for t in (cos, sin, q_weight, k_weight) if t is not None]
        for t in held[1:]:
            if t.device != held[0].device:
                raise ValueError(f"the weights and tables are on {held[0].device} and {t.device}")
        self.c = c_qk_norm(q_heads, kv_heads, head_dim, 2 * half, int(bool(interleaved)), rows,
                           eps, 0, _vector(q_weight, head_dim, torch.float32, "q_weight"),
                           _vector(k_weight, head_dim, torch.float32, "k_weight"),
                           _vector(cos, rows * half, torch.float32, "cos"),
                           _vector(sin, rows * half, torch.float32, "sin"))
        self._ref = ctypes.byref(self.c)


def qk_norm_rope(norm: QKNorm, qkv, q_out, k_out=None, positions=None, cache: KVCache = None,
                 seq=None, place=None, stream=None):
    """Head norm and rotation of the rows of qkv [T][heads * D], queries to
    q_out, keys to k_out and/or with the values into the cache (slot place[t]
    of sequence seq[t], or of sequence t).  q_out and k_out may be the parts
    of qkv itself."""
    import torch
    T, D = int(qkv.shape[0]), norm.head_dim
    dt = _io_dtype(qkv)
    if q_out.dtype is not qkv.dtype or (k_out is not None and k_out.dtype is not qkv.dtype):
        raise TypeError("q_out and k_out must have qkv's type")
    qw, kw = norm.q_heads * D, norm.kv_heads * D
    _on_device(qkv.get_device(), q_out, k_out, positions, seq, place, norm.cos, norm.q_weight,
               norm.k_weight, None if cache is None else cache.k)
    p_in, ld = _rows(qkv, T, qw + kw * (1 if cache is None else 2), "qkv")
    p_q, q_ld = _rows(q_out, T, qw, "q_out")
    p_k, k_ld = (None, 0) if k_out is None else _rows(k_out, T, kw, "k_out")
    i32 = torch.int32
    _check(load().rq_qk_norm_rope(
        norm._ref, p_in, dt, ld, T, _vector(positions, T, i32, "positions"), p_q, q_ld, p_k, k_ld,
        None if cache is None else cache._ref, _vector(seq, T, i32, "seq"),
        _vector(place, T, i32, "place"), _stream(stream)))


def paged_attention_workspace_bytes(cache: KVCache, q_heads: int, max_len: int, track=False) -> int:
    n = ctypes.c_size_t(0)
    _check(load().rq_paged_attention_workspace_bytes(cache._ref, q_heads, max_len, int(track),
                                                     ctypes.byref(n)))
    return n.value


def paged_attention(q, cache: KVCache, lens, out, scale=None, max_len=None, mask=None, lse=None,
                    track=False, weight_out=None, workspace=None, stream=None):
    """Attention of q [batch][q_heads * D] over the cache: softmax of scale
    (default 1 / sqrt(D)) times the scores over the first lens[b] slots whose
    mask [batch][>= max_len] (uint8 or bool) is not 0.  lse fp32
    [batch][q_heads].  track adds the weights to the cache's weight, written
    to weight_out (default: in place)."""
    import torch
    B, D = cache.batch, cache.head_dim
    dt = _io_dtype(q)
    if out.dtype is not q.dtype:
        raise TypeError("out must have q's type")
    width = q.shape[1] if q.dim() == 2 else q.shape[1] * q.shape[2]
    if width % D:
        raise ValueError(f"a row of q must be whole heads of {D}, got {width}")
    _on_device(q.get_device(), cache.k, lens, out, mask, lse, weight_out, workspace)
    p_q, q_ld = _rows(q, B, width, "q")
    p_o, o_ld = _rows(out, B, width, "out")
    if max_len is None:
        max_len = cache.slots
    p_m, m_ld = None, 0
    if mask is not None:
        if mask.dtype not in (torch.uint8, torch.bool):
            raise TypeError("mask must be uint8 or bool")
        p_m, m_ld = _rows(mask, B, max_len, "mask")
    if track:
        if cache.weight is None:
            raise ValueError("track needs a cache with weight")
        weight_out = cache.weight if weight_out is None else weight_out
    p_ws, ws_bytes = _workspace(workspace)
    _check(load().rq_paged_attention(
        cache._ref, p_q, dt, q_ld, width // D, D ** -0.5 if scale is None else scale,
        _vector(lens, B, torch.int32, "lens"), max_len, p_m, m_ld, p_o, o_ld,
        _vector(lse, B * (width // D), torch.float32, "lse"), int(track),
        _vector(weight_out, B * cache.heads * cache.slots, torch.float32, "weight_out") if track else None,
        p_ws, ws_bytes, _stream(stream)))


def cache_evict_workspace_bytes(cache: KVCache, keep: int, max_len: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().rq_cache_evict_workspace_bytes(cache._ref, keep, max_len, ctypes.byref(n)))
    return n.value


def cache_evict(cache: KVCache, lens, keep, recent=0, sink=0, max_len=None, lens_out=None,
                weight_out=None, pos_out=None, workspace=None, stream=None):
    """Cut every sequence of the cache to its `keep` best tokens per head
    (protected, then by weight); lens, weight and pos are updated in place
    unless lens_out, weight_out and pos_out are given."""
    import torch
    B = cache.batch
    if cache.weight is None or cache.pos is None:
        raise ValueError("eviction needs a cache with weight and pos")
    _on_device(cache.k.get_device(), lens, lens_out, weight_out, pos_out, workspace)
    n = B * cache.heads * cache.slots
    p_lens = _vector(lens, B, torch.int32, "lens")
    p_ws, ws_bytes = _workspace(workspace)
    _check(load().rq_cache_evict(
        cache._ref, p_lens, cache.slots if max_len is None else max_len, keep, recent, sink,
        p_lens if lens_out is None else _vector(lens_out, B, torch.int32, "lens_out"),
        cache.c.weight if weight_out is None else _vector(weight_out, n, torch.float32, "weight_out"),
        cache.c.pos if pos_out is None else _vector(pos_out, n, torch.int32, "pos_out"),
        p_ws, ws_bytes, _stream(stream)))


# ---------------------------------------------------------------------------
# between the blocks; many queries to the same keys
# ---------------------------------------------------------------------------

NORMS = {"rms": 0, "layer": 1}


class Norm:
    """An RMS ("rms") or layer norm ("layer") over rows of `width` values, with
    weight and bias fp32 [width] (None: ones, zeros)."""

    def __init__(self, width, kind="rms", weight=None, bias=None, eps=1e-6):
        import torch
        if kind not in NORMS:
            raise ValueError(f"kind must be one of {sorted(NORMS)}, got {kind!r}")
        if weight is not None and bias is not None and weight.device != bias.device:
            raise ValueError(f"weight and bias are on {weight.device} and {bias.device}")
        self.width, self.weight, self.bias = width, weight, bias
        held = bias if weight is None else weight
        self.device_index = None if held is None else held.get_device()
        self.c = c_norm(NORMS[kind], eps, _vector(weight, width, torch.float32, "weight"),
                        _vector(bias, width, torch.float32, "bias"))
        self._ref = ctypes.byref(self.c)


class Modulation:
    """What a conditioning network gives a block: gate, shift and scale, fp32
    [rows][width] each or None, possibly parts of one wider tensor; token t
    takes row index[t] (int32), or t // per (default: one row for all)."""

    def __init__(self, gate=None, shift=None, scale=None, per=None, index=None):
        import torch
        held = [(n, t) for n, t in (("gate", gate), ("shift", shift), ("scale", scale)) if t is not None]
        if not held:
            raise ValueError("modulations need a gate, a shift or a scale")
        rows, width = held[0][1].shape
        ld = None
        for n, t in held:
            if t.dtype is not torch.float32 or t.dim() != 2 or t.shape != (rows, width) or (t.stride(1) != 1 and width > 1):
                raise ValueError(f"{n} must be a float32 [rows][width] tensor of contiguous rows, all of one shape")
            if t.device != held[0][1].device:
                raise ValueError(f"{n} is on {t.device}, not on {held[0][1].device}")
            if rows > 1:
                if ld is not None and t.stride(0) != ld:
                    raise ValueError("gate, shift and scale must have one stride from row to row")
                ld = t.stride(0)
        if index is not None and per is not None:
            per = None   # (the index alone counts)
        if index is not None and (index.dtype is not torch.int32 or index.dim() != 1 or not index.is_contiguous()):
            raise ValueError("index must be a contiguous int32 [tokens] tensor")
        if index is not None and index.device != held[0][1].device:
            raise ValueError(f"index is on {index.device}, not on {held[0][1].device}")
        self.gate, self.shift, self.scale, self.index = gate, shift, scale, index
        self.rows, self.width = rows, width
        ptr = (lambda t: None if t is None else t.data_ptr())
        self.c = c_modulation(rows, 0, width if ld is None else ld, (1 << 62) if per is None else per, ptr(index),
                              ptr(gate), ptr(shift), ptr(scale))
        self._ref = ctypes.byref(self.c)
        self.device_index = held[0][1].get_device()


def block_norm(x, z=None, pre: Norm = None, y=None, post: Norm = None, h=None, mod: Modulation = None, alpha=1.0,
               beta=1.0, stream=None):
    """The residual stream between two blocks in one pass: h = alpha x + beta gate
    post(y) and z = pre(h) (1 + scale) + shift, for rows x, h [T][width] of one
    type and y, z of one (fp32 or bf16 each).  Leave out y (nothing is added), h
    or z (not written).  h may be x itself, and z may be y."""
    if x.dim() != 2:
        raise ValueError("x must be rows [T][width]")
    T, K = x.shape
    index = x.get_device()
    if h is not None and h.dtype is not x.dtype:
        raise TypeError("h must have x's type")
    if y is not None and z is not None and y.dtype is not z.dtype:
        raise TypeError("z must have y's type")
    for n in (post, pre, mod):
        if n is not None:
            if n.width != K:
                raise ValueError(f"the rows have {K} values, a norm or the modulations {n.width}")
            if n.device_index is not None and n.device_index != index:
                raise ValueError(f"a norm or the modulations are on device {n.device_index}, x on {index}")
    if mod is not None and mod.index is not None and mod.index.numel() != T:
        raise ValueError(f"index must have {T} elements, got {mod.index.numel()}")
    _on_device(index, y, h, z)
    p_x, x_ld = _rows(x, T, K, "x")
    p_y, y_ld = (None, 0) if y is None else _rows(y, T, K, "y")
    p_h, h_ld = (None, 0) if h is None else _rows(h, T, K, "h")
    p_z, z_ld = (None, 0) if z is None else _rows(z, T, K, "z")
    io = y if y is not None else z
    _check((_lib or load()).rq_block_norm(
        None if post is None else post._ref, None if pre is None else pre._ref, None if mod is None else mod._ref, K,
        p_x, _io_dtype(x), x_ld, p_y, RQ_BF16 if io is None else _io_dtype(io), y_ld, T, alpha, beta, p_h, h_ld, p_z,
        z_ld, _stream(stream, index)))


def _tokens(t, name):
    """Address, token stride and sequence stride of a [batch][tokens][heads][D]
    tensor whose tokens' heads lie together."""
    B, T, H, D = t.shape
    s = t.stride()
    if t.numel() == 0:
        return t.data_ptr(), H * D, 0
    if (s[3] != 1 and D > 1) or (s[2] != D and H > 1):
        raise ValueError(f"the heads of a token of {name} must lie together")
    # (single tokens and sequences have no stride to keep to)
    return t.data_ptr(), s[1] if T > 1 else H * D, s[0] if B > 1 else 0


class States:
    """Keys and values of a batch, bf16 [batch][tokens][heads][D] (views of a
    projection's output are fine; so is one sequence expanded over the batch),
    with lens int32 [batch] and mask uint8 or bool [batch][tokens] (None: all
    tokens count).  The tensors are held."""

    def __init__(self, k, v, lens=None, mask=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [batch][tokens][heads][D] tensors of one shape")
        if k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16:
            raise TypeError(f"k and v must be bfloat16, got {k.dtype} and {v.dtype}")
        B, S, H, D = k.shape
        for name, t in (("v", v), ("lens", lens), ("mask", mask)):
            if t is not None and t.device != k.device:
                raise ValueError(f"{name} is on {t.device}, not on {k.device}")
        p_m, m_ld = None, 0
        if mask is not None:
            if mask.dtype not in (torch.uint8, torch.bool):
                raise TypeError("mask must be uint8 or bool")
            if mask.shape != (B, S) or (mask.stride(1) != 1 and S > 1):
                raise ValueError(f"mask must be rows [{B}][{S}]")
            p_m, m_ld = mask.data_ptr(), mask.stride(0) if B > 1 else S
        (p_k, k_ld, k_b), (p_v, v_ld, v_b) = _tokens(k, "k"), _tokens(v, "v")
        self.k, self.v, self.lens, self.mask = k, v, lens, mask
        self.batch, self.keys, self.heads, self.head_dim = B, S, H, D
        self.c = c_states(H, D, B, 0, S, k_ld, v_ld, k_b, v_b, m_ld, p_k, p_v,
                          _vector(lens, B, torch.int32, "lens"), p_m)
        self._ref = ctypes.byref(self.c)


def _code(dtype) -> int:
    import torch
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"expected torch.float32 or torch.bfloat16, got {dtype}")
    return RQ_BF16 if dtype is torch.bfloat16 else RQ_F32


def cross_attention_workspace_bytes(states: States, queries: int, q_heads: int, dtype) -> int:
    """dtype: the queries' torch type."""
    n = ctypes.c_size_t(0)
    _check(load().rq_cross_attention_workspace_bytes(states._ref, queries, q_heads, _code(dtype), ctypes.byref(n)))
    return n.value


def cross_attention(q, states: States, out, scale=None, q_lens=None, lse=None, workspace=None, stream=None):
    """Attention of q [batch][queries][q_heads][D] to its sequences' states
    (softmax of scale, default 1 / sqrt(D), times the scores), to out of q's
    shape and type; lse fp32 [batch][queries][q_heads].  Rows from q_lens[b]
    (int32) on are left as they are."""
    import torch
    if q.dim() != 4 or q.shape != out.shape:
        raise ValueError("q and out must be [batch][queries][heads][D] tensors of one shape")
    if out.dtype is not q.dtype:
        raise TypeError("out must have q's type")
    B, T, H, D = q.shape
    if B != states.batch or D != states.head_dim:
        raise ValueError(f"q has {B} sequences of heads of {D}, the states {states.batch} of {states.head_dim}")
    index = q.get_device()
    _on_device(index, out, states.k, q_lens, lse, workspace)
    (p_q, q_ld, q_b), (p_o, o_ld, o_b) = _tokens(q, "q"), _tokens(out, "out")
    p_ws, ws_bytes = _workspace(workspace)
    _check(load().rq_cross_attention(
        states._ref, p_q, _io_dtype(q), q_ld, q_b, T, H, D ** -0.5 if scale is None else scale,
        _vector(q_lens, B, torch.int32, "q_lens"), p_o, o_ld, o_b, _vector(lse, B * T * H, torch.float32, "lse"),
        p_ws, ws_bytes, _stream(stream, index)))


def prefix_attention_workspace_bytes(cache: KVCache, q_heads: int, prefix: int, max_len: int, dtype) -> int:
    """dtype: the queries' torch type."""
    n = ctypes.c_size_t(0)
    _check(load().rq_prefix_attention_workspace_bytes(cache._ref, q_heads, _code(dtype), prefix, max_len, ctypes.byref(n)))
    return n.value


def prefix_attention(q, cache: KVCache, prefix_table, prefix, lens, out, scale=None, max_len=None, mask=None, lse=None,
                     workspace=None, stream=None):
    """paged_attention for a batch that shares its first `prefix` tokens, which
    lie in the pages of prefix_table int32 [>= ceil(prefix / page)] and are read
    once for all.  lens counts the prefix too; columns of mask below it are not
    read.  A sequence shorter than the prefix gets 0."""
    import torch
    B, D = cache.batch, cache.head_dim
    dt = _io_dtype(q)
    if out.dtype is not q.dtype:
        raise TypeError("out must have q's type")
    width = q.shape[1] if q.dim() == 2 else q.shape[1] * q.shape[2]
    if width % D:
        raise ValueError(f"a row of q must be whole heads of {D}, got {width}")
    index = q.get_device()
    _on_device(index, cache.k, prefix_table, lens, out, mask, lse, workspace)
    p_q, q_ld = _rows(q, B, width, "q")
    p_o, o_ld = _rows(out, B, width, "out")
    if max_len is None:
        max_len = cache.slots
    if prefix_table is not None:
        n = -(-prefix // cache.page)
        if prefix_table.dim() != 1 or prefix_table.numel() < n or prefix_table.dtype is not torch.int32 or not prefix_table.is_contiguous():
            raise ValueError(f"prefix_table must be a contiguous int32 tensor of at least {n} pages")
    p_m, m_ld = None, 0
    if mask is not None:
        if mask.dtype not in (torch.uint8, torch.bool):
            raise TypeError("mask must be uint8 or bool")
        p_m, m_ld = _rows(mask, B, max_len, "mask")
    p_ws, ws_bytes = _workspace(workspace)
    _check(load().rq_prefix_attention(
        cache._ref, None if prefix_table is None or prefix == 0 else prefix_table.data_ptr(), prefix, p_q, dt, q_ld,
        width // D, D ** -0.5 if scale is None else scale, _vector(lens, B, torch.int32, "lens"), max_len, p_m, m_ld,
        p_o, o_ld, _vector(lse, B * (width // D), torch.float32, "lse"), p_ws, ws_bytes, _stream(stream, index)))
