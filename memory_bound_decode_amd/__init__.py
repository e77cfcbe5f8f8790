"""Python binding of libmbd (include/mbd.h): weight-only low-bit decode GEMV on MI355X.

The functions keep the C names and only marshal arguments: numpy arrays for the
CPU packer, torch device tensors (memory and streams) for the GPU calls.  Every
computation runs in libmbd; if the library is not built, importing the native
symbols raises.
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np

from ._native import (  # noqa: F401
    MBD_CASSANDRA, MBD_EALIGN, MBD_EFORMAT, MBD_EHIP, MBD_EINVAL, MBD_ENOMEM, MBD_ERANGE,
    MBD_CASSANDRA_MX, MBD_ESHAPE, MBD_INT4_G128, MBD_MX32, MBD_OK, MBD_TERNARY_B128, MBD_TERNARY_SKIP, MbdDWeights, MbdError,
    MbdEncodePlan, MbdPackParams, MbdSection, MbdStats, check, lib,
    MBD_BF16, MBD_F32, MBD_KV_E4M3, MBD_KV_INT8, MbdKvAttnArgs, MbdKvCache, MbdKvPool,
)

SECTION_NAMES = {
    MBD_TERNARY_B128: ["codes", "scales"],
    MBD_INT4_G128: ["codes", "scales"],
    MBD_CASSANDRA: ["bitmap", "spec_nib", "unary", "codebook", "bitoff", "kprefix", "lo_nib", "pruned"],
    MBD_MX32: ["mx_exp", "mx_sign", "mx_mag"],
    MBD_TERNARY_SKIP: ["codes", "scales", "slabs", "tile_base"],
    MBD_CASSANDRA_MX: ["bitmap", "mx_nib", "mx_sign", "mx_exp", "kprefix"],
}
SPEC_SECTIONS = ("bitmap", "spec_nib", "unary", "codebook", "bitoff", "kprefix")


class Packed:
    """Owns an mbd_packed handle (host sections written by the C++ packer)."""

    def __init__(self, handle: ctypes.c_void_p, fmt: int, M: int, K: int, n_mats: int = 1):
        self._h = handle
        self._free = lib().mbd_packed_free        # the library that allocated the handle frees it
        self.fmt, self.M, self.K, self.n_mats = fmt, M, K, n_mats

    def __del__(self):
        h, free = getattr(self, "_h", None), getattr(self, "_free", None)
        if h is not None and h.value and free is not None:
            free(h)
            self._h = None

    def sections(self) -> dict:
        """name -> (uint8 copy of the padded section, meaningful byte count)."""
        L = lib()
        n = ctypes.c_int32(0)
        check(L.mbd_packed_sections(self._h, None, 0, ctypes.byref(n)), "mbd_packed_sections")
        arr = (MbdSection * n.value)()
        check(L.mbd_packed_sections(self._h, arr, n.value, ctypes.byref(n)), "mbd_packed_sections")
        out = {}
        for s in arr:
            buf = (ctypes.c_uint8 * s.padded_bytes).from_address(s.data)
            out[s.name.decode()] = (np.frombuffer(buf, dtype=np.uint8).copy(), int(s.bytes))
        return out

    def section(self, name: str, dtype) -> np.ndarray:
        """Meaningful bytes of one section viewed as ``dtype``."""
        raw, nbytes = self.sections()[name]
        return raw[:nbytes].view(dtype)

    def stats(self) -> MbdStats:
        st = MbdStats()
        check(lib().mbd_packed_stats(self._h, ctypes.byref(st)), "mbd_packed_stats")
        return st

    def validate(self) -> None:
        check(lib().mbd_validate(self._h), "mbd_validate")


def mbd_pack(fmt: int, w_bits: np.ndarray, act_norm: np.ndarray | None = None,
             keep_num: int = 3, keep_den: int = 10, n_mats: int = 1) -> Packed:
    """Pack bf16 bits [M][K] (numpy uint16) on the CPU; n_mats > 1 packs the rows as
    that many stacked matrices (ternary / INT4, for the expert GEMV)."""
    w = np.ascontiguousarray(w_bits, dtype=np.uint16)
    if w.ndim != 2:
        raise ValueError("w_bits must be 2-D [M][K]")
    M, K = w.shape
    nrm = None
    if act_norm is not None:
        nrm = np.ascontiguousarray(act_norm, dtype=np.float32)
    params = MbdPackParams(keep_num, keep_den, n_mats)
    h = ctypes.c_void_p()
    st = lib().mbd_pack(fmt, w.ctypes.data_as(ctypes.POINTER(ctypes.c_uint16)), M, K,
                        None if nrm is None else nrm.ctypes.data, ctypes.byref(params), ctypes.byref(h))
    check(st, "mbd_pack")
    return Packed(h, fmt, M, K, n_mats)


class DeviceWeights:
    """Device copies (torch uint8 tensors) of packed sections plus the mbd_dweights
    descriptor that points at them.  ``n_mats`` > 1 describes stacked matrices."""

    def __init__(self, packed: Packed, device="cuda", n_mats: int = 1, only=None):
        import torch
        secs = packed.sections()
        names = SECTION_NAMES[packed.fmt]
        st = packed.stats()
        self.tensors = {}
        self.desc = MbdDWeights()
        self.desc.fmt = packed.fmt
        self.desc.n_sym = st.n_sym
        if packed.M % n_mats:
            raise ValueError("rows not divisible by n_mats")
        if n_mats != packed.n_mats and packed.fmt in (MBD_TERNARY_B128, MBD_INT4_G128):
            raise ValueError("packed as %d matrices, described as %d: pack with mbd_pack(..., n_mats=%d)"
                             % (packed.n_mats, n_mats, n_mats))
        self.desc.M = packed.M // n_mats
        self.desc.K = packed.K
        self.desc.n_kept = st.n_kept
        self.desc.n_mats = n_mats
        self.bytes = {}
        for i, name in enumerate(names):
            raw, nbytes = secs[name]
            self.bytes[name] = nbytes
            if only is not None and name not in only:
                self.desc.sec[i] = None
                continue
            t = torch.from_numpy(raw).to(device)
            self.tensors[name] = t
            self.desc.sec[i] = t.data_ptr()
        self.fmt, self.M, self.K, self.n_mats = packed.fmt, self.desc.M, packed.K, n_mats

    def ref(self):
        return ctypes.byref(self.desc)


def to_device(packed: Packed, device="cuda", n_mats: int = 1, only=None) -> DeviceWeights:
    return DeviceWeights(packed, device, n_mats, only)


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def mbd_gemv(dw: DeviceWeights, x, y, stream=None) -> None:
    """y [B][M] fp32 = W x for bf16 x [B][K] (torch tensors on the device)."""
    check(lib().mbd_gemv(dw.ref(), _ptr(x), int(x.shape[0]), _ptr(y), _stream(stream)), "mbd_gemv")


def mbd_dequant(dw: DeviceWeights, out, stream=None) -> None:
    check(lib().mbd_dequant(dw.ref(), _ptr(out), _stream(stream)), "mbd_dequant")


def mbd_moe_workspace_bytes(n_mats: int, T: int, k: int) -> int:
    b = ctypes.c_uint64(0)
    check(lib().mbd_moe_workspace_bytes(n_mats, T, k, ctypes.byref(b)), "mbd_moe_workspace_bytes")
    return int(b.value)


def mbd_moe_gemv(dw: DeviceWeights, route, x, x_per_pair: bool, y, ws, stream=None) -> None:
    T, k = int(route.shape[0]), int(route.shape[1])
    check(lib().mbd_moe_gemv(dw.ref(), _ptr(route), T, k, _ptr(x), int(bool(x_per_pair)), _ptr(y),
                             _ptr(ws), int(ws.numel() * ws.element_size()), _stream(stream)), "mbd_moe_gemv")


def mbd_moe_gemv_noalloc(dw: DeviceWeights, route, x, x_per_pair: bool, y, stream=None) -> None:
    """mbd_moe_gemv without a workspace (the library's static device scratch)."""
    T, k = int(route.shape[0]), int(route.shape[1])
    check(lib().mbd_moe_gemv_noalloc(dw.ref(), _ptr(route), T, k, _ptr(x), int(bool(x_per_pair)), _ptr(y),
                                     _stream(stream)), "mbd_moe_gemv_noalloc")


def mbd_spec_decode(dw: DeviceWeights, out, stream=None) -> None:
    check(lib().mbd_spec_decode(dw.ref(), _ptr(out), _stream(stream)), "mbd_spec_decode")


def mbd_spec_gemv(dw: DeviceWeights, x, y, stream=None) -> None:
    check(lib().mbd_spec_gemv(dw.ref(), _ptr(x), int(x.shape[0]), _ptr(y), _stream(stream)), "mbd_spec_gemv")


def mbd_verify_restore(dw: DeviceWeights, out, stream=None) -> None:
    check(lib().mbd_verify_restore(dw.ref(), _ptr(out), _stream(stream)), "mbd_verify_restore")


def mbd_encode_workspace_bytes(M: int) -> int:
    n = ctypes.c_uint64(0)
    check(lib().mbd_encode_workspace_bytes(M, ctypes.byref(n)), "mbd_encode_workspace_bytes")
    return int(n.value)


def mbd_encode_plan(w, act_norm, keep_num: int, keep_den: int, ws, stream=None) -> MbdEncodePlan:
    """Device encoder, first call (synchronises the stream): section sizes of the
    Cassandra sections of device bf16 w [M][K] (int16 tensor) and fp32 act_norm."""
    M, K = w.shape
    plan = MbdEncodePlan()
    check(lib().mbd_encode_plan(_ptr(w), _ptr(act_norm), M, K, keep_num, keep_den, _ptr(ws), ws.numel() * ws.element_size(),
                                ctypes.byref(plan), _stream(stream)), "mbd_encode_plan")
    return plan


def mbd_encode_cassandra(w, act_norm, keep_num: int, keep_den: int, plan: MbdEncodePlan, sections, ws, stream=None) -> None:
    """Device encoder, second call: writes the eight sections into ``sections``
    (device uint8 tensors of at least plan.padded_bytes[i] bytes each)."""
    M, K = w.shape
    arr = (ctypes.c_void_p * 8)(*[t.data_ptr() for t in sections])
    check(lib().mbd_encode_cassandra(_ptr(w), _ptr(act_norm), M, K, keep_num, keep_den, ctypes.byref(plan), arr, _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), "mbd_encode_cassandra")


# ------------------------------------------------------------------ KV cache

# A decode step makes these calls for every layer, and a launch takes 3 us: the checks look
# at each tensor once, and build nothing.

def _gpu(name, t):
    """The index of the GPU that holds ``t``, which has to be the current one: its stream is taken."""
    import torch
    here = t.get_device()
    if here < 0 or here != torch.cuda.current_device():
        raise ValueError("%s is on %s, not on the current GPU" % (name, t.device))
    return here


def _refuse(here, name, t, dtype, n=None):
    if t.get_device() != here:
        raise ValueError("%s is on %s, not on the current GPU" % (name, t.device))
    raise ValueError("%s must be a contiguous %s tensor%s" % (name, dtype, "" if n is None else " of %d values" % n))


def _held(here, name, held):
    """A cache's or pool's memory is where it was built, whatever GPU is current now."""
    if held.gpu != here:
        raise ValueError("the %s is on cuda:%d, not on the current GPU" % (name, held.gpu))


def _ints(here, i32, *checks):
    """(name, tensor, values) each: contiguous int32 on GPU ``here``."""
    for name, t, n in checks:
        if t.dtype is not i32 or t.numel() != n or t.get_device() != here or not t.is_contiguous():
            _refuse(here, name, t, "int32", n)


def _rows(here, name, t, heads, dim, dtypes):
    """[T][heads][dim] with dense rows on GPU ``here``; returns the elements from one token to the next."""
    if t.dim() != 3 or t.dtype not in dtypes:
        raise ValueError("%s must be [T][%d][%d] of %s" % (name, heads, dim, " or ".join(str(d) for d in dtypes)))
    (n, h, d), (s0, s1, s2) = t.shape, t.stride()
    if h != heads or d != dim:
        raise ValueError("%s must be [T][%d][%d]" % (name, heads, dim))
    if (heads > 1 and s1 != dim) or s2 != 1:
        raise ValueError("%s: one token's heads must be dense" % name)
    if t.get_device() != here:
        _refuse(here, name, t, "")
    return s0 if n > 1 else heads * dim


def _queue(stream, here):
    """The raw handle of ``stream``, or of the current one (0: the default stream)."""
    if stream is not None:
        return int(stream)
    import torch
    return torch._C._cuda_getCurrentRawStream(here)


class KvCache:
    """An 8-bit paged KV cache over the caller's device tensors: codes uint8
    [n_blocks][n_heads][block_size * head_dim] in the tile order of mbd.h, scales fp32
    [n_blocks][n_heads].  Holds the tensors and the mbd_kv_cache that points at them."""

    def __init__(self, fmt: int, block_size: int, head_dim: int, k_codes, v_codes, k_scale, v_scale):
        import torch
        if k_codes.dim() != 3 or k_codes.shape[2] != block_size * head_dim:
            raise ValueError("codes must be [n_blocks][n_heads][block_size * head_dim]")
        for t, shape, dtype in ((k_codes, k_codes.shape, torch.uint8), (v_codes, k_codes.shape, torch.uint8),
                                (k_scale, k_codes.shape[:2], torch.float32), (v_scale, k_codes.shape[:2], torch.float32)):
            if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
                raise ValueError("codes are contiguous uint8 tensors of one shape, scales contiguous fp32 [n_blocks][n_heads]")
        for t in (k_codes, v_codes, k_scale, v_scale):
            self.gpu = _gpu("the cache", t)
        self.tensors = dict(k_codes=k_codes, v_codes=v_codes, k_scale=k_scale, v_scale=v_scale)
        self.fmt, self.block_size, self.n_heads, self.head_dim = fmt, block_size, k_codes.shape[1], head_dim
        self.n_blocks = k_codes.shape[0]
        self.desc = MbdKvCache(fmt, block_size, self.n_heads, head_dim, self.n_blocks, k_codes.data_ptr(), v_codes.data_ptr(),
                               k_scale.data_ptr(), v_scale.data_ptr())
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, fmt: int, n_blocks: int, n_heads: int, head_dim: int, block_size: int, device="cuda"):
        import torch
        codes = [torch.empty((n_blocks, n_heads, block_size * head_dim), dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.empty((n_blocks, n_heads), dtype=torch.float32, device=device) for _ in range(2)]
        return cls(fmt, block_size, head_dim, *codes, *scales)

    def ref(self):
        return self._ref


class KvPool:
    """Block tables int32 [n_seqs][max_blocks] and the stack of free blocks int32 [n_blocks]."""

    def __init__(self, block_size: int, block_table, free_blocks):
        if block_table.dim() != 2 or free_blocks.dim() != 1:
            raise ValueError("block_table must be [n_seqs][max_blocks], free_blocks [n_blocks]")
        import torch
        self.gpu = _gpu("block_table", block_table)
        _ints(self.gpu, torch.int32, ("block_table", block_table, block_table.numel()),
              ("free_blocks", free_blocks, free_blocks.numel()))
        self.block_table, self.free_blocks, self.block_size = block_table, free_blocks, block_size
        self.n_seqs, self.max_blocks = block_table.shape
        self.desc = MbdKvPool(self.n_seqs, block_size, self.max_blocks, free_blocks.shape[0], block_table.data_ptr(),
                              free_blocks.data_ptr())
        self._ref = ctypes.byref(self.desc)

    def ref(self):
        return self._ref


def mbd_kv_slots(pool: KvPool, new_tokens, lens, held, n_free, seq_start, slots, positions, lens_out, held_out, n_free_out,
                 status, stream=None) -> None:
    """One step's block tables, slot map and ragged starts from request lengths; slots has
    one value for each row of the step's token batch, positions may be None."""
    import torch
    n, T, here, i32 = pool.n_seqs, slots.numel(), _gpu("slots", slots), torch.int32
    _held(here, "pool", pool)
    _ints(here, i32, ("new_tokens", new_tokens, n), ("lens", lens, n), ("held", held, n), ("n_free", n_free, 1), ("seq_start", seq_start, n + 1),
          ("slots", slots, T), ("lens_out", lens_out, n), ("held_out", held_out, n), ("n_free_out", n_free_out, 1), ("status", status, n))
    if positions is not None:
        _ints(here, i32, ("positions", positions, T))
    st = lib().mbd_kv_slots(pool._ref, new_tokens.data_ptr(), lens.data_ptr(), held.data_ptr(), n_free.data_ptr(), T, seq_start.data_ptr(),
                            slots.data_ptr(), None if positions is None else positions.data_ptr(), lens_out.data_ptr(),
                            held_out.data_ptr(), n_free_out.data_ptr(), status.data_ptr(), _queue(stream, here))
    check(st, "mbd_kv_slots")


def mbd_kv_append(cache: KvCache, k, v, slots, stream=None) -> None:
    """Quantise k, v [T][n_heads][head_dim] (bf16 or fp32; rows may be slices) into their slots."""
    import torch
    here, heads, dim, T, dt = _gpu("k", k), cache.n_heads, cache.head_dim, k.shape[0], k.dtype
    _held(here, "cache", cache)
    ks, vs = _rows(here, "k", k, heads, dim, (torch.bfloat16, torch.float32)), _rows(here, "v", v, heads, dim, (dt,))
    if v.shape[0] != T:
        raise ValueError("k and v must have as many tokens")
    _ints(here, torch.int32, ("slots", slots, T))
    st = lib().mbd_kv_append(cache._ref, k.data_ptr(), v.data_ptr(), MBD_BF16 if dt is torch.bfloat16 else MBD_F32, ks, vs, slots.data_ptr(), T,
                             _queue(stream, here))
    check(st, "mbd_kv_append")


def mbd_kv_gather(cache: KvCache, slots, k_out, v_out, stream=None) -> None:
    """Dense keys and values [T][n_heads][head_dim] (bf16 or fp32) of the tokens in ``slots``."""
    import torch
    here, heads, dim, T, dt = _gpu("k_out", k_out), cache.n_heads, cache.head_dim, k_out.shape[0], k_out.dtype
    _held(here, "cache", cache)
    _rows(here, "k_out", k_out, heads, dim, (torch.bfloat16, torch.float32))
    _rows(here, "v_out", v_out, heads, dim, (dt,))
    if v_out.shape[0] != T or not k_out.is_contiguous() or not v_out.is_contiguous():
        raise ValueError("k_out and v_out must be contiguous and alike")
    _ints(here, torch.int32, ("slots", slots, T))
    st = lib().mbd_kv_gather(cache._ref, slots.data_ptr(), T, MBD_BF16 if dt is torch.bfloat16 else MBD_F32, k_out.data_ptr(), v_out.data_ptr(),
                             _queue(stream, here))
    check(st, "mbd_kv_gather")


def mbd_kv_attn_workspace_bytes(cache: KvCache, n_heads: int, n_seqs: int, max_new: int, max_blocks: int) -> int:
    """Bytes of mbd_kv_attn's workspace for these sizes and all smaller ones."""
    b = ctypes.c_uint64(0)
    check(lib().mbd_kv_attn_workspace_bytes(cache.ref(), n_heads, n_seqs, max_new, max_blocks, ctypes.byref(b)),
          "mbd_kv_attn_workspace_bytes")
    return int(b.value)


_ATTN_ARGS = struct.Struct("@6i2fPqq")                 # MbdKvAttnArgs, in the machine's own layout


def mbd_kv_attn(cache: KvCache, q, seq_start, lens, block_table, out, ws=None, max_new: int = 1, scale: float | None = None,
                softcap: float = 0.0, window: int = 0, slopes=None, lse=None, stream=None) -> None:
    """Causal attention of the requests' newest tokens q [T][n_heads][head_dim] bf16 over
    their cached tokens, into out (alike; rows may be slices) and lse fp32 [T][n_heads].
    scale defaults to head_dim ** -0.5."""
    import torch
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [T][n_heads][head_dim], block_table [n_seqs][max_blocks]")
    here, (T, heads, dim), (n, width) = _gpu("q", q), q.shape, block_table.shape
    _held(here, "cache", cache)
    qs = _rows(here, "q", q, heads, cache.head_dim, (torch.bfloat16,))
    outs = _rows(here, "out", out, heads, dim, (torch.bfloat16,))
    if out.shape[0] != T:
        raise ValueError("out must have as many rows as q")
    _ints(here, torch.int32, ("block_table", block_table, n * width), ("lens", lens, n), ("seq_start", seq_start, n + 1))
    for name, t, size in (("lse", lse, T * heads), ("slopes", slopes, heads)):
        if t is not None and (t.dtype is not torch.float32 or t.numel() != size or t.get_device() != here or not t.is_contiguous()):
            _refuse(here, name, t, "fp32", size)
    if ws is not None and (ws.get_device() != here or not ws.is_contiguous()):
        _refuse(here, "ws", ws, "")
    args = _ATTN_ARGS.pack(heads, n, width, T, max_new, window, dim ** -0.5 if scale is None else scale, softcap,
                           0 if slopes is None else slopes.data_ptr(), qs, outs)
    st = lib().mbd_kv_attn(cache._ref, args, q.data_ptr(), seq_start.data_ptr(), lens.data_ptr(), block_table.data_ptr(), out.data_ptr(),
                           None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes,
                           _queue(stream, here))
    check(st, "mbd_kv_attn")


def mbd_probe_stream_read(src, sink, blocks: int, threads: int, stream=None) -> None:
    """Streaming-read probe over the whole of ``src`` (a device tensor); measurement aid."""
    check(lib().mbd_probe_stream_read(_ptr(src), int(src.numel() * src.element_size()), _ptr(sink), int(blocks),
                                      int(threads), _stream(stream)), "mbd_probe_stream_read")
