"""Python binding of libcf (argument marshalling only).

Every function here forwards to the C ABI declared in ``include/cf.h``; all
arithmetic runs in the HIP kernels of ``libcf.so``.  PyTorch supplies device memory
and streams.  Importing this module fails loudly when ``libcf.so`` is missing: there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcf.so")

CF_BF16, CF_F32 = 0, 1
CF_MODE_NOEF, CF_MODE_NAIVE = 1, 2
CF_NORM_NONE, CF_NORM_RMS, CF_NORM_LAYER = 0, 1, 2
CF_ROPE_NONE, CF_ROPE_INTERLEAVED, CF_ROPE_HALF = 0, 1, 2
CF_ATTN_CAUSAL = 1
GROUP = 128

STATUS = {0: "CF_OK", -1: "CF_E_NULL", -2: "CF_E_SHAPE", -3: "CF_E_ALIGN", -4: "CF_E_ARG",
          -5: "CF_E_ALIAS", -6: "CF_E_WORKSPACE", -7: "CF_E_DEVICE", -8: "CF_E_HIP", -9: "CF_E_SCRATCH"}
NOALLOC_SCRATCH_BYTES = 64 << 20  # CF_NOALLOC_SCRATCH_BYTES

# name -> (restype, argtypes) ; i=int, l=int64, p=pointer, z=size_t
_SIG = {
    "cf_init_state": ("i", "ippplp"),
    "cf_compress": ("i", "iippppplp"),
    "cf_decompress": ("i", "ippplp"),
    "cf_decompress_bf16": ("i", "ipppplp"),
    "cf_compress_ablation": ("i", "iiipppppl" "p"),
    "cf_topk_compress": ("i", "iippppplp"),
    "cf_topk_decompress": ("i", "ippplp"),
    "cf_lowrank_compress": ("i", "ipppllii" "iipppppp" "zp"),
    "cf_lowrank_compress_noalloc": ("i", "ipppllii" "iippppp" "p"),
    "cf_lowrank_decompress": ("i", "ipppp" "pllii" "p"),
    "cf_lowrank_workspace_bytes": ("z", "llii"),
    "cf_codes_bytes": ("l", "li"),
    "cf_qk_norm_rope": ("i", "iliii" "rrrr" "ipppp" "fi" "ppli" "pp"),
    "cf_kv4_cache_bytes": ("l", "liii"),
    "cf_kv4_append": ("i", "irrpl" "pliii" "p"),
    "cf_kv4_read": ("i", "ipliii" "plrr" "p"),
    "cf_kv4_attention": ("i", "irli" "pliii" "ipipp" "liif" "rppzp"),
    "cf_kv4_attention_workspace_bytes": ("z", "iliii"),
    "cf_kv8_cache_bytes": ("l", "liii"),
    "cf_kv8_append": ("i", "irrlp" "liiii" "pipp" "p"),
    "cf_kv8_read": ("i", "ipliii" "plrr" "p"),
    "cf_kv8_attention": ("i", "irli" "pliii" "ipipp" "liif" "rppzp"),
    "cf_kv8_attention_workspace_bytes": ("z", "iliii"),
    "cf_attention": ("i", "irli" "rrl" "iii" "pp" "liif" "rppzp"),
    "cf_attention_workspace_bytes": ("z", "iliii"),
    "cf_pages_workspace_bytes": ("z", "li"),
    "cf_pages_resize": ("i", "gg" "liii" "pp" "pzp"),
    "cf_pages_fork": ("i", "gg" "liii" "pppp" "pzp"),
    "cf_pages_fork_own": ("i", "gg" "liii" "pppp" "pzp"),
    "cf_pages_compact": ("i", "gg" "lii" "ppp" "pzp"),
    "cf_pages_copy": ("i", "pllil" "pplpp"),
    "cf_strerror": ("s", "i"),
    "cf_abi_version": ("i", ""),
}


class Rows(ctypes.Structure):
    """cf_rows: where the rows of a (tokens, heads, head_dim) tensor start."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Pages(ctypes.Structure):
    """cf_pages: the arrays that say who holds which page."""
    _fields_ = [("refs", ctypes.c_void_p), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p)]


# r: a pointer to cf_rows, g: a pointer to cf_pages, f: float
_CT = {"r": ctypes.POINTER(Rows), "g": ctypes.POINTER(Pages), "f": ctypes.c_float, "i": ctypes.c_int, "l": ctypes.c_int64, "p": ctypes.c_void_p, "z": ctypes.c_size_t,
       "s": ctypes.c_char_p}


class CFError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({strerror(status)})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(the HIP library is required; there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIG.items():
        f = getattr(lib, name)
        f.restype = _CT[res]
        f.argtypes = [_CT[c] for c in args]
    return lib


lib = _load()


def strerror(status: int) -> str:
    return lib.cf_strerror(status).decode()


def _check(fn: str, rc: int):
    if rc != 0:
        raise CFError(fn, rc)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libcf takes device tensors (a host pointer would fault the kernel)")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{torch.cuda.current_device()} "
                         "(libcf launches on the current device)")
    if not t.is_contiguous():
        raise ValueError("libcf needs contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _need(name: str, t: torch.Tensor | None, nbytes: int, valid: bool = True):
    """The C ABI cannot see buffer sizes: refuse a buffer smaller than the call uses.
    With ``valid`` False (an argument the C ABI rejects anyway) nothing is checked, so
    the call reports the library's own status."""
    if valid and t is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} B, the call needs {nbytes} B")


_F32, _U8 = torch.float32, torch.uint8
_BITS16 = (torch.int16, torch.uint16, torch.bfloat16)  # raw 16-bit (bf16) storage


def _dtype(name: str, t: torch.Tensor | None, *allowed):
    """The C ABI takes untyped pointers: refuse a buffer whose element type the kernel
    would misread (state and scales are fp32, codes and index bytes uint8)."""
    if t is not None and t.dtype not in allowed:
        raise TypeError(f"{name} is {t.dtype}; libcf wants {' or '.join(map(str, allowed))}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _allocate(make, stream, returned: bool = True):
    """make(), one buffer or several, for the launch stream to write.

    PyTorch's caching allocator hands a freed block to the stream it was allocated on, behind that stream's work and no
    other's.  A block of the caller's stream may still be written by what is queued there, which the launch stream does
    not wait for, so the buffer comes from the launch stream's own blocks: what used it before is done when the
    launch gets there.  Of a buffer that the caller gets, the caller's stream is on record too, so that the block is not
    reused before the work that is queued there when it is freed.  One that is freed when the call returns needs
    no more."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        here = torch.cuda.current_stream()
        if stream.cuda_stream != here.cuda_stream:
            with torch.cuda.stream(stream):
                made = make()
            if returned:
                for t in made if isinstance(made, tuple) else (made,):
                    if t is not None:
                        t.record_stream(here)
            return made
    return make()


def _act_dtype(a: torch.Tensor) -> int:
    if a.dtype == torch.bfloat16:
        return CF_BF16
    if a.dtype == torch.float32:
        return CF_F32
    raise TypeError(f"activation dtype {a.dtype}: want torch.bfloat16 or torch.float32")


def require_device() -> torch.device:
    """cuda:0 if it is an MI355X (gfx950); raises otherwise."""
    if not torch.cuda.is_available():
        raise RuntimeError("no HIP device visible")
    arch = torch.cuda.get_device_properties(0).gcnArchName
    if not arch.startswith("gfx950"):
        raise RuntimeError(f"device 0 is {arch}, libcf is built for gfx950 only")
    return torch.device("cuda", 0)


def codes_bytes(numel: int, bits: int) -> int:
    n = lib.cf_codes_bytes(numel, bits)
    if n < 0:
        raise CFError("cf_codes_bytes", n)
    return n


@dataclass
class SenderState:
    """Sender-side state of one tensor (or slab): reconstruction and error buffer."""
    ahat: torch.Tensor
    err: torch.Tensor

    @staticmethod
    def create(numel: int, device=None) -> "SenderState":
        device = device or require_device()
        return SenderState(torch.empty(numel, dtype=torch.float32, device=device),
                           torch.empty(numel, dtype=torch.float32, device=device))


def init_state(a: torch.Tensor, ahat: torch.Tensor, err: torch.Tensor | None = None, stream=None):
    """Warmup: ahat = a, err = 0 (err None on the receiver)."""
    _dtype("ahat", ahat, _F32)
    _dtype("err", err, _F32)
    _need("ahat", ahat, 4 * a.numel())
    _need("err", err, 4 * a.numel())
    _check("cf_init_state", lib.cf_init_state(_act_dtype(a), _ptr(a), _ptr(ahat), _ptr(err),
                                              a.numel(), _stream(stream)))


def compress(bits: int, a: torch.Tensor, ahat: torch.Tensor, err: torch.Tensor | None,
             codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """One sender step; returns (codes uint8[numel*bits/8], scales fp32[numel/128]).
    err None skips the (diagnostic) error buffer."""
    n = a.numel()
    if codes is None:
        codes = _allocate(lambda: torch.empty(max(n * bits // 8, 0), dtype=torch.uint8, device=a.device), stream)
    if scales is None:
        scales = _allocate(lambda: torch.empty(max(n // GROUP, 0), dtype=torch.float32, device=a.device), stream)
    for nm, t, dt in (("ahat", ahat, _F32), ("err", err, _F32), ("codes", codes, _U8), ("scales", scales, _F32)):
        _dtype(nm, t, dt)
    for nm, t, nb in (("ahat", ahat, 4 * n), ("err", err, 4 * n), ("codes", codes, n * bits // 8),
                      ("scales", scales, 4 * (n // GROUP))):
        _need(nm, t, nb, bits in (1, 2))
    _check("cf_compress", lib.cf_compress(bits, _act_dtype(a), _ptr(a), _ptr(ahat), _ptr(err),
                                          _ptr(codes), _ptr(scales), n, _stream(stream)))
    return codes, scales


def decompress(bits: int, codes: torch.Tensor, scales: torch.Tensor, ahat: torch.Tensor,
               stream=None, out_bf16: torch.Tensor | None = None):
    """Receiver step: ahat += decoded residual; with out_bf16 (a bfloat16 tensor of the
    same size) also writes the updated reconstruction rounded to bf16."""
    n = ahat.numel()
    for nm, t, dt in (("codes", codes, _U8), ("scales", scales, _F32), ("ahat", ahat, _F32)):
        _dtype(nm, t, dt)
    _need("codes", codes, n * bits // 8, bits in (1, 2))
    _need("scales", scales, 4 * (n // GROUP), bits in (1, 2))
    if out_bf16 is None:
        _check("cf_decompress", lib.cf_decompress(bits, _ptr(codes), _ptr(scales), _ptr(ahat),
                                                  ahat.numel(), _stream(stream)))
        return
    if out_bf16.dtype != torch.bfloat16 or out_bf16.numel() != ahat.numel():
        raise ValueError("out_bf16 must be a bfloat16 tensor of ahat's size")
    _check("cf_decompress_bf16", lib.cf_decompress_bf16(bits, _ptr(codes), _ptr(scales), _ptr(ahat),
                                                        _ptr(out_bf16), ahat.numel(), _stream(stream)))


def compress_ablation(mode: int, bits: int, a: torch.Tensor, ahat: torch.Tensor,
                      a_prev: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None, stream=None):
    """Ablation sender step (CF_MODE_NOEF needs a_prev); returns (codes, scales)."""
    n = a.numel()
    if codes is None:
        codes = _allocate(lambda: torch.empty(n * bits // 8, dtype=torch.uint8, device=a.device), stream)
    if scales is None:
        scales = _allocate(lambda: torch.empty(n // GROUP, dtype=torch.float32, device=a.device), stream)
    for nm, t, dt in (("ahat", ahat, _F32), ("a_prev", a_prev, a.dtype), ("codes", codes, _U8),
                      ("scales", scales, _F32)):
        _dtype(nm, t, dt)
    for nm, t, nb in (("ahat", ahat, 4 * n), ("a_prev", a_prev, n * a.element_size()),
                      ("codes", codes, n * bits // 8), ("scales", scales, 4 * (n // GROUP))):
        _need(nm, t, nb, bits in (1, 2))
    _check("cf_compress_ablation", lib.cf_compress_ablation(
        mode, bits, _act_dtype(a), _ptr(a), _ptr(a_prev), _ptr(ahat), _ptr(codes), _ptr(scales), n,
        _stream(stream)))
    return codes, scales


def topk_compress(k: int, a: torch.Tensor, ahat: torch.Tensor, err: torch.Tensor | None,
                  idx: torch.Tensor | None = None, vals: torch.Tensor | None = None, stream=None):
    """One top-k sender step; returns (idx uint8[numel/128*k], vals bf16 bits int16[numel/128*k])."""
    slots = max(a.numel() // GROUP * k, 0)
    if idx is None:
        idx = _allocate(lambda: torch.empty(slots, dtype=torch.uint8, device=a.device), stream)
    if vals is None:
        vals = _allocate(lambda: torch.empty(slots, dtype=torch.int16, device=a.device), stream)
    n = a.numel()
    for nm, t, dts in (("ahat", ahat, (_F32,)), ("err", err, (_F32,)), ("idx", idx, (_U8,)), ("vals", vals, _BITS16)):
        _dtype(nm, t, *dts)
    for nm, t, nb in (("ahat", ahat, 4 * n), ("err", err, 4 * n), ("idx", idx, slots), ("vals", vals, 2 * slots)):
        _need(nm, t, nb, 1 <= k <= GROUP)
    _check("cf_topk_compress", lib.cf_topk_compress(k, _act_dtype(a), _ptr(a), _ptr(ahat), _ptr(err),
                                                    _ptr(idx), _ptr(vals), a.numel(), _stream(stream)))
    return idx, vals


def topk_decompress(k: int, idx: torch.Tensor, vals: torch.Tensor, ahat: torch.Tensor, stream=None):
    """Receiver step: ahat[group, idx] += bf16 value, for every sent slot."""
    slots = max(ahat.numel() // GROUP * k, 0)
    _dtype("idx", idx, _U8)
    _dtype("vals", vals, *_BITS16)
    _dtype("ahat", ahat, _F32)
    _need("idx", idx, slots, 1 <= k <= GROUP)
    _need("vals", vals, 2 * slots, 1 <= k <= GROUP)
    _check("cf_topk_decompress", lib.cf_topk_decompress(k, _ptr(idx), _ptr(vals), _ptr(ahat), ahat.numel(),
                                                        _stream(stream)))


def _dev_ptr(t: torch.Tensor) -> int:
    return _ptr(t).value


class Slab:
    """1/2-bit state of ``count`` tensors of ``numel`` elements laid out back to back
    (e.g. the K and V activations of every layer of one sequence-parallel shard).

    ``compress``/``decompress``/``init`` issue one C-ABI call per ``per_call``
    consecutive tensors (2 = one layer's K and V, the serving pattern; ``count`` = one
    call for the whole step).  Pointers are computed once; each call only forwards
    integers to libcf.
    """

    def __init__(self, count: int, numel: int, bits: int, device=None, receiver: bool = False):
        if numel % GROUP:
            raise ValueError("numel must be a multiple of 128")
        device = device or require_device()
        self.count, self.numel, self.bits = count, numel, bits
        f32 = torch.float32
        self.ahat = torch.empty((count, numel), dtype=f32, device=device)
        self.err = None if receiver else torch.empty((count, numel), dtype=f32, device=device)
        self.codes = torch.empty((count, numel * bits // 8), dtype=torch.uint8, device=device)
        self.scales = torch.empty((count, numel // GROUP), dtype=f32, device=device)

    def _chunks(self, per_call: int):
        per_call = max(1, min(per_call, self.count))
        for i in range(0, self.count, per_call):
            yield i, min(per_call, self.count - i)

    def init(self, a: torch.Tensor, per_call: int = 2, stream=None):
        if a.numel() != self.count * self.numel:
            raise ValueError("activation slab has the wrong size")
        dt, s = _act_dtype(a), _stream(stream)
        ab, esz = _dev_ptr(a), a.element_size()
        hb = _dev_ptr(self.ahat)
        eb = _dev_ptr(self.err) if self.err is not None else None
        n = self.numel
        for i, c in self._chunks(per_call):
            _check("cf_init_state", lib.cf_init_state(
                dt, ab + i * n * esz, hb + i * n * 4, None if eb is None else eb + i * n * 4,
                c * n, s))

    def compress(self, a: torch.Tensor, per_call: int = 2, stream=None, timer: list | None = None,
                 streams: list | None = None):
        """Compress one step.  With ``timer`` a list, a pair of timing events recorded on
        the launch stream just before and after every call is appended to it.  With
        ``streams`` a list of streams, call i goes to streams[i % len(streams)] instead (the
        calls touch disjoint tensors, so they may overlap); ordering those streams against
        the inputs and the later consumers is the caller's."""
        if self.err is None:
            raise RuntimeError("receiver slab has no error buffer")
        if a.numel() != self.count * self.numel:
            raise ValueError("activation slab has the wrong size")
        dt, s, bits, n = _act_dtype(a), _stream(stream), self.bits, self.numel
        ab, esz = _dev_ptr(a), a.element_size()
        hb, eb = _dev_ptr(self.ahat), _dev_ptr(self.err)
        cb, sb = _dev_ptr(self.codes), _dev_ptr(self.scales)
        cbytes, ng = n * bits // 8, n // GROUP
        f = lib.cf_compress
        ts = None if timer is None else (torch.cuda.current_stream() if stream is None else stream)
        rr = [_stream(x) for x in streams] if streams else None
        for j, (i, c) in enumerate(self._chunks(per_call)):
            if ts is not None:
                ev0 = torch.cuda.Event(enable_timing=True)
                ev0.record(ts)
            rc = f(bits, dt, ab + i * n * esz, hb + i * n * 4, eb + i * n * 4, cb + i * cbytes,
                   sb + i * ng * 4, c * n, s if rr is None else rr[j % len(rr)])
            if rc:
                raise CFError("cf_compress", rc)
            if ts is not None:
                ev1 = torch.cuda.Event(enable_timing=True)
                ev1.record(ts)
                timer.append((ev0, ev1))

    def decompress(self, codes: torch.Tensor, scales: torch.Tensor, per_call: int = 2, stream=None):
        s, bits, n = _stream(stream), self.bits, self.numel
        _dtype("codes", codes, _U8)
        _dtype("scales", scales, _F32)
        _need("codes", codes, self.count * n * bits // 8)
        _need("scales", scales, 4 * self.count * (n // GROUP))
        cb, sb, hb = _dev_ptr(codes), _dev_ptr(scales), _dev_ptr(self.ahat)
        cbytes, ng = n * bits // 8, n // GROUP
        f = lib.cf_decompress
        for i, c in self._chunks(per_call):
            rc = f(bits, cb + i * cbytes, sb + i * ng * 4, hb + i * n * 4, c * n, s)
            if rc:
                raise CFError("cf_decompress", rc)


def lowrank_workspace_bytes(m: int, n: int, rank: int, batch: int = 1) -> int:
    nb = lib.cf_lowrank_workspace_bytes(m, n, rank, batch)
    if nb == 0:
        raise CFError("cf_lowrank_workspace_bytes", -2)
    return nb


def lowrank_payload(batch: int, m: int, n: int, rank: int, factor_bits: int, device):
    """Empty payload buffers (u, u_scales, v, v_scales) for `batch` tensors."""
    if factor_bits == 4:
        return (torch.empty(batch * m * rank // 2, dtype=torch.uint8, device=device),
                torch.empty(batch * rank, dtype=torch.float32, device=device),
                torch.empty(batch * n * rank // 2, dtype=torch.uint8, device=device),
                torch.empty(batch * rank, dtype=torch.float32, device=device))
    dt = torch.int16 if factor_bits == 16 else torch.float32  # bf16 bits or fp32
    return (torch.empty(batch * m * rank, dtype=dt, device=device), None,
            torch.empty(batch * n * rank, dtype=dt, device=device), None)


def _check_lowrank_buffers(batch, m, n, rank, factor_bits, payload):
    u, us, v, vs = payload
    esz = {4: 0.5, 16: 2, 32: 4}.get(factor_bits)
    if esz is None or rank < 1:
        return  # the C ABI rejects these arguments itself
    fdt = {4: (_U8,), 16: _BITS16, 32: (_F32,)}[factor_bits]
    _dtype("u", u, *fdt)
    _dtype("v", v, *fdt)
    _dtype("u_scales", us, _F32)
    _dtype("v_scales", vs, _F32)
    _need("u", u, int(batch * m * rank * esz))
    _need("v", v, int(batch * n * rank * esz))
    if factor_bits == 4:
        _need("u_scales", us, 4 * batch * rank)
        _need("v_scales", vs, 4 * batch * rank)


def lowrank_compress(a: torch.Tensor, ahat: torch.Tensor, err: torch.Tensor | None,
                     q_state: torch.Tensor, rank: int, iters: int, factor_bits: int = 4,
                     payload=None, workspace: torch.Tensor | None = None, stream=None):
    """One low-rank sender step on a (batch, m, n) activation; returns the payload
    (u, u_scales, v, v_scales).  q_state is (batch, n, rank) fp32, updated in place."""
    batch, m, n = a.shape
    if payload is None:
        payload = _allocate(lambda: lowrank_payload(batch, m, n, rank, factor_bits, a.device), stream)
    u, us, v, vs = payload
    need = lowrank_workspace_bytes(m, n, rank, batch)
    if workspace is None:
        # freed when this call returns, possibly before the launch stream has used it
        workspace = _allocate(lambda: torch.empty(need, dtype=torch.uint8, device=a.device), stream, False)
    _check_lowrank_buffers(batch, m, n, rank, factor_bits, payload)
    numel = batch * m * n
    for nm, t in (("ahat", ahat), ("err", err), ("q_state", q_state)):
        _dtype(nm, t, _F32)
    for nm, t, nb in (("ahat", ahat, 4 * numel), ("err", err, 4 * numel), ("q_state", q_state, 4 * batch * n * rank)):
        _need(nm, t, nb, rank >= 1)
    _check("cf_lowrank_compress", lib.cf_lowrank_compress(
        _act_dtype(a), _ptr(a), _ptr(ahat), _ptr(err), m, n, rank, iters, factor_bits, batch,
        _ptr(q_state), _ptr(u), _ptr(us), _ptr(v), _ptr(vs), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return u, us, v, vs


def lowrank_compress_noalloc(a: torch.Tensor, ahat: torch.Tensor, err: torch.Tensor | None,
                             q_state: torch.Tensor, rank: int, iters: int, factor_bits: int, payload,
                             stream=None):
    """cf_lowrank_compress_noalloc: one low-rank sender step that uses the library's fixed
    device scratch instead of a workspace, for callers that cannot allocate.  Every buffer,
    the payload (u, u_scales, v, v_scales) included, comes from the caller; nothing is
    allocated here.  Calls that may overlap on one GPU race on that scratch."""
    batch, m, n = a.shape
    u, us, v, vs = payload
    _check_lowrank_buffers(batch, m, n, rank, factor_bits, payload)
    numel = batch * m * n
    for nm, t in (("ahat", ahat), ("err", err), ("q_state", q_state)):
        _dtype(nm, t, _F32)
    for nm, t, nb in (("ahat", ahat, 4 * numel), ("err", err, 4 * numel), ("q_state", q_state, 4 * batch * n * rank)):
        _need(nm, t, nb, rank >= 1)
    _check("cf_lowrank_compress_noalloc", lib.cf_lowrank_compress_noalloc(
        _act_dtype(a), _ptr(a), _ptr(ahat), _ptr(err), m, n, rank, iters, factor_bits, batch,
        _ptr(q_state), _ptr(u), _ptr(us), _ptr(v), _ptr(vs), _stream(stream)))
    return u, us, v, vs


def lowrank_decompress(factor_bits: int, payload, ahat: torch.Tensor, rank: int, stream=None):
    """Receiver step on a (batch, m, n) reconstruction: ahat += U^ V^^T."""
    batch, m, n = ahat.shape
    u, us, v, vs = payload
    _dtype("ahat", ahat, _F32)
    _check_lowrank_buffers(batch, m, n, rank, factor_bits, payload)
    _check("cf_lowrank_decompress", lib.cf_lowrank_decompress(
        factor_bits, _ptr(u), _ptr(us), _ptr(v), _ptr(vs), _ptr(ahat), m, n, rank, batch,
        _stream(stream)))


# The calls below are a few microseconds on the device, so their marshalling asks the runtime for
# the current device and stream once, and for nothing twice.


def _here(name: str, t: torch.Tensor, dev: int):
    """Refuses a tensor that is not on the current device ``dev``."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError("libcf takes device tensors (a host pointer would fault the kernel)")
        raise ValueError(f"{name} on {t.device}, but the current device is cuda:{dev} "
                         "(libcf launches on the current device)")


def _rows(name: str, t: torch.Tensor, dev: int) -> Rows:
    """The rows of a (tokens, heads, head_dim) tensor, of any strides but the last."""
    _here(name, t, dev)
    st, sh, sd = t.stride()
    if sd != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the channels of a row must be consecutive")
    return Rows(t.data_ptr(), st, sh)


def _flat(name: str, t: torch.Tensor | None, dev: int, dtype: torch.dtype, shape: tuple):
    """Address of a contiguous tensor of this type and shape, None for None."""
    if t is None:
        return None
    if t.dtype == dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}; libcf wants {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, the call needs {shape}")
    _here(name, t, dev)
    if not t.is_contiguous():
        raise ValueError("libcf needs contiguous tensors")
    return t.data_ptr()


def _shaped(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple):
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}; libcf wants {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, the call needs {tuple(shape)}")


def _fit(fn: str, status: int, form: str, *numbers):
    """Refuses numbers that the C ABI's int (i) and int64_t (q) cannot hold: ctypes would hand on their
    lowest bits."""
    try:
        struct.pack(form, *numbers)
    except struct.error:
        raise CFError(fn, status) from None


def _device(t: torch.Tensor) -> int:
    """The current device; no tensor's where t is not on one (there may be none)."""
    return torch._C._cuda_getDevice() if t.is_cuda else -2


def _on(stream, dev: int):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    return torch.empty_like(t) if stream is None else _allocate(lambda: torch.empty_like(t), stream)


def _new(like: torch.Tensor, shape, stream, dtype: torch.dtype | None = None, returned: bool = True) -> torch.Tensor:
    """A buffer for the launch stream to write."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    return _allocate(lambda: like.new_empty(shape, dtype=dtype), stream, returned)


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, norm: int = CF_NORM_RMS,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                 q_bias: torch.Tensor | None = None, k_bias: torch.Tensor | None = None, eps: float = 1e-6,
                 rope: int = CF_ROPE_NONE, cos: torch.Tensor | None = None, sin: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None, stream=None):
    """Per-head norms of q and k (tokens, heads, head_dim) and the position rotation, in one
    pass; returns (q_out, k_out).  Either side may be None.  Slices of a packed projection and
    head-major views are taken as they are; q_out may be q itself, and k_out k.  cos and sin
    are (positions, rot_dim / 2) fp32, weights and biases (head_dim,) fp32, positions
    (tokens,) int32 (negative: a padding token, whose output rows stay as they are)."""
    a = q if q is not None else k
    if a is None or a.dim() != 3:
        raise ValueError("q or k must be a (tokens, heads, head_dim) tensor")
    tokens, _, dim = a.shape
    dt, kind = _act_dtype(a), a.dtype
    hq = 0 if q is None else q.shape[1] if q.dim() == 3 else -1
    hk = 0 if k is None else k.shape[1] if k.dim() == 3 else -1
    for nm, t, o, h in (("q", q, q_out, hq), ("k", k, k_out, hk)):
        if t is not None:
            _shaped(nm, t, kind, (tokens, h, dim))
            if o is not None:
                _shaped(nm + "_out", o, kind, t.shape)
    _fit("cf_qk_norm_rope", -4, "iiii", norm, rope, hq, hk)
    dev = _device(a)
    rq = rk = rqo = rko = None
    if q is not None:
        rq = _rows("q", q, dev)
        q_out = _like(q, stream) if q_out is None else q_out
        rqo = _rows("q_out", q_out, dev)
    if k is not None:
        rk = _rows("k", k, dev)
        k_out = _like(k, stream) if k_out is None else k_out
        rko = _rows("k_out", k_out, dev)
    n_pos = rot = 0
    pc = ps = pp = None
    if rope != CF_ROPE_NONE:
        if cos is None or sin is None or cos.dim() != 2:
            raise ValueError("a rotation needs cos and sin, (positions, rot_dim / 2) fp32")
        n_pos, rot = cos.shape
        _fit("cf_qk_norm_rope", -2, "i", 2 * rot)
        pc, ps = _flat("cos", cos, dev, _F32, (n_pos, rot)), _flat("sin", sin, dev, _F32, (n_pos, rot))
        pp = _flat("positions", positions, dev, torch.int32, (tokens,))
    row = (dim,)
    rc = lib.cf_qk_norm_rope(
        dt, tokens, hq, hk, dim, rq, rk, rqo, rko, norm, _flat("q_weight", q_weight, dev, _F32, row),
        _flat("q_bias", q_bias, dev, _F32, row), _flat("k_weight", k_weight, dev, _F32, row),
        _flat("k_bias", k_bias, dev, _F32, row), eps, rope, pc, ps, n_pos, 2 * rot, pp, _on(stream, dev))
    if rc:
        raise CFError("cf_qk_norm_rope", rc)
    return q_out, k_out


@dataclass
class KV4Cache:
    """A paged K/V cache of 4-bit codes: ``data`` is (pages, kv_heads, page_size * head_dim *
    17 / 16) uint8.  A copy of ``data`` is a checkpoint of it."""
    data: torch.Tensor
    page_size: int
    head_dim: int

    @staticmethod
    def create(pages: int, page_size: int, kv_heads: int, head_dim: int, device=None) -> "KV4Cache":
        _fit("cf_kv4_cache_bytes", -2, "qiii", pages, page_size, kv_heads, head_dim)
        nb = lib.cf_kv4_cache_bytes(pages, page_size, kv_heads, head_dim)
        if nb < 0:
            raise CFError("cf_kv4_cache_bytes", nb)
        return KV4Cache(torch.zeros((pages, kv_heads, nb // pages // kv_heads), dtype=torch.uint8,
                                    device=device or require_device()), page_size, head_dim)

    def _args(self, dev: int):
        d = self.data
        if d.dim() != 3 or d.shape[2] * 16 != self.page_size * self.head_dim * 17:
            raise ValueError(f"cache data is {tuple(d.shape)}: want (pages, kv_heads, page_size * head_dim * 17 / 16)")
        _fit("KV4Cache", -2, "iii", self.page_size, d.shape[1], self.head_dim)
        return _flat("cache", d, dev, _U8, d.shape), d.shape[0], self.page_size, d.shape[1], self.head_dim


def kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None):
    """Quantize rows k, v (tokens, kv_heads, head_dim) into the cache's slots (tokens,) int64,
    page * page_size + place; a negative slot takes nothing."""
    tokens = k.shape[0] if k.dim() == 3 else -1
    want = (tokens, cache.data.shape[1], cache.head_dim)
    dt, dev = _act_dtype(k), _device(k)
    _shaped("k", k, k.dtype, want)
    _shaped("v", v, k.dtype, want)
    ps = _flat("slots", slots, dev, torch.int64, (tokens,))
    rc = lib.cf_kv4_append(dt, _rows("k", k, dev), _rows("v", v, dev), ps, tokens, *cache._args(dev), _on(stream, dev))
    if rc:
        raise CFError("cf_kv4_append", rc)


def kv4_read(cache: KV4Cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
             k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """The rows that the cache holds in slots (tokens,) int64, as (k, v) of (tokens, kv_heads,
    head_dim); zeros for slots that are not in the cache."""
    return _read("cf_kv4_read", lib.cf_kv4_read, cache, slots, dtype, k, v, stream)


def _read(fn, call, cache, slots, dtype, k, v, stream):
    tokens = slots.numel()
    want = (tokens, cache.data.shape[1], cache.head_dim)
    k = _new(cache.data, want, stream, dtype) if k is None else k
    v = _new(cache.data, want, stream, k.dtype) if v is None else v
    dt, dev = _act_dtype(k), _device(k)
    _shaped("k", k, k.dtype, want)
    _shaped("v", v, k.dtype, want)
    ps = _flat("slots", slots, dev, torch.int64, (tokens,))
    rc = call(dt, *cache._args(dev), ps, tokens, _rows("k", k, dev), _rows("v", v, dev), _on(stream, dev))
    if rc:
        raise CFError(fn, rc)
    return k, v


def _workspace_bytes(fn: str, dtype: torch.dtype, *sizes: int) -> int:
    dt = CF_BF16 if dtype == torch.bfloat16 else CF_F32 if dtype == torch.float32 else -1
    _fit(fn, -2, "qiii", *sizes)
    nb = getattr(lib, fn)(dt, *sizes)
    if nb == 0:
        raise CFError(fn, -2)
    return nb


def kv4_attention_workspace_bytes(dtype: torch.dtype, max_q: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return _workspace_bytes("cf_kv4_attention_workspace_bytes", dtype, max_q, q_heads, kv_heads, head_dim)


def kv4_attention(q: torch.Tensor, cache: KV4Cache, kv_lens: torch.Tensor, table: torch.Tensor | None = None,
                  q_starts: torch.Tensor | None = None, max_q: int = 0, causal: bool = False, window: int = 0,
                  scale: float | None = None, table_width: int = 0, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of q (total_q, q_heads, head_dim) over the cache; returns out.  kv_lens
    (batch,), table (batch, pages) and q_starts (batch + 1,) are int32; without a table
    sequence b has pages b * table_width and on, without q_starts every sequence has
    total_q / batch queries.  lse (total_q, q_heads) fp32 is written where it is given.  Rows
    that belong to no sequence stay as they are.  max_q: the most queries of a sequence, if
    known (a bound above total_q is as good as total_q); scale: head_dim ** -0.5 if None."""
    return _paged_attention("cf_kv4_attention", lib.cf_kv4_attention, lib.cf_kv4_attention_workspace_bytes, q, cache, kv_lens, table,
                            q_starts, max_q, causal, window, scale, table_width, out, lse, workspace, stream)


def _paged_attention(fn, call, workspace_bytes, q, cache, kv_lens, table, q_starts, max_q, causal, window, scale, table_width, out,
                     lse, workspace, stream):
    if q.dim() != 3:
        raise ValueError("q must be (total_q, q_heads, head_dim)")
    total, heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError(f"q has rows of {dim}, the cache of {cache.head_dim}")
    dt, dev, kv_heads = _act_dtype(q), _device(q), cache.data.shape[1]
    batch = kv_lens.numel()
    if max_q > total:
        max_q = total
    if kv_lens.dtype != torch.int32:
        raise TypeError(f"kv_lens is {kv_lens.dtype}; libcf wants torch.int32")
    pt = None
    if table is not None:
        table_width = table.shape[-1]
        pt = _flat("table", table, dev, torch.int32, (batch, table_width))
    _fit(fn, -2, "qiiiii", max_q, window, batch, table_width, heads, kv_heads)
    pq = _flat("q_starts", q_starts, dev, torch.int32, (batch + 1,))
    pe = _flat("lse", lse, dev, _F32, (total, heads))
    pl = _flat("kv_lens", kv_lens, dev, torch.int32, (batch,))
    if out is None:
        out = _like(q, stream)
    else:
        _shaped("out", out, q.dtype, q.shape)
    workspace, pw, nw = _workspace(workspace_bytes, dt, q, max_q or (total if q_starts is not None else total // max(batch, 1)), heads, kv_heads,
                        workspace, dev, stream)
    rc = call(
        dt, _rows("q", q, dev), total, heads, *cache._args(dev), batch, pt, table_width, pl, pq, max_q,
        CF_ATTN_CAUSAL if causal else 0, window, dim ** -0.5 if scale is None else scale, _rows("out", out, dev), pe,
        pw, nw, _on(stream, dev))
    if rc:
        raise CFError(fn, rc)
    return out


@dataclass
class KV8Cache:
    """A paged K/V cache of 8-bit codes with a scale for each 16 tokens and head: ``data`` is (pages, kv_heads, 2 * page_size *
    head_dim + max(16, page_size / 8)) uint8.  A copy of ``data`` is a checkpoint of it."""
    data: torch.Tensor
    page_size: int
    head_dim: int

    @staticmethod
    def create(pages: int, page_size: int, kv_heads: int, head_dim: int, device=None) -> "KV8Cache":
        _fit("cf_kv8_cache_bytes", -2, "qiii", pages, page_size, kv_heads, head_dim)
        nb = lib.cf_kv8_cache_bytes(pages, page_size, kv_heads, head_dim)
        if nb < 0:
            raise CFError("cf_kv8_cache_bytes", nb)
        return KV8Cache(torch.zeros((pages, kv_heads, nb // pages // kv_heads), dtype=torch.uint8,
                                    device=device or require_device()), page_size, head_dim)

    def _args(self, dev: int):
        d, page_size, head_dim = self.data, self.page_size, self.head_dim
        shape = d.shape
        if len(shape) != 3 or shape[2] != 2 * page_size * head_dim + max(16, page_size // 8):
            raise ValueError(f"cache data is {tuple(shape)}: want (pages, kv_heads, 2 * page_size * head_dim + max(16, page_size / 8))")
        pages, heads, _ = shape
        _fit("KV8Cache", -2, "iii", page_size, heads, head_dim)
        return _flat("cache", d, dev, _U8, shape), pages, page_size, heads, head_dim


def kv8_append(cache: KV8Cache, k: torch.Tensor, v: torch.Tensor, kv_lens: torch.Tensor, table: torch.Tensor | None = None,
               starts: torch.Tensor | None = None, table_width: int = 0, stream=None):
    """Quantize rows k, v (tokens, kv_heads, head_dim), the last tokens of sequences, into the cache.  kv_lens (batch,) are the
    sequences' tokens with them, starts (batch + 1,) where each one's rows begin, table (batch, pages) their pages, all
    int32; without a table sequence b has pages b * table_width and on, without starts every sequence gets
    tokens / batch.  Behind a pages_resize that may have found too few pages kv_lens are its append_lens."""
    tokens = k.shape[0] if k.dim() == 3 else -1
    want = (tokens, cache.data.shape[1], cache.head_dim)
    dt, dev, batch = _act_dtype(k), _device(k), kv_lens.numel()
    _shaped("k", k, k.dtype, want)
    _shaped("v", v, k.dtype, want)
    pt = None
    if table is not None:
        table_width = table.shape[-1]
        pt = _flat("table", table, dev, torch.int32, (batch, table_width))
    _fit("cf_kv8_append", -2, "ii", batch, table_width)
    ps = _flat("starts", starts, dev, torch.int32, (batch + 1,))
    pl = _flat("kv_lens", kv_lens, dev, torch.int32, (batch,))
    rc = lib.cf_kv8_append(dt, _rows("k", k, dev), _rows("v", v, dev), tokens, *cache._args(dev), batch, pt, table_width, pl, ps,
                           _on(stream, dev))
    if rc:
        raise CFError("cf_kv8_append", rc)


def kv8_read(cache: KV8Cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
             k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """The rows that the cache holds in slots (tokens,) int64 (page * page_size + place), as (k, v) of (tokens, kv_heads,
    head_dim); zeros for slots that are not in the cache."""
    return _read("cf_kv8_read", lib.cf_kv8_read, cache, slots, dtype, k, v, stream)


def kv8_attention_workspace_bytes(dtype: torch.dtype, max_q: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return _workspace_bytes("cf_kv8_attention_workspace_bytes", dtype, max_q, q_heads, kv_heads, head_dim)


def kv8_attention(q: torch.Tensor, cache: KV8Cache, kv_lens: torch.Tensor, table: torch.Tensor | None = None,
                  q_starts: torch.Tensor | None = None, max_q: int = 0, causal: bool = False, window: int = 0,
                  scale: float | None = None, table_width: int = 0, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of q (total_q, q_heads, head_dim) over an 8-bit cache; arguments and results as for kv4_attention."""
    return _paged_attention("cf_kv8_attention", lib.cf_kv8_attention, lib.cf_kv8_attention_workspace_bytes, q, cache, kv_lens, table,
                            q_starts, max_q, causal, window, scale, table_width, out, lse, workspace, stream)


def attention_workspace_bytes(dtype: torch.dtype, max_q: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return _workspace_bytes("cf_attention_workspace_bytes", dtype, max_q, q_heads, kv_heads, head_dim)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor | None = None,
              k_starts: torch.Tensor | None = None, batch: int = 1, max_q: int = 0, causal: bool = False, window: int = 0,
              scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None):
    """Attention of q (total_q, q_heads, head_dim) over k and v (total_k, kv_heads, head_dim), packed sequences of which
    sequence b has rows q_starts[b] .. q_starts[b + 1] - 1 of q and likewise k_starts of k and v (batch + 1 int32 each);
    without starts each of `batch` sequences has as many.  Returns out; lse (total_q, q_heads) fp32 is written where it is given.
    Slices of a packed projection and head-major views are taken as they are.  Rows that belong to no sequence stay as they are.
    max_q: the most queries of a sequence, if known (a bound above total_q is as good as total_q); scale: head_dim ** -0.5
    if None."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be (total_q, q_heads, head_dim), k and v (total_k, kv_heads, head_dim)")
    total, heads, dim = q.shape
    keys, kv_heads = k.shape[:2]
    dt, dev = _act_dtype(q), _device(q)
    _shaped("k", k, q.dtype, (keys, kv_heads, dim))
    _shaped("v", v, q.dtype, (keys, kv_heads, dim))
    if q_starts is not None:
        batch = q_starts.numel() - 1
    elif k_starts is not None:
        batch = k_starts.numel() - 1
    if max_q > total:
        max_q = total
    _fit("cf_attention", -2, "qiiiii", max_q, window, batch, heads, kv_heads, dim)
    pq = _flat("q_starts", q_starts, dev, torch.int32, (batch + 1,))
    pk = _flat("k_starts", k_starts, dev, torch.int32, (batch + 1,))
    pe = _flat("lse", lse, dev, _F32, (total, heads))
    if out is None:
        out = _like(q, stream)
    else:
        _shaped("out", out, q.dtype, q.shape)
    workspace, pw, nw = _workspace(lib.cf_attention_workspace_bytes, dt, q, max_q or (total if q_starts is not None else total // max(batch, 1)), heads,
                        kv_heads, workspace, dev, stream)
    rc = lib.cf_attention(
        dt, _rows("q", q, dev), total, heads, _rows("k", k, dev), _rows("v", v, dev), keys, kv_heads, dim, batch, pq, pk, max_q,
        CF_ATTN_CAUSAL if causal else 0, window, dim ** -0.5 if scale is None else scale, _rows("out", out, dev), pe, pw, nw,
        _on(stream, dev))
    if rc:
        raise CFError("cf_attention", rc)
    return out


def _workspace(workspace_bytes, dt, q, most, heads, kv_heads, workspace, dev, stream):
    """An attention call's workspace, the caller's or one to be held until the call has returned: (tensor, address, bytes)."""
    if workspace is None:
        need = workspace_bytes(dt, most, heads, kv_heads, q.shape[2])
        if not need or not q.shape[0]:
            return None, None, 0
        # freed when the call returns, possibly before the launch stream has used it
        workspace = _new(q, need, stream, _U8, False)
        return workspace, workspace.data_ptr(), need
    return workspace, _flat("workspace", workspace, dev, workspace.dtype, workspace.shape), workspace.numel() * workspace.element_size()


@dataclass
class PageTable:
    """Who holds which page of a cache: refs (pages,) how many entries hold each, table (rows, width) the pages of each
    sequence, lens (rows,) its tokens, all int32.  The same table serves every cache whose pages it numbers (each layer's)."""
    refs: torch.Tensor
    table: torch.Tensor
    lens: torch.Tensor
    page_size: int

    @staticmethod
    def create(pages: int, rows: int, width: int, page_size: int, device=None) -> "PageTable":
        """All pages free, all sequences empty."""
        dev = device or require_device()
        return PageTable(torch.zeros(pages, dtype=torch.int32, device=dev),
                         torch.full((rows, width), -1, dtype=torch.int32, device=dev),
                         torch.zeros(rows, dtype=torch.int32, device=dev), page_size)

    def append_lens(self, want: torch.Tensor) -> torch.Tensor:
        """kv_lens for an append of the tokens that a resize to want (rows,) was for: want where a row has so many, and 0, so
        that nothing is written, where it found too few pages and still has its old length.  On the current stream."""
        return torch.where(self.lens == want, want, 0)

    def _pages(self, name: str, dev: int, shape: tuple) -> Pages:
        pages, rows, width = shape
        i32 = torch.int32
        return Pages(_flat(name + ".refs", self.refs, dev, i32, (pages,)), _flat(name + ".table", self.table, dev, i32, (rows, width)),
                     _flat(name + ".lens", self.lens, dev, i32, (rows,)))

    def _like(self, stream) -> "PageTable":
        return PageTable(_like(self.refs, stream), _like(self.table, stream), _like(self.lens, stream), self.page_size)


def _pages_call(fn: str, have: PageTable, out: PageTable | None, workspace, stream):
    """Of an operation on pages: the sequences in and out, out, sizes, the workspace's address and bytes, the device, and
    the workspace, to be held until the call has returned."""
    if have.table.dim() != 2 or have.refs.dim() != 1:
        raise ValueError("table must be (rows, width), refs (pages,)")
    dev = _device(have.table)
    rows, width = have.table.shape
    shape = (have.refs.numel(), rows, width)
    _fit(fn, -2, "qiii", *shape, have.page_size)
    if out is not None and out.page_size != have.page_size:
        raise ValueError(f"pages of {have.page_size} tokens in, of {out.page_size} out")
    pin = have._pages("have", dev, shape)
    if out is None:
        out = have._like(stream)
        pout = Pages(out.refs.data_ptr(), out.table.data_ptr(), out.lens.data_ptr())
    else:
        pout = pin if out is have else out._pages("out", dev, shape)
    need = lib.cf_pages_workspace_bytes(shape[0], rows)
    if workspace is None:
        workspace = _new(have.table, max(need, 4) // 4, stream, returned=False)
        ws = (workspace.data_ptr(), need)
    else:
        ws = (_flat("workspace", workspace, dev, workspace.dtype, workspace.shape), workspace.numel() * workspace.element_size())
    return pin, pout, out, shape, ws, dev, workspace


def _words(like: torch.Tensor, n: int, t: torch.Tensor | None, name: str, dev: int, stream):
    """(a buffer of n int32, its address)."""
    if t is None:
        t = _new(like, n, stream)
        return t, t.data_ptr()
    return t, _flat(name, t, dev, torch.int32, (n,))


def pages_resize(have: PageTable, want: torch.Tensor, out: PageTable | None = None, missing: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """Sequences of want (rows,) int32 tokens each (negative: as it is): those that shrink let go pages, then those that
    grow take the first free ones.  Returns (out, missing): missing (1,) int32 says how many rows found too few and stay as they
    are; an append takes out.append_lens(want), since out.lens would place their new tokens over their last.  Rows that shrink to
    inside a page that others hold need pages_fork(own=True) before anything is appended to them.  out may be `have`."""
    pin, pout, out, shape, ws, dev, workspace = _pages_call("cf_pages_resize", have, out, workspace, stream)
    missing, pm = _words(have.table, 1, missing, "missing", dev, stream)
    rc = lib.cf_pages_resize(pin, pout, *shape, have.page_size, _flat("want", want, dev, torch.int32, (shape[1],)), pm, *ws, _on(stream, dev))
    if rc:
        raise CFError("cf_pages_resize", rc)
    return out, missing


def pages_fork(have: PageTable, parents: torch.Tensor, out: PageTable | None = None, src: torch.Tensor | None = None,
               dst: torch.Tensor | None = None, missing: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               stream=None, own: bool = False):
    """Row r becomes a copy of row parents[r] (rows,) int32 (itself: it stays; outside the rows: empty).  Whole pages are
    shared.  Returns (out, src, dst, missing): pages src[r] have to be copied to dst[r], with pages_copy in every cache, before
    anything is appended; missing (1,) says how many rows found no page for that and end before it.  Where a pages_resize
    may have shrunk rows to inside pages that others hold, own=True: every row's last, partly filled page is then its alone,
    whoever its parent is (parents = 0, 1, 2, .. changes nothing else)."""
    fn, call = ("cf_pages_fork_own", lib.cf_pages_fork_own) if own else ("cf_pages_fork", lib.cf_pages_fork)
    pin, pout, out, shape, ws, dev, workspace = _pages_call(fn, have, out, workspace, stream)
    src, p1 = _words(have.table, shape[1], src, "src", dev, stream)
    dst, p2 = _words(have.table, shape[1], dst, "dst", dev, stream)
    missing, pm = _words(have.table, 1, missing, "missing", dev, stream)
    rc = call(pin, pout, *shape, have.page_size, _flat("parents", parents, dev, torch.int32, (shape[1],)), p1, p2, pm, *ws, _on(stream, dev))
    if rc:
        raise CFError(fn, rc)
    return out, src, dst, missing


def pages_compact(have: PageTable, out: PageTable | None = None, src: torch.Tensor | None = None, dst: torch.Tensor | None = None,
                  count: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """The pages that are held become the first ones.  Returns (out, src, dst, count): the first count (1,) of src and dst
    (pages / 2 each) are the pages to copy, with pages_copy in every cache.  Every entry of the table is renumbered, behind a
    row's last page too.  out may be `have`."""
    pin, pout, out, shape, ws, dev, workspace = _pages_call("cf_pages_compact", have, out, workspace, stream)
    src, p1 = _words(have.table, shape[0] // 2, src, "src", dev, stream)
    dst, p2 = _words(have.table, shape[0] // 2, dst, "dst", dev, stream)
    count, pm = _words(have.table, 1, count, "count", dev, stream)
    rc = lib.cf_pages_compact(pin, pout, *shape, p1, p2, pm, *ws, _on(stream, dev))
    if rc:
        raise CFError("cf_pages_compact", rc)
    return out, src, dst, count


def pages_copy(data: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, count: torch.Tensor | None = None, stream=None):
    """Copies page src[i] to page dst[i] (int32) of data, (layers, pages, bytes) uint8 of one or
    several caches that are numbered alike; with count (1,) int32 the first of them.  Pairs with a -1 copy nothing."""
    if data.dtype != _U8 or data.dim() != 3:
        raise TypeError("data must be (layers, pages, bytes) uint8; of one cache: cache.data.flatten(1)[None]")
    dev = _device(data)
    layers, pages, size = data.shape
    n = src.numel()
    _fit("cf_pages_copy", -2, "i", layers)
    _here("data", data, dev)
    if data.stride(2) != 1 or data.stride(1) != size:
        raise ValueError("a layer's pages must lie behind each other")
    rc = lib.cf_pages_copy(data.data_ptr(), pages, size, layers, data.stride(0), _flat("src", src, dev, torch.int32, (n,)),
                           _flat("dst", dst, dev, torch.int32, (n,)), n, _flat("count", count, dev, torch.int32, (1,)), _on(stream, dev))
    if rc:
        raise CFError("cf_pages_copy", rc)
