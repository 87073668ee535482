"""The decode step around the quantized products, on PyTorch tensors.

RMS norm with the residual add, rotary positions with the paged cache write, attention of one
new token over that cache, and the mixture-of-experts layer of a few tokens.  PyTorch only
allocates device buffers and supplies the stream; every operation is a libwq kernel.

Calls run on the current stream of their tensors' device, enqueue and return; none
synchronizes, so all of them may be captured into a graph.  A plan (PagedAttention, MoELayer)
owns a workspace: its calls must not overlap on different streams.  Tensors that a call is given
follow PyTorch's rules for streams other than their own; a plan's own memory is not reused before
the calls made on any stream are done.

The arguments of a call are packed as the bytes of its C struct and checked here only where
the library cannot see them (types, devices, shapes, strides): a call of a few microseconds on
the GPU should not take longer than that to make.
"""

from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import (WQ_ABI_VERSION, WQ_FLAG_BF16, WQ_FLAG_FP8, WQ_FLAG_HAS_ZP, WQ_MAX_ROPE_AXES,
               WQ_MOE_MAX_TOKENS, _check, lib, wq_attn_args, wq_expert_bank, wq_kv_cache,
               wq_moe_args, wq_moe_layer_workspace_bytes, wq_norm_args,
               wq_paged_attention_workspace_bytes, wq_rope_args)

_TYPE_FLAGS = {torch.float16: 0, torch.bfloat16: WQ_FLAG_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _layout(cls, fields: str) -> struct.Struct:
    """The native layout of a C argument struct after its version and size."""
    s = struct.Struct("@II" + fields + "0P")
    assert s.size == ctypes.sizeof(cls), cls
    return s


_CACHE = f"{ctypes.sizeof(wq_kv_cache)}s"
_BANK = f"{ctypes.sizeof(wq_expert_bank)}s"
_NORM = _layout(wq_norm_args, "6P6ifIi")
_ROPE = _layout(wq_rope_args, _CACHE + "8P8i" + f"{WQ_MAX_ROPE_AXES}iiIi")
_ATTN = _layout(wq_attn_args, _CACHE + "7PNP7iffiIi")
_MOE = _layout(wq_moe_args, "2P" + 2 * _BANK + "5PNP8ifiIi")


def _stream(dev: int) -> int:
    """The current stream of GPU `dev`, which has to be the current device."""
    if dev < 0:
        raise TypeError("GPU tensors expected")
    if _current_device() != dev:
        raise ValueError(f"the tensors are on GPU {dev}, the current device is "
                         f"{_current_device()}: call under torch.cuda.device({dev})")
    return _raw_stream(dev)


class _PlanMemory:
    """A plan's own tensors, and the stream they were allocated on."""

    def __init__(self, dev: int, *tensors: torch.Tensor):
        self.tensors, self.home = tensors, _raw_stream(dev) if dev >= 0 else None

    def stream(self, dev: int) -> int:
        """The current stream, for a call that uses the memory there."""
        stream = _stream(dev)
        if stream != self.home:
            for t in self.tensors:
                t.record_stream(torch.cuda.current_stream(dev))
        return stream


class _Call:
    """A library call that takes the bytes of its argument struct."""

    def __init__(self, name: str):
        self.name, self.fn = name, None

    def __call__(self, packed: bytes) -> None:
        if self.fn is None:
            self.fn = getattr(lib(), self.name)
        status = self.fn(packed)
        if status:
            _check(status)


_norm_call, _rope_call = _Call("wq_add_rms_norm"), _Call("wq_rope_append")
_attn_call, _moe_call = _Call("wq_paged_attention"), _Call("wq_moe_layer")


def _type_flag(dtype: torch.dtype) -> int:
    flag = _TYPE_FLAGS.get(dtype)
    if flag is None:
        raise TypeError(f"fp16 or bf16 expected, got {dtype}")
    return flag


def _check_type(t: torch.Tensor, name: str, dtype: torch.dtype, dev: int) -> None:
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name}: {dtype} on device {dev} expected, got {t.dtype} on "
                        f"{t.get_device()}")


def _rows(t: torch.Tensor, name: str, dtype, dev: int, shape) -> int:
    """The row stride of a [rows][cols] tensor of this shape."""
    if t.dtype is not dtype or t.get_device() != dev:
        _check_type(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name}: {tuple(shape)} expected, got {tuple(t.shape)}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    return ld if shape[0] > 1 else shape[1]


def _heads(t: torch.Tensor, name: str, dtype, dev: int, rows: int, heads: int, d: int) -> int:
    """The row stride of a [rows][heads][d] tensor whose heads lie one after another."""
    if t.dtype is not dtype or t.get_device() != dev:
        _check_type(t, name, dtype, dev)
    if t.shape != (rows, heads, d):
        raise ValueError(f"{name}: {(rows, heads, d)} expected, got {tuple(t.shape)}")
    ld, head, one = t.stride()
    if one != 1 or (head != d and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return ld if rows > 1 else heads * d


def _dense(t: torch.Tensor, name: str, dtype, dev: int, shape: tuple) -> int:
    """The address of a contiguous tensor of this shape."""
    if t.dtype is not dtype or t.get_device() != dev:
        _check_type(t, name, dtype, dev)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {shape} expected, got {tuple(t.shape)}")
    return t.data_ptr()


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
                 delta: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(y, s) of [rows][n] tensors: s = x + delta, y = s / sqrt(mean(s^2) + eps) * weight.
    Without delta, s is x itself.  sum_out may be x or delta (the residual stream kept in
    place), out likewise, but not both the same."""
    dtype, dev, shape = x.dtype, x.get_device(), x.shape
    flags = _type_flag(dtype)
    if len(shape) != 2:
        raise ValueError(f"x: two dimensions expected, got {tuple(shape)}")
    rows, n = shape
    ldx = _rows(x, "x", dtype, dev, shape)
    w = _dense(weight, "weight", dtype, dev, (n,))
    ldy = n
    if out is None:
        out = torch.empty_like(x)
    else:
        ldy = _rows(out, "out", dtype, dev, shape)
    dp = sp = ldd = lds = 0
    s = x
    if delta is not None:
        dp, ldd, lds = delta.data_ptr(), _rows(delta, "delta", dtype, dev, shape), n
        if sum_out is None:
            s = torch.empty_like(x)
        else:
            s, lds = sum_out, _rows(sum_out, "sum_out", dtype, dev, shape)
        sp = s.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs delta")
    if rows:
        _norm_call(_NORM.pack(WQ_ABI_VERSION, _NORM.size, x.data_ptr(), dp, w, sp, out.data_ptr(),
                              _stream(dev), rows, n, ldx, ldd, lds, ldy, eps, flags, 0))
    return out, s


class PagedCache:
    """A paged KV cache over two tensors seen as [page][slot][kv_head][head_dim] (any page,
    slot and head strides, the same for both; head-major storage is passed transposed):
    fp16, bf16, or float8_e4m3fn with fp32 scales per KV head (None: 1)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("K and V: two [page][slot][kv_head][head_dim] tensors of the same "
                             "shape and strides expected")
        if k.dtype != v.dtype or k.device != v.device:
            raise TypeError("K and V differ in type or device")
        self.fp8 = k.dtype is torch.float8_e4m3fn
        if not self.fp8:
            _type_flag(k.dtype)
        if k.stride(3) != 1:
            raise ValueError("the elements of a head must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dtype, self.device, self.dev = k.dtype, k.device, k.get_device()
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None:
                if not self.fp8:
                    raise ValueError(f"{name}: only an E4M3 cache has scales")
                _dense(s, name, torch.float32, self.dev, (self.kv_heads,))
        strides = [k.stride(i) if k.shape[i] > 1 else 0 for i in range(3)]
        self.packed = bytes(wq_kv_cache(
            k=k.data_ptr(), v=v.data_ptr(),
            k_scale=None if k_scale is None else k_scale.data_ptr(),
            v_scale=None if v_scale is None else v_scale.data_ptr(), page_stride=strides[0],
            slot_stride=strides[1], head_stride=strides[2], num_pages=self.num_pages,
            page_size=self.page_size, kv_heads=self.kv_heads, head_dim=self.head_dim))

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
              dtype: torch.dtype, device="cuda", k_scale=None, v_scale=None) -> "PagedCache":
        """A new cache, pages stored head-major: a KV head's slots of a page are contiguous."""
        k, v = (torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=dtype,
                            device=device).transpose(1, 2) for _ in range(2))
        return cls(k, v, k_scale, v_scale)

    def flags(self, dtype: torch.dtype) -> int:
        """The flags of a call whose q (or k and v) have this type."""
        if self.fp8:
            return _type_flag(dtype) | WQ_FLAG_FP8
        if dtype is not self.dtype:
            raise TypeError(f"the cache holds {self.dtype}, the call's tensors are {dtype}")
        return _type_flag(dtype)


def rope_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: PagedCache,
                slots: torch.Tensor, *, positions: torch.Tensor | None = None,
                inv_freq: torch.Tensor | None = None, sections=None, interleaved: bool = False,
                q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Rotates q [tokens][q_heads][d] and k [tokens][kv_heads][d] and writes k and v to their
    cache slots (int64 page * page_size + slot; -1 writes nothing).  Pair i turns by
    positions[axis(i)][token] * inv_freq[i]: positions int32 [axes][tokens] (or [tokens]),
    inv_freq fp32 [rot / 2] (None or empty: no rotation), sections the number of pairs of each
    axis.  Returns the rotated q (q_out, which may be q; a new tensor by default)."""
    dtype, dev, d, kv_heads = k.dtype, cache.dev, cache.head_dim, cache.kv_heads
    flags = cache.flags(dtype)
    tokens = k.shape[0]
    ldk = _heads(k, "k", dtype, dev, tokens, kv_heads, d)
    ldv = _heads(v, "v", dtype, dev, tokens, kv_heads, d)
    sl = _dense(slots, "slots", torch.int64, dev, (tokens,))
    qp = qo = heads = ldq = ldqo = 0
    if q is not None:
        heads = q.shape[1]
        ldq = _heads(q, "q", dtype, dev, tokens, heads, d)
        ldqo = heads * d
        if q_out is None:
            q_out = torch.empty_like(q)
        else:
            ldqo = _heads(q_out, "q_out", dtype, dev, tokens, heads, d)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    half = pp = fp = 0
    axes, pairs = 1, [0, 0, 0, 0]
    if inv_freq is not None:
        half = inv_freq.numel()
    if half:
        if positions is None:
            raise ValueError("inv_freq needs positions")
        shape = positions.shape
        axes = 1 if len(shape) == 1 else shape[0]
        if sections is None:
            if axes != 1:
                raise ValueError("several axes need sections")
            sections = (half,)
        if len(sections) != axes or axes > WQ_MAX_ROPE_AXES:
            raise ValueError(f"{axes} axes of positions, {len(sections)} sections")
        pairs[:axes] = sections
        fp = _dense(inv_freq, "inv_freq", torch.float32, dev, (half,))
        pp = _dense(positions, "positions", torch.int32, dev,
                    (tokens,) if len(shape) == 1 else (axes, tokens))
    if tokens:
        _rope_call(_ROPE.pack(WQ_ABI_VERSION, _ROPE.size, cache.packed, qp, k.data_ptr(),
                              v.data_ptr(), qo, sl, pp, fp, _stream(dev), tokens, heads, ldq, ldk,
                              ldv, ldqo, 2 * half, axes, *pairs, interleaved, flags, 0))
    return q_out


class PagedAttention:
    """Attention of one new token for `batch` sequences of up to `max_len` positions over a
    paged cache: the plan of a call and its workspace.  window: only the last that many
    positions; softcap: scores become softcap * tanh(score / softcap); scale: 1/sqrt(head_dim)
    by default.  One of its calls must not overlap another on a different stream."""

    def __init__(self, cache: PagedCache, batch: int, q_heads: int, max_len: int, *,
                 dtype: torch.dtype, scale: float | None = None, window: int = 0,
                 softcap: float = 0.0):
        self.cache, self.batch, self.q_heads, self.max_len = cache, batch, q_heads, max_len
        self.dtype, self.device = dtype, cache.device
        nbytes = wq_paged_attention_workspace_bytes(batch, q_heads, cache.kv_heads,
                                                    cache.head_dim, max_len, window,
                                                    cache.flags(dtype))
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self._space = (self.workspace.data_ptr(), nbytes)
        self._lse = torch.empty((batch, q_heads), dtype=torch.float32, device=self.device)
        self._memory = _PlanMemory(cache.dev, self.workspace)
        scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else scale
        self._last = (scale, softcap, window, cache.flags(dtype), 0)

    def __call__(self, q: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, *,
                 keep: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 lse: bool | torch.Tensor = False):
        """q [batch][q_heads][d]; block_table int32 [batch][pages]; lens int32 [batch]; keep
        uint8 [batch][>= max_len] (0: position left out).  Returns out, or (out, lse) when lse
        is True or a fp32 [batch][q_heads] tensor to write."""
        cache, b, heads, dtype = self.cache, self.batch, self.q_heads, self.dtype
        dev, d = cache.dev, cache.head_dim
        ldq = _heads(q, "q", dtype, dev, b, heads, d)
        ldo = heads * d
        if out is None:
            out = torch.empty_like(q)
        else:
            ldo = _heads(out, "out", dtype, dev, b, heads, d)
        pages = block_table.shape[-1]
        table = _dense(block_table, "block_table", torch.int32, dev, (b, pages))
        n = _dense(lens, "lens", torch.int32, dev, (b,))
        kp = lp = keep_stride = 0
        if keep is not None:
            keep_stride = keep.shape[-1]
            kp = _dense(keep, "keep", torch.uint8, dev, (b, keep_stride))
        if lse is not False:
            if lse is True:
                lse = torch.empty_like(self._lse)
                lp = lse.data_ptr()
            else:
                lp = _dense(lse, "lse", torch.float32, dev, (b, heads))
        _attn_call(_ATTN.pack(WQ_ABI_VERSION, _ATTN.size, cache.packed, q.data_ptr(),
                              out.data_ptr(), lp, table, n, kp, *self._space,
                              self._memory.stream(dev), b, heads, self.max_len, pages,
                              keep_stride, ldq, ldo, *self._last))
        return out if lse is False else (out, lse)


def _bank(bank) -> bytes:
    """The C view of a torch_ops.ExpertBank."""
    return bytes(wq_expert_bank(b=bank.b.data_ptr(), s=bank.s.data_ptr(),
                                zp=None if bank.z is None else bank.z.data_ptr(),
                                b_stride_bytes=bank.b_stride, s_stride_bytes=bank.s_stride,
                                zp_stride_bytes=bank.z_stride, group_size=bank.group_size))


class MoELayer:
    """A mixture-of-experts layer of up to `max_tokens` tokens over two torch_ops.ExpertBank
    (gate_up packed with the SwiGLU pairing, down) and a router weight [n_expert][hidden]:
    routing and all products on the device.  After a call, ids and weights hold the chosen
    experts and routing weights of its tokens.  One of its calls must not overlap another on a
    different stream."""

    def __init__(self, gate_up, down, router: torch.Tensor, top_k: int, *,
                 renormalize: bool = True, routed_scale: float = 1.0,
                 max_tokens: int = WQ_MOE_MAX_TOKENS):
        if not gate_up.swiglu or down.swiglu:
            raise ValueError("gate_up has to be a paired gate/up bank, down a plain one")
        self.hidden, self.inter, self.n_expert = gate_up.k, gate_up.n // 2, gate_up.n_expert
        if (down.k, down.n, down.n_expert) != (self.inter, self.hidden, self.n_expert):
            raise ValueError(f"down: {self.n_expert} experts of {self.inter} x {self.hidden} "
                             f"expected, got {down.n_expert} of {down.k} x {down.n}")
        if (gate_up.bf16, gate_up.fp8, gate_up.z is None) != (down.bf16, down.fp8, down.z is None):
            raise TypeError("the two banks differ in type")
        self.dtype = torch.bfloat16 if gate_up.bf16 else torch.float16
        self.device, self.dev = gate_up.b.device, gate_up.b.get_device()
        self.gate_up, self.down, self.router, self.top_k = gate_up, down, router, top_k
        nbytes = wq_moe_layer_workspace_bytes(max_tokens, self.n_expert, top_k, self.hidden,
                                              self.inter)
        self.max_tokens = max_tokens
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.ids = torch.empty((max_tokens, top_k), dtype=torch.int32, device=self.device)
        self.weights = torch.empty((max_tokens, top_k), dtype=torch.float32, device=self.device)
        self._memory = _PlanMemory(self.dev, self.workspace, self.ids, self.weights)
        r = _dense(router, "router", self.dtype, self.dev, (self.n_expert, self.hidden))
        self._banks = (r, _bank(gate_up), _bank(down))
        self._space = (self.ids.data_ptr(), self.weights.data_ptr(), self.workspace.data_ptr(),
                       nbytes)
        self._last = (routed_scale, int(renormalize),
                      _type_flag(self.dtype) | (WQ_FLAG_FP8 if gate_up.fp8 else 0)
                      | (WQ_FLAG_HAS_ZP if gate_up.z is not None else 0), 0)

    def __call__(self, x: torch.Tensor, *, residual: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """residual + the layer's output for x [tokens][hidden] (out may be residual or x)."""
        hidden, dtype, dev, shape = self.hidden, self.dtype, self.dev, x.shape
        tokens = shape[0]
        if not 0 < tokens <= self.max_tokens or shape[1:] != (hidden,):
            raise ValueError(f"x: [1 to {self.max_tokens}][{hidden}] expected, got {tuple(shape)}")
        ldx = _rows(x, "x", dtype, dev, shape)
        ldy = hidden
        if out is None:
            out = torch.empty_like(x)
        else:
            ldy = _rows(out, "out", dtype, dev, shape)
        rp = ldr = 0
        if residual is not None:
            rp, ldr = residual.data_ptr(), _rows(residual, "residual", dtype, dev, shape)
        router, gate_up, down = self._banks
        _moe_call(_MOE.pack(WQ_ABI_VERSION, _MOE.size, x.data_ptr(), router, gate_up, down, rp,
                            out.data_ptr(), *self._space, self._memory.stream(dev), tokens,
                            self.n_expert, self.top_k, hidden, self.inter, ldx, ldr, ldy,
                            *self._last))
        return out
