"""The decode step around the quantized products, on PyTorch tensors.

RMS norm with the residual add, rotary positions with the paged cache write, attention of one
new token over that cache, and the mixture-of-experts layer of a few tokens.  PyTorch only
allocates device buffers and supplies the stream; every operation is a libwq kernel.

Calls run on the current stream of their tensors' device, enqueue and return; none
synchronizes, so all of them may be captured into a graph (pass the outputs then, or keep
what the call returns).  A plan (PagedAttention, MoELayer) owns a workspace: its calls must
not overlap on different streams.
"""

from __future__ import annotations

import math

import torch

from . import (WQ_FLAG_BF16, WQ_FLAG_FP8, WQ_FLAG_HAS_ZP, WQ_MOE_MAX_TOKENS, versioned,
               wq_add_rms_norm, wq_attn_args, wq_expert_bank, wq_kv_cache, wq_moe_args,
               wq_moe_layer, wq_moe_layer_workspace_bytes, wq_norm_args, wq_paged_attention,
               wq_paged_attention_workspace_bytes, wq_rope_append, wq_rope_args)

_FLOATS = (torch.float16, torch.bfloat16)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else None


def _enqueue(call, args, device: torch.device) -> None:
    """call(args) on the device's current stream, with that device current."""
    index = device.index
    if _raw_stream is None:
        raise RuntimeError("this PyTorch build has no GPU support")
    args.stream = _raw_stream(index)
    if index == torch.cuda.current_device():
        call(args)
    else:
        with torch.cuda.device(index):
            call(args)


def _flag(dtype: torch.dtype) -> int:
    if dtype is torch.float16:
        return 0
    if dtype is torch.bfloat16:
        return WQ_FLAG_BF16
    raise TypeError(f"fp16 or bf16 expected, got {dtype}")


def _rows(t: torch.Tensor, name: str, dtype, device, cols: int, rows: int | None = None) -> int:
    """The row stride of a [rows][cols] tensor, checked."""
    if t.dtype is not dtype or t.device != device:
        raise TypeError(f"{name}: {dtype} on {device} expected, got {t.dtype} on {t.device}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name}: [{rows or 'rows'}][{cols}] expected, got {tuple(shape)}")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    return ld if shape[0] > 1 else max(ld, cols)


def _heads(t: torch.Tensor, name: str, dtype, device, rows: int, heads: int, d: int) -> int:
    """The row stride of a [rows][heads][d] tensor whose heads lie one after another."""
    if t.dtype is not dtype or t.device != device:
        raise TypeError(f"{name}: {dtype} on {device} expected, got {t.dtype} on {t.device}")
    if t.shape != (rows, heads, d):
        raise ValueError(f"{name}: {(rows, heads, d)} expected, got {tuple(t.shape)}")
    ld, head, one = t.stride()
    if one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return ld if rows > 1 else max(ld, heads * d)


def _index(t: torch.Tensor, name: str, dtype, device, shape) -> int:
    if t.dtype is not dtype or t.device != device:
        raise TypeError(f"{name}: {dtype} on {device} expected, got {t.dtype} on {t.device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {tuple(shape)} expected, got {tuple(t.shape)}")
    return t.data_ptr()


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
                 delta: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(y, s) of [rows][n] tensors: s = x + delta, y = s / sqrt(mean(s^2) + eps) * weight.
    Without delta, s is x itself.  sum_out may be x or delta (the residual stream kept in
    place), out likewise, but not both the same."""
    if x.dtype not in _FLOATS:
        raise TypeError(f"fp16 or bf16 expected, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"x: two dimensions expected, got {tuple(x.shape)}")
    rows, n = x.shape
    dtype, device = x.dtype, x.device
    if out is None:
        out = torch.empty((rows, n), dtype=dtype, device=device)
    args = versioned(wq_norm_args, x=x.data_ptr(), y=out.data_ptr(),
                     weight=_index(weight, "weight", dtype, device, (n,)), rows=rows, n=n,
                     ldx=_rows(x, "x", dtype, device, n), eps=eps, flags=_flag(dtype),
                     ldy=_rows(out, "out", dtype, device, n, rows))
    if delta is not None:
        if sum_out is None:
            sum_out = torch.empty((rows, n), dtype=dtype, device=device)
        args.delta, args.ldd = delta.data_ptr(), _rows(delta, "delta", dtype, device, n, rows)
        args.sum_out, args.lds = (sum_out.data_ptr(),
                                  _rows(sum_out, "sum_out", dtype, device, n, rows))
    elif sum_out is not None:
        raise ValueError("sum_out needs delta")
    else:
        sum_out = x
    if rows:
        _enqueue(wq_add_rms_norm, args, device)
    return out, sum_out


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
        if not self.fp8 and k.dtype not in _FLOATS:
            raise TypeError(f"fp16, bf16 or float8_e4m3fn expected, got {k.dtype}")
        if k.stride(3) != 1:
            raise ValueError("the elements of a head must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dtype, self.device = k.dtype, k.device
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None:
                if not self.fp8:
                    raise ValueError(f"{name}: only an E4M3 cache has scales")
                _index(s, name, torch.float32, self.device, (self.kv_heads,))
        strides = [k.stride(i) if k.shape[i] > 1 else 0 for i in range(3)]
        self.args = wq_kv_cache(
            k=k.data_ptr(), v=v.data_ptr(),
            k_scale=None if k_scale is None else k_scale.data_ptr(),
            v_scale=None if v_scale is None else v_scale.data_ptr(), page_stride=strides[0],
            slot_stride=strides[1], head_stride=strides[2], num_pages=self.num_pages,
            page_size=self.page_size, kv_heads=self.kv_heads, head_dim=self.head_dim)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
              dtype: torch.dtype, device="cuda", k_scale=None, v_scale=None) -> "PagedCache":
        """A new cache, pages stored head-major: a KV head's slots of a page are contiguous."""
        k, v = (torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=dtype,
                            device=device).transpose(1, 2) for _ in range(2))
        return cls(k, v, k_scale, v_scale)

    def check_type(self, dtype: torch.dtype) -> int:
        """The flags of a call whose q (or k and v) have this type."""
        if not self.fp8 and dtype is not self.dtype:
            raise TypeError(f"the cache holds {self.dtype}, the call's tensors are {dtype}")
        return _flag(dtype) | (WQ_FLAG_FP8 if self.fp8 else 0)


def rope_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: PagedCache,
                slots: torch.Tensor, *, positions: torch.Tensor | None = None,
                inv_freq: torch.Tensor | None = None, sections=None, interleaved: bool = False,
                q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Rotates q [tokens][q_heads][d] and k [tokens][kv_heads][d] and writes k and v to their
    cache slots (int64 page * page_size + slot; -1 writes nothing).  Pair i turns by
    positions[axis(i)][token] * inv_freq[i]: positions int32 [axes][tokens] (or [tokens]),
    inv_freq fp32 [rot / 2] (None or empty: no rotation), sections the number of pairs of each
    axis.  Returns the rotated q (q_out, which may be q; a new tensor by default)."""
    tokens = k.shape[0]
    dtype, device, d = k.dtype, k.device, cache.head_dim
    if device != cache.device:
        raise TypeError(f"the cache is on {cache.device}, k on {device}")
    args = versioned(wq_rope_args, cache=cache.args, k=k.data_ptr(), v=v.data_ptr(),
                     ldk=_heads(k, "k", dtype, device, tokens, cache.kv_heads, d),
                     ldv=_heads(v, "v", dtype, device, tokens, cache.kv_heads, d),
                     slots=_index(slots, "slots", torch.int64, device, (tokens,)),
                     tokens=tokens, axes=1, interleaved=int(interleaved),
                     flags=cache.check_type(dtype))
    if q is not None:
        heads = q.shape[1]
        if q_out is None:
            q_out = torch.empty((tokens, heads, d), dtype=dtype, device=device)
        args.q, args.q_out, args.q_heads = q.data_ptr(), q_out.data_ptr(), heads
        args.ldq = _heads(q, "q", dtype, device, tokens, heads, d)
        args.ldqo = _heads(q_out, "q_out", dtype, device, tokens, heads, d)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if inv_freq is not None and inv_freq.numel():
        half = inv_freq.numel()
        if positions is None:
            raise ValueError("inv_freq needs positions")
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        if sections is None:
            if axes != 1:
                raise ValueError("several axes need sections")
            sections = (half,)
        if len(sections) != axes or axes > len(args.sections):
            raise ValueError(f"{axes} axes of positions, {len(sections)} sections")
        args.rot_dim, args.axes = 2 * half, axes
        for i, pairs in enumerate(sections):
            args.sections[i] = pairs
        args.inv_freq = _index(inv_freq, "inv_freq", torch.float32, device, (half,))
        args.positions = _index(positions, "positions", torch.int32, device,
                                (tokens,) if positions.dim() == 1 else (axes, tokens))
    if tokens:
        _enqueue(wq_rope_append, args, device)
    return q_out


class PagedAttention:
    """Attention of one new token for up to `batch` sequences of up to `max_len` positions
    over a paged cache: the plan of a call and its workspace.  window: only the last that many
    positions; softcap: scores become softcap * tanh(score / softcap); scale: 1/sqrt(head_dim)
    by default.  One of its calls must not overlap another on a different stream."""

    def __init__(self, cache: PagedCache, batch: int, q_heads: int, max_len: int, *,
                 dtype: torch.dtype, scale: float | None = None, window: int = 0,
                 softcap: float = 0.0):
        self.cache, self.batch, self.q_heads, self.max_len = cache, batch, q_heads, max_len
        self.dtype, self.device = dtype, cache.device
        nbytes = wq_paged_attention_workspace_bytes(batch, q_heads, cache.kv_heads,
                                                    cache.head_dim, max_len, window)
        self.workspace = (torch.empty(nbytes, dtype=torch.uint8, device=self.device)
                          if nbytes else None)
        self._args = versioned(
            wq_attn_args, cache=cache.args, q_heads=q_heads, max_len=max_len, window=window,
            softcap=softcap, flags=cache.check_type(dtype),
            scale=1.0 / math.sqrt(cache.head_dim) if scale is None else scale,
            workspace=None if self.workspace is None else self.workspace.data_ptr(),
            workspace_bytes=nbytes)

    def __call__(self, q: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, *,
                 keep: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 lse: bool | torch.Tensor = False):
        """q [batch][q_heads][d]; block_table int32 [batch][pages]; lens int32 [batch]; keep
        uint8 [batch][>= max_len] (0: position left out).  Returns out, or (out, lse) when lse
        is True or a fp32 [batch][q_heads] tensor to write."""
        b, d, device = self.batch, self.cache.head_dim, self.device
        args = wq_attn_args.from_buffer_copy(self._args)
        if out is None:
            out = torch.empty((b, self.q_heads, d), dtype=self.dtype, device=device)
        if lse is True:
            lse = torch.empty((b, self.q_heads), dtype=torch.float32, device=device)
        args.batch = b
        args.q, args.out = q.data_ptr(), out.data_ptr()
        args.ldq = _heads(q, "q", self.dtype, device, b, self.q_heads, d)
        args.ldo = _heads(out, "out", self.dtype, device, b, self.q_heads, d)
        args.table_stride = block_table.shape[-1]
        args.block_table = _index(block_table, "block_table", torch.int32, device,
                                  (b, block_table.shape[-1]))
        args.lens = _index(lens, "lens", torch.int32, device, (b,))
        if keep is not None:
            args.keep_stride = keep.shape[-1]
            args.keep = _index(keep, "keep", torch.uint8, device, (b, keep.shape[-1]))
        if lse is not False:
            args.lse = _index(lse, "lse", torch.float32, device, (b, self.q_heads))
        _enqueue(wq_paged_attention, args, device)
        return out if lse is False else (out, lse)


def _bank(bank) -> wq_expert_bank:
    """The C view of a torch_ops.ExpertBank."""
    return wq_expert_bank(b=bank.b.data_ptr(), s=bank.s.data_ptr(),
                          zp=None if bank.z is None else bank.z.data_ptr(),
                          b_stride_bytes=bank.b_stride, s_stride_bytes=bank.s_stride,
                          zp_stride_bytes=bank.z_stride, group_size=bank.group_size)


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
        self.device = gate_up.b.device
        self.gate_up, self.down, self.router, self.top_k = gate_up, down, router, top_k
        nbytes = wq_moe_layer_workspace_bytes(max_tokens, self.n_expert, top_k, self.hidden,
                                              self.inter)
        self.max_tokens = max_tokens
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.ids = torch.empty((max_tokens, top_k), dtype=torch.int32, device=self.device)
        self.weights = torch.empty((max_tokens, top_k), dtype=torch.float32, device=self.device)
        self._args = versioned(
            wq_moe_args, gate_up=_bank(gate_up), down=_bank(down),
            router=_index(router, "router", self.dtype, self.device,
                          (self.n_expert, self.hidden)),
            ids=self.ids.data_ptr(), weights=self.weights.data_ptr(),
            workspace=self.workspace.data_ptr(), workspace_bytes=nbytes,
            n_expert=self.n_expert, top_k=top_k, hidden=self.hidden, inter=self.inter,
            routed_scale=routed_scale, renormalize=int(renormalize),
            flags=_flag(self.dtype) | (WQ_FLAG_FP8 if gate_up.fp8 else 0)
            | (WQ_FLAG_HAS_ZP if gate_up.z is not None else 0))

    def __call__(self, x: torch.Tensor, *, residual: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """residual + the layer's output for x [tokens][hidden] (out may be residual or x)."""
        tokens, device = x.shape[0], self.device
        if not 0 < tokens <= self.max_tokens:
            raise ValueError(f"1 to {self.max_tokens} tokens expected, got {tokens}")
        args = wq_moe_args.from_buffer_copy(self._args)
        if out is None:
            out = torch.empty((tokens, self.hidden), dtype=self.dtype, device=device)
        args.tokens, args.x, args.y = tokens, x.data_ptr(), out.data_ptr()
        args.ldx = _rows(x, "x", self.dtype, device, self.hidden)
        args.ldy = _rows(out, "out", self.dtype, device, self.hidden, tokens)
        if residual is not None:
            args.residual = residual.data_ptr()
            args.ldr = _rows(residual, "residual", self.dtype, device, self.hidden, tokens)
        _enqueue(wq_moe_layer, args, device)
        return out
