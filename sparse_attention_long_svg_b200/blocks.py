"""Query/key preparation and attention over key blocks chosen for each query.

Argument marshalling for the second group of libsvg.so calls (include/svg.h):
``qk_norm_rope`` turns a projection's token-major Q, K and V into the
head-major rows every attention call of the package reads (or appends them to a
K/V cache), ``block_mean`` -> ``block_select`` -> ``block_attn`` is attention in
which every query has its own block list (causal or not, shared key heads, a
growing context), and ``*_backward`` are the gradients.

All tensors of a call lie on one CUDA device, which need not be the current
one.  With ``stream`` the call runs, and allocates what it returns, on that
stream of the device.

Calls record nothing for autograd.  Those whose results depend smoothly on a
tensor that requires grad are refused, unless gradients are off: under
``torch.no_grad()``, or in the ``forward`` of a ``torch.autograd.Function``
whose ``backward`` calls the ``*_backward`` of the same name.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Sequence, Tuple

import torch

from . import _check, _need as _needs, load_library

_SIDE = contextlib.nullcontext()
_Strides = ctypes.c_int64 * 3

# A single token's call takes a few microseconds on the device, so the checks
# here are written to cost little on the host: attributes are read once, and
# ctypes converts plain integers.


def _side(stream, *tensors):
    """Checks that the tensors share a device; the context in which to allocate and launch."""
    index = tensors[0].get_device()
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on {tensors[0].device}, got {t.device}")
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream of {stream.device} for tensors on {tensors[0].device}")
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return torch.cuda.stream(stream)
    if index != _device():
        return torch.cuda.device(index)
    return _SIDE


def _constant(call: str, instead: str, *tensors):
    """Refuses tensors whose gradient would be lost."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{call} records no gradient, but an input requires grad: {instead}")


def _device() -> int:
    return torch._C._cuda_getDevice()


def _stream() -> int:
    """The current stream of the current device, as the library takes it."""
    return torch._C._cuda_getCurrentRawStream(_device())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, dims: int):
    if not (t.dtype == dtype and t.dim() == dims and t.is_contiguous() and t.is_cuda):
        _needs(t, name, dtype, dims)


def _same(t: torch.Tensor, name: str, shape, dtype):
    if not (t.dtype == dtype and t.shape == shape and t.is_contiguous()):
        _needs(t, name, dtype, len(shape))
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, device) -> torch.Tensor:
    """An output buffer: made here, or the caller's, checked."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _same(t, name, shape, dtype)
    return t


def _scratch(workspace, nbytes: int, device):
    """(workspace or None, its size): nothing is allocated where a call needs none."""
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return workspace, workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, 0
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def _seqs(kv_len, BHk: int) -> int:
    if kv_len is None:
        return 1
    _need(kv_len, "kv_len", torch.int32, 1)
    B = kv_len.shape[0]
    if B < 1 or BHk % B != 0:
        raise ValueError(f"kv_len has {B} entries, which do not divide {BHk} key heads")
    return B


# ----------------------------------------------------------------------- norm and rotation

def rope_table(grid: Sequence[int], D: int, theta: float = 10000.0, split: Optional[Sequence[int]] = None,
               device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """Cosines and sines [prod(grid), D/2] fp32 of the rotation by a token's place in `grid`.

    One entry (a sequence) or several, e.g. (frames, height, width) of a clip in raster order; `split` says how
    many of the D/2 pairs turn by each coordinate (default: as even as possible, the first ones get the rest).
    Pair i of a coordinate with n pairs turns by coordinate * theta^(-i/n).  Angles are formed in float64.
    """
    half, axes = D // 2, len(grid)
    if split is None:
        split = [half // axes + (1 if i < half % axes else 0) for i in range(axes)]
    if len(split) != axes or sum(split) != half or min(split) < 0 or min(grid) < 1:
        raise ValueError(f"split {tuple(split)} must give {half} pairs to the {axes} coordinates of {tuple(grid)}")
    parts = []
    for axis, (size, pairs) in enumerate(zip(grid, split)):
        speed = theta ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
        angle = torch.arange(size, dtype=torch.float64)[:, None] * speed
        shape = [1] * axes + [pairs]
        shape[axis] = size
        parts.append(angle.view(shape).expand(*grid, pairs))
    angle = torch.cat(parts, -1).reshape(-1, half)
    return angle.cos().float().to(device), angle.sin().float().to(device)


def _view(t: torch.Tensor, name: str, shape):
    """A token-major [B, N, H, D] bf16 view: channels contiguous.  Returns (pointer, int64[3] strides)."""
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    sb, sn, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    if 1 in shape:                   # the stride of a dimension of size 1 is of no account
        B, N, H, _ = shape
        sb, sn, sh = sb if B > 1 else 0, sn if N > 1 else 0, sh if H > 1 else 0
    return t.data_ptr(), _Strides(sb, sn, sh)


def _overlaps(t: torch.Tensor) -> bool:
    """Whether a [B, N, H, D] view with contiguous channels may name an element twice."""
    reach = t.shape[3]
    for size, stride in sorted(((t.shape[i], t.stride(i)) for i in range(3)), key=lambda x: x[1]):
        if size > 1:
            if stride < reach:
                return True
            reach = stride * (size - 1) + reach
    return False


def _rope_common(q, k, v, w_q, w_k, cos, sin, start):
    if q.dim() != 4:
        raise ValueError(f"q must be [B, N, heads, D], got {tuple(q.shape)}")
    B, N, Hq, D = q.shape
    if v is not None and k is None:
        raise ValueError("v without k")
    Hk = 0 if k is None else k.shape[2] if k.dim() == 4 else -1
    for w, n in ((w_q, "w_q"), (w_k, "w_k")):
        if w is not None:
            _same(w, n, (D,), torch.float32)
    P = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        P = cos.shape[0]
        _same(cos, "cos", (P, D // 2), torch.float32)
        _same(sin, "sin", (P, D // 2), torch.float32)
    if start is not None:
        _same(start, "start", (B,), torch.int32)
    return B, N, Hq, Hk, D, P


def _cap(t, name: str, rows: int, D: int, N: int) -> int:
    _need(t, name, torch.bfloat16, 3)
    if t.shape[0] != rows or t.shape[2] != D:
        raise ValueError(f"{name} must be [{rows}, rows, {D}], got {tuple(t.shape)}")
    return t.shape[1]


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                 w_q: Optional[torch.Tensor] = None, w_k: Optional[torch.Tensor] = None,
                 cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = True, start: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 v_out: Optional[torch.Tensor] = None, stream=None):
    """RMS norm of every head of Q and K, rotation by position, and the move to head-major rows, in one pass.

    q [B, N, Hq, D], k and v [B, N, Hk, D] bf16: views of token-major data (e.g. slices of one projection's
    output); w_q, w_k [D] fp32 or None (ones); cos, sin [P, D/2] fp32 or None (no rotation), one row per position;
    start [B] int32: position of each sequence's token 0 (None: 0).  q_out [B*Hq, N, D]; k_out, v_out
    [B*Hk, cap, D]: token n goes to row start[b] + n, other rows stay as they are (None: new buffers of N rows,
    without start only; a new v_out has k_out's rows, zeros behind the N).  Negative positions are padding (see
    svg_qk_norm_rope).  Returns (q_out, k_out, v_out).
    """
    lib = load_library()
    _constant("qk_norm_rope", "call it under torch.no_grad() and qk_norm_rope_backward for the gradient",
              q, k, v, w_q, w_k)
    B, N, Hq, Hk, D, P = _rope_common(q, k, v, w_q, w_k, cos, sin, start)
    with _side(stream, q, k, v, w_q, w_k, cos, sin, start, q_out, k_out, v_out):
        dev, bf = q.device, torch.bfloat16
        pq, sq = _view(q, "q", (B, N, Hq, D))
        pk = pv = sk = sv = None
        cap = 0
        if start is not None and ((k is not None and k_out is None) or (v is not None and v_out is None)):
            raise ValueError("start places rows in k_out and v_out: give both buffers")
        q_out = _out(q_out, "q_out", (B * Hq, N, D), bf, dev)
        if k is not None:
            pk, sk = _view(k, "k", (B, N, Hk, D))
            if k_out is None:
                k_out = torch.empty((B * Hk, N, D), dtype=bf, device=dev)
            cap = _cap(k_out, "k_out", B * Hk, D, N)
        if v is not None:
            pv, sv = _view(v, "v", (B, N, Hk, D))
            if v_out is None and cap > N:             # beside a longer k_out: rows that nobody writes are zero
                v_out = torch.zeros((B * Hk, cap, D), dtype=bf, device=dev)
            v_out = _out(v_out, "v_out", (B * Hk, cap, D), bf, dev)
        _check("svg_qk_norm_rope", lib.svg_qk_norm_rope(
            pq, sq, pk, sk, pv, sv, _ptr(w_q), _ptr(w_k), _ptr(cos), _ptr(sin), P, B, N, Hq, Hk, D, float(eps),
            1 if interleaved else 0, _ptr(start), _ptr(q_out), _ptr(k_out if k is not None else None),
            _ptr(v_out if v is not None else None), cap, _stream()))
    return q_out, k_out if k is not None else None, v_out if v is not None else None


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], dv_out: Optional[torch.Tensor],
                          q: torch.Tensor, k: Optional[torch.Tensor] = None,
                          w_q: Optional[torch.Tensor] = None, w_k: Optional[torch.Tensor] = None,
                          cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          interleaved: bool = True, start: Optional[torch.Tensor] = None,
                          dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                          dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of qk_norm_rope.  dq_out, dk_out, dv_out: gradients of its outputs, laid out like them; q, k and
    the rest: what the forward call was given.  dq, dk, dv: views like the inputs (None: new contiguous ones).
    Returns (dq, dk, dv, dw_q, dw_k), the weights' [D] fp32."""
    lib = load_library()
    B, N, Hq, Hk, D, P = _rope_common(q, k, None, w_q, w_k, cos, sin, start)
    if (k is None) != (dk_out is None) or (dv_out is not None and k is None):
        raise ValueError("k and dk_out go together, and dv_out needs them")
    with _side(stream, q, k, w_q, w_k, cos, sin, start, dq_out, dk_out, dv_out, dq, dk, dv, workspace):
        dev, bf = q.device, torch.bfloat16
        pq, sq = _view(q, "q", (B, N, Hq, D))
        _same(dq_out, "dq_out", (B * Hq, N, D), bf)
        pk = sk = sdk = sdv = pdk = pdv = None
        cap = 0

        def grad(t, name, H):
            if t is None:
                t = torch.empty((B, N, H, D), dtype=bf, device=dev)
            elif t.dim() == 4 and _overlaps(t):
                raise ValueError(f"{name} must not name an element twice")
            return (t, *_view(t, name, (B, N, H, D)))

        dq, pdq, sdq = grad(dq, "dq", Hq)
        if k is not None:
            pk, sk = _view(k, "k", (B, N, Hk, D))
            cap = _cap(dk_out, "dk_out", B * Hk, D, N)
            dk, pdk, sdk = grad(dk, "dk", Hk)
        if dv_out is not None:
            _same(dv_out, "dv_out", (B * Hk, cap, D), bf)
            dv, pdv, sdv = grad(dv, "dv", Hk)
        dw_q = torch.empty(D, dtype=torch.float32, device=dev)
        dw_k = torch.empty(D, dtype=torch.float32, device=dev) if k is not None else None
        workspace, nbytes = _scratch(workspace, lib.svg_qk_norm_rope_backward_workspace_size(B, N, Hq, Hk, D), dev)
        _check("svg_qk_norm_rope_backward", lib.svg_qk_norm_rope_backward(
            _ptr(dq_out), _ptr(dk_out), _ptr(dv_out), pq, sq, pk, sk, _ptr(w_q), _ptr(w_k), _ptr(cos), _ptr(sin), P,
            B, N, Hq, Hk, D, float(eps), 1 if interleaved else 0, _ptr(start), cap, pdq, sdq, pdk, sdk, pdv, sdv,
            _ptr(dw_q), _ptr(dw_k), _ptr(workspace), nbytes, _stream()))
    return dq, dk if k is not None else None, dv if dv_out is not None else None, dw_q, dw_k


# ----------------------------------------------------------------------- blocks chosen for each query

def block_mean(k: torch.Tensor, block: int, kv_len: Optional[torch.Tensor] = None, new: int = 0,
               mean: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Mean key of every block of `block` rows of k [BHk, Nk, D] bf16: [BHk, ceil(Nk/block), D] fp32.

    kv_len [B] int32: keys in use (None: all).  With `new` > 0 only the blocks that hold any of a sequence's last
    `new` keys are formed, in place in `mean` (the means of a cache after a decoding step)."""
    lib = load_library()
    _constant("block_mean", "give it k.detach(): means serve the choice of blocks, which is constant", k)
    _need(k, "k", torch.bfloat16, 3)
    BHk, Nk, D = k.shape
    B = _seqs(kv_len, BHk)
    if block < 1:
        raise ValueError(f"block must be positive, got {block}")
    if new and mean is None:
        raise ValueError("new updates the means of a cache in place: give mean")
    with _side(stream, k, kv_len, mean):
        mean = _out(mean, "mean", (BHk, -(-Nk // block), D), torch.float32, k.device)
        _check("svg_block_mean", lib.svg_block_mean(_ptr(k), BHk, B, Nk, D, int(block), _ptr(kv_len), int(new),
                                                    _ptr(mean), _stream()))
    return mean


def block_select(q: torch.Tensor, mean: torch.Tensor, block: int, topk: int, Nk: int, sink: int = 1, local: int = 2,
                 causal: bool = True, kv_len: Optional[torch.Tensor] = None, sel: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Block list of every query: the first `sink` blocks, the `local` ones up to the query's own, and those with
    the largest (sum of the group's q) . mean, `topk` in all; ascending, filled up with -1.

    q [BHq, Nq, D] bf16 (the last Nq tokens of their sequences), mean [BHk, ceil(Nk/block), D] fp32 of buffers of
    Nk rows.  Returns sel [BHk, Nq, topk] int32."""
    lib = load_library()
    _need(q, "q", torch.bfloat16, 3)
    _need(mean, "mean", torch.float32, 3)
    BHq, Nq, D = q.shape
    BHk = mean.shape[0]
    B = _seqs(kv_len, BHk)
    if block < 1:
        raise ValueError(f"block must be positive, got {block}")
    if topk < 1:
        raise ValueError(f"topk must be positive, got {topk}")
    _same(mean, "mean", (BHk, -(-Nk // block), D), torch.float32)
    with _side(stream, q, mean, kv_len, sel, workspace):
        sel = _out(sel, "sel", (BHk, Nq, topk), torch.int32, q.device)
        workspace, nbytes = _scratch(
            workspace, lib.svg_block_select_workspace_size(BHk, Nq, int(Nk), D, int(block)), q.device)
        _check("svg_block_select", lib.svg_block_select(
            _ptr(q), _ptr(mean), BHq, BHk, B, Nq, int(Nk), D, int(block), int(topk), int(sink), int(local),
            1 if causal else 0, _ptr(kv_len), _ptr(sel), _ptr(workspace), nbytes, _stream()))
    return sel


_ATTN_INSTEAD = "call it under torch.no_grad() and block_attn_backward for the gradient"


def _attn_shapes(q, k, v, sel, kv_len):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 3)
    _need(sel, "sel", torch.int32, 3)
    BHq, Nq, D = q.shape
    BHk, Nk, _ = k.shape
    _same(k, "k", (BHk, Nk, D), torch.bfloat16)
    _same(v, "v", (BHk, Nk, D), torch.bfloat16)
    topk = sel.shape[2]
    _same(sel, "sel", (BHk, Nq, topk), torch.int32)
    return BHq, BHk, _seqs(kv_len, BHk), Nq, Nk, D, topk


def block_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, sel: torch.Tensor, block: int,
               causal: bool = True, scale: float = 0.0, kv_len: Optional[torch.Tensor] = None,
               o: Optional[torch.Tensor] = None, want_lse: bool = False, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None):
    """Softmax attention of every query over the keys of its listed blocks.

    q [BHq, Nq, D], k, v [BHk, Nk, D] bf16, sel [BHk, Nq, topk] int32 (block_select; -1 is passed over).  Query
    head h reads key head h // (BHq / BHk).  A query without a visible key gets zeros.  Returns (o, lse or None)."""
    lib = load_library()
    _constant("block_attn", _ATTN_INSTEAD, q, k, v)
    BHq, BHk, B, Nq, Nk, D, topk = _attn_shapes(q, k, v, sel, kv_len)
    with _side(stream, q, k, v, sel, kv_len, o, lse, workspace):
        o = _out(o, "o", (BHq, Nq, D), torch.bfloat16, q.device)
        if want_lse or lse is not None:
            lse = _out(lse, "lse", (BHq, Nq), torch.float32, q.device)
        workspace, nbytes = _scratch(
            workspace, lib.svg_block_attn_workspace_size(BHq, BHk, Nq, Nk, D, topk, int(block)), q.device)
        _check("svg_block_attn", lib.svg_block_attn(
            _ptr(q), _ptr(k), _ptr(v), BHq, BHk, B, Nq, Nk, D, _ptr(sel), topk, int(block), 1 if causal else 0,
            float(scale), _ptr(kv_len), _ptr(o), _ptr(lse), _ptr(workspace), nbytes, _stream()))
    return o, lse


def block_attn_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                        lse: torch.Tensor, sel: torch.Tensor, block: int, causal: bool = True, scale: float = 0.0,
                        kv_len: Optional[torch.Tensor] = None, dq: Optional[torch.Tensor] = None,
                        dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of block_attn from do and the forward call's inputs, o and lse.  Returns (dq, dk, dv)."""
    lib = load_library()
    BHq, BHk, B, Nq, Nk, D, topk = _attn_shapes(q, k, v, sel, kv_len)
    _same(do, "do", (BHq, Nq, D), torch.bfloat16)
    _same(o, "o", (BHq, Nq, D), torch.bfloat16)
    _same(lse, "lse", (BHq, Nq), torch.float32)
    with _side(stream, q, k, v, o, lse, do, sel, kv_len, dq, dk, dv, workspace):
        dev = q.device
        dq = _out(dq, "dq", (BHq, Nq, D), torch.bfloat16, dev)
        dk = _out(dk, "dk", (BHk, Nk, D), torch.bfloat16, dev)
        dv = _out(dv, "dv", (BHk, Nk, D), torch.bfloat16, dev)
        workspace, nbytes = _scratch(
            workspace, lib.svg_block_attn_backward_workspace_size(BHq, BHk, Nq, Nk, D, topk, int(block)), dev)
        _check("svg_block_attn_backward", lib.svg_block_attn_backward(
            _ptr(do), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), BHq, BHk, B, Nq, Nk, D, _ptr(sel), topk,
            int(block), 1 if causal else 0, float(scale), _ptr(kv_len), _ptr(dq), _ptr(dk), _ptr(dv),
            _ptr(workspace), nbytes, _stream()))
    return dq, dk, dv


def block_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block: int, topk: int, sink: int = 1,
                    local: int = 2, causal: bool = True, scale: float = 0.0,
                    kv_len: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None, new: int = 0,
                    want_lse: bool = False, stream=None):
    """block_mean, block_select and block_attn on head-major Q, K and V.

    `mean` with `new` > 0: the means of a cache, brought up to date for its last `new` keys; else all are formed
    (into `mean` if given).  Returns (o, lse or None, sel, mean)."""
    _constant("block_attention", _ATTN_INSTEAD, q, k, v)
    mean = block_mean(k, block, kv_len, new, mean, stream)
    sel = block_select(q, mean, block, topk, k.shape[1], sink, local, causal, kv_len, stream=stream)
    o, lse = block_attn(q, k, v, sel, block, causal, scale, kv_len, want_lse=want_lse, stream=stream)
    return o, lse, sel, mean
