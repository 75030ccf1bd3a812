"""The layer operators on packed ragged batches and single tokens.

Binding of the second half of ``include/bidir_ssd.h``:

  ssd_conv / ssd_conv_bwd     the causal convolution with carried states, and its gradients
  ssd_scan_ragged             the scan over packed ragged sequences, states in slots
  mamba2_step                 one token per row: convolution, SiLU, softplus, recurrence
  ffn_block / ffn_block_bwd   the gated feed-forward block, and its gradients

Packed batches: the rows of every tensor are the tokens of all sequences, one sequence behind
another, and ``cu_seqlens`` (int32, on the device, ``nseq + 1`` entries) holds where each starts.
Without ``cu_seqlens`` the tensors have a batch dimension in front and every sequence that many rows.
Rows may be any stride apart (column blocks of a packed projection need no copy); the elements of a
row are contiguous.  Outputs are contiguous unless ``out`` is given.

``workspace``: a uint8 CUDA tensor whose first 256 bytes are zero before its first use, read by
``workspace_status`` afterwards; it tells of index arrays that do not keep the contract.  Without one
the call takes its scratch from PyTorch and nothing is reported.
"""
from __future__ import annotations

import ctypes

import torch

from . import SSDError, _check, _stream, lib  # noqa: F401

__all__ = ["ssd_conv", "ssd_conv_bwd", "ssd_scan_ragged", "ragged_workspace_bytes", "mamba2_step", "step_workspace_bytes",
           "ffn_block", "ffn_block_bwd", "ffn_workspace_bytes", "ffn_bwd_workspace_bytes"]

_VP, _SZ, _LL, _I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_int


class _Packed(ctypes.Structure):
    _fields_ = [("cu_seqlens", _VP), ("nseq", _I), ("tokens", _I)]


class _Slots(ctypes.Structure):
    _fields_ = [("pool_in", _VP), ("pool_out", _VP), ("slots_in", _VP), ("slots_out", _VP), ("n_in", _I), ("n_out", _I)]


class _ConvShape(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("channels", "width", "direction", "silu", "io")]


class _RaggedShape(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("nheads", "headdim", "dstate", "ngroups", "io")]


class _RaggedParams(ctypes.Structure):
    _fields_ = [(n, _VP) for n in ("x", "dt", "B", "C")] + [(n, _LL) for n in ("ldx", "lddt", "ldB", "ldC")] + \
               [(n, _VP) for n in ("A", "D", "dt_bias")]


class _StepShape(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("rows", "n_slots", "nheads", "headdim", "dstate", "ngroups", "d_conv", "io")]


class _FfnShape(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("tokens", "d_model", "d_ff", "activation")]


_P = ctypes.POINTER
lib.ssd_conv.argtypes = [_P(_ConvShape), _P(_Packed), _VP, _LL, _VP, _VP, _P(_Slots), _VP, _LL, _VP, _SZ, _VP]
lib.ssd_conv_bwd_workspace_bytes.argtypes = [_P(_ConvShape), _I]
lib.ssd_conv_bwd_workspace_bytes.restype = _SZ
lib.ssd_conv_bwd.argtypes = [_P(_ConvShape), _P(_Packed), _VP, _LL, _VP, _VP, _VP, _LL, _VP, _LL, _VP, _VP, _VP, _SZ, _VP]
lib.ssd_ragged_workspace_bytes.argtypes = [_P(_RaggedShape), _I, _I]
lib.ssd_ragged_workspace_bytes.restype = _SZ
lib.ssd_scan_ragged.argtypes = [_P(_RaggedShape), _P(_Packed), _P(_RaggedParams), _I, _P(_Slots), _VP, _LL, _VP, _SZ, _VP]
lib.ssd_step_workspace_bytes.argtypes = [_P(_StepShape)]
lib.ssd_step_workspace_bytes.restype = _SZ
lib.mamba2_step.argtypes = [_P(_StepShape), _VP, _LL, _VP, _LL] + [_VP] * 8 + [_VP, _LL, _VP, _SZ, _VP]
lib.ssd_ffn_workspace_bytes.argtypes = lib.ssd_ffn_bwd_workspace_bytes.argtypes = [_P(_FfnShape)]
lib.ssd_ffn_workspace_bytes.restype = lib.ssd_ffn_bwd_workspace_bytes.restype = _SZ
lib.ffn_block.argtypes = [_P(_FfnShape)] + [_VP] * 6 + [_SZ, _VP]
lib.ffn_block_bwd.argtypes = [_P(_FfnShape)] + [_VP] * 9 + [_SZ, _VP]
for _f in (lib.ssd_conv, lib.ssd_conv_bwd, lib.ssd_scan_ragged, lib.mamba2_step, lib.ffn_block, lib.ffn_block_bwd):
    _f.restype = _I

_IO = {torch.bfloat16: 0, torch.float32: 1}


def _call(dev, f, *args):
    """The C call on ``dev``'s current stream, with ``dev`` as the current device."""
    if torch.cuda.current_device() == dev.index:
        _check(f(*args, _stream(dev)))
    else:
        with torch.cuda.device(dev):
            _check(f(*args, _stream(dev)))


def _io_of(t) -> int:
    io = _IO.get(t.dtype)
    if io is None:
        raise TypeError(f"unsupported io dtype {t.dtype} (bfloat16 or float32)")
    return io


def _sizes(*ns):
    """Refuse sizes past the C entry points' ints (ctypes would pass them on modulo 2^32)."""
    if max(ns) > 0x7fffffff:
        raise ValueError(f"sizes {ns}: at most 2^31 - 1 tokens, sequences, channels or slots")


def _cuda(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _f32(name, t, shape, dev):
    """Pointer of a contiguous float32 tensor of this shape (None for None)."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != shape or t.get_device() != dev.index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 of shape {tuple(shape)} on {dev}")
    return t.data_ptr()


def _i32(name, t, n, dev):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.shape != (n,) or t.get_device() != dev.index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 of shape ({n},) on {dev}")
    return t.data_ptr()


def _rows(name, t, batched, lead, tail, dtype, dev):
    """(pointer, elements from one row to the next) of a [tokens, *tail] or [batch, len, *tail] tensor.

    The common case, one token dimension, is told by few tensor calls (a cost of every decoding step); what
    is not it goes through the checks one by one."""
    if not batched and t.dtype is dtype and t.shape == lead + tail and t.get_device() == dev.index:
        st = t.stride()
        if len(st) == 2:
            if st[1] == 1 and st[0] >= tail[0]:
                return t.data_ptr(), st[0]
        elif st[2] == 1 and st[1] == tail[1] and st[0] >= tail[0] * tail[1]:
            return t.data_ptr(), st[0]
    return _rows_checked(name, t, batched, lead, tail, dtype, dev)


def _rows_checked(name, t, batched, lead, tail, dtype, dev):
    if t.dtype is not dtype or t.device != dev:
        raise ValueError(f"{name} must be {dtype} on {dev}")
    if t.shape != lead + tail:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(lead + tail)}")
    if t.numel() == 0:
        return t.data_ptr(), _width(tail)
    st = t.stride()
    want = 1
    for size, s in zip(reversed(t.shape[len(lead):]), reversed(st[len(lead):])):
        if size > 1 and s != want:
            raise ValueError(f"{name}: the elements of a token must be contiguous")
        want *= size
    ld = st[len(lead) - 1] if t.shape[len(lead) - 1] > 1 else (st[0] if batched and t.shape[0] > 1 else want)
    if batched and t.shape[0] > 1 and st[0] != t.shape[1] * ld:
        raise ValueError(f"{name}: the sequences of a batch must lie one behind another")
    if ld < want:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), ld


def _width(tail) -> int:
    w = 1
    for n in tail:
        w *= n
    return w


def _packed(x, tail_dims, cu_seqlens, dev):
    """(packed, has a batch dimension, leading shape) of a call whose main tensor is x."""
    shape = x.shape
    if cu_seqlens is None:
        if len(shape) != tail_dims + 2:
            raise ValueError("without cu_seqlens the tensors need a batch and a token dimension")
        b, n = shape[:2]
        _sizes(b, b * n)
        return _Packed(None, b, b * n), True, shape[:2]
    if len(shape) != tail_dims + 1:
        raise ValueError("with cu_seqlens the tensors have one token dimension and no batch dimension")
    n = cu_seqlens.numel()
    if n < 1:
        raise ValueError("cu_seqlens must be int32 of shape (nseq + 1,)")
    _sizes(n, shape[0])
    return _Packed(_i32("cu_seqlens", cu_seqlens, n, dev), n - 1, shape[0]), False, shape[:1]


def _pool(name, t, tail, dtype, dev):
    if t is None:
        return None, 0
    shape = t.shape
    if t.dtype is not dtype or shape[1:] != tail or len(shape) != len(tail) + 1 or t.get_device() != dev.index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} of shape (slots, {', '.join(map(str, tail))}) on {dev}")
    _sizes(shape[0])
    return t.data_ptr(), shape[0]


def _slots(state_in, state_out, slots_in, slots_out, tail, dtype, nseq, dev):
    if state_in is None and state_out is None:
        if slots_in is not None or slots_out is not None:
            raise ValueError("slots without a state pool")
        return None
    p_in, n_in = _pool("state_in", state_in, tail, dtype, dev)
    p_out, n_out = _pool("state_out", state_out, tail, dtype, dev)
    return ctypes.byref(_Slots(p_in, p_out, _i32("slots_in", slots_in, nseq, dev), _i32("slots_out", slots_out, nseq, dev),
                               n_in, n_out))


_need: dict = {}


def _bytes(f, *key) -> int:
    """Workspace size f(*key) (a pure function of the shape), asked for once per shape."""
    n = _need.get(key)
    if n is None:
        if len(_need) > 4096:
            _need.clear()
        n = _need[key] = max(256, int(f(*key[1:])))
    return n


def _scratch(workspace, need, like):
    """(tensor, pointer, bytes) of the caller's workspace, or of one taken here on ``like``'s device."""
    if workspace is None:
        workspace = like.new_empty(need, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), need
    dev = like.device
    if workspace.device != dev or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel()


def _no_overlap(out, yp, ldy, width, rows, *ins):
    """Refuse an ``out`` that shares elements with an input; ins: (tensor, pointer, row stride, row width).
    Column blocks of one buffer (equal row strides) are told apart."""
    es = out.element_size()
    for t, p, ld, w in ins:
        if t.untyped_storage().data_ptr() != out.untyped_storage().data_ptr() or rows == 0:
            continue
        d = (yp - p) // es
        if d >= (rows - 1) * ld + w or -d >= (rows - 1) * ldy + width:
            continue
        if ld == ldy and d % ld >= w and (-d) % ld >= width:
            continue
        raise ValueError("out overlaps an input")


def _apart(out, *states):
    """Refuse an ``out`` laid over a state that the call reads or writes."""
    for t in states:
        if t is None or t.untyped_storage().data_ptr() != out.untyped_storage().data_ptr() or t.numel() == 0 or out.numel() == 0:
            continue
        last = sum((n - 1) * s for n, s in zip(out.shape, out.stride()))
        if out.data_ptr() < t.data_ptr() + t.numel() * t.element_size() and \
                t.data_ptr() < out.data_ptr() + (last + 1) * out.element_size():
            raise ValueError("out overlaps a state")


def _conv_bwd_bytes(C, K, tokens):
    return lib.ssd_conv_bwd_workspace_bytes(_ConvShape(C, K, 1, 1, 0), tokens)


def _ragged_bytes(H, P, N, G, io, tokens, nseq):
    return lib.ssd_ragged_workspace_bytes(_RaggedShape(H, P, N, G, io), tokens, nseq)


def _step_bytes(R, H, P, N, G, K):
    return lib.ssd_step_workspace_bytes(_StepShape(R, R, H, P, N, G, K, 0))


def ssd_conv(x, w, bias=None, cu_seqlens=None, direction: int = 1, silu: bool = True, state_in=None, state_out=None,
             slots_in=None, slots_out=None, out=None, workspace=None):
    """The depthwise causal convolution (then SiLU): returns y shaped like x.

    x [tokens, channels] with ``cu_seqlens``, or [batch, seqlen, channels]; w float32 [channels, width],
    bias float32 [channels] or None.  States: pools [slots, width - 1, channels] of x's dtype, the last
    inputs in scan order, oldest first; ``slots_in`` / ``slots_out`` int32 [nseq] say where a sequence
    starts from and where it leaves its state (negative: zero / not stored; None: slot i).
    Rows of x in no sequence leave their rows of ``out`` as they were."""
    dev, io = _cuda("x", x), _io_of(x)
    if w.dim() != 2:
        raise ValueError("w must be float32 [channels, width]")
    C, K = w.shape
    _sizes(C, K)
    seq, batched, lead = _packed(x, 1, cu_seqlens, dev)
    xp, ldx = _rows("x", x, batched, lead, (C,), x.dtype, dev)
    y = x.new_empty(x.shape) if out is None else out
    yp, ldy = (y.data_ptr(), C) if out is None else _rows("out", y, batched, lead, (C,), x.dtype, dev)
    if out is not None:
        _no_overlap(out, yp, ldy, C, seq.tokens, (x, xp, ldx, C))
        _apart(out, state_in, state_out)
    slots = _slots(state_in, state_out, slots_in, slots_out, (K - 1, C), x.dtype, seq.nseq, dev)
    ws, wp, wn = (None, None, 0) if workspace is None else _scratch(workspace, 256, x)
    _call(dev, lib.ssd_conv, _ConvShape(C, K, int(direction), int(silu), io), seq, xp, ldx, _f32("w", w, (C, K), dev),
          _f32("bias", bias, (C,), dev), slots, yp, ldy, wp, wn)
    return y


def ssd_conv_bwd(x, w, bias, gy, cu_seqlens=None, direction: int = 1, silu: bool = True, workspace=None) -> dict:
    """Gradients of ssd_conv (zero starting states) for dL/dy = gy: dict of x (x's dtype), w and bias
    (float32; bias None without one).  Rows of x in no sequence have gradient zero."""
    dev, io = _cuda("x", x), _io_of(x)
    if w.dim() != 2:
        raise ValueError("w must be float32 [channels, width]")
    C, K = w.shape
    _sizes(C, K)
    seq, batched, lead = _packed(x, 1, cu_seqlens, dev)
    xp, ldx = _rows("x", x, batched, lead, (C,), x.dtype, dev)
    gp, ldg = _rows("gy", gy, batched, lead, (C,), x.dtype, dev)
    gx = x.new_empty(x.shape)
    gw = torch.empty_like(w, memory_format=torch.contiguous_format)
    gb = torch.empty_like(bias, memory_format=torch.contiguous_format) if bias is not None else None
    shape = _ConvShape(C, K, int(direction), int(silu), io)
    ws, wp, wn = _scratch(workspace, _bytes(_conv_bwd_bytes, "conv", C, K, seq.tokens), x)
    _call(dev, lib.ssd_conv_bwd, shape, seq, xp, ldx, _f32("w", w, (C, K), dev), _f32("bias", bias, (C,), dev), gp, ldg,
          gx.data_ptr(), C, gw.data_ptr(), gb.data_ptr() if gb is not None else None, wp, wn)
    return {"x": gx, "w": gw, "bias": gb}


def ragged_workspace_bytes(tokens: int, nseq: int, nheads: int, headdim: int, dstate: int, ngroups: int = 1,
                           io: torch.dtype = torch.bfloat16) -> int:
    """Workspace size of ssd_scan_ragged (0: refused); it never falls as tokens or sequences grow."""
    _sizes(tokens, nseq)
    return int(lib.ssd_ragged_workspace_bytes(_RaggedShape(nheads, headdim, dstate, ngroups, _IO[io]), tokens, nseq))


def ssd_scan_ragged(x, dt, A, B, C, D=None, cu_seqlens=None, dt_bias=None, direction: int = 1, state_in=None,
                    state_out=None, slots_in=None, slots_out=None, out=None, workspace=None):
    """The scan over packed ragged sequences of any lengths: returns y shaped like x.

    x [tokens, nheads, headdim], dt [tokens, nheads], B and C [tokens, ngroups, dstate] with
    ``cu_seqlens``, or each with [batch, seqlen] in front; A, D, dt_bias float32 [nheads].  ``dt_bias``:
    softplus(dt + dt_bias) is used (None: dt is positive already).  States: float32 pools
    [slots, nheads, headdim, dstate], addressed as in ssd_conv."""
    dev, io = _cuda("x", x), _io_of(x)
    seq, batched, lead = _packed(x, 2, cu_seqlens, dev)
    if B.dim() != x.dim():
        raise ValueError("x must be [..., nheads, headdim] and B, C [..., ngroups, dstate]")
    H, P = x.shape[-2:]
    G, N = B.shape[-2:]
    xp, ldx = _rows("x", x, batched, lead, (H, P), x.dtype, dev)
    dp, ldd = _rows("dt", dt, batched, lead, (H,), x.dtype, dev)
    bp, ldb = _rows("B", B, batched, lead, (G, N), x.dtype, dev)
    cp, ldc = _rows("C", C, batched, lead, (G, N), x.dtype, dev)
    y = x.new_empty(x.shape) if out is None else out
    yp, ldy = (y.data_ptr(), H * P) if out is None else _rows("out", y, batched, lead, (H, P), x.dtype, dev)
    if out is not None:
        _no_overlap(out, yp, ldy, H * P, seq.tokens, (x, xp, ldx, H * P), (dt, dp, ldd, H), (B, bp, ldb, G * N),
                    (C, cp, ldc, G * N))
        _apart(out, state_in, state_out)
    slots = _slots(state_in, state_out, slots_in, slots_out, (H, P, N), torch.float32, seq.nseq, dev)
    shape = _RaggedShape(H, P, N, G, io)
    prm = _RaggedParams(xp, dp, bp, cp, ldx, ldd, ldb, ldc, _f32("A", A, (H,), dev), _f32("D", D, (H,), dev),
                        _f32("dt_bias", dt_bias, (H,), dev))
    ws, wp, wn = _scratch(workspace, _bytes(_ragged_bytes, "ragged", H, P, N, G, io, seq.tokens, seq.nseq), x)
    _call(dev, lib.ssd_scan_ragged, shape, seq, prm, int(direction), slots, yp, ldy, wp, wn)
    return y


def step_workspace_bytes(rows: int, nheads: int, headdim: int, dstate: int, ngroups: int = 1, d_conv: int = 4) -> int:
    """Workspace size of mamba2_step (0: refused)."""
    _sizes(rows)
    return int(lib.ssd_step_workspace_bytes(_StepShape(rows, rows, nheads, headdim, dstate, ngroups, d_conv, 0)))


def mamba2_step(xBC, dt, conv_w, conv_b, dt_bias, A, D, conv_state, ssm_state, slots=None, ngroups: int = 1, out=None,
                workspace=None):
    """One token of the Mamba-2 layer per row: returns y [rows, nheads, headdim] and updates both states in place.

    xBC [rows, nheads*headdim + 2*ngroups*dstate] before the convolution, dt [rows, nheads] before bias and
    softplus (rows any stride apart); conv_w, conv_b, dt_bias, A, D float32 as in mixer_bidir (conv_b, dt_bias
    and D may be None).  conv_state [slots, d_conv - 1, channels] of xBC's dtype, ssm_state float32
    [slots, nheads, headdim, dstate]; ``slots`` int32 [rows] (None: slot r; negative: a padding row, whose
    rows of ``out`` are left as they were)."""
    dev, io = _cuda("xBC", xBC), _io_of(xBC)
    if xBC.dim() != 2 or ssm_state.dim() != 4 or conv_w.dim() != 2:
        raise ValueError("xBC must be [rows, channels], ssm_state [slots, nheads, headdim, dstate], conv_w [channels, d_conv]")
    R, Cc = xBC.shape
    _sizes(R, Cc)
    n, H, P, N = ssm_state.shape
    K = conv_w.shape[1]
    if Cc != H * P + 2 * ngroups * N:
        raise ValueError(f"xBC has {Cc} channels, the states say {H * P + 2 * ngroups * N}")
    dtype, lead = xBC.dtype, xBC.shape[:1]
    xp, ldx = _rows("xBC", xBC, False, lead, (Cc,), dtype, dev)
    dp, ldd = _rows("dt", dt, False, lead, (H,), dtype, dev)
    sp, _ = _pool("ssm_state", ssm_state, (H, P, N), torch.float32, dev)
    vp, nc = _pool("conv_state", conv_state, (K - 1, Cc), dtype, dev)
    if nc != n:
        raise ValueError(f"conv_state has {nc} slots, ssm_state {n}")
    y = xBC.new_empty((R, H, P)) if out is None else out
    yp, ldy = (y.data_ptr(), H * P) if out is None else _rows("out", y, False, lead, (H, P), dtype, dev)
    if out is not None:
        _no_overlap(out, yp, ldy, H * P, R, (xBC, xp, ldx, Cc), (dt, dp, ldd, H))
        _apart(out, conv_state, ssm_state)
    shape = _StepShape(R, n, H, P, N, ngroups, K, io)
    ws, wp, wn = _scratch(workspace, _bytes(_step_bytes, "step", R, H, P, N, ngroups, K), xBC)
    _call(dev, lib.mamba2_step, shape, xp, ldx, dp, ldd, _f32("conv_w", conv_w, (Cc, K), dev), _f32("conv_b", conv_b, (Cc,), dev),
          _f32("dt_bias", dt_bias, (H,), dev), _f32("A", A, (H,), dev), _f32("D", D, (H,), dev), vp, sp,
          _i32("slots", slots, R, dev), yp, ldy, wp, wn)
    return y


_ACT = {"silu": 0, "gelu": 1}


def _ffn_shape(u, W_in, W_out, activation, dev):
    if activation not in _ACT:
        raise ValueError(f"unknown activation {activation!r} (silu or gelu)")
    if W_in.dim() != 2 or W_out.dim() != 2 or u.dim() < 1:
        raise ValueError("u must be [..., d_model], W_in [2 d_ff, d_model], W_out [d_model, d_ff]")
    D, F = W_out.shape
    T = u.numel() // D if D else 0
    _sizes(T, D, F)
    return _FfnShape(T, D, F, _ACT[activation])


def _bf16(name, t, shape, dev):
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != dev.index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous bf16 of shape {tuple(shape)} on {dev}")
    return t.data_ptr()


def ffn_workspace_bytes(tokens: int, d_model: int, d_ff: int) -> int:
    """Workspace size of ffn_block (0: refused)."""
    _sizes(tokens, d_model, d_ff)
    return int(lib.ssd_ffn_workspace_bytes(_FfnShape(tokens, d_model, d_ff, 0)))


def ffn_bwd_workspace_bytes(tokens: int, d_model: int, d_ff: int) -> int:
    """Workspace size of ffn_block_bwd (0: refused)."""
    _sizes(tokens, d_model, d_ff)
    return int(lib.ssd_ffn_bwd_workspace_bytes(_FfnShape(tokens, d_model, d_ff, 0)))


def ffn_block(u, W_in, W_out, activation: str = "silu", save: bool = False, out=None, workspace=None):
    """The gated feed-forward block: out = (act(u Wg^T) * (u Wu^T)) W_out^T, with W_in = [Wg; Wu].

    u [..., d_model] bf16, W_in [2 d_ff, d_model], W_out [d_model, d_ff]; activation "silu" or "gelu".
    ``save``: return (out, gu), gu [..., 2 d_ff] the two projections that ffn_block_bwd needs."""
    dev = _cuda("u", u)
    shape = _ffn_shape(u, W_in, W_out, activation, dev)
    D, F, lead = shape.d_model, shape.d_ff, u.shape[:-1]
    up, wi, wo = _bf16("u", u, lead + (D,), dev), _bf16("W_in", W_in, (2 * F, D), dev), _bf16("W_out", W_out, (D, F), dev)
    y = u.new_empty(u.shape) if out is None else out
    yp = y.data_ptr() if out is None else _bf16("out", y, lead + (D,), dev)
    if out is not None:
        for name, t in (("u", u), ("W_in", W_in), ("W_out", W_out)):
            if yp < t.data_ptr() + 2 * t.numel() and t.data_ptr() < yp + 2 * y.numel():
                raise ValueError(f"out overlaps {name}")
    gu = u.new_empty(lead + (2 * F,)) if save else None
    ws, wp, wn = _scratch(workspace, _bytes(ffn_workspace_bytes, "ffn", shape.tokens, D, F), u)
    _call(dev, lib.ffn_block, shape, up, wi, wo, yp, gu.data_ptr() if save else None, wp, wn)
    return (y, gu) if save else y


def ffn_block_bwd(u, W_in, W_out, gu, gy, activation: str = "silu", workspace=None) -> dict:
    """Gradients of ffn_block for dL/dout = gy, from the saved projections: dict of u, W_in, W_out (bf16)."""
    dev = _cuda("u", u)
    shape = _ffn_shape(u, W_in, W_out, activation, dev)
    D, F, lead = shape.d_model, shape.d_ff, u.shape[:-1]
    ptrs = [_bf16("u", u, lead + (D,), dev), _bf16("W_in", W_in, (2 * F, D), dev), _bf16("W_out", W_out, (D, F), dev),
            _bf16("gu", gu, lead + (2 * F,), dev), _bf16("gy", gy, lead + (D,), dev)]
    g = {"u": torch.empty_like(u), "W_in": torch.empty_like(W_in), "W_out": torch.empty_like(W_out)}
    ws, wp, wn = _scratch(workspace, _bytes(ffn_bwd_workspace_bytes, "ffn bwd", shape.tokens, D, F), u)
    _call(dev, lib.ffn_block_bwd, shape, *ptrs, g["u"].data_ptr(), g["W_in"].data_ptr(), g["W_out"].data_ptr(), wp, wn)
    return g
