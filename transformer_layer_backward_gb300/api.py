"""Python binding of the C ABI: one function per entry point, with the same names.

Each function checks devices, dtypes and contiguity of torch tensors, then passes
raw device pointers to the library.  No arithmetic of the backward pass happens
here; every step runs in the CUDA kernels of ``lib/libtlb.so``.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math

import torch

from . import _abi as A

_WDTYPE = {A.W_F32: torch.float32, A.W_BF16: torch.bfloat16, A.W_TERNARY_I8: torch.int8,
           A.W_TERNARY_2B: torch.uint8}
_WCODE = {"f32": A.W_F32, "bf16": A.W_BF16, "ternary": A.W_TERNARY_I8, "ternary2": A.W_TERNARY_2B}


_NO_GUARD = contextlib.nullcontext()

_STATUS_BYTES = 256     # of a workspace, at its start


def _queued(t, stream=None):
    """Guard for work on t: its device is the current one, and so is the stream that the work is
    queued on, to which what is allocated meanwhile then belongs."""
    if not t.is_cuda:
        return _NO_GUARD
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != t.device:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, t.device))
        return torch.cuda.stream(stream)
    if t.device.index == torch.cuda.current_device():
        return _NO_GUARD
    return torch.cuda.device(t.device)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _ptr(t, dtype=torch.float32, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return C.c_void_p(t.data_ptr()) if t.numel() else None


# ------------------------------------------------------------------ standalone steps

def softmax_backward(attn, dattn, out=None, stream=None):
    """dS = attn * (dAttn - rowsum(attn * dAttn)) over the last axis."""
    out = torch.empty_like(attn) if out is None else out
    rows = attn.numel() // attn.shape[-1] if attn.dim() and attn.shape[-1] else 0
    A.call("tlb_softmax_backward", _ptr(attn, name="attn"), _ptr(dattn, name="dattn"),
           _ptr(out, name="out"), rows, attn.shape[-1] if attn.dim() else 0, _stream(stream))
    return out


def act_backward(act, gate, up, dh, silu_gate=None, dgate=None, dup=None, stream=None):
    """Gated activation backward; act is 'relu2_mul' or 'silu_mul'."""
    code = {"relu2_mul": A.ACT_RELU2_MUL, "silu_mul": A.ACT_SILU_MUL}[act]
    dgate = torch.empty_like(gate) if dgate is None else dgate
    dup = torch.empty_like(gate) if dup is None else dup
    A.call("tlb_act_backward", code, _ptr(gate, name="gate"), _ptr(up, name="up"),
           _ptr(silu_gate, name="silu_gate"), _ptr(dh, name="dh"), _ptr(dgate, name="dgate"),
           _ptr(dup, name="dup"), gate.numel(), _stream(stream))
    return dgate, dup


def rmsnorm_backward(x, gamma, dy, eps=1e-6, out=None, accumulate=False, stream=None):
    """Row-wise RMSNorm backward over the last axis; accumulate adds into out."""
    out = torch.empty_like(x) if out is None else out
    n = x.shape[-1]
    rows = x.numel() // n if n else 0
    A.call("tlb_rmsnorm_backward", _ptr(x, name="x"), _ptr(gamma, name="gamma"),
           _ptr(dy, name="dy"), _ptr(out, name="out"), rows, n, float(eps),
           1 if accumulate else 0, _stream(stream))
    return out


def rope_backward(dy, pos0, base=10000.0, out=None, stream=None):
    """Inverse NeoX rotation of dy [rows, n_heads, head_dim]; row r at position pos0 + r."""
    out = torch.empty_like(dy) if out is None else out
    rows, nh, hd = dy.shape
    A.call("tlb_rope_backward", _ptr(dy, name="dy"), _ptr(out, name="out"), rows, nh, hd,
           int(pos0), float(base), _stream(stream))
    return out


def linear_workspace(wtype, S, out_dim, in_dim, device="cuda"):
    code = _WCODE[wtype]
    n = int(A.load().tlb_linear_workspace_bytes(code, int(S), int(out_dim), int(in_dim)))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def linear_backward(wtype, W, dY, scale=1.0, out=None, accumulate=False, ws=None, stream=None):
    """dX = scale * dY @ W^T for W stored [in, out] (wtype 'f32', 'bf16', 'ternary', or
    'ternary2': uint8 [in, out / 4], four 2-bit codes per byte)."""
    code = _WCODE[wtype]
    in_dim, out_dim = W.shape
    if code == A.W_TERNARY_2B:
        out_dim *= 4
    S = dY.shape[0]
    out = torch.zeros(S, in_dim, dtype=torch.float32, device=dY.device) if out is None else out
    ws = linear_workspace(wtype, S, out_dim, in_dim, dY.device) if ws is None else ws
    A.call("tlb_linear_backward", code, _ptr(W, _WDTYPE[code], "W"), float(scale), _ptr(dY, name="dY"),
           S, out_dim, in_dim, _ptr(out, name="out"), 1 if accumulate else 0,
           _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream))
    return out


def launch_count() -> int:
    return int(A.load().tlb_launch_count())


def launch_names(first: int, last: int | None = None):
    """Names of the library's launches numbered first .. last - 1 (launch_count() values
    taken before and after a call); None where the log no longer holds one."""
    lib = A.load()
    last = launch_count() if last is None else last
    out = []
    for i in range(first, last):
        nm = lib.tlb_launch_name(i)
        out.append(nm.decode() if nm is not None else None)
    return out


def profile_events(events):
    """events[0] (torch.cuda.Event) is recorded at the start of each later layer call and
    events[k + 1] after its k-th kernel; None turns it off.  Returns the ctypes array,
    which must stay alive while in use."""
    lib = A.load()
    if events is None:
        lib.tlb_profile_events(None, 0)
        return None
    for e in events:            # torch creates the CUDA event on its first record
        e.record()
    arr = (C.c_void_p * len(events))(*[C.c_void_p(e.cuda_event) for e in events])
    lib.tlb_profile_events(arr, len(events))
    return arr


def adamw_cfg(lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, lr_b_mult=16.0):
    return A.AdamwCfg(lr, beta1, beta2, eps, weight_decay, lr_b_mult, int(step))


def adamw(p, g, m, v, cfg: A.AdamwCfg, lr_mult=1.0, sumsq=None, stream=None):
    """One AdamW step in place on p, m, v; sumsq (float64 device scalar) += sum(g^2)."""
    A.call("tlb_adamw", _ptr(p, name="p"), _ptr(g, name="g"), _ptr(m, name="m"),
           _ptr(v, name="v"), p.numel(), C.byref(cfg), float(lr_mult),
           _ptr(sumsq, torch.float64, "sumsq"), _stream(stream))


def muon_cfg(lr, momentum=0.95, weight_decay=0.0, eps=1e-7, coefficients=(3.4445, -4.7750, 2.0315), steps=5,
             nesterov=True):
    a, b, c = coefficients
    return A.MuonCfg(lr, momentum, weight_decay, eps, a, b, c, int(steps), 1 if nesterov else 0)


def muon_mats(params, grads, momenta, lr_mults=None, scales=None):
    """The matrices of a Muon step, for muon() and muon_workspace(): equally long lists of
    float32 matrices [rows, cols], min(rows, cols) <= 64.  lr_mults (1) multiply the learning
    rate, scales (sqrt(max(1, rows / cols))) the orthogonal update.  Holds the tensors,
    whose memory must stay where it is (a gradient is written into, not replaced)."""
    n = len(params)
    if not (len(grads) == len(momenta) == n and (lr_mults is None or len(lr_mults) == n)
            and (scales is None or len(scales) == n)):
        raise ValueError("muon_mats: the lists differ in length")
    mats = (A.MuonMat * max(n, 1))()
    for i, (p, g, m) in enumerate(zip(params, grads, momenta)):
        if p.dim() != 2 or g.shape != p.shape or m.shape != p.shape:
            raise ValueError("muon_mats: matrix %d: param, grad and momentum must be matrices of one shape" % i)
        if any(t.device != params[0].device for t in (p, g, m)):
            raise ValueError("muon_mats: matrix %d is on another device" % i)
        rows, cols = p.shape
        mats[i] = A.MuonMat(_ptr(p, name="param"), _ptr(g, name="grad"), _ptr(m, name="momentum"), rows, cols,
                            1.0 if lr_mults is None else float(lr_mults[i]),
                            math.sqrt(max(1.0, rows / max(cols, 1))) if scales is None else float(scales[i]))
    written = [q for mat in mats[:n] for q in (mat.p, mat.m) if q]
    if len(set(written)) != len(written):
        raise ValueError("muon_mats: the same tensor twice")
    if set(written) & {mat.g for mat in mats[:n] if mat.g}:
        raise ValueError("muon_mats: a gradient that is also a param or momentum")
    mats.n, mats.device = n, params[0].device if n else None
    mats.tensors = list(params), list(grads), list(momenta)
    return mats


def muon_workspace(mats, device="cuda"):
    """A zeroed workspace tensor for muon() on these matrices (or on others of their shapes)."""
    n = int(A.load().tlb_muon_workspace_bytes(mats, mats.n))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=mats.device or device)


def muon(mats, cfg: A.MuonCfg, ws, stream=None):
    """One Muon step in place on the params and momenta of muon_mats(): momentum, the update
    made orthogonal by Newton-Schulz steps, weight decay.  The counterpart of adamw()."""
    if mats.device is not None and ws.device != mats.device:
        raise ValueError("ws is on %s, the matrices on %s" % (ws.device, mats.device))
    with _queued(ws, stream):
        A.call("tlb_muon", mats, mats.n, C.byref(cfg), _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream))


# ------------------------------------------------------------------ the loss above the stack

_XENT_CODE = {torch.float32: A.W_F32, torch.bfloat16: A.W_BF16}


def _xent_code(dtype, name):
    if dtype not in _XENT_CODE:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, dtype))
    return _XENT_CODE[dtype]


def _xent_shapes(hidden, W, targets, ws, **per_row):
    if hidden.dim() != 2 or W.dim() != 2 or hidden.shape[1] != W.shape[1]:
        raise ValueError("hidden [rows, dim] and W [vocab, dim] expected, got %s and %s"
                         % (tuple(hidden.shape), tuple(W.shape)))
    rows = hidden.shape[0]
    for name, t in dict(per_row, targets=targets).items():
        if t is not None and tuple(t.shape) != (rows,):
            raise ValueError("%s must have shape (%d,), got %s" % (name, rows, tuple(t.shape)))
    for name, t in dict(per_row, W=W, targets=targets, ws=ws).items():
        if t is not None and t.device != hidden.device:
            raise ValueError("%s is on %s, hidden on %s" % (name, t.device, hidden.device))
    return rows, W.shape[0], W.shape[1]


def xent_workspace(hidden_dtype, weight_dtype, rows, vocab, dim, grad_w=False, device="cuda", grad=True):
    """A workspace tensor, its status block zeroed, for xent_forward and xent_backward (grad_w:
    with the head's gradient) of these sizes; grad=False: for xent_forward alone."""
    sizes = (_xent_code(hidden_dtype, "hidden"), _xent_code(weight_dtype, "W"), int(rows), int(vocab), int(dim))
    n = int(A.load().tlb_xent_workspace_bytes(*sizes, 1 if grad_w else 0) if grad or grad_w else
            A.load().tlb_xent_forward_workspace_bytes(*sizes))
    ws = torch.empty(max(n, _STATUS_BYTES), dtype=torch.uint8, device=device)
    ws[:_STATUS_BYTES].zero_()
    return ws


# Status words of the workspaces that calls made for themselves, by device and stream.
_own_status = {}


def _keep_status(ws):
    """Keeps the status words of a workspace that the caller will not see, for workspace_status().
    (The first call on a stream cannot keep them while it is captured into a graph.)"""
    words = ws[:_STATUS_BYTES].view(torch.int32)
    key = ws.device, torch.cuda.current_stream(ws.device).cuda_stream
    if key in _own_status:
        torch.maximum(_own_status[key], words, out=_own_status[key])
    elif not torch.cuda.is_current_stream_capturing():
        _own_status[key] = words.clone()


def xent_forward(hidden, W, targets, loss=None, lse=None, ws=None, stream=None):
    """Per-row cross entropy of the linear head W [vocab, dim] on hidden [rows, dim], without
    the logits: (loss, lse).  Targets (int64) outside [0, vocab) mark rows without one.
    Without ws the call makes one of its own, which workspace_status() without one looks after."""
    rows, vocab, dim = _xent_shapes(hidden, W, targets, ws, loss=loss, lse=lse)
    ht, wt = _xent_code(hidden.dtype, "hidden"), _xent_code(W.dtype, "W")
    with _queued(hidden, stream):
        loss = torch.empty(rows, dtype=torch.float32, device=hidden.device) if loss is None else loss
        lse = torch.empty(rows, dtype=torch.float32, device=hidden.device) if lse is None else lse
        own = ws is None
        if own:
            ws = xent_workspace(hidden.dtype, W.dtype, rows, vocab, dim, device=hidden.device, grad=False)
        A.call("tlb_xent_forward", ht, _ptr(hidden, None, "hidden"), wt, _ptr(W, None, "W"),
               _ptr(targets, torch.int64, "targets"), rows, vocab, dim, _ptr(loss, name="loss"), _ptr(lse, name="lse"),
               _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream))
        if own:
            _keep_status(ws)
    return loss, lse


def xent_backward(hidden, W, targets, lse, d_loss, d_hidden=None, d_w=None, grad_w=False, ws=None, stream=None):
    """Gradient of sum(d_loss * loss): (d_hidden, d_w), in hidden's dtype; d_w [vocab, dim] is
    None unless grad_w is set or a tensor for it is given.  lse as xent_forward returned it; ws
    as there."""
    rows, vocab, dim = _xent_shapes(hidden, W, targets, ws, lse=lse, d_loss=d_loss)
    ht, wt = _xent_code(hidden.dtype, "hidden"), _xent_code(W.dtype, "W")
    with _queued(hidden, stream):
        d_hidden = torch.empty_like(hidden) if d_hidden is None else d_hidden
        if d_w is None and grad_w:
            d_w = torch.empty(vocab, dim, dtype=hidden.dtype, device=hidden.device)
        for name, t, shape in (("d_hidden", d_hidden, hidden.shape), ("d_w", d_w, W.shape)):
            if t is not None and (t.shape != shape or t.device != hidden.device):
                raise ValueError("%s must have shape %s on %s" % (name, tuple(shape), hidden.device))
        own = ws is None
        if own:
            ws = xent_workspace(hidden.dtype, W.dtype, rows, vocab, dim, d_w is not None, hidden.device)
        A.call("tlb_xent_backward", ht, _ptr(hidden, None, "hidden"), wt, _ptr(W, None, "W"),
               _ptr(targets, torch.int64, "targets"), _ptr(lse, name="lse"), _ptr(d_loss, name="d_loss"), rows, vocab,
               dim, _ptr(d_hidden, hidden.dtype, "d_hidden"), _ptr(d_w, hidden.dtype, "d_w"),
               _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream))
        if own:
            _keep_status(ws)
    return d_hidden, d_w


# ------------------------------------------------------------------ 8-bit blocks

_FP8_BLOCK = 128
_E4M3 = torch.float8_e4m3fn


def _raw_stream(stream, device):
    """The stream's address, the current one of the device where none is given (a guard of _queued() set it)."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _int32(n, name):
    """n for a 32-bit argument, of which ctypes would pass the low 32 bits."""
    n = int(n)
    if not -1 << 31 <= n < 1 << 31:
        raise ValueError("%s does not fit 32 bits: %d" % (name, n))
    return n


def _at(t, shape, dtype, device, name):
    """Address of a contiguous tensor of this shape (None: any), type and device."""
    if t.dtype is dtype and t.is_contiguous() and t.device == device and (shape is None or t.shape == shape) and t.is_cuda:
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s is on %s, expected on %s" % (name, t.device, device))
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _status_cleared(n, device):
    """A workspace of n bytes, its status block zeroed."""
    ws = torch.empty(max(n, _STATUS_BYTES), dtype=torch.uint8, device=device)
    ws[:_STATUS_BYTES].zero_()
    return ws


def fp8_quantize(x, block_rows=1, q=None, scales=None, stream=None):
    """x [rows, cols] (float32 or bfloat16) in 8-bit blocks of block_rows (1, or 128 for weights) x 128
    columns: (q, scales), q float8_e4m3fn [rows, cols] and scales float32 [ceil(rows / block_rows),
    ceil(cols / 128)], powers of two.  x is about q * scales."""
    code = _xent_code(x.dtype, "x")
    if x.dim() != 2:
        raise ValueError("x [rows, cols] expected, got %s" % (tuple(x.shape),))
    rows, cols = x.shape
    block_rows = _int32(block_rows, "block_rows")
    blocks = (-(-rows // max(block_rows, 1)), -(-cols // _FP8_BLOCK))
    with _queued(x, stream):
        at_x = _at(x, None, x.dtype, x.device, "x")
        if q is None:
            q = torch.empty((rows, cols), dtype=_E4M3, device=x.device)
        else:
            _at(q, x.shape, _E4M3, x.device, "q")
        if scales is None:
            scales = torch.empty(blocks, dtype=torch.float32, device=x.device)
        else:
            _at(scales, blocks, torch.float32, x.device, "scales")
        A.call("tlb_fp8_quantize", code, at_x, rows, cols, block_rows, q.data_ptr(), scales.data_ptr(),
               _raw_stream(stream, x.device))
    return q, scales


def linear_fp8_workspace(S, out_dim, in_dim, device="cuda"):
    """A workspace tensor, its status block zeroed, for linear_fp8_backward of these sizes."""
    return _status_cleared(int(A.load().tlb_linear_fp8_workspace_bytes(int(S), int(out_dim), int(in_dim))), device)


def linear_fp8_backward(W, w_scales, dY, dy_scales, out=None, accumulate=False, dtype=torch.float32, ws=None, stream=None):
    """dX = dY @ W^T [S, in] of fp8_quantize()d dY [S, out] (block_rows 1) and W [in, out] (block_rows 128),
    in dtype (float32 or bfloat16; that of out where it is given); accumulate adds into out.
    Without ws the call makes one of its own, which workspace_status() without one looks after."""
    if W.dim() != 2 or dY.dim() != 2 or W.shape[1] != dY.shape[1]:
        raise ValueError("W [in, out] and dY [S, out] expected, got %s and %s" % (tuple(W.shape), tuple(dY.shape)))
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    (in_dim, out_dim), S, dev = W.shape, dY.shape[0], W.device
    dtype = dtype if out is None else out.dtype
    code = _xent_code(dtype, "out")
    columns = -(-out_dim // _FP8_BLOCK)
    with _queued(W, stream):
        if out is None:
            out = torch.empty((S, in_dim), dtype=dtype, device=dev)
        else:
            _at(out, (S, in_dim), dtype, dev, "out")
        own = ws is None
        if own:
            ws = linear_fp8_workspace(S, out_dim, in_dim, dev)
        A.call("tlb_linear_fp8_backward", _at(W, None, _E4M3, dev, "W"),
               _at(w_scales, (-(-in_dim // _FP8_BLOCK), columns), torch.float32, dev, "w_scales"),
               _at(dY, None, _E4M3, dev, "dY"), _at(dy_scales, (S, columns), torch.float32, dev, "dy_scales"), S, out_dim, in_dim,
               code, out.data_ptr(), 1 if accumulate else 0,
               _at(ws, None, torch.uint8, dev, "ws"), ws.numel(), _raw_stream(stream, dev))
        if own:
            _keep_status(ws)
    return out


def kv8_cache(n_slots, n_kv_heads, head_dim, device="cuda"):
    """An 8-bit K/V cache of n_slots positions, all 0, for kv8_write, kv8_read and kv8_attn_*."""
    rows = [torch.zeros(n_slots, n_kv_heads, head_dim, dtype=torch.uint8, device=device).view(_E4M3) for _ in range(2)]
    scales = [torch.zeros(n_kv_heads, n_slots, dtype=torch.float32, device=device) for _ in range(2)]
    return kv8_cache_of(rows[0], scales[0], rows[1], scales[1])


def kv8_cache_of(k, k_scale, v, v_scale):
    """An 8-bit K/V cache in these tensors: k, v float8_e4m3fn [n_slots, n_kv_heads, head_dim], k_scale, v_scale
    float32 [n_kv_heads, n_slots].  Holds them (as .k, .k_scale, .v, .v_scale); their memory must stay where it is."""
    if k.dim() != 3:
        raise ValueError("k [n_slots, n_kv_heads, head_dim] expected, got %s" % (tuple(k.shape),))
    n_slots, n_kv, hd = k.shape
    at = (_at(k, None, _E4M3, k.device, "k"), _at(v, k.shape, _E4M3, k.device, "v"),
          _at(k_scale, (n_kv, n_slots), torch.float32, k.device, "k_scale"),
          _at(v_scale, (n_kv, n_slots), torch.float32, k.device, "v_scale"))
    cache = A.Kv8(*at, n_slots, n_kv, hd)
    cache.tensors = k, k_scale, v, v_scale
    cache.device = k.device
    return cache


def kv8_write(cache, k, v, slots, stream=None):
    """Quantises new rows k, v [rows, n_kv_heads, head_dim] (float32 or bfloat16; head_dim dense, other strides any)
    into slots (int64 [rows], distinct; those outside the cache, such as -1, are skipped)."""
    rows = slots.numel()
    code = _xent_code(k.dtype, "k")
    for name, t in (("k", k), ("v", v)):
        if t.shape != (rows, cache.n_kv_heads, cache.head_dim) or t.dtype != k.dtype or t.device != cache.device:
            raise ValueError("%s must be %s [%d, %d, %d] on %s" % (name, k.dtype, rows, cache.n_kv_heads, cache.head_dim,
                                                                 cache.device))
        if t.numel() and t.stride(2) != 1:
            raise ValueError("%s: the values of a head must be dense" % name)
    with _queued(k, stream):
        A.call("tlb_kv8_write", cache, code, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
               _at(slots, (rows,), torch.int64, cache.device, "slots"), rows, _raw_stream(stream, cache.device))


def kv8_read(cache, slots, dtype=torch.float32, kv_layout="shd", k=None, v=None, stream=None):
    """The keys and values of slots (int64 [rows]; 0 for those outside the cache) as (k, v) in dtype: [rows, n_kv_heads,
    head_dim] for kv_layout 'shd', [n_kv_heads, rows, head_dim] for 'hsd', the layouts that layer_acts() takes."""
    rows, n_kv, hd = slots.numel(), cache.n_kv_heads, cache.head_dim
    if kv_layout not in ("shd", "hsd"):
        raise ValueError("kv_layout must be 'shd' or 'hsd', got %r" % (kv_layout,))
    if (k is None) != (v is None):
        raise ValueError("k and v are given together or not at all")
    shape = (rows, n_kv, hd) if kv_layout == "shd" else (n_kv, rows, hd)
    dtype = dtype if k is None else k.dtype
    code = _xent_code(dtype, "k")
    with _queued(slots, stream):
        if k is None:
            k, v = (torch.empty(shape, dtype=dtype, device=cache.device) for _ in range(2))
        else:
            _at(k, shape, dtype, cache.device, "k")
            _at(v, shape, dtype, cache.device, "v")
        strides = (n_kv * hd, hd) if kv_layout == "shd" else (hd, rows * hd)
        A.call("tlb_kv8_read", cache, _at(slots, (rows,), torch.int64, cache.device, "slots"), rows, code, k.data_ptr(),
               v.data_ptr(), *strides, _raw_stream(stream, cache.device))
    return k, v


def kv8_attn_workspace(cache, n_seq, n_heads, max_len, grad=False):
    """A workspace tensor, its status block zeroed, for kv8_attn_forward and, with grad, kv8_attn_backward."""
    n = A.load().tlb_kv8_attn_workspace_bytes(cache, int(n_seq), int(n_heads), int(max_len), 1 if grad else 0)
    return _status_cleared(int(n), cache.device)


def _kv8_over(cache, q, pages, page, lengths):
    page = _int32(page, "page")
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q [n_seq, n_heads, %d] expected, got %s" % (cache.head_dim, tuple(q.shape)))
    n_seq, n_heads = q.shape[:2]
    if pages.dim() != 2 or pages.shape[0] != n_seq:
        raise ValueError("pages [%d, max_pages] expected, got %s" % (n_seq, tuple(pages.shape)))
    return (n_seq, n_heads, _xent_code(q.dtype, "q"), _at(q, None, q.dtype, cache.device, "q"),
            _at(pages, None, torch.int32, cache.device, "pages"), pages.shape[1], page,
            _at(lengths, (n_seq,), torch.int32, cache.device, "lengths"))


def kv8_attn_forward(cache, q, pages, page, lengths, max_len, scale=None, ctx=None, lse=None, ws=None, stream=None):
    """Attention of one query row q [n_seq, n_heads, head_dim] for each sequence over the 8-bit cache: (ctx, lse).
    Key j < lengths[b] (int32 [n_seq]) of sequence b is in slot pages[b, j // page] * page + j % page (pages int32
    [n_seq, max_pages]); max_len is at least the longest length; scale 1 / sqrt(head_dim) unless given.
    Without ws the call makes one of its own, which workspace_status() without one looks after."""
    n_seq, n_heads, code, at_q, at_pages, max_pages, page, at_lengths = _kv8_over(cache, q, pages, page, lengths)
    dev = cache.device
    with _queued(q, stream):
        if ctx is None:
            ctx = torch.empty_like(q)
        else:
            _at(ctx, q.shape, q.dtype, dev, "ctx")
        if lse is None:
            lse = torch.empty((n_seq, n_heads), dtype=torch.float32, device=dev)
        else:
            _at(lse, (n_seq, n_heads), torch.float32, dev, "lse")
        own = ws is None
        if own:
            ws = kv8_attn_workspace(cache, n_seq, n_heads, max_len)
        A.call("tlb_kv8_attn_forward", cache, at_pages, max_pages, page, at_lengths, n_seq, int(max_len), n_heads,
               1.0 / math.sqrt(cache.head_dim) if scale is None else float(scale), code, at_q,
               ctx.data_ptr(), lse.data_ptr(), _at(ws, None, torch.uint8, dev, "ws"), ws.numel(), _raw_stream(stream, dev))
        if own:
            _keep_status(ws)
    return ctx, lse


def kv8_attn_backward(cache, q, pages, page, lengths, max_len, lse, d_ctx, scale=None, d_q=None, d_k=None, d_v=None, ws=None,
                      stream=None):
    """Gradient of kv8_attn_forward() for d_ctx: (d_q, d_k, d_v) in q's dtype, d_k and d_v [n_seq, n_kv_heads, head_dim]
    of each sequence's newest key and value.  lse as kv8_attn_forward returned it; ws as there."""
    n_seq, n_heads, code, at_q, at_pages, max_pages, page, at_lengths = _kv8_over(cache, q, pages, page, lengths)
    dev, newest = cache.device, (n_seq, cache.n_kv_heads, cache.head_dim)
    with _queued(q, stream):
        if d_q is None:
            d_q = torch.empty_like(q)
        else:
            _at(d_q, q.shape, q.dtype, dev, "d_q")
        if d_k is None:
            d_k = torch.empty(newest, dtype=q.dtype, device=dev)
        else:
            _at(d_k, newest, q.dtype, dev, "d_k")
        if d_v is None:
            d_v = torch.empty(newest, dtype=q.dtype, device=dev)
        else:
            _at(d_v, newest, q.dtype, dev, "d_v")
        own = ws is None
        if own:
            ws = kv8_attn_workspace(cache, n_seq, n_heads, max_len, grad=True)
        A.call("tlb_kv8_attn_backward", cache, at_pages, max_pages, page, at_lengths, n_seq, int(max_len), n_heads,
               1.0 / math.sqrt(cache.head_dim) if scale is None else float(scale), code, at_q,
               _at(lse, (n_seq, n_heads), torch.float32, dev, "lse"), _at(d_ctx, q.shape, q.dtype, dev, "d_ctx"),
               d_q.data_ptr(), d_k.data_ptr(), d_v.data_ptr(), _at(ws, None, torch.uint8, dev, "ws"), ws.numel(), _raw_stream(stream, dev))
        if own:
            _keep_status(ws)
    return d_q, d_k, d_v


# ------------------------------------------------------------------ layer pieces

def layer_cfg(dim, ffn_dim, n_heads, n_kv_heads, head_dim, rank, lora_alpha, act="relu2_mul",
              wtype="f32", sub_norm=False, pre_norm=False, residual=True, rope=True,
              use_silu_cache=False, causal=True, rope_base=10000.0, norm_eps=1e-6,
              attn_scale=None, persistent=False, qk_norm=False, check_finite=False,
              exact_din=False, recompute_p=False) -> A.LayerCfg:
    flags = ((A.SUB_NORM if sub_norm else 0) | (A.PRE_NORM if pre_norm else 0) |
             (A.RESIDUAL if residual else 0) | (A.ROPE if rope else 0) |
             (A.USE_SILU_CACHE if use_silu_cache else 0) | (A.CAUSAL if causal else 0) |
             (A.PERSISTENT if persistent else 0) | (A.QK_NORM if qk_norm else 0) |
             (A.CHECK_FINITE if check_finite else 0) | (A.EXACT_DIN if exact_din else 0) |
             (A.RECOMPUTE_P if recompute_p else 0))
    return A.LayerCfg(dim, ffn_dim, n_heads, n_kv_heads, head_dim, rank, float(lora_alpha),
                      float(rope_base), float(norm_eps),
                      float(1.0 / math.sqrt(head_dim) if attn_scale is None else attn_scale),
                      {"relu2_mul": A.ACT_RELU2_MUL, "silu_mul": A.ACT_SILU_MUL}[act],
                      _WCODE[wtype], flags)


def layer_cfg_of(c, persistent=False, check_finite=False) -> A.LayerCfg:
    """The layer struct for any object with the attributes of a layer configuration
    (dim, ffn_dim, n_heads, n_kv_heads, head_dim, rank, lora_alpha, act, wtype, sub_norm,
    pre_norm, residual, rope, use_silu_cache, rope_base, norm_eps, attn_scale, qk_norm);
    the attention is causal."""
    return layer_cfg(c.dim, c.ffn_dim, c.n_heads, c.n_kv_heads, c.head_dim, c.rank, c.lora_alpha,
                     act=c.act, wtype=c.wtype, sub_norm=c.sub_norm, pre_norm=c.pre_norm,
                     residual=c.residual, rope=c.rope,
                     use_silu_cache=(c.act == "silu_mul" and c.use_silu_cache), causal=True,
                     rope_base=c.rope_base, norm_eps=c.norm_eps, attn_scale=c.attn_scale,
                     persistent=persistent, qk_norm=c.qk_norm, check_finite=check_finite,
                     exact_din=getattr(c, "exact_din", False), recompute_p=getattr(c, "recompute_p", False))


def adamw_cfg_of(c) -> A.AdamwCfg:
    """The AdamW struct for an object with lr, beta1, beta2, adam_eps, weight_decay, step
    and lr_b_mult attributes."""
    return adamw_cfg(c.lr, c.beta1, c.beta2, c.adam_eps, c.weight_decay, c.step, c.lr_b_mult)


def workspace_bytes(cfg: A.LayerCfg, S: int, L: int) -> int:
    return int(A.load().tlb_workspace_bytes(C.byref(cfg), int(S), int(L)))


def workspace(cfg: A.LayerCfg, S: int, L: int, device="cuda"):
    """A zeroed workspace tensor of the size the library asks for."""
    return torch.zeros(max(workspace_bytes(cfg, S, L), 256), dtype=torch.uint8, device=device)


def debug_skip_barrier_arrival(block: int):
    """Test hook of the device-side timeout path (see tlb_debug_skip_barrier_arrival)."""
    A.call("tlb_debug_skip_barrier_arrival", int(block))


def workspace_status(ws=None, stream=None):
    """Raises TlbError for an error that a kernel recorded in ws, and clears it (waits for the
    stream).  Without ws: for errors of calls that made a workspace of their own, on any stream
    (waits for their devices)."""
    if ws is not None:
        A.call("tlb_workspace_status", _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream))
        return
    failed = None
    for (device, _), words in _own_status.items():
        with torch.cuda.device(device):
            torch.cuda.synchronize()
            try:
                A.call("tlb_workspace_status", _ptr(words, torch.int32, "status"), _STATUS_BYTES, _stream(stream))
            except A.TlbError as e:
                failed = failed or e
    if failed is not None:
        raise failed


def layer_weights(cfg: A.LayerCfg, t: dict):
    """Weights from a dict: w_down/w_gate/w_up/w_o (+ s_* scales); the gains g_sub_ffn,
    g_ffn, g_sub_attn, g_q are optional, and so are w_q/w_k/w_v, g_attn, g_k (the exact
    layer-input gradient)."""
    wd = _WDTYPE[cfg.wtype]

    def w(name):
        if name not in t:
            return A.Weight(None, 1.0)
        return A.Weight(_ptr(t[name], wd, name), float(t.get("s_" + name[2:], 1.0)))

    return A.LayerWeights(w("w_down"), w("w_gate"), w("w_up"), w("w_o"),
                          _ptr(t.get("g_sub_ffn"), name="g_sub_ffn"),
                          _ptr(t.get("g_ffn"), name="g_ffn"),
                          _ptr(t.get("g_sub_attn"), name="g_sub_attn"),
                          _ptr(t.get("g_q"), name="g_q"),
                          w("w_q"), w("w_k"), w("w_v"),
                          _ptr(t.get("g_attn"), name="g_attn"), _ptr(t.get("g_k"), name="g_k"))


def layer_acts(cfg: A.LayerCfg, t: dict, kv_layout: str, L: int):
    """Cached activations from a dict; kv_layout 'shd' = [L, kv_dim], 'hsd' = [n_kv, L, hd]."""
    hd = cfg.head_dim
    if kv_layout == "shd":
        sh, sp = hd, cfg.n_kv_heads * hd
    else:
        sh, sp = L * hd, hd
    g = lambda k: _ptr(t.get(k), name=k)
    return A.LayerActs(g("x"), g("gate"), g("up"), g("silu_gate"), g("hidden"), g("r1"),
                       g("ctx"), g("k"), g("v"), sh, sp, g("attn"), g("lora_q_h"), g("lora_v_h"),
                       g("q_raw"), g("x_in"), g("q"), g("k_raw"), g("lse"))


def lora(t: dict, tag: str, grads: dict | None = None):
    g = grads or {}
    p = lambda k: _ptr(t[k], name=k)
    return A.Lora(p("a_" + tag), p("b_" + tag), p("m_a_" + tag), p("v_a_" + tag),
                  p("m_b_" + tag), p("v_b_" + tag),
                  _ptr(g.get("dA_" + tag), name="dA"), _ptr(g.get("dB_" + tag), name="dB"))


def ffn_backward(cfg, S, d_out, weights, acts, d_residual, ws, stream=None):
    A.call("tlb_ffn_backward", C.byref(cfg), int(S), _ptr(d_out, name="d_out"), C.byref(weights),
           C.byref(acts), _ptr(d_residual, name="d_residual"), _ptr(ws, torch.uint8, "ws"),
           ws.numel(), _stream(stream))


def attn_backward(cfg, S, L, d_attn_out, weights, acts, d_qpre, d_v, ws, stream=None):
    A.call("tlb_attn_backward", C.byref(cfg), int(S), int(L), _ptr(d_attn_out, name="d_attn_out"),
           C.byref(weights), C.byref(acts), _ptr(d_qpre, name="d_qpre"), _ptr(d_v, name="d_v"),
           _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream))


def lora_grad_adamw(S, out_dim, in_dim, rank, alpha, G, h, x, lora_: A.Lora, adam: A.AdamwCfg,
                    sumsq, ws, stream=None):
    A.call("tlb_lora_grad_adamw", int(S), int(out_dim), int(in_dim), int(rank), float(alpha),
           _ptr(G, name="G"), _ptr(h, name="h"), _ptr(x, name="x"), C.byref(lora_), C.byref(adam),
           _ptr(sumsq, torch.float64, "sumsq"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
           _stream(stream))


def lora_grad_adamw_noalloc(S, out_dim, in_dim, rank, alpha, G, h, x, lora_: A.Lora, adam: A.AdamwCfg,
                            sumsq, stream=None):
    """lora_grad_adamw without a workspace: for callers that cannot allocate device memory.
    Its scratch is a fixed array inside the library (S * rank <= 65536); calls sharing it
    must not overlap on the GPU."""
    A.call("tlb_lora_grad_adamw_noalloc", int(S), int(out_dim), int(in_dim), int(rank), float(alpha),
           _ptr(G, name="G"), _ptr(h, name="h"), _ptr(x, name="x"), C.byref(lora_), C.byref(adam),
           _ptr(sumsq, torch.float64, "sumsq"), _stream(stream))


def layer_backward(cfg, S, L, weights, acts, lora_q, lora_v, adam, d_hidden, sumsq, ws, stream=None):
    A.call("tlb_layer_backward", C.byref(cfg), int(S), int(L), C.byref(weights), C.byref(acts),
           C.byref(lora_q), C.byref(lora_v), C.byref(adam), _ptr(d_hidden, name="d_hidden"),
           _ptr(sumsq, torch.float64, "sumsq"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
           _stream(stream))


def stack_workspace(cfg: A.LayerCfg, S: int, L: int, device="cuda"):
    """A zeroed workspace tensor for stack_backward."""
    n = int(A.load().tlb_stack_workspace_bytes(C.byref(cfg), int(S), int(L)))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def stack_backward(cfg, S, L, weights, acts, lora_q, lora_v, adam, d_hidden, sumsq, ws, stream=None):
    """Layers len(weights) - 1 .. 0 of a stack (entry l of each list is layer l); d_hidden
    holds the top layer's dOut on entry and layer 0's d_in on return."""
    n = len(weights)
    if not (len(acts) == len(lora_q) == len(lora_v) == n):
        raise ValueError("stack_backward: the four layer lists differ in length")
    W = (A.LayerWeights * max(n, 1))(*weights)
    X = (A.LayerActs * max(n, 1))(*acts)
    Q = (A.Lora * max(n, 1))(*lora_q)
    V = (A.Lora * max(n, 1))(*lora_v)
    A.call("tlb_stack_backward", C.byref(cfg), int(S), int(L), n, W, X, Q, V, C.byref(adam),
           _ptr(d_hidden, name="d_hidden"), _ptr(sumsq, torch.float64, "sumsq"), _ptr(ws, torch.uint8, "ws"),
           ws.numel(), _stream(stream))
