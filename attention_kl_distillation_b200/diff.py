"""Differential attention and paged single-token attention (the second part of include/streamkl.h).

    O = (softmax(s1 Q1 K1^T) - lam softmax(s2 Q2 K2^T)) V

``diff_attn`` is the autograd entry point, ``diff_attn_fwd`` and ``diff_attn_bwd`` its two halves,
``diff_attn_paged`` its form for one new token over paged caches, ``attn_paged`` the same with one
softmax map, ``paged_write`` puts new tokens' rows into the caches.

As in ``binding``, this is argument marshalling only: tensors are checked for dtype, device, shape and
layout, and every step of the computation runs in the library's kernels on the current stream.
Tensors are bf16 or fp16 (one type for all of a call), with contiguous features; the other axes may
have any positive strides that are multiples of 8 elements, so a projection's [B, N, H, d] output
passes as ``.transpose(1, 2)`` without a copy.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import EINVAL, OK, StreamKLError, _lib, _stream, _vp

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class _Tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("b", ctypes.c_int64), ("h", ctypes.c_int64),
                ("n", ctypes.c_int64)]


class DiffProblem(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int) for k in ("B", "H", "HK", "NQ", "NK", "d", "dv", "causal", "dtype",
                                            "lam_fp32")] + [("s1", ctypes.c_float), ("s2", ctypes.c_float)]


class PagedProblem(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int) for k in ("B", "H", "HK", "d", "dv", "dtype", "lam_fp32", "pages",
                                            "page_size", "max_pages")] + [("s1", ctypes.c_float),
                                                                          ("s2", ctypes.c_float)]


_tp = ctypes.POINTER(_Tensor)
_dp = ctypes.POINTER(DiffProblem)
_gp = ctypes.POINTER(PagedProblem)
_lib.streamkl_diff_fwd.argtypes = [_dp] + [_tp] * 6 + [_vp] * 2 + [_tp] * 2 + [_vp] * 3
_lib.streamkl_diff_fwd.restype = ctypes.c_int
_lib.streamkl_diff_bwd_workspace_size.argtypes = [_dp]
_lib.streamkl_diff_bwd_workspace_size.restype = ctypes.c_size_t
_lib.streamkl_diff_bwd.argtypes = [_dp] + [_tp] * 9 + [_vp] * 4 + [_tp] * 5 + [_vp] * 2 + [ctypes.c_size_t, _vp]
_lib.streamkl_diff_bwd.restype = ctypes.c_int
_lib.streamkl_paged_workspace_size.argtypes = [_gp, ctypes.c_int]
_lib.streamkl_paged_workspace_size.restype = ctypes.c_size_t
_lib.streamkl_paged_attn.argtypes = [_gp] + [_tp] * 6 + [_vp, ctypes.c_int64, _vp, _tp, _vp, ctypes.c_size_t, _vp]
_lib.streamkl_paged_attn.restype = ctypes.c_int
_lib.streamkl_paged_write.argtypes = [ctypes.c_int, _tp, _tp, ctypes.POINTER(ctypes.c_int), _vp] + \
    [ctypes.c_int] * 5 + [_vp]
_lib.streamkl_paged_write.restype = ctypes.c_int


def _ptr(t):
    return _vp(t.data_ptr()) if t is not None else None


def _layout_ok(t) -> bool:
    """Contiguous features, 16-byte aligned, outer strides positive multiples of 8 elements."""
    return (t.data_ptr() % 16 == 0 and (t.shape[-1] == 1 or t.stride(-1) == 1)
            and all(n == 1 or (s > 0 and s % 8 == 0) for n, s in zip(t.shape[:-1], t.stride()[:-1])))


def _check(name, t, shape, like, what):
    """One 16-bit operand: its shape (None matches anything), type, device and layout."""
    if not isinstance(t, torch.Tensor) or t.dim() != len(shape) or \
            any(want is not None and want != got for want, got in zip(shape, t.shape)):
        raise ValueError(f"{name} must be a tensor {what}")
    if t.dtype not in _DTYPES or t.dtype != like.dtype:
        raise ValueError(f"{name} must be bf16 or fp16, the same type as the other operands")
    if t.device != like.device:
        raise ValueError("tensors must be on one device")
    if t.numel() and not _layout_ok(t):
        raise ValueError(f"{name} must have contiguous features, 16-byte alignment and outer strides "
                         "that are positive multiples of 8 elements")


def _check_out(name, t, ref_shape, like):
    """A caller's output: as an operand, and no two of its elements in one place."""
    _check(name, t, tuple(ref_shape), like, f"of shape {tuple(ref_shape)}")
    need = 1
    for n, s in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n > 1), key=lambda p: p[1]):
        if s < need:
            raise ValueError(f"{name} must not overlap itself")
        need = s * n


def _check_cuda(t):
    if not t.is_cuda:
        raise ValueError("inputs must be CUDA tensors")


def _check_lens(name, t, B, like):
    if t is not None and (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.shape != (B,)
                          or not t.is_contiguous() or t.device != like.device):
        raise ValueError(f"{name} must be a contiguous int32 tensor [B] on the inputs' device")


def _check_lam(lam, extents, like):
    """lam as a tensor with one axis per extent, broadcast axes of stride 0."""
    names = "[H], [B, H, N]" if len(extents) == 3 else "[H], [B, H]"
    if not isinstance(lam, torch.Tensor) or lam.dtype not in (like.dtype, torch.float32) or \
            lam.device != like.device:
        raise ValueError("lam must be a tensor of the inputs' type or fp32 on their device")
    if lam.dim() == 0:
        shape = (1,) * len(extents)
    elif lam.dim() == 1:
        shape = (1, lam.shape[0]) + (1,) * (len(extents) - 2)
    else:
        shape = tuple(lam.shape)
    if len(shape) != len(extents) or any(n not in (1, e) for n, e in zip(shape, extents)):
        raise ValueError(f"lam must be a scalar or {names} (extents of 1 broadcast)")
    view = lam.reshape(shape)
    if any(n > 1 and s <= 0 for n, s in zip(view.shape, view.stride())):
        view = view.contiguous()
    return view


def _tensor(t):
    """The streamkl_tensor of [.., .., .., width] (or, with fewer axes, of the leading ones)."""
    if t is None:
        return None
    st = t.stride()
    return ctypes.byref(_Tensor(t.data_ptr(), *(st[k] if k < t.dim() - 1 else 0 for k in range(3))))


def _lam_tensor(view):
    st = [s if n > 1 else 0 for n, s in zip(view.shape, view.stride())]
    return ctypes.byref(_Tensor(view.data_ptr(), *(st + [0])[:3]))


def _scale(s):
    return float(s) if s is not None else 0.0


def _check_diff(Q1, K1, Q2, K2, V, lam, q_lens, k_lens):
    if not isinstance(Q1, torch.Tensor) or Q1.dim() != 4:
        raise ValueError("Q1 must be a tensor [B, H, NQ, d]")
    B, H, NQ, d = Q1.shape
    _check("Q1", Q1, (B, H, NQ, d), Q1, "[B, H, NQ, d]")
    _check("Q2", Q2, (B, H, NQ, d), Q1, "[B, H, NQ, d], as Q1")
    _check("K1", K1, (B, None, None, d), Q1, "[B, HK, NK, d]")
    HK, NK = K1.shape[1:3]
    _check("K2", K2, (B, HK, NK, d), Q1, "[B, HK, NK, d], as K1")
    _check("V", V, (B, HK, NK, None), Q1, "[B, HK, NK, dv]")
    if (HK == 0) != (H == 0) or (HK and H % HK != 0):
        raise ValueError("the key heads must divide the query heads")
    _check_lens("q_lens", q_lens, B, Q1)
    _check_lens("k_lens", k_lens, B, Q1)
    view = _check_lam(lam, (B, H, NQ), Q1)
    _check_cuda(Q1)
    return (B, H, HK, NQ, NK, d, V.shape[3]), view


def diff_problem(B, H, HK, NQ, NK, d, dv, causal=False, s1=None, s2=None, dtype=torch.bfloat16,
                 lam_fp32=False) -> DiffProblem:
    return DiffProblem(B, H, HK, NQ, NK, d, dv, int(bool(causal)), _DTYPES[dtype], int(lam_fp32),
                       _scale(s1), _scale(s2))


def _like(t, width):
    """An empty tensor of t's shape but `width` features, its axes in t's memory order."""
    order = sorted(range(t.dim() - 1), key=lambda k: (-t.stride(k), k))
    out = torch.empty([t.shape[k] for k in order] + [width], dtype=t.dtype, device=t.device)
    back = [0] * t.dim()
    for place, k in enumerate(order):
        back[k] = place
    back[-1] = t.dim() - 1
    return out.permute(back)


def diff_attn_fwd(Q1, K1, Q2, K2, V, lam, causal=False, s1=None, s2=None, q_lens=None, k_lens=None,
                  save=True, out=None):
    """O, O2, LSE1, LSE2 of differential attention on the current stream (streamkl_diff_fwd).

    Q1, Q2 [B, H, NQ, d], K1, K2 [B, HK, NK, d], V [B, HK, NK, dv]; (d, dv) one of (64, 64),
    (64, 128), (128, 128), (128, 256); HK divides H.  ``lam`` is a scalar tensor, [H], or
    [B, H, NQ] with extents of 1 broadcast, in the inputs' type or fp32.  ``q_lens`` / ``k_lens``
    (int32 [B]) give the valid rows of a right-padded batch; the causal mask is bottom-right
    aligned on them (key j is visible from row i when j <= i + k_len - q_len), so a padded
    self-attention batch passes both.  Rows that see no key give O = 0 and LSE = -inf.
    O2 = P2 V and the LSEs are what ``diff_attn_bwd`` needs; ``save=False`` leaves them out (None).
    ``out`` may hold a preallocated O, and with ``save`` O2, LSE1, LSE2."""
    (B, H, HK, NQ, NK, d, dv), lv = _check_diff(Q1, K1, Q2, K2, V, lam, q_lens, k_lens)
    if out is None:
        O = _like(Q1, dv)
        O2 = torch.empty_like(O) if save else None
        LSE1, LSE2 = (torch.empty((B, H, NQ), dtype=torch.float32, device=Q1.device)
                      if save else None for _ in range(2))
    else:
        O, O2, LSE1, LSE2 = tuple(out) if save else (*tuple(out)[:1], None, None, None)
        for name, t in (("O", O), ("O2", O2)):
            if t is not None or name == "O" or save:
                _check_out(name, t, (B, H, NQ, dv), Q1)
        if save and O.numel() and any(n > 1 and a != b for n, a, b in zip(O.shape, O.stride(), O2.stride())):
            raise ValueError("O and O2 must have the same strides")
        if save:
            _check_rows((("LSE1", LSE1), ("LSE2", LSE2)), (B, H, NQ), Q1)
    if O.numel() == 0:
        return O, O2, LSE1, LSE2
    if NK == 0:
        for t in (O, O2):
            if t is not None:
                t.zero_()
        for t in (LSE1, LSE2):
            if t is not None:
                t.fill_(-float("inf"))
        return O, O2, LSE1, LSE2
    prob = diff_problem(B, H, HK, NQ, NK, d, dv, causal, s1, s2, Q1.dtype, lv.dtype == torch.float32)
    with torch.cuda.device(Q1.device):
        st = _lib.streamkl_diff_fwd(ctypes.byref(prob), *map(_tensor, (Q1, K1, Q2, K2, V)), _lam_tensor(lv),
                                    _ptr(q_lens), _ptr(k_lens), _tensor(O), _tensor(O2), _ptr(LSE1),
                                    _ptr(LSE2), _stream(Q1.device))
    if st != OK:
        raise StreamKLError(st, "streamkl_diff_fwd")
    return O, O2, LSE1, LSE2


def _check_rows(named, shape, like):
    for name, t in named:
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.shape != shape \
                or not t.is_contiguous() or t.device != like.device:
            raise ValueError(f"{name} must be a contiguous fp32 tensor [B, H, NQ] on the inputs' device")


def diff_attn_workspace_size(B, H, HK, NQ, NK, d, dv, causal=False) -> int:
    """Bytes of the workspace of ``diff_attn_bwd`` (0 on a bad problem)."""
    prob = diff_problem(B, H, HK, NQ, NK, d, dv, causal)
    return int(_lib.streamkl_diff_bwd_workspace_size(ctypes.byref(prob)))


def diff_attn_bwd(dO, Q1, K1, Q2, K2, V, lam, O, O2, LSE1, LSE2, causal=False, s1=None, s2=None,
                  q_lens=None, k_lens=None, need=(True,) * 6, workspace=None, out=None):
    """dQ1, dK1, dQ2, dK2, dV, dlam (None where not needed) via streamkl_diff_bwd.

    O, O2, LSE1, LSE2 come from ``diff_attn_fwd`` on the same inputs.  Gradients have their inputs'
    shapes and types, key heads summed over the query heads that share them, dlam over what lam is
    broadcast over.  Accumulation is in fp32 and in a fixed order: results repeat bit for bit.  dS is
    rounded to the inputs' 16-bit type for the products, so an fp32 lam's gradient is as exact as
    16-bit operands allow, and fp16 training wants the usual loss scale.
    ``out`` may pass preallocated gradients (None entries are skipped), ``workspace`` a device buffer
    of at least ``diff_attn_workspace_size`` bytes, 256-byte aligned."""
    (B, H, HK, NQ, NK, d, dv), lv = _check_diff(Q1, K1, Q2, K2, V, lam, q_lens, k_lens)
    for name, t in (("dO", dO), ("O", O), ("O2", O2)):
        _check(name, t, (B, H, NQ, dv), Q1, "[B, H, NQ, dv]")
    if O.numel() and any(n > 1 and a != b for n, a, b in zip(O.shape, O.stride(), O2.stride())):
        raise ValueError("O and O2 must have the same strides")
    _check_rows((("LSE1", LSE1), ("LSE2", LSE2)), (B, H, NQ), Q1)
    inputs = (Q1, K1, Q2, K2, V, lam)
    if out is not None:
        if len(out) != 6:
            raise ValueError("out must hold six entries: dQ1, dK1, dQ2, dK2, dV, dlam (None skips one)")
        outs = list(out)
        for name, o, t in zip(("dQ1", "dK1", "dQ2", "dK2", "dV"), outs, inputs):
            if o is not None:
                _check_out(name, o, t.shape, Q1)
        o = outs[5]
        if o is not None and (not isinstance(o, torch.Tensor) or o.shape != lam.shape or o.dtype != lam.dtype
                              or not o.is_contiguous() or o.device != lam.device):
            raise ValueError("dlam must be contiguous, of lam's shape and type")
    else:
        if len(need) != 6:
            raise ValueError("need must hold six entries: dQ1, dK1, dQ2, dK2, dV, dlam")
        outs = [_like(t, t.shape[-1]) if want else None for t, want in zip(inputs[:5], need)]
        outs.append(torch.empty(lam.shape, dtype=lam.dtype, device=lam.device) if need[5] else None)
    if all(o is None for o in outs):
        raise ValueError("no gradient is asked for")
    if Q1.numel() == 0 or K1.numel() == 0:
        for o in outs:
            if o is not None:
                o.zero_()
        return tuple(outs)
    prob = diff_problem(B, H, HK, NQ, NK, d, dv, causal, s1, s2, Q1.dtype, lv.dtype == torch.float32)
    ws_bytes = int(_lib.streamkl_diff_bwd_workspace_size(ctypes.byref(prob)))
    workspace = _workspace(workspace, ws_bytes, Q1)
    with torch.cuda.device(Q1.device):
        st = _lib.streamkl_diff_bwd(ctypes.byref(prob), _tensor(dO), *map(_tensor, (Q1, K1, Q2, K2, V)),
                                    _lam_tensor(lv), _tensor(O), _tensor(O2), _ptr(LSE1), _ptr(LSE2),
                                    _ptr(q_lens), _ptr(k_lens), *map(_tensor, outs[:5]), _ptr(outs[5]),
                                    *workspace, _stream(Q1.device))
    if st != OK:
        raise StreamKLError(st, "streamkl_diff_bwd")
    return tuple(outs)


def _workspace(ws, need, like):
    """(pointer, bytes) of the caller's workspace, or of one from the caching allocator."""
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=like.device)
    elif not isinstance(ws, torch.Tensor) or ws.device != like.device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    elif ws.numel() * ws.element_size() < need:
        raise ValueError("workspace too small")
    return _vp(ws.data_ptr()), ctypes.c_size_t(ws.numel() * ws.element_size())


class _DiffAttnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q1, K1, Q2, K2, V, lam, causal, s1, s2, q_lens, k_lens):
        O, O2, LSE1, LSE2 = diff_attn_fwd(Q1, K1, Q2, K2, V, lam, causal, s1, s2, q_lens, k_lens)
        ctx.save_for_backward(Q1, K1, Q2, K2, V, lam, O, O2, LSE1, LSE2, q_lens, k_lens)
        ctx.cfg = (causal, s1, s2)
        return O

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO):
        *state, q_lens, k_lens = ctx.saved_tensors
        need = tuple(bool(x) for x in ctx.needs_input_grad[:6])
        if not any(need):
            return (None,) * 11
        if not _layout_ok(dO):  # an expanded or sliced upstream gradient
            dO = dO.contiguous()
        return (*diff_attn_bwd(dO, *state, *ctx.cfg, q_lens, k_lens, need=need), *(None,) * 5)


def diff_attn(Q1, K1, Q2, K2, V, lam, causal=False, s1=None, s2=None, q_lens=None, k_lens=None):
    """Differential attention O [B, H, NQ, dv] with autograd for Q1, K1, Q2, K2, V and lam.

    Arguments as in ``diff_attn_fwd``.  O's axes are in Q1's memory order.  Where no gradient is
    wanted, nothing is saved."""
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad
                                       for t in (Q1, K1, Q2, K2, V, lam)):
        return _DiffAttnFunction.apply(Q1, K1, Q2, K2, V, lam, causal, s1, s2, q_lens, k_lens)
    return diff_attn_fwd(Q1, K1, Q2, K2, V, lam, causal, s1, s2, q_lens, k_lens, save=False)[0]


def _paged(Q1, K1, Q2, K2, V, lam, table, lens, s1, s2, workspace, out, where):
    if not isinstance(Q1, torch.Tensor) or Q1.dim() != 3:
        raise ValueError("the query must be a tensor [B, H, d]")
    B, H, d = Q1.shape
    _check("Q1" if Q2 is not None else "Q", Q1, (B, H, d), Q1, "[B, H, d]")
    _check("K1" if Q2 is not None else "K", K1, (None, None, None, d), Q1, "[pages, page_size, HK, d]")
    pages, page_size, HK, _ = K1.shape
    _check("V", V, (pages, page_size, HK, None), Q1, "[pages, page_size, HK, dv]")
    if HK == 0 or H % HK != 0:
        raise ValueError("the key heads must divide the query heads")
    lv = None
    if Q2 is not None:
        _check("Q2", Q2, (B, H, d), Q1, "[B, H, d], as Q1")
        _check("K2", K2, (pages, page_size, HK, d), Q1, "[pages, page_size, HK, d], as K1")
        lv = _check_lam(lam, (B, H), Q1)
    if not isinstance(table, torch.Tensor) or table.dtype != torch.int32 or table.dim() != 2 or \
            table.shape[0] != B or table.device != Q1.device or (table.shape[1] > 1 and table.stride(1) != 1) \
            or (B > 1 and table.stride(0) < table.shape[1]):
        raise ValueError("table must be an int32 tensor [B, pages of a sequence] on the inputs' device, "
                         "its rows contiguous and apart")
    if lens is None:
        raise ValueError("lens must be a contiguous int32 tensor [B] on the inputs' device")
    _check_lens("lens", lens, B, Q1)
    dv = V.shape[3]
    if out is None:
        out = torch.empty((B, H, dv), dtype=Q1.dtype, device=Q1.device)
    else:
        _check_out("out", out, (B, H, dv), Q1)
    _check_cuda(Q1)
    if out.numel() == 0:
        return out
    if K1.numel() == 0 or V.numel() == 0 or table.shape[1] == 0:
        return out.zero_()
    prob = PagedProblem(B, H, HK, d, dv, _DTYPES[Q1.dtype], int(lv is not None and lv.dtype == torch.float32),
                        pages, page_size, table.shape[1], _scale(s1), _scale(s2))
    with torch.cuda.device(Q1.device):
        need = int(_lib.streamkl_paged_workspace_size(ctypes.byref(prob), 1 if Q2 is None else 2))
        # a cache's axes in the order that the library names them: page, head, row
        caches = [t.transpose(1, 2) if t is not None else None for t in (K1, K2, V)]
        st = _lib.streamkl_paged_attn(
            ctypes.byref(prob), _tensor(Q1), _tensor(caches[0]), _tensor(Q2), _tensor(caches[1]),
            _tensor(caches[2]), _lam_tensor(lv) if lv is not None else None, _ptr(table),
            table.stride(0), _ptr(lens), _tensor(out), *_workspace(workspace, need, Q1),
            _stream(Q1.device))
    if st != OK:
        raise StreamKLError(st, where)
    return out


def attn_paged(Q, K, V, table, lens, s=None, workspace=None, out=None):
    """softmax(s Q K^T) V [B, H, dv] of one new token per sequence over paged caches.

    Q [B, H, d]; K [pages, page_size, HK, d] and V [pages, page_size, HK, dv], in any memory order
    of their outer axes; (d, dv) as in ``diff_attn_fwd``; HK divides H.  Token t of sequence b is
    row t % page_size of page table[b, t // page_size] (int32); lens[b] (int32) tokens are attended
    to, none giving 0.  Table entries behind a sequence's end are not read; one outside the cache is
    not followed and, like a length past the table, recorded for ``query_device_status``.
    The work is split over the device by lens as they are when the kernel runs, so a captured call
    follows lengths that grow.  Results repeat bit for bit.  ``workspace`` may pass a device buffer
    of at least ``paged_workspace_size`` bytes, 256-byte aligned."""
    return _paged(Q, K, None, None, V, None, table, lens, s, None, workspace, out, "streamkl_paged_attn")


def diff_attn_paged(Q1, K1, Q2, K2, V, lam, table, lens, s1=None, s2=None, workspace=None, out=None):
    """Differential attention [B, H, dv] of one new token per sequence over paged caches K1, K2 and V
    that share one table.  Arguments as in ``attn_paged``; lam is a scalar tensor, [H] or [B, H]."""
    if Q2 is None or K2 is None or lam is None:
        raise ValueError("Q2, K2 and lam are needed")
    return _paged(Q1, K1, Q2, K2, V, lam, table, lens, s1, s2, workspace, out, "streamkl_paged_attn")


def paged_workspace_size(dv, maps, device=None) -> int:
    """Bytes of the workspace of ``attn_paged`` (maps 1) or ``diff_attn_paged`` (maps 2) on a device."""
    prob = PagedProblem(1, 1, 1, 64 if dv == 64 else 128 if dv == 256 else 64, dv, 0, 0, 1, 1, 1, 0.0, 0.0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = int(_lib.streamkl_paged_workspace_size(ctypes.byref(prob), int(maps)))
    if n == 0:
        raise StreamKLError(EINVAL, "streamkl_paged_workspace_size")
    return n


def paged_write(rows, caches, slots):
    """Writes new tokens' rows into paged caches in one launch (streamkl_paged_write).

    ``rows`` and ``caches`` are tuples of up to four: rows[k] [T, HK, width] goes into caches[k]
    [pages, page_size, HK, width], row t into slot slots[t] = page * page_size + row of the page
    (int32 or int64 [T]).  A negative slot is skipped, one past the cache is skipped and recorded for
    ``query_device_status``.  Slots must be distinct; the rest of the caches stays as it was."""
    rows, caches = tuple(rows), tuple(caches)
    if not 1 <= len(rows) <= 4 or len(rows) != len(caches):
        raise ValueError("rows and caches must be tuples of the same length, one to four")
    first = rows[0]
    if not isinstance(first, torch.Tensor) or first.dim() != 3:
        raise ValueError("rows[0] must be a tensor [T, HK, width]")
    T, HK = first.shape[:2]
    for k, (r, c) in enumerate(zip(rows, caches)):
        _check(f"rows[{k}]", r, (T, HK, None), first, "[T, HK, width]")
        shape = (None, None, HK, r.shape[2])
        _check(f"caches[{k}]", c, shape, first, "[pages, page_size, HK, width]")
        _check_out(f"caches[{k}]", c, c.shape, first)
        if c.shape[:2] != caches[0].shape[:2]:
            raise ValueError("the caches must have the same pages and page size")
        if r.shape[2] % 8 != 0:
            raise ValueError("widths must be multiples of 8")
    if not isinstance(slots, torch.Tensor) or slots.dtype not in (torch.int32, torch.int64) or \
            slots.shape != (T,) or not slots.is_contiguous() or slots.device != first.device:
        raise ValueError("slots must be a contiguous int32 or int64 tensor [T] on the rows' device")
    _check_cuda(first)
    if any(r.numel() == 0 for r in rows) or caches[0].numel() == 0:
        if all(r.numel() == 0 for r in rows):
            return
        raise ValueError("there is no slot to write to")
    n = len(rows)
    rt = (_Tensor * n)(*(_Tensor(r.data_ptr(), 0, r.stride(1), r.stride(0)) for r in rows))
    ct = (_Tensor * n)(*(_Tensor(c.data_ptr(), c.stride(0), c.stride(2), c.stride(1)) for c in caches))
    widths = (ctypes.c_int * n)(*(r.shape[2] for r in rows))
    pages, page_size = caches[0].shape[:2]
    with torch.cuda.device(first.device):
        st = _lib.streamkl_paged_write(n, rt, ct, widths, _ptr(slots), int(slots.dtype == torch.int64), T, HK,
                                       pages, page_size, _stream(first.device))
    if st != OK:
        raise StreamKLError(st, "streamkl_paged_write")
