"""Differential attention and paged single-token attention (the second part of include/streamkl.h).

    O = (softmax(s1 Q1 K1^T) - lam softmax(s2 Q2 K2^T)) V

``diff_attn`` is the autograd entry point, ``diff_attn_fwd`` and ``diff_attn_bwd`` its two halves,
``diff_attn_paged`` its form for one new token over paged caches, ``attn_paged`` the same with one
softmax map, ``paged_write`` puts new tokens' rows into the caches.

As in ``binding``, this is argument marshalling only: tensors are checked for dtype, device, shape and
layout, and every step of the computation runs in the library's kernels on the current stream.
The checks of shapes, types and layouts are a function of these alone; their results (and the
problem's C structs without pointers) are kept by them, since for one token's step they would take
longer than the kernels.
Tensors are bf16 or fp16 (one type for all of a call), with contiguous features; the other axes may
have any positive strides that are multiples of 8 elements, so a projection's [B, N, H, d] output
passes as ``.transpose(1, 2)`` without a copy.
"""
from __future__ import annotations

import ctypes
import functools
from collections import namedtuple

import torch
from torch.autograd import forward_ad

from .binding import EINVAL, OK, StreamKLError, _lib, _vp

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


# Pointers to structs are passed as addresses.
_sz = ctypes.c_size_t
_lib.streamkl_diff_fwd.argtypes = [_vp] * 14
_lib.streamkl_diff_fwd.restype = ctypes.c_int
_lib.streamkl_diff_bwd_workspace_size.argtypes = [_vp]
_lib.streamkl_diff_bwd_workspace_size.restype = _sz
_lib.streamkl_diff_bwd.argtypes = [_vp] * 21 + [_sz, _vp]
_lib.streamkl_diff_bwd.restype = ctypes.c_int
_lib.streamkl_paged_workspace_size.argtypes = [_vp, ctypes.c_int]
_lib.streamkl_paged_workspace_size.restype = _sz
_lib.streamkl_paged_attn.argtypes = [_vp] * 8 + [ctypes.c_int64] + [_vp] * 3 + [_sz, _vp]
_lib.streamkl_paged_attn.restype = ctypes.c_int
_lib.streamkl_paged_write.argtypes = [ctypes.c_int] + [_vp] * 4 + [ctypes.c_int] * 5 + [_vp]
_lib.streamkl_paged_write.restype = ctypes.c_int

# The current stream's handle, without a Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

# What the checks look at.
_Meta = namedtuple("_Meta", "shape stride dtype device")


def _keys(*tensors):
    """What the checks depend on, as it comes; None for None."""
    try:
        return [None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in tensors]
    except AttributeError:
        raise ValueError("operands must be tensors") from None


def _meta(t):
    """The same with names."""
    return _Meta(*_keys(t)[0]) if t is not None else None


def _planned(plan):
    """A plan class as a function of keys: each key becomes a _Meta, the result is kept."""
    return functools.lru_cache(maxsize=512)(
        lambda *keys: plan(*(_Meta(*k) if isinstance(k, tuple) else k for k in keys)))


def _contiguous(m) -> bool:
    want = 1
    for n, s in zip(reversed(m.shape), reversed(m.stride)):
        if n != 1 and s != want and 0 not in m.shape:
            return False
        want *= n
    return True


def _layout_ok(m) -> bool:
    """Contiguous features, outer strides positive multiples of 8 elements."""
    return (m.shape[-1] == 1 or m.stride[-1] == 1) and \
        all(n == 1 or (s > 0 and s % 8 == 0) for n, s in zip(m.shape[:-1], m.stride[:-1]))


def _check(name, m, shape, like, what):
    """One 16-bit operand: its shape (None matches anything), type, device and layout."""
    if m is None or len(m.shape) != len(shape) or \
            any(want is not None and want != got for want, got in zip(shape, m.shape)):
        raise ValueError(f"{name} must be a tensor {what}")
    if m.dtype not in _DTYPES or m.dtype != like.dtype:
        raise ValueError(f"{name} must be bf16 or fp16, the same type as the other operands")
    if m.device != like.device:
        raise ValueError("tensors must be on one device")
    if max(m.shape) >= 2 ** 31:
        raise ValueError(f"{name} must have extents below 2^31")
    if 0 not in m.shape and not _layout_ok(m):
        raise ValueError(f"{name} must have contiguous features and outer strides that are positive "
                         "multiples of 8 elements")


def _check_out(name, m, shape, like):
    """A caller's output: as an operand, and no two of its elements in one place."""
    _check(name, m, tuple(shape), like, f"of shape {tuple(shape)}")
    need = 1
    for s, n in sorted((s, n) for n, s in zip(m.shape, m.stride) if n > 1):
        if s < need:
            raise ValueError(f"{name} must not overlap itself")
        need = s * n


def _check_cuda(device):
    if device.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")


def _check_lens(name, m, B, like):
    if m is not None and (m.dtype != torch.int32 or tuple(m.shape) != (B,) or not _contiguous(m)
                          or m.device != like.device):
        raise ValueError(f"{name} must be a contiguous int32 tensor [B] on the inputs' device")


def _check_rows(name, m, shape, like):
    if m is None or m.dtype != torch.float32 or tuple(m.shape) != tuple(shape) or not _contiguous(m) \
            or m.device != like.device:
        raise ValueError(f"{name} must be a contiguous fp32 tensor [B, H, NQ] on the inputs' device")


def _check_same_strides(O, O2):
    if 0 not in O.shape and any(n > 1 and a != b for n, a, b in zip(O.shape, O.stride, O2.stride)):
        raise ValueError("O and O2 must have the same strides")


def _lam_strides(m, extents, like):
    """Element strides of lam along the extents, 0 where it is broadcast."""
    if m is None or m.dtype not in (like.dtype, torch.float32) or m.device != like.device:
        raise ValueError("lam must be a tensor of the inputs' type or fp32 on their device")
    shape, stride = tuple(m.shape), tuple(m.stride)
    if len(shape) == 0:
        shape, stride = (1,) * len(extents), (0,) * len(extents)
    elif len(shape) == 1:
        shape, stride = (1, *shape) + (1,) * (len(extents) - 2), (0, *stride) + (0,) * (len(extents) - 2)
    if len(shape) != len(extents) or any(n not in (1, e) for n, e in zip(shape, extents)):
        raise ValueError("lam must be a scalar, [H], or one weight per " +
                         ("[B, H, NQ]" if len(extents) == 3 else "[B, H]") + " (extents of 1 broadcast)")
    return (*(s if n > 1 else 0 for n, s in zip(shape, stride)), 0)[:3]


def _lam(lam):
    """lam itself, or a copy where an axis of it was expanded: each element then has a place."""
    if not isinstance(lam, torch.Tensor) or lam.is_contiguous():
        return lam
    return lam.contiguous() if any(n > 1 and s <= 0 for n, s in zip(lam.shape, lam.stride())) else lam


def _scale(s):
    """A scale's value when the call is made: plans are kept by it."""
    return float(s) if s is not None else 0.0


class _Structs:
    """streamkl_tensor structs without their pointers; ``at`` puts the pointers in, in a new copy, and
    gives the addresses to pass, NULL for a pointer of 0."""

    def __init__(self, strides):
        words = []
        for st in strides:
            words += [0, *(st if st is not None else (0, 0, 0))]
        self.type = ctypes.c_uint64 * len(words)
        self.template = bytes(self.type(*(w % 2 ** 64 for w in words)))

    def at(self, pointers):
        block = self.type.from_buffer_copy(self.template)
        block[::4] = pointers
        base = ctypes.addressof(block)
        return block, [base + 32 * k if p else None for k, p in enumerate(pointers)]


def _outer(m):
    """The three outer strides of an operand, or of a row operand with fewer axes the leading ones."""
    return (*m.stride[:-1], 0, 0)[:3]


def _order(m):
    """The outer axes from the slowest to the fastest in memory, and where each one went."""
    order = sorted(range(len(m.shape) - 1), key=lambda k: (-m.stride[k], k))
    back = [0] * len(m.shape)
    for place, k in enumerate(order):
        back[k] = place
    back[-1] = len(m.shape) - 1
    return tuple(order), tuple(back)


@functools.lru_cache(maxsize=512)
def _like_shape(shape, stride, width):
    order, back = _order(_Meta(shape, stride, None, None))
    return [*(shape[k] for k in order), width], back if order != tuple(range(len(order))) else None


def _low_bits(*tensors):
    """What the addresses have under 16 bytes."""
    low = 0
    for t in tensors:
        low |= t.data_ptr()
    return low & 15


def _readable(t):
    """t, or a copy where the kernels cannot read it as it lies."""
    return t if t.data_ptr() % 16 == 0 and _layout_ok(_meta(t)) else t.clone(memory_format=torch.contiguous_format)


def _pointers(*tensors):
    """Data pointers, 0 for None; operands start on 16 bytes."""
    out = [0 if t is None else t.data_ptr() for t in tensors]
    low = 0
    for p in out:
        low |= p
    if low & 15:
        raise ValueError("operands must be 16-byte aligned")
    return out


def _check_places(outs, operands=()):
    """A caller's outputs start in different places, and not where an operand does."""
    outs = [p for p in outs if p]
    if len(set(outs)) != len(outs) or not set(outs).isdisjoint(operands):
        raise ValueError("outputs must not be in one place with each other or with an operand")


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _run(fn, where, device, *args):
    """Calls the library on the current stream of `device`, that device current."""
    if torch.cuda.current_device() == device.index:
        st = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device.index))
    if st != OK:
        raise StreamKLError(st, where)


def _workspace(ws, need, like):
    """The caller's workspace, or one from the caching allocator: (tensor, pointer, bytes)."""
    if ws is None:
        ws = like.new_empty(need, dtype=torch.uint8)
        return ws, ws.data_ptr(), need
    if not isinstance(ws, torch.Tensor) or ws.device != like.device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    have = ws.numel() * ws.element_size()
    if have < need:
        raise ValueError("workspace too small")
    return ws, ws.data_ptr(), have


def diff_problem(B, H, HK, NQ, NK, d, dv, causal=False, s1=None, s2=None, dtype=torch.bfloat16,
                 lam_fp32=False) -> DiffProblem:
    return DiffProblem(B, H, HK, NQ, NK, d, dv, int(bool(causal)), _DTYPES[dtype], int(lam_fp32),
                       _scale(s1), _scale(s2))


class _DiffPlan:
    """One problem's checked dimensions and C structs."""

    def __init__(self, Q1, K1, Q2, K2, V, lam, q_lens, k_lens, causal, s1, s2):
        if Q1 is None or len(Q1.shape) != 4:
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
        lam_strides = _lam_strides(lam, (B, H, NQ), Q1)
        _check_cuda(Q1.device)
        dv = V.shape[3]
        self.saved = None   # the keys of what the forward saves for the backward
        self.options = causal, s1, s2
        self.device = Q1.device
        self.rows, self.out, self.q = (B, H, NQ), (B, H, NQ, dv), Q1
        self.empty = 0 in self.out or HK == 0
        self.out_shape, self.out_back = _like_shape(Q1.shape, Q1.stride, dv)
        self.grads = [_like_shape(m.shape, m.stride, m.shape[-1]) for m in (Q1, K1, Q2, K2, V)]
        self.fwd = {}   # the forward's C structs for outputs in Q1's memory order, with and without O2
        self.bwd = {}   # the backward's, by the gradients asked for and the layouts of dO and the state
        self.no_keys = NK == 0
        self.prob = diff_problem(B, H, HK, NQ, NK, d, dv, causal, s1, s2, Q1.dtype, lam.dtype == torch.float32)
        self.prob_at = ctypes.addressof(self.prob)
        self.inputs = [*map(_outer, (Q1, K1, Q2, K2, V)), lam_strides]
        self.ws_bytes = max(256, int(_lib.streamkl_diff_bwd_workspace_size(self.prob_at)))


_diff_plan = _planned(_DiffPlan)


def _plan_of(Q1, K1, Q2, K2, V, lam, q_lens, k_lens, causal, s1, s2):
    return _diff_plan(*_keys(Q1, K1, Q2, K2, V, lam, q_lens, k_lens), bool(causal), _scale(s1), _scale(s2))


def _fwd_structs(plan, O, O2):
    return _Structs([*plan.inputs, _outer(O), _outer(O2) if O2 is not None else None])


def diff_attn_fwd(Q1, K1, Q2, K2, V, lam, causal=False, s1=None, s2=None, q_lens=None, k_lens=None,
                  save=True, out=None):
    """O, O2, LSE1, LSE2 of differential attention on the current stream (streamkl_diff_fwd).

    Q1, Q2 [B, H, NQ, d], K1, K2 [B, HK, NK, d], V [B, HK, NK, dv]; (d, dv) one of (64, 64),
    (64, 128), (128, 128), (128, 256); HK divides H.  ``lam`` is a scalar tensor, [H], or
    [B, H, NQ] with extents of 1 broadcast, in the inputs' type or fp32.  ``q_lens`` / ``k_lens``
    (int32 [B]) give the valid rows of a right-padded batch; the causal mask is bottom-right
    aligned on them (key j is visible from row i when j <= i + k_len - q_len), so a padded
    self-attention batch passes both.  Rows that see no key give O = 0 and LSE = -inf.  Scales of
    None (or <= 0) are 1/sqrt(d).
    O2 = P2 V and the LSEs are what ``diff_attn_bwd`` needs; ``save=False`` leaves them out (None).
    ``out`` may hold a preallocated O, and with ``save`` O2, LSE1, LSE2, none of them in memory that
    another output, K1, K2 or V has."""
    lam = _lam(lam)
    plan = _plan_of(Q1, K1, Q2, K2, V, lam, q_lens, k_lens, causal, s1, s2)
    return _forward(plan, Q1, K1, Q2, K2, V, lam, q_lens, k_lens, save, out)


def _forward(plan, Q1, K1, Q2, K2, V, lam, q_lens, k_lens, save, out):
    if out is None:
        O, O2 = (Q1.new_empty(plan.out_shape) if k == 0 or save else None for k in range(2))
        if plan.out_back is not None:
            O, O2 = O.permute(plan.out_back), O2.permute(plan.out_back) if save else None
        LSE1, LSE2 = (Q1.new_empty(plan.rows, dtype=torch.float32) if save else None for _ in range(2))
        structs = plan.fwd.get(save)
        if structs is None:
            structs = plan.fwd[save] = _fwd_structs(plan, _meta(O), _meta(O2))
            if save:
                plan.saved = _keys(Q1, K1, Q2, K2, V, lam, O, O2, LSE1, LSE2, q_lens, k_lens)
    else:
        out = tuple(out)
        if len(out) != 4:
            raise ValueError("out must hold four entries: O, O2, LSE1, LSE2")
        O, O2, LSE1, LSE2 = out if save else (out[0], None, None, None)
        mO, mO2 = _meta(O), _meta(O2)
        _check_out("O", mO, plan.out, plan.q)
        if save:
            _check_out("O2", mO2, plan.out, plan.q)
            _check_same_strides(mO, mO2)
            _check_rows("LSE1", _meta(LSE1), plan.rows, plan.q)
            _check_rows("LSE2", _meta(LSE2), plan.rows, plan.q)
        structs = _fwd_structs(plan, mO, mO2)
    if plan.empty or plan.no_keys:
        for t, v in ((O, 0.0), (O2, 0.0), (LSE1, -float("inf")), (LSE2, -float("inf"))):
            if t is not None:
                t.fill_(v)
        return O, O2, LSE1, LSE2
    p = _pointers(Q1, K1, Q2, K2, V, O, O2)
    if out is not None:
        # over Q is well: a block reads its rows of Q before it writes those of O
        _check_places([*p[5:], *((LSE1.data_ptr(), LSE2.data_ptr()) if save else ())], (p[1], p[3], p[4]))
    block, at = structs.at([*p[:5], lam.data_ptr(), *p[5:]])
    _run(_lib.streamkl_diff_fwd, "streamkl_diff_fwd", plan.device, plan.prob_at, *at[:6], _ptr(q_lens),
         _ptr(k_lens), *at[6:], _ptr(LSE1), _ptr(LSE2))
    return O, O2, LSE1, LSE2


def diff_attn_workspace_size(B, H, HK, NQ, NK, d, dv, causal=False) -> int:
    """Bytes of the workspace of ``diff_attn_bwd`` (0 on a bad problem)."""
    prob = diff_problem(B, H, HK, NQ, NK, d, dv, causal)
    return int(_lib.streamkl_diff_bwd_workspace_size(ctypes.addressof(prob)))


def _bwd_structs(plan, dO, O, O2, LSE1, LSE2, grads):
    for name, m in (("dO", dO), ("O", O), ("O2", O2)):
        _check(name, m, plan.out, plan.q, "[B, H, NQ, dv]")
    _check_same_strides(O, O2)
    _check_rows("LSE1", LSE1, plan.rows, plan.q)
    _check_rows("LSE2", LSE2, plan.rows, plan.q)
    return _Structs([_outer(dO), *plan.inputs, _outer(O), _outer(O2),
                     *(_outer(m) if m is not None else None for m in grads)])


def diff_attn_bwd(dO, Q1, K1, Q2, K2, V, lam, O, O2, LSE1, LSE2, causal=False, s1=None, s2=None,
                  q_lens=None, k_lens=None, need=(True,) * 6, workspace=None, out=None):
    """dQ1, dK1, dQ2, dK2, dV, dlam (None where not needed) via streamkl_diff_bwd.

    O, O2, LSE1, LSE2 come from ``diff_attn_fwd`` on the same inputs.  Gradients have their inputs'
    shapes and types, key heads summed over the query heads that share them, dlam over what lam is
    broadcast over.  Accumulation is in fp32 and in a fixed order: results repeat bit for bit.  dS is
    rounded to the inputs' 16-bit type for the products, so an fp32 lam's gradient is as exact as
    16-bit operands allow, and fp16 training wants the usual loss scale.
    ``out`` may pass preallocated gradients (None entries are skipped), each in memory that no other
    gradient, dO, Q, K or V has, ``workspace`` a device buffer
    of at least ``diff_attn_workspace_size`` bytes, 256-byte aligned."""
    lam = _lam(lam)
    plan = _plan_of(Q1, K1, Q2, K2, V, lam, q_lens, k_lens, causal, s1, s2)
    return _backward(plan, dO, Q1, K1, Q2, K2, V, lam, O, O2, LSE1, LSE2, q_lens, k_lens, tuple(need),
                     workspace, out)


def _backward(plan, dO, Q1, K1, Q2, K2, V, lam, O, O2, LSE1, LSE2, q_lens, k_lens, need, workspace, out,
              state=None):
    """``state``: the keys of O, O2, LSE1 and LSE2 where the caller has them."""
    inputs = (Q1, K1, Q2, K2, V)
    key = structs = None
    if out is not None:
        if len(out) != 6:
            raise ValueError("out must hold six entries: dQ1, dK1, dQ2, dK2, dV, dlam (None skips one)")
        outs = list(out)
        for name, o, t in zip(("dQ1", "dK1", "dQ2", "dK2", "dV"), outs, inputs):
            if o is not None:
                _check_out(name, _meta(o), t.shape, plan.q)
        o = outs[5]
        if o is not None and (not isinstance(o, torch.Tensor) or o.shape != lam.shape or o.dtype != lam.dtype
                              or not o.is_contiguous() or o.device != lam.device):
            raise ValueError("dlam must be contiguous, of lam's shape and type")
    else:
        if len(need) != 6:
            raise ValueError("need must hold six entries: dQ1, dK1, dQ2, dK2, dV, dlam")
        key = (need, *_keys(dO), *(state or _keys(O, O2, LSE1, LSE2)))
        structs = plan.bwd.get(key)
        outs = []
        for (shape, back), want in zip(plan.grads, need):
            o = Q1.new_empty(shape) if want else None
            outs.append(o if o is None or back is None else o.permute(back))
        outs.append(lam.new_empty(lam.shape) if need[5] else None)
    if all([o is None for o in outs]):
        raise ValueError("no gradient is asked for")
    if structs is None:
        structs = _bwd_structs(plan, *map(_meta, (dO, O, O2, LSE1, LSE2)), tuple(map(_meta, outs[:5])))
        if key is not None and len(plan.bwd) < 64:
            plan.bwd[key] = structs
    if plan.empty or plan.no_keys:
        for o in outs:
            if o is not None:
                o.zero_()
        return tuple(outs)
    p = _pointers(dO, *inputs, O, O2, *outs[:5])
    if out is not None:
        # lam, O and O2 are read by the first kernel alone, before anything is written
        _check_places([*p[8:], _ptr(outs[5])], p[:6])
    block, at = structs.at([*p[:6], lam.data_ptr(), *p[6:]])
    ws, ws_at, ws_bytes = _workspace(workspace, plan.ws_bytes, Q1)
    _run(_lib.streamkl_diff_bwd, "streamkl_diff_bwd", plan.device, plan.prob_at, *at[:9], _ptr(LSE1),
         _ptr(LSE2), _ptr(q_lens), _ptr(k_lens), *at[9:], _ptr(outs[5]), ws_at, ws_bytes)
    return tuple(outs)


def _tracked(Q1, K1, Q2, K2, V, lam):
    """Whether autograd looks at a call (of one map: Q2, K2 and lam are None): a gradient is wanted, or in
    a level of forward-mode differentiation (-1 is none) an operand has a tangent."""
    if torch.is_grad_enabled() and (Q1.requires_grad or K1.requires_grad or V.requires_grad or
                                    (lam is not None and (Q2.requires_grad or K2.requires_grad or
                                                          lam.requires_grad))):
        return True
    if getattr(forward_ad, "_current_level", 0) < 0:
        return False
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None
               for t in (Q1, K1, Q2, K2, V, lam))


class _DiffAttnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, Q1, K1, Q2, K2, V, lam, q_lens, k_lens):
        saved = _forward(plan, Q1, K1, Q2, K2, V, lam, q_lens, k_lens, True, None)
        ctx.save_for_backward(Q1, K1, Q2, K2, V, lam, *saved, q_lens, k_lens)
        ctx.plan = plan
        return saved[0]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO):
        need = ctx.needs_input_grad[1:7]
        dO = _readable(dO)   # expanded or sliced
        Q1, K1, Q2, K2, V, lam, O, O2, LSE1, LSE2, q_lens, k_lens = saved = ctx.saved_tensors
        plan = ctx.plan
        # hooks on saved tensors (offloading, say) may give them back in another layout
        given = _keys(*saved)
        state = given[6:10]
        if given != plan.saved or _low_bits(Q1, K1, Q2, K2, V, O, O2):
            Q1, K1, Q2, K2, V, O, O2 = map(_readable, (Q1, K1, Q2, K2, V, O, O2))
            if O.stride() != O2.stride():
                O, O2 = O.contiguous(), O2.contiguous()
            lam, LSE1, LSE2 = _lam(lam), LSE1.contiguous(), LSE2.contiguous()
            plan = _plan_of(Q1, K1, Q2, K2, V, lam, q_lens, k_lens, *plan.options)
            state = None
        return (None, *_backward(plan, dO, Q1, K1, Q2, K2, V, lam, O, O2, LSE1, LSE2, q_lens, k_lens, need,
                                 None, None, state), None, None)


def diff_attn(Q1, K1, Q2, K2, V, lam, causal=False, s1=None, s2=None, q_lens=None, k_lens=None):
    """Differential attention O [B, H, NQ, dv] with autograd for Q1, K1, Q2, K2, V and lam.

    Arguments as in ``diff_attn_fwd``.  O's axes are in Q1's memory order.  Where no gradient is
    wanted, nothing is saved.  Gradients of gradients and forward-mode tangents are refused."""
    lam = _lam(lam)
    plan = _plan_of(Q1, K1, Q2, K2, V, lam, q_lens, k_lens, causal, s1, s2)
    if _tracked(Q1, K1, Q2, K2, V, lam):
        return _DiffAttnFunction.apply(plan, Q1, K1, Q2, K2, V, lam, q_lens, k_lens)
    return _forward(plan, Q1, K1, Q2, K2, V, lam, q_lens, k_lens, False, None)[0]


class _PagedPlan:
    """One paged problem's checked dimensions and C structs."""

    def __init__(self, Q1, K1, Q2, K2, V, lam, table, lens, out, s1, s2):
        if Q1 is None or len(Q1.shape) != 3:
            raise ValueError("the query must be a tensor [B, H, d]")
        B, H, d = Q1.shape
        two = Q2 is not None
        _check("Q1" if two else "Q", Q1, (B, H, d), Q1, "[B, H, d]")
        _check("K1" if two else "K", K1, (None, None, None, d), Q1, "[pages, page_size, HK, d]")
        pages, page_size, HK, _ = K1.shape
        _check("V", V, (pages, page_size, HK, None), Q1, "[pages, page_size, HK, dv]")
        if HK == 0 or H % HK != 0:
            raise ValueError("the key heads must divide the query heads")
        if two:
            _check("Q2", Q2, (B, H, d), Q1, "[B, H, d], as Q1")
            _check("K2", K2, (pages, page_size, HK, d), Q1, "[pages, page_size, HK, d], as K1")
        lam_strides = _lam_strides(lam, (B, H), Q1) if two else None
        if table is None or table.dtype != torch.int32 or len(table.shape) != 2 or table.shape[0] != B or \
                table.device != Q1.device or (table.shape[1] > 1 and table.stride[1] != 1) or \
                (B > 1 and table.stride[0] < table.shape[1]) or table.shape[1] >= 2 ** 31:
            raise ValueError("table must be an int32 tensor [B, pages of a sequence] on the inputs' device, "
                             "its rows contiguous and apart")
        if lens is None:
            raise ValueError("lens must be a contiguous int32 tensor [B] on the inputs' device")
        _check_lens("lens", lens, B, Q1)
        dv = V.shape[3]
        self.out, self.device = (B, H, dv), Q1.device
        if out is not None:
            _check_out("out", out, self.out, Q1)
        _check_cuda(Q1.device)
        self.empty = 0 in self.out
        self.no_keys = pages == 0 or page_size == 0 or table.shape[1] == 0
        self.table_stride = table.stride[0]
        self.prob = PagedProblem(B, H, HK, d, dv, _DTYPES[Q1.dtype], int(two and lam.dtype == torch.float32),
                                 pages, page_size, table.shape[1], _scale(s1), _scale(s2))
        self.prob_at = ctypes.addressof(self.prob)

        def cache(m):  # page, head, row
            return (m.stride[0], m.stride[2], m.stride[1]) if m is not None else None

        self.structs = _Structs([_outer(Q1), cache(K1), _outer(Q2) if two else None, cache(K2), cache(V),
                                 lam_strides, _outer(out) if out is not None else (H * dv, dv, 0)])
        self.ws_bytes = 0
        if not (self.empty or self.no_keys):
            with torch.cuda.device(Q1.device):
                # 0 for a problem that the call itself refuses
                self.ws_bytes = max(256, int(_lib.streamkl_paged_workspace_size(self.prob_at, 2 if two else 1)))


_paged_plan = _planned(_PagedPlan)


class _PagedFunction(torch.autograd.Function):
    """The paged forms in autograd: their outputs want a gradient where an operand does, and refuse to give
    one, rather than that it is lost without a word."""

    @staticmethod
    def forward(ctx, call, out, *operands):
        O = call()
        # the caller's buffer stays outside the graph: what is returned shares its memory
        return O.new_empty(0).set_(O) if O is out[0] else O

    @staticmethod
    def backward(ctx, dO):
        raise NotImplementedError("attention over paged caches has no backward: call diff_attn where gradients "
                                  "are wanted, or detach its operands")


def _paged(Q1, K1, Q2, K2, V, lam, table, lens, s1, s2, workspace, out):
    lam = _lam(lam)
    plan = _paged_plan(*_keys(Q1, K1, Q2, K2, V, lam, table, lens, out), _scale(s1), _scale(s2))
    if _tracked(Q1, K1, Q2, K2, V, lam):
        return _PagedFunction.apply(
            lambda: _paged_forward(plan, Q1, K1, Q2, K2, V, lam, table, lens, workspace, out), [out],
            Q1, K1, Q2, K2, V, lam)
    return _paged_forward(plan, Q1, K1, Q2, K2, V, lam, table, lens, workspace, out)


def _paged_forward(plan, Q1, K1, Q2, K2, V, lam, table, lens, workspace, out):
    if out is None:
        out = Q1.new_empty(plan.out)
    if plan.empty or plan.no_keys:
        return out.zero_()
    p = _pointers(Q1, K1, Q2, K2, V, out)
    block, at = plan.structs.at([*p[:5], lam.data_ptr() if lam is not None else 0, p[5]])
    ws, ws_at, ws_bytes = _workspace(workspace, plan.ws_bytes, Q1)
    _run(_lib.streamkl_paged_attn, "streamkl_paged_attn", plan.device, plan.prob_at, *at[:6],
         table.data_ptr(), plan.table_stride, lens.data_ptr(), at[6], ws_at, ws_bytes)
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
    of at least ``paged_workspace_size`` bytes, 256-byte aligned.
    At most 2048 sequences a call.  There is no backward: where an operand wants a gradient the
    output does too, and asking for it raises NotImplementedError."""
    return _paged(Q, K, None, None, V, None, table, lens, s, None, workspace, out)


def diff_attn_paged(Q1, K1, Q2, K2, V, lam, table, lens, s1=None, s2=None, workspace=None, out=None):
    """Differential attention [B, H, dv] of one new token per sequence over paged caches K1, K2 and V
    that share one table.  Arguments as in ``attn_paged``; lam is a scalar tensor, [H] or [B, H]."""
    if Q2 is None or K2 is None or lam is None:
        raise ValueError("Q2, K2 and lam are needed")
    return _paged(Q1, K1, Q2, K2, V, lam, table, lens, s1, s2, workspace, out)


def paged_workspace_size(dv, maps, device=None) -> int:
    """Bytes of the workspace of ``attn_paged`` (maps 1) or ``diff_attn_paged`` (maps 2) on a device."""
    prob = PagedProblem(1, 1, 1, 128 if dv == 256 else 64, dv, 0, 0, 1, 1, 1, 0.0, 0.0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = int(_lib.streamkl_paged_workspace_size(ctypes.addressof(prob), int(maps)))
    if n == 0:
        raise StreamKLError(EINVAL, "streamkl_paged_workspace_size")
    return n


class _WritePlan:
    """One write's checked dimensions and C structs."""

    def __init__(self, n, *metas):
        rows, caches, slots = metas[:n], metas[n:-1], metas[-1]
        first = rows[0]
        if first is None or len(first.shape) != 3:
            raise ValueError("rows[0] must be a tensor [T, HK, width]")
        T, HK = first.shape[:2]
        for k, (r, c) in enumerate(zip(rows, caches)):
            _check(f"rows[{k}]", r, (T, HK, None), first, "[T, HK, width]")
            _check(f"caches[{k}]", c, (None, None, HK, r.shape[2]), first, "[pages, page_size, HK, width]")
            _check_out(f"caches[{k}]", c, c.shape, first)
            if c.shape[:2] != caches[0].shape[:2]:
                raise ValueError("the caches must have the same pages and page size")
            if r.shape[2] % 8 != 0:
                raise ValueError("widths must be multiples of 8")
        if slots is None or slots.dtype not in (torch.int32, torch.int64) or tuple(slots.shape) != (T,) or \
                not _contiguous(slots) or slots.device != first.device:
            raise ValueError("slots must be a contiguous int32 or int64 tensor [T] on the rows' device")
        _check_cuda(first.device)
        self.empty = any(0 in r.shape for r in rows)
        if self.empty and not all(0 in r.shape for r in rows):
            raise ValueError("rows must all be empty or none")
        if not self.empty and 0 in caches[0].shape:
            raise ValueError("there is no slot to write to")
        self.device, self.n = first.device, len(rows)
        self.structs = _Structs([(0, r.stride[1], r.stride[0]) for r in rows] +
                                [(c.stride[0], c.stride[2], c.stride[1]) for c in caches])
        self.widths = (ctypes.c_int * self.n)(*(r.shape[2] for r in rows))
        self.widths_at = ctypes.addressof(self.widths)
        self.tail = (int(slots.dtype == torch.int64), T, HK, *caches[0].shape[:2])


_write_plan = _planned(_WritePlan)


def paged_write(rows, caches, slots):
    """Writes new tokens' rows into paged caches in one launch (streamkl_paged_write).

    ``rows`` and ``caches`` are tuples of up to four: rows[k] [T, HK, width] goes into caches[k]
    [pages, page_size, HK, width], row t into slot slots[t] = page * page_size + row of the page
    (int32 or int64 [T]).  A negative slot is skipped, one past the cache is skipped and recorded for
    ``query_device_status``.  Slots must be distinct, and rows that are views of
    the caches apart from the slots written; the rest of the caches stays as it was.  No gradient
    passes through the caches."""
    n = len(rows)
    if not 1 <= n <= 4 or n != len(caches):
        raise ValueError("rows and caches must be tuples of the same length, one to four")
    plan = _write_plan(n, *_keys(*rows, *caches, slots))
    if plan.empty:
        return
    p = _pointers(*rows, *caches)
    if len(set(p[n:])) != n:
        raise ValueError("the caches must not be in one place with each other")
    block, at = plan.structs.at(p)
    _run(_lib.streamkl_paged_write, "streamkl_paged_write", plan.device, n, at[0], at[n], plan.widths_at,
         slots.data_ptr(), *plan.tail)
