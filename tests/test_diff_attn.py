"""CPU tests of differential attention and the paged caches: what is refused, before any CUDA call, by the
binding and by the C ABI, and the formulas of the reference against differences."""
import ctypes
import math

import pytest
import torch

from attention_kl_distillation_b200 import binding as B
from attention_kl_distillation_b200 import diff as D
from diff_ref import Reference

BF, HF = torch.bfloat16, torch.float16


def ops(dtype=BF, d=64, dv=64, H=4, HK=2):
    z = lambda h, n, w: torch.zeros(2, h, n, w, dtype=dtype)  # noqa: E731
    return dict(Q1=z(H, 9, d), K1=z(HK, 12, d), Q2=z(H, 9, d), K2=z(HK, 12, d), V=z(HK, 12, dv),
                lam=torch.zeros(H, dtype=dtype))


BAD = {
    "fp32": dict(Q1=torch.zeros(2, 4, 9, 64)),
    "mixed types": dict(K2=torch.zeros(2, 2, 12, 64, dtype=HF)),
    "three axes": dict(Q1=torch.zeros(2, 9, 64, dtype=BF)),
    "other keys": dict(K2=torch.zeros(2, 2, 11, 64, dtype=BF)),
    "other width": dict(Q2=torch.zeros(2, 4, 9, 128, dtype=BF)),
    "other batch": dict(V=torch.zeros(1, 2, 12, 64, dtype=BF)),
    "heads": dict(K1=torch.zeros(2, 3, 12, 64, dtype=BF), K2=torch.zeros(2, 3, 12, 64, dtype=BF),
                  V=torch.zeros(2, 3, 12, 64, dtype=BF)),
    "expanded": dict(V=torch.zeros(2, 1, 12, 64, dtype=BF).expand(2, 2, 12, 64)),
    "features apart": dict(Q1=torch.zeros(2, 4, 64, 9, dtype=BF).transpose(2, 3)),
    "odd stride": dict(Q1=torch.zeros(2, 4, 9, 68, dtype=BF)[..., :64]),
    "unaligned": dict(Q1=torch.zeros(2, 4, 9, 72, dtype=BF)[..., 4:68]),
    "lam type": dict(lam=torch.zeros(4, dtype=torch.float64)),
    "lam heads": dict(lam=torch.zeros(3, dtype=BF)),
    "lam axes": dict(lam=torch.zeros(4, 9, dtype=BF)),
    "lam rows": dict(lam=torch.zeros(2, 4, 8, dtype=BF)),
    "lam number": dict(lam=0.5),
    "q_lens type": dict(q_lens=torch.zeros(2, dtype=torch.int64)),
    "k_lens size": dict(k_lens=torch.zeros(3, dtype=torch.int32)),
    "on the CPU": {},
}


@pytest.mark.parametrize("case", BAD)
def test_forward_refuses(case):
    calls = B.launch_count()
    with pytest.raises(ValueError):
        D.diff_attn_fwd(**{**ops(), **BAD[case]})
    with pytest.raises(ValueError):
        D.diff_attn(**{**ops(), **BAD[case]})
    assert B.launch_count() == calls


def test_backward_refuses(monkeypatch):
    monkeypatch.setattr(D, "_check_cuda", lambda t: None)  # the checks behind it run on the CPU too
    o = ops()
    state = dict(O=torch.zeros(2, 4, 9, 64, dtype=BF), O2=torch.zeros(2, 4, 9, 64, dtype=BF),
                 LSE1=torch.zeros(2, 4, 9), LSE2=torch.zeros(2, 4, 9))
    dO = torch.zeros(2, 4, 9, 64, dtype=BF)
    grads = [torch.zeros_like(o[k]) for k in ("Q1", "K1", "Q2", "K2", "V", "lam")]
    for bad in (dict(dO=dO.float()), dict(dO=dO[:, :, :8]), dict(O2=state["O2"].transpose(1, 2).contiguous().transpose(1, 2)),
                dict(LSE1=state["LSE1"].to(BF)), dict(LSE2=state["LSE2"][:1]), dict(need=(False,) * 6),
                dict(need=(True,) * 5), dict(out=grads[:5]), dict(out=[None] * 6),
                dict(out=[grads[1], *grads[1:]]), dict(out=[*grads[:5], torch.zeros(4)]),
                dict(out=[grads[0].expand(2, 4, 9, 64).as_strided((2, 4, 9, 64), (64, 64, 64, 1)), *grads[1:]]),
                dict(dO=dO[:, :, :1].expand(2, 4, 9, 64))):
        with pytest.raises(ValueError):
            D.diff_attn_bwd(**{**o, **state, "dO": dO, **bad})


def paged(**more):
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    c = dict(Q1=z(3, 4, 64), K1=z(10, 16, 2, 64), Q2=z(3, 4, 64), K2=z(10, 16, 2, 64), V=z(10, 16, 2, 128),
             lam=z(4), table=torch.zeros(3, 2, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32))
    return {**c, **more}


@pytest.mark.parametrize("bad", [
    dict(Q1=torch.zeros(3, 4, 1, 64, dtype=BF)), dict(Q1=torch.zeros(3, 4, 64)), dict(Q2=None), dict(K2=None),
    dict(lam=None), dict(lam=torch.zeros(3, dtype=BF)), dict(K1=torch.zeros(10, 16, 3, 64, dtype=BF)),
    dict(V=torch.zeros(9, 16, 2, 128, dtype=BF)), dict(V=torch.zeros(10, 8, 2, 128, dtype=BF)),
    dict(K2=torch.zeros(10, 16, 2, 64, dtype=HF)), dict(table=torch.zeros(3, 2, dtype=torch.int64)),
    dict(table=torch.zeros(2, 2, dtype=torch.int32)), dict(table=torch.zeros(1, 2, dtype=torch.int32).expand(3, 2)),
    dict(lens=None), dict(lens=torch.zeros(3, dtype=torch.int64)), dict(lens=torch.zeros(4, dtype=torch.int32)),
    dict(out=torch.zeros(3, 4, 64, dtype=BF)), dict(out=torch.zeros(1, 4, 128, dtype=BF).expand(3, 4, 128)), {},
])
def test_paged_refuses(bad):
    calls = B.launch_count()
    with pytest.raises(ValueError):
        D.diff_attn_paged(**paged(**bad))
    assert B.launch_count() == calls


def test_one_map_refuses():
    c = paged()
    with pytest.raises(ValueError):
        D.attn_paged(c["Q1"], c["K1"], c["V"], c["table"], c["lens"])       # on the CPU
    with pytest.raises(ValueError):
        D.attn_paged(c["Q1"], c["K1"][..., :32], c["V"], c["table"], c["lens"])


def test_write_refuses():
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    rows, caches, slots = (z(5, 2, 64),), (z(3, 16, 2, 64),), torch.zeros(5, dtype=torch.int64)
    for r, c, s in ((rows, caches, slots), ((), (), slots), (rows * 5, caches * 5, slots), (rows, caches * 2, slots),
                    (rows, caches, slots[:4]), (rows, caches, slots.float()), (rows, (z(3, 16, 1, 64),), slots),
                    (rows, (z(3, 16, 2, 72),), slots), (rows, (z(3, 16, 2, 64).to(HF),), slots),
                    (rows * 2, (z(3, 16, 2, 64), z(4, 16, 2, 64)), slots), ((z(5, 2, 12),), (z(3, 16, 2, 12),), slots),
                    (rows, (z(1, 16, 2, 64).expand(3, 16, 2, 64),), slots)):
        with pytest.raises(ValueError):
            D.paged_write(r, c, s)


def test_extents_past_32_bits_are_refused():
    """Sizes are passed as C ints, which would keep only their low bits."""
    z = lambda *s: torch.empty(*s, dtype=BF, device="meta")  # noqa: E731
    n = (1 << 32) + 8
    o = dict(Q1=z(1, 2, 8, 64), K1=z(1, 2, n, 64), Q2=z(1, 2, 8, 64), K2=z(1, 2, n, 64), V=z(1, 2, n, 64), lam=z(2))
    with pytest.raises(ValueError, match="2\\^31"):
        D.diff_attn_fwd(**o)
    with pytest.raises(ValueError, match="2\\^31"):
        D.attn_paged(z(1, 2, 64), z(n, 16, 2, 64), z(n, 16, 2, 64), z(1, 4).int(), z(1).int())
    with pytest.raises(ValueError, match="table"):
        D.attn_paged(z(1, 2, 64), z(4, 16, 2, 64), z(4, 16, 2, 64), z(1, n).int(), z(1).int())
    with pytest.raises(ValueError, match="2\\^31"):
        D.paged_write((z(n, 2, 64),), (z(4, 16, 2, 64),), z(n).long())


def test_scales_are_read_at_every_call(monkeypatch):
    """A scale passed as a tensor may change between calls: what is kept goes by its value."""
    monkeypatch.setattr(D, "_check_cuda", lambda t: None)
    o, s = ops(), torch.tensor(0.5)
    plan = lambda: D._plan_of(*o.values(), None, None, False, s, s).prob  # noqa: E731
    assert (plan().s1, plan().s2) == (0.5, 0.5)
    s.fill_(0.25)
    assert (plan().s1, plan().s2) == (0.25, 0.25)
    c, kept = paged(), []
    c.update(K1=c["K1"][:0], K2=c["K2"][:0], V=c["V"][:0])     # no pages: nothing is launched
    planned = D._paged_plan
    monkeypatch.setattr(D, "_paged_plan", lambda *k: kept.append(planned(*k)) or kept[-1])
    D.diff_attn_paged(**c, s1=s, s2=s)
    s.fill_(0.125)
    D.diff_attn_paged(**c, s1=s, s2=s)
    assert [(p.prob.s1, p.prob.s2) for p in kept] == [(0.25, 0.25), (0.125, 0.125)]


# ---------------------------------------------------------------- C ABI
def tensor(ptr, b=4096, h=1024, n=64):
    return ctypes.byref(D._Tensor(ptr, b, h, n))


def raw_fwd(prob, **bad):
    a = dict(Q1=tensor(256), K1=tensor(512), Q2=tensor(768), K2=tensor(1024), V=tensor(1280), lam=tensor(2, 0, 1, 0),
             ql=None, kl=None, O=tensor(1536), O2=tensor(1792), L1=B._vp(2048), L2=B._vp(4096))
    a.update(bad)
    return B.lib().streamkl_diff_fwd(ctypes.byref(prob) if prob else None, *a.values(), None)


def problem(**kw):
    c = dict(B=2, H=4, HK=2, NQ=9, NK=12, d=64, dv=64)
    c.update(kw)
    return D.diff_problem(**c)


def test_forward_abi_refuses():
    for bad in (dict(B=0), dict(H=0), dict(HK=0), dict(HK=3), dict(NQ=0), dict(NK=0), dict(s1=math.nan), dict(s2=math.inf),
                dict(NQ=1 << 30), dict(B=1 << 16, H=1 << 16, HK=1)):
        assert raw_fwd(problem(**bad)) == B.EINVAL, bad
    for d, dv in ((64, 256), (128, 64), (96, 96), (256, 256), (0, 0)):
        assert raw_fwd(problem(d=d, dv=dv)) == B.EUNSUPPORTED
    p = problem()
    p.dtype = 2
    assert raw_fwd(p) == B.EUNSUPPORTED
    p = problem()
    p.causal = 3
    assert raw_fwd(p) == B.EINVAL
    assert raw_fwd(None) == B.EINVAL
    for name in ("Q1", "K1", "Q2", "K2", "V", "O", "lam"):
        assert raw_fwd(problem(), **{name: None}) == B.EINVAL
        assert raw_fwd(problem(), **{name: tensor(0)}) == B.EINVAL
    for name in ("Q1", "V", "O", "O2"):
        for layout in (tensor(264), tensor(256, b=0), tensor(256, h=-8), tensor(256, n=68), tensor(256, b=1 << 40)):
            assert raw_fwd(problem(), **{name: layout}) == B.EINVAL
    assert raw_fwd(problem(), O2=tensor(1792, n=128)) == B.EINVAL       # not O's strides
    assert raw_fwd(problem(), L1=None) == B.EINVAL                      # one LSE without the other
    assert raw_fwd(problem(), lam=tensor(2, -1, 1, 0)) == B.EINVAL
    assert raw_fwd(problem(lam_fp32=True), lam=tensor(2, 0, 1, 0)) == B.EINVAL
    assert raw_fwd(problem(), ql=B._vp(3)) == B.EINVAL


def raw_bwd(prob, **bad):
    a = dict(dO=tensor(128), Q1=tensor(256), K1=tensor(512), Q2=tensor(768), K2=tensor(1024), V=tensor(1280),
             lam=tensor(2, 0, 1, 0), O=tensor(1536), O2=tensor(1792), L1=B._vp(2048), L2=B._vp(4096), ql=None, kl=None,
             dQ1=tensor(16), dK1=None, dQ2=None, dK2=None, dV=None, dlam=None, ws=B._vp(1 << 20),
             n=ctypes.c_size_t(1 << 30))
    a.update(bad)
    return B.lib().streamkl_diff_bwd(ctypes.byref(prob), *a.values(), None)


def test_backward_abi_refuses():
    for bad in (dict(dO=None), dict(O=None), dict(O2=None), dict(O2=tensor(1792, b=8192)), dict(L1=None), dict(L2=B._vp(2)),
                dict(dQ1=None), dict(dQ1=tensor(8)), dict(dK1=tensor(16, n=0)), dict(dV=tensor(16, b=4)), dict(dlam=B._vp(1)),
                dict(ws=None), dict(ws=B._vp(64)), dict(n=ctypes.c_size_t(64))):
        assert raw_bwd(problem(), **bad) == B.EINVAL, bad
    assert raw_bwd(problem(d=96)) == B.EUNSUPPORTED
    for nq, rows in ((9, 64), (64, 64), (65, 128)):   # a record of 5 per row of 64, 4 sums per row of 128
        need = 2 * 4 * (rows * 5 + 128 * 4) * 4
        assert 0 <= D.diff_attn_workspace_size(2, 4, 2, nq, 12, 64, 64) - need < 256
    assert D.diff_attn_workspace_size(2, 4, 3, 9, 12, 64, 64) == 0


def test_paged_abi_refuses():
    def call(prob=None, **bad):
        p = dict(B=3, H=4, HK=2, d=64, dv=64, dtype=0, lam_fp32=0, pages=10, page_size=16, max_pages=4, s1=0.0, s2=0.0)
        p.update(prob or {})
        a = dict(Q1=tensor(256), K1=tensor(512), Q2=tensor(768), K2=tensor(1024), V=tensor(1280), lam=tensor(2, 0, 1, 0),
                 table=B._vp(64), ts=4, lens=B._vp(64), O=tensor(1536), ws=B._vp(1 << 20), n=ctypes.c_size_t(1 << 30))
        a.update(bad)
        return B.lib().streamkl_paged_attn(ctypes.byref(D.PagedProblem(*p.values())), *a.values(), None)

    for bad in (dict(B=0), dict(B=2049), dict(H=0), dict(HK=3), dict(pages=0), dict(page_size=0), dict(max_pages=0),
                dict(s1=math.nan), dict(max_pages=1 << 28, page_size=16), dict(B=2048, H=4096, HK=4096, max_pages=1 << 16)):
        assert call(bad) == B.EINVAL, bad
    for bad in (dict(d=64, dv=256), dict(d=32), dict(dtype=5)):
        assert call(bad) == B.EUNSUPPORTED
    for bad in (dict(Q1=None), dict(K1=None), dict(V=None), dict(O=None), dict(K2=None), dict(Q2=None), dict(lam=None),
                dict(table=None), dict(lens=None), dict(ts=3), dict(ws=None), dict(ws=B._vp(16)), dict(table=B._vp(2)),
                dict(K1=tensor(512, n=4)), dict(V=tensor(1288)), dict(Q1=tensor(256, h=0))):
        assert call(**bad) == B.EINVAL, bad


def test_write_abi_refuses():
    def call(n=1, T=5, HK=2, pages=3, page=16, width=64, slots=64, wide=1, row=(256, 0, 64, 128), cache=(512, 2048, 64, 128)):
        rows, caches = (D._Tensor * max(n, 1))(*[D._Tensor(*row)] * max(n, 1)), (D._Tensor * max(n, 1))(*[D._Tensor(*cache)] * max(n, 1))
        return B.lib().streamkl_paged_write(n, rows, caches, (ctypes.c_int * max(n, 1))(*[width] * max(n, 1)), B._vp(slots),
                                            wide, T, HK, pages, page, None)

    for bad in (dict(n=0), dict(n=5), dict(T=0), dict(HK=0), dict(pages=0), dict(page=0), dict(width=12), dict(width=0),
                dict(slots=0), dict(slots=4), dict(wide=2), dict(pages=1 << 20, page=1 << 11), dict(row=(0, 0, 64, 128)), dict(row=(256, 0, 0, 128)),
                dict(cache=(520, 2048, 64, 128)), dict(cache=(512, 2044, 64, 128))):
        assert call(**bad) == B.EINVAL, bad


# ---------------------------------------------------------------- the reference itself
def test_reference_against_differences():
    """The formulas that the GPU tests compare with, against central differences of the definition."""
    g = torch.Generator().manual_seed(3)
    B_, H, HK, NQ, NK, d, dv = 2, 4, 2, 7, 9, 4, 6
    t = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64).to(BF)  # noqa: E731
    x = [t(B_, H, NQ, d), t(B_, HK, NK, d), t(B_, H, NQ, d), t(B_, HK, NK, d), t(B_, HK, NK, dv), t(H)]
    kw = dict(causal=True, q_lens=torch.tensor([7, 5]), k_lens=torch.tensor([9, 4]))
    dO = t(B_, H, NQ, dv)
    grads = Reference(*x, **kw).backward(dO)

    def value(ops):
        # the definition in 64 bits, on operands that are not rounded
        out = 0.0
        for b in range(B_):
            q, k = int(kw["q_lens"][b]), int(kw["k_lens"][b])
            for h in range(H):
                s = h * HK // H
                for i in range(q):
                    n = min(k, i + k - q + 1)
                    if n <= 0:
                        continue
                    P = [torch.softmax(ops[1 + m][b, s, :n] @ ops[m][b, h, i] / math.sqrt(d), 0) for m in (0, 2)]
                    out += float(((P[0] - ops[5][h] * P[1]) @ ops[4][b, s, :n]) @ dO[b, h, i].double())
        return out

    wide = [v.double() for v in x]
    for k, name in enumerate(("dQ1", "dK1", "dQ2", "dK2", "dV", "dlam")):
        way = torch.randn(x[k].shape, generator=g, dtype=torch.float64)
        ends = [value([v + e * way if m == k else v for m, v in enumerate(wide)]) for e in (1e-5, -1e-5)]
        slope = (ends[0] - ends[1]) / 2e-5
        got = float((grads[name][0] * way).sum())
        assert abs(got - slope) <= 1e-7 * max(1.0, abs(slope)), name
