"""fp16 holds weights far below a row's largest, and gradients of diffuse rows: differential attention and the
paged forms in fp16 against the definition in 64 bits, with bounds that allow less than half a step of fp16's
smallest number per weight.

Bounds (u = 2^-11, half a step of fp16; c = Reference's bound of a weight's relative error in fp32 and of the
hardware exponential): a weight relative to the row's sum is off by u + c of itself (paged: u^2 + c, its rounding's
remainder goes in too) or by 2^-36: weights are kept relative to a reference that puts the row's largest at 2^11 or
above, where half of fp16's smallest step, 2^-25, is 2^-36 of it and the row's sum is no less than that largest
weight. Outputs are rounded once more: u of the value, or 2^-25.
"""
import math

import pytest
import torch

from diff_ref import FLUSH, Reference, group_sum, within

pytestmark = pytest.mark.gpu

HF = torch.float16
WIDTHS = [(64, 64), (64, 128), (128, 128), (128, 256)]


def sink(N, H, HK, d, dv, gaps, at, seed=0):
    """One token's queries [H, d], keys [HK, N, d] and values of two maps: key `at` scores gaps[t] nats above
    the others and has the value 0, so that the outputs are what the others' small weights make them."""
    g = torch.Generator().manual_seed(seed)
    s = 1 / math.sqrt(d)
    Q, K = [], []
    for gap in gaps:
        q, k = torch.randn(H, d, generator=g) * 0.3, torch.randn(HK, N, d, generator=g)
        q[:, 0], k[:, :, 0], k[:, at] = 16.0, 0.0, 0.0
        k[:, at, 0] = gap / 16.0 / s
        Q.append(q.to(HF).cuda())
        K.append(k.to(HF).cuda())
    V = (1 + 0.25 * torch.randn(HK, N, dv, generator=g)) * 2000
    V[:, at] = 0.0
    return Q, K, V.to(HF).cuda()


def bound(r, factors):
    low = (2.0 ** -36 + FLUSH) * (r.seen.double() @ r.V.abs())
    e = [(r.u ** factors + r.c) * (P @ r.V.abs()) + low for P in r.P]
    return (e[0] + r.lam.abs() * e[1]) * (1 + r.u) + r.u * r.O.abs() + 2.0 ** -25


@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("gaps", [(12.0, 14.0), (16.0, 13.0), (18.0, 17.0), (20.0, 3.0)])
@pytest.mark.parametrize("at", [0, 130, 2998])
def test_forward_weights_far_below_the_largest(at, gaps, d, dv):
    import attention_kl_distillation_b200 as skl
    Q, K, V = sink(3000, 4, 2, d, dv, gaps, at)
    rows = 140
    Q1, Q2 = (q[None, :, None].expand(1, 4, rows, d).contiguous() for q in Q)
    lam = torch.tensor([0.5, -0.25, 2.0, 0.0], dtype=HF, device="cuda")
    ops = (Q1, K[0][None], Q2, K[1][None], V[None], lam)
    r = Reference(*ops)
    O, _, L1, L2 = skl.diff_attn_fwd(*ops)
    assert skl.query_device_status() == 0
    within("O", O, r.O, bound(r, 1))
    for got, want in ((L1, r.LSE[0]), (L2, r.LSE[1])):
        within("LSE", got, want, r.tol_LSE)


def test_forward_very_large_scores():
    """Scores of 2^27 and more, whose rounding in 32 bits is many nats: weights stay finite, whichever way they round."""
    import attention_kl_distillation_b200 as skl
    g = torch.Generator().manual_seed(1)
    t = lambda h: (torch.randn(1, h, 1000, 64, generator=g) * 12000).to(HF).cuda()  # noqa: E731
    ops = (t(4), t(4), t(4), t(4), torch.randn(1, 4, 1000, 64, generator=g).to(HF).cuda(), torch.ones(4, dtype=HF).cuda())
    for O in skl.diff_attn_fwd(*ops)[:2]:
        assert bool(torch.isfinite(O).all())


def paged(K, V, lens, page=32):
    """Whole sequences' keys and values [HK, N, width] in pages, the same for every sequence."""
    N = V.shape[1]
    per = (N + page - 1) // page
    table = torch.arange(per - 1, -1, -1, dtype=torch.int32, device="cuda").expand(len(lens), per).contiguous()

    def cache(t):
        c = torch.zeros(per * page, t.shape[0], t.shape[2], dtype=HF, device="cuda")
        c[:N] = t.transpose(0, 1)
        return c.view(per, page, *c.shape[1:]).flip(0).contiguous()

    return cache(K[0]), cache(K[1]), cache(V), table, torch.tensor(lens, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("gaps", [(12.0, 14.0), (16.0, 13.0), (18.0, 17.0), (20.0, 3.0)])
@pytest.mark.parametrize("at", [0, 130, 2998])
@pytest.mark.parametrize("maps", [1, 2])
def test_paged_weights_far_below_the_largest(maps, at, gaps, d, dv):
    import attention_kl_distillation_b200 as skl
    Q, K, V = sink(3000, 8, 2, d, dv, gaps, at)
    K1, K2, Vc, table, lens = paged(K, V, [3000, 3000, 2999])
    Q1, Q2 = (q.expand(3, 8, d).contiguous() for q in Q)
    lam = torch.linspace(-0.5, 2.0, 8).to(HF).cuda()
    if maps == 1:
        got = skl.attn_paged(Q1, K1, Vc, table, lens)
    else:
        got = skl.diff_attn_paged(Q1, K1, Q2, K2, Vc, lam, table, lens)
    assert skl.query_device_status() == 0
    for b in range(3):      # equal sequences are cut at different tokens: each against the definition
        n = int(lens[b])
        r = Reference(Q1[b].view(1, 8, 1, d), K[0][None, :, :n], Q2[b].view(1, 8, 1, d), K[1][None, :, :n], V[None, :, :n],
                      lam if maps == 2 else torch.zeros((), dtype=HF, device="cuda"))
        within("O", got[b], r.O[0, :, 0], bound(r, 2)[0, :, 0])


@pytest.mark.parametrize("maps", [1, 2])
def test_paged_very_large_scores(maps):
    import attention_kl_distillation_b200 as skl
    g = torch.Generator().manual_seed(1)
    t = lambda *s: (torch.randn(*s, generator=g) * 12000).to(HF).cuda()  # noqa: E731
    K1, K2, Vc, table, lens = paged([t(4, 3000, 64) for _ in range(2)], t(4, 3000, 64) / 12000, [3000, 1500])
    Q1, Q2 = t(2, 4, 64), t(2, 4, 64)
    got = skl.attn_paged(Q1, K1, Vc, table, lens) if maps == 1 else \
        skl.diff_attn_paged(Q1, K1, Q2, K2, Vc, torch.ones(4, dtype=HF).cuda(), table, lens)
    assert bool(torch.isfinite(got).all())


def dv_bound(r, dO, lam_max):
    """dV and its bound, with chains of additions as the kernels have them."""
    u, eps = r.u, 2.0 ** -23
    amp = max(float((Q.abs() @ K.abs().transpose(2, 3)).max()) * x for Q, K, x in zip(r.Q, r.K, r.s))
    c = eps * ((r.d + 4) * amp + r.NK / 128 + 40 + 16)
    dO = torch.where(r.rows, dO.double(), 0.0)
    A = r.P[0] - r.lam * r.P[1]
    e = torch.where(r.seen, u * A.abs() + c * (r.P[0] + r.lam.abs() * r.P[1]) + 2.0 ** -38 * (1 + lam_max)
                    + FLUSH * (1 + r.lam.abs()), 0.0)
    v = group_sum(A.transpose(2, 3) @ dO, r.HK)
    e = group_sum(e.transpose(2, 3) @ dO.abs() + r.NQ * eps * (A.abs().transpose(2, 3) @ dO.abs()), r.HK)
    return v, e * (1 + u) + u * v.abs() + 2.0 ** -25


@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("NK", [20001, 200001])
def test_value_gradient_of_diffuse_rows(NK, d, dv):
    """Rows that spread over very many keys: A is below fp16's normal numbers, the same for a whole row in the
    first heads (so that its rounding does not average out)."""
    import attention_kl_distillation_b200 as skl
    g = torch.Generator(device="cuda").manual_seed(5)
    t = lambda h, n, w, x: (torch.randn(1, h, n, w, generator=g, device="cuda") * x).to(HF)  # noqa: E731
    ops = [t(2, 70, d, 0.5), t(1, NK, d, 0.5), t(2, 70, d, 0.5), t(1, NK, d, 0.5), t(1, NK, dv, 1.0),
           torch.tensor([0.37, -0.21], dtype=HF, device="cuda")]
    ops[0][:, 0], ops[2][:, 0] = 0.0, 0.0
    dO = t(2, 70, dv, 1000.0)
    saved = skl.diff_attn_fwd(*ops)
    dV = skl.diff_attn_bwd(dO, *ops, *saved, need=(False,) * 4 + (True, False))[4]
    assert skl.query_device_status() == 0
    within("dV", dV, *dv_bound(Reference(*ops), dO, 0.37))


@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("weights", ["large", "rows", "late", "zero"])
def test_value_gradient_of_any_weight(weights, d, dv):
    """Weights past fp16's range, and weights of very different size in one key head's rows."""
    import attention_kl_distillation_b200 as skl
    g = torch.Generator(device="cuda").manual_seed(6)
    t = lambda h, n, w, x: (torch.randn(2, h, n, w, generator=g, device="cuda") * x).to(HF)  # noqa: E731
    n = torch.tensor([333, 200], dtype=torch.int32, device="cuda")
    lam = {"large": torch.tensor([2.0e5, -3.0, 0.5, 1.0e5], device="cuda"), "zero": torch.zeros((), device="cuda"),
           "rows": torch.randn(2, 4, 333, generator=g, device="cuda") * 0.1,
           "late": torch.randn(2, 4, 333, generator=g, device="cuda") * 0.1}[weights]
    if weights == "rows":
        lam[0, 1, 65], lam[1, 3, 199] = -1000.0, 70.0
        lam[1, :, 200:] = math.nan                # behind the end
    if weights == "late":
        lam[:, 3, -1] = 5.0e4                     # the last row: every key tile's
    big = float(lam.nan_to_num(0.0).abs().max())
    ops = [t(4, 333, d, 1.5), t(2, 333, d, 1.0), t(4, 333, d, 1.5), t(2, 333, d, 1.0), t(2, 333, dv, 0.01), lam]
    dO = t(4, 333, dv, 0.001)
    kw = dict(causal=True, q_lens=n, k_lens=n)
    saved = skl.diff_attn_fwd(*ops, **kw)
    dV = skl.diff_attn_bwd(dO, *ops, *saved, **kw)[4]
    assert skl.query_device_status() == 0
    r = Reference(*ops[:5], lam.nan_to_num(0.0), **kw)
    within("dV", dV, *dv_bound(r, dO, big))


def test_a_row_of_infinite_weight_hides_no_other():
    """One row whose weight overflows: keys that it does not see, in other tiles, keep their gradients."""
    import attention_kl_distillation_b200 as skl
    g = torch.Generator(device="cuda").manual_seed(6)
    t = lambda w, x: (torch.randn(1, 2, 400, w, generator=g, device="cuda") * x).to(HF)  # noqa: E731
    lam = torch.rand(1, 2, 400, generator=g, device="cuda")
    lam[0, 0, 100] = 1e30
    ops, dO = [t(64, 1.0), t(64, 1.0), t(64, 1.0), t(64, 1.0), t(64, 1.0), lam], t(64, 1.0)
    saved = [x.nan_to_num(0.0, 0.0, 0.0) for x in skl.diff_attn_fwd(*ops, causal=True)]
    dV = skl.diff_attn_bwd(dO, *ops, *saved, causal=True)[4]
    assert not bool(torch.isfinite(dV[0, 0, 0]).any())          # key 0 is seen by row 100
    tame = lam.clone()
    tame[0, 0, 100] = 0.0                                       # as far as later keys go, the row is not there
    r = Reference(*ops[:5], tame, True)
    v, tol = dv_bound(r, dO, 2.0 ** 20)
    within("dV", dV[:, :, 128:], v[:, :, 128:], tol[:, :, 128:])
