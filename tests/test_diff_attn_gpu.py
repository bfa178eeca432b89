"""Differential attention on the GPU against its definition in 64 bits: forward, backward, layouts,
lengths, masks that leave rows empty, captured calls."""
import math

import pytest
import torch

from diff_ref import Reference, within

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
WIDTHS = [(64, 64), (64, 128), (128, 128), (128, 256)]


def make(B, H, HK, NQ, NK, d, dv, dtype=BF, seed=0, lam="head", token_major=False, scale=1.0):
    g = torch.Generator().manual_seed(seed)

    def t(h, n, w):
        x = torch.randn(B, n, h, w, generator=g) if token_major else torch.randn(B, h, n, w, generator=g)
        x = (x * scale).to(dtype).cuda()
        return x.transpose(1, 2) if token_major else x

    shape = {"head": (H,), "scalar": (), "row": (B, H, NQ), "batch": (B, 1, 1), "token": (1, 1, NQ)}[lam]
    lam_t = (torch.rand(shape, generator=g) * 1.2 - 0.3).to(dtype).cuda()
    return [t(H, NQ, d), t(HK, NK, d), t(H, NQ, d), t(HK, NK, d), t(HK, NK, dv), lam_t], t(H, NQ, dv)


def lens_of(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda") if values is not None else None


def check(ops, dO, causal=False, s1=None, s2=None, q_lens=None, k_lens=None):
    import attention_kl_distillation_b200 as skl
    ql, kl = lens_of(q_lens), lens_of(k_lens)
    kw = dict(causal=causal, s1=s1, s2=s2, q_lens=ql, k_lens=kl)
    ref = Reference(*ops, causal, s1, s2, ql, kl)
    O, O2, L1, L2 = skl.diff_attn_fwd(*ops, **kw)
    grads = skl.diff_attn_bwd(dO, *ops, O, O2, L1, L2, **kw)
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    within("O", O, ref.O, ref.tol_O)
    within("O2", O2, ref.O_t[1], ref.tol_O2)
    for n, got, want in (("LSE1", L1, ref.LSE[0]), ("LSE2", L2, ref.LSE[1])):
        dead = torch.isinf(want)
        assert torch.equal(torch.isinf(got), dead) and bool((got[dead] < 0).all()), n
        within(n, got[~dead], want[~dead], ref.tol_LSE)
    for (name, (want, tol)), got in zip(ref_order(ref.backward(dO)), grads):
        within(name, got, want, tol)
    return ref, O, grads


def ref_order(d):
    return [(n, d[n]) for n in ("dQ1", "dK1", "dQ2", "dK2", "dV", "dlam")]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_widths_and_types(d, dv, dtype, causal):
    check(*make(2, 2, 2, 200, 200, d, dv, dtype), causal=causal)


@pytest.mark.parametrize("d,dv", [(64, 128), (128, 128)])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("NQ,NK", [(1, 1), (1, 300), (2, 65), (63, 64), (64, 63), (65, 129), (127, 128), (128, 127),
                                   (129, 257), (300, 130), (5, 1000), (513, 700)])
def test_lengths(NQ, NK, d, dv, causal):
    check(*make(1, 2, 1, NQ, NK, d, dv, seed=NQ + NK), causal=causal)


@pytest.mark.parametrize("H,HK", [(4, 1), (6, 2), (8, 8), (16, 2)])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (128, 256)])
def test_shared_key_heads(H, HK, d, dv):
    check(*make(1, H, HK, 150, 210, d, dv, seed=H), causal=True)


@pytest.mark.parametrize("lam", ["scalar", "head", "row", "batch", "token"])
def test_weights(lam):
    check(*make(2, 3, 3, 130, 130, 64, 64, lam=lam), causal=True)


def test_fp32_weight():
    ops, dO = make(2, 2, 2, 100, 100, 64, 128)
    ops[5] = torch.tensor([0.3, -0.7], device="cuda")
    _, _, grads = check(ops, dO)
    assert grads[5].dtype == torch.float32


@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_padded_batch_with_garbage_behind_the_ends(d, dv, causal):
    """Rows behind a sequence's end hold NaN and infinities; outputs and gradients there are 0."""
    ql, kl = [200, 1, 0, 130, 64, 77], [200, 1, 140, 0, 190, 50]
    ops, dO = make(6, 2, 1, 200, 200, d, dv, seed=3)
    clean = [t.clone() for t in ops] + [dO.clone()]
    for b in range(6):
        for t, n in ((ops[0], ql[b]), (ops[2], ql[b]), (dO, ql[b]), (ops[1], kl[b]), (ops[3], kl[b]), (ops[4], kl[b])):
            t[b, :, n:] = math.nan
            t[b, :, n + 3:n + 5] = math.inf
    ref, O, grads = check(ops, dO, causal=causal, q_lens=ql, k_lens=kl)
    dead = ~ref.live.expand(6, 2, 200, 1)
    assert bool((O.masked_select(dead) == 0).all())
    for g, lens in zip(grads[:5], (ql, kl, ql, kl, kl)):
        for b in range(6):
            assert bool((g[b, :, lens[b]:] == 0).all())
    # and what was behind the ends does not matter
    import attention_kl_distillation_b200 as skl
    kw = dict(causal=causal, q_lens=lens_of(ql), k_lens=lens_of(kl))
    saved = skl.diff_attn_fwd(*clean[:6], **kw)
    assert torch.equal(saved[0], O)
    for a, b in zip(skl.diff_attn_bwd(clean[6], *clean[:6], *saved, **kw), grads):
        assert torch.equal(a, b)


def test_lengths_outside_the_tensors_are_cut():
    check(*make(2, 2, 2, 90, 140, 64, 64), q_lens=[-5, 1000], k_lens=[10, 1000])


@pytest.mark.parametrize("d,dv", [(64, 128), (128, 128), (128, 256)])
def test_rows_that_see_no_key(d, dv):
    """Causal with more rows than keys: the first rows see nothing, whatever dO holds there."""
    ops, dO = make(1, 2, 1, 300, 100, d, dv, seed=5)
    dO[:, :, :150] = math.nan
    ref, O, grads = check(ops, dO, causal=True)
    assert bool((O[:, :, :200] == 0).all()) and bool((grads[0][:, :, :200] == 0).all())


@pytest.mark.parametrize("token_major", [False, True], ids=["head_major", "token_major"])
def test_memory_orders(token_major):
    """Projections' [B, N, H, d] layout is taken as it is, and the outputs come in it too."""
    ops, dO = make(2, 4, 2, 140, 160, 64, 128, token_major=token_major)
    _, O, grads = check(ops, dO, causal=True)
    for got, like in zip((O, *grads[:5]), (ops[0], *ops[:5])):
        assert got.transpose(1, 2).is_contiguous() == like.transpose(1, 2).is_contiguous() == token_major


def test_sliced_operands():
    """Operands that are slices of one projection, offset and strided, the value head in the middle."""
    g = torch.Generator().manual_seed(9)
    packed = torch.randn(2, 170, 3, 64 * 4 + 128 + 8, generator=g).to(BF).cuda().transpose(1, 2)
    ops = [packed[..., a:b] for a, b in ((0, 64), (64, 128), (136, 200), (200, 264), (264, 392))]
    lam = torch.full((3,), 0.5, dtype=BF, device="cuda")
    dO = torch.randn(2, 3, 170, 128, generator=g).to(BF).cuda()
    check([ops[0], ops[1], ops[2], ops[3], ops[4], lam], dO, causal=True)


def test_large_logits_and_scales():
    """Logits over hundreds of nats in both directions: references move between tiles."""
    ops, dO = make(1, 2, 2, 260, 700, 64, 64, scale=4.0)
    check(ops, dO, s1=0.5, s2=0.3)
    ramp = torch.linspace(0.1, 6.0, 700, device="cuda").view(1, 1, 700, 1)
    ops[1] = (ops[1].float() * ramp / 4).to(BF)   # every key tile raises the maximum
    check(ops, dO, s1=0.5, causal=False)


def test_identical_maps_and_unit_weight_cancel():
    """With Q1 = Q2, K1 = K2 and lam = 1 the output is 0 exactly: both maps take the same steps."""
    import attention_kl_distillation_b200 as skl
    ops, _ = make(1, 2, 2, 300, 300, 64, 128)
    ops[2], ops[3], ops[5] = ops[0], ops[1], torch.ones(2, dtype=BF, device="cuda")
    assert bool((skl.diff_attn(*ops, causal=True) == 0).all())


def test_zero_weight_is_the_first_map():
    ops, dO = make(1, 2, 2, 200, 200, 64, 64)
    ops[5] = torch.zeros(2, dtype=BF, device="cuda")
    _, _, grads = check(ops, dO)
    assert bool((grads[2] == 0).all()) and bool((grads[3] == 0).all())


@pytest.mark.parametrize("B,NQ,NK", [(0, 5, 5), (2, 0, 5), (2, 5, 0)])
def test_empty_tensors(B, NQ, NK):
    import attention_kl_distillation_b200 as skl
    ops, dO = make(B, 2, 2, NQ, NK, 64, 64)
    saved = skl.diff_attn_fwd(*ops)
    assert saved[0].shape == (B, 2, NQ, 64) and bool((saved[0] == 0).all())
    assert bool(torch.isinf(saved[2]).all())
    for g, t in zip(skl.diff_attn_bwd(dO, *ops, *saved), ops):
        assert g.shape == t.shape and bool((g == 0).all())


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 256)])
def test_single_gradients(which, d, dv):
    """Each gradient asked for alone equals the one of the full call, bit for bit."""
    import attention_kl_distillation_b200 as skl
    ops, dO = make(1, 4, 2, 150, 170, d, dv)
    saved = skl.diff_attn_fwd(*ops)
    full = skl.diff_attn_bwd(dO, *ops, *saved)
    one = skl.diff_attn_bwd(dO, *ops, *saved, need=[k == which for k in range(6)])
    assert [g is not None for g in one] == [k == which for k in range(6)]
    assert torch.equal(one[which], full[which])


def test_more_units_than_multiprocessors_and_repeatability():
    import attention_kl_distillation_b200 as skl
    ops, dO = make(2, 16, 4, 1100, 1100, 64, 128, seed=11)
    kw = dict(causal=True, q_lens=lens_of([1100, 700]), k_lens=lens_of([1100, 700]))
    saved = skl.diff_attn_fwd(*ops, **kw)
    grads = skl.diff_attn_bwd(dO, *ops, *saved, **kw)
    ref = Reference(*ops, True, None, None, kw["q_lens"], kw["k_lens"])
    within("O", saved[0], ref.O, ref.tol_O)
    for (name, (want, tol)), got in zip(ref_order(ref.backward(dO)), grads):
        within(name, got, want, tol)
    again = skl.diff_attn_fwd(*ops, **kw)
    for a, b in zip((*saved, *grads), (*again, *skl.diff_attn_bwd(dO, *ops, *again, **kw))):
        assert torch.equal(a, b)


def test_autograd_and_expanded_upstream():
    import attention_kl_distillation_b200 as skl
    ops, _ = make(2, 4, 2, 120, 120, 64, 64, lam="scalar")
    leaves = [t.clone().requires_grad_() for t in ops]
    O = skl.diff_attn(*leaves, causal=True)
    O.sum().backward()   # an upstream gradient expanded from one number
    want = Reference(*ops, True).backward(torch.ones_like(O))
    for (name, (v, tol)), t in zip(ref_order(want), leaves):
        within(name, t.grad, v, tol)
    with torch.no_grad():
        assert torch.equal(skl.diff_attn(*leaves, causal=True), O)
    only = [t.detach() for t in leaves]
    only[5] = leaves[5]
    (g,) = torch.autograd.grad(skl.diff_attn(*only, causal=True).sum(), [leaves[5]])
    within("dlam", g, *want["dlam"])


def test_gradients_against_differences():
    """The gradient along a direction is the definition's central difference along it."""
    import attention_kl_distillation_b200 as skl
    ops, dO = make(1, 2, 1, 70, 90, 64, 64, seed=21)
    saved = skl.diff_attn_fwd(*ops, causal=True)
    grads = skl.diff_attn_bwd(dO, *ops, *saved, causal=True)
    bounds = Reference(*ops, True).backward(dO)
    g = torch.Generator().manual_seed(5)
    for k, name in enumerate(("dQ1", "dK1", "dQ2", "dK2", "dV", "dlam")):
        way = torch.randn(ops[k].shape, generator=g).double().cuda()
        side = []
        for e in (1e-4, -1e-4):
            moved = [t.double() for t in ops]
            moved[k] = moved[k] + e * way
            side.append(float((definition(*moved) * dO.double()).sum()))
        slope = (side[0] - side[1]) / 2e-4
        got = float((grads[k].double() * way).sum())
        # the gradients' own bounds along the direction, and the difference's truncation
        tol = float((bounds[name][1] * way.abs()).sum()) + 1e-5 * max(1.0, abs(slope))
        assert abs(got - slope) <= tol, (name, got, slope, tol)


def definition(Q1, K1, Q2, K2, V, lam):
    H, d, NQ, NK = Q1.shape[1], Q1.shape[3], Q1.shape[2], K1.shape[2]
    K1, K2, V = (t.repeat_interleave(H // t.shape[1], 1) for t in (K1, K2, V))
    hide = torch.ones(NQ, NK, dtype=torch.bool, device=Q1.device).triu(NK - NQ + 1)
    P1, P2 = (torch.softmax((Q @ K.transpose(2, 3) / math.sqrt(d)).masked_fill(hide, -math.inf), -1)
              for Q, K in ((Q1, K1), (Q2, K2)))
    return (P1 - lam.view(1, -1, 1, 1) * P2) @ V


def test_captured_step_and_two_streams():
    """A captured forward and backward replays on new inputs and lengths; two graphs share a workspace."""
    import attention_kl_distillation_b200 as skl
    ops, dO = make(2, 4, 2, 200, 200, 64, 128, seed=31)
    ql, kl = lens_of([200, 150]), lens_of([200, 150])
    ws = torch.empty(skl.diff_attn_workspace_size(2, 4, 2, 200, 200, 64, 128), dtype=torch.uint8, device="cuda")
    kw = dict(causal=True, q_lens=ql, k_lens=kl)

    def step():
        saved = skl.diff_attn_fwd(*ops, **kw)
        return (saved[0], *skl.diff_attn_bwd(dO, *ops, *saved, workspace=ws, **kw))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
    other, dO2 = make(2, 4, 2, 200, 200, 64, 128, seed=32)
    for t, n in zip(ops, other):
        t.copy_(n)
    dO.copy_(dO2)
    ql.copy_(lens_of([90, 200]))
    kl.copy_(lens_of([120, 200]))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    for a, b in zip(outs[0], step()):
        assert torch.equal(a, b)




def test_two_streams_at_once():
    """Calls on two streams at the same time do not touch each other."""
    import attention_kl_distillation_b200 as skl
    sets = [make(1, 8, 4, 700, 700, 64, 128, seed=41 + k) for k in range(2)]

    def step(ops, dO):
        saved = skl.diff_attn_fwd(*ops, causal=True)
        return (saved[0], *skl.diff_attn_bwd(dO, *ops, *saved, causal=True))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(step(*sets[k]))
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, r))


def test_captured_autograd_step():
    """A training step through autograd, captured with no eager graph of the leaves alive."""
    import attention_kl_distillation_b200 as skl
    ops, dO = make(1, 4, 2, 130, 130, 64, 64, seed=51)
    leaves = [t.requires_grad_() for t in ops]

    def step():
        O = skl.diff_attn(*leaves, causal=True)
        return (O.detach(), *torch.autograd.grad(O, leaves, dO))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for t in out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,dv", [(64, 128), (128, 256)])
def test_a_query_tile_per_multiprocessor(d, dv):
    """Long sequences run one key head at a time: the first and last rows of every head against rows of a
    smaller problem (the last 100 rows see the same keys under the bottom-right causal mask)."""
    import attention_kl_distillation_b200 as skl
    N, H = 148 * 128 + 77, 4
    ops, dO = make(2, H, 2, N, N, d, dv, seed=61)
    saved = skl.diff_attn_fwd(*ops, causal=True)
    dQ1, _, dQ2 = skl.diff_attn_bwd(dO, *ops, *saved, causal=True, need=(True, False, True, False, False, False))[:3]
    assert skl.query_device_status() == 0
    Q1, K1, Q2, K2, V, lam = ops
    for rows, keys in ((slice(0, 100), slice(0, 100)), (slice(N - 100, N), slice(0, N))):
        r = Reference(Q1[:, :, rows], K1[:, :, keys], Q2[:, :, rows], K2[:, :, keys], V[:, :, keys], lam, True)
        within("O", saved[0][:, :, rows], r.O, r.tol_O)
        g = r.backward(dO[:, :, rows])
        within("dQ1", dQ1[:, :, rows], *g["dQ1"])
        within("dQ2", dQ2[:, :, rows], *g["dQ2"])
