"""NaN and infinities in what a row sees come out of the differential and paged calls, of those rows only."""
import math

import pytest
import torch

from diff_ref import Reference, within

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
WIDTHS = [(64, 64), (64, 128), (128, 128), (128, 256)]
N, KEY, ROW = 300, 150, 170


def operands(d, dv, dtype, seed=3):
    g = torch.Generator().manual_seed(seed)
    t = lambda h, w: torch.randn(2, h, N, w, generator=g).to(dtype).cuda()  # noqa: E731
    return [t(4, d), t(2, d), t(4, d), t(2, d), t(2, dv), torch.tensor([0.3, 0.6, 0.9, -0.2], dtype=dtype).cuda()], t(4, dv)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("where", ["Q1", "K1", "Q2", "K2"])
def test_nan_in_a_row_or_key(where, d, dv, causal, dtype):
    """A NaN in a row of Q_t, or in a key of K_t that a row sees, makes that row's O and LSE_t NaN; the other
    map's state and all other rows stay as they are."""
    import attention_kl_distillation_b200 as skl
    ops, dO = operands(d, dv, dtype)
    n = torch.tensor([N, 160], dtype=torch.int32, device="cuda")
    kw = dict(causal=causal, q_lens=n, k_lens=n)
    clean = skl.diff_attn_fwd(*ops, **kw)
    clean_dQ = skl.diff_attn_bwd(dO, *ops, *clean, **kw)
    hit = torch.zeros(2, 4, N, dtype=torch.bool, device="cuda")
    at = {"Q1": 0, "K1": 1, "Q2": 2, "K2": 3}[where]
    if where[0] == "Q":
        ops[at][0, 1, ROW, d - 1] = math.nan
        hit[0, 1, ROW] = True
    else:
        ops[at][:, 1, KEY, 3] = math.nan        # key head 1: query heads 2 and 3, of both sequences
        hit[:, 2:] = (torch.arange(N, device="cuda") >= (KEY if causal else 0)) & \
            (torch.arange(N, device="cuda") < n.view(2, 1, 1))
    got = skl.diff_attn_fwd(*ops, **kw)
    grads = skl.diff_attn_bwd(dO, *ops, *got, **kw)
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    mine, other = (2, 3) if where[1] == "1" else (3, 2)
    touched = [0, mine] if where[1] == "1" else [0, 1, mine]
    for k in range(4):
        if k in touched:
            assert bool(torch.isnan(got[k][hit]).all()), k
            assert torch.equal(got[k][~hit], clean[k][~hit]), k
        else:
            assert torch.equal(got[k], clean[k]), k
    assert torch.equal(skl.diff_attn(*ops, **kw).isnan(), got[0].isnan())
    name = 0 if where[1] == "1" else 2
    assert bool(torch.isnan(grads[name][hit]).all())
    if where[0] == "Q":
        assert torch.equal(grads[name][~hit], clean_dQ[name][~hit])


@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("t", [1, 2])
@pytest.mark.parametrize("sign", [1, -1])
def test_a_score_that_overflows(sign, t, d, dv):
    """A score of +infinity has no softmax; one of -infinity has the weight 0."""
    import attention_kl_distillation_b200 as skl
    ops, dO = operands(d, dv, BF)
    Q, K = ops[2 * t - 2], ops[2 * t - 1]
    Q[..., 0], K[..., 0] = 1.0, 0.0
    K[:, :, KEY, 0] = -1600.0                   # exp(-100) or less: no weight either
    ref = Reference(*ops, True)
    want = ref.backward(dO)
    Q[..., 0] = 3e38
    K[:, :, KEY, 0] = sign * 16.0
    got = skl.diff_attn_fwd(*ops, causal=True)
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    sees = torch.arange(N, device="cuda") >= KEY
    if sign > 0:
        for k in (0, 1 + t):
            assert bool(torch.isnan(got[k][:, :, sees]).all())
            assert bool(torch.isfinite(got[k][:, :, ~sees]).all())
        return
    within("O", got[0], ref.O, ref.tol_O)
    within("O2", got[1], ref.O_t[1], ref.tol_O2)
    for k in (0, 1):
        within("LSE", got[2 + k], ref.LSE[k], ref.tol_LSE)
    grads = skl.diff_attn_bwd(dO, *ops, *got, causal=True)
    for k, name in ((4, "dV"), (5, "dlam")):
        within(name, grads[k], *want[name])


@pytest.mark.parametrize("t", [1, 2])
def test_a_map_without_weights(t):
    """A row whose scores of one map are all -infinity has no weights there: the other map's output is whole."""
    import attention_kl_distillation_b200 as skl
    ops, dO = operands(64, 64, BF)
    Q, K = ops[2 * t - 2], ops[2 * t - 1]
    clean = skl.diff_attn_fwd(*ops, causal=True)
    Q[:, :, 0, 0], K[:, :, 0, 0] = 3e38, -16.0  # row 0 sees key 0 alone
    got = skl.diff_attn_fwd(*ops, causal=True)
    assert bool(torch.isneginf(got[1 + t][:, :, 0]).all())
    lam = ops[5].view(1, 4, 1).float()
    row = got[0][:, :, 0].float()
    if t == 1:
        assert torch.equal(got[1][:, :, 0], clean[1][:, :, 0])
        # one key: O_2 is its values, and the product is rounded once
        assert torch.equal(row, (-lam * clean[1][:, :, 0].float()).to(BF).float())
    else:
        assert bool((got[1][:, :, 0] == 0).all())
        assert torch.equal(row, ops[4][:, :, 0].float().repeat_interleave(2, 1))
    dV, dlam = skl.diff_attn_bwd(dO, *ops, *got, causal=True)[4:]
    assert bool(torch.isfinite(dV).all()) and bool(torch.isfinite(dlam).all())


@pytest.mark.parametrize("d,dv", WIDTHS)
def test_nan_in_values(d, dv):
    import attention_kl_distillation_b200 as skl
    ops, _ = operands(d, dv, BF)
    clean = skl.diff_attn_fwd(*ops)
    ops[4][0, 1, KEY, dv - 1] = math.nan
    got = skl.diff_attn_fwd(*ops)
    for k in (0, 1):
        assert bool(torch.isnan(got[k][0, 2:, :, dv - 1]).all())
        got[k][0, 2:, :, dv - 1] = clean[k][0, 2:, :, dv - 1]
        assert torch.equal(got[k], clean[k])
    assert torch.equal(got[2], clean[2]) and torch.equal(got[3], clean[3])


@pytest.mark.parametrize("maps", [1, 2])
@pytest.mark.parametrize("d,dv", WIDTHS)
@pytest.mark.parametrize("where", ["Q1", "K1", "Q2", "K2", "V", "inf"])
def test_paged(where, d, dv, maps):
    """The same of the paged forms, in sequences that lie in one stretch or in many."""
    import attention_kl_distillation_b200 as skl
    if maps == 1 and where[1:] == "2":
        return
    g = torch.Generator().manual_seed(5)
    lens, page, H, HK = [4000, 9, 70], 16, 8, 2
    held = [(x + page - 1) // page for x in lens]
    table = torch.zeros(3, max(held), dtype=torch.int32)
    order, at = torch.randperm(sum(held), generator=g).int(), 0
    for b, x in enumerate(held):
        table[b, :x] = order[at:at + x]
        at += x
    c = {k: torch.randn(sum(held), page, HK, w, generator=g).to(BF).cuda() for k, w in (("K1", d), ("K2", d), ("V", dv))}
    q = {k: torch.randn(3, H, d, generator=g).to(BF).cuda() for k in ("Q1", "Q2")}
    n, lam = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.rand(H, generator=g).to(BF).cuda()

    def call():
        if maps == 1:
            return skl.attn_paged(q["Q1"], c["K1"], c["V"], table.cuda(), n)
        return skl.diff_attn_paged(q["Q1"], c["K1"], q["Q2"], c["K2"], c["V"], lam, table.cuda(), n)

    clean = call()
    hit = torch.zeros(3, H, dv, dtype=torch.bool, device="cuda")
    for b in (0, 2):
        p, r = int(table[b, 40 // page]), 40 % page
        if where[0] == "Q":
            q[where][b, 5, d - 1] = math.nan
            hit[b, 5] = True
        elif where[0] == "K":
            c[where][p, r, 1, 2] = math.nan
            hit[b, 4:] = True
        elif where == "V":
            c["V"][p, r, 1, dv - 1] = math.nan
            hit[b, 4:, dv - 1] = True
        else:
            q["Q1"][b, 5] = 0.0
            q["Q1"][b, 5, 0] = 3e38
            c["K1"][p, r, 1, 0] = 16.0
            hit[b, 5] = True
    got = call()
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    assert bool(torch.isnan(got[hit]).all())
    if where != "inf":
        assert torch.equal(got[~hit], clean[~hit])
    else:
        assert bool(torch.isfinite(got[~hit]).all())
