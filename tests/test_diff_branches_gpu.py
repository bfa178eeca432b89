"""Differential attention and the paged forms on the branches that one width or type alone takes."""
import pytest
import torch

import test_paged_gpu as paged
from test_diff_attn_gpu import HF, check, lens_of, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("d,dv", [(64, 128), (128, 128)])
def test_single_gradients(d, dv, causal, which):
    """Each gradient asked for alone equals the one of the full call, bit for bit, in a padded batch."""
    import attention_kl_distillation_b200 as skl
    ops, dO = make(2, 4, 2, 150, 170, d, dv)
    kw = dict(causal=causal, q_lens=lens_of([150, 90]), k_lens=lens_of([170, 64]))
    saved = skl.diff_attn_fwd(*ops, **kw)
    full = skl.diff_attn_bwd(dO, *ops, *saved, **kw)
    one = skl.diff_attn_bwd(dO, *ops, *saved, need=[k == which for k in range(6)], **kw)
    assert [g is not None for g in one] == [k == which for k in range(6)]
    assert torch.equal(one[which], full[which])


@pytest.mark.parametrize("pair", [(0, 2), (1, 3), (0, 4), (2, 5), (1, 4), (3, 4)])
@pytest.mark.parametrize("d,dv", [(128, 128), (128, 256)])
def test_pairs_of_gradients(d, dv, pair):
    import attention_kl_distillation_b200 as skl
    ops, dO = make(1, 4, 2, 150, 170, d, dv, seed=2)
    saved = skl.diff_attn_fwd(*ops, causal=True)
    full = skl.diff_attn_bwd(dO, *ops, *saved, causal=True)
    some = skl.diff_attn_bwd(dO, *ops, *saved, causal=True, need=[k in pair for k in range(6)])
    for k in range(6):
        assert (some[k] is None) if k not in pair else torch.equal(some[k], full[k])


@pytest.mark.parametrize("lam", ["scalar", "head", "row", "batch", "token"])
@pytest.mark.parametrize("d,dv", [(64, 128), (128, 128), (128, 256)])
def test_weights(d, dv, lam):
    """Weights of every shape, their gradients summed over what they are broadcast over, in a padded batch."""
    check(*make(2, 4, 2, 200, 200, d, dv, lam=lam), causal=True, q_lens=[200, 77], k_lens=[200, 77])


@pytest.mark.parametrize("lam", ["head", "row"])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 256)])
def test_one_query_row(d, dv, lam):
    check(*make(3, 4, 2, 1, 150, d, dv, lam=lam), causal=True, q_lens=[1, 0, 1], k_lens=[150, 9, 1])


@pytest.mark.parametrize("d,dv", [(64, 64), (64, 128), (128, 128), (128, 256)])
def test_large_logits_in_fp16(d, dv):
    """Logits over hundreds of nats in both directions: references move between tiles."""
    ops, dO = make(1, 2, 2, 260, 700, d, dv, HF, scale=4.0)
    check(ops, dO, s1=0.5, s2=0.3)
    ramp = torch.linspace(0.1, 6.0, 700, device="cuda").view(1, 1, 700, 1)
    ops[1] = (ops[1].float() * ramp / 4).to(HF)   # every key tile raises the maximum
    check(ops, dO, s1=0.5, causal=False)


@pytest.mark.parametrize("maps", [1, 2])
@pytest.mark.parametrize("d,dv", [(64, 64), (64, 128), (128, 128), (128, 256)])
def test_paged_large_logits_in_fp16(d, dv, maps):
    c = paged.make([900, 1700], 4, 2, d, dv, dtype=HF)
    ramp = torch.linspace(0.1, 8.0, c["K1"].shape[0], device="cuda").view(-1, 1, 1, 1)
    for k in ("K1", "K2"):
        c[k] = (c[k].float() * ramp).to(HF)
    paged.check(c, maps, s1=0.7)
