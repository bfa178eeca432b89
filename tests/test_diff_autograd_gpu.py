"""Differential attention and the paged calls in autograd on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def operands(layout, seed=7):
    """Projections read head by head, or slices of one packed projection; lam every second of its elements."""
    g = torch.Generator().manual_seed(seed)
    B, N, H, d, dv = 2, 140, 4, 64, 128
    if layout == "packed":
        packed = torch.randn(B, N, H, 4 * d + dv + 8, generator=g).to(BF).cuda().transpose(1, 2)
        views = [packed[..., a:a + w] for a, w in ((0, d), (d, d), (2 * d, d), (3 * d, d), (4 * d + 8, dv))]
    else:
        views = [torch.randn(B, N, H, w, generator=g).to(BF).cuda().transpose(1, 2) for w in (d, d, d, d, dv)]
    lam = torch.rand(2 * H, generator=g).to(BF).cuda()[::2]
    dO = torch.randn(B, H, N, dv, generator=g).to(BF).cuda()
    return [t.detach().requires_grad_() for t in (*views, lam)], dO


def offload(pin):
    return torch.autograd.graph.save_on_cpu(pin_memory=pin)


def relayout():
    return torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t.contiguous())


@pytest.mark.parametrize("layout", ["token_major", "packed"])
@pytest.mark.parametrize("hooks", [relayout, lambda: offload(False), lambda: offload(True)],
                         ids=["contiguous", "save_on_cpu", "save_on_cpu_pinned"])
def test_saved_tensors_in_another_layout(layout, hooks):
    """Hooks that give the saved tensors back in another layout leave the gradients as they are, bit for bit."""
    import attention_kl_distillation_b200 as skl
    ops, dO = operands(layout)
    n = torch.tensor([140, 77], dtype=torch.int32, device="cuda")
    step = lambda: skl.diff_attn(*ops, causal=True, s1=0.2, q_lens=n, k_lens=n)  # noqa: E731
    want = torch.autograd.grad(step(), ops, dO)
    with hooks():
        O = step()
    got = torch.autograd.grad(O, ops, dO)
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("maps", [1, 2])
def test_paged_forms_in_a_graph(maps):
    """A query that wants a gradient changes nothing of the output; asking for the gradient raises."""
    import attention_kl_distillation_b200 as skl
    g = torch.Generator().manual_seed(3)
    t = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    Q1, Q2, K1, K2, V, lam = t(2, 4, 64), t(2, 4, 64), t(8, 16, 2, 64), t(8, 16, 2, 64), t(8, 16, 2, 128), t(4)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([64, 33], dtype=torch.int32, device="cuda")

    def call(out=None):
        if maps == 1:
            return skl.attn_paged(Q1, K1, V, table, lens, out=out)
        return skl.diff_attn_paged(Q1, K1, Q2, K2, V, lam, table, lens, out=out)

    want, out = call(), torch.empty(2, 4, 128, dtype=BF, device="cuda")
    Q1.requires_grad_()
    for buffer in (None, out):
        O = call(buffer)
        assert torch.equal(O, want) and O.requires_grad
        with pytest.raises(NotImplementedError):
            O.sum().backward()
    assert torch.equal(out, want) and not out.requires_grad


def test_outputs_over_what_has_been_read():
    """O over Q1, and gradients over O, O2 and lam, are as in places of their own."""
    import attention_kl_distillation_b200 as skl
    g = torch.Generator().manual_seed(9)
    t = lambda h: torch.randn(2, h, 500, 64, generator=g).to(BF).cuda()  # noqa: E731
    ops, dO = [t(8), t(8), t(8), t(8), t(8), torch.rand(8, generator=g).to(BF).cuda()], t(8)
    want = skl.diff_attn_fwd(*ops, causal=True)
    grads = skl.diff_attn_bwd(dO, *ops, *want, causal=True)
    O, O2, L1, L2 = (x.clone() for x in want)
    lam = ops[5].clone()
    new = [torch.empty_like(x) for x in ops[1:4]]
    got = skl.diff_attn_bwd(dO, *ops[:5], lam, O, O2, L1, L2, causal=True, out=[O, *new, O2, lam])
    for a, b in zip(got, grads):
        assert torch.equal(a, b)
    over = ops[0].clone()
    skl.diff_attn_fwd(over, *ops[1:], causal=True, save=False, out=(over, None, None, None))
    assert torch.equal(over, want[0])
    assert skl.query_device_status() == 0


@pytest.mark.parametrize("unpack", ["misaligned", "features_apart", "half_of_them"])
def test_saved_tensors_of_any_layout(unpack):
    """Saved tensors that the kernels cannot read as they come back are copied; lam and dO may be anything."""
    import attention_kl_distillation_b200 as skl
    ops, dO = operands("token_major", seed=8)
    seen = [0]

    def restore(t):
        seen[0] += 1
        if unpack == "misaligned":
            flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
            return flat[1:1 + t.numel()].view(t.shape).copy_(t)
        if unpack == "features_apart":
            return t.transpose(-1, -2).contiguous().transpose(-1, -2) if t.dim() == 4 else t
        return t.contiguous() if seen[0] % 2 else t

    want = torch.autograd.grad(skl.diff_attn(*ops, causal=True), ops, dO)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, restore):
        O = skl.diff_attn(*ops, causal=True)
    got = torch.autograd.grad(O, ops, dO, retain_graph=True)
    again = torch.autograd.grad(O, ops, dO.transpose(2, 3).contiguous().transpose(2, 3))
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    for a, b, c in zip(got, again, want):
        assert torch.equal(a, c) and torch.equal(b, c)
