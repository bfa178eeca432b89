"""CPU tests of how the differential and paged calls stand in autograd, with the launches replaced by a
record of what the library would get."""
import ctypes

import pytest
import torch

from attention_kl_distillation_b200 import diff as D

BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as lists of arguments, structs of tensors as (pointer, strides)."""
    made = []

    def run(fn, where, device, *args):
        made.append((where, [args[0], *(D._Tensor.from_address(a) if isinstance(a, int) and a in kept else a
                                        for a in args[1:])]))

    kept, at = set(), D._Structs.at

    def structs(self, pointers):
        block, addresses = at(self, pointers)
        kept.update(a for a in addresses if a)
        made.append(block)     # alive as long as the record
        return block, addresses

    monkeypatch.setattr(D, "_check_cuda", lambda device: None)
    monkeypatch.setattr(D, "_run", run)
    monkeypatch.setattr(D._Structs, "at", structs)
    return lambda where: [a for entry in made if isinstance(entry, tuple) and entry[0] == where for a in [entry[1]]]


def operands(sliced):
    """Projections read head by head, or slices of one packed projection."""
    B, N, H, d, dv = 2, 9, 4, 64, 128
    if sliced:
        packed = torch.zeros(B, N, H, 4 * d + dv + 8, dtype=BF).transpose(1, 2)
        views = [packed[..., a:a + w] for a, w in ((0, d), (d, d), (2 * d, d), (3 * d, d), (4 * d + 8, dv))]
    else:
        views = [torch.zeros(B, N, H, w, dtype=BF).transpose(1, 2) for w in (d, d, d, d, dv)]
    return [t.detach().requires_grad_() for t in views] + [torch.zeros(2 * H, dtype=BF)[::2].detach().requires_grad_()]


@pytest.mark.parametrize("sliced", [False, True], ids=["token_major", "packed"])
@pytest.mark.parametrize("unpack", [lambda t: t, lambda t: t.contiguous(), lambda t: t.clone()],
                         ids=["as_saved", "contiguous", "clone"])
def test_backward_takes_the_layout_of_what_was_saved(calls, sliced, unpack):
    """Hooks on saved tensors (offloading, compression) may give back tensors of another layout: addresses
    and strides that reach the library belong to the same tensors."""
    ops, back = operands(sliced), []

    def restore(t):
        t = unpack(t)
        back.append(t)
        return t

    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, restore):
        O = D.diff_attn(*ops, causal=True)
    torch.autograd.grad(O, ops, torch.zeros_like(O))
    (args,) = calls("streamkl_diff_bwd")
    given = {t.data_ptr(): t for t in back}
    for place, like in zip(args[2:8], ops):       # Q1, K1, Q2, K2, V, lam
        assert place.ptr in given
        t = given[place.ptr]
        assert t.shape == like.shape
        want = t.stride()[:-1] if t.dim() == 4 else (0, t.stride(0), 0)
        assert (place.b, place.h, place.n) == want


def off_by_one_element(t):
    """The same values in memory that starts 2 bytes behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype)
    at = flat[1:1 + t.numel()].view(t.shape)
    return at.copy_(t)


def features_apart(t):
    return t.transpose(-1, -2).contiguous().transpose(-1, -2) if t.dim() == 4 else t


def only_small_offsets(t):
    """A hook that treats some tensors and not others."""
    only_small_offsets.calls += 1
    return t.contiguous() if only_small_offsets.calls % 2 else t


@pytest.mark.parametrize("unpack", [off_by_one_element, features_apart, only_small_offsets])
def test_backward_takes_saved_tensors_of_any_layout(calls, unpack):
    """What the kernels cannot read as it lies is copied, as dO is."""
    only_small_offsets.calls = 0
    ops = operands(False)
    for k, t in enumerate(ops):
        t.data.copy_(torch.arange(t.numel()).view(t.shape) % 251 + k)

    def restore(t):
        return unpack(t) if t.dtype == BF else t

    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, restore):
        O = D.diff_attn(*ops, causal=True)
    torch.autograd.grad(O, ops, torch.zeros_like(O))
    (args,) = calls("streamkl_diff_bwd")
    for place, like in zip(args[2:7], ops):
        assert place.ptr % 16 == 0 and all(s % 8 == 0 for s in (place.b, place.h, place.n))
    O_at, O2_at = args[8], args[9]
    assert (O_at.b, O_at.h, O_at.n) == (O2_at.b, O2_at.h, O2_at.n)


def test_forward_mode_is_refused(calls):
    """A tangent is not dropped: the call raises, as streamkl's does."""
    ops = [t.detach() for t in operands(False)]
    for k in range(6):
        with torch.autograd.forward_ad.dual_level():
            dual = [torch.autograd.forward_ad.make_dual(t, torch.ones_like(t)) if j == k else t for j, t in enumerate(ops)]
            with pytest.raises(NotImplementedError):
                D.diff_attn(*dual)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                D.diff_attn(*dual)
            assert not D.diff_attn(*ops).requires_grad      # no operand has a tangent
    assert len(calls("streamkl_diff_fwd")) > 0


def paged():
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    return dict(Q1=z(3, 4, 64), K1=z(0, 16, 2, 64), Q2=z(3, 4, 64), K2=z(0, 16, 2, 64), V=z(0, 16, 2, 128),
                lam=z(4), table=torch.zeros(3, 2, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("name", ["Q1", "K1", "Q2", "K2", "V", "lam"])
@pytest.mark.parametrize("own", [False, True], ids=["new", "out"])
def test_paged_forms_refuse_gradients(calls, name, own):
    """Where an operand wants a gradient the output does too, and asking for it raises. (Caches without pages:
    nothing is launched.)"""
    c = paged()
    c[name].requires_grad_()
    out = torch.ones(3, 4, 128, dtype=BF) if own else None
    one = lambda **k: D.attn_paged(c["Q1"], c["K1"], c["V"], c["table"], c["lens"], **k)  # noqa: E731
    for call in (lambda **k: D.diff_attn_paged(**c, **k), one):
        if call is one and name in ("Q2", "K2", "lam"):
            continue
        for _ in range(2):      # a buffer is used again and again
            O = call(out=out)
            assert O.requires_grad and bool((O == 0).all())
            if own:
                assert O.data_ptr() == out.data_ptr() and not out.requires_grad
            with pytest.raises(NotImplementedError):
                O.sum().backward()
        with torch.no_grad():
            O = call(out=out)
            assert not O.requires_grad and (out is None or O is out)
        with torch.autograd.forward_ad.dual_level():
            d = {**c, name: torch.autograd.forward_ad.make_dual(c[name].detach(), torch.ones_like(c[name]))}
            with pytest.raises(NotImplementedError):
                D.diff_attn_paged(**d)
    c[name].requires_grad_(False)
    O = D.diff_attn_paged(**c, out=out)
    assert not O.requires_grad and (out is None or O is out)


def test_public_names_follow_the_binding(monkeypatch):
    """A function replaced in the binding is the one that the package gives, also after its first use."""
    import attention_kl_distillation_b200 as skl
    from attention_kl_distillation_b200 import binding
    assert skl.fwd is binding.fwd and skl.diff_attn is D.diff_attn
    monkeypatch.setattr(binding, "fwd", lambda *a: 7)
    monkeypatch.setattr(D, "diff_attn", lambda *a: 8)
    assert skl.fwd() == 7 and skl.diff_attn() == 8


def test_outputs_in_one_place_are_refused(calls):
    """Two outputs in one place, or an output over an operand that other blocks still read, would be a race."""
    B, H, N, d = 2, 4, 9, 64
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    ops = [z(B, H, N, d) for _ in range(5)] + [z(H)]
    O, O2, L1, L2 = z(B, H, N, d), z(B, H, N, d), torch.zeros(B, H, N), torch.zeros(B, H, N)
    for out in ((O, O, L1, L2), (O, O2, L1, L1), (ops[1], O2, L1, L2), (ops[3], O2, L1, L2), (O, ops[4], L1, L2)):
        with pytest.raises(ValueError, match="one place"):
            D.diff_attn_fwd(*ops, out=out)
    for K in (1, 3, 4):
        with pytest.raises(ValueError, match="one place"):
            D.diff_attn_fwd(*ops, save=False, out=(ops[K], None, None, None))
    dO, grads = z(B, H, N, d), [z(B, H, N, d) for _ in range(5)] + [z(H)]
    for k in range(5):
        for other in [*(g for j, g in enumerate(grads[:5]) if j != k), *ops[:5], dO]:
            out = list(grads)
            out[k] = other
            with pytest.raises(ValueError, match="one place"):
                D.diff_attn_bwd(dO, *ops, O, O2, L1, L2, out=out)
    assert not calls("streamkl_diff_fwd") and not calls("streamkl_diff_bwd")
    D.diff_attn_fwd(*ops, out=(O, O2, L1, L2))
    D.diff_attn_fwd(*ops, out=(ops[0], O2, L1, L2))      # over Q: a block reads its rows before it writes them
    D.diff_attn_bwd(dO, *ops, O, O2, L1, L2, out=grads)
    same = ops[:2] + ops[:2] + ops[4:]                   # operands may be the same
    D.diff_attn_bwd(dO, *same, O, O2, L1, L2, out=grads)
    D.diff_attn_bwd(dO, *ops, O, O2, L1, L2, out=[O, *grads[1:4], O2, ops[5]])   # read before the passes begin
    assert len(calls("streamkl_diff_fwd")) == 2 and len(calls("streamkl_diff_bwd")) == 3

    cache, rows, slots = z(3, 16, 2, 64), z(5, 2, 64), torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="one place"):
        D.paged_write((rows, rows), (cache, cache), slots)
    D.paged_write((rows, rows), (cache, z(3, 16, 2, 64)), slots)
    assert len(calls("streamkl_paged_write")) == 1
