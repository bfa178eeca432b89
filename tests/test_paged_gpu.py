"""Single-token attention over paged caches on the GPU against its definition in 64 bits, and the write of
new rows into the pages."""
import math

import pytest
import torch

from diff_ref import Reference, paged_reference, within

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
WIDTHS = [(64, 64), (64, 128), (128, 128), (128, 256)]


def make(lens, H, HK, d, dv, page=16, dtype=BF, seed=0, spare=2, head_major=False, fill=None):
    """Queries, caches, table and lens; what no sequence holds is `fill` where given."""
    g = torch.Generator().manual_seed(seed)
    held = [(n + page - 1) // page for n in lens]
    pages = sum(held) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(max(held), 1)), -1, dtype=torch.int32)
    used = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n].int()
        for k in range(n):
            used[order[at + k], :min(page, lens[b] - k * page)] = True
        at += n

    def cache(w):
        t = torch.randn(pages, page, HK, w, generator=g).to(dtype)
        if fill is not None:
            t[~used] = fill
        t = t.cuda()
        return t.transpose(1, 2).contiguous().transpose(1, 2) if head_major else t

    q = [torch.randn(len(lens), H, d, generator=g).to(dtype).cuda() for _ in range(2)]
    lam = (torch.rand(H, generator=g) * 1.2 - 0.3).to(dtype).cuda()
    return dict(Q1=q[0], K1=cache(d), Q2=q[1], K2=cache(d), V=cache(dv), lam=lam, table=table.cuda(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def run(c, maps, **kw):
    import attention_kl_distillation_b200 as skl
    if maps == 1:
        return skl.attn_paged(c["Q1"], c["K1"], c["V"], c["table"], c["lens"], s=kw.pop("s1", None), **kw)
    return skl.diff_attn_paged(c["Q1"], c["K1"], c["Q2"], c["K2"], c["V"], c["lam"], c["table"], c["lens"], **kw)


def reference(c, maps, **kw):
    two = maps == 2
    return paged_reference(c["Q1"], c["K1"], c["Q2"] if two else None, c["K2"] if two else None, c["V"],
                           c["lam"] if two else None, c["table"].clamp(min=0), c["lens"], s1=kw.get("s1"))


def check(c, maps, **kw):
    import attention_kl_distillation_b200 as skl
    got = run(c, maps, **kw)
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    within("O", got, *reference(c, maps, **kw))
    return got


@pytest.mark.parametrize("maps", [1, 2])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d,dv", WIDTHS)
def test_widths_and_types(d, dv, dtype, maps):
    check(make([1, 700, 16, 0, 129, 64], 8, 2, d, dv, dtype=dtype), maps)


@pytest.mark.parametrize("maps", [1, 2])
@pytest.mark.parametrize("page", [1, 3, 16, 48, 100, 256])
def test_page_sizes(page, maps):
    """Pages that end inside a tile, hold several tiles, or a single row."""
    check(make([257, 1, 100, 640], 4, 4, 64, 128, page=page, seed=page), maps)


@pytest.mark.parametrize("maps", [1, 2])
@pytest.mark.parametrize("H,HK", [(1, 1), (3, 1), (8, 1), (9, 1), (32, 2), (40, 8)])
def test_shared_key_heads(H, HK, maps):
    check(make([300, 77], H, HK, 64, 64, seed=H), maps)
    check(make([300, 77], H, HK, 128, 256, seed=H), maps)


@pytest.mark.parametrize("maps", [1, 2])
@pytest.mark.parametrize("lens", [[5000], [20000, 3], [40] * 300, [0, 0, 9, 0], [0, 0], [16384, 1, 16384]])
def test_uneven_batches(lens, maps):
    """One long sequence over every multiprocessor, many short ones, empty ones anywhere."""
    got = check(make(lens, 4, 2, 128, 128, page=64, seed=len(lens)), maps)
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((got[b] == 0).all())


@pytest.mark.parametrize("d,dv,maps", [(64, 64, 1), (64, 128, 2), (128, 128, 2), (128, 256, 2)])
def test_largest_batch(d, dv, maps):
    """The most sequences a call takes, most of them short or empty."""
    lens = [(7 * k) % 40 if k % 3 else 0 for k in range(2048)]
    c = make(lens, 2, 1, d, dv, page=8)
    import attention_kl_distillation_b200 as skl
    got = run(c, maps)
    assert skl.query_device_status() == 0
    pick = torch.tensor([0, 1, 2, 5, 777, 1024, 2045, 2046, 2047], device="cuda")
    part = {**c, **{k: c[k][pick] for k in ("Q1", "Q2", "table", "lens")}}
    within("O", got[pick], *reference(part, maps))
    assert bool((got[c["lens"] == 0] == 0).all()) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("maps", [1, 2])
def test_what_no_sequence_holds_does_not_matter(maps):
    check(make([33, 500, 0, 129], 8, 4, 64, 128, page=24, fill=math.nan), maps)


@pytest.mark.parametrize("maps", [1, 2])
def test_memory_orders(maps):
    """Caches whose pages hold head after head, and sliced queries and outputs."""
    c = make([200, 70], 8, 4, 128, 128, head_major=True)
    wide = torch.zeros(2, 8, 264, dtype=BF, device="cuda")
    wide[..., 8:136] = c["Q1"]
    c["Q1"] = wide[..., 8:136]
    out = torch.full((2, 16, 128), 7.0, dtype=BF, device="cuda")[:, ::2]
    got = check(c, maps, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert bool((out._base[:, 1::2] == 7).all())


@pytest.mark.parametrize("maps", [1, 2])
def test_large_logits(maps):
    c = make([900, 1700], 4, 2, 64, 64)
    ramp = torch.linspace(0.1, 8.0, c["K1"].shape[0], device="cuda").view(-1, 1, 1, 1)
    for k in ("K1", "K2"):
        c[k] = (c[k].float() * ramp).to(BF)
    check(c, maps, s1=0.7)


def test_weights():
    c = make([100, 40], 4, 2, 64, 64)
    for lam in (torch.tensor(0.4, device="cuda"), torch.rand(2, 4, device="cuda", dtype=torch.float32).to(BF),
                torch.rand(2, 1, device="cuda"), torch.rand(4, device="cuda")):
        c["lam"] = lam
        check(c, 2)


def test_bad_pages_and_lengths_are_reported_and_left_out():
    """An entry outside the cache is not followed; its tokens are left out and the status word says so."""
    import attention_kl_distillation_b200 as skl
    from attention_kl_distillation_b200 import binding
    c = make([64, 40], 4, 2, 64, 64)
    clean = run(c, 2)
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    good = c["table"].clone()
    c["table"][0, 1] = c["K1"].shape[0]
    c["table"][0, 2] = -7
    got = run(c, 2)
    torch.cuda.synchronize()
    assert skl.query_device_status() == binding.EDEVICE
    assert torch.equal(got[1], clean[1])
    # the same as a sequence without those tokens
    c["table"] = good.clone()
    c["table"][0, 1] = good[0, 3]
    c["lens"][0] = 32
    want, tol = reference(c, 2)
    within("O", got, want, tol)
    c["table"], c["lens"] = good, torch.tensor([64, 100000], dtype=torch.int32, device="cuda")
    c["table"][1, 3] = c["table"][1, 0]
    got = run(c, 2)
    torch.cuda.synchronize()
    assert skl.query_device_status() == binding.EDEVICE
    c["lens"][1] = 64
    within("O", got, *reference(c, 2))


def test_captured_steps_follow_growing_lengths():
    """A decode step as it is used: the new rows are written, then attended to, captured once and replayed
    while the sequences grow over page borders; two graphs share one workspace."""
    import attention_kl_distillation_b200 as skl
    page, H, HK, d, dv, B = 16, 4, 2, 64, 128, 3
    g = torch.Generator().manual_seed(1)
    caches = [torch.zeros(30, page, HK, w, dtype=BF, device="cuda") for w in (d, d, dv)]
    table = torch.randperm(30, generator=g).int().view(B, 10).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = [torch.zeros(B, HK, w, dtype=BF, device="cuda") for w in (d, d, dv)]
    Q1, Q2 = (torch.zeros(B, H, d, dtype=BF, device="cuda") for _ in range(2))
    lam = torch.full((H,), 0.6, dtype=BF, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    ws = torch.empty(skl.paged_workspace_size(dv, 2), dtype=torch.uint8, device="cuda")

    def step():
        at = lens.long()
        slots.copy_(table.long().gather(1, (at // page).unsqueeze(1)).squeeze(1) * page + at % page)
        skl.paged_write(rows, caches, slots)
        lens.add_(1)
        return skl.diff_attn_paged(Q1, caches[0], Q2, caches[1], caches[2], lam, table, lens, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step())
        graphs.append(gr)
    lens.copy_(torch.tensor([0, 5, 31], dtype=torch.int32))
    seen = [torch.zeros(B, 160, HK, w, dtype=torch.float64, device="cuda") for w in (d, d, dv)]
    for c in caches:
        c.zero_()
    for n in range(40):
        for t in (*rows, Q1, Q2):
            t.copy_(torch.randn(t.shape, generator=g))
        at = lens.tolist()
        for b in range(B):
            for s, r in zip(seen, rows):
                s[b, at[b]] = r[b].double()
        graphs[n % 2].replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [x + 1 for x in at]
        for b in range(B):   # the caches hold what was written, in the order of the table
            for s, c in zip(seen, caches):
                got = c[table[b].long()].reshape(160, HK, -1)
                assert torch.equal(got[:at[b] + 1].double(), s[b, :at[b] + 1])
        want = paged_reference(Q1, caches[0], Q2, caches[1], caches[2], lam, table, lens)
        within(f"step {n}", outs[n % 2], *want)
    assert skl.query_device_status() == 0


def test_paged_and_whole_sequence_forms_agree():
    """The last row of a prompt by diff_attn and the same token by diff_attn_paged are within both bounds."""
    import attention_kl_distillation_b200 as skl
    n = 333
    c = make([n], 4, 2, 64, 128, page=32)
    K1, K2, V = (c[k][c["table"][0].long()].reshape(1, -1, 2, c[k].shape[3])[:, :n].transpose(1, 2) for k in ("K1", "K2", "V"))
    Q1, Q2 = (c[k].view(1, 4, 1, 64) for k in ("Q1", "Q2"))
    whole = skl.diff_attn(Q1, K1, Q2, K2, V, c["lam"], causal=True)
    r = Reference(Q1, K1, Q2, K2, V, c["lam"], True)
    within("whole", whole, r.O, r.tol_O)
    within("paged", run(c, 2), *reference(c, 2))


@pytest.mark.parametrize("maps", [1, 2])
def test_repeatability(maps):
    c = make([3000, 10, 777], 16, 4, 128, 128, page=32)
    first = run(c, maps)
    for _ in range(3):
        assert torch.equal(run(c, maps), first)


def test_cache_past_32_bit_offsets():
    """A cache of more than 2^31 elements, its last pages in use."""
    import attention_kl_distillation_b200 as skl
    page, HK, d = 64, 8, 128
    pages = 2 ** 31 // (page * HK * d) + 40
    K, V = (torch.zeros(pages, page, HK, d, dtype=BF, device="cuda") for _ in range(2))
    table = torch.arange(pages - 1, pages - 9, -1, dtype=torch.int32, device="cuda").view(2, 4)
    n = torch.tensor([256, 200], dtype=torch.int32, device="cuda")
    slots = torch.cat([table[b].long().repeat_interleave(page) * page + torch.arange(256, device="cuda") % page
                       for b in range(2)])
    rows = [torch.randn(512, HK, d, device="cuda").to(BF) for _ in range(2)]
    skl.paged_write(rows, (K, V), slots)
    Q = torch.randn(2, 16, d, device="cuda").to(BF)
    got = skl.attn_paged(Q, K, V, table, n)
    assert skl.query_device_status() == 0
    assert torch.equal(K.view(-1, HK, d)[slots], rows[0]) and torch.equal(V.view(-1, HK, d)[slots], rows[1])
    within("O", got, *paged_reference(Q, K, None, None, V, None, table, n))


@pytest.mark.parametrize("index", [torch.int32, torch.int64], ids=["int32", "int64"])
@pytest.mark.parametrize("T,HK,widths,head_major", [(1, 1, (8,), False), (7, 3, (64, 64, 128), False),
                                                    (500, 2, (128, 128, 256), True), (33, 16, (24, 8, 40, 64), False)])
def test_write(T, HK, widths, head_major, index):
    """Rows land in their slots; negative slots are skipped; everything else stays."""
    import attention_kl_distillation_b200 as skl
    g = torch.Generator().manual_seed(T)
    pages, page = T // 5 + 3, 12
    slots = torch.randperm(pages * page, generator=g)[:T].to(index).cuda()
    if T > 1:
        slots[T // 2] = -1
    caches, rows = [], []
    for w in widths:
        c = torch.randn(pages, page, HK, w, generator=g).to(HF).cuda()
        caches.append(c.transpose(1, 2).contiguous().transpose(1, 2) if head_major else c)
        rows.append(torch.randn(T, HK, w + 8, generator=g).to(HF).cuda()[..., 8:])
    want = []
    keep = slots >= 0
    for c, r in zip(caches, rows):
        x = c.clone()
        s = slots[keep].long()
        x[s // page, s % page] = r[keep]
        want.append(x)
    skl.paged_write(tuple(rows), tuple(caches), slots)
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    for c, x in zip(caches, want):
        assert torch.equal(c, x)


def test_write_past_the_cache_is_reported():
    import attention_kl_distillation_b200 as skl
    from attention_kl_distillation_b200 import binding
    cache = torch.zeros(2, 4, 1, 8, dtype=BF, device="cuda")
    rows = torch.ones(3, 1, 8, dtype=BF, device="cuda")
    skl.paged_write((rows,), (cache,), torch.tensor([8, 2, 10 ** 12], device="cuda"))
    torch.cuda.synchronize()
    assert skl.query_device_status() == binding.EDEVICE
    want = torch.zeros_like(cache)
    want[0, 2] = 1
    assert torch.equal(cache, want)
    skl.paged_write((rows[:0],), (cache,), torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert torch.equal(cache, want)


def test_prompts_then_tokens():
    """Served as it is used: a padded batch of prompts through diff_attn, their rows into the pages, then single
    tokens through paged_write and diff_attn_paged; every output against the whole sequence in 64 bits."""
    import attention_kl_distillation_b200 as skl
    B, H, HK, d, dv, page, N, more = 3, 8, 2, 64, 128, 32, 90, 5
    g = torch.Generator().manual_seed(77)
    n = torch.tensor([90, 31, 64], dtype=torch.int32, device="cuda")
    total = N + more
    rnd = lambda h, w: torch.randn(B, total, h, w, generator=g).to(BF).cuda()  # noqa: E731
    q1, k1, q2, k2, v = rnd(H, d), rnd(HK, d), rnd(H, d), rnd(HK, d), rnd(HK, dv)
    lam = torch.rand(H, generator=g).to(BF).cuda()
    caches = [torch.zeros(16, page, HK, w, dtype=BF, device="cuda") for w in (d, d, dv)]
    table = torch.randperm(16, generator=g)[:B * 3].int().view(B, 3).cuda()
    heads_first = [t.transpose(1, 2) for t in (q1, k1, q2, k2, v)]
    O = skl.diff_attn(*(t[:, :, :N] for t in heads_first), lam, causal=True, q_lens=n, k_lens=n)
    r = Reference(*(t[:, :, :N] for t in heads_first), lam, True, q_lens=n, k_lens=n)
    within("prompt", O, r.O, r.tol_O)
    at = torch.arange(N, device="cuda").expand(B, N)
    slots = table.long().gather(1, at // page) * page + at % page
    slots = torch.where(at < n.view(B, 1), slots, -1)     # the padding is not written
    skl.paged_write([t[:, :N].reshape(B * N, HK, -1) for t in (k1, k2, v)], caches, slots.reshape(-1))
    b = torch.arange(B, device="cuda")
    for _ in range(more):
        pos = n.long()
        new = table.long()[b, pos // page] * page + pos % page
        skl.paged_write([t[b, pos] for t in (k1, k2, v)], caches, new)
        n = n + 1
        got = skl.diff_attn_paged(q1[b, pos], caches[0], q2[b, pos], caches[1], caches[2], lam, table, n)
        for s in range(B):
            p = int(pos[s])
            one = Reference(*(t[s:s + 1, :, sl] for t, sl in zip(heads_first, (slice(p, p + 1), slice(0, p + 1)) * 2
                                                                 + (slice(0, p + 1),))), lam, True, factors=2)
            within(f"token {p} of sequence {s}", got[s], one.O[0, :, 0], one.tol_O[0, :, 0])
    assert skl.query_device_status() == 0


def test_paged_calls_on_two_streams_at_once():
    import attention_kl_distillation_b200 as skl
    sets = [make([900, 3, 2000], 16, 4, 64, 128, seed=k) for k in range(2)]
    want = [run(c, 2) for c in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(10):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(run(sets[k], 2))
    torch.cuda.synchronize()
    assert skl.query_device_status() == 0
    for w, runs in zip(want, got):
        assert all(torch.equal(w, r) for r in runs)
