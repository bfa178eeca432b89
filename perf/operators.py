"""What the differential-attention and paged-cache operators are measured on.

Cases of real use, their inputs, one pass through an operator (plain torch in 32 bits, or the package's
kernels when ``own`` is true), the work a pass cannot do without, and the same results in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a short question to a small model: one tile per head, latency is all that counts
        dict(name="prompt_short", op="fwd", type="bf16", B=1, H=4, HK=4, NQ=100, NK=100, d=64, dv=128, causal=True, low=1.0),
        # one prompt of 4096 tokens, heads of 64 with values twice as wide
        dict(name="prompt_4k", op="fwd", type="bf16", B=1, H=16, HK=16, NQ=4096, NK=4096, d=64, dv=128, causal=True, low=1.0),
        # a right-padded batch of prompts of different lengths, four query heads to a key head, wide heads
        dict(name="prompt_batch", op="fwd", type="bf16", B=4, H=32, HK=8, NQ=2048, NK=2048, d=128, dv=128, causal=True, low=0.25),
        # a training step at 4096 tokens
        dict(name="train_4k", op="train", type="bf16", B=1, H=16, HK=16, NQ=4096, NK=4096, d=64, dv=128, causal=True, low=1.0),
        # a training step with shared key heads, two padded sequences, the largest case
        dict(name="train_shared", op="train", type="bf16", B=2, H=32, HK=8, NQ=4096, NK=4096, d=128, dv=128, causal=True, low=0.7),
        # cross attention in fp16, values twice as wide as wide heads, odd lengths, no causal mask
        dict(name="train_cross", op="train", type="fp16", B=1, H=8, HK=4, NQ=1111, NK=1501, d=128, dv=256, causal=False, low=1.0),
        # one user's next token
        dict(name="paged_one", op="paged", type="bf16", B=1, H=32, HK=8, NK=1000, d=128, dv=128, page=16, low=1.0),
        # a served batch's next tokens, lengths spread widely
        dict(name="paged_batch", op="paged", type="bf16", B=64, H=32, HK=8, NK=8192, d=128, dv=128, page=64, low=0.05),
        # the same through two maps, a key head to every query head
        dict(name="diff_paged_batch", op="diff_paged", type="bf16", B=32, H=16, HK=16, NK=4096, d=64, dv=128, page=32, low=0.1),
        # two long documents, values twice as wide, fp16, pages that are no power of two
        dict(name="diff_paged_long", op="diff_paged", type="fp16", B=2, H=16, HK=4, NK=65537, d=128, dv=256, page=48, low=0.9),
        # the rows of a served batch's new tokens
        dict(name="write_step", op="write", type="bf16", B=64, HK=16, NK=1, d=64, dv=128, page=32, low=1.0),
        # the rows of a batch of prompts
        dict(name="write_prompts", op="write", type="bf16", B=7, HK=8, NK=2048, d=128, dv=256, page=64, low=0.3),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    wide = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["fwd", "train", "paged", "diff_paged", "write"])
        d, dv = rng.choice([(64, 64), (64, 128), (128, 128), (128, 256)])
        c = dict(op=op, type=rng.choice(["bf16", "fp16"]), d=d, dv=dv)
        c["HK"] = rng.choice([1, 2, 4, 8, 16])
        if op in ("fwd", "train"):
            c["H"] = c["HK"] * rng.choice([1, 2, 4])
            c["B"] = rng.randint(1, 4)
            c["NQ"] = _spread(rng, 64, 4096)
            c["NK"] = c["NQ"] if rng.random() < 0.6 else _spread(rng, c["NQ"], 4096)
            c["causal"] = rng.random() < 0.7
            c["low"] = rng.choice([1.0, rng.uniform(0.1, 1.0)])
        else:
            if op != "write":
                c["H"] = c["HK"] * rng.choice([1, 2, 4, 8])
            c["B"] = _spread(rng, 1, 96)
            c["NK"] = _spread(rng, 100, 65536) if op != "write" else rng.choice([1, _spread(rng, 1, 2048)])
            c["page"] = rng.choice([16, 32, 48, 64, 128])
            c["low"] = rng.uniform(0.05, 1.0)
        w = work(c)
        room = c["B"] * c["H"] * c["NQ"] * c["NK"] <= 2 * 32 * 4096 * 4096 if op in ("fwd", "train") else c["B"] * c["NK"] <= 64 * 8192
        if w["flops"] <= most and w["bytes"] <= wide and room:
            return c


def _lens(n, count, low):
    """`count` lengths from low*n to n, the first n itself, spread evenly and in no order."""
    return [max(1, n - int((n - low * n) * ((k * 0.6180339887) % 1.0))) for k in range(count)]


def _pairs(case):
    """Visible (query, key) pairs of one head over the batch."""
    if case["op"] in ("paged", "diff_paged"):
        return sum(_lens(case["NK"], case["B"], case["low"]))
    total = 0
    for q, k in zip(_lens(case["NQ"], case["B"], case["low"]), _lens(case["NK"], case["B"], case["low"])):
        total += sum(max(0, min(k, i + k - q + 1)) for i in range(q)) if case["causal"] else q * k
    return total


def work(case):
    d, dv = case["d"], case["dv"]
    if case["op"] == "write":
        rows = sum(_lens(case["NK"], case["B"], case["low"])) * case["HK"]
        return {"bytes": 2 * rows * (2 * d + dv) * 2, "flops": 0}
    pairs, maps = _pairs(case), 1 if case["op"] == "paged" else 2
    if case["op"] in ("paged", "diff_paged"):
        return {"bytes": 2 * (pairs * case["HK"] + case["B"] * case["H"]) * (maps * d + dv),
                "flops": pairs * case["H"] * (2 * maps * d + 2 * dv)}
    q, k = case["B"] * case["H"] * case["NQ"], case["B"] * case["HK"] * case["NK"]
    elements = q * (2 * d + dv) + k * (2 * d + dv)
    if case["op"] == "fwd":
        return {"bytes": 2 * elements, "flops": pairs * case["H"] * (4 * d + 2 * dv)}
    return {"bytes": 2 * (2 * elements + q * dv), "flops": pairs * case["H"] * (12 * d + 6 * dv)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["type"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    B, HK, NK, d, dv, low = (case[k] for k in ("B", "HK", "NK", "d", "dv", "low"))
    st = {"case": dict(case)}
    lens = _lens(NK, B, low)
    if case["op"] in ("fwd", "train"):
        H, NQ = case["H"], case["NQ"]
        # as a projection lays them out: [batch, token, head, feature], read as [batch, head, token, feature]
        for name, heads, n, width in (("Q1", H, NQ, d), ("K1", HK, NK, d), ("Q2", H, NQ, d), ("K2", HK, NK, d), ("V", HK, NK, dv)):
            st[name] = normal(B, n, heads, width).transpose(1, 2)
        st["lam"] = (torch.rand((H,), generator=g, device="cuda") * 0.6 + 0.2).to(dtype)
        st["q_lens"] = st["k_lens"] = None
        if low < 1.0:
            st["q_lens"] = torch.tensor(_lens(NQ, B, low), dtype=torch.int32, device="cuda")
            st["k_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if case["op"] == "train":
            for name in ("Q1", "K1", "Q2", "K2", "V", "lam"):
                st[name].requires_grad_(True)
            st["dO"] = normal(B, NQ, H, dv).transpose(1, 2)
        return st
    page = case["page"]
    held = [(n + page - 1) // page for n in lens]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(held)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    for name, width in (("K1", d), ("K2", d), ("V", dv)):
        if name != "K2" or case["op"] != "paged":
            st[name] = normal(pages, page, HK, width)
    st["table"], st["lens"] = table, torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "write":
        at = torch.cat([table[b].long().repeat_interleave(page)[:n] * page + torch.arange(n, device="cuda") % page
                        for b, n in enumerate(lens)])
        st["slots"] = at
        for name, width in (("k1", d), ("k2", d), ("v", dv)):
            st[name] = normal(at.numel(), HK, width)
        return st
    st["Q1"] = normal(B, case["H"], d)
    if case["op"] == "diff_paged":
        st["Q2"] = normal(B, case["H"], d)
        st["lam"] = (torch.rand((case["H"],), generator=g, device="cuda") * 0.6 + 0.2).to(dtype)
    return st


def _seen(st):
    """Which keys each row sees: [B, 1, NQ, NK] truth values."""
    B, _, NQ, _ = st["Q1"].shape
    NK = st["K1"].shape[2]
    i = torch.arange(NQ, device="cuda").view(1, 1, NQ, 1)
    j = torch.arange(NK, device="cuda").view(1, 1, 1, NK)
    q = st["q_lens"].view(B, 1, 1, 1) if st["q_lens"] is not None else NQ
    k = st["k_lens"].view(B, 1, 1, 1) if st["k_lens"] is not None else NK
    seen = (i < q) & (j < k)
    return seen & (j <= i + k - q) if st["case"]["causal"] else seen


def _softmax(x, seen):
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def _over_heads(t, H):
    return t.float().repeat_interleave(H // t.shape[1], 1)


def _plain_maps(st):
    H, scale, seen = st["Q1"].shape[1], 1.0 / math.sqrt(st["Q1"].shape[3]), _seen(st)
    P1 = _softmax(st["Q1"].float() @ _over_heads(st["K1"], H).transpose(2, 3) * scale, seen)
    P2 = _softmax(st["Q2"].float() @ _over_heads(st["K2"], H).transpose(2, 3) * scale, seen)
    return P1, P2, _over_heads(st["V"], H), st["lam"].float().view(1, H, 1, 1), scale


def _plain_fwd(st):
    P1, P2, V, lam, _ = _plain_maps(st)
    return ((P1 - lam * P2) @ V).to(st["V"].dtype)


def _plain_train(st):
    P1, P2, V, lam, scale = _plain_maps(st)
    dtype, B, H = st["V"].dtype, *st["Q1"].shape[:2]
    group = lambda t: t.view(B, -1, H // st["K1"].shape[1], *t.shape[2:]).sum(2).to(dtype)  # noqa: E731
    dO = st["dO"].float()
    G = dO @ V.transpose(2, 3)
    D1, D2 = (P1 * G).sum(-1, keepdim=True), (P2 * G).sum(-1, keepdim=True)
    A = P1.addcmul(lam.expand(B, H, 1, 1), P2, value=-1.0)
    O, dV = A @ V, group(A.transpose(2, 3) @ dO)
    del A
    X1 = P1.mul_(G - D1).mul_(scale)
    X2 = P2.mul_(D2 - G).mul_(lam * scale)
    dQ1, dQ2 = X1 @ _over_heads(st["K1"], H), X2 @ _over_heads(st["K2"], H)
    dK1, dK2 = X1.transpose(2, 3) @ st["Q1"].float(), X2.transpose(2, 3) @ st["Q2"].float()
    return (O.to(dtype), dQ1.to(dtype), group(dK1), dQ2.to(dtype), group(dK2), dV, -D2.sum((0, 2, 3)).to(dtype))


def _pages(cache, table):
    """A cache's rows of every sequence, in 32 bits: [B, key heads, tokens, width]."""
    t = cache[table.long()]
    return t.reshape(t.shape[0], -1, *t.shape[3:]).permute(0, 2, 1, 3).float()


def _plain_paged(st):
    B, H, d = st["Q1"].shape
    heads = (B, st["K1"].shape[2], -1, d)  # query heads by the key head that they share
    K, V = _pages(st["K1"], st["table"]), _pages(st["V"], st["table"])
    seen = torch.arange(K.shape[2], device="cuda").view(1, 1, 1, -1) < st["lens"].view(B, 1, 1, 1)
    A = _softmax(st["Q1"].float().view(heads) @ K.transpose(2, 3) / math.sqrt(d), seen)
    if st["case"]["op"] == "diff_paged":
        x = st["Q2"].float().view(heads) @ _pages(st["K2"], st["table"]).transpose(2, 3) / math.sqrt(d)
        A = A - st["lam"].float().view(1, heads[1], -1, 1) * _softmax(x, seen)
    return (A @ V).reshape(B, H, -1).to(st["V"].dtype)


def _plain_write(st):
    st["K1"].view(-1, *st["K1"].shape[2:])[st["slots"]] = st["k1"]
    st["K2"].view(-1, *st["K2"].shape[2:])[st["slots"]] = st["k2"]
    st["V"].view(-1, *st["V"].shape[2:])[st["slots"]] = st["v"]
    return st["K1"], st["K2"], st["V"]


def _own_run(st):
    import attention_kl_distillation_b200 as skl
    op = st["case"]["op"]
    if op == "write":
        skl.paged_write((st["k1"], st["k2"], st["v"]), (st["K1"], st["K2"], st["V"]), st["slots"])
        return st["K1"], st["K2"], st["V"]
    if op == "paged":
        return skl.attn_paged(st["Q1"], st["K1"], st["V"], st["table"], st["lens"])
    if op == "diff_paged":
        return skl.diff_attn_paged(st["Q1"], st["K1"], st["Q2"], st["K2"], st["V"], st["lam"], st["table"], st["lens"])
    leaves = [st[n] for n in ("Q1", "K1", "Q2", "K2", "V", "lam")]
    O = skl.diff_attn(*leaves, causal=st["case"]["causal"], q_lens=st["q_lens"], k_lens=st["k_lens"])
    return (O.detach(), *torch.autograd.grad(O, leaves, st["dO"])) if op == "train" else O


def run(state):
    if own:
        return _own_run(state)
    with torch.no_grad():
        return {"fwd": _plain_fwd, "train": _plain_train, "paged": _plain_paged, "diff_paged": _plain_paged,
                "write": _plain_write}[state["case"]["op"]](state)


def exact(case, seed):
    """run's results from the definition in 64 bits: one head of one sequence at a time over its own visible
    keys, gradients by differentiating the definition."""
    st = prepare(case, seed)
    lens = _lens(case["NK"], case["B"], case["low"])
    if case["op"] == "write":
        out = []
        for cache, rows in (("K1", "k1"), ("K2", "k2"), ("V", "v")):
            t = st[cache].double()
            t[st["slots"] // case["page"], st["slots"] % case["page"]] = st[rows].double()
            out.append(t)
        return tuple(out)
    H, per = case["H"], case["H"] // case["HK"]
    if case["op"] in ("paged", "diff_paged"):
        out = torch.zeros((case["B"], H, case["dv"]), dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            at = torch.arange(n, device="cuda")
            page, row = st["table"][b].long()[at // case["page"]], at % case["page"]
            for h in range(case["HK"]):
                heads = slice(h * per, (h + 1) * per)
                v = st["V"][page, row, h].double()
                x = st["Q1"][b, heads].double() @ st["K1"][page, row, h].double().T / math.sqrt(case["d"])
                out[b, heads] = torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) @ v
                if case["op"] == "diff_paged":
                    x = st["Q2"][b, heads].double() @ st["K2"][page, row, h].double().T / math.sqrt(case["d"])
                    out[b, heads] -= st["lam"][heads].double()[:, None] * (torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) @ v)
        return out
    names = ("Q1", "K1", "Q2", "K2", "V", "lam")
    wide = {n: st[n].detach().double() for n in names}
    grads = {n: torch.zeros_like(wide[n]) for n in names}
    O = torch.zeros((case["B"], H, case["NQ"], case["dv"]), dtype=torch.float64, device="cuda")
    for b, (q, k) in enumerate(zip(_lens(case["NQ"], case["B"], case["low"]), lens)):
        for h in range(H):
            s = h // per
            one = [wide["Q1"][b, h, :q], wide["K1"][b, s, :k], wide["Q2"][b, h, :q], wide["K2"][b, s, :k], wide["V"][b, s, :k], wide["lam"][h]]
            one = [t.clone().requires_grad_(case["op"] == "train") for t in one]
            maps = []
            for Q, K in (one[:2], one[2:4]):
                x = Q @ K.T / math.sqrt(case["d"])
                if case["causal"]:
                    x = x.masked_fill(torch.ones(q, k, dtype=torch.bool, device="cuda").triu(k - q + 1), -math.inf)
                maps.append(torch.softmax(x, 1))
            o = (maps[0] - one[5] * maps[1]) @ one[4]
            O[b, h, :q] = o.detach()
            if case["op"] == "train":
                got = torch.autograd.grad(o, one, st["dO"][b, h, :q].double())
                grads["Q1"][b, h, :q], grads["Q2"][b, h, :q] = got[0], got[2]
                grads["K1"][b, s, :k] += got[1]
                grads["K2"][b, s, :k] += got[3]
                grads["V"][b, s, :k] += got[4]
                grads["lam"][h] += got[5]
    return (O, *(grads[n] for n in names)) if case["op"] == "train" else O
