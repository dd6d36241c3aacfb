"""What is measured of the operators for a bounded view and a bounded cache:
the cases, their inputs, their plain form in elementary torch operations, and
the framework's calls.

  wprefill   causal attention over packed prompts with a sliding window and a
             few first tokens that stay visible (sinks): token i attends the
             tokens j <= i with i - j < window or j < sinks (grouped heads,
             optional sigmoid output gate):       kda_attn_window_prefill
  wbackward  its gradients:                       kda_attn_window_prefill_backward
  wtree      the same view for a tree of drafted tokens over a paged cache
             (one token per sequence is plain decode): of a row's tokens, the
             cached ones and then the drafts of its mask word, the first
             `sinks` and the last `window` are attended:  kda_attn_window_tree
  weigh      each cached token's attention weight, summed over the heads and
             the queries of its sequence's last tokens, added to what it has
             gathered:                            kda_cache_weigh
  evict      slots cut down to `keep` tokens: the first and the most recent
             ones and, of the others, the heaviest, moved to the front of the
             slots' pages in their order; the pages behind are given back:
             kda_cache_evict

A cache is two pools of pages, k_cache [pages, Hkv, page, dk] and v_cache
[pages, Hkv, page, dv], a page table [slots, max_pages] (-1: no page), the
slots' lengths in tokens and each page's count of table entries (0: free).
The gathered weights are fp32 [slots, max_pages * page].
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the library's smallest core shape (64 tokens, 2 heads of 16, fp32): launch latency
        dict(name="wprefill_tiny_f32", op="wprefill", dtype="f32", seqs=1, min_len=64, max_len=64, lens_seed=0,
             H=2, Hkv=2, dk=16, dv=16, gate=False, window=16, sinks=2),
        # a serving batch of ragged prompts, the hybrid's attention heads (192 with the rotary part, values 128, gated)
        dict(name="wprefill_packed", op="wprefill", dtype="bf16", seqs=12, min_len=1, max_len=2048, lens_seed=3,
             H=32, Hkv=32, dk=192, dv=128, gate=True, window=512, sinks=4),
        # one long prompt with grouped heads
        dict(name="wprefill_long", op="wprefill", dtype="bf16", seqs=1, min_len=16384, max_len=16384, lens_seed=0,
             H=32, Hkv=8, dk=128, dv=128, gate=False, window=4096, sinks=4),
        # a small fp32 training batch of ragged sequences, gated, an odd window
        dict(name="wbackward_packed_f32", op="wbackward", dtype="f32", seqs=6, min_len=5, max_len=500, lens_seed=5,
             H=8, Hkv=2, dk=64, dv=64, gate=True, window=100, sinks=3),
        # a training layer of 8192 tokens, each attending the last 1024
        dict(name="wbackward_layer_t8k", op="wbackward", dtype="bf16", seqs=1, min_len=8192, max_len=8192, lens_seed=0,
             H=32, Hkv=8, dk=128, dv=128, gate=False, window=1024, sinks=4),
        # plain decode, 256 sequences, one token each
        dict(name="wdecode_b256", op="wtree", dtype="bf16", seqs=256, min_len=1024, max_len=4096, lens_seed=7,
             T=1, chain=True, H=32, Hkv=8, dk=128, dv=128, page=64, gate=False, window=1024, sinks=4),
        # 32 sequences with a tree of 16 drafted tokens each, gated
        dict(name="wtree_b32_t16", op="wtree", dtype="bf16", seqs=32, min_len=100, max_len=8000, lens_seed=8,
             T=16, chain=False, H=32, Hkv=8, dk=128, dv=128, page=64, gate=True, window=2000, sinks=4),
        # a decode step's weights over the whole cache, 256 sequences
        dict(name="weigh_decode_b256", op="weigh", dtype="bf16", seqs=256, min_len=1024, max_len=4096, lens_seed=7,
             last=1, tree=4, H=32, Hkv=8, dk=128, page=64, window=0, sinks=0),
        # the last 64 tokens of each prompt of a batch weigh the prompt
        dict(name="weigh_last64_prompts", op="weigh", dtype="bf16", seqs=8, min_len=900, max_len=8000, lens_seed=10,
             last=64, tree=0, H=32, Hkv=8, dk=128, page=64, window=0, sinks=0),
        # every token of one long prompt weighs those before it
        dict(name="weigh_prompt_8000", op="weigh", dtype="bf16", seqs=1, min_len=8000, max_len=8000, lens_seed=0,
             last=8000, tree=0, H=32, Hkv=8, dk=128, page=64, window=0, sinks=0),
        # one conversation cut to its budget: latency
        dict(name="evict_one", op="evict", dtype="bf16", seqs=1, min_len=5000, max_len=5000, lens_seed=13,
             keep=1024, first=4, recent=256, Hkv=8, dk=128, dv=128, page=64),
        # a batch of prompts cut to theirs; some are shorter than it
        dict(name="evict_b64", op="evict", dtype="bf16", seqs=64, min_len=500, max_len=8000, lens_seed=14,
             keep=2048, first=4, recent=512, Hkv=8, dk=128, dv=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["wprefill", "wbackward", "wtree", "wtree", "weigh", "weigh", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dk, dv = rng.choice([(128, 128), (128, 128), (192, 128), (64, 64), (32, 32), (16, 16)])
    H, Hkv = rng.choice([(32, 8), (32, 32), (8, 1), (8, 2), (32, 4)])
    seed = rng.randrange(1 << 30)
    heads = dict(H=H, Hkv=Hkv, dk=dk, dv=dv)
    page = rng.choice([16, 32, 64, 128])
    sinks = rng.choice([0, 1, 4, 4, 33, 128])
    most = int(2e9) // (Hkv * (dk + dv) * (2 if dtype == "bf16" else 4))  # tokens in 2 GB of cache
    if op in ("wprefill", "wbackward"):
        seqs = rng.choice([1, 1, 2, 5, 16])
        longest = max(2, _log(rng, 16, (6000 if op == "wprefill" else 4000) // (1 if seqs < 5 else 4)))
        return dict(op=op, dtype=dtype, seqs=seqs, min_len=max(1, longest // rng.choice([1, 2, 50])), max_len=longest,
                    lens_seed=seed, gate=rng.random() < 0.5, window=_log(rng, 1, 3000), sinks=sinks, **heads)
    if op == "wtree":
        seqs = _log(rng, 1, 200)
        longest = _log(rng, 30, min(200000, max(40, min(500000, most) // seqs)))
        return dict(op=op, dtype=dtype, seqs=seqs, min_len=max(0, longest // rng.choice([1, 3, 1000])),
                    max_len=longest, lens_seed=seed, T=rng.choice([1, 1, 4, 7, 16, 33]), chain=rng.random() < 0.3,
                    gate=rng.random() < 0.5, page=page, window=_log(rng, 1, 20000), sinks=sinks, **heads)
    if op == "weigh":
        tree = rng.choice([0, 0, 4, 16])
        last = rng.choice([1, 1, 3, 4]) if tree else _log(rng, 1, 4000)
        seqs = _log(rng, 1, max(2, 200 // last))
        room = min(500000, most, int(1.5e9) // (H * last)) // seqs  # fp32 scores of at most 6 GB
        longest = _log(rng, last + 1, max(last + 2, min(100000, room)))
        return dict(op=op, dtype=dtype, seqs=seqs, min_len=max(1, longest // rng.choice([1, 3, 20])), max_len=longest,
                    lens_seed=seed, last=last, tree=tree, H=H, Hkv=Hkv, dk=dk, page=page,
                    window=rng.choice([0, 0, _log(rng, 1, 20000)]), sinks=sinks)
    seqs = _log(rng, 1, 64)
    longest = _log(rng, 20, max(30, min(100000, most // seqs)))
    keep = max(1, int(longest * rng.choice([0.1, 0.3, 0.5, 0.9])))
    first = min(rng.choice([0, 1, 4, 32]), keep // 2)
    return dict(op=op, dtype=dtype, seqs=seqs, min_len=max(1, longest // rng.choice([1, 3, 20])), max_len=longest,
                lens_seed=seed, keep=keep, first=first, recent=min(rng.choice([0, 1, 64, 500]), keep - first),
                Hkv=Hkv, dk=dk, dv=dv, page=page)


def _lens(case):
    """The lengths of a case's sequences: the longest first named, the others
    anywhere between the two bounds."""
    r = random.Random(case["lens_seed"])
    lens = [case["max_len"]] + [r.randint(case["min_len"], case["max_len"]) for _ in range(case["seqs"] - 1)]
    r.shuffle(lens)
    return lens


def _counts(case):
    """Queries of each sequence of a weigh: its last tokens, fewer where the
    sequence is shorter; of a draft tree any number up to `last` is accepted."""
    r = random.Random(case["lens_seed"] + 1)
    return [min(n, r.randint(1, case["last"]) if case["tree"] else case["last"]) for n in _lens(case)]


def _item(case):
    return 2 if case["dtype"] == "bf16" else 4


def _pages_of(n, page):
    return -(-n // page)


def _pairs(n, window, sinks, first=0):
    """Pairs of the tokens first .. n - 1 with what they attend."""
    if window == 0:
        window = n
    total = 0
    for i in range(first, n):
        far = max(0, i + 1 - window)
        total += i + 1 - far + min(sinks, far)
    return total


def _parents(T, seed):
    """A draft tree as each token's parent (-1: the committed context), the
    same shape for every sequence of a case, as a server keeps it."""
    r = random.Random(seed + 1)
    return [-1] + [r.choice([t - 1, r.randint(-1, t - 1)]) for t in range(1, T)]


def _ancestors(parents, t):
    got = []
    while t >= 0:
        got.append(t)
        t = parents[t]
    return got


def _paths(case):
    """Each drafted token's own path, itself included, in order."""
    T = case["T"]
    parents = list(range(-1, T - 1)) if case["chain"] else _parents(T, case["lens_seed"])
    return [sorted(_ancestors(parents, t)) for t in range(T)]


def work(case):
    op, e = case["op"], _item(case)
    lens = _lens(case)
    Hkv, dk = case["Hkv"], case["dk"]
    if op in ("wprefill", "wbackward"):
        T, pairs = sum(lens), sum(_pairs(n, case["window"], case["sinks"]) for n in lens)
        H, dv = case["H"], case["dv"]
        one = T * (H * dk + Hkv * (dk + dv) + H * dv * (2 if case["gate"] else 1)) * e + T * H * 4
        if op == "wprefill":
            return {"bytes": one, "flops": 2 * (dk + dv) * pairs * H}
        # also reads dy; writes dq, dk, dv (and dz)
        return {"bytes": one + T * H * dv * e + T * (H * dk + Hkv * (dk + dv) + (H * dv if case["gate"] else 0)) * e,
                "flops": 2 * (3 * dk + 2 * dv) * pairs * H}
    if op == "wtree":
        T, H, dv, B = case["T"], case["H"], case["dv"], case["seqs"]
        window, sinks = case["window"], case["sinks"]
        read = pairs = entries = 0
        depths = [len(p) for p in _paths(case)]
        for n in lens:
            seen = [_pairs(n + d, window, sinks, n + d - 1) for d in depths]
            pairs += sum(seen)
            read += min(n, max(0, window - min(depths)) + sinks)
            entries += min(_pages_of(n, case["page"]), _pages_of(window, case["page"]) + _pages_of(sinks, case["page"]) + 1)
        return {"bytes": (read + B * T) * Hkv * (dk + dv) * e + B * T * H * (dk + dv * (2 if case["gate"] else 1)) * e
                + B * T * H * 4 + entries * 4 + (0 if case["chain"] else B * T * 8),
                "flops": 2 * (dk + dv) * H * pairs}
    if op == "weigh":
        counts, H, window, sinks = _counts(case), case["H"], case["window"], case["sinks"]
        pairs = sum(_pairs(n, window, sinks, n - c) for n, c in zip(lens, counts))
        read = sum(min(n, (window or n) + c - 1 + sinks) for n, c in zip(lens, counts))
        return {"bytes": read * (Hkv * dk * e + 8) + sum(counts) * H * (dk * e + 4), "flops": 2 * dk * H * pairs}
    cut = [n for n in lens if n > case["keep"]]
    moved = len(cut) * (case["keep"] - case["first"])
    return {"bytes": 2 * moved * Hkv * (dk + case["dv"]) * e + 4 * sum(cut) + 4 * sum(cut) + 4 * len(lens) * case["keep"],
            "flops": 0}


# --------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return c


def _attn_inputs(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    lens = _lens(case)
    T, H, Hkv, dk, dv = sum(lens), case["H"], case["Hkv"], case["dk"], case["dv"]
    s = dict(case=dict(case), longest=max(lens), cu=_ints(_cu(lens)), q=_normal(g, (T, H, dk), dt),
             k=_normal(g, (T, Hkv, dk), dt), v=_normal(g, (T, Hkv, dv), dt),
             z=_normal(g, (T, H, dv), dt) if case["gate"] else None)
    if case["op"] == "wbackward":
        s["dy"] = _normal(g, (T, H, dv), dt)
        s["out"], s["lse"] = _plain_prefill(s)
    return s


def _table(case, g, r, lens, spare):
    """A page table of slots in any order over pages in any order: each
    sequence's slot, the table, the slots' lengths, the pages' counts."""
    page, B = case["page"], len(lens)
    need = [_pages_of(n, page) for n in lens]
    width, pages = max(max(need), 1), sum(need) + 8
    slots = B + spare  # a server's table has rows that this batch does not use
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    row = r.sample(range(slots), B)
    table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    length = torch.zeros(slots, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:sum(need)].long()] = 1
    at = 0
    for b in range(B):
        table[row[b], :need[b]] = order[at:at + need[b]]
        at += need[b]
    length[torch.tensor(row, device="cuda")] = _ints(lens)
    return row, table, length, refs


def _tree_inputs(case, seed):
    g, dt, r = _gen(seed), DTYPES[case["dtype"]], random.Random(seed)
    lens, B, T, page = _lens(case), case["seqs"], case["T"], case["page"]
    H, Hkv, dk, dv = case["H"], case["Hkv"], case["dk"], case["dv"]
    row, table, length, refs = _table(case, g, r, lens, 3)
    pages = refs.numel()
    mask = None
    if not case["chain"]:
        words = [sum(1 << a for a in p) for p in _paths(case)]
        mask = torch.tensor(words, dtype=torch.int64, device="cuda").expand(B, T).contiguous()
    return dict(case=dict(case), longest=max(lens), rows=_ints(row), table=table, lens=length, mask=mask,
                q=_normal(g, (B, T, H, dk), dt), k_new=_normal(g, (B, T, Hkv, dk), dt),
                v_new=_normal(g, (B, T, Hkv, dv), dt), k_cache=_normal(g, (pages, Hkv, page, dk), dt),
                v_cache=_normal(g, (pages, Hkv, page, dv), dt),
                z=_normal(g, (B, T, H, dv), dt) if case["gate"] else None)


def _weigh_inputs(case, seed):
    g, dt, r = _gen(seed), DTYPES[case["dtype"]], random.Random(seed)
    lens, counts, N, page = _lens(case), _counts(case), case["seqs"], case["page"]
    row, table, length, refs = _table(case, g, r, lens, 3)
    slots, width = table.shape
    total, tree = sum(counts), max(case["tree"], case["last"]) if case["tree"] else 0
    src = N * tree if tree else total
    rows = None
    if tree:  # an accepted path: rising positions in the sequence's tree
        rows = _ints([b * tree + t for b, n in enumerate(counts) for t in sorted(r.sample(range(tree), n))])
    s = dict(case=dict(case), longest=max(lens), most=max(counts), slot=_ints(row), cu=_ints(_cu(counts)), rows=rows, table=table, lens=length,
             q=_normal(g, (src, case["H"], case["dk"]), dt), k_cache=_normal(g, (refs.numel(), case["Hkv"], page, case["dk"]), dt),
             # gathered by a few such calls before this one
             weights=torch.rand((slots, width * page), generator=g, device="cuda") * (4 * case["H"] * max(counts) / max(lens)))
    # what the attention of these queries gave: the logarithm of each row's sum
    x, there = _weigh_scores(s)
    m = x.amax(-1, keepdim=True)
    lse = (m + (x - m).exp_().sum(-1, keepdim=True).log())[..., 0]  # [N, Hkv, G, C]
    lse = lse.permute(0, 3, 1, 2).reshape(N, s["most"], case["H"])[there]
    s["lse"] = torch.zeros((src, case["H"]), device="cuda")
    s["lse"][torch.arange(total, device="cuda") if rows is None else rows.long()] = lse
    return s


def _evict_inputs(case, seed):
    g, dt, r = _gen(seed), DTYPES[case["dtype"]], random.Random(seed)
    lens, page, Hkv = _lens(case), case["page"], case["Hkv"]
    row, table, length, refs = _table(case, g, r, lens, 2)
    slots, width = table.shape
    # gathered weights: a few heavy tokens, many light ones, some that nobody has attended
    w = (_normal(g, (slots, width * page), torch.float32) * 1.5).exp()
    w = w * (torch.rand(w.shape, generator=g, device="cuda") > 0.2)
    shape = (refs.numel(), Hkv, page)
    s = dict(case=dict(case), longest=max(lens), slot=_ints(row), table0=table, lens0=length, refs0=refs, weights0=w,
             k_cache=_normal(g, shape + (case["dk"],), dt), v_cache=_normal(g, shape + (case["dv"],), dt))
    for name in ("table", "lens", "refs", "weights"):
        s[name] = s[name + "0"].clone()
    return s


def prepare(case, seed):
    return {"wprefill": _attn_inputs, "wbackward": _attn_inputs, "wtree": _tree_inputs, "weigh": _weigh_inputs,
            "evict": _evict_inputs}[case["op"]](case, seed)


# ----------------------------------------------------------- the plain form

def _padded(x, cu, longest):
    """[T, heads, d] of packed sequences as fp32 [N, heads, longest, d]."""
    at = cu[:-1, None].long() + torch.arange(longest, device=x.device)
    at = at.clamp(max=x.shape[0] - 1)
    return x[at].float().transpose(1, 2)


def _packed(x, cu, longest, T, dtype):
    """[N, heads, longest, d] back to [T, heads, d]."""
    t = torch.arange(T, device=x.device)
    n = torch.searchsorted(cu[1:].contiguous(), t.to(cu.dtype), right=True)
    return x.transpose(1, 2)[n, t - cu[n].long()].to(dtype)


def _scores(s):
    """Scaled scores [N, Hkv, G, L, L] with what a token may not attend at -inf."""
    c, cu, L = s["case"], s["cu"], s["longest"]
    Hkv, G = c["Hkv"], c["H"] // c["Hkv"]
    q = _padded(s["q"], cu, L)
    k = _padded(s["k"], cu, L)
    N = q.shape[0]
    x = torch.matmul((q * c["dk"] ** -0.5).reshape(N, Hkv, G * L, c["dk"]), k.transpose(2, 3)).view(N, Hkv, G, L, L)
    t = torch.arange(L, device=q.device)
    i, j = t[:, None], t[None, :]
    hidden = (j > i) | ((i - j >= c["window"]) & (j >= c["sinks"]))
    return x.masked_fill_(hidden, -math.inf), q, k


def _plain_prefill(s):
    c, cu, L = s["case"], s["cu"], s["longest"]
    T, H, Hkv, dv = s["q"].shape[0], c["H"], c["Hkv"], c["dv"]
    x, q, k = _scores(s)
    N = q.shape[0]
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (m + total.log()).view(N, H, L, 1)
    v = _padded(s["v"], cu, L)
    o = torch.matmul(x.view(N, Hkv, -1, L), v).view(N, Hkv, H // Hkv, L, dv) / total
    o = o.view(N, H, L, dv)
    if s["z"] is not None:
        o = o * torch.sigmoid(_padded(s["z"], cu, L))
    return _packed(o, cu, L, T, s["q"].dtype), _packed(lse, cu, L, T, torch.float32)[..., 0]


def _plain_backward(s):
    c, cu, L, dt = s["case"], s["cu"], s["longest"], s["q"].dtype
    T, H, Hkv, dk, dv = s["q"].shape[0], c["H"], c["Hkv"], c["dk"], c["dv"]
    G = H // Hkv
    x, q, k = _scores(s)
    N = q.shape[0]
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    p = x.div_(x.sum(-1, keepdim=True)).view(N, Hkv, G * L, L)
    # rows behind a sequence's end are padding: their output gradient is nothing
    there = torch.arange(L, device=q.device) < (cu[1:] - cu[:-1])[:, None]
    v = _padded(s["v"], cu, L)
    do = _padded(s["dy"], cu, L) * there[:, None, :, None]
    dz = None
    if s["z"] is not None:
        gate = torch.sigmoid(_padded(s["z"], cu, L))
        o = torch.matmul(p, v).view(N, H, L, dv)
        dz = _packed(do * o * gate * (1 - gate), cu, L, T, dt)
        do = do * gate
    do = do.reshape(N, Hkv, G * L, dv)
    gv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds = ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(dk ** -0.5)
    gk = torch.matmul(ds.transpose(2, 3), q.reshape(N, Hkv, G * L, dk))
    gq = torch.matmul(ds, k).view(N, H, L, dk)
    return {"dq": _packed(gq, cu, L, T, dt), "dk": _packed(gk, cu, L, T, dt), "dv": _packed(gv, cu, L, T, dt), "dz": dz}


def _plain_tree(s):
    c = s["case"]
    B, T, H, Hkv, dk, dv, page = c["seqs"], c["T"], c["H"], c["Hkv"], c["dk"], c["dv"], c["page"]
    G, rows = H // Hkv, s["rows"].long()
    n = max(_pages_of(s["longest"], page), 1)
    at = s["table"][rows][:, :n].long().clamp(min=0)
    lens = s["lens"][rows].long()
    k = s["k_cache"][at].float().transpose(1, 2).reshape(B, Hkv, n * page, dk)
    v = s["v_cache"][at].float().transpose(1, 2).reshape(B, Hkv, n * page, dv)
    k = torch.cat([k, s["k_new"].float().transpose(1, 2)], 2)
    v = torch.cat([v, s["v_new"].float().transpose(1, 2)], 2)
    q = (s["q"].float() * dk ** -0.5).view(B, T, Hkv, G, dk).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, dk)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, T, -1)
    bits = torch.arange(T, device=q.device)
    if s["mask"] is None:
        new = (bits[None, :] <= bits[:, None]).expand(B, T, T)
    else:
        new = (s["mask"][:, :, None] >> bits) & 1 > 0
    # the place of each key among a row's tokens: the cached ones, then its drafts
    old = torch.arange(n * page, device=q.device)
    place = torch.cat([old.expand(B, T, n * page), lens[:, None, None] + new.cumsum(2) - 1], 2)
    all_of = (lens[:, None] + new.sum(2))[..., None]
    seen = torch.cat([(old < lens[:, None])[:, None].expand(B, T, n * page), new], 2)
    seen = seen & ((place < c["sinks"]) | (place >= all_of - c["window"]))
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, G * T, -1), v).view(B, Hkv, G, T, dv) / total
    lse = (m + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, T, H)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, H, dv)
    if s["z"] is not None:
        o = o * torch.sigmoid(s["z"].float())
    return o.to(s["q"].dtype), lse.contiguous()


def _weigh_scores(s):
    """Scaled scores [N, Hkv, G, C, L] of each sequence's queries over its slot,
    what they may not attend at -inf, and which of the [N, C] rows are queries."""
    c, cu = s["case"], s["cu"].long()
    N, C, H, Hkv, dk, page = c["seqs"], s["most"], c["H"], c["Hkv"], c["dk"], c["page"]
    n, G, slot = _pages_of(s["longest"], page), H // Hkv, s["slot"].long()
    at = s["table"][slot][:, :n].long().clamp(min=0)
    lens, counts = s["lens"][slot].long(), cu[1:] - cu[:-1]
    k = s["k_cache"][at].float().transpose(1, 2).reshape(N, Hkv, n * page, dk)
    t = torch.arange(C, device="cuda")
    there = t < counts[:, None]
    row = (cu[:-1, None] + t).clamp(max=int(s["q"].shape[0]) - 1 if s["rows"] is None else s["rows"].numel() - 1)
    q = s["q"][row if s["rows"] is None else s["rows"].long()[row]].float() * dk ** -0.5  # [N, C, H, dk]
    q = q.view(N, C, Hkv, G, dk).permute(0, 2, 3, 1, 4).reshape(N, Hkv, G * C, dk)
    x = torch.matmul(q, k.transpose(2, 3)).view(N, Hkv, G, C, n * page)
    i, j = (lens - counts)[:, None, None] + t[:, None], torch.arange(n * page, device="cuda")
    hidden = (j > i) | ~there[..., None]
    if c["window"]:
        hidden = hidden | ((i - j >= c["window"]) & (j >= c["sinks"]))
    return x.masked_fill_(hidden[:, None, None], -math.inf), there


def _plain_weigh(s):
    c, cu = s["case"], s["cu"].long()
    N, C, H, Hkv = c["seqs"], s["most"], c["H"], c["Hkv"]
    x, there = _weigh_scores(s)
    lse = torch.zeros((N, C, H), device="cuda")
    lse[there] = s["lse"] if s["rows"] is None else s["lse"][s["rows"].long()]
    x = x.sub_(lse.view(N, C, Hkv, H // Hkv).permute(0, 2, 3, 1)[..., None]).exp_()
    slot = s["slot"].long()
    s["weights"][slot, :x.shape[-1]] += x.view(N, -1, x.shape[-1]).sum(1)
    return s["weights"]


def _reset(s):
    for name in ("table", "lens", "refs", "weights"):
        s[name].copy_(s[name + "0"])


def _plain_evict(s):
    _reset(s)
    c, slot, table, refs = s["case"], s["slot"].long(), s["table"], s["refs"]
    keep, first, recent, page = c["keep"], c["first"], c["recent"], c["page"]
    L = max(s["longest"], keep)
    lens = s["lens"][slot].long()[:, None]
    new = lens.clamp(max=keep)
    pos = torch.arange(L, device="cuda")
    w = s["weights"][slot][:, :L]
    w = torch.cat([w, w.new_zeros(w.shape[0], L - w.shape[1])], 1)
    rank = torch.where((pos < first) | (pos >= lens - recent), math.inf, w)
    rank = torch.where(pos < lens, rank, -math.inf)
    kept = rank.sort(dim=1, descending=True, stable=True).indices[:, :keep]
    d = torch.arange(keep, device="cuda")
    kept = torch.where(d < new, kept, L).sort(dim=1).values
    e, to = (d < new).nonzero(as_tuple=True)
    at = kept[e, to]
    for name in ("k_cache", "v_cache"):
        pool = s[name]
        pool[table[slot[e], to // page].long(), :, to % page] = pool[table[slot[e], at // page].long(), :, at % page]
    moved = torch.where(pos < lens, 0.0, w)
    moved[e, to] = w[e, at]
    room = min(L, s["weights"].shape[1])
    s["weights"][slot, :room] = moved[:, :room]
    rows = table[slot]
    gone = (torch.arange(rows.shape[1], device="cuda") >= (new + page - 1) // page) & (rows >= 0)
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), -gone.flatten().to(torch.int32))
    table[slot] = torch.where(gone, -1, rows)
    s["lens"][slot] = new[:, 0].to(torch.int32)
    kept = torch.where(d < new, kept, -1).to(torch.int32)
    return {"kept": kept, "status": torch.zeros_like(s["slot"]), "table": table, "lens": s["lens"], "refs": refs,
            "weights": s["weights"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


PLAIN = {"wprefill": _plain_prefill, "wbackward": _plain_backward, "wtree": _plain_tree, "weigh": _plain_weigh,
         "evict": _plain_evict}


# -------------------------------------------------------- the framework's calls

def _own(s):
    from gated_delta_rule_64_amd import kda
    c = s["case"]
    op = c["op"]
    if op == "wprefill":
        return kda.kda_attn_window_prefill(s["q"], s["k"], s["v"], c["window"], sinks=c["sinks"], out_gate=s["z"],
                                           cu_seqlens=s["cu"])
    if op == "wbackward":
        return kda.kda_attn_window_prefill_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dy"], c["window"],
                                                    sinks=c["sinks"], out_gate=s["z"], cu_seqlens=s["cu"])
    if op == "wtree":
        return kda.kda_attn_window_tree(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                        c["window"], sinks=c["sinks"], tree_mask=s["mask"], out_gate=s["z"],
                                        slot_indices=s["rows"])
    if op == "weigh":
        kda.kda_cache_weigh(s["q"], s["lse"], s["k_cache"], s["table"], s["lens"], s["weights"], cu_seqlens=s["cu"],
                            rows=s["rows"], slot_indices=s["slot"], window=c["window"], sinks=c["sinks"])
        return s["weights"]
    _reset(s)
    kept, status = kda.kda_cache_evict(s["slot"], c["keep"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["refs"],
                                       s["weights"], first=c["first"], recent=c["recent"])
    return {"kept": kept, "status": status, "table": s["table"], "lens": s["lens"], "refs": s["refs"],
            "weights": s["weights"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------- the definition in 64 bits

def _view(i, window, sinks, keys):
    """What the tokens at places i attend of `keys` tokens."""
    j = torch.arange(keys, device="cuda")
    d = i[:, None] - j
    return (d >= 0) & ((d < (window or keys + 1)) | (j < sinks))


def _exact_rows(q, k, v, scale, seen):
    """One head in 64 bits: softmax(q k^T scale over what is seen) v, and the
    log of the softmax's sum.  seen: [rows, keys] truth values."""
    w = torch.where(seen, (q @ k.T) * scale, -math.inf)
    lse = torch.logsumexp(w, 1)
    p = torch.exp(w - lse[:, None])
    return p @ v, lse, p


def _exact_prefill(case, s):
    c, grads = case, case["op"] == "wbackward"
    lens, G, scale = _lens(c), c["H"] // c["Hkv"], c["dk"] ** -0.5
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    z = torch.sigmoid(s["z"].double()) if c["gate"] else None
    y, lse = torch.empty(q.shape[0], c["H"], c["dv"], dtype=torch.float64, device="cuda"), \
        torch.empty(q.shape[0], c["H"], dtype=torch.float64, device="cuda")
    if grads:
        dy = s["dy"].double()
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dz = torch.empty_like(y) if c["gate"] else None
    at = 0
    for n in lens:
        r = slice(at, at + n)
        at += n
        seen = _view(torch.arange(n, device="cuda"), c["window"], c["sinks"], n)
        for h in range(c["H"]):
            f = h // G
            o, l, p = _exact_rows(q[r, h], k[r, f], v[r, f], scale, seen)
            y[r, h], lse[r, h] = o if z is None else o * z[r, h], l
            if grads:
                do = dy[r, h]
                if z is not None:
                    dz[r, h] = do * o * z[r, h] * (1 - z[r, h])
                    do = do * z[r, h]
                dv[r, f] += p.T @ do
                ds = p * (do @ v[r, f].T - (do * o).sum(1, keepdim=True)) * scale
                dq[r, h] = ds @ k[r, f]
                dk[r, f] += ds.T @ q[r, h]
    return {"dq": dq, "dk": dk, "dv": dv, "dz": dz} if grads else (y, lse)


def _cached(pool, pages, n):
    """A slot's first n tokens of a pool, [heads, n, d] in 64 bits."""
    x = pool[pages].double().transpose(0, 1)
    return x.reshape(x.shape[0], x.shape[1] * x.shape[2], x.shape[3])[:, :n]


def _exact_tree(case, s):
    c = case
    B, T, H, G, page, scale = c["seqs"], c["T"], c["H"], c["H"] // c["Hkv"], c["page"], c["dk"] ** -0.5
    y = torch.empty(B, T, H, c["dv"], dtype=torch.float64, device="cuda")
    lse = torch.empty(B, T, H, dtype=torch.float64, device="cuda")
    paths = _paths(c)
    rows, table, lens = s["rows"].tolist(), s["table"].long(), s["lens"].tolist()
    for b in range(B):
        n = lens[rows[b]]
        at = table[rows[b], :_pages_of(n, page)]
        seen = torch.zeros(T, n + T, dtype=torch.bool, device="cuda")
        for t, path in enumerate(paths):  # the row's tokens in order, and its place behind them
            line = torch.cat([torch.arange(n, device="cuda"), torch.tensor(path, device="cuda") + n])
            view = _view(torch.tensor([n + len(path) - 1], device="cuda"), c["window"], c["sinks"], n + len(path))[0]
            seen[t, line[view]] = True
        seen = seen.repeat(G, 1)
        k, v = _cached(s["k_cache"], at, n), _cached(s["v_cache"], at, n)
        for f in range(c["Hkv"]):
            qs = s["q"][b, :, f * G:(f + 1) * G].double().transpose(0, 1).reshape(G * T, c["dk"])
            o, l, _ = _exact_rows(qs, torch.cat([k[f], s["k_new"][b, :, f].double()]),
                                  torch.cat([v[f], s["v_new"][b, :, f].double()]), scale, seen)
            y[b, :, f * G:(f + 1) * G] = o.view(G, T, -1).transpose(0, 1)
            lse[b, :, f * G:(f + 1) * G] = l.view(G, T).transpose(0, 1)
    if c["gate"]:
        y = y * torch.sigmoid(s["z"].double())
    return y, lse


def _exact_weigh(case, s):
    c = case
    G, page, scale = c["H"] // c["Hkv"], c["page"], c["dk"] ** -0.5
    total = s["weights"].double()
    slot, table, lens, cu = s["slot"].tolist(), s["table"].long(), s["lens"].tolist(), s["cu"].tolist()
    rows = s["rows"].long() if s["rows"] is not None else torch.arange(cu[-1], device="cuda")
    for b in range(c["seqs"]):
        n, mine = lens[slot[b]], rows[cu[b]:cu[b + 1]]
        k = _cached(s["k_cache"], table[slot[b], :_pages_of(n, page)], n)
        seen = _view(torch.arange(n - mine.numel(), n, device="cuda"), c["window"], c["sinks"], n)
        for h in range(c["H"]):
            x = (s["q"][mine, h].double() @ k[h // G].T) * scale - s["lse"][mine, h].double()[:, None]
            total[slot[b], :n] += torch.where(seen, torch.exp(x), 0.0).sum(0)
    return total


def exact(case, seed):
    if case["op"] == "evict":
        return None  # what it writes is whole numbers and copied rows
    s = prepare(case, seed)
    return {"wprefill": _exact_prefill, "wbackward": _exact_prefill, "wtree": _exact_tree, "weigh": _exact_weigh}[case["op"]](case, s)
