"""What is measured of the full-attention operators: the cases, their inputs,
their plain form in elementary torch operations, and the framework's calls.

The operators are those of the full-attention layers that stand between the
KDA layers of a hybrid model, for training and for serving:

  prefill    causal attention over packed prompts (grouped heads, optional
             sigmoid output gate):          kda_attn_prefill
  backward   its gradients:                 kda_attn_prefill_backward
  tree       attention of a tree of drafted tokens over a paged cache; one
             token per sequence is plain decode:  kda_attn_tree
  append     keys and values written into the cache's pages (a whole prompt,
             or the accepted path of a draft tree):  kda_cache_append
  fork       one step of a beam over the cache's pages: the old beams are
             freed, the new ones forked (full pages shared, the last one
             copied) and given pages for their next tokens:
             kda_cache_free, kda_cache_fork, kda_cache_reserve
  compact    the pages in use moved to the front of the pool:
             kda_cache_compact

A cache is two pools of pages, k_cache [pages, Hkv, page, dk] and v_cache
[pages, Hkv, page, dv], a page table [slots, max_pages] (-1: no page), the
slots' lengths in tokens and each page's count of table entries (0: free).
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
        dict(name="prefill_tiny_f32", op="prefill", dtype="f32", seqs=1, min_len=64, max_len=64, lens_seed=0,
             H=2, Hkv=2, dk=16, dv=16, gate=False),
        # a serving batch of ragged prompts, the hybrid's attention heads (192 with the rotary part, values 128, gated)
        dict(name="prefill_packed", op="prefill", dtype="bf16", seqs=12, min_len=1, max_len=2048, lens_seed=3,
             H=32, Hkv=32, dk=192, dv=128, gate=True),
        # one long prompt with grouped heads
        dict(name="prefill_long", op="prefill", dtype="bf16", seqs=1, min_len=16384, max_len=16384, lens_seed=0,
             H=32, Hkv=8, dk=128, dv=128, gate=False),
        # a small fp32 training batch of ragged sequences, gated, grouped heads
        dict(name="backward_packed_f32", op="backward", dtype="f32", seqs=6, min_len=5, max_len=500, lens_seed=5,
             H=8, Hkv=2, dk=64, dv=64, gate=True),
        # the 4096-token training layer
        dict(name="backward_layer_t4k", op="backward", dtype="bf16", seqs=1, min_len=4096, max_len=4096, lens_seed=0,
             H=32, Hkv=8, dk=128, dv=128, gate=False),
        # plain decode, 256 sequences, one token each
        dict(name="decode_b256", op="tree", dtype="bf16", seqs=256, min_len=1024, max_len=4096, lens_seed=7,
             T=1, chain=True, H=32, Hkv=8, dk=128, dv=128, page=64, gate=False),
        # 32 sequences with a tree of 16 drafted tokens each, gated
        dict(name="tree_b32_t16", op="tree", dtype="bf16", seqs=32, min_len=100, max_len=8000, lens_seed=8,
             T=16, chain=False, H=32, Hkv=8, dk=128, dv=128, page=64, gate=True),
        # one long conversation, a chain of four tokens: the split over the cache carries it
        dict(name="tree_b1_256k", op="tree", dtype="bf16", seqs=1, min_len=262144, max_len=262144, lens_seed=0,
             T=4, chain=True, H=32, Hkv=8, dk=128, dv=128, page=64, gate=False),
        # the accepted tokens of 256 draft trees written to the cache: latency
        dict(name="append_commit_b256", op="append", dtype="bf16", seqs=256, min_len=1, max_len=5, lens_seed=9,
             ctx_max=4000, tree=16, Hkv=8, dk=128, dv=128, page=64),
        # a packed batch of prompts written to the cache
        dict(name="append_prompts", op="append", dtype="bf16", seqs=8, min_len=900, max_len=8000, lens_seed=10,
             ctx_max=0, tree=0, Hkv=8, dk=128, dv=128, page=64),
        # one beam step: 64 parents with four beams each
        dict(name="fork_beams_256", op="fork", dtype="bf16", parents=64, beams=4, min_len=200, max_len=4000,
             lens_seed=11, more=8, Hkv=8, dk=128, dv=128, page=64),
        # a pool of which a third was freed at random
        dict(name="compact_8k_pages", op="compact", dtype="bf16", pages=8192, live=0.66, seqs=64, lens_seed=12,
             Hkv=8, dk=128, dv=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "backward", "tree", "tree", "append", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dk, dv = rng.choice([(128, 128), (128, 128), (192, 128), (64, 64), (32, 32), (16, 16)])
    H, Hkv = rng.choice([(32, 8), (32, 32), (8, 1), (8, 2), (32, 4)])
    seed = rng.randrange(1 << 30)
    heads = dict(H=H, Hkv=Hkv, dk=dk, dv=dv)
    cache = dict(Hkv=Hkv, dk=dk, dv=dv, page=rng.choice([16, 32, 64, 128]))
    most = int(2e9) // (Hkv * (dk + dv) * (2 if dtype == "bf16" else 4))  # tokens in 2 GB of cache
    if op in ("prefill", "backward"):
        seqs = rng.choice([1, 1, 2, 5, 16])
        longest = max(2, _log(rng, 16, (6000 if op == "prefill" else 4000) // (1 if seqs < 5 else 4)))
        return dict(op=op, dtype=dtype, seqs=seqs, min_len=max(1, longest // rng.choice([1, 2, 50])), max_len=longest,
                    lens_seed=seed, gate=rng.random() < 0.5, **heads)
    if op == "tree":
        seqs = _log(rng, 1, 200)
        longest = _log(rng, 30, min(200000, max(40, min(500000, most) // seqs)))
        return dict(op=op, dtype=dtype, seqs=seqs, min_len=max(0, longest // rng.choice([1, 3, 1000])),
                    max_len=longest, lens_seed=seed, T=rng.choice([1, 1, 4, 7, 16, 33]), chain=rng.random() < 0.3,
                    gate=rng.random() < 0.5, **heads, page=cache["page"])
    if op == "append":
        if rng.random() < 0.5:
            return dict(op=op, dtype=dtype, seqs=_log(rng, 1, 300), min_len=0, max_len=rng.choice([1, 4, 8]),
                        lens_seed=seed, ctx_max=_log(rng, 1, 4000), tree=16, **cache)
        seqs = _log(rng, 1, 16)
        return dict(op=op, dtype=dtype, seqs=seqs, min_len=1, max_len=_log(rng, 50, max(60, min(40000, most // 2) // seqs)), lens_seed=seed,
                    ctx_max=0, tree=0, **cache)
    if op == "fork":
        longest = _log(rng, 20, 4000)
        return dict(op=op, dtype=dtype, parents=_log(rng, 1, max(2, min(64, most // longest))), beams=rng.choice([1, 2, 4]),
                    min_len=max(1, longest // 10), max_len=longest, lens_seed=seed, more=rng.choice([1, 8, 70]), **cache)
    return dict(op=op, dtype=dtype, pages=_log(rng, 64, max(80, min(4000, most // cache["page"]))), live=rng.choice([0.1, 0.5, 0.66, 0.95]),
                seqs=_log(rng, 1, 64), lens_seed=seed, **cache)


def _lens(case, count=None):
    """The lengths of a case's sequences: the longest first named, the others
    anywhere between the two bounds."""
    r = random.Random(case["lens_seed"])
    n = case["seqs"] if count is None else count
    lens = [case["max_len"]] + [r.randint(case["min_len"], case["max_len"]) for _ in range(n - 1)]
    r.shuffle(lens)
    return lens


def _item(case):
    return 2 if case["dtype"] == "bf16" else 4


def _pages_of(n, page):
    return -(-n // page)


def _tree_visible(case):
    """Draft tokens that the tokens of one tree attend, themselves included."""
    if case["chain"]:
        return case["T"] * (case["T"] + 1) // 2
    return sum(len(_ancestors(_parents(case["T"], case["lens_seed"]), t)) for t in range(case["T"]))


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


def _fork_plan(case):
    return _lens(case, case["parents"])


def work(case):
    op, e = case["op"], _item(case)
    if op in ("prefill", "backward"):
        lens = _lens(case)
        T, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
        H, Hkv, dk, dv = case["H"], case["Hkv"], case["dk"], case["dv"]
        one = T * (H * dk + Hkv * (dk + dv) + H * dv * (2 if case["gate"] else 1)) * e + T * H * 4
        if op == "prefill":
            return {"bytes": one, "flops": 2 * (dk + dv) * pairs * H}
        # also reads dy; writes dq, dk, dv (and dz)
        return {"bytes": one + T * H * dv * e + T * (H * dk + Hkv * (dk + dv) + (H * dv if case["gate"] else 0)) * e,
                "flops": 2 * (3 * dk + 2 * dv) * pairs * H}
    if op == "tree":
        lens, T, H, Hkv, dk, dv = _lens(case), case["T"], case["H"], case["Hkv"], case["dk"], case["dv"]
        B, ctx = case["seqs"], sum(lens)
        entries = sum(_pages_of(n, case["page"]) for n in lens)
        return {"bytes": (ctx + B * T) * Hkv * (dk + dv) * e + B * T * H * (dk + dv * (2 if case["gate"] else 1)) * e
                + B * T * H * 4 + entries * 4 + (0 if case["chain"] else B * T * 8),
                "flops": 2 * (dk + dv) * H * (T * ctx + B * _tree_visible(case))}
    if op == "append":
        n = sum(_lens(case))
        return {"bytes": 2 * n * case["Hkv"] * (case["dk"] + case["dv"]) * e + n * 4 + case["seqs"] * 12, "flops": 0}
    page = case["page"]
    token = case["Hkv"] * (case["dk"] + case["dv"]) * e
    if op == "fork":
        lens = _fork_plan(case)
        old = _pages_of(case["max_len"], page)
        copied = sum(n % page for n in lens) * case["beams"]
        shared = sum(n // page for n in lens) * case["beams"]
        pages = _fork_pages(case)
        # the old beams' entries out, the new ones' in, their pages' counts, the free pages found, the rows copied
        return {"bytes": 2 * copied * token + 8 * case["parents"] * case["beams"] * old + 16 * shared + 4 * pages, "flops": 0}
    live = _live(case)
    kept = len(live)
    moved = sum(p >= kept for p in live)
    return {"bytes": 2 * moved * page * token + 8 * case["pages"] + 8 * case["pages"], "flops": 0}


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
    if case["op"] == "backward":
        s["dy"] = _normal(g, (T, H, dv), dt)
        s["out"], s["lse"] = _plain_prefill(s)
    return s


def _tree_inputs(case, seed):
    g, dt, r = _gen(seed), DTYPES[case["dtype"]], random.Random(seed)
    lens, B, T, page = _lens(case), case["seqs"], case["T"], case["page"]
    H, Hkv, dk, dv = case["H"], case["Hkv"], case["dk"], case["dv"]
    need = [_pages_of(n, page) for n in lens]
    width, pages = max(max(need), 1), sum(need) + 8
    slots = B + 3  # a server's table has rows that this batch does not use
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    row = r.sample(range(slots), B)
    table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    length = torch.zeros(slots, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[row[b], :need[b]] = order[at:at + need[b]]
        at += need[b]
    length[torch.tensor(row, device="cuda")] = _ints(lens)
    mask = None
    if not case["chain"]:
        parents = _parents(T, case["lens_seed"])
        words = [sum(1 << a for a in _ancestors(parents, t)) for t in range(T)]
        mask = torch.tensor(words, dtype=torch.int64, device="cuda").expand(B, T).contiguous()
    return dict(case=dict(case), longest=max(lens), rows=_ints(row), table=table, lens=length, mask=mask,
                q=_normal(g, (B, T, H, dk), dt), k_new=_normal(g, (B, T, Hkv, dk), dt),
                v_new=_normal(g, (B, T, Hkv, dv), dt), k_cache=_normal(g, (pages, Hkv, page, dk), dt),
                v_cache=_normal(g, (pages, Hkv, page, dv), dt),
                z=_normal(g, (B, T, H, dv), dt) if case["gate"] else None)


def _append_inputs(case, seed):
    g, dt, r = _gen(seed), DTYPES[case["dtype"]], random.Random(seed)
    counts, N, page = _lens(case), case["seqs"], case["page"]
    Hkv, dk, dv = case["Hkv"], case["dk"], case["dv"]
    fixed = random.Random(case["lens_seed"] + 1)  # the sizes go by the case, not by the seed
    ctx = [fixed.randint(0, case["ctx_max"]) for _ in counts]
    need = [_pages_of(a + n, page) for a, n in zip(ctx, counts)]
    pages, width = max(sum(need), 1) + 4, max(max(need), 1)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((N, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(N):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    total, tree = sum(counts), case["tree"]
    src = N * tree if tree else total
    rows = None
    if tree:  # an accepted path: rising positions in the sequence's tree
        rows = [b * tree + t for b, n in enumerate(counts) for t in sorted(r.sample(range(tree), n))]
        rows = _ints(rows) if rows else torch.zeros(0, dtype=torch.int32, device="cuda")
    cu = _ints(_cu(counts))
    return dict(case=dict(case), total=total, cu=cu, rows=rows, table=table, lens=_ints(ctx),
                k_new=_normal(g, (src, Hkv, dk), dt), v_new=_normal(g, (src, Hkv, dv), dt),
                k_cache=_normal(g, (pages, Hkv, page, dk), dt), v_cache=_normal(g, (pages, Hkv, page, dv), dt))


def _fork_pages(case):
    lens = _fork_plan(case)
    page = case["page"]
    beams = case["parents"] * case["beams"]
    return sum(_pages_of(n, page) for n in lens) + beams * (1 + _pages_of(case["more"] + page, page)) + \
        beams * _pages_of(case["max_len"], page) // 4 + 16


def _fork_inputs(case, seed):
    g, dt, r = _gen(seed), DTYPES[case["dtype"]], random.Random(seed)
    lens, page, Hkv, dk, dv = _fork_plan(case), case["page"], case["Hkv"], case["dk"], case["dv"]
    parents, beams = case["parents"], case["parents"] * case["beams"]
    pages = _fork_pages(case)
    width = _pages_of(case["max_len"] + case["more"], page) + 1
    slots = parents + beams
    order = list(range(pages))
    r.shuffle(order)
    table = torch.full((slots, width), -1, dtype=torch.int32)
    length = torch.zeros(slots, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        for j in range(_pages_of(n, page)):
            table[b, j] = order[at]
            refs[order[at]] += 1
            at += 1
        length[b] = n
    # the beams of the step before: each shares its parent's first pages and has one of its own
    for i in range(beams):
        p, d = i % parents, parents + i
        n = r.randint(1, lens[p])
        full = n // page
        table[d, :full] = table[p, :full]
        refs[table[p, :full].long()] += 1
        if n % page:
            table[d, full] = order[at]
            refs[order[at]] += 1
            at += 1
        length[d] = n
    src = [r.randrange(parents) for _ in range(beams)]
    k_cache, v_cache = _normal(g, (pages, Hkv, page, dk), dt), _normal(g, (pages, Hkv, page, dv), dt)
    s = dict(case=dict(case), table=table.cuda(), lens=length.cuda(), refs=refs.cuda(), k_cache=k_cache,
             v_cache=v_cache, src=_ints(src), dst=_ints(list(range(parents, slots))),
             new_lens=_ints([lens[p] + case["more"] for p in src]))
    return s


def _live(case):
    r = random.Random(case["lens_seed"])
    n = case["pages"]
    return sorted(r.sample(range(n), max(1, int(n * case["live"]))))


def _compact_inputs(case, seed):
    g, dt, r = _gen(seed), DTYPES[case["dtype"]], random.Random(seed)
    live = _live(case)
    slots, page = case["seqs"], case["page"]
    order = list(live)
    r.shuffle(order)
    width = _pages_of(len(live), slots) + 4
    table = torch.full((slots, width), -1, dtype=torch.int32)
    refs = torch.zeros(case["pages"], dtype=torch.int32)
    for i, p in enumerate(order):
        table[i % slots, i // slots] = p
        refs[p] = 1
    for s in range(1, slots, 2):  # every other slot shares a page of its neighbour
        j = _pages_of(len(live), slots)
        p = int(table[s - 1, 0])
        table[s, j] = p
        refs[p] += 1
    shape = (case["pages"], case["Hkv"], page)
    return dict(case=dict(case), table0=table.cuda(), refs0=refs.cuda(), table=table.cuda(), refs=refs.cuda(),
                k_cache=_normal(g, shape + (case["dk"],), dt), v_cache=_normal(g, shape + (case["dv"],), dt))


def prepare(case, seed):
    return {"prefill": _attn_inputs, "backward": _attn_inputs, "tree": _tree_inputs, "append": _append_inputs,
            "fork": _fork_inputs, "compact": _compact_inputs}[case["op"]](case, seed)


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
    return x.masked_fill_(t[None, :] > t[:, None], -math.inf), q, k


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
    n = _pages_of(s["longest"], page)
    at = s["table"][rows][:, :n].long().clamp(min=0)
    lens = s["lens"][rows]
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
    old = torch.arange(n * page, device=q.device) < lens[:, None]
    seen = torch.cat([old[:, None].expand(B, T, n * page), new], 2)
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


def _plain_append(s):
    page = s["case"]["page"]
    t = torch.arange(s["total"], device="cuda")
    n = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    pos = s["lens"][n].long() + t - s["cu"][n].long()
    at, off = s["table"][n, pos // page].long(), pos % page
    k, v = (s["k_new"], s["v_new"]) if s["rows"] is None else (s["k_new"][s["rows"].long()], s["v_new"][s["rows"].long()])
    s["k_cache"][at, :, off] = k
    s["v_cache"][at, :, off] = v
    return s["k_cache"], s["v_cache"]


def _lowest_free(refs, count):
    """The `count` lowest-numbered free pages."""
    return (refs == 0).to(torch.uint8).sort(descending=True, stable=True).indices[:count]


def _plain_fork(s):
    page, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    src, dst = s["src"].long(), s["dst"].long()
    beams, width = dst.numel(), table.shape[1]
    # the old beams go
    old = table[dst]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().to(torch.int32))
    table[dst] = -1
    # the new ones share the full pages and copy the rows of the last
    n = lens[src].long()
    full, part = n // page, n % page
    col = torch.arange(width, device="cuda")
    rows = torch.where(col < full[:, None], table[src], -1)
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).flatten().to(torch.int32))
    need = part > 0
    rank = need.cumsum(0) - 1
    new = _lowest_free(refs, beams)[rank.clamp(min=0)]
    last = table[src, full.clamp(max=width - 1)].long()
    last = torch.where(need, last, new)
    kept = (torch.arange(page, device="cuda") < part[:, None])[:, None, :, None]
    at = torch.where(need, new, s["k_cache"].shape[0])  # no page: a row behind the pool's own, dropped
    for name in ("k_cache", "v_cache"):
        pool = s[name]
        rows_of = torch.where(kept, pool[last], pool[new])
        put = need.nonzero()[:, 0]
        pool[at[put]] = rows_of[put]
    rows = torch.where((col == full[:, None]) & need[:, None], new[:, None].to(torch.int32), rows)
    refs.index_add_(0, new, need.to(torch.int32))
    lens[dst] = lens[src]
    # and get the pages that their next tokens need
    wants = (col < ((s["new_lens"].long() + page - 1) // page)[:, None]) & (rows < 0)
    rank = (wants.flatten().cumsum(0) - 1).clamp(min=0)
    free = _lowest_free(refs, wants.numel())
    new = free[rank.clamp(max=free.numel() - 1)].view_as(wants)
    rows = torch.where(wants, new.to(torch.int32), rows)
    refs.index_add_(0, new.flatten(), wants.flatten().to(torch.int32))
    table[dst] = rows
    return {"table": table, "lens": lens, "refs": refs, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    table, refs = s["table"], s["refs"]
    used = refs > 0
    count = used.sum()
    number = torch.arange(refs.numel(), device="cuda")
    src = (used & (number >= count)).nonzero()[:, 0]
    dst = (~used & (number < count)).nonzero()[:, 0]
    s["k_cache"][dst] = s["k_cache"][src]
    s["v_cache"][dst] = s["v_cache"][src]
    to = number.to(torch.int32)
    to[src] = dst.to(torch.int32)
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    return {"table": table, "refs": refs, "live": count.to(torch.int32).view(1), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


PLAIN = {"prefill": _plain_prefill, "backward": _plain_backward, "tree": _plain_tree, "append": _plain_append,
         "fork": _plain_fork, "compact": _plain_compact}


# -------------------------------------------------------- the framework's calls

def _own(s):
    from gated_delta_rule_64_amd import kda
    op = s["case"]["op"]
    if op == "prefill":
        return kda.kda_attn_prefill(s["q"], s["k"], s["v"], out_gate=s["z"], cu_seqlens=s["cu"])
    if op == "backward":
        return kda.kda_attn_prefill_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dy"], out_gate=s["z"],
                                             cu_seqlens=s["cu"])
    if op == "tree":
        return kda.kda_attn_tree(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                 tree_mask=s["mask"], out_gate=s["z"], slot_indices=s["rows"])
    if op == "append":
        kda.kda_cache_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                             rows=s["rows"])
        return s["k_cache"], s["v_cache"]
    if op == "fork":
        kda.kda_cache_free(s["dst"], s["table"], s["lens"], s["refs"])
        kda.kda_cache_fork(s["src"], s["dst"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["refs"])
        kda.kda_cache_reserve(s["dst"], s["new_lens"], s["case"]["page"], s["table"], s["lens"], s["refs"])
        return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "k_cache": s["k_cache"],
                "v_cache": s["v_cache"]}
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    live = kda.kda_cache_compact(s["k_cache"], s["v_cache"], s["table"], s["refs"])
    return {"table": s["table"], "refs": s["refs"], "live": live, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------- the definition in 64 bits

def _exact_rows(q, k, v, scale, seen):
    """One head in 64 bits: softmax(q k^T scale over what is seen) v, and the
    log of the softmax's sum.  seen: [rows, keys] truth values."""
    w = torch.where(seen, (q @ k.T) * scale, -math.inf)
    lse = torch.logsumexp(w, 1)
    p = torch.exp(w - lse[:, None])
    return p @ v, lse, p


def _exact_prefill(case, s):
    c, grads = case, case["op"] == "backward"
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
        seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
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


def _exact_tree(case, s):
    c = case
    B, T, H, G, page, scale = c["seqs"], c["T"], c["H"], c["H"] // c["Hkv"], c["page"], c["dk"] ** -0.5
    y = torch.empty(B, T, H, c["dv"], dtype=torch.float64, device="cuda")
    lse = torch.empty(B, T, H, dtype=torch.float64, device="cuda")
    parents = list(range(-1, T - 1)) if c["chain"] else _parents(T, c["lens_seed"])
    tree = torch.zeros(T, T, dtype=torch.bool, device="cuda")
    for t in range(T):
        tree[t, _ancestors(parents, t)] = True
    rows, table, lens = s["rows"].tolist(), s["table"].long(), s["lens"].tolist()
    for b in range(B):
        n = lens[rows[b]]
        at = table[rows[b], :_pages_of(n, page)]
        seen = torch.cat([torch.ones(T, n, dtype=torch.bool, device="cuda"), tree], 1).repeat(G, 1)
        k = s["k_cache"][at].double().transpose(0, 1).reshape(-1, at.numel() * page, c["dk"])[:, :n] \
            if n else torch.empty(c["Hkv"], 0, c["dk"], dtype=torch.float64, device="cuda")
        v = s["v_cache"][at].double().transpose(0, 1).reshape(-1, at.numel() * page, c["dv"])[:, :n] \
            if n else torch.empty(c["Hkv"], 0, c["dv"], dtype=torch.float64, device="cuda")
        for f in range(c["Hkv"]):
            qs = s["q"][b, :, f * G:(f + 1) * G].double().transpose(0, 1).reshape(G * T, c["dk"])
            o, l, _ = _exact_rows(qs, torch.cat([k[f], s["k_new"][b, :, f].double()]),
                                  torch.cat([v[f], s["v_new"][b, :, f].double()]), scale, seen)
            y[b, :, f * G:(f + 1) * G] = o.view(G, T, -1).transpose(0, 1)
            lse[b, :, f * G:(f + 1) * G] = l.view(G, T).transpose(0, 1)
    if c["gate"]:
        y = y * torch.sigmoid(s["z"].double())
    return y, lse


def exact(case, seed):
    if case["op"] not in ("prefill", "backward", "tree"):
        return None  # what these write is whole numbers and copied rows
    s = (_tree_inputs if case["op"] == "tree" else _attn_inputs)(case, seed)
    return (_exact_tree if case["op"] == "tree" else _exact_prefill)(case, s)
