"""Serving a DSA layer from a paged cache: the cases that are measured, each
operator's plain form in elementary torch operations, and the framework's call.

The cache of one layer lies in pages of `page` tokens: keys and values
[pages, page, 128], indexer keys [pages, page, 64] and pooled indexer keys
[pages, page / 4, 128] (the fp32 mean of four indexer keys as a bf16 pair, hi
in columns 0..63 and lo in 64..127).  block_table[b] lists sequence b's pages;
seq_lens[b] counts its tokens, the new ones among them; rows cu_q[b] ..
cu_q[b+1]-1 are its new tokens, the last of the sequence.

Operators ("op" of a case):
  append  new tokens' rows into their pages, and the pooled key of every pool
          of four that they complete
  fork    sequences forked (full pages shared, a partly filled last page
          copied), then the children freed: one step of parallel sampling
  compact used pages moved down over the free ones, tables and counts with them
  index   the new tokens' indexer scores over all complete earlier pools and
          the top-k of each row
  attn    the new tokens' attention over their selected pools and their own
          partial pool
"""
import math
import random

import torch

own = False

D, DI, HQ = 128, 64, 16


def listed():
    return [
        # one decoding step of a batch of 64 sequences writes its tokens: a latency case
        {"name": "append_decode_64", "op": "append", "B": 64, "q": 1, "ctx": 32768, "page": 64, "ragged": True},
        # two sequences' prompt chunks are written, 8192 and some thousand tokens, ends inside pages
        {"name": "append_chunk", "op": "append", "B": 2, "q": 8191, "ctx": 40001, "page": 64, "ragged": True},
        # 8 prompts sampled 4 times each
        {"name": "fork_8x4", "op": "fork", "B": 8, "children": 4, "ctx": 8190, "page": 64},
        # 32 long prompts sampled 8 times each, large pages: 256 last pages copied
        {"name": "fork_32x8", "op": "fork", "B": 32, "children": 8, "ctx": 65500, "page": 256},
        # a cache in which every third sequence has ended
        {"name": "compact_64", "op": "compact", "B": 64, "ctx": 16001, "page": 64},
        # one sequence decodes at the 131072-token context of the layer's benchmark
        {"name": "index_decode_1", "op": "index", "B": 1, "q": 1, "ctx": 131072, "page": 64, "Hi": 32, "topk": 512,
         "ragged": False},
        # a batch of 64 sequences of 13 to 131 thousand tokens decodes
        {"name": "index_decode_64", "op": "index", "B": 64, "q": 1, "ctx": 131072, "page": 64, "Hi": 32, "topk": 512,
         "ragged": True},
        # a prompt's chunk of 2048 tokens, the last of a context of 131072
        {"name": "index_chunk_2048", "op": "index", "B": 1, "q": 2048, "ctx": 131072, "page": 64, "Hi": 32,
         "topk": 512, "ragged": False},
        # one token attends to its 2048 selected keys: a latency case
        {"name": "attn_decode_1", "op": "attn", "B": 1, "q": 1, "ctx": 131072, "page": 64, "topk": 512,
         "ragged": False},
        # a batch of 64 sequences decodes
        {"name": "attn_decode_64", "op": "attn", "B": 64, "q": 1, "ctx": 65536, "page": 64, "topk": 512,
         "ragged": True},
        # 16 sequences verify up to 7 drafted tokens each, odd selection size, small pages
        {"name": "attn_draft_16x7", "op": "attn", "B": 16, "q": 7, "ctx": 30011, "page": 16, "topk": 255,
         "ragged": True},
        # a prompt's chunk of 4096 tokens, the last of a context of 131072
        {"name": "attn_chunk_4096", "op": "attn", "B": 1, "q": 4096, "ctx": 131072, "page": 64, "topk": 512,
         "ragged": False},
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "fork", "compact", "index", "index", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        B = logint(1, 128)
        q = rng.choice([1, logint(2, max(2, 16384 // B))])
        return {"op": op, "B": B, "q": q, "ctx": q + logint(16, 32768), "page": page, "ragged": rng.random() < 0.7}
    if op == "fork":
        return {"op": op, "B": logint(1, 32), "children": logint(1, 8), "ctx": logint(64, 65536), "page": page}
    if op == "compact":
        return {"op": op, "B": logint(2, 64), "ctx": logint(64, 16384), "page": page}
    # single tokens, drafted tokens, or a chunk of a prompt
    kind = rng.choice(["one", "draft", "chunk"])
    B = logint(1, 64) if kind != "chunk" else logint(1, 4)
    q = {"one": 1, "draft": rng.randint(2, 8), "chunk": logint(16, 2048 // B)}[kind]
    ctx = q + logint(16 if op == "attn" else 256, 131072 if kind == "one" else 65536)
    c = {"op": op, "B": B, "q": q, "ctx": ctx, "page": page, "topk": logint(8, 512), "ragged": rng.random() < 0.7}
    if op == "index":
        c["Hi"] = rng.choice([8, 16, 32, 32])
    return c


def lengths(case):
    """(new tokens, length with them) of each sequence."""
    r = random.Random("%d %d" % (case["B"], case["ctx"]))
    q, n = [], []
    for b in range(case["B"]):
        ragged = case.get("ragged", True) and b > 0
        qb = case.get("q", 1)
        qb = r.randint(1, qb) if ragged else qb
        q.append(qb)
        n.append(max(qb, int(case["ctx"] * r.uniform(0.1, 1.0))) if ragged else case["ctx"])
    return q, n


def work(case):
    q, n = lengths(case)
    T, page_bytes = sum(q), case["page"] * 704
    if case["op"] == "append":
        pools = sum(l // 4 - (l - a) // 4 for a, l in zip(q, n))
        older = sum(min((l - a) % 4, l - a) for a, l in zip(q, n))
        return {"bytes": T * 2 * 640 + pools * 256 + older * 128, "flops": pools * 5 * DI}
    if case["op"] == "fork":
        # the parents' rows read, the children's written; counts of shared pages read and written; last pages copied
        # and the counts searched for free pages; then the children's rows read and cleared
        c, P = case["children"], case["page"]
        rows = sum(l // P for l in n)
        part = sum(1 for l in n if l % P)
        return {"bytes": c * part * 2 * page_bytes + 4 * rows * (1 + 5 * c) + 8 * sum(-(-l // P) for l in n), "flops": 0}
    if case["op"] == "compact":
        used, total = used_pages(case)
        moved = sum(1 for p in used if p >= len(used))
        return {"bytes": moved * 2 * page_bytes + 8 * total + 8 * len(used), "flops": 0}
    pairs = sum(sum((l - a + j) // 4 for j in range(a)) for a, l in zip(q, n))
    if case["op"] == "index":
        Hi = case["Hi"]
        return {"bytes": sum((l - 1) // 4 for l in n) * 256 + T * (Hi * 132 + case["topk"] * 4),
                "flops": pairs * Hi * (2 * DI + 3)}
    k = case["topk"]
    keys = [[4 * min(k, (l - a + j) // 4) + (l - a + j) % 4 + 1 for j in range(a)] for a, l in zip(q, n)]
    kv = sum(min(sum(x), l) for x, l in zip(keys, n)) * 512
    return {"bytes": kv + T * (2 * HQ * D * 2 + HQ * 4 + k * 4), "flops": sum(sum(x) for x in keys) * HQ * D * 4}


def used_pages(case):
    """Pages in use and pages in all of a compaction case: page numbers are dealt to the sequences in turn, as a
    server's growing sequences take them, and every third sequence has ended."""
    _, n = lengths(case)
    P = case["page"]
    need = [-(-l // P) for l in n]
    used, p = [], 0
    for j in range(max(need)):
        for b in range(len(n)):
            if j < need[b]:
                if b % 3 != 2:
                    used.append(p)
                p += 1
    return used, p


class State:
    pass


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = State()
    s.case = dict(case)
    s.q, s.n = lengths(case)
    P, B = case["page"], case["B"]
    s.T, s.P = sum(s.q), P
    need = [-(-l // P) for l in s.n]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    def grid(*shape, step, top):
        # values on a grid of at most 8 bits, as an indexer quantised to 8 bits holds them: every sum of the
        # scores is exact in 32 bits, so that the selection is one and the same in any order of summing
        x = torch.randn(*shape, generator=g, device=dev)
        return (x / step).round_().clamp_(-top / step + 1, top / step - 1).mul_(step)

    op = case["op"]
    children = case.get("children", 0)
    spare = B * children
    if op == "compact":
        _, pages = used_pages(case)
    else:
        pages = sum(need) + spare + 3
    s.k = randn(pages, P, D) if op != "index" else torch.empty(pages, P, D, device=dev, dtype=torch.bfloat16)
    s.v = randn(pages, P, D) if op != "index" else torch.empty(pages, P, D, device=dev, dtype=torch.bfloat16)
    s.k_idx = grid(pages, P, DI, step=1 / 32, top=4).to(torch.bfloat16)
    s.khat = split(pool_mean(s.k_idx.view(-1, 4, DI).float())).view(pages, P // 4, 2 * DI)
    # the pages of a sequence lie anywhere in the cache
    width = max(need) + 2
    table = torch.full((B + spare, width), -1, dtype=torch.int32)
    if op == "compact":
        p = 0
        for j in range(max(need)):
            for b in range(B):
                if j < need[b]:
                    table[b, j] = p
                    p += 1
    else:
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        at = 0
        for b in range(B):
            table[b, : need[b]] = order[at : at + need[b]]
            at += need[b]
    lens = torch.tensor(s.n + [0] * spare, dtype=torch.int32)
    if op == "compact":
        table[2::3] = -1
        lens[2::3] = 0
    s.table, s.lens = table.to(dev), lens.to(dev)
    cu = [0]
    for x in s.q:
        cu.append(cu[-1] + x)
    s.cu = torch.tensor(cu, dtype=torch.int32, device=dev)
    if op in ("fork", "compact"):
        flat = s.table.view(-1)
        s.count = torch.zeros(pages, dtype=torch.int32, device=dev)
        s.count.index_add_(0, flat.clamp(min=0).long(), (flat >= 0).to(torch.int32))
        s.table0, s.count0 = s.table.clone(), s.count.clone()
        s.src = torch.arange(B, dtype=torch.int32, device=dev).repeat_interleave(max(children, 1))
        s.dst = torch.arange(B, B + spare, dtype=torch.int32, device=dev)
    elif op == "append":
        s.new_k, s.new_v = randn(s.T, D), randn(s.T, D)
        s.new_idx = randn(s.T, DI)
    elif op == "index":
        Hi = case["Hi"]
        s.q_idx = grid(s.T, Hi, DI, step=1 / 8, top=4).to(torch.bfloat16)
        s.w = torch.randint(0, 17, (s.T, Hi), generator=g, device=dev).float() / 16
    else:
        s.qq = randn(s.T, HQ, D)
        s.pool_idx = selection(s, case["topk"], g)
    if own:  # the handles that a serving program keeps: they hold the tensors above
        import long_context_sparse_index_gb300 as dsa
        s.cache = dsa.PagedCache(s.k, s.v, s.k_idx, s.khat)
        if op in ("fork", "compact"):
            s.pages = dsa.PageTable(s.table, s.lens, s.count)
        else:
            s.batch = dsa.PagedBatch(s.table, s.lens, s.cu)
    return s


def selection(s, topk, g):
    """A selection as the indexer gives it: pools that many rows of a sequence share, and pools of a row's own."""
    b, pos = rows(s)
    P = max(max(s.n) // 4, 1)
    liked = torch.rand(len(s.n), P, generator=g, device="cuda")
    x = liked[b] + torch.rand(s.T, P, generator=g, device="cuda")
    n = pos // 4
    x.masked_fill_(torch.arange(P, device="cuda") >= n[:, None], -1.0)
    k = min(topk, P)
    at = x.topk(k, dim=1).indices
    at = torch.where(torch.arange(k, device="cuda") < n[:, None], at, P).sort(dim=1).values
    out = torch.full((s.T, topk), -1, dtype=torch.int32, device="cuda")
    out[:, :k] = torch.where(at < P, at, -1)
    return out


def rows(s):
    """Sequence and position of each new token."""
    r = torch.arange(s.T, device=s.cu.device)
    cu = s.cu.long()
    b = torch.searchsorted(cu[1:], r, right=True)
    return b, s.lens.long()[b] - cu[b + 1] + r


def pool_mean(x):
    return ((x[:, 0] + x[:, 1]) + (x[:, 2] + x[:, 3])) * 0.25


def split(x):
    hi = x.to(torch.bfloat16)
    return torch.cat([hi, (x - hi.float()).to(torch.bfloat16)], dim=1)


def run(s):
    return globals()["run_" + s.case["op"]](s)


def run_append(s):
    if own:
        import long_context_sparse_index_gb300 as dsa
        dsa.dsa_cache_append(s.cache, s.batch, s.new_k, s.new_v, s.new_idx)
        return {"k": s.k, "v": s.v, "k_idx": s.k_idx, "khat": s.khat}
    b, pos = rows(s)
    slot = s.table[b, pos // s.P].long() * s.P + pos % s.P
    s.k.view(-1, D)[slot] = s.new_k
    s.v.view(-1, D)[slot] = s.new_v
    s.k_idx.view(-1, DI)[slot] = s.new_idx
    pool = slot // 4  # every row writes its pool: the pooled key if the pool is complete, else what was there
    four = s.k_idx.view(-1, DI)[4 * pool[:, None] + torch.arange(4, device=pool.device)].float()
    whole = (pos | 3) < s.lens.long()[b]
    khat = s.khat.view(-1, 2 * DI)
    khat[pool] = torch.where(whole[:, None], split(pool_mean(four)), khat[pool])
    return {"k": s.k, "v": s.v, "k_idx": s.k_idx, "khat": s.khat}


def run_fork(s):
    if own:
        import long_context_sparse_index_gb300 as dsa
        taken = dsa.dsa_cache_fork(s.cache, s.pages, s.src, s.dst)
        table, count, lens = s.table[s.case["B"]:].clone(), s.count.clone(), s.lens.clone()
        dsa.dsa_cache_free(s.cache, s.pages, s.dst)
        return [taken, table, count, lens, s.table, s.count, s.lens, s.k, s.v, s.k_idx, s.khat]
    src, dst = s.src.long(), s.dst.long()
    P, width = s.P, s.table.shape[1]
    n = s.lens[src].long()
    part = n % P != 0
    free = torch.sort((s.count != 0).to(torch.int32), stable=True).indices  # free pages first, the lowest first
    fresh = free[part.long().cumsum(0) - 1]
    row = s.table[src]
    at = torch.arange(width, device=row.device)
    last = (n // P)[:, None]
    old = torch.where(part, row.gather(1, last.clamp(max=width - 1))[:, 0].long(), 0)
    to = torch.where(part, fresh, 0)  # where nothing is copied, page 0 is copied onto itself
    for_full = (at < last).to(torch.int32)
    s.count.index_add_(0, row.clamp(min=0).long().view(-1), for_full.view(-1))
    s.count.index_add_(0, to, part.to(torch.int32))
    s.table[dst] = torch.where(at < last, row, torch.where((at == last) & part[:, None], to[:, None], -1).int())
    s.lens[dst] = n.int()
    s.k[to], s.v[to], s.k_idx[to], s.khat[to] = s.k[old], s.v[old], s.k_idx[old], s.khat[old]
    taken = part.int().sum(dim=0, keepdim=True).int()
    table, count, lens = s.table[s.case["B"]:].clone(), s.count.clone(), s.lens.clone()
    row = s.table[dst]
    s.count.index_add_(0, row.clamp(min=0).long().view(-1), -(row >= 0).to(torch.int32).view(-1))
    s.table[dst] = -1
    s.lens[dst] = 0
    return [taken, table, count, lens, s.table, s.count, s.lens, s.k, s.v, s.k_idx, s.khat]


def run_compact(s):
    s.table.copy_(s.table0)  # the fragmented cache again
    s.count.copy_(s.count0)
    if own:
        import long_context_sparse_index_gb300 as dsa
        info = dsa.dsa_cache_compact(s.cache, s.pages)
        return [info, s.table, s.count, s.k, s.v, s.k_idx, s.khat]
    N = s.count.shape[0]
    at = torch.arange(N, device=s.count.device)
    is_used = s.count != 0
    used = is_used.sum()
    hole = ~is_used & (at < used)
    high = is_used & (at >= used)
    to = torch.sort((~hole).to(torch.int32), stable=True).indices  # the k-th hole
    rank = high.long().cumsum(0) - 1
    new = torch.where(high, to[rank.clamp(min=0)], at)  # where every page goes; a free one stays
    # every page below `used` takes what comes to it (itself, unless it is a hole)
    come = at.clone().scatter_(0, torch.where(high, new, N - 1 - at * 0), torch.where(high, at, N - 1))
    come = torch.where(hole, come, at)
    s.k.copy_(s.k[come]), s.v.copy_(s.v[come]), s.k_idx.copy_(s.k_idx[come]), s.khat.copy_(s.khat[come])
    s.count.copy_(torch.where(at < used, s.count[come], 0))
    s.table.copy_(torch.where(s.table >= 0, new[s.table.clamp(min=0).long()].int(), s.table))
    return [torch.stack([used, high.sum()]).int(), s.table, s.count, s.k, s.v, s.k_idx, s.khat]


def run_index(s):
    topk = s.case["topk"]
    if own:
        import long_context_sparse_index_gb300 as dsa
        return dsa.dsa_paged_index_topk(s.cache, s.batch, s.q_idx, s.w, topk)
    b, pos = rows(s)
    B, Q, Hi = len(s.n), max(s.q), s.w.shape[1]
    P, per = max(max(s.n) // 4, 1), s.P // 4
    p = torch.arange(P, device=b.device)
    kh = s.khat.view(-1, 2 * DI)[s.table[:, p // per].clamp(min=0).long() * per + p % per]
    keys = kh[..., :DI].float() + kh[..., DI:].float()  # [B, P, DI]
    cu = s.cu.long()
    pad = (cu[:B, None] + torch.arange(Q, device=b.device)).clamp(max=s.T - 1)  # rows in a rectangle [B, Q]
    x = torch.bmm(s.q_idx[pad].view(B, Q * Hi, DI).float(), keys.transpose(1, 2)).view(B, Q, Hi, P)
    score = x.clamp_(min=0).mul_(s.w[pad][..., None]).sum(dim=2)
    score = score[b, torch.arange(s.T, device=b.device) - cu[b]]  # [T, P]
    n = pos // 4
    score.masked_fill_(p >= n[:, None], -math.inf)
    k = min(topk, P)
    at = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k]
    at = torch.where(torch.arange(k, device=b.device) < n[:, None], at, P).sort(dim=1).values
    out = torch.full((s.T, topk), -1, dtype=torch.int32, device=b.device)
    out[:, :k] = torch.where(at < P, at, -1)
    return out


def run_attn(s):
    if own:
        import long_context_sparse_index_gb300 as dsa
        return dsa.dsa_paged_sparse_attn_fwd(s.cache, s.batch, s.qq, s.pool_idx)
    b, pos = rows(s)
    four = torch.arange(4, device=b.device)
    sel = s.pool_idx.long()
    tok = torch.cat([(4 * sel[:, :, None] + four).view(s.T, -1), 4 * (pos // 4)[:, None] + four], dim=1)
    ok = (tok >= 0) & (tok <= pos[:, None])
    tok = torch.where(ok, tok, 0)
    slot = s.table[b[:, None], tok // s.P].long() * s.P + tok % s.P
    x = torch.bmm(s.qq.float(), s.k.view(-1, D)[slot].float().transpose(1, 2)) * (1 / math.sqrt(D))
    x.masked_fill_(~ok[:, None, :], -math.inf)
    top = x.amax(dim=2, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(dim=2, keepdim=True)
    o = torch.bmm(p, s.v.view(-1, D)[slot].float()) / total
    return o.to(torch.bfloat16), (top + torch.log(total))[..., 0]


def exact(case, seed):
    if case["op"] == "append":
        s = prepare(case, seed)
        out = {x: getattr(s, x).double() for x in ("k", "v", "k_idx", "khat")}
        table, r = s.table.tolist(), 0
        at, pool, first = [], [], []
        for b, (a, l) in enumerate(zip(s.q, s.n)):
            for i in range(l - a, l):
                at.append(table[b][i // s.P] * s.P + i % s.P)
            for i in range((l - a) // 4 * 4, l - 3, 4):
                pool.append((table[b][i // s.P] * s.P + i % s.P) // 4)
        at = torch.tensor(at, device="cuda")
        for x, y in (("k", s.new_k), ("v", s.new_v), ("k_idx", s.new_idx)):
            flat = out[x].view(-1, y.shape[1])
            flat[at] = y.double()
        if pool:
            pool = torch.tensor(pool, device="cuda")
            mean = out["k_idx"].view(-1, 4, DI)[pool].mean(dim=1)
            hi = mean.to(torch.bfloat16).double()
            out["khat"].view(-1, 2 * DI)[pool] = torch.cat([hi, mean - hi], dim=1)
        return out
    if case["op"] != "attn":
        return None  # page numbers, counts, copies and pool numbers
    s = prepare(case, seed)
    o = torch.empty(s.T, HQ, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(s.T, HQ, dtype=torch.float64, device="cuda")
    r = 0
    for b, (a, l) in enumerate(zip(s.q, s.n)):
        # this sequence's keys and values end to end
        of = s.table[b, : -(-l // s.P)].long()
        k = s.k[of].view(-1, D)[:l].double()
        v = s.v[of].view(-1, D)[:l].double()
        for i in range(l - a, l):
            pools = s.pool_idx[r]
            keep = torch.zeros((l + 3) // 4, dtype=torch.bool, device="cuda")
            keep[i // 4] = True
            keep.index_fill_(0, torch.where(pools < 0, i // 4, pools).long(), True)
            at = keep.repeat_interleave(4)[: i + 1].nonzero()[:, 0]
            x = s.qq[r].double() @ k[at].T / math.sqrt(D)
            lse[r] = torch.logsumexp(x, dim=1)
            o[r] = torch.softmax(x, dim=1) @ v[at]
            r += 1
    return o, lse
