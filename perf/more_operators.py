"""A DSA layer with rotated positions, and its cache held in 4 bits: the cases that are measured, each operator's plain
form in elementary torch operations, and the framework's call.

Rotation.  A table cos_sin [positions, R] (fp32: cosines in columns 0..R/2-1, sines in the rest) turns the first R
dimensions of a head: pair j of the row at position p becomes (a c - b s, b c + a s), with c = cos_sin[p, j] and s =
cos_sin[p, R/2 + j].  A pair is (j, j + R/2), or (2j, 2j + 1) where the case says "inter".  The inverse turns back: it
is the rotation's gradient.

The cache in 4 bits.  Pages of `page` tokens: kv uint8 [pages, page / 4, 576], indexer keys [pages, page, 64] and pooled
indexer keys [pages, page / 4, 128] (bf16, as in the bf16 cache).  The 128 values of a key or a value lie in 8 groups of
16; a group has one scale, its values are 4-bit codes e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign in bit 3) and stand
for code * scale / 16.  A scale is 8 bits without a sign, 5 of exponent and 3 of mantissa, the upper half of a half
precision number less its sign: scale = bits << 7 read as fp16.  For x_1..x_16, in bf16: scale = the nearest to
16 max|x| / 6, at most 10240, and code = the nearest to 16 x / scale (ties to even in both).
The 576 bytes of a pool of four tokens t:
  0    keys' codes [t][64]: byte b holds dimension 2b in its low half and 2b + 1 in its high one
  256  values' codes [group][t][8], the same order within a group
  512  keys' scales [group / 2][t % 2][t / 2][group % 2]
  544  values' scales [group][t]

Operators ("op" of a case):
  rope     a tensor of heads turned, or turned back
  append   new tokens' rows into the pages of a bf16 cache, keys and indexer keys turned on the way, and the step's
           queries turned with them
  append4  the same into a cache in 4 bits; the written rows are read back as the values that they stand for
  attn4    the new tokens' attention over their selected pools and their own partial pool of a cache in 4 bits
"""
import math
import random

import torch

own = False

D, DI, HQ = 128, 64, 16
POOL = 576


def listed():
    return [
        # queries of one step of 61 sequences, before a contiguous attention: a latency case
        {"name": "rope_rows_61", "op": "rope", "S": 61, "H": 16, "D": 128, "R": 128, "inter": False, "inverse": False,
         "packed": True},
        # the queries of the layer's benchmark sequence, in training
        {"name": "rope_q_131072", "op": "rope", "S": 131072, "H": 16, "D": 128, "R": 128, "inter": False,
         "inverse": False, "packed": False},
        # the gradient of a packed batch's indexer queries, half of their dimensions turned
        {"name": "rope_idx_back", "op": "rope", "S": 40001, "H": 32, "D": 64, "R": 32, "inter": True, "inverse": True,
         "packed": True},
        # one decoding step of a batch of 64 sequences: a latency case
        {"name": "append_decode_64", "op": "append", "B": 64, "q": 1, "ctx": 32768, "page": 64, "R": 128, "Ri": 64,
         "inter": False, "Hi": 32, "ragged": True},
        # 16 sequences with up to 7 drafted tokens, small pages
        {"name": "append_draft_16x7", "op": "append", "B": 16, "q": 7, "ctx": 30011, "page": 16, "R": 64, "Ri": 32,
         "inter": True, "Hi": 8, "ragged": True},
        # two sequences' prompt chunks, 8191 and some thousand tokens, ends inside pages
        {"name": "append_chunk", "op": "append", "B": 2, "q": 8191, "ctx": 40001, "page": 64, "R": 128, "Ri": 64,
         "inter": False, "Hi": 32, "ragged": True},
        # the same decoding step and chunk into 4 bits
        {"name": "append4_decode_64", "op": "append4", "B": 64, "q": 1, "ctx": 32768, "page": 64, "R": 128, "Ri": 64,
         "inter": False, "Hi": 32, "ragged": True},
        {"name": "append4_chunk", "op": "append4", "B": 2, "q": 8191, "ctx": 40001, "page": 64, "R": 64, "Ri": 64,
         "inter": True, "Hi": 32, "ragged": True},
        # one token attends to its 2048 selected keys: a latency case
        {"name": "attn4_decode_1", "op": "attn4", "B": 1, "q": 1, "ctx": 131072, "page": 64, "topk": 512,
         "ragged": False},
        # a batch of 64 sequences decodes
        {"name": "attn4_decode_64", "op": "attn4", "B": 64, "q": 1, "ctx": 65536, "page": 64, "topk": 512,
         "ragged": True},
        # 16 sequences verify up to 7 drafted tokens each, odd selection size, small pages
        {"name": "attn4_draft_16x7", "op": "attn4", "B": 16, "q": 7, "ctx": 30011, "page": 16, "topk": 255,
         "ragged": True},
        # a prompt's chunk of 4096 tokens, the last of a context of 131072
        {"name": "attn4_chunk_4096", "op": "attn4", "B": 1, "q": 4096, "ctx": 131072, "page": 64, "topk": 512,
         "ragged": False},
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "append", "append4", "attn4", "attn4"])
    inter = rng.random() < 0.5
    if op == "rope":
        d, h = rng.choice([64, 128]), rng.choice([1, 4, 7, 16, 32])
        return {"op": op, "S": logint(1, min(131072, 131072 * 16 * 128 // (h * d))), "H": h, "D": d,
                "R": 16 * rng.randint(1, d // 16), "inter": inter, "inverse": rng.random() < 0.5,
                "packed": rng.random() < 0.5}
    page = rng.choice([16, 32, 64, 128, 256])
    if op != "attn4":
        B = logint(1, 128)
        q = rng.choice([1, logint(2, max(2, 8192 // B))])
        return {"op": op, "B": B, "q": q, "ctx": q + logint(16, 32768), "page": page, "R": 16 * rng.randint(1, 8),
                "Ri": 16 * rng.randint(1, 4), "inter": inter, "Hi": rng.choice([8, 16, 32, 32]),
                "ragged": rng.random() < 0.7}
    # single tokens, drafted tokens, or a chunk of a prompt
    kind = rng.choice(["one", "draft", "chunk"])
    B = logint(1, 64) if kind != "chunk" else logint(1, 4)
    q = {"one": 1, "draft": rng.randint(2, 8), "chunk": logint(16, 2048 // B)}[kind]
    ctx = q + logint(16, 131072 if kind == "one" else 65536)
    return {"op": op, "B": B, "q": q, "ctx": ctx, "page": page, "topk": logint(8, 512), "ragged": rng.random() < 0.7}


def lengths(case):
    """(new tokens, length with them) of each sequence."""
    r = random.Random("%d %d" % (case["B"], case["ctx"]))
    q, n = [], []
    for b in range(case["B"]):
        ragged = case["ragged"] and b > 0
        qb = r.randint(1, case["q"]) if ragged else case["q"]
        q.append(qb)
        n.append(max(qb, int(case["ctx"] * r.uniform(0.1, 1.0))) if ragged else case["ctx"])
    return q, n


def work(case):
    if case["op"] == "rope":
        rows = case["S"]
        return {"bytes": rows * (case["H"] * case["D"] * 4 + case["R"] * 4 + (4 if case["packed"] else 0)),
                "flops": rows * case["H"] * case["R"] * 3}
    q, n = lengths(case)
    T = sum(q)
    if case["op"] != "attn4":
        pools = sum(l // 4 - (l - a) // 4 for a, l in zip(q, n))
        older = sum(min((l - a) % 4, l - a) for a, l in zip(q, n))
        heads = HQ * case["R"] + case["Hi"] * case["Ri"]
        held = 2 * D * 2 if case["op"] == "append" else 2 * 72 + 2 * D * 2  # in 4 bits: read back, too
        return {"bytes": T * (640 + held + DI * 2 + (HQ * D + case["Hi"] * DI) * 4 + (case["R"] + case["Ri"]) * 4)
                + pools * 256 + older * 128,
                "flops": T * 3 * (heads + case["R"] + case["Ri"]) + pools * 5 * DI}
    k = case["topk"]
    keys = [[4 * min(k, (l - a + j) // 4) + (l - a + j) % 4 + 1 for j in range(a)] for a, l in zip(q, n)]
    kv = sum(min(sum(x), l) for x, l in zip(keys, n)) * 144
    return {"bytes": kv + T * (2 * HQ * D * 2 + HQ * 4 + k * 4), "flops": sum(sum(x) for x in keys) * HQ * D * 4}


class State:
    pass


def angles(positions, R):
    """cos_sin [positions, R], from angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(R // 2, device="cuda", dtype=torch.float64) * 2 / R)
    x = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([x.cos(), x.sin()], dim=1).float()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = State()
    s.case = dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    if case["op"] == "rope":
        S = case["S"]
        s.x = randn(S, case["H"], case["D"])
        s.table = angles(S, case["R"])
        s.pos = None
        if case["packed"]:  # sequences of some lengths, one behind another
            cut = torch.rand(S, generator=g, device=dev) < 8 / S
            at = torch.arange(S, device=dev)
            s.pos = (at - torch.where(cut, at, 0).cummax(0).values).int()
        if own:
            import long_context_sparse_index_gb300 as dsa
            s.rope = dsa.Rope(s.table, interleaved=case["inter"])
        return s
    s.q, s.n = lengths(case)
    P, B = case["page"], case["B"]
    s.T, s.P = sum(s.q), P
    need = [-(-l // P) for l in s.n]
    pages = sum(need) + 3
    # the pages of a sequence lie anywhere in the cache
    table = torch.full((B, max(need) + 2), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = 0
    for b in range(B):
        table[b, : need[b]] = order[at : at + need[b]]
        at += need[b]
    s.table, s.lens = table.to(dev), torch.tensor(s.n, dtype=torch.int32, device=dev)
    cu = [0]
    for x in s.q:
        cu.append(cu[-1] + x)
    s.cu = torch.tensor(cu, dtype=torch.int32, device=dev)
    s.k_idx = randn(pages, P, DI)
    s.khat = split(pool_mean(s.k_idx.view(-1, 4, DI).float())).view(pages, P // 4, 2 * DI)
    if case["op"] == "attn4":
        s.kv = torch.empty(pages, P // 4, POOL, dtype=torch.uint8, device=dev)
        few = max(1, (1 << 19) // P)
        for p in range(0, pages, few):
            m = min(few, pages - p) * P // 4
            pools = torch.cat([pack(*quantise(randn(m, 4, D))), pack(*quantise(randn(m, 4, D)))], 1)
            s.kv[p : p + few].view(-1, POOL)[:] = pools[:, ORDER.to(dev)]
        s.qq = randn(s.T, HQ, D)
        s.pool_idx = selection(s, case["topk"], g)
    else:
        if case["op"] == "append":
            s.k, s.v = randn(pages, P, D), randn(pages, P, D)
        else:
            s.kv = torch.zeros(pages, P // 4, POOL, dtype=torch.uint8, device=dev)
        s.new_k, s.new_v, s.new_idx = randn(s.T, D), randn(s.T, D), randn(s.T, DI)
        s.new_q, s.new_qi = randn(s.T, HQ, D), randn(s.T, case["Hi"], DI)
        s.turn, s.turn_idx = angles(max(s.n), case["R"]), angles(max(s.n), case["Ri"])
    if own:  # the handles that a serving program keeps: they hold the tensors above
        import long_context_sparse_index_gb300 as dsa
        s.cache = dsa.PagedCache(s.k, s.v, s.k_idx, s.khat) if case["op"] == "append" else \
            dsa.PagedCache4(s.kv, s.k_idx, s.khat)
        s.batch = dsa.PagedBatch(s.table, s.lens, s.cu)
        if case["op"] != "attn4":
            s.rope = dsa.Rope(s.turn, interleaved=case["inter"])
            s.rope_idx = dsa.Rope(s.turn_idx, interleaved=case["inter"])
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


def turned(x, cs, inter, kind=torch.float32):
    """x [rows, heads, d] bf16 turned by cs [rows, R]; `kind`: the arithmetic's type."""
    R = cs.shape[1]
    c, s = cs[:, None, : R // 2].to(kind), cs[:, None, R // 2 :].to(kind)
    head = x[..., :R].to(kind)
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = head[..., : R // 2], head[..., R // 2 :]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y.float().to(torch.bfloat16), x[..., R:]], dim=-1)


# the values of the 16 codes, and each byte of a pool's 576 in the order in which pack() leaves them
CODES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def _order():
    at = torch.arange(POOL)
    k, v = at[:288], at[288:]  # pack(): codes [t][64], then scales [t][8]
    kc, ks = k[:256], k[256:].view(2, 2, 4, 2).permute(2, 1, 0, 3)  # [t/2][t%2][group/2][group%2] ->
    vc, vs = v[:256].view(4, 8, 8).transpose(0, 1), v[256:].view(4, 8).T
    return torch.cat([x.reshape(-1) for x in (kc, vc, ks, vs)])


ORDER = _order()
# the 144 bytes of each of a pool's four tokens
TOKEN = torch.cat([torch.arange(256) // 64, torch.arange(32) // 8]).repeat(2)[ORDER]
PLACES = torch.stack([(TOKEN == t).nonzero()[:, 0] for t in range(4)])


def quantise(x):
    """x [n, 4, 128] bf16: codes [n, 4, 128] (uint8) and scales' bits [n, 4, 8] (uint8)."""
    y = 16 * x.float().view(-1, 4, 8, 16)
    m = y.abs().amax(dim=3) / 6
    e = torch.frexp(m).exponent.clamp(min=-13) - 1  # 2^e <= m, or the smallest normal number's
    step = torch.ldexp(torch.ones_like(m), e - 3)
    scale = (torch.round(m / step) * step).clamp(max=10240.0)
    r = torch.where(scale[..., None] > 0, y / scale[..., None], 0.0)
    a = r.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code += torch.where(y < 0, 8, 0).to(torch.uint8)
    bits = (scale.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)
    return code.view(-1, 4, D), bits


def pack(code, bits):
    """The 288 bytes of a pool's keys (or values): codes, then scales."""
    two = code.view(-1, 4, D // 2, 2)
    return torch.cat([(two[..., 0] | two[..., 1] << 4).view(-1, 256), bits.view(-1, 32)], dim=1)


def values(pool):
    """pool [n, 576] uint8: keys and values [n, 4, 128] fp32 that they stand for."""
    back = torch.empty_like(pool)
    back[:, ORDER.to(pool.device)] = pool
    out = []
    for x in (back[:, :288], back[:, 288:]):
        two = x[:, :256].reshape(-1, 4, 64)
        code = CODES.to(pool.device)[torch.stack([two & 15, two >> 4], dim=-1).long()].view(-1, 4, 8, 16)
        scale = (x[:, 256:].to(torch.int16) << 7).view(torch.float16).float().view(-1, 4, 8, 1)
        out.append((code * scale / 16).view(-1, 4, D))
    return out


def run(s):
    return globals()["run_" + s.case["op"]](s)


def run_rope(s):
    if own:
        import long_context_sparse_index_gb300 as dsa
        return dsa.dsa_rope(s.x, s.rope, positions=s.pos, inverse=s.case["inverse"])
    cs = s.table if s.pos is None else s.table[s.pos.long()]
    if s.case["inverse"]:
        R = cs.shape[1]
        cs = torch.cat([cs[:, : R // 2], -cs[:, R // 2 :]], dim=1)
    return turned(s.x, cs, s.case["inter"])


def append_indexer(s, b, pos, kind):
    """The indexer keys' part of an append: rows, and the pooled key of every pool that they complete."""
    slot = s.table[b, pos // s.P].long() * s.P + pos % s.P
    s.k_idx.view(-1, DI)[slot] = turned(s.new_idx[:, None], s.turn_idx[pos], s.case["inter"], kind)[:, 0]
    pool = slot // 4  # every row writes its pool: the pooled key if the pool is complete, else what was there
    four = s.k_idx.view(-1, DI)[4 * pool[:, None] + torch.arange(4, device=pool.device)].float()
    whole = (pos | 3) < s.lens.long()[b]
    khat = s.khat.view(-1, 2 * DI)
    khat[pool] = torch.where(whole[:, None], split(pool_mean(four)), khat[pool])
    return slot


def run_append(s):
    if own:
        import long_context_sparse_index_gb300 as dsa
        q, qi = dsa.dsa_cache_append_rope(s.cache, s.batch, s.new_k, s.new_v, s.new_idx, s.rope, s.rope_idx,
                                          q=s.new_q, q_idx=s.new_qi)
        return {"k": s.k, "v": s.v, "k_idx": s.k_idx, "khat": s.khat, "q": q, "q_idx": qi}
    b, pos = rows(s)
    inter = s.case["inter"]
    slot = append_indexer(s, b, pos, torch.float32)
    s.k.view(-1, D)[slot] = turned(s.new_k[:, None], s.turn[pos], inter)[:, 0]
    s.v.view(-1, D)[slot] = s.new_v
    return {"k": s.k, "v": s.v, "k_idx": s.k_idx, "khat": s.khat, "q": turned(s.new_q, s.turn[pos], inter),
            "q_idx": turned(s.new_qi, s.turn_idx[pos], inter)}


def run_append4(s):
    if own:
        import long_context_sparse_index_gb300 as dsa
        q, qi = dsa.dsa_cache4_append(s.cache, s.batch, s.new_k, s.new_v, s.new_idx, s.rope, s.rope_idx,
                                      q=s.new_q, q_idx=s.new_qi)
        k, v = dsa.dsa_cache4_read(s.cache, s.batch, s.T)
        return {"k": k, "v": v, "k_idx": s.k_idx, "khat": s.khat, "q": q, "q_idx": qi}
    b, pos = rows(s)
    inter = s.case["inter"]
    # the codes' borders: in 64 bits, so that a key's code does not hang on an order of operations
    slot = append_indexer(s, b, pos, torch.float64)
    k = turned(s.new_k[:, None], s.turn[pos], inter, torch.float64)[:, 0]
    # a row's bytes go to the places of its token t within its pool
    t = slot % 4
    halves = [pack(*quantise(x[:, None].expand(-1, 4, -1).contiguous())) for x in (k, s.new_v)]
    place = PLACES.to(t.device)[t]  # [rows, 144]
    byte = torch.cat(halves, dim=1)[:, ORDER.to(t.device)].gather(1, place)
    s.kv.view(-1)[slot[:, None] // 4 * POOL + place] = byte
    kk, vv = values(s.kv.view(-1, POOL)[slot // 4])
    r = torch.arange(s.T, device=t.device)
    return {"k": kk[r, t].to(torch.bfloat16), "v": vv[r, t].to(torch.bfloat16), "k_idx": s.k_idx, "khat": s.khat,
            "q": turned(s.new_q, s.turn[pos], inter), "q_idx": turned(s.new_qi, s.turn_idx[pos], inter)}


def run_attn4(s):
    if own:
        import long_context_sparse_index_gb300 as dsa
        return dsa.dsa_paged4_sparse_attn_fwd(s.cache, s.batch, s.qq, s.pool_idx)
    b, pos = rows(s)
    per = s.P // 4
    pool = torch.cat([s.pool_idx.long(), (pos // 4)[:, None]], dim=1)
    tok = 4 * pool[:, :, None] + torch.arange(4, device=b.device)
    ok = ((pool[:, :, None] >= 0) & (tok <= pos[:, None, None])).flatten(1)
    pool = pool.clamp(min=0)
    at = s.table[b[:, None], pool // per].long() * per + pool % per
    k, v = values(s.kv.view(-1, POOL)[at].view(-1, POOL))
    k, v = k.view(s.T, -1, D), v.view(s.T, -1, D)
    v = torch.where(ok[:, :, None], v, 0.0)
    x = torch.bmm(s.qq.float(), k.transpose(1, 2)) * (1 / math.sqrt(D))
    x.masked_fill_(~ok[:, None, :], -math.inf)
    top = x.amax(dim=2, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(dim=2, keepdim=True)
    o = torch.bmm(p, v) / total
    return o.to(torch.bfloat16), (top + torch.log(total))[..., 0]


def whole_turn(x, cs, inter):
    """x [rows, heads, d] turned in 64 bits: a product with each row's complex number."""
    R = cs.shape[1]
    z = torch.complex(cs[:, None, : R // 2].double(), cs[:, None, R // 2 :].double())
    y = x.double().clone()
    h = y[..., :R].reshape(*y.shape[:2], -1, 2) if inter else y[..., :R].reshape(*y.shape[:2], 2, -1).transpose(2, 3)
    w = torch.view_as_real(torch.view_as_complex(h.contiguous()) * z)
    y[..., :R] = w.flatten(2) if inter else w.transpose(2, 3).flatten(2)
    return y


def held4(x):
    """What a row x [n, 128] of bf16 numbers stands for in 4 bits, in 64 bits: the nearest scale and the nearest code of
    all that there are."""
    y = 16 * x.double().view(-1, 8, 16)
    every = torch.arange(0xE3, device=x.device, dtype=torch.int16)
    every = (every << 7).view(torch.float16).double()  # ascending; an even place has an even mantissa
    code = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device, dtype=torch.float64)

    def nearest(v, of):
        hi = torch.searchsorted(of, v).clamp(max=len(of) - 1)
        lo = (hi - 1).clamp(min=0)
        up, down = (of[hi] - v).abs(), (v - of[lo]).abs()
        return of[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]

    scale = nearest(y.abs().amax(dim=2) / 6, every)[..., None]
    near = nearest(torch.where(scale > 0, y.abs() / scale, 0.0).contiguous(), code)
    return (y.sign() * near * scale / 16).view(-1, D)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        cs = s.table if s.pos is None else s.table[s.pos.long()]
        if case["inverse"]:
            cs = torch.cat([cs[:, : case["R"] // 2], -cs[:, case["R"] // 2 :]], dim=1)
        return torch.cat([whole_turn(x, c, case["inter"]) for x, c in zip(s.x.split(16384), cs.split(16384))])
    table = s.table.tolist()
    if op != "attn4":
        at, pos, pool = [], [], []
        for b, (a, l) in enumerate(zip(s.q, s.n)):
            for i in range(l - a, l):
                at.append(table[b][i // s.P] * s.P + i % s.P)
                pos.append(i)
            for i in range((l - a) // 4 * 4, l - 3, 4):
                pool.append((table[b][i // s.P] * s.P + i % s.P) // 4)
        at, pos = torch.tensor(at, device="cuda"), torch.tensor(pos, device="cuda")
        new_idx = whole_turn(s.new_idx[:, None], s.turn_idx[pos], case["inter"])[:, 0]
        new_k = whole_turn(s.new_k[:, None], s.turn[pos], case["inter"])[:, 0]
        out = {"k_idx": s.k_idx.double(), "khat": s.khat.double(),
               "q": whole_turn(s.new_q, s.turn[pos], case["inter"]),
               "q_idx": whole_turn(s.new_qi, s.turn_idx[pos], case["inter"])}
        out["k_idx"].view(-1, DI)[at] = new_idx
        if pool:  # the mean of the four keys as the cache holds them
            pool = torch.tensor(pool, device="cuda")
            mean = out["k_idx"].view(-1, 4, DI)[pool].float().to(torch.bfloat16).double().mean(dim=1)
            hi = mean.to(torch.bfloat16).double()
            out["khat"].view(-1, 2 * DI)[pool] = torch.cat([hi, mean - hi], dim=1)
        if op == "append":
            out["k"], out["v"] = s.k.double(), s.v.double()
            out["k"].view(-1, D)[at] = new_k
            out["v"].view(-1, D)[at] = s.new_v.double()
        else:
            out["k"], out["v"] = held4(new_k.float().to(torch.bfloat16)), held4(s.new_v)
        return out
    o = torch.empty(s.T, HQ, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(s.T, HQ, dtype=torch.float64, device="cuda")
    size = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device="cuda", dtype=torch.float64) / 2
    r = 0
    for b, (a, l) in enumerate(zip(s.q, s.n)):
        # this sequence's pools end to end, decoded place by place
        x = s.kv[s.table[b, : -(-l // s.P)].long()].view(-1, POOL)

        def decoded(codes, bits):  # codes [n, 4, 8, 8] bytes, bits [n, 4, 8]
            nib = torch.stack([codes % 16, codes // 16], dim=4).flatten(3).long()
            e, m = (bits // 8).double(), (bits % 8).double()
            scale = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 15), m / 8 * torch.exp2(e - 14))
            return (torch.where(nib < 8, size[nib % 8], -size[nib % 8]) * scale[..., None] / 16).reshape(-1, D)[:l]

        bits = x[:, 512:544].reshape(-1, 4, 2, 2, 2).permute(0, 3, 2, 1, 4)
        k = decoded(x[:, :256].reshape(-1, 4, 8, 8), bits.reshape(-1, 4, 8))
        v = decoded(x[:, 256:512].reshape(-1, 8, 4, 8).transpose(1, 2), x[:, 544:].reshape(-1, 8, 4).transpose(1, 2))
        for i in range(l - a, l):
            keep = torch.zeros((l + 3) // 4, dtype=torch.bool, device="cuda")
            keep[i // 4] = True
            keep.index_fill_(0, torch.where(s.pool_idx[r] < 0, i // 4, s.pool_idx[r]).long(), True)
            at = keep.repeat_interleave(4)[: i + 1].nonzero()[:, 0]
            y = s.qq[r].double() @ k[at].T / math.sqrt(D)
            lse[r] = torch.logsumexp(y, dim=1)
            o[r] = torch.softmax(y, dim=1) @ v[at]
            r += 1
    return o, lse
