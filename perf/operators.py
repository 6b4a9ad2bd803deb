"""Speculative decoding with a tree of drafted tokens over a paged Q8_0 cache: its operators, measured.

Three operators that one verification step runs one after the other:

* ``attention``  epq_attention_tree: the drafted tokens' keys and values are
                 quantized and appended, and every drafted token attends over
                 the sequence's cached positions and the drafted tokens that
                 its mask names;
* ``verify``     epq_verify_tree: the walk through the tree that accepts or
                 rejects drafted tokens against the target's probabilities,
                 with given random numbers, and the next token;
* ``pages``      epq_pages_truncate, epq_pages_fork, epq_pages_reserve and
                 epq_pages_compact: pages freed, shared, copied on write, and
                 the accepted rows moved together.

The cache is a pool of pages, [layers][pages][kv heads][2][page size][row]
bytes; a row of D elements is D/32 fp16 factors, then D int8 codes (element =
factor * code).  ``table`` [sequences][max pages] names a sequence's pages (-1:
none), ``length`` its committed positions, ``refs`` how many sequences hold a
page.
"""
import math

import torch

own = False

VOCAB = 128256  # the dense decode configuration's vocabulary


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token on a short context, dense 8B-class heads: the smallest serving call
        _attn("attn_1tok_ctx37", 32, 8, 128, 64, "37", 1),
        # 8 verify columns over the decode benchmark's 1024-position context
        _attn("attn_8tok_ctx1024", 32, 8, 128, 64, "1024", 8),
        # three branches of unequal length, one still empty, with unequal trees; one key/value head per query head, small pages
        _attn("attn_ragged_16heads", 16, 16, 128, 16, "0,333,4001", 13, "13,5,1"),
        # a wide tree over a long prompt
        _attn("attn_64tok_ctx8193", 32, 8, 128, 64, "8193", 64),
        # four branches over long contexts: the cache is the cost
        _attn("attn_8tok_4x32k", 32, 8, 128, 64, "32768,32001,32768,30000", 8),
        # plain sampling: a tree of the last token alone, dense 8B-class vocabulary
        _ver("verify_1tok", 1, 1, VOCAB, 1.0, False, ""),
        # 8 verify columns against the draft's probabilities
        _ver("verify_8tok", 1, 8, VOCAB, 0.8, True, ""),
        # greedy decoding, unequal trees, an odd vocabulary
        _ver("verify_greedy_3seq", 3, 13, 50001, 0.0, False, "13,1,7"),
        # four branches with wide trees
        _ver("verify_64tok_4seq", 4, 64, VOCAB, 1.0, True, ""),
        # one sequence's accepted rows moved together after a step, dense 8B-class cache
        _pages("pages_commit_1seq", 32, 8, 128, 64, 1037, 1, 8, 24),
        # one prompt forked into 8 branches, its last page copied on write
        _pages("pages_fork_8seq", 32, 8, 128, 64, 1037, 8, 8, 40),
        # the MoE decode model's cache (40 layers, 16 heads), 24 branches, large pages
        _pages("pages_fork_24seq_moe", 40, 16, 128, 128, 2047, 24, 16, 64),
    ]


def _attn(name, heads, kv, dim, page, lengths, ntok, ragged=""):
    return {"name": name, "kind": "attention", "heads": heads, "kv": kv, "dim": dim, "page": page, "lengths": lengths, "ntok": ntok, "ragged": ragged}


def _ver(name, nseq, ntok, vocab, temperature, draft, ragged):
    return {"name": name, "kind": "verify", "nseq": nseq, "ntok": ntok, "vocab": vocab, "temperature": temperature, "draft": draft, "ragged": ragged}


def _pages(name, layers, kv, dim, page, length, nseq, ntok, npages):
    return {"name": name, "kind": "pages", "layers": layers, "kv": kv, "dim": dim, "page": page, "length": length, "nseq": nseq, "ntok": ntok, "npages": npages}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "verify", "pages"])
    if kind == "attention":
        kv = rng.choice([1, 2, 4, 8, 16])
        group = rng.choice([1, 2, 3, 4, 8]) if kv < 16 else 1
        dim, page = rng.choice([128, 128, 256]), rng.choice([16, 32, 64, 128])
        nseq, ntok = rng.choice([1, 1, 2, 3, 5]), min(64, _log(rng, 1, 70))
        # at most the largest listed case's positions, and its products where the tree is wide
        most = min(32768, 131072 * 8 * 128 // (nseq * kv * dim), 131072 * 32 * 8 * 128 // (nseq * kv * group * ntok * dim))
        lengths = [_log(rng, 1, most) - (rng.random() < 0.1) for _ in range(nseq)]
        ragged = ",".join(str(rng.randint(1, ntok)) for _ in range(nseq)) if rng.random() < 0.4 else ""
        case = _attn("", kv * group, kv, dim, page, ",".join(map(str, lengths)), ntok, ragged)
    elif kind == "verify":
        vocab, nseq = _log(rng, 1000, 200000), rng.choice([1, 1, 2, 4])
        ntok = _log(rng, 1, max(1, min(64, 4 * 64 * VOCAB // (nseq * vocab))))
        draft = rng.random() < 0.6
        ragged = ",".join(str(rng.randint(1, ntok)) for _ in range(nseq)) if rng.random() < 0.4 else ""
        case = _ver("", nseq, ntok, vocab, rng.choice([0.0, 0.6, 1.0, 1.3]), draft, ragged)
    else:
        kv, dim, page = rng.choice([1, 2, 4, 8, 16]), rng.choice([128, 128, 256]), rng.choice([16, 32, 64, 128])
        layers, nseq, ntok = rng.choice([1, 4, 16, 32]), _log(rng, 1, 24), min(64, _log(rng, 1, 70))
        length = _log(rng, 1, 4000)
        # a fork needs its copied page and the pages of its drafted tokens
        npages = -(-length // page) + nseq * (2 + ntok // page) + rng.randint(0, 20)
        case = _pages("", layers, kv, dim, page, length, nseq, ntok, npages)
    del case["name"]
    return case


def _ints(text):
    return [int(v) for v in text.split(",")]


def _ragged(case, nseq):
    return _ints(case["ragged"]) if case["ragged"] else [case["ntok"]] * nseq


# ---------------------------------------------------------------- inputs
def _parents(gen, nseq, ntok):
    """Random trees: a node's parent is one of the few nodes before it."""
    i = torch.arange(ntok, device="cuda").expand(nseq, ntok)
    back = 1 + (torch.rand((nseq, ntok), generator=gen, device="cuda") ** 2 * 4).long()
    return torch.where(i == 0, -1, (i - back).clamp(min=0)).int()


def _ancestors(parent):
    """int64 [nseq][ntok]: bit j of entry i says that token j is i or one of its ancestors."""
    nseq, ntok = parent.shape
    p = parent.tolist()
    mask = [[0] * ntok for _ in range(nseq)]
    for s in range(nseq):
        for i in range(ntok):
            m = (mask[s][p[s][i]] if p[s][i] >= 0 else 0) | 1 << i
            mask[s][i] = m
    wrap = lambda m: m - (1 << 64) if m >= 1 << 63 else m  # noqa: E731
    return torch.tensor([[wrap(m) for m in r] for r in mask], dtype=torch.int64, device="cuda")


def _fill(gen, pool):
    """Rows of N(0,1) values in Q8_0, written page block by page block."""
    flat, row = pool.view(-1, pool.shape[-1]), pool.shape[-1]
    dim = row * 16 // 17
    for a in range(0, flat.shape[0], 1 << 20):
        part = flat[a:a + (1 << 20)]
        x = torch.randn((part.shape[0], dim // 32, 32), generator=gen, device="cuda")
        d = (x.abs().amax(2, keepdim=True) / 127).half()
        part[:, : dim // 16] = d[..., 0].contiguous().view(torch.uint8)
        part[:, dim // 16:] = (x / d.float()).round().clamp(-127, 127).to(torch.int8).view(torch.uint8).view(part.shape[0], dim)


def _views(pool):
    dim = pool.shape[-1] * 16 // 17
    return pool[..., dim // 16:].view(torch.int8), pool[..., : dim // 16].view(torch.float16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    kind, ntok = case["kind"], case["ntok"]
    st = {"kind": kind, "ntok": ntok}
    if kind == "attention":
        lengths, dim, page, kv = _ints(case["lengths"]), case["dim"], case["page"], case["kv"]
        nseq = len(lengths)
        each = [-(-(n + ntok) // page) for n in lengths]
        npages, most = sum(each) + 3, max(each)
        pool = torch.empty((1, npages, kv, 2, page, dim + dim // 16), dtype=torch.uint8, device="cuda")
        _fill(gen, pool)
        order = torch.randperm(npages, generator=gen, device="cuda").int()
        table = torch.full((nseq, most), -1, dtype=torch.int32, device="cuda")
        at = 0
        for s, n in enumerate(each):
            table[s, :n] = order[at:at + n]
            at += n
        refs = torch.zeros(npages, dtype=torch.int32, device="cuda")
        refs[order[:at].long()] = 1
        width = (case["heads"] + 2 * kv) * dim
        st["qkv"] = torch.randn((nseq, ntok, width), generator=gen, device="cuda")
        st["qkv"][..., : case["heads"] * dim] *= 2.0
        st.update(pool=pool, table=table, refs=refs, length=torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                  mask=_ancestors(_parents(gen, nseq, ntok)), heads=case["heads"], kv=kv, dim=dim, page=page, most=max(lengths) + ntok,
                  n_tok=torch.tensor(_ragged(case, nseq), dtype=torch.int32, device="cuda"), views=_views(pool), scale=1 / math.sqrt(dim))
    elif kind == "verify":
        nseq, vocab = case["nseq"], case["vocab"]
        st.update(parent=_parents(gen, nseq, ntok), vocab=vocab, temperature=case["temperature"], draft=None,
                  n_tok=torch.tensor(_ragged(case, nseq), dtype=torch.int32, device="cuda"),
                  u=torch.rand((nseq, ntok), generator=gen, device="cuda"))
        logits = torch.randn((nseq, ntok, vocab), generator=gen, device="cuda") * 3.0
        drafted = logits + torch.randn(logits.shape, generator=gen, device="cuda") * 0.5
        # a node's token is drawn from what the draft model said at its parent
        p = torch.softmax(drafted / (case["temperature"] or 1.0), 2)
        up = st["parent"].long().clamp(min=0)
        noise = torch.rand((nseq, ntok, vocab), generator=gen, device="cuda").clamp_(min=1e-30).log_().neg_()
        st["tokens"] = (p.gather(1, up[..., None].expand(-1, -1, vocab)) / noise).argmax(2).int()
        del noise
        st["logits"] = logits
        if case["draft"]:
            st["draft"] = p
    else:
        nseq, dim, page, kv, length = case["nseq"], case["dim"], case["page"], case["kv"], case["length"]
        pool = torch.empty((case["layers"], case["npages"], kv, 2, page, dim + dim // 16), dtype=torch.uint8, device="cuda")
        _fill(gen, pool)
        have, most = -(-length // page), -(-(length + 4 * ntok) // page)
        table = torch.full((nseq, most), -1, dtype=torch.int32, device="cuda")
        held = torch.randperm(case["npages"], generator=gen, device="cuda")[:have]
        table[0, :have] = held.int()
        refs = torch.zeros(case["npages"], dtype=torch.int32, device="cuda")
        refs[held] = 1
        lengths = torch.zeros(nseq, dtype=torch.int32, device="cuda")
        lengths[0] = length
        # an accepted path: the root, then nodes of rising index
        keep = 1 + (torch.rand((nseq,), generator=gen, device="cuda") * ntok).long()
        pick = torch.rand((nseq, ntok), generator=gen, device="cuda")
        pick[:, 0] = -1.0
        chosen = pick.argsort(1).argsort(1) < keep[:, None]
        index = torch.arange(ntok, device="cuda")
        path = torch.where(chosen, index, ntok).sort(1).values
        st.update(pool=pool, table=table, refs=refs, length=lengths, kv=kv, dim=dim, page=page, n_keep=keep.int(),
                  path=torch.where(path < ntok, path, -1).int(), extra=torch.full((nseq,), ntok, dtype=torch.int32, device="cuda"),
                  back=lengths.clone(), src=torch.zeros(nseq - 1, dtype=torch.int32, device="cuda"),
                  dst=torch.arange(1, nseq, dtype=torch.int32, device="cuda"), views=_views(pool))
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    return {"attention": _run_attention, "verify": _run_verify, "pages": _run_pages}[state["kind"]](state)


def _cache(epq, st):
    """The handle and the workspace that a user's program makes once and keeps."""
    if "cache" not in st:
        st["cache"] = epq.PagedKVCache.over(st["pool"], st["table"], st["length"], st["refs"])
    return st["cache"]


def _run_attention(st):
    nq, nkv = st["heads"] * st["dim"], st["kv"] * st["dim"]
    q, k, v = st["qkv"][..., :nq], st["qkv"][..., nq:nq + nkv], st["qkv"][..., nq + nkv:]
    if own:
        import moe_experts_gb300 as epq
        cache = _cache(epq, st)
        if "ws" not in st:
            st["ws"] = epq.epq_attention_tree_workspace(cache, st["heads"], st["ntok"])
        out = epq.epq_attention_tree(q, k, v, cache, 0, st["heads"], st["scale"], mask=st["mask"], n_tok=st["n_tok"], workspace=st["ws"])
    else:
        out = _plain_attention(st, q, k, v)
    return [out, *st["views"]]


def _run_verify(st):
    if own:
        import moe_experts_gb300 as epq
        if "ws" not in st:
            st["ws"] = epq.epq_verify_tree_workspace(st["logits"])
        return epq.epq_verify_tree(st["logits"], st["tokens"], st["parent"], st["u"], draft=st["draft"], n_tok=st["n_tok"],
                                   temperature=st["temperature"], workspace=st["ws"])
    return _plain_verify(st)


def _run_pages(st):
    # the last pass's branches are freed first, so that a pass can be run again
    if own:
        import moe_experts_gb300 as epq
        cache = _cache(epq, st)
        epq.epq_pages_truncate(cache, st["back"])
        epq.epq_pages_fork(cache, st["src"], st["dst"])
        status = epq.epq_pages_reserve(cache, st["extra"])
        epq.epq_pages_compact(cache, st["path"], st["n_keep"])
    else:
        _plain_truncate(st)
        _plain_fork(st)
        status = _plain_reserve(st)
        _plain_compact(st)
    return [st["table"], st["length"], st["refs"], status, *st["views"]]


# ---------------------------------------------------------------- plain forms
def _plain_rows(x, dim):
    """float32 [..., dim] -> the cache rows [..., dim + dim/16] in bytes."""
    b = (x + 0.0).reshape(*x.shape[:-1], dim // 32, 32)
    n = torch.full((), 127.0, device=x.device)
    d = (b.abs().amax(-1, keepdim=True) / n).half()
    f = d.float()
    c = torch.where(f == 0, torch.zeros_like(b), (b / torch.where(f == 0, torch.ones_like(f), f)).round().clamp(-127, 127)).to(torch.int8)
    return torch.cat([d[..., 0].contiguous().view(torch.uint8), c.view(torch.uint8).reshape(*x.shape[:-1], dim)], -1)


def _plain_attention(st, q, k, v):
    pool, table, length, dim, page, kv, ntok = st["pool"][0], st["table"].long(), st["length"].long(), st["dim"], st["page"], st["kv"], st["ntok"]
    nseq, group = table.shape[0], st["heads"] // kv
    # the new rows, at positions length ... of their sequence
    i = torch.arange(ntok, device=pool.device)
    live = i < st["n_tok"][:, None]
    pos = length[:, None] + i
    pg, slot = table.gather(1, pos // page), pos % page
    rows = _plain_rows(torch.stack([k, v], 2).reshape(nseq, ntok, 2, kv, dim), dim).transpose(2, 3)
    pool[pg, :, :, slot] = torch.where(live[:, :, None, None, None], rows, pool[pg, :, :, slot])
    # every sequence's rows, padded to the longest
    n = -(-st["most"] // page)
    t = torch.arange(n * page, device=pool.device)
    held = pool[table[:, :n].clamp(min=0)].permute(0, 2, 3, 1, 4, 5).reshape(nseq, kv, 2, n * page, dim + dim // 16)
    f = held[..., : dim // 16].contiguous().view(torch.float16).float()
    x = held[..., dim // 16:].contiguous().view(torch.int8).float().view(nseq, kv, 2, n * page, dim // 32, 32)
    x = (x * f[..., None]).view(nseq, kv, 2, n * page, dim)
    # scores, masked, and their softmax
    s = torch.matmul(q.reshape(nseq, ntok, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(nseq, kv, group * ntok, dim), x[:, :, 0].transpose(2, 3)) * st["scale"]
    j = t - length[:, None]
    bit = (st["mask"][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    drafted = (j >= 0) & (j < st["n_tok"][:, None])
    may = ((j < 0)[:, None, :] | (drafted[:, None, :] & (bit == 1))) & live[:, :, None]
    s = s.view(nseq, kv, group, ntok, -1).masked_fill(~may[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(nseq, kv, group * ntok, -1), x[:, :, 1]).view(nseq, kv, group, ntok, dim) / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 3, 1, 2, 4).reshape(nseq, ntok, st["heads"] * dim)


def _plain_verify(st):
    """In 64 bits: an acceptance and a drawn token are comparisons of long sums."""
    logits, tokens, parent, u, draft = st["logits"], st["tokens"].long(), st["parent"].long(), st["u"].double(), st["draft"]
    nseq, ntok, vocab = logits.shape
    live = torch.arange(ntok, device=logits.device) < st["n_tok"][:, None]
    greedy = st["temperature"] == 0
    every = torch.arange(nseq, device=logits.device)
    x = logits.double() / (1.0 if greedy else st["temperature"])
    top = x.amax(2, keepdim=True)
    lse = (top[..., 0] + torch.exp(x - top).sum(2).log()).masked_fill(~live, 0.0).float()
    node = torch.zeros(nseq, dtype=torch.int64, device=logits.device)
    path = torch.full((nseq, ntok + 1), -1, dtype=torch.int64, device=logits.device)
    path[:, 0] = torch.where(live[:, 0], 0, -1)
    count = live[:, 0].long()

    def weights(at):
        row = x[every, at]
        best = logits[every, at].argmax(1)
        first = (logits[every, at] == logits[every, at].amax(1, keepdim=True)).int().argmax(1)
        if greedy:
            return torch.nn.functional.one_hot(first, vocab).double()
        return torch.exp(row - row.gather(1, best[:, None]))

    r = weights(node)
    for i in range(1, ntok):
        tok = tokens[:, i].clamp(0, vocab - 1)
        total = r.sum(1)
        here = r[every, tok]
        test = live[:, i] & (parent[:, i] == node)
        qx = draft[every, node, tok].double() if draft is not None and not greedy else torch.ones_like(total)
        if greedy:
            yes = test & (here > 0)
        else:
            yes = test & (u[:, i] * qx * total < here)
        no = test & ~yes
        if not greedy:
            if draft is not None:
                less = (r - total[:, None] * draft[every, node].double()).clamp(min=0)
                less = torch.where(less.sum(1, keepdim=True) > 0, less, r)
            else:
                less = r.scatter(1, tok[:, None], 0.0)
            r = torch.where(no[:, None], less, r)
        node = torch.where(yes, i, node)
        path[every, torch.where(yes, count, ntok)] = i
        count = count + yes.long()
        r = torch.where(yes[:, None], weights(node), r)
    upto = r.cumsum(1)
    # the total is the last running sum, so that a u just below 1 still names a token
    # (where nothing is left: the row's largest logit)
    drawn = (upto > u[:, :1] * upto[:, -1:]).int().argmax(1)
    last = logits[every, node]
    drawn = torch.where(upto[:, -1] > 0, drawn, (last == last.amax(1, keepdim=True)).int().argmax(1))
    path[:, ntok] = -1
    return [path[:, :ntok].int(), count.int(), torch.where(live[:, 0], drawn, -1).int(), lse]


def _plain_truncate(st):
    table, page = st["table"], st["page"]
    new = torch.where(st["back"] < 0, st["length"], torch.minimum(st["back"], st["length"]))
    j = torch.arange(table.shape[1], device=table.device)
    gone = (j >= (new[:, None] + page - 1) // page) & (table >= 0) & (st["back"][:, None] >= 0)
    st["refs"].index_add_(0, table.clamp(min=0).view(-1).long(), -gone.int().view(-1))
    table.copy_(torch.where(gone, -1, table))
    st["length"].copy_(new)


def _plain_fork(st):
    table, length, page = st["table"], st["length"], st["page"]
    src, dst = st["src"].long(), st["dst"].long()
    if not src.numel():
        return
    j = torch.arange(table.shape[1], device=table.device)
    used = j < (length[src][:, None] + page - 1) // page
    table[dst] = torch.where(used, table[src], -1)
    length[dst] = length[src]
    st["refs"].index_add_(0, table[dst].clamp(min=0).view(-1).long(), used.int().view(-1))


def _plain_reserve(st):
    pool, table, length, refs, page, extra = st["pool"], st["table"], st["length"].long(), st["refs"], st["page"], st["extra"].long()
    nseq, most = table.shape
    j = torch.arange(most, device=table.device)
    first, last = length // page, (length + extra + page - 1) // page
    fits = last <= most
    active = (extra > 0) & fits
    at = first.clamp(max=most - 1)
    mine = table.gather(1, at[:, None])[:, 0].long()
    partly = active & (length % page > 0) & (mine >= 0)
    # the holders of a shared page copy it one after the other; the last one left keeps it
    before = torch.ones((nseq, nseq), dtype=torch.bool, device=table.device).tril(-1)
    rank = (before & (mine[:, None] == mine[None, :]) & partly[None, :]).sum(1)
    copies = partly & (refs[mine.clamp(min=0)] - rank > 1)
    need = active[:, None] & (j >= first[:, None]) & (j < last[:, None]) & ((table < 0) | (copies[:, None] & (j == first[:, None])))
    free = refs == 0
    order = free.long().cumsum(0) - 1
    ids = torch.zeros(refs.shape[0] + 1, dtype=torch.int64, device=table.device)
    ids.scatter_(0, torch.where(free, order, refs.shape[0]), torch.arange(refs.shape[0], device=table.device))
    ids[refs.shape[0]] = 0
    ok = need.sum(1).cumsum(0) <= free.sum()
    take = need & ok[:, None]
    nth = (need.view(-1).long().cumsum(0) - 1).view(nseq, most)
    new = ids[nth.clamp(0, refs.shape[0])]
    copies = copies & ok
    refs.index_add_(0, mine.clamp(min=0), -copies.int())
    refs.index_add_(0, torch.where(take, new, 0).view(-1), take.int().view(-1))
    table.copy_(torch.where(take, new.int(), table))
    to = torch.where(copies, table.gather(1, at[:, None])[:, 0].long(), mine.clamp(min=0))
    row = torch.arange(page, device=table.device)
    moved = (copies[:, None] & (row < (length % page)[:, None]))[None, :, None, None, :, None]
    pool[:, to] = torch.where(moved, pool[:, mine.clamp(min=0)], pool[:, to])
    return torch.where(extra <= 0, 0, torch.where(~fits, 2, torch.where(ok, 0, 1))).int()


def _plain_compact(st):
    pool, table, length, page, ntok = st["pool"], st["table"].long(), st["length"].long(), st["page"], st["ntok"]
    i = torch.arange(ntok, device=table.device)
    to = length[:, None] + i
    moved = (i < st["n_keep"][:, None]) & (st["path"] >= 0)
    come = length[:, None] + torch.where(moved, st["path"].long(), i)
    pool[:, table.gather(1, to // page), :, :, to % page] = pool[:, table.gather(1, come // page), :, :, come % page]
    st["length"].copy_((length + st["n_keep"]).int())


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    ntok = case["ntok"]
    if case["kind"] == "attention":
        lengths = _ints(case["lengths"])
        n_tok, dim, kv, heads = _ragged(case, len(lengths)), case["dim"], case["kv"], case["heads"]
        row = dim + dim // 16
        old = sum(lengths) * kv * 2 * row
        new = sum(n_tok) * (kv * 2 * (row + 4 * dim) + heads * dim * 4) + len(lengths) * ntok * heads * dim * 4
        seen = sum(t * (n + (t + 1) / 2) for n, t in zip(lengths, n_tok))
        return {"bytes": old + new, "flops": 4 * heads * dim * seen}
    if case["kind"] == "verify":
        rows = sum(_ragged(case, case["nseq"]))
        # the logits once; of the draft's rows, one of each sequence, where the walk ends
        many = rows + (case["nseq"] if case["draft"] and case["temperature"] else 0)
        return {"bytes": 4 * many * case["vocab"] + 16 * case["nseq"] * ntok, "flops": 4 * many * case["vocab"]}
    row = case["dim"] + case["dim"] // 16
    each = case["layers"] * case["kv"] * 2 * row
    live = case["length"] % case["page"]
    copies = case["nseq"] - 1 if live else 0
    moved = case["nseq"] * (ntok + 1) // 2
    return {"bytes": each * ((live if copies else 0) + copies * live + 2 * moved) + 8 * case["nseq"] * -(-case["length"] // case["page"]), "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "attention":
        return [_exact_attention(st), None, None]
    if case["kind"] == "verify":
        rows = [torch.logsumexp(st["logits"][s].double() / (st["temperature"] or 1.0), 1) for s in range(case["nseq"])]
        return [None, None, None, torch.stack([torch.where(torch.arange(case["ntok"], device="cuda") < st["n_tok"][s], r, 0.0) for s, r in enumerate(rows)])]
    return None  # whole numbers and copied bytes


def _exact_values(rows, dim):
    f = rows[:, : dim // 16].contiguous().view(torch.float16).double().repeat_interleave(32, 1)
    return f * rows[:, dim // 16:].contiguous().view(torch.int8).double()


def _exact_attention(st):
    dim, page, heads, kv, ntok = st["dim"], st["page"], st["heads"], st["kv"], st["ntok"]
    nseq = st["table"].shape[0]
    out = torch.zeros((nseq, ntok, heads, dim), dtype=torch.float64, device="cuda")
    x = st["qkv"].view(nseq, ntok, heads + 2 * kv, dim)
    masks = st["mask"].tolist()
    for s in range(nseq):
        length, n = int(st["length"][s]), int(st["n_tok"][s])
        pages = st["table"][s, : -(-length // page)].long()
        see = torch.tensor([[(masks[s][i] >> j) & 1 == 1 for j in range(n)] for i in range(n)], device="cuda").view(n, n)
        see = torch.cat([torch.ones((n, length), dtype=torch.bool, device="cuda"), see], 1)
        for h in range(kv):
            old = [st["pool"][0, pages, h, c].reshape(-1, dim + dim // 16)[:length] for c in (0, 1)]
            new = [_plain_rows(x[s, :n, heads + c * kv + h], dim) for c in (0, 1)]
            K, V = (_exact_values(torch.cat([old[c], new[c]]), dim) for c in (0, 1))
            for g in range(h * (heads // kv), (h + 1) * (heads // kv)):
                w = (x[s, :n, g].double() @ K.T) * st["scale"]
                w = torch.softmax(w.masked_fill(~see, -math.inf), 1).nan_to_num(0.0)
                out[s, :n, g] = w @ V
    return out.view(nseq, ntok, heads * dim)
