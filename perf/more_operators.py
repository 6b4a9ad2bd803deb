"""A sequence from its prompt to its constrained tokens over a paged Q8_0 cache: its operators, measured.

* ``rope``    epq_rope: query and key heads rotated by their tokens' positions;
* ``append``  epq_pages_append: any number of keys and values quantized into the
              pages behind a sequence's committed positions, the keys rotated
              on the way;
* ``prompt``  epq_attention_prompt: causal attention of any number of appended
              rows over the cached ones and themselves;
* ``logits``  epq_logits_adjust: biases, penalties for repeated tokens and
              grammar masks on the logits of drafted tokens, each with the
              tokens before it in its tree.

The cache is a pool of pages, [layers][pages][kv heads][2][page size][row]
bytes; a row of D elements is D/32 fp16 factors, then D int8 codes (element =
factor * code).  ``table`` [sequences][max pages] names a sequence's pages (-1:
none), ``length`` its committed positions, ``refs`` how many sequences hold a
page.  The rotation's table is float32 [positions][rotated / 2][2]: cosine and
sine of an angle, times a magnitude.
"""
import math

import torch

own = False

VOCAB = 128256  # the dense decode configuration's vocabulary


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the heads of one verification step's 8 drafted tokens (32 query and 8 key heads of one buffer): latency
        _rope("rope_8tok_tree", 40, 128, 128, 0, False, "1037", 8, tree=True, scaling="none"),
        # a long prompt's heads, a part of each rotated, neighbours paired, angles stretched for a longer context
        _rope("rope_4096tok_part", 40, 128, 64, 64, True, "28672", 4096, scaling="parts"),
        # a step's 8 drafted rows, at their depths in the tree: latency
        _append("append_8tok_tree", 8, 128, 64, 128, 0, False, "1037", 8, tree=True),
        # prompts of unequal length behind an empty, a short and a long context; small pages, part of the head rotated
        _append("append_ragged_16heads", 16, 128, 16, 64, 0, True, "0,333,4001", 517, "517,64,1"),
        # a whole prompt at once
        _append("append_8192tok", 8, 128, 64, 128, 0, False, "0", 8192),
        # the first prompt length past a tree's 64 tokens: latency
        _prompt("prompt_65tok", 32, 8, 128, 64, "0", 65),
        # unequal prompts, one of a single token, a window of positions, one key/value head per query head, small pages
        _prompt("prompt_ragged_window", 16, 16, 128, 16, "0,333,4001", 517, "517,129,1", window=1024),
        # a whole prompt
        _prompt("prompt_4096tok", 32, 8, 128, 64, "0", 4096),
        # a chunk of a prompt behind a long context
        _prompt("prompt_2048tok_ctx32k", 32, 8, 128, 64, "32768", 2048),
        # plain sampling with penalties over a short history: latency
        _logits("logits_1tok", 1, 1, VOCAB, 100, 8, False, ""),
        # unequal trees, an odd vocabulary, a grammar
        _logits("logits_13tok_3seq", 3, 13, 50001, 1037, 20, True, "13,1,7"),
        # four branches with wide trees, long histories, a grammar
        _logits("logits_64tok_4seq", 4, 64, VOCAB, 8193, 64, True, ""),
    ]


def _rope(name, heads, dim, rot, first, interleaved, lengths, ntok, ragged="", tree=False, scaling="none"):
    return {"name": name, "kind": "rope", "heads": heads, "dim": dim, "rot": rot, "first": first, "interleaved": interleaved,
            "lengths": lengths, "ntok": ntok, "ragged": ragged, "tree": tree, "scaling": scaling}


def _append(name, kv, dim, page, rot, first, interleaved, lengths, ntok, ragged="", tree=False):
    return {"name": name, "kind": "append", "kv": kv, "dim": dim, "page": page, "rot": rot, "first": first, "interleaved": interleaved,
            "lengths": lengths, "ntok": ntok, "ragged": ragged, "tree": tree, "scaling": "none"}


def _prompt(name, heads, kv, dim, page, lengths, ntok, ragged="", window=0):
    return {"name": name, "kind": "prompt", "heads": heads, "kv": kv, "dim": dim, "page": page, "lengths": lengths, "ntok": ntok,
            "ragged": ragged, "window": window}


def _logits(name, nseq, ntok, vocab, history, nbias, grammar, ragged):
    return {"name": name, "kind": "logits", "nseq": nseq, "ntok": ntok, "vocab": vocab, "history": history, "nbias": nbias,
            "grammar": grammar, "ragged": ragged}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _some(rng, nseq, ntok):
    return ",".join(str(rng.randint(1, ntok)) for _ in range(nseq)) if rng.random() < 0.4 else ""


def draw(rng):
    kind = rng.choice(["rope", "append", "prompt", "logits"])
    nseq = rng.choice([1, 1, 2, 3, 5])
    if kind in ("rope", "append"):
        dim = rng.choice([128, 128, 256]) if kind == "append" else rng.choice([64, 80, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8, 16]) if kind == "append" else rng.choice([1, 5, 10, 20, 40])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        first, inter = rng.choice([0, 0, dim - rot]), rng.random() < 0.4
        most = min(8192, (8192 * 8 * 128 if kind == "append" else 4096 * 40 * 128) // (nseq * kv * dim))
        ntok = _log(rng, 1, most)
        tree = ntok <= 64 and rng.random() < 0.6
        lengths = ",".join(str(_log(rng, 1, 32768 if kind == "rope" else 8192) - (rng.random() < 0.1)) for _ in range(nseq))
        ragged = _some(rng, nseq, ntok)
        if kind == "rope":
            case = _rope("", kv, dim, rot, first, inter, lengths, ntok, ragged, tree, rng.choice(["none", "linear", "parts", "bands"]))
        else:
            case = _append("", kv, dim, rng.choice([16, 32, 64, 128]), rot, first, inter, lengths, ntok, ragged, tree)
    elif kind == "prompt":
        kv = rng.choice([1, 2, 4, 8, 16])
        group = rng.choice([1, 2, 3, 4, 8]) if kv < 16 else 1
        dim = rng.choice([128, 128, 256])
        ntok = _log(rng, 1, 4096)
        # at most the largest listed case's products and cached rows
        room = 2048 * 32768 * 32 * 128 // (nseq * kv * group * dim * ntok)
        ntok = min(ntok, 2 * room + 1, 4096)
        most = max(1, min(32768, room - ntok, 32768 * 8 * 128 // (nseq * kv * dim)))
        lengths = ",".join(str(_log(rng, 1, most) - (rng.random() < 0.2)) for _ in range(nseq))
        case = _prompt("", kv * group, kv, dim, rng.choice([16, 32, 64, 128]), lengths, ntok, _some(rng, nseq, ntok),
                       rng.choice([0, 0, 0, _log(rng, 1, 8192)]))
    else:
        vocab = _log(rng, 1000, 200000)
        nseq = rng.choice([1, 1, 2, 4])
        ntok = _log(rng, 1, max(1, min(64, 4 * 64 * VOCAB // (nseq * vocab))))
        case = _logits("", nseq, ntok, vocab, _log(rng, 1, 9000) - 1, rng.choice([0, 1, 8, 33, 300]), rng.random() < 0.6, _some(rng, nseq, ntok))
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
            mask[s][i] = (mask[s][p[s][i]] if p[s][i] >= 0 else 0) | 1 << i
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


def _frequencies(rot, scaling):
    """float64 [rot / 2] angles per position, and what cosine and sine are multiplied by."""
    base, factor, before = 500000.0, 8.0, 8192
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if scaling == "linear":  # all angles smaller
        return f / factor, 1.0
    if scaling == "parts":  # slow pairs stretched, fast ones kept, a ramp in the pair's index between them
        at = lambda turns: rot * math.log(before / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64, device="cuda") - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "bands":  # the same by wavelength, a ramp in the turns that the pair makes over the first context
        smooth = ((before * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - smooth) * f / factor + smooth * f, 1.0
    return f, 1.0


def _angles(st, case, gen, nseq):
    """The table of the positions that the sequences reach, and what the tokens' positions come from."""
    lengths, ntok = _ints(case["lengths"]), case["ntok"]
    f, magnitude = _frequencies(case["rot"], case["scaling"])
    a = torch.arange(max(lengths) + ntok, dtype=torch.float64, device="cuda")[:, None] * f
    st["table"] = (torch.stack([a.cos(), a.sin()], 2) * magnitude).float()
    st["exact_table"] = (f, magnitude)
    st["mask"] = _ancestors(_parents(gen, nseq, ntok)) if case["tree"] else None
    st.update(rot=case["rot"], first=case["first"], interleaved=case["interleaved"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    kind, ntok = case["kind"], case["ntok"]
    st = {"kind": kind, "ntok": ntok}
    i32 = dict(dtype=torch.int32, device="cuda")
    if kind == "logits":
        nseq, vocab, history, nbias = case["nseq"], case["vocab"], case["history"], case["nbias"]
        st["logits"] = torch.randn((nseq, ntok, vocab), generator=gen, device="cuda") * 3.0
        # text repeats itself: tokens by falling frequency
        often = lambda *n: (torch.rand(n, generator=gen, device="cuda") ** 4 * vocab).int().clamp(max=vocab - 1)  # noqa: E731
        st["tokens"] = often(nseq, ntok)
        st["history"] = often(nseq, history) if history else None
        st["history_len"] = torch.tensor([max(0, history - 17 * s) for s in range(nseq)], **i32)
        st["prompt_len"] = st["history_len"] // 3
        st["mask"] = _ancestors(_parents(gen, nseq, ntok))
        st["n_tok"] = torch.tensor(_ragged(case, nseq), **i32)
        pen = torch.rand((nseq, 3), generator=gen, device="cuda")
        st["penalties"] = pen * torch.tensor([0.3, 0.5, 0.5], device="cuda") + torch.tensor([1.0, 0.0, 0.0], device="cuda")
        st["bias_ids"] = st["bias"] = st["allowed"] = None
        if nbias:
            st["bias_ids"] = torch.stack([torch.randperm(vocab, generator=gen, device="cuda")[:nbias] for _ in range(nseq)]).int()
            st["bias"] = torch.randn((nseq, nbias), generator=gen, device="cuda") * 4.0
        if case["grammar"]:  # runs of 32 tokens all out, all in, or some in
            n = -(-vocab // 32)
            word = torch.randint(-(1 << 31), 1 << 31, (nseq, ntok, n), generator=gen, device="cuda").int()
            how = torch.rand((nseq, ntok, n), generator=gen, device="cuda")
            st["allowed"] = torch.where(how < 0.5, 0, torch.where(how < 0.7, -1, word)).int()
        return st
    lengths, dim = _ints(case["lengths"]), case["dim"]
    nseq = len(lengths)
    st.update(dim=dim, length=torch.tensor(lengths, **i32), n_tok=torch.tensor(_ragged(case, nseq), **i32))
    if kind == "rope":
        st["heads"] = case["heads"]
        _angles(st, case, gen, nseq)
        st["x"] = torch.randn((nseq, ntok, case["heads"] * dim), generator=gen, device="cuda")
        return st
    page, kv = case["page"], case["kv"]
    each = [-(-(n + ntok) // page) for n in lengths]
    npages, most = sum(each) + 3, max(each)
    pool = torch.empty((1, npages, kv, 2, page, dim + dim // 16), dtype=torch.uint8, device="cuda")
    _fill(gen, pool)
    order = torch.randperm(npages, generator=gen, device="cuda").int()
    pages = torch.full((nseq, most), -1, **i32)
    at = 0
    for s, n in enumerate(each):
        pages[s, :n] = order[at:at + n]
        at += n
    refs = torch.zeros(npages, **i32)
    refs[order[:at].long()] = 1
    st.update(pool=pool, pages=pages, refs=refs, kv=kv, page=page, most=max(lengths) + ntok, views=_views(pool))
    if kind == "append":
        _angles(st, case, gen, nseq)
        st["kv_new"] = torch.randn((nseq, ntok, 2 * kv * dim), generator=gen, device="cuda")
    else:
        st.update(heads=case["heads"], window=case["window"], scale=1 / math.sqrt(dim))
        st["q"] = torch.randn((nseq, ntok, case["heads"] * dim), generator=gen, device="cuda") * 2.0
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    return {"rope": _run_rope, "append": _run_append, "prompt": _run_prompt, "logits": _run_logits}[state["kind"]](state)


def _plan(epq, st):
    """The handles that a user's program makes once and keeps."""
    if "plan" not in st:
        st["plan"] = {}
        if "pool" in st:
            st["plan"]["cache"] = epq.PagedKVCache.over(st["pool"], st["pages"], st["length"], st["refs"])
        if "table" in st:
            st["plan"]["rope"] = epq.RopeTable.over(st["table"], first=st["first"], interleaved=st["interleaved"])
        if st["kind"] == "prompt":
            st["plan"]["ws"] = epq.epq_attention_prompt_workspace(st["plan"]["cache"], st["heads"], st["ntok"])
    return st["plan"]


def _run_rope(st):
    if own:
        import moe_experts_gb300 as epq
        return epq.epq_rope(st["x"], _plan(epq, st)["rope"], st["heads"], start=st["length"], mask=st["mask"], n_tok=st["n_tok"])
    x = st["x"].view(*st["x"].shape[:2], st["heads"], st["dim"])
    live = torch.arange(st["ntok"], device=x.device) < st["n_tok"][:, None]
    return torch.where(live[:, :, None, None], _plain_rotate(x, _plain_turn(st), st), x).view(st["x"].shape)


def _run_append(st):
    n = st["kv"] * st["dim"]
    k, v = st["kv_new"][..., :n], st["kv_new"][..., n:]
    if own:
        import moe_experts_gb300 as epq
        plan = _plan(epq, st)
        epq.epq_pages_append(k, v, plan["cache"], 0, rope=plan["rope"], mask=st["mask"], n_tok=st["n_tok"])
    else:
        _plain_append(st, k, v)
    return list(st["views"])


def _run_prompt(st):
    if own:
        import moe_experts_gb300 as epq
        plan = _plan(epq, st)
        return epq.epq_attention_prompt(st["q"], plan["cache"], 0, st["heads"], st["scale"], window=st["window"], n_tok=st["n_tok"],
                                        workspace=plan["ws"])
    return _plain_prompt(st)


def _run_logits(st):
    if own:
        import moe_experts_gb300 as epq
        return epq.epq_logits_adjust(st["logits"], penalties=st["penalties"], history=st["history"], history_len=st["history_len"],
                                     prompt_len=st["prompt_len"], tokens=st["tokens"], mask=st["mask"], n_tok=st["n_tok"],
                                     bias_ids=st["bias_ids"], bias=st["bias"], allowed=st["allowed"])
    return _plain_logits(st)


# ---------------------------------------------------------------- plain forms
def _bits(mask):
    """bool [nseq][ntok][ntok]: whether bit j of entry i is set."""
    return ((mask[:, :, None] >> torch.arange(mask.shape[1], device=mask.device)) & 1) == 1


def _plain_positions(st):
    """A token's position: behind the committed ones, at its depth in its tree or at its place in the prompt."""
    i = torch.arange(st["ntok"], device="cuda")
    depth = i if st["mask"] is None else _bits(st["mask"]).sum(2) - 1
    return st["length"].long()[:, None] + depth


def _plain_turn(st):
    return st["table"][_plain_positions(st).clamp(max=st["table"].shape[0] - 1)][:, :, None]


def _plain_rotate(x, turn, st):
    """x [nseq][ntok][heads][dim]; turn [nseq][ntok][1][rot / 2][2]."""
    a, rot = st["first"], st["rot"]
    part = x[..., a:a + rot]
    c, s = turn[..., 0].to(x.dtype), turn[..., 1].to(x.dtype)
    if st["interleaved"]:
        x0, x1 = part[..., 0::2], part[..., 1::2]
    else:
        x0, x1 = part[..., : rot // 2], part[..., rot // 2:]
    y0, y1 = x0 * c - x1 * s, x1 * c + x0 * s
    turned = torch.stack([y0, y1], -1).flatten(-2) if st["interleaved"] else torch.cat([y0, y1], -1)
    return torch.cat([x[..., :a], turned, x[..., a + rot:]], -1)


def _plain_rows(x, dim):
    """float32 [..., dim] -> the cache rows [..., dim + dim/16] in bytes."""
    b = (x + 0.0).reshape(*x.shape[:-1], dim // 32, 32)
    n = torch.full((), 127.0, device=x.device)
    d = (b.abs().amax(-1, keepdim=True) / n).half()
    f = d.float()
    c = torch.where(f == 0, torch.zeros_like(b), (b / torch.where(f == 0, torch.ones_like(f), f)).round().clamp(-127, 127)).to(torch.int8)
    return torch.cat([d[..., 0].contiguous().view(torch.uint8), c.view(torch.uint8).reshape(*x.shape[:-1], dim)], -1)


def _plain_append(st, k, v):
    pool, dim, page, kv, ntok = st["pool"][0], st["dim"], st["page"], st["kv"], st["ntok"]
    nseq = st["pages"].shape[0]
    k = _plain_rotate(k.reshape(nseq, ntok, kv, dim), _plain_turn(st), st)
    i = torch.arange(ntok, device=pool.device)
    live = i < st["n_tok"][:, None]
    pos = st["length"].long()[:, None] + i
    pg, slot = st["pages"].long().gather(1, pos // page), pos % page
    rows = _plain_rows(torch.stack([k, v.reshape(nseq, ntok, kv, dim)], 3), dim)
    pool[pg, :, :, slot] = torch.where(live[:, :, None, None, None], rows, pool[pg, :, :, slot])


def _plain_prompt(st):
    pool, table, length, dim, page, kv, ntok = st["pool"][0], st["pages"].long(), st["length"].long(), st["dim"], st["page"], st["kv"], st["ntok"]
    nseq, group = table.shape[0], st["heads"] // kv
    # every sequence's rows, padded to the longest
    n = -(-st["most"] // page)
    t = torch.arange(n * page, device=pool.device)
    held = pool[table[:, :n].clamp(min=0)].permute(0, 2, 3, 1, 4, 5).reshape(nseq, kv, 2, n * page, dim + dim // 16)
    f = held[..., : dim // 16].contiguous().view(torch.float16).float()
    x = held[..., dim // 16:].contiguous().view(torch.int8).float().view(nseq, kv, 2, n * page, dim // 32, 32)
    x = (x * f[..., None]).view(nseq, kv, 2, n * page, dim)
    # scores, masked, and their softmax
    i = torch.arange(ntok, device=pool.device)
    pos = length[:, None] + i
    live = i < st["n_tok"][:, None]
    may = (t <= pos[:, :, None]) & live[:, :, None]
    if st["window"]:
        may = may & (t > pos[:, :, None] - st["window"])
    s = torch.matmul(st["q"].view(nseq, ntok, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(nseq, kv, group * ntok, dim), x[:, :, 0].transpose(2, 3))
    s = s.mul_(st["scale"]).view(nseq, kv, group, ntok, -1).masked_fill_(~may[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    e = s.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(nseq, kv, group * ntok, -1), x[:, :, 1]).view(nseq, kv, group, ntok, dim) / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 3, 1, 2, 4).reshape(nseq, ntok, st["heads"] * dim)


def _plain_counts(st, vocab):
    """int32 [nseq][ntok][vocab]: how often each token was generated before, and whether it occurs in the prompt."""
    nseq, ntok = st["tokens"].shape
    dev = st["tokens"].device
    n = torch.zeros((nseq, vocab), dtype=torch.int32, device=dev)
    before = torch.zeros((nseq, vocab), dtype=torch.int32, device=dev)
    if st["history"] is not None:
        i = torch.arange(st["history"].shape[1], device=dev)
        said, given = i < st["history_len"][:, None], i < st["prompt_len"][:, None]
        n.scatter_add_(1, st["history"].long(), (said & ~given).int())
        before.scatter_add_(1, st["history"].long(), (said & given).int())
    live = torch.arange(ntok, device=dev) < st["n_tok"][:, None]
    on = (_bits(st["mask"]) & live[:, None, :]).int()
    n = n[:, None].repeat(1, ntok, 1).scatter_add_(2, st["tokens"].long()[:, None].expand(-1, ntok, -1), on)
    return n, before[:, None] > 0


def _plain_logits(st):
    x = st["logits"]
    nseq, ntok, vocab = x.shape
    if st["bias"] is not None:
        x = x.scatter_add(2, st["bias_ids"].long()[:, None].expand(-1, ntok, -1), st["bias"][:, None].expand(-1, ntok, -1))
    n, before = _plain_counts(st, vocab)
    r, f, p = (st["penalties"][:, k, None, None] for k in range(3))
    x = torch.where((n > 0) | before, torch.where(x > 0, x / r, x * r), x)
    x = torch.where(n > 0, x - (f * n + p), x)
    if st["allowed"] is not None:
        v = torch.arange(vocab, device=x.device)
        x = torch.where(((st["allowed"][:, :, v // 32] >> (v % 32)) & 1) == 1, x, -math.inf)
    live = torch.arange(ntok, device=x.device) < st["n_tok"][:, None]
    return torch.where(live[:, :, None], x, st["logits"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["kind"] == "logits":
        rows, vocab, nseq = sum(_ragged(case, case["nseq"])), case["vocab"], case["nseq"]
        rest = nseq * case["ntok"] - rows
        return {"bytes": (8 * rows + 8 * rest) * vocab + (rows * (vocab / 8) if case["grammar"] else 0) + 4 * nseq * case["history"] + 8 * nseq * case["nbias"],
                "flops": 2 * rows * vocab}
    lengths = _ints(case["lengths"])
    n_tok, dim, ntok = _ragged(case, len(lengths)), case["dim"], case["ntok"]
    if case["kind"] == "rope":
        width = 4 * case["heads"] * dim
        return {"bytes": sum(n_tok) * 4 * case["rot"] + 2 * len(lengths) * ntok * width, "flops": 3 * sum(n_tok) * case["heads"] * case["rot"]}
    row = dim + dim // 16
    if case["kind"] == "append":
        return {"bytes": sum(n_tok) * (case["kv"] * 2 * (4 * dim + row) + 4 * case["rot"]), "flops": 8 * sum(n_tok) * case["kv"] * dim}
    heads, window = case["heads"], case["window"]
    seen, held = 0, 0
    for n, t in zip(lengths, n_tok):
        w = window or n + t
        # token i sees min(n + i + 1, w) positions
        full = min(t, max(0, n + t - w))  # tokens whose window is full
        seen += full * w + (t - full) * n + (t - full) * (t - full + 1) / 2
        held += min(n + t, w + t - 1)
    return {"bytes": held * case["kv"] * 2 * row + (sum(n_tok) + len(lengths) * ntok) * heads * dim * 4, "flops": 4 * heads * dim * seen}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "prompt": _exact_prompt, "logits": _exact_logits}[case["kind"]](st)


def _exact_turned(st, x):
    """x float64 [nseq][ntok][heads][dim] as complex pairs times exp(i angle)."""
    f, magnitude = st["exact_table"]
    nseq, ntok = x.shape[:2]
    if st["mask"] is None:
        pos = torch.arange(ntok, dtype=torch.float64, device="cuda") + st["length"].double()[:, None]
    else:
        depth = [[bin(m & (1 << 64) - 1).count("1") - 1.0 for m in r] for r in st["mask"].tolist()]
        pos = torch.tensor(depth, dtype=torch.float64, device="cuda") + st["length"].double()[:, None]
    turn = torch.polar(torch.full((), magnitude, dtype=torch.float64, device="cuda"), pos[..., None] * f)[:, :, None]
    a, b, half = st["first"], st["first"] + st["rot"], st["rot"] // 2
    index = torch.arange(half, device="cuda")
    one, two = (a + 2 * index, a + 2 * index + 1) if st["interleaved"] else (a + index, a + half + index)
    z = torch.complex(x[..., one], x[..., two]) * turn
    y = x.clone()
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_rope(st):
    nseq, ntok = st["x"].shape[:2]
    y = _exact_turned(st, st["x"].double().view(nseq, ntok, st["heads"], st["dim"])).view(nseq, ntok, -1)
    for s in range(nseq):
        n = int(st["n_tok"][s])
        y[s, n:] = st["x"][s, n:].double()
    return y


def _exact_append(st):
    """The factors; the codes are whole numbers."""
    nseq, ntok, kv, dim, page = *st["kv_new"].shape[:2], st["kv"], st["dim"], st["page"]
    x = st["kv_new"].double().view(nseq, ntok, 2, kv, dim)
    x = torch.stack([_exact_turned(st, x[:, :, 0]), x[:, :, 1]], 3)
    d = (x.view(nseq, ntok, kv, 2, dim // 32, 32).abs().amax(5) / 127)
    factors = st["views"][1].double()
    for s in range(nseq):
        p = int(st["length"][s]) + torch.arange(int(st["n_tok"][s]), device="cuda")
        factors[0, st["pages"][s].long()[p // page], :, :, p % page] = d[s, : len(p)]
    return [None, factors]


def _exact_values(rows, dim):
    f = rows[:, : dim // 16].contiguous().view(torch.float16).double().repeat_interleave(32, 1)
    return f * rows[:, dim // 16:].contiguous().view(torch.int8).double()


def _exact_prompt(st):
    dim, page, heads, kv, ntok = st["dim"], st["page"], st["heads"], st["kv"], st["ntok"]
    nseq = st["pages"].shape[0]
    out = torch.zeros((nseq, ntok, heads, dim), dtype=torch.float64, device="cuda")
    q = st["q"].view(nseq, ntok, heads, dim)
    for s in range(nseq):
        length, n = int(st["length"][s]), int(st["n_tok"][s])
        held = st["pages"][s, : -(-(length + n) // page)].long()
        behind = torch.arange(length, length + n, device="cuda")[:, None] - torch.arange(length + n, device="cuda")
        see = behind >= 0
        if st["window"]:
            see &= behind < st["window"]
        for h in range(kv):
            K, V = (_exact_values(st["pool"][0, held, h, c].reshape(-1, dim + dim // 16)[: length + n], dim) for c in (0, 1))
            for g in range(h * (heads // kv), (h + 1) * (heads // kv)):
                w = (q[s, :n, g].double() @ K.T) * st["scale"]
                out[s, :n, g] = torch.softmax(w.masked_fill_(~see, -math.inf), 1) @ V
    return out.view(nseq, ntok, heads * dim)


def _exact_logits(st):
    nseq, ntok, vocab = st["logits"].shape
    out = st["logits"].double()
    v = torch.arange(vocab, device="cuda")
    for s in range(nseq):
        r, f, p = (float(x) for x in st["penalties"][s].double())
        said, given = int(st["history_len"][s]), int(st["prompt_len"][s])
        past = st["history"][s].long() if st["history"] is not None else torch.zeros(0, dtype=torch.int64, device="cuda")
        known = torch.bincount(past[given:said], minlength=vocab)
        read = torch.bincount(past[:given], minlength=vocab)
        masks, n = st["mask"][s].tolist(), int(st["n_tok"][s])
        for i in range(n):
            path = [j for j in range(n) if masks[i] >> j & 1]
            count = known + torch.bincount(st["tokens"][s].long()[path], minlength=vocab)
            x = out[s, i]
            if st["bias"] is not None:
                x[st["bias_ids"][s].long()] += st["bias"][s].double()
            again = count + read > 0
            x[again & (x > 0)] /= r
            x[again & (x < 0)] *= r
            x -= f * count.double() + p * (count > 0).double()
            if st["allowed"] is not None:
                x[(st["allowed"][s, i].long()[v // 32] >> (v % 32)) & 1 == 0] = -math.inf
    return out
