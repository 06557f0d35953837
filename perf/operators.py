"""The measured cases of the attention and key-value cache operators.

Four operators, in the order in which a serving loop meets them:

  prompt   attention over whole prompts, packed, causal, grouped heads: K and V
           packed like Q ("prompt"), or read from the cache's pages, with a
           prefix before the new rows ("chunk")
  decode   attention of one new token per sequence over the paged cache
  append   new K and V rows into the pages
  pages    forking, granting (with copy on write), freeing and compacting pages

`own` false: elementary torch operations in 32 bits; true: the library's entry
points.  Head counts are Llama-3-8B's (32 query heads over 8 key-value heads of
128 channels: the 4096 / 1024 / 1024 outputs of the q, k and v projections that
the benchmark's decoder layer has) or small generic ones.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    llama = dict(q_heads=32, kv_heads=8, head_dim=128)
    return [
        # a chat turn's first tokens: one short prompt, launch-bound
        dict(name="prompt_17", kind="prompt", dtype="bf16", new="17", **llama),
        # a batch of prompts packed to 4096 rows, from one token to long, odd lengths
        dict(name="prompt_packed_4096", kind="prompt", dtype="bf16", new="1,700,33,1500,257,64,1541", **llama),
        # one prompt that fills an 8k context
        dict(name="prompt_8192", kind="prompt", dtype="f16", new="8192", **llama),
        # prompts' suffixes over cached prefixes, 7 query heads to a kv head, 64-channel heads
        dict(name="chunk_ragged", kind="chunk", dtype="f16", new="1,40,129,300,64", prefix="500,0,1000,37,2047",
             page=16, q_heads=14, kv_heads=2, head_dim=64),
        # a later chunk of one long prompt
        dict(name="chunk_2048_of_14336", kind="chunk", dtype="bf16", new="2048", prefix="12288", page=64, **llama),
        # one user's next token in a short chat, latency-bound
        dict(name="decode_1", kind="decode", dtype="bf16", lengths="777", page=16, **llama),
        # a serving step of 64 users, contexts up to 4096
        dict(name="decode_64", kind="decode", dtype="bf16", lengths=_ramp(64, 4096), page=16, **llama),
        # two users with very long contexts: few rows, the length has to be split
        dict(name="decode_long", kind="decode", dtype="f16", lengths="131072,100001", page=64, **llama),
        # the cache write of that serving step: one row each
        dict(name="append_64", kind="append", dtype="bf16", new=",".join(["1"] * 64), prefix=_ramp(64, 4096), page=16,
             kv_heads=8, head_dim=128),
        # the cache write of the packed prompts
        dict(name="append_4096", kind="append", dtype="f16", new="1,700,33,1500,257,64,1541", prefix="0,0,5,100,0,31,64",
             page=16, kv_heads=8, head_dim=128),
        # one prompt branches into eight answers: fork, one new token each (copy on write), all of a model's layers
        dict(name="pages_branch", kind="branch", dtype="bf16", layers=32, length=1000, children=8, grow=1, page=16,
             pages=160, kv_heads=8, head_dim=128),
        # a fragmented pool is compacted
        dict(name="pages_compact", kind="compact", dtype="bf16", layers=4, slots=64, used=1200, moves=500, page=16,
             pages=2048, kv_heads=8, head_dim=128),
    ]


def _ramp(n, most):
    """n lengths spread unevenly over 1..most, as contexts of users at different turns are."""
    return ",".join(str(1 + (i * i * 37 + i * 611) % most) for i in range(n))


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _split(rng, total, parts):
    cuts = sorted(rng.randint(0, total) for _ in range(parts - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "chunk", "decode", "decode", "append", "branch", "compact"])
    kv_heads = rng.choice([1, 2, 4, 8])
    case = dict(kind=kind, dtype=rng.choice(["f16", "bf16"]), kv_heads=kv_heads, head_dim=rng.choice([64, 128, 128]))
    group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8])
    if kind == "prompt":
        group = min(group, 32 // kv_heads)
        total = _log(rng, 1, 8000)
        case.update(q_heads=kv_heads * group, new=",".join(map(str, _split(rng, total, _log(rng, 1, 16)))))
    elif kind == "chunk":
        group = min(group, 32 // kv_heads)
        n = _log(rng, 1, 8)
        new = _split(rng, _log(rng, 1, 2048), n)
        prefix = _split(rng, _log(rng, 1, 12000 // n), n)
        case.update(q_heads=kv_heads * group, new=",".join(map(str, new)), prefix=",".join(map(str, prefix)),
                    page=rng.choice([16, 32, 64, 128]))
    elif kind == "decode":
        n = _log(rng, 1, 256)
        longest = min(131072, 200000 // n)
        case.update(q_heads=kv_heads * group, lengths=",".join(str(_log(rng, 1, longest)) for _ in range(n)),
                    page=rng.choice([16, 32, 64, 128]))
    elif kind == "append":
        n = _log(rng, 1, 128)
        new = _split(rng, _log(rng, 1, 4096), n)
        case.update(new=",".join(map(str, new)), prefix=",".join(str(rng.randint(0, 2000)) for _ in range(n)),
                    page=rng.choice([16, 32, 64, 128]))
    elif kind == "branch":
        page, length, children = rng.choice([16, 32, 64]), _log(rng, 1, 1000), rng.randint(1, 8)
        grow = _log(rng, 1, 40)
        case.update(layers=_log(rng, 1, 16), length=length, children=children, grow=grow, page=page,
                    pages=-(-length // page) + children * (-(-grow // page) + 1) + rng.randint(0, 20))
    else:
        pages = _log(rng, 32, 1024)
        used = rng.randint(1, pages - 1)
        case.update(layers=_log(rng, 1, 4), slots=rng.randint(1, 100), used=used,
                    moves=rng.randint(0, min(used, pages - used)), page=rng.choice([16, 32]), pages=pages)
    return case


# ---- inputs ----

def _numbers(text):
    return [int(t) for t in text.split(",")]


def _offsets(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _randn(shape, dtype, gen):
    return torch.randn(shape, dtype=torch.float32, device="cuda", generator=gen).to(dtype)


def _pool(case, gen, lengths, spare=3):
    """A cache whose sequences of these lengths lie in randomly ordered pages: slot i holds sequence i."""
    page, dtype = case["page"], DTYPES[case["dtype"]]
    counts = [-(-n // page) for n in lengths]
    pages = case.get("pages") or sum(counts) + spare
    shape = (case.get("layers", 1), pages, case["kv_heads"], page, case["head_dim"])
    k = torch.randn(shape, dtype=dtype, device="cuda", generator=gen)
    v = torch.randn(shape, dtype=dtype, device="cuda", generator=gen)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(gen.initial_seed()) + 1))
    slots, width = len(lengths), max(max(counts), 1) + 4
    refs = torch.zeros(pages, dtype=torch.int32)
    table = torch.full((slots, width), -1, dtype=torch.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c].to(torch.int32)
        refs[order[at:at + c]] = 1
        at += c
    return dict(k=k, v=v, refs=refs, table=table, lengths=torch.tensor(lengths, dtype=torch.int32))


def _kept(pool):
    """The pool's tensors on the GPU; its three tables are views of one buffer, with a copy to start each pass from."""
    parts = [pool["refs"].reshape(-1), pool["table"].reshape(-1), pool["lengths"]]
    words = torch.cat(parts).cuda()
    refs, table, lengths = words.split([p.numel() for p in parts])
    return dict(k=pool["k"], v=pool["v"], words=words, words0=words.clone(), refs=refs,
                table=table.view(pool["table"].shape), lengths=lengths)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, dtype, dim = case["kind"], DTYPES[case["dtype"]], case["head_dim"]
    heads, kv_heads = case.get("q_heads", 0), case["kv_heads"]
    s = dict(kind=kind)
    if kind == "prompt":
        cu = _offsets(_numbers(case["new"]))
        rows = cu[-1]
        s.update(q=1.5 * _randn((rows, heads, dim), dtype, gen), k=_randn((rows, kv_heads, dim), dtype, gen),
                 v=_randn((rows, kv_heads, dim), dtype, gen), cu=torch.tensor(cu, device="cuda"))
        s["y"] = torch.empty_like(s["q"])
    elif kind == "chunk":
        new, prefix = _numbers(case["new"]), _numbers(case["prefix"])
        s.update(_kept(_pool(case, gen, [a + b for a, b in zip(new, prefix)])))
        cu = _offsets(new)
        s.update(q=1.5 * _randn((cu[-1], heads, dim), dtype, gen), cu=torch.tensor(cu, device="cuda"),
                 slots=torch.arange(len(new), dtype=torch.int32, device="cuda"))
        s["y"] = torch.empty_like(s["q"])
    elif kind == "decode":
        lengths = _numbers(case["lengths"])
        s.update(_kept(_pool(case, gen, lengths)))
        order = torch.randperm(len(lengths), generator=torch.Generator().manual_seed(int(seed) + 2))
        s.update(q=1.5 * _randn((len(lengths), heads, dim), dtype, gen), slots=order.to(torch.int32).cuda())
        s["y"] = torch.empty_like(s["q"])
    elif kind == "append":
        new, prefix = _numbers(case["new"]), _numbers(case["prefix"])
        s.update(_kept(_pool(case, gen, [a + b for a, b in zip(new, prefix)])))
        cu = _offsets(new)
        s.update(new_k=_randn((cu[-1], kv_heads, dim), dtype, gen), new_v=_randn((cu[-1], kv_heads, dim), dtype, gen),
                 cu=torch.tensor(cu, device="cuda"),
                 slots=torch.arange(len(new), dtype=torch.int32, device="cuda"))
    elif kind == "branch":
        n = case["children"]
        pool = _pool(case, gen, [case["length"]] + [0] * n)
        grown = -(-(case["length"] + case["grow"]) // case["page"])
        if pool["table"].shape[1] < grown:
            pool["table"] = torch.nn.functional.pad(pool["table"], (0, grown - pool["table"].shape[1]), value=-1)
        s.update(_kept(pool))
        s.update(parents=torch.zeros(n, dtype=torch.int32, device="cuda"),
                 children=torch.arange(1, n + 1, dtype=torch.int32, device="cuda"),
                 grow=torch.full((n,), case["grow"], dtype=torch.int32, device="cuda"),
                 forked=torch.empty(n, dtype=torch.int32, device="cuda"),
                 granted=torch.empty(n, dtype=torch.int32, device="cuda"))
    else:
        # `used` pages in use, `moves` of them behind the used-th page, dealt to the slots
        host = torch.Generator().manual_seed(int(seed) + 3)
        used, moves, pages, slots = case["used"], case["moves"], case["pages"], case["slots"]
        low = torch.randperm(used, generator=host)[:used - moves]
        high = used + torch.randperm(pages - used, generator=host)[:moves]
        mine = torch.cat([low, high])[torch.randperm(used, generator=host)]
        counts = [used // slots + (i < used % slots) for i in range(slots)]
        pool = _pool(case, gen, [0] * slots)
        table = torch.full((slots, max(counts) + 1), -1, dtype=torch.int32)
        at = 0
        for i, c in enumerate(counts):
            table[i, :c] = mine[at:at + c].to(torch.int32)
            at += c
        refs = torch.zeros(pages, dtype=torch.int32)
        refs[mine] = 1
        lengths = [max(0, c * case["page"] - (i * 5) % case["page"]) for i, c in enumerate(counts)]
        pool.update(refs=refs, table=table, lengths=torch.tensor(lengths, dtype=torch.int32))
        s.update(_kept(pool))
        s["used"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return s


# ---- one pass ----

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import rotation_int4_weight_amd as paro

    kind = s["kind"]
    if kind == "prompt":
        paro.paro_attention_prompt(s["q"], s["k"], s["v"], s["cu"], s["cu"], s["y"])
        return s["y"]
    if "cache" not in s:
        s["cache"] = paro.KVCache(s["k"], s["v"], s["refs"], s["table"], s["lengths"])
        if kind == "decode":
            s["workspace"] = paro.make_workspace(
                paro.paro_attention_decode_workspace_bytes(s["cache"], s["q"].shape[0], s["q"].shape[1]))
        elif kind in ("branch", "compact"):
            s["workspace"] = paro.make_workspace(paro.paro_kv_workspace_bytes(s["cache"]))
    cache = s["cache"]
    if kind == "chunk":
        paro.paro_attention_prompt_cached(cache, 0, s["q"], s["slots"], s["cu"], s["y"])
        return s["y"]
    if kind == "decode":
        paro.paro_attention_decode(cache, 0, s["q"], s["slots"], s["y"], s["workspace"])
        return s["y"]
    if kind == "append":
        paro.paro_kv_append(cache, 0, s["new_k"], s["new_v"], s["slots"], s["cu"])
        return s["k"], s["v"]
    s["words"].copy_(s["words0"])
    if kind == "branch":
        paro.paro_kv_fork(cache, s["parents"], s["children"], s["forked"], s["workspace"])
        paro.paro_kv_reserve(cache, s["children"], s["grow"], s["granted"], s["workspace"])
        grown = s["words"].clone()
        paro.paro_kv_free(cache, s["parents"])
        return s["k"], s["v"], grown, s["words"], s["forked"], s["granted"]
    paro.paro_kv_compact(cache, s["used"], s["workspace"])
    return s["k"], s["v"], s["words"], s["used"]


def _attend(q, k, v, allowed, scale):
    """q [B, H, T, D], k and v [B, Hkv, S, D], allowed [B, 1, 1, T, S]: attention in 32 bits, rows with no key 0."""
    b, heads, t, dim = q.shape
    kv_heads, n = k.shape[1], k.shape[2]
    q = q.reshape(b * kv_heads, heads // kv_heads * t, dim)
    k = k.reshape(b * kv_heads, n, dim).transpose(1, 2).contiguous()
    scores = torch.bmm(q, k).view(b, kv_heads, heads // kv_heads, t, n)
    scores = scores.mul_(scale).masked_fill_(~allowed, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = scores.sum(-1, keepdim=True)
    y = torch.bmm(scores.view(b * kv_heads, -1, n), v.reshape(b * kv_heads, n, dim))
    total = total.view(b * kv_heads, -1, 1)
    return (y / total.masked_fill(total == 0, 1.0)).view(b, heads, t, dim)


def _rows(cu, n):
    """The sequence of each of n packed rows."""
    return torch.searchsorted(cu, torch.arange(n, device=cu.device), right=True) - 1


def _run_plain(s):
    kind = s["kind"]
    if kind == "prompt":
        q, k, v = (s[name].float().transpose(0, 1)[None] for name in "qkv")
        at = torch.arange(q.shape[2], device="cuda")
        seq = _rows(s["cu"], q.shape[2])
        allowed = (seq[:, None] == seq[None, :]) & (at[:, None] >= at[None, :])
        y = _attend(q, k, v, allowed[None, None, None], 1.0 / math.sqrt(q.shape[-1]))
        return y[0].transpose(0, 1).to(s["q"].dtype).contiguous()
    page = s["k"].shape[3]
    if kind in ("chunk", "decode"):
        table, lengths = s["table"][s["slots"].long()].long().clamp(min=0), s["lengths"][s["slots"].long()].long()
        dim, kv_heads = s["k"].shape[4], s["k"].shape[2]
        k, v = (s[name][0][table].float().transpose(1, 2).reshape(table.shape[0], kv_heads, -1, dim) for name in "kv")
        scale, where = 1.0 / math.sqrt(dim), torch.arange(k.shape[2], device="cuda")
        if kind == "decode":
            allowed = (where[None] < lengths[:, None])[:, None, None, None]
            return _attend(s["q"].float()[:, :, None], k, v, allowed, scale)[:, :, 0].to(s["q"].dtype)
        # all sequences' keys side by side: a row sees its own sequence's, up to its own position
        rows = s["q"].shape[0]
        seq = _rows(s["cu"], rows)
        position = lengths[seq] - s["cu"][1:][seq] + torch.arange(rows, device="cuda")
        allowed = (torch.arange(table.shape[0], device="cuda")[None, :, None] == seq[:, None, None]) \
            & (where[None, None] <= position[:, None, None])
        k, v = (x.transpose(0, 1).reshape(1, kv_heads, -1, dim) for x in (k, v))
        y = _attend(s["q"].float().transpose(0, 1)[None], k, v, allowed.view(1, 1, 1, rows, -1), scale)
        return y[0].transpose(0, 1).to(s["q"].dtype).contiguous()
    if kind == "append":
        rows = s["new_k"].shape[0]
        seq = _rows(s["cu"], rows)
        slot = s["slots"].long()[seq]
        position = s["lengths"].long()[slot] - s["cu"][1:][seq] + torch.arange(rows, device="cuda")
        where = s["table"][slot, position // page].long()
        s["k"][0, where, :, position % page] = s["new_k"]
        s["v"][0, where, :, position % page] = s["new_v"]
        return s["k"], s["v"]
    s["words"].copy_(s["words0"])
    if kind == "branch":
        _fork(s)
        _reserve(s, page)
        grown = s["words"].clone()
        _free(s, s["parents"][:1].long(), page)
        return s["k"], s["v"], grown, s["words"], s["forked"], s["granted"]
    refs, pages = s["refs"], s["refs"].numel()
    index = torch.arange(pages, device="cuda")
    live = refs > 0
    used = live.sum()
    s["used"].copy_(used)
    moving, hole = live & (index >= used), ~live & (index < used)
    source, target = index[moving], index[hole]
    where = index.clone()
    where[source] = target
    s["k"][:, target] = s["k"][:, source]
    s["v"][:, target] = s["v"][:, source]
    refs[target] = refs[source]
    refs[source] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, where[s["table"].long().clamp(min=0)].int(), s["table"]))
    return s["k"], s["v"], s["words"], s["used"]


def _fork(s):
    """Distinct empty children of live parents: each takes its parent's pages and length."""
    parents, children = s["parents"].long(), s["children"].long()
    rows = s["table"][parents]
    s["table"][children] = rows
    s["lengths"][children] = s["lengths"][parents]
    s["refs"].index_add_(0, rows[rows >= 0].long(), torch.ones_like(rows[rows >= 0]))
    s["forked"].fill_(1)


def _reserve(s, page):
    """Distinct slots grow: new pages in ascending order, a shared last page that is not full copied first."""
    slots = s["children"].long()
    length, grow = s["lengths"][slots].long(), s["grow"].long()
    have, want = (length + page - 1) // page, (length + grow + page - 1) // page
    last = s["table"][slots, (have - 1).clamp(min=0)].long().clamp(min=0)
    shared = (length % page != 0) & (s["refs"][last] > 1)
    need = want - have + shared.long()
    ends = need.cumsum(0)
    free = torch.nonzero(s["refs"] == 0)[:, 0]
    granted = (need == 0) | (ends <= free.numel())
    s["granted"].copy_(granted)
    at = torch.arange(s["table"].shape[1], device="cuda")[None]
    first = have - shared.long()
    taken = (at >= first[:, None]) & (at < want[:, None]) & granted[:, None]
    rank = (ends - need)[:, None] + at - first[:, None]
    new = free[rank.clamp(0, max(free.numel() - 1, 0))] if free.numel() else torch.zeros_like(rank)
    s["table"][slots] = torch.where(taken, new.int(), s["table"][slots])
    copied = shared & granted
    target = new.gather(1, first.clamp(min=0, max=at.shape[1] - 1)[:, None])[:, 0][copied]
    s["k"][:, target] = s["k"][:, last[copied]]
    s["v"][:, target] = s["v"][:, last[copied]]
    s["refs"].index_add_(0, last[copied], torch.full_like(target, -1, dtype=torch.int32))
    s["refs"][new[taken]] = 1
    s["lengths"][slots] = torch.where(granted, length + grow, length).int()


def _free(s, slots, page):
    """Distinct slots let go of their pages."""
    rows = s["table"][slots]
    s["refs"].index_add_(0, rows[rows >= 0].long(), torch.full_like(rows[rows >= 0], -1))
    s["table"][slots] = -1
    s["lengths"][slots] = 0


# ---- what a pass cannot do without ----

def work(case):
    kind, dim, kv_heads = case["kind"], case["head_dim"], case["kv_heads"]
    heads, row = case.get("q_heads", 0), 2 * kv_heads * dim * 2
    if kind in ("prompt", "chunk"):
        new = _numbers(case["new"])
        prefix = _numbers(case["prefix"]) if kind == "chunk" else [0] * len(new)
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, prefix))
        keys = sum(n + p for n, p in zip(new, prefix) if n)
        return {"bytes": 4 * sum(new) * heads * dim + keys * row, "flops": 4 * dim * heads * pairs}
    if kind == "decode":
        lengths = _numbers(case["lengths"])
        return {"bytes": 4 * len(lengths) * heads * dim + sum(lengths) * row, "flops": 4 * dim * heads * sum(lengths)}
    if kind == "append":
        return {"bytes": 2 * sum(_numbers(case["new"])) * row, "flops": 0}
    page = case["layers"] * case["page"] * row
    if kind == "branch":
        copies = case["children"] if case["length"] % case["page"] else 0
        held = -(-case["length"] // case["page"])
        return {"bytes": 2 * copies * page + 4 * (case["pages"] + 4 * held * (case["children"] + 1)), "flops": 0}
    return {"bytes": 2 * case["moves"] * page + 8 * (case["pages"] + case["used"]), "flops": 0}


# ---- the definition in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("prompt", "chunk", "decode"):
        q, page = s["q"], case.get("page")
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        group = q.shape[1] // case["kv_heads"]
        if kind == "decode":
            lengths = _numbers(case["lengths"])
            spans = [(r, r + 1, slot, lengths[slot]) for r, slot in enumerate(s["slots"].tolist())]
        else:
            new = _numbers(case["new"])
            cu = _offsets(new)
            prefix = _numbers(case["prefix"]) if kind == "chunk" else [0] * len(new)
            spans = [(cu[i], cu[i + 1], i, new[i] + prefix[i]) for i in range(len(new))]
        for low, high, slot, n in spans:
            if low == high:
                continue
            if kind == "prompt":
                k, v = s["k"][low:high].double(), s["v"][low:high].double()
            else:
                pages = s["table"][slot, :-(-n // page)].long()
                k, v = (s[name][0, pages].double().movedim(1, 2).flatten(0, 1)[:n] for name in "kv")
            limit = torch.arange(n - (high - low), n, device="cuda")[:, None]
            hidden = torch.arange(n, device="cuda")[None] > limit
            for h in range(q.shape[1]):
                a = q[low:high, h].double() @ k[:, h // group].t().contiguous() / math.sqrt(q.shape[2])
                out[low:high, h] = torch.softmax(a.masked_fill_(hidden, -math.inf), -1) @ v[:, h // group].contiguous()
        return out
    # the cache's steps, one page at a time on the host; the pages' values are copies
    refs, table, lengths = (s[name].tolist() for name in ("refs", "table", "lengths"))
    page = case["page"]
    k, v = s["k"].double(), s["v"].double()

    def copy(source, target):
        k[:, target], v[:, target] = k[:, source].clone(), v[:, source].clone()

    def words():
        return torch.tensor(refs + [p for row in table for p in row] + lengths, dtype=torch.int32, device="cuda")

    if kind == "append":
        new = _numbers(case["new"])
        cu = _offsets(new)
        for i in range(len(new)):
            for p0 in range(lengths[i] - new[i], lengths[i], 1):
                where, r = table[i][p0 // page], cu[i] + p0 - (lengths[i] - new[i])
                k[0, where, :, p0 % page], v[0, where, :, p0 % page] = s["new_k"][r].double(), s["new_v"][r].double()
        return k, v
    if kind == "branch":
        n = case["children"]
        held = -(-case["length"] // page)
        for c in range(1, n + 1):
            table[c], lengths[c] = list(table[0]), lengths[0]
            for p in table[0][:held]:
                refs[p] += 1
        free = [p for p in range(len(refs)) if refs[p] == 0]
        before, total, granted = list(refs), 0, []
        for c in range(1, n + 1):
            last = table[c][held - 1]
            shared = lengths[c] % page != 0 and before[last] > 1
            want = -(-(lengths[c] + case["grow"]) // page)
            need = want - held + shared
            total += need
            granted.append(int(need == 0 or total <= len(free)))
            if not granted[-1]:
                continue
            mine = free[total - need:total]
            if shared:
                copy(last, mine[0])
                refs[last] -= 1
            for i, p in enumerate(mine):
                table[c][held - shared + i] = p
                refs[p] = 1
            lengths[c] += case["grow"]
        grown = words()
        for p in table[0][:held]:
            refs[p] -= 1
        table[0], lengths[0] = [-1] * len(table[0]), 0
        return (k, v, grown, words(), torch.ones(n, dtype=torch.int32, device="cuda"),
                torch.tensor(granted, dtype=torch.int32, device="cuda"))
    live = [p for p, r in enumerate(refs) if r]
    used = len(live)
    holes = [p for p in range(used) if not refs[p]]
    to = {p: h for p, h in zip([p for p in live if p >= used], holes)}
    for a, b in to.items():
        copy(a, b)
        refs[b], refs[a] = refs[a], 0
    table = [[to.get(p, p) for p in row] for row in table]
    return k, v, words(), torch.tensor([used], dtype=torch.int32, device="cuda")
