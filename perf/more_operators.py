"""The measured cases of rotary positions and of the key-value cache held in four bits.

Four operators, in the order in which a serving loop meets them:

  rotary   queries and keys turned by their positions (and turned back: the gradient)
  write    new K and V rows quantised to four bits as they are written into the
           pages, and read back as the values that attention will see
  read     a slot's rows out of the pages into packed K and V, as a prompt's
           next chunk needs them
  decode   attention of one new token per sequence over the four-bit cache

`own` false: elementary torch operations in 32 bits (angles, and the quantiser's
decisions, in 64); true: the library's entry points.  Head counts are
Llama-3-8B's (32 query heads over 8 key-value heads of 128 channels, as the
benchmark's decoder layer has) or small generic ones.

A four-bit page of one head holds its codes, then a (scale, lowest value) pair
in 16 bits per position and group of 64 channels; a value is
lowest + scale * code.  With P positions of D channels:
  K codes  [P][4][D/32] words of 32 bits; word (p, g, t) holds channels
           32 t + 8 g + (0, 2, 4, 6, 1, 3, 5, 7), lowest bits first
  V codes  [P/4][16][D/64][4] words of 16 bits; word (p/4, r, u, p%4) holds
           channels 64 u + 4 r + (0, 1, 2, 3), lowest bits first
  pairs    [P][D/64][2]
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 64                           # channels that share a scale
ORDER = (0, 2, 4, 6, 1, 3, 5, 7)     # channels of a K word, lowest bits first


def listed():
    llama = dict(kv_heads=8, head_dim=128)
    return [
        # one user's next token: q and k heads of a fused q/k/v row, launch-bound
        dict(name="rotary_1", kind="rotary", dtype="bf16", new="1", prefix="776", heads=40, fused=48, head_dim=128, rot=128,
             layout="half", scaling="none", inverse=False),
        # the q and k heads of packed prompts, out of the fused q/k/v buffer; frequencies in bands for a long context
        dict(name="rotary_4096", kind="rotary", dtype="bf16", new="1,700,33,1500,257,64,1541", prefix="0,0,5,100,0,31,64",
             heads=40, fused=48, head_dim=128, rot=128, layout="half", scaling="bands", inverse=False),
        # far positions of a long context, neighbouring channels paired, half of each head turned
        dict(name="rotary_far", kind="rotary", dtype="f16", new="777,1", prefix="1047799,300001", heads=14, fused=18,
             head_dim=64, rot=32, layout="interleaved", scaling="ramp", inverse=False),
        # the gradient of 2048 rows of queries, held in 32 bits
        dict(name="rotary_gradient", kind="rotary", dtype="f32", new="1024,1,1023", prefix="0,0,0", heads=32, fused=32,
             head_dim=128, rot=128, layout="half", scaling="linear", inverse=True),
        # the cache write of a serving step of 64 users: one row each
        dict(name="write_64", kind="write", dtype="bf16", new=",".join(["1"] * 64), prefix=_ramp(64, 4096), page=16, **llama),
        # the cache write of packed prompts
        dict(name="write_4096", kind="write", dtype="f16", new="1,700,33,1500,257,64,1541", prefix="0,0,5,100,0,31,64",
             page=16, **llama),
        # everything that five slots hold, for the prompt attention of their next chunks
        dict(name="read_ragged", kind="read", dtype="f16", out="f16", lengths="501,40,1129,337,2111", page=16, kv_heads=2,
             head_dim=64),
        # a long prompt's prefix before its next chunk, and a second one's
        dict(name="read_long", kind="read", dtype="bf16", out="bf16", lengths="65536,30001", page=64, **llama),
        # one user's next token in a short chat, latency-bound
        dict(name="decode4_1", kind="decode", dtype="bf16", lengths="777", page=16, q_heads=32, **llama),
        # a serving step of 64 users, contexts up to 4096
        dict(name="decode4_64", kind="decode", dtype="bf16", lengths=_ramp(64, 4096), page=16, q_heads=32, **llama),
        # heads of 64 channels, 7 query heads to a kv head, short odd lengths
        dict(name="decode4_narrow", kind="decode", dtype="f16", lengths=_ramp(40, 1500), page=32, q_heads=14, kv_heads=2,
             head_dim=64),
        # two users with very long contexts: few rows, the length has to be split
        dict(name="decode4_long", kind="decode", dtype="f16", lengths="131072,100001", page=64, q_heads=32, **llama),
    ]


def _ramp(n, most):
    """n lengths spread unevenly over 1..most, as contexts of users at different turns are."""
    return ",".join(str(1 + (i * i * 37 + i * 611) % most) for i in range(n))


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _split(rng, total, parts):
    cuts = sorted(rng.randint(0, total) for _ in range(parts - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _text(numbers):
    return ",".join(map(str, numbers))


def draw(rng):
    kind = rng.choice(["rotary", "rotary", "write", "write", "read", "decode", "decode", "decode"])
    if kind == "rotary":
        dim = rng.choice([64, 80, 128, 128, 256])
        heads = _log(rng, 1, 48 * 64 // dim)
        n = _log(rng, 1, 16)
        new = _split(rng, _log(rng, 1, 4096), n)
        return dict(kind=kind, dtype=rng.choice(["f16", "bf16", "f32"]), new=_text(new),
                    prefix=_text(_log(rng, 1, 1 << 20) - 1 for _ in new), heads=heads, fused=heads + rng.randint(0, 8),
                    head_dim=dim, rot=rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "bands", "ramp"]), inverse=rng.random() < 0.4)
    kv_heads = rng.choice([1, 2, 4, 8])
    case = dict(kind=kind, dtype=rng.choice(["f16", "bf16"]), kv_heads=kv_heads, head_dim=rng.choice([64, 128, 128]),
                page=rng.choice([16, 32, 64, 128, 256]))
    if kind == "write":
        n = _log(rng, 1, 128)
        case.update(new=_text(_split(rng, _log(rng, 1, 4096), n)), prefix=_text(rng.randint(0, 2000) for _ in range(n)))
    elif kind == "read":
        case.update(out=rng.choice([case["dtype"], "f32"]),
                    lengths=_text(_split(rng, _log(rng, 1, 80000), _log(rng, 1, 40))))
    else:
        n = _log(rng, 1, 256)
        longest = min(131072, 200000 // n)
        case.update(q_heads=kv_heads * rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8]),
                    lengths=_text(_log(rng, 1, longest) for _ in range(n)))
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


def _frequencies(case):
    """Radians per position of each pair of channels, and what multiplies cosine and sine."""
    rot, context, factor = case["rot"], 8192.0, 8.0
    f = [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "bands":
        # by the turns over the trained context: slower than 1 stretched, faster than 4 kept, blended between
        share = [min(1.0, max(0.0, (context * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        return [x * (s + (1.0 - s) / factor) for x, s in zip(f, share)], 1.0
    if case["scaling"] == "ramp":
        # by the pair's index: kept up to the one with 32 turns, stretched from the one with 1, a ramp between
        def index(turns):
            return rot * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(500000.0))
        low, high = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rot - 1)
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(rot // 2)]
        return [x * (1.0 - r) + x / factor * r for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _quantise(x):
    """x (..., D) in 16 bits: codes (..., D/64, 64) and pairs (..., D/64, 2) of (scale, lowest value) in x's type.

    scale: a fifteenth of the group's range, taken in 64 bits, rounded to 32 and then to the type; a code is the
    whole number nearest to (x - lowest) / scale (a tie: the even one), at most 15, and 0 where the scale is 0."""
    g = x.unflatten(-1, (-1, GROUP)).double()
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((high - low) / 15.0).float().to(x.dtype)
    step = scale.double()
    codes = torch.where(step == 0, torch.zeros_like(g), torch.round((g - low) / torch.where(step == 0, 1.0, step)))
    return codes.clamp_(max=15.0).to(torch.uint8), torch.cat([scale, low.to(x.dtype)], -1)


def _k_bytes(codes):
    """codes (..., P, D/64, 64) of K rows as the bytes (..., P, D/2) of their words."""
    c = codes.flatten(-2)
    c = c.unflatten(-1, (c.shape[-1] // 32, 4, 8)).transpose(-3, -2)[..., list(ORDER)].contiguous()
    return (c[..., 0::2] | c[..., 1::2] << 4).flatten(-3)


def _v_words(codes):
    """codes (..., P, D/64, 64) of V rows as the two bytes of their words (..., P, 16, D/64, 2)."""
    c = codes.unflatten(-1, (16, 4)).transpose(-3, -2).contiguous()
    return c[..., 0::2] | c[..., 1::2] << 4


def _pages(x, key):
    """x (pages, heads, P, D) as the bytes of its four-bit pages (pages, heads, P, 9 D / 16)."""
    n, heads, page, dim = x.shape
    codes, pairs = _quantise(x)
    if key:
        body = _k_bytes(codes).flatten(2)
    else:
        body = _v_words(codes).unflatten(2, (page // 4, 4)).movedim(3, 5).contiguous().flatten(2)
    return torch.cat([body, pairs.view(torch.uint8).flatten(2)], -1).view(n, heads, page, dim * 9 // 16)


def _pool(case, gen, lengths):
    """A cache of one layer whose sequences of these lengths lie in randomly ordered pages: slot i holds sequence i."""
    page, dtype, dim, heads = case["page"], DTYPES[case["dtype"]], case["head_dim"], case["kv_heads"]
    counts = [-(-n // page) for n in lengths]
    pages = sum(counts) + 3
    # keys have a few channels that are larger than the others
    gain = torch.ones((heads, 1, dim), device="cuda")
    gain[:, :, 3::37] = 4.0
    k = _pages((torch.randn((pages, heads, page, dim), device="cuda", generator=gen) * gain).to(dtype), True)
    v = _pages(_randn((pages, heads, page, dim), dtype, gen), False)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(gen.initial_seed()) + 1))
    table = torch.full((len(lengths), max(max(counts), 1) + 4), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c].to(torch.int32)
        refs[order[at:at + c]] = 1
        at += c
    return dict(k=k[None].contiguous(), v=v[None].contiguous(), refs=refs.cuda(), table=table.cuda(),
                lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"), dtype=dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, dtype, dim = case["kind"], DTYPES[case["dtype"]], case["head_dim"]
    s = dict(kind=kind)
    if kind == "rotary":
        new, prefix = _numbers(case["new"]), _numbers(case["prefix"])
        x = _randn((sum(new), case["fused"], dim), dtype, gen)[:, :case["heads"]]
        at = torch.cat([torch.arange(p, p + n, dtype=torch.int32) for n, p in zip(new, prefix)])
        freqs, magnitude = _frequencies(case)
        s.update(x=x, positions=at.cuda(), freqs=torch.tensor(freqs, dtype=torch.float64, device="cuda"),
                 magnitude=magnitude, interleaved=case["layout"] == "interleaved", inverse=case["inverse"])
        s["y"] = torch.empty(x.shape, dtype=dtype, device="cuda")
    elif kind == "write":
        new, prefix = _numbers(case["new"]), _numbers(case["prefix"])
        s.update(_pool(case, gen, [a + b for a, b in zip(new, prefix)]))
        cu = _offsets(new)
        s.update(new_k=_randn((cu[-1], case["kv_heads"], dim), dtype, gen),
                 new_v=_randn((cu[-1], case["kv_heads"], dim), dtype, gen), cu=torch.tensor(cu, device="cuda"),
                 slots=torch.arange(len(new), dtype=torch.int32, device="cuda"))
        s["out_k"], s["out_v"] = (torch.empty(s["new_k"].shape, device="cuda") for _ in range(2))
    elif kind == "read":
        lengths = _numbers(case["lengths"])
        s.update(_pool(case, gen, lengths))
        cu = _offsets(lengths)
        s.update(cu=torch.tensor(cu, device="cuda"),
                 slots=torch.arange(len(lengths), dtype=torch.int32, device="cuda"))
        s["out_k"], s["out_v"] = (torch.empty((cu[-1], case["kv_heads"], dim), dtype=DTYPES[case["out"]], device="cuda")
                                  for _ in range(2))
    else:
        lengths = _numbers(case["lengths"])
        s.update(_pool(case, gen, lengths))
        order = torch.randperm(len(lengths), generator=torch.Generator().manual_seed(int(seed) + 2))
        s.update(q=1.5 * _randn((len(lengths), case["q_heads"], dim), dtype, gen), slots=order.to(torch.int32).cuda())
        s["y"] = torch.empty_like(s["q"])
    return s


# ---- one pass ----

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import rotation_int4_weight_amd as paro

    kind = s["kind"]
    if kind == "rotary":
        paro.paro_rotary(s["x"], s["positions"], s["freqs"], s["y"], interleaved=s["interleaved"], inverse=s["inverse"],
                         magnitude=s["magnitude"])
        return s["y"]
    if "cache" not in s:
        s["cache"] = paro.KVCache(s["k"], s["v"], s["refs"], s["table"], s["lengths"], dtype=s["dtype"])
        if kind == "decode":
            s["workspace"] = paro.make_workspace(
                paro.paro_attention_decode_workspace_bytes(s["cache"], s["q"].shape[0], s["q"].shape[1]))
    cache = s["cache"]
    if kind == "decode":
        paro.paro_attention_decode(cache, 0, s["q"], s["slots"], s["y"], s["workspace"])
        return s["y"]
    if kind == "write":
        paro.paro_kv_append(cache, 0, s["new_k"], s["new_v"], s["slots"], s["cu"])
    paro.paro_kv_read(cache, 0, s["out_k"], s["out_v"], s["slots"], s["cu"])
    return s["out_k"], s["out_v"]


def _rows(cu, n):
    """The sequence of each of n packed rows."""
    return torch.searchsorted(cu, torch.arange(n, device=cu.device), right=True) - 1


def _nibbles(b):
    """bytes (..., n) as their codes (..., 2 n), lowest bits first."""
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _values(pages, key, dtype):
    """Four-bit pages (..., P, 9 D / 16) as the values (..., P, D) in 32 bits that they hold."""
    page, dim = pages.shape[-2], pages.shape[-1] * 16 // 9
    flat = pages.flatten(-2)
    pairs = flat[..., page * dim // 2:].contiguous().view(dtype).float().unflatten(-1, (page, dim // GROUP, 2))
    body = flat[..., :page * dim // 2]
    if key:
        c = _nibbles(body.unflatten(-1, (page, 4, dim // 32, 4)))
        inverse = [ORDER.index(i) for i in range(8)]
        c = c[..., inverse].transpose(-3, -2).flatten(-3)
    else:
        c = _nibbles(body.unflatten(-1, (page // 4, 16, dim // GROUP, 4, 2)))
        c = c.movedim(-2, -4).transpose(-3, -2).flatten(-3).flatten(-3, -2)
    c = c.float().unflatten(-1, (dim // GROUP, GROUP))
    return (pairs[..., 1:] + pairs[..., :1] * c).flatten(-2)


def _where(s, rows, page):
    """Page and row in it of the newest positions of the slots, for packed rows."""
    seq = _rows(s["cu"], rows)
    slot = s["slots"].long()[seq]
    position = s["lengths"].long()[slot] - s["cu"][1:][seq] + torch.arange(rows, device="cuda")
    return s["table"][slot, position // page].long(), position % page


def _run_plain(s):
    kind = s["kind"]
    if kind == "rotary":
        rot = 2 * s["freqs"].numel()
        angle = s["positions"].double()[:, None] * s["freqs"]
        cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
        if s["inverse"]:
            sin = -sin
        x = s["x"].float()
        if s["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = (a * cos - b * sin, b * cos + a * sin)
        turned = torch.stack(turned, -1).flatten(-2) if s["interleaved"] else torch.cat(turned, -1)
        return torch.cat([turned, x[..., rot:]], -1).to(s["x"].dtype)
    page, dim, dtype = s["k"].shape[3], s["k"].shape[4] * 16 // 9, s["dtype"]
    if kind == "write":
        where, at = _where(s, s["new_k"].shape[0], page)
        size = page * dim // 2
        for name, key in (("k", True), ("v", False)):
            codes, pairs = _quantise(s["new_" + name])
            flat = s[name][0].flatten(-2)
            tail = flat[..., size:].unflatten(-1, (page, -1))
            tail[where, :, at] = pairs.view(torch.uint8).flatten(2)
            if key:
                flat[..., :size].unflatten(-1, (page, -1))[where, :, at] = _k_bytes(codes[..., None, :, :])[:, :, 0]
            else:
                words = flat[..., :size].unflatten(-1, (page // 4, 16, dim // GROUP, 4, 2))
                words[where, :, at // 4, :, :, at % 4] = _v_words(codes[..., None, :, :])[:, :, 0]
    if kind in ("write", "read"):
        # whole pages of the slots, then the rows asked for
        rows = s["out_k"].shape[0]
        where, at = _where(s, rows, page)
        used, index = torch.unique(where, return_inverse=True)
        return tuple(_values(s[name][0][used], key, dtype)[index, :, at].to(s["out_k"].dtype)
                     for name, key in (("k", True), ("v", False)))
    table, lengths = s["table"][s["slots"].long()].long().clamp(min=0), s["lengths"][s["slots"].long()].long()
    kv_heads = s["k"].shape[2]
    k, v = (_values(s[name][0][table], key, dtype).transpose(1, 2).reshape(table.shape[0], kv_heads, -1, dim)
            for name, key in (("k", True), ("v", False)))
    n, heads = k.shape[2], s["q"].shape[1]
    q = s["q"].float().view(-1, kv_heads, heads // kv_heads, dim)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(1.0 / math.sqrt(dim))
    scores.masked_fill_((torch.arange(n, device="cuda") >= lengths[:, None])[:, None, None], -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    y = torch.matmul(scores, v) / scores.sum(-1, keepdim=True)
    return y.view(-1, heads, dim).to(s["q"].dtype)


# ---- what a pass cannot do without ----

def work(case):
    kind, dim = case["kind"], case["head_dim"]
    if kind == "rotary":
        rows, size = sum(_numbers(case["new"])), 4 if case["dtype"] == "f32" else 2
        turned = rows * case["heads"] * case["rot"]
        return {"bytes": 2 * rows * case["heads"] * dim * size + rows * 4 + case["rot"] * 4, "flops": 3 * turned}
    held = 2 * case["kv_heads"] * dim * 9 // 16  # bytes of one position's K and V
    if kind == "write":
        rows = sum(_numbers(case["new"]))
        # read, written in four bits, and handed out in 32
        return {"bytes": rows * (2 * case["kv_heads"] * dim * (2 + 4) + held), "flops": 0}
    rows = sum(_numbers(case["lengths"]))
    if kind == "read":
        return {"bytes": rows * (held + 2 * case["kv_heads"] * dim * (4 if case["out"] == "f32" else 2)), "flops": 0}
    sequences = len(_numbers(case["lengths"]))
    return {"bytes": 4 * sequences * case["q_heads"] * dim + rows * held, "flops": 4 * dim * case["q_heads"] * rows}


# ---- the definition in 64 bits ----

def _held(case, pages, key, dtype):
    """Pages (n, heads, P, 9 D / 16) as the values (n P, heads, D) in 64 bits: each channel's byte by its address."""
    n, heads, page, _ = pages.shape
    dim = case["head_dim"]
    flat = pages.flatten(2)
    p, c = torch.arange(page, device="cuda")[:, None], torch.arange(dim, device="cuda")[None]
    if key:
        place = (c % 8) // 2 + 4 * (c % 2)                     # which nibble of the word
        byte = 4 * ((p * 4 + c % 32 // 8) * (dim // 32) + c // 32) + place // 2
    else:
        place = c % 4
        byte = 2 * ((((p // 4) * 16 + c % 64 // 4) * (dim // 64) + c // 64) * 4 + p % 4) + place // 2
    code = (flat[:, :, byte.flatten()] >> (4 * (place % 2)).expand(page, dim).flatten()) & 15
    pair = flat[:, :, page * dim // 2:].contiguous().view(dtype).double().view(n, heads, page, dim // 64, 2)
    pair = pair.repeat_interleave(64, 3)
    out = pair[..., 1] + pair[..., 0] * code.view(n, heads, page, dim)
    return out.transpose(1, 2).reshape(n * page, heads, dim)


def _rounded(rows):
    """What a written row stands for, group by group, in 64 bits."""
    out = torch.empty(rows.shape, dtype=torch.float64, device="cuda")
    for first in range(0, rows.shape[-1], 64):
        x = rows[..., first:first + 64].double()
        low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        step = ((high - low) / 15).to(torch.float32).to(rows.dtype).double()
        code = torch.nan_to_num((x - low) / step, nan=0.0, posinf=0.0).round().clamp(0, 15)
        out[..., first:first + 64] = low + step * code
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind, dim = case["kind"], case["head_dim"]
    if kind == "rotary":
        x, rot = s["x"].double(), case["rot"]
        y = x.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + rot // 2)
            angle = (s["positions"].double() * float(s["freqs"][i]))[:, None]
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.full_like(angle, s["magnitude"]),
                                                                  -angle if s["inverse"] else angle)
            y[..., a], y[..., b] = z.real, z.imag
        return y
    if kind == "write":
        return _rounded(s["new_k"]), _rounded(s["new_v"])
    lengths, page, dtype = _numbers(case["lengths"]), case["page"], s["dtype"]

    def rows(name, slot):
        mine = s["table"][slot, :-(-lengths[slot] // page)].long()
        return _held(case, s[name][0, mine], name == "k", dtype)[:lengths[slot]]

    if kind == "read":
        return tuple(torch.cat([rows(name, i) for i in range(len(lengths))]) for name in ("k", "v"))
    q = s["q"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    group = q.shape[1] // case["kv_heads"]
    for r, slot in enumerate(s["slots"].tolist()):
        k, v = rows("k", slot), rows("v", slot)
        for h in range(case["kv_heads"]):
            mine = slice(h * group, (h + 1) * group)
            a = q[r, mine].double() @ k[:, h].t().contiguous() / math.sqrt(dim)
            out[r, mine] = torch.softmax(a, -1) @ v[:, h].contiguous()
    return out
