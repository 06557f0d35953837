"""The attention half of a decoder layer as a serving loop runs it: rotated
W4A16 q/k/v projections, pages granted and written, attention over the prompts
and then token by token, the output projection; with a branch, a compaction,
a captured step, two streams and workspaces shared by two graphs."""
import numpy as np
import pytest

import synth
from _attention import check_rows, default_scale, offsets
from _helpers import LIN_TOL, torch_dtype

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")
from oracle import ref  # noqa: E402

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV_HEADS = 512, 8, 2


class Block:
    """q, k, v and output projections of one layer and a cache for their heads."""

    def __init__(self, dim, dt, slots, pages, page_size=16, max_pages=12, layers=2):
        self.dim, self.dt, self.dtype, self.layer = dim, dt, torch_dtype(dt), layers - 1
        wide = HEADS * dim
        self.host = [synth.make_layer(900 + dim, i, I, O) for i, (I, O) in
                     enumerate([(HIDDEN, wide), (HIDDEN, KV_HEADS * dim), (HIDDEN, KV_HEADS * dim), (wide, HIDDEN)])]
        self.dev = [paro.DeviceLayer(h) for h in self.host]
        self.hl = []
        for d in self.dev:
            hl = torch.empty(paro.paro_rotation_matrix_bytes(d), dtype=torch.uint8, device="cuda")
            paro.paro_rotation_matrix(d, dt, hl)
            self.hl.append(hl)
        self.cache = paro.KVCache.empty(layers, pages, KV_HEADS, page_size, dim, slots, max_pages, self.dtype)
        most = 256
        need = max(paro.paro_w4a16_linear_prepared_multi_workspace_bytes(self.dev[:3], m) for m in (1, 16, most))
        need = max([need] + [paro.paro_w4a16_linear_prepared_workspace_bytes(self.dev[3], m) for m in (1, 16, most)])
        self.ws = paro.make_workspace(need)
        self.kv_ws = paro.make_workspace(paro.paro_kv_workspace_bytes(self.cache))
        self.dec_ws = paro.make_workspace(
            max(paro.paro_attention_decode_workspace_bytes(self.cache, r, HEADS) for r in range(1, slots + 1)))

    def buffers(self, rows):
        e = lambda *s: torch.full(s, float("nan"), dtype=self.dtype, device="cuda")  # noqa: E731
        return dict(q=e(rows, HEADS, self.dim), k=e(rows, KV_HEADS, self.dim), v=e(rows, KV_HEADS, self.dim),
                    a=e(rows, HEADS, self.dim), y=e(rows, HIDDEN),
                    granted=torch.full((self.cache.c.slots,), -1, dtype=torch.int32, device="cuda"))

    def step(self, x, slots, cu, grow, b, prompt):
        """One step; slots, grow: int32, cu: int64 offsets (None: one row each)."""
        n = slots.numel()
        flat = [b[name].view(x.shape[0], -1) for name in "qkv"]
        paro.paro_w4a16_linear_prepared_multi(self.dev[:3], self.hl[:3], x, flat, self.ws)
        paro.paro_kv_reserve(self.cache, slots, grow, b["granted"][:n], self.kv_ws)
        paro.paro_kv_append(self.cache, self.layer, b["k"], b["v"], slots, cu, granted=b["granted"][:n])
        if prompt == "packed":
            paro.paro_attention_prompt(b["q"], b["k"], b["v"], cu, cu, b["a"])
        elif prompt == "cached":
            paro.paro_attention_prompt_cached(self.cache, self.layer, b["q"], slots, cu, b["a"])
        else:
            paro.paro_attention_decode(self.cache, self.layer, b["q"], slots, b["a"], self.dec_ws)
        paro.paro_w4a16_linear_prepared(self.dev[3], self.hl[3], b["a"].view(x.shape[0], -1), b["y"], self.ws)
        return b

    def x(self, rows, seed):
        x = synth.make_x(950, seed, rows, HIDDEN, self.dt)
        return torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).cuda().view(self.dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dim,dt", [(64, synth.F16), (128, synth.BF16)])
def test_serving_loop(dim, dt):
    blk = Block(dim, dt, slots=6, pages=60)
    held = {}  # slot -> the K and V rows it must hold, as the projections gave them

    def check(b, slots, counts):
        torch.cuda.synchronize()
        assert b["granted"][:len(slots)].tolist() == [1] * len(slots)
        at = 0
        for s, n in zip(slots, counts):
            k, v = (torch.cat([old, b[name][at:at + n]]) for old, name in zip(held[s], "kv"))
            held[s] = (k, v)
            assert int(blk.cache.lengths[s]) == k.shape[0]
            check_rows(b["a"][at:at + n], b["q"][at:at + n], k, v, default_scale(dim))
            at += n
        x_bits = b["a"].reshape(at, -1).cpu().view(torch.int16).numpy().view(np.uint16)
        rc, err, top, _ = ref.paro_linear_ref_check(blk.host[3], x_bits, dt, b["y"].float().cpu().numpy(), ref.F32,
                                                    LIN_TOL)
        assert rc == ref.OK, f"output projection off by {err / top:.2e}"

    empty = torch.empty((0, KV_HEADS, dim), dtype=blk.dtype, device="cuda")
    for s in range(6):
        held[s] = (empty, empty)
    # three prompts in one call, then a second chunk for one of them beside a new prompt
    slots, counts = [4, 0, 2], [37, 70, 1]
    check(blk.step(blk.x(108, 0), ints(slots), offsets(counts), ints(counts), blk.buffers(108), "packed"), slots, counts)
    slots, counts = [0, 1], [25, 20]
    check(blk.step(blk.x(45, 1), ints(slots), offsets(counts), ints(counts), blk.buffers(45), "cached"), slots, counts)
    # slot 4 branches into 3 and 5; five rows of decode, several times
    b = blk.buffers(1)
    paro.paro_kv_fork(blk.cache, ints([4, 4]), ints([3, 5]), b["granted"][:2], blk.kv_ws)
    held[3] = held[5] = held[4]
    for i in range(20):
        slots = [5, 0, 4, 2, 3][:5 - i % 2]
        check(blk.step(blk.x(len(slots), 2 + i), ints(slots), None, ints([1] * len(slots)), blk.buffers(len(slots)),
                       "decode"), slots, [1] * len(slots))
        if i == 8:
            paro.paro_kv_free(blk.cache, ints([0]))
            held[0] = (empty, empty)
            used = ints([0])
            paro.paro_kv_compact(blk.cache, used, blk.kv_ws)
            assert int((blk.cache.refs[:int(used)] > 0).sum()) == int(used) and not blk.cache.refs[int(used):].any()
    # the two branches went their own ways from a shared prefix
    n = 37
    assert torch.equal(held[3][0][:n], held[5][0][:n]) and not torch.equal(held[3][0][n:n + 1], held[5][0][n:n + 1])


def prefilled(dim=128, dt=synth.BF16, seed=0):
    blk = Block(dim, dt, slots=4, pages=40)
    counts = [50, 31, 16, 7]
    blk.step(blk.x(104, seed), ints([0, 1, 2, 3]), offsets(counts), ints(counts), blk.buffers(104), "packed")
    torch.cuda.synchronize()
    return blk


def test_captured_steps_replay_as_eager_ones():
    """Two graphs of whole decode steps (three rows and one) share one block's workspaces and are replayed in turn,
    with eager work and synchronizations between; every replay grants, writes and attends as the eager step does."""
    graphed, eager = prefilled(), prefilled()
    rows = {"a": [2, 0, 3], "b": [1]}
    xs = {g: graphed.x(len(r), 40 + len(r)) for g, r in rows.items()}
    slots = {g: ints(r) for g, r in rows.items()}
    ones = {g: ints([1] * len(r)) for g, r in rows.items()}
    bufs = {g: graphed.buffers(len(r)) for g, r in rows.items()}
    graphs = {}
    for g in rows:
        graphs[g] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[g], stream=torch.cuda.Stream()):
            graphed.step(xs[g], slots[g], None, ones[g], bufs[g], "decode")
    torch.cuda.synchronize()
    for i, g in enumerate("abbaabab" * 3):
        xs[g].copy_(graphed.x(len(rows[g]), 60 + i))
        graphs[g].replay()
        torch.cuda.synchronize()
        want = eager.step(graphed.x(len(rows[g]), 60 + i), slots[g], None, ones[g], eager.buffers(len(rows[g])), "decode")
        torch.cuda.synchronize()
        n = len(rows[g])
        assert torch.equal(bufs[g]["granted"][:n], want["granted"][:n])
        for name in ("lengths", "refs", "table"):
            assert torch.equal(getattr(graphed.cache, name), getattr(eager.cache, name)), f"replay {i}: {name}"
        for name in ("q", "k", "v", "a", "y"):
            assert torch.equal(bufs[g][name], want[name]), f"replay {i}: {name}"
    assert eager.cache.lengths.tolist() == [62, 43, 28, 19]


def test_captured_prompt_and_bookkeeping_replay():
    """A prompt over the cache, a fork, a free and a compaction in one graph."""
    blk = prefilled(64, synth.F16)
    q = torch.randn((20, HEADS, 64), device="cuda").half()
    y, want = torch.empty_like(q), torch.empty_like(q)
    cu, s = offsets([12, 8]), ints([0, 1])
    got, used = ints([0]), ints([0])
    start = [t.clone() for t in (blk.cache.refs, blk.cache.table, blk.cache.lengths, blk.cache.k, blk.cache.v)]
    paro.paro_attention_prompt_cached(blk.cache, blk.layer, q, s, cu, want)

    def work():
        paro.paro_attention_prompt_cached(blk.cache, blk.layer, q, s, cu, y)
        paro.paro_kv_free(blk.cache, ints_free)
        paro.paro_kv_fork(blk.cache, parent, child, got, blk.kv_ws)
        paro.paro_kv_compact(blk.cache, used, blk.kv_ws)

    ints_free, parent, child = ints([2]), ints([1]), ints([2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        work()
    ends = []
    for i in range(4):
        for t, t0 in zip((blk.cache.refs, blk.cache.table, blk.cache.lengths, blk.cache.k, blk.cache.v), start):
            t.copy_(t0)
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        if i == 1:
            work()  # once eagerly
        else:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and got.tolist() == [1]
        ends.append([t.clone() for t in (blk.cache.refs, blk.cache.table, blk.cache.lengths, used, blk.cache.k)])
        for a, b in zip(ends[0], ends[-1]):
            assert torch.equal(a, b), f"pass {i}"
    assert blk.cache.lengths.tolist() == [50, 31, 31, 7]


def test_two_streams_with_their_own_workspaces():
    """Decode over one cache from two streams at once, each with a workspace; the bits are those of single calls."""
    blk = Block(128, synth.F16, slots=3, pages=700, max_pages=320)
    n = [3000, 777, 1500]
    blk.cache.k.copy_(torch.randn_like(blk.cache.k))
    blk.cache.v.copy_(torch.randn_like(blk.cache.v))
    paro.paro_kv_reserve(blk.cache, ints([0, 1, 2]), ints(n), ints([0, 0, 0]), blk.kv_ws)
    calls = []
    for i, order in enumerate(([0, 1, 2], [2, 0])):
        q = torch.randn((len(order), HEADS, 128), device="cuda").half()
        need = paro.paro_attention_decode_workspace_bytes(blk.cache, len(order), HEADS)
        calls.append((torch.cuda.Stream(), q, ints(order), torch.empty_like(q), paro.make_workspace(need)))
    want = []
    for _, q, s, y, ws in calls:
        paro.paro_attention_decode(blk.cache, 1, q, s, y, ws)
        torch.cuda.synchronize()
        want.append(y.clone())
    for _ in range(10):
        for _, _, _, y, _ in calls:
            y.fill_(float("nan"))
        torch.cuda.synchronize()
        for st, q, s, y, ws in calls:
            for _ in range(4):
                paro.paro_attention_decode(blk.cache, 1, q, s, y, ws, stream=st)
        torch.cuda.synchronize()
        for (_, _, _, y, _), w in zip(calls, want):
            assert torch.equal(y, w)


def test_stream_argument_forms():
    """A torch stream, its raw handle and the default give the same."""
    blk = prefilled(64, synth.F16)
    q, s = torch.randn((2, HEADS, 64), device="cuda").half(), ints([3, 0])
    st = torch.cuda.Stream()
    ys = []
    torch.cuda.synchronize()
    for stream in (None, st, st.cuda_stream):
        y = torch.empty_like(q)
        torch.cuda.synchronize()
        paro.paro_attention_decode(blk.cache, 1, q, s, y, blk.dec_ws, stream=stream)
        torch.cuda.synchronize()
        ys.append(y)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_one_workspace_for_linears_attention_and_pages():
    """The linears, the attention's join and the page calls share their workspace's counter area, one after another."""
    dt, rows, dim = synth.F16, 2, 128
    host = synth.make_layer(970, 0, 1024, 16384)
    lin = paro.DeviceLayer(host)
    cache = paro.KVCache.empty(1, 600, 2, 16, dim, 4, 300, torch_dtype(dt))
    lengths = [2500, 1800]
    e = lambda *s: torch.full(s, float("nan"), dtype=cache.dtype, device="cuda")  # noqa: E731
    x = torch.from_numpy(np.ascontiguousarray(synth.make_x(971, 0, rows, 1024, dt)).view(np.int16)).cuda()
    x = x.view(cache.dtype)
    need = max(paro.paro_w4a16_linear_workspace_bytes(lin, rows), paro.paro_kv_workspace_bytes(cache),
               max(paro.paro_attention_decode_workspace_bytes(cache, r, 8) for r in (1, 2)),
               paro.paro_attention_prompt_cached_workspace_bytes(cache, 1, 2, 8))
    assert paro.paro_attention_prompt_cached_workspace_bytes(cache, 1, 2, 8) > 0
    shared, alone = paro.make_workspace(need), paro.make_workspace(need)
    want, got = e(rows, 16384), e(rows, 16384)
    paro.paro_w4a16_linear(lin, x, want, alone)
    granted = ints([-1, -1])
    paro.paro_kv_reserve(cache, ints([1, 3]), ints(lengths), granted, shared)
    assert granted.tolist() == [1, 1]
    k = torch.randn((sum(lengths), 2, dim), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    k = k.to(cache.dtype)
    paro.paro_kv_append(cache, 0, k, -k, ints([1, 3]), offsets(lengths))
    q = k[5:7].repeat(1, 4, 1).contiguous()
    for i in range(3):
        a = e(rows, 8, dim)
        paro.paro_attention_decode(cache, 0, q, ints([1, 3]), a, shared)
        paro.paro_attention_decode(cache, 0, q[:1], ints([3]), e(1, 8, dim), shared)
        chunk = e(2, 8, dim)
        paro.paro_attention_prompt_cached(cache, 0, q, ints([1]), offsets([2]), chunk, workspace=shared)
        check_rows(chunk, q, k[:2500], -k[:2500], default_scale(dim))
        paro.paro_w4a16_linear(lin, x, got, shared)
        assert torch.equal(got, want)
        paro.paro_kv_fork(cache, ints([1]), ints([0]), granted[:1], shared)
        paro.paro_kv_free(cache, ints([0]))
        paro.paro_kv_compact(cache, granted[:1], shared)
        paro.paro_w4a16_linear(lin, x, got.fill_(float("nan")), shared)
        assert torch.equal(got, want)
        for r, (lo, n) in enumerate(((0, 2500), (2500, 1800))):
            check_rows(a[r:r + 1], q[r:r + 1], k[lo:lo + n], -k[lo:lo + n], default_scale(dim))


def test_captured_split_chunk_follows_the_lengths():
    """Few rows, their keys split over workgroups, in a graph: replays see the lengths of the moment."""
    cache = paro.KVCache.empty(1, 250, 2, 16, 64, 2, 250, torch.float16)
    cache.k.normal_()
    cache.v.normal_()
    cache.table[1] = torch.randperm(250, device="cuda").to(torch.int32)
    cache.refs.fill_(1)
    q = torch.randn((6, 8, 64), device="cuda").half()
    y, want, s, cu = torch.empty_like(q), torch.empty_like(q), ints([1]), offsets([6])
    need = paro.paro_attention_prompt_cached_workspace_bytes(cache, 1, 6, 8)
    ws, other = paro.make_workspace(need), paro.make_workspace(need)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        paro.paro_attention_prompt_cached(cache, 0, q, s, cu, y, workspace=ws)
    for n in (4000, 6, 0, 700, 3, 513, 512, 3999, 4000):
        cache.lengths[1] = n
        y.fill_(float("nan"))
        g.replay()
        paro.paro_attention_prompt_cached(cache, 0, q, s, cu, want, workspace=other)
        torch.cuda.synchronize()
        assert torch.equal(y, want), n
    k, v = (x[0, cache.table[1].long()].transpose(1, 2).reshape(4000, 2, 64) for x in (cache.k, cache.v))
    check_rows(y, q, k, v, default_scale(64))
