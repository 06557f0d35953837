"""The attention half of a decoder layer as a serving loop runs it with rotary positions and a cache in four bits:
rotated W4A16 q/k/v projections, positions, pages granted and written, attention over the prompts, over a read-back
prefix and then token by token, the output projection; with a branch and a compaction, captured steps, and one
workspace for everything."""
import numpy as np
import pytest

import synth
from _attention import check_rows, default_scale, offsets
from _helpers import torch_dtype

torch = pytest.importorskip("torch")
paro = pytest.importorskip("rotation_int4_weight_amd")
import _kv4  # noqa: E402

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV_HEADS, PAGE = 512, 8, 2, 16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Block:
    """q, k, v and output projections of one layer, and a cache in four bits for their heads."""

    def __init__(self, dim, dt, slots, pages, max_pages=16, layers=2):
        self.dim, self.dt, self.dtype, self.layer = dim, dt, torch_dtype(dt), layers - 1
        wide = HEADS * dim
        self.dev = [paro.DeviceLayer(synth.make_layer(980 + dim, i, I, O)) for i, (I, O) in
                    enumerate([(HIDDEN, wide), (HIDDEN, KV_HEADS * dim), (HIDDEN, KV_HEADS * dim), (wide, HIDDEN)])]
        self.hl = []
        for d in self.dev:
            hl = torch.empty(paro.paro_rotation_matrix_bytes(d), dtype=torch.uint8, device="cuda")
            paro.paro_rotation_matrix(d, dt, hl)
            self.hl.append(hl)
        self.cache = paro.KVCache.empty(layers, pages, KV_HEADS, PAGE, dim, slots, max_pages, self.dtype, bits=4)
        self.freqs, self.magnitude = paro.paro_rotary_frequencies(dim // 2, kind="ramp", factor=4.0, context=128.0, high=8.0)
        need = max(paro.paro_w4a16_linear_prepared_multi_workspace_bytes(self.dev[:3], m) for m in (1, 16, 256))
        need = max([need, paro.paro_kv_workspace_bytes(self.cache)] +
                   [paro.paro_w4a16_linear_prepared_workspace_bytes(self.dev[3], m) for m in (1, 16, 256)] +
                   [paro.paro_attention_decode_workspace_bytes(self.cache, r, HEADS) for r in range(1, slots + 1)])
        self.ws = paro.make_workspace(need)  # one for all, one call after another

    def buffers(self, rows):
        """The heads of q, k and v lie side by side in one row, as a fused projection would leave them."""
        e = lambda *s: torch.full(s, float("nan"), dtype=self.dtype, device="cuda")  # noqa: E731
        fused = e(rows, HEADS + 2 * KV_HEADS, self.dim)
        return dict(fused=fused, q=fused[:, :HEADS], k=fused[:, HEADS:HEADS + KV_HEADS], v=fused[:, HEADS + KV_HEADS:],
                    flat=[e(rows, n * self.dim) for n in (HEADS, KV_HEADS, KV_HEADS)], a=e(rows, HEADS, self.dim),
                    y=e(rows, HIDDEN), granted=torch.full((self.cache.c.slots,), -1, dtype=torch.int32, device="cuda"))

    def step(self, x, slots, cu, grow, positions, b, prompt, before=None):
        """One step; slots, grow, positions: int32, cu: int64 offsets (None: one row each)."""
        n = slots.numel()
        paro.paro_w4a16_linear_prepared_multi(self.dev[:3], self.hl[:3], x, b["flat"], self.ws)
        for name, flat in zip("qkv", b["flat"]):
            b[name].copy_(flat.view(b[name].shape))
        turned = b["fused"][:, :HEADS + KV_HEADS]
        paro.paro_rotary(turned, positions, self.freqs, turned, magnitude=self.magnitude)
        paro.paro_kv_reserve(self.cache, slots, grow, b["granted"][:n], self.ws)
        paro.paro_kv_append(self.cache, self.layer, b["k"], b["v"], slots, cu, granted=b["granted"][:n])
        if prompt == "packed":
            paro.paro_attention_prompt(b["q"], b["k"], b["v"], cu, cu, b["a"])
        elif prompt == "chunk":  # the whole slots back, then the rows over them
            cu_k, keys = before
            paro.paro_kv_read(self.cache, self.layer, *keys, slots, cu_k)
            paro.paro_attention_prompt(b["q"], *keys, cu, cu_k, b["a"])
        else:
            paro.paro_attention_decode(self.cache, self.layer, b["q"], slots, b["a"], self.ws)
        paro.paro_w4a16_linear_prepared(self.dev[3], self.hl[3], b["a"].view(x.shape[0], -1), b["y"], self.ws)
        return b

    def x(self, rows, seed):
        x = synth.make_x(990, seed, rows, HIDDEN, self.dt)
        return torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).cuda().view(self.dtype)


def positions(starts, counts):
    return ints([p for s, n in zip(starts, counts) for p in range(s, s + n)])


@pytest.mark.parametrize("dim,dt", [(64, synth.F16), (128, synth.BF16)])
def test_serving_loop(dim, dt):
    blk = Block(dim, dt, slots=6, pages=60)
    empty = torch.empty((0, KV_HEADS, dim), dtype=blk.dtype)
    held = {s: (empty, empty) for s in range(6)}  # slot -> the K and V rows that were written to it

    def run(slots, counts, seed, prompt):
        starts = [held[s][0].shape[0] for s in slots]
        rows, b = sum(counts), blk.buffers(sum(counts))
        cu = offsets(counts) if prompt != "decode" else None
        before = None
        if prompt == "chunk":
            lengths = [a + n for a, n in zip(starts, counts)]
            before = (offsets(lengths), [torch.empty((sum(lengths), KV_HEADS, dim), dtype=blk.dtype, device="cuda")
                                         for _ in range(2)])
        blk.step(blk.x(rows, seed), ints(slots), cu, ints(counts), positions(starts, counts), b, prompt, before)
        torch.cuda.synchronize()
        assert b["granted"][:len(slots)].tolist() == [1] * len(slots) and bool(torch.isfinite(b["y"]).all())
        at = 0
        for s, n in zip(slots, counts):
            held[s] = tuple(torch.cat([old, b[name][at:at + n].cpu()]) for old, name in zip(held[s], "kv"))
            at += n
        # what the slots hold, as the format defines it; attention over that (a packed prompt sees its own rows)
        at = 0
        for i, (s, n) in enumerate(zip(slots, counts)):
            k, v = (_kv4.stands_for(*_kv4.quantise(t)) for t in held[s])
            got, q = b["a"][at:at + n], b["q"][at:at + n]
            if prompt == "decode":
                _kv4.check_decode(got[0], q[0], k, v, default_scale(dim))
            elif prompt == "packed":
                check_rows(got, q, b["k"][at:at + n], b["v"][at:at + n], default_scale(dim))
            else:
                lo, hi = int(before[0][i]), int(before[0][i + 1])
                read = [t[lo:hi] for t in before[1]]
                for t, want in zip(read, (k, v)):
                    u = _kv4.HALF_STEP[blk.dtype]
                    off = (t.cpu().double() - want).abs()
                    assert bool((off <= (u + 2.0 ** -23) * want.abs() + (2.0 ** -25 if dt == synth.F16 else 0)).all())
                check_rows(got, q, *read, default_scale(dim))
            at += n

    # three prompts in one call, a second chunk for one of them beside a new prompt
    run([4, 0, 2], [37, 70, 1], 0, "packed")
    run([0, 1], [25, 20], 1, "chunk")
    # slot 4 branches into 3 and 5; rows of decode, several times
    got = ints([0, 0])
    paro.paro_kv_fork(blk.cache, ints([4, 4]), ints([3, 5]), got, blk.ws)
    assert got.tolist() == [1, 1]
    held[3] = held[5] = held[4]
    for i in range(16):
        slots = [5, 0, 4, 2, 3][:5 - i % 2]
        run(slots, [1] * len(slots), 2 + i, "decode")
        if i == 7:
            paro.paro_kv_free(blk.cache, ints([0]))
            held[0] = (empty, empty)
            used = ints([0])
            paro.paro_kv_compact(blk.cache, used, blk.ws)
            assert int((blk.cache.refs > 0).sum()) == int(used) and not blk.cache.refs[int(used):].any()
    run([3, 0], [9, 30], 40, "chunk")
    # the branches went their own ways from a shared prefix
    assert torch.equal(held[3][0][:37], held[5][0][:37]) and not torch.equal(held[3][0][37], held[5][0][37])


def test_captured_steps_replay_as_eager_ones():
    """Two graphs of whole decode steps (three rows and one) that share one workspace are replayed in turn, with eager
    work and synchronizations between; positions follow the lengths on the device."""
    def make():
        blk = Block(128, synth.BF16, slots=4, pages=60)
        counts = [50, 31, 16, 7]
        blk.step(blk.x(104, 0), ints([0, 1, 2, 3]), offsets(counts), ints(counts), positions([0] * 4, counts),
                 blk.buffers(104), "packed")
        torch.cuda.synchronize()
        return blk

    graphed, eager = make(), make()
    rows = {"a": [2, 0, 3], "b": [1]}
    xs = {g: graphed.x(len(r), 40 + len(r)) for g, r in rows.items()}
    slots = {g: ints(r) for g, r in rows.items()}
    ones = {g: ints([1] * len(r)) for g, r in rows.items()}
    bufs = {g: graphed.buffers(len(r)) for g, r in rows.items()}

    def step(blk, g, x, b):
        at = blk.cache.lengths.index_select(0, slots[g])
        return blk.step(x, slots[g], None, ones[g], at, b, "decode")

    graphs = {}
    for g in rows:
        graphs[g] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[g], stream=torch.cuda.Stream()):
            step(graphed, g, xs[g], bufs[g])
    torch.cuda.synchronize()
    for i, g in enumerate("abbaabab" * 3):
        x = graphed.x(len(rows[g]), 60 + i)
        xs[g].copy_(x)
        graphs[g].replay()
        torch.cuda.synchronize()
        want = step(eager, g, x, eager.buffers(len(rows[g])))
        torch.cuda.synchronize()
        for name in ("lengths", "refs", "table"):
            assert torch.equal(getattr(graphed.cache, name), getattr(eager.cache, name)), f"replay {i}: {name}"
        for s in range(4):
            n = int(eager.cache.lengths[s])
            for a, b in zip(_kv4.held_rows(graphed.cache, 1, s, n), _kv4.held_rows(eager.cache, 1, s, n)):
                assert torch.equal(a, b), f"replay {i}: slot {s}"
        for name in ("q", "k", "v", "a", "y"):
            assert torch.equal(bufs[g][name], want[name]), f"replay {i}: {name}"
    assert eager.cache.lengths.tolist() == [62, 43, 28, 19]
