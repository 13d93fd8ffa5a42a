"""GPU parity of tree attention on the 4-bit cache against the definition in 64 bits, on the values that the cache
holds (oracle/kv4.py, exact) and the nodes' own keys.

Bounds (reference()). ds, a score's absolute error in natural-log units: the fp32 sum of D products errs by at most D 2^-22 of
the sum of their magnitudes (each of D / 16 MMA steps adds 17 terms cut at 2^-23 of the largest); scaling, the
difference from the running maximum and ex2.approx add 2^-20 of the score and 2^-18. o: each p moves by a factor within
e^(2 dsum) (its own error and the sum's, dsum with the fp32 sum's n 2^-23), P is rounded to fp16 (2^-11, or
2^-25 absolute against a sum of at least 1), PV's fp32 sum of n terms errs by n 2^-22, the output is rounded (2^-11, or 2^-25). The
LSE adds q . shift, D products in fp32 (D 2^-23 of the sum of their magnitudes).
"""
import threading

import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from oracle import kv4
from test_gpu_kv4 import host, new_cache, rows

pytestmark = pytest.mark.gpu


def pasa():
    import precision_flashattention_numerics_gb300 as p

    return p


def tree(rng, B, n, kind):
    if kind == "chain":
        return np.tile(np.arange(-1, n - 1), (B, 1)).astype(np.int32)
    if kind == "roots":
        return np.full((B, n), -1, np.int32)
    p = (rng.random((B, n)) * (np.arange(n) + 1)).astype(np.int32) - 1
    if kind == "odd":    # numbers that are not before the node end the path
        p[rng.random((B, n)) < 0.2] = 2 ** 31 - 1
        p[rng.random((B, n)) < 0.1] = -2 ** 31
        p[:, n // 2] = n // 2
    return p


def path(parents, i):
    seen = []
    while i >= 0:
        seen.append(i)
        i = parents[i] if parents[i] < i else -1
    return seen


def reference(q, kn, vn, kv, vv, lengths, parents, counts, scale, shift):
    """o, lse and bounds on their errors; kv, vv: the cache's values (without the shift), kn, vn: the nodes' (all 64 bits)."""
    q = q.astype(np.float64)
    B, Hq, n, D = q.shape
    H = kv.shape[1]
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(B):
        see = np.zeros((n, lengths[b] + n), bool)
        for i in range(counts[b]):
            see[i, :lengths[b]] = True
            see[i, lengths[b] + np.array(path(parents[b], i))] = True
        alive = see.any(1)
        if not alive.any():
            continue
        for h in range(Hq):
            g = h // (Hq // H)
            k = np.concatenate([kv[b, g, :lengths[b]], kn[b, g] - shift[b, g]])
            raw = np.concatenate([np.abs(kv[b, g, :lengths[b]]), np.abs(kn[b, g]) + np.abs(shift[b, g])])   # of a score's products
            v = np.concatenate([vv[b, g, :lengths[b]], vn[b, g]])
            qs = q[b, h][alive]
            s = see[alive]
            x = np.where(s, scale * (qs @ k.T), -np.inf)
            top = x.max(1, keepdims=True)
            p = np.exp(x - top)
            total = p.sum(1, keepdims=True)
            p /= total
            off = scale * (qs @ shift[b, g])
            lse[b, h, alive] = (top + np.log(total))[:, 0] + off
            o[b, h, alive] = p @ v
            mag = scale * np.where(s, np.abs(qs) @ raw.T, 0).max(1)
            ds = mag * (D * 2.0 ** -22 + 2.0 ** -20) + 2.0 ** -18
            dsum = ds + (s.sum(1) + 2) * 2.0 ** -23
            bl[b, h, alive] = (dsum + scale * (np.abs(qs) @ np.abs(shift[b, g])) * D * 2.0 ** -23
                               + np.abs(lse[b, h, alive]) * 2.0 ** -21 + np.abs(off) * 2.0 ** -22 + 2.0 ** -20)
            bo[b, h, alive] = ((p @ np.abs(v)) * (2.0 ** -11 + np.expm1(2 * dsum) + s.sum(1) * 2.0 ** -22)[:, None]
                               + (s @ np.abs(v)) * 2.0 ** -25 + np.abs(o[b, h, alive]) * 2.0 ** -11 + 2.0 ** -25)
    return o, lse, bo, bl


def check(got, ref):
    (o, lse), (ro, rl, bo, bl) = host(*got), ref
    off = np.abs(o.astype(np.float64) - ro)
    assert (off <= bo).all(), (float(np.nanmax(off / np.maximum(bo, 1e-300))), np.isnan(off).any())
    fin = np.isfinite(rl)
    assert np.array_equal(np.isneginf(lse), ~fin)
    off = np.abs(lse[fin] - rl[fin])
    assert (off <= bl[fin]).all(), float((off / bl[fin]).max())


class Case:
    """Inputs on the device, with garbage wherever nothing may be read, and the reference."""

    def __init__(self, seed, B, Hq, H, n, Sk, cap, D, lengths=None, counts=None, kind="tree", shifted=True):
        rng = np.random.default_rng(seed)
        self.B, self.D, self.Sk, self.scale = B, D, Sk, D ** -0.5
        self.len_arg, self.count_arg, self.kind = lengths, counts, kind
        self.lengths = np.clip(lengths if lengths is not None else [Sk] * B, 0, Sk)
        self.counts = np.clip(counts if counts is not None else [n] * B, 0, n)
        bias = 10 * rng.standard_normal((B, H, 1, D)) if shifted else 0
        k = (rng.standard_normal((B, H, cap, D)) + bias).astype(np.float16)
        v = rows(rng, B, H, cap, D, "plain")
        self.kn = (rng.standard_normal((B, H, n, D)) + bias).astype(np.float16)
        self.vn = rows(rng, B, H, n, D, "plain")
        self.q = rng.standard_normal((B, Hq, n, D)).astype(np.float16)
        self.parents = tree(rng, B, n, kind)
        shift = k[:, :, 0].copy() if shifted else None
        self.zero_shift = (shift if shifted else np.zeros((B, H, D))).astype(np.float64)
        self.cache = new_cache(B, H, cap, D)
        kt, vt = to_dev(k, v)
        self.shift = to_dev(shift)[0] if shifted else None
        pasa().kv4_append(kt, vt, *self.cache, shift=self.shift)
        for b in range(B):
            for x, fill in zip(self.cache, (255, float("nan"), 255, float("inf"))):
                x[b, :, self.lengths[b]:] = fill
        self.held = kv4.values(*kv4.quantise(k, shift)), kv4.values(*kv4.quantise(v))
        self.nodes = self.kn.astype(np.float64), self.vn.astype(np.float64)
        foul = [x.copy() for x in (self.q, self.kn, self.vn, self.parents)]
        for b in range(B):
            for x in foul[:3]:
                x[b, :, self.counts[b]:] = np.nan
            foul[3][b, self.counts[b]:] = 5
        self.dev = to_dev(*foul)

    def ints(self, x):
        return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")

    def run(self, scale=None, **kw):
        q, k, v, parents = self.dev
        got = pasa().attn_fwd_tree_kv4(q, k, v, *self.cache, None if self.kind == "chain" else parents, scale=scale, shift=self.shift,
                                       length=self.Sk, lengths=self.ints(self.len_arg), counts=self.ints(self.count_arg), **kw)
        pasa().check_device_error()
        return got

    def reference(self, scale=None):
        return reference(self.q, *self.nodes, *self.held, self.lengths, self.parents, self.counts, scale or self.scale, self.zero_shift)


CASES = [
    # B, Hq, Hkv, n, Sk, cap, D, lengths, counts, kind
    (1, 1, 1, 1, 1, 1, 128, None, None, "tree"),
    (1, 1, 1, 1, 0, 5, 64, None, None, "tree"),                       # an empty cache
    (1, 28, 4, 8, 300, 301, 128, None, None, "tree"),
    (2, 8, 1, 16, 128, 128, 128, None, None, "chain"),                # 128 rows, a whole block
    (2, 8, 1, 16, 129, 131, 64, None, None, "odd"),
    (3, 14, 2, 9, 1000, 1003, 128, [1000, 0, 385], [9, 9, 0], "tree"),
    (3, 14, 2, 9, 1000, 1003, 64, [1000, 0, 1], [0, 1, 4], "roots"),
    (4, 16, 2, 61, 700, 700, 64, [700, 128, 127, 640], [61, 1, 33, 0], "tree"),   # several tiles of rows
    (2, 4, 4, 128, 260, 260, 128, None, [128, 127], "tree"),          # the most nodes
    (1, 2, 1, 128, 257, 260, 128, None, None, "chain"),
    (1, 40, 1, 31, 500, 500, 64, None, None, "odd"),                  # 1240 rows
    (2, 7, 1, 5, 9001, 9001, 128, [9001, 4096], None, "tree"),        # shared by many CTAs
    (5, 10, 2, 3, 5000, 5001, 64, [5000, 0, 2500, 128, 6000], [3, 3, 9, -2, 2], "tree"),
    (70, 2, 1, 4, 300, 300, 128, [(37 * i) % 301 for i in range(70)], [i % 6 for i in range(70)], "tree"),   # more segments than CTAs
    (300, 1, 1, 2, 10, 10, 64, [i % 11 for i in range(300)], [i % 3 for i in range(300)], "tree"),
    (2, 2, 2, 4, 300, 300, 128, [0, 0], [0, 0], "tree"),              # nothing at all
]


@pytest.mark.parametrize("shifted", [True, False], ids=["", "plain"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_parity(case, shifted):
    *sizes, lengths, counts, kind = CASES[case]
    c = Case(600 + case, *sizes, lengths, counts, kind, shifted)
    got = c.run()
    check(got, c.reference())
    again = c.run()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    if case < 6:
        check(c.run(scale=0.3), c.reference(0.3))


MANY = [
    # more segments than CTAs share, of which some end in the CTA where they began: B, Hq, Hkv, n, Sk, D, lengths, counts
    (90, 4, 2, 3, 900, 128, [(97 * i) % 901 for i in range(90)], [i % 4 for i in range(90)]),
    (90, 4, 2, 3, 900, 64, None, None),
    (160, 2, 1, 2, 800, 64, [800 if i % 40 == 7 else i % 3 for i in range(160)], [2 * (i % 40 == 7) for i in range(160)]),
    (200, 1, 1, 1, 1000, 128, [1000] * 200, [int(i == 131) for i in range(200)]),      # fewer items than CTAs
    (20, 18, 2, 61, 700, 64, [(311 * i) % 701 for i in range(20)], [61 - 3 * i for i in range(20)]),   # tiles of rows
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_more_segments_than_ctas(case):
    B, Hq, H, n, Sk, D, lengths, counts = MANY[case]
    c = Case(660 + case, B, Hq, H, n, Sk, Sk + 1, D, lengths, counts)
    size = pasa().tree_kv4_workspace_bytes(B, Hq, H, n, Sk, D)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    got = c.run(workspace=ws)
    check(got, c.reference())
    again = c.run(workspace=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1]) and (ws[size:] == 0xFF).all()


def test_a_chain_equals_the_causal_decode_on_a_cache_that_holds_it():
    """Against the library's own decode on the 4-bit cache, with nodes that the cache holds exactly."""
    c = Case(700, 2, 8, 2, 5, 600, 700, 128, None, None, "chain", False)
    nodes = [torch.randint(-7, 8, c.dev[i].shape, device="cuda").half() for i in (1, 2)]
    for x in nodes:
        x[..., ::32] = 7
    got = pasa().attn_fwd_tree_kv4(c.dev[0], *nodes, *c.cache, length=600)
    pasa().kv4_append(*nodes, *c.cache, start=600)
    want = pasa().attn_fwd_decode_kv4(c.dev[0], *c.cache, causal=True, length=605)
    # both are within the bounds of the exact result: P in fp16 and the output's rounding, on values of at most 7
    assert (got[0].float() - want[0].float()).abs().max() <= 2 * 7 * 2.0 ** -10
    assert (got[1] - want[1]).abs().max() <= 2.0 ** -10


def test_large_growing_scores():
    """Scores that grow along the cache (the blocks are read from the last one on, so these shrink) and ones that shrink."""
    for seed, sign in ((1, 1), (2, -1)):
        c = Case(710 + seed, 1, 4, 1, 8, 1500, 1500, 128, None, None, "tree", False)
        k = (sign * np.arange(1500)[:, None] / 100 + np.random.default_rng(seed).standard_normal((1, 1, 1500, 128)) * 0.1).astype(np.float16)
        v = rows(np.random.default_rng(seed), 1, 1, 1500, 128, "plain")
        pasa().kv4_append(*to_dev(k, v), *c.cache)
        c.held = kv4.values(*kv4.quantise(k)), kv4.values(*kv4.quantise(v))
        c.q = np.abs(c.q)
        c.dev[0] = to_dev(c.q)[0]
        check(c.run(), c.reference())


@pytest.mark.parametrize("D", [64, 128])
def test_values_of_every_size(D):
    """Cached rows up to fp16's largest values (scales past 2729, where a code is expanded in two steps), down to subnormal
    scales, and rows of zeros."""
    c = Case(720 + D, 2, 4, 2, 5, 700, 700, D, None, None, "tree", False)
    rng = np.random.default_rng(D)
    size = 2.0 ** rng.integers(-24, 16, (2, 2, 700, D // 32)).repeat(32, -1)
    k = np.clip(rng.standard_normal((2, 2, 700, D)) * size, -65504, 65504)
    v = np.clip(rng.standard_normal((2, 2, 700, D)) * size[:, :, ::-1], -60000, 60000)
    k[:, :, ::50], v[:, :, 7::50] = 0, 0
    k, v = k.astype(np.float16), v.astype(np.float16)
    c.q = (c.q * 2.0 ** -12).astype(np.float16)      # scores of some tens
    c.dev[0] = to_dev(c.q)[0]
    pasa().kv4_append(*to_dev(k, v), *c.cache)
    c.held = kv4.values(*kv4.quantise(k)), kv4.values(*kv4.quantise(v))
    assert (kv4.quantise(k)[1] > 2729).any() and (kv4.quantise(v)[1] > 2729).any()
    check(c.run(), c.reference())


def test_offsets_past_32_bits():
    """The last head's rows lie behind 2^32 bytes of codes."""
    B, H, cap, D, n = 2, 1, 36_000_000, 128, 4
    c = Case(720, B, 3, H, n, 400, 400, D, None, None, "tree")
    big = new_cache(B, H, cap, D)
    for x, y in zip(big, c.cache):
        x[:, :, :400] = y
    got = pasa().attn_fwd_tree_kv4(*c.dev[:3], *big, c.dev[3], shift=c.shift, length=400)
    check(got, c.reference())


def test_captured_steps_follow_lengths_and_counts_and_share_a_workspace():
    c = Case(730, 3, 8, 2, 7, 900, 900, 128, [900, 900, 900], [7, 7, 7])
    lengths, counts = c.ints([900] * 3), c.ints([7] * 3)
    ws = torch.empty(pasa().tree_kv4_workspace_bytes(3, 8, 2, 7, 900, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.dev[0]), torch.empty((3, 8, 7), device="cuda")
    q, k, v, parents = to_dev(c.q, c.kn, c.vn, c.parents)

    def call():
        pasa().attn_fwd_tree_kv4(q, k, v, *c.cache, parents, shift=c.shift, lengths=lengths, counts=counts, out=out, lse=lse, workspace=ws)

    call()
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        call()
    with torch.cuda.graph(two):
        call()
        call()
    for n, m in (([900, 1, 0], [7, 7, 7]), ([128, 800, 129], [0, 5, 1]), ([0, 0, 0], [0, 0, 0])):
        lengths.copy_(torch.tensor(n)), counts.copy_(torch.tensor(m))
        c.lengths, c.counts = np.array(n), np.array(m)
        out.fill_(7), lse.fill_(7)
        one.replay()
        two.replay()
        one.replay()
        check((out, lse), c.reference())
    pasa().check_device_error()


def test_two_threads_on_two_streams():
    c = Case(740, 2, 8, 2, 9, 3000, 3000, 64)
    want = c.run()
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(20):
                got[i] = c.run()
        st.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_a_serving_loop_of_drafts():
    """The operators in a row, as a program makes them: a packed prompt with rotary positions into the cache, then steps in which
    drafted tokens are turned to their positions, looked at, and the accepted ones stored."""
    p = pasa()
    rng = np.random.default_rng(750)
    B, Hq, H, D, n, cap = 3, 8, 2, 128, 6, 400
    lens = [150, 3, 77]
    T = sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    f, _ = p.rope_frequencies(D)
    qkv = to_dev(rng.standard_normal((T, Hq + 2 * H, D)).astype(np.float16))[0]
    pos = torch.cat([torch.arange(x) for x in lens]).int().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    p.rope(q, k, f, positions=pos, out_q=q, out_k=k)
    o, _ = p.attn_fwd_packed(q, k, v, cu, mode=1)
    assert o.isfinite().all()
    cache, shift = new_cache(B, H, cap, D), torch.stack([k[cu[b]] for b in range(B)])
    padded = [torch.zeros((B, H, max(lens), D), dtype=torch.float16, device="cuda") for _ in range(2)]
    for b, m in enumerate(lens):
        for x, y in zip(padded, (k, v)):
            x[b, :, :m] = y[cu[b]:cu[b + 1]].transpose(0, 1)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    p.kv4_append(*padded, *cache, counts=lengths, shift=shift)
    held = [x.cpu().numpy().astype(np.float64) for x in p.kv4_read(*cache, cap)]      # without the shift: K' = s c
    sh = shift.cpu().numpy().astype(np.float64)
    for step in range(3):
        parents = tree(rng, B, n, "tree")
        depth = np.array([[len(path(parents[b], i)) - 1 for i in range(n)] for b in range(B)], np.int32)
        counts = np.array([n, n - step, 1], np.int32)
        dq, dk, dv = (rng.standard_normal((B, x, n, D)).astype(np.float16) for x in (Hq, H, H))
        tq, tk, tv, tp, tc = to_dev(dq, dk, dv, parents, counts)
        at = lengths[:, None] + to_dev(depth)[0]
        p.rope(tq, tk, f, positions=at, out_q=tq, out_k=tk)
        got = p.attn_fwd_tree_kv4(tq, tk, tv, *cache, tp, lengths=lengths, counts=tc, shift=shift)
        qn, kn, vn = (x.cpu().numpy() for x in (tq, tk, tv))
        check(got, reference(qn, kn.astype(np.float64), vn.astype(np.float64), *held, lengths.cpu().numpy(), parents, counts, D ** -0.5, sh))
        # the longest path of each tree is accepted
        best = [max((path(parents[b], i)[::-1] for i in range(counts[b])), key=len) for b in range(B)]
        accepted = np.array([len(x) for x in best], np.int32)
        pick = np.full((B, n), -1, np.int32)
        for b in range(B):
            pick[b, :accepted[b]] = best[b]
        tr, ta = to_dev(pick, accepted)
        p.kv4_append(tk, tv, *cache, start=lengths, counts=ta, rows=tr, shift=shift)
        new = kv4.values(*kv4.quantise(kn, shift.cpu().numpy())), kv4.values(*kv4.quantise(vn))
        old = lengths.cpu().numpy()
        for b in range(B):
            for x, y in zip(held, new):
                x[b, :, old[b]:old[b] + accepted[b]] = y[b][:, best[b]]
        lengths += ta
    now = p.kv4_read(*cache, cap)
    for x, y in zip(held, now):
        assert np.array_equal(x, y.cpu().numpy().astype(np.float64))
    p.check_device_error()


def test_binding_refusals():
    p = pasa()
    c = Case(760, 2, 4, 2, 5, 100, 100, 64)
    q, k, v, parents = c.dev
    for bad in ((q.float(), k, v), (q, k.cpu(), v), (q, k, v.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(TypeError):
            p.attn_fwd_tree_kv4(*bad, *c.cache)
    for bad in ((q, k[:, :, :4].contiguous(), v), (q[0], k, v), (q, k[:1].contiguous(), v)):
        with pytest.raises(ValueError):
            p.attn_fwd_tree_kv4(*bad, *c.cache)
    for kw in ({"parents": parents.long()}, {"counts": torch.zeros(2, device="cuda")}, {"lengths": torch.zeros(2, device="cuda")},
               {"out": q.float()}, {"workspace": torch.zeros(4, device="cuda")}):
        with pytest.raises(TypeError):
            p.attn_fwd_tree_kv4(q, k, v, *c.cache, **kw)
    for kw in ({"out": q}, {"length": 101}, {"length": -1}):
        with pytest.raises(p.PasaError):
            p.attn_fwd_tree_kv4(q, k, v, *c.cache, **kw)
    wide = [torch.zeros((2, h, 129, 64), dtype=torch.float16, device="cuda") for h in (4, 2, 2)]
    with pytest.raises(p.PasaError):
        p.attn_fwd_tree_kv4(*wide, *c.cache)


@pytest.mark.parametrize("Sk", [512, 1280])
@pytest.mark.parametrize("D", [64, 128])
def test_maximum_moves_at_every_32_keys(D, Sk):
    """A block is taken 32 keys at a time, and what is stored of its first keys is scaled when a later key raises the maximum by
    more than 8 (log2 units). Here each 32 keys do so, in every block and in the order in which the kernel takes them."""
    c = Case(770 + D, 1, 4, 1, 8, Sk, Sk, D, None, None, "tree", False)
    i = np.arange(Sk)
    step = (Sk // 128 - 1 - i // 128) * 4 + i % 128 // 32
    k = np.broadcast_to((step * (1.8 if D == 64 else 1.3))[:, None], (1, 1, Sk, D)).astype(np.float16)
    v = rows(np.random.default_rng(D), 1, 1, Sk, D, "plain")
    pasa().kv4_append(*to_dev(k, v), *c.cache)
    c.held = kv4.values(*kv4.quantise(k)), kv4.values(*kv4.quantise(v))
    c.q = np.abs(c.q)
    c.dev[0] = to_dev(c.q)[0]
    x = c.scale * np.einsum("bhid,bgjd->hij", c.q.astype(np.float64), c.held[0])
    top = np.stack([x[..., step == e].max(-1) for e in range(Sk // 32)])
    assert (np.diff(top, axis=0) > 8.1 * np.log(2)).all()
    check(c.run(), c.reference())


@pytest.mark.parametrize("below", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_probabilities_are_rounded_once(D, below):
    """One score holds the maximum and all others of a block are equal, so that whatever scales the block's probabilities scales
    the whole output. below = 0: the block's maximum is less than the node's, so that its probabilities are scaled to that. below = 1: a
    key behind the first 32 raises the maximum by more than 8 (log2 units).

    The probabilities' errors, of reference()'s bounds: once to fp16 (2^-11 or, where they are subnormal, 2^-25), and 2^-25 for each
    scaling that leaves them subnormal, which later ones at least halve: less than 2^-24 in all, against a sum of at
    least 1. Scaling itself is by powers of two."""
    H, g = 14, 128
    c = Case(780 + D, 1, H * g, H, 1, 128, 128, D, None, None, "tree", False)
    rng = np.random.default_rng(780 + below)
    k = np.zeros((1, H, 128, D))
    k[..., 1] = 7                                                  # every row's scale is 1; channel 1 of q is 0
    code = np.arange(H) - 7.0
    k[0, :, :, 0] = code[:, None]
    k[0, :, 0 if below == 0 else 100, 0] = 7
    node = rng.uniform(7.5, 11, H) if below == 0 else code - 40
    weight = rng.uniform(0.05, 0.6, (H, g)) if below == 0 else 8.1 * np.log(2) / (7 - code)[:, None] * rng.uniform(1, 1.5, (H, g))
    v = np.repeat(rng.uniform(0.5, 1, (1, 1, 1, D // 32)), 32, -1) * np.ones((1, H, 128, D))
    if below == 1:
        v[:, :, 100] = 0
    c.q = np.zeros((1, H * g, 1, D), np.float16)
    c.q[0, :, 0, 0] = weight.reshape(-1)
    c.kn, c.vn = np.zeros((1, H, 1, D), np.float16), np.zeros((1, H, 1, D), np.float16)
    c.kn[0, :, 0, 0] = node
    k, v = k.astype(np.float16), v.astype(np.float16)
    pasa().kv4_append(*to_dev(k, v), *c.cache)
    c.held, c.nodes = (kv4.values(*kv4.quantise(k)), kv4.values(*kv4.quantise(v))), (c.kn.astype(np.float64), c.vn.astype(np.float64))
    assert np.array_equal(c.held[0], k)
    c.dev[:3] = to_dev(c.q, c.kn, c.vn)
    o, lse, bo, bl = c.reference(1.0)
    bo = bo + (np.abs(c.held[1]).sum(2)[:, :, None] * 2.0 ** -25).repeat(g, 1)
    check(c.run(scale=1.0), (o, lse, bo, bl))


@pytest.mark.parametrize("B,n,Sk,D", [(2, 5, 300, 128), (2, 5, 9000, 64), (2, 5, 9000, 128), (80, 3, 900, 64)])
def test_a_nan_query_stays_in_its_row(B, n, Sk, D):
    """As in the decode on this cache: an output and an LSE of NaN, not those of a row without keys, and the other rows as they were.
    A CTA to a segment, segments that CTAs share, and more segments than CTAs."""
    c = Case(790, B, 4, 2, n, Sk, Sk, D)
    want, lse = c.run()
    assert want.isfinite().all() and lse.isfinite().all()
    bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    bad[B - 1, 3, 0] = bad[0, 0, n - 1] = True
    c.dev[0] = c.dev[0].clone()
    c.dev[0][B - 1, 3, 0, 5] = c.dev[0][0, 0, n - 1, D - 1] = float("nan")
    o, other = c.run()
    assert o[bad].isnan().all() and other[bad].isnan().all()
    assert torch.equal(o[~bad], want[~bad]) and torch.equal(other[~bad], lse[~bad])
