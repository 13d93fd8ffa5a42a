"""GPU parity of attention over packed sequences against the definition in 64 bits, sequence by sequence.

The keys of the shifted modes are the oracle's K' + m (exact integer arithmetic on each sequence alone,
oracle/pseudo_average.py), so the rounding of K' is part of the reference and a block that is not counted
from its sequence's first key shows.

Bounds (bounds()). ds, a score's absolute error in natural-log units: the fp32 sum of D products errs by at most D 2^-22
of the sum of their magnitudes (each of D / 16 MMA steps adds 17 terms cut at 2^-23 of the largest), likewise the offset
q . m; scaling, the difference from the running maximum and ex2.approx add 2^-20 of the score and 2^-18. fp16
scores: D / 16 roundings of at most 2^-11 of the sum of magnitudes, and 2^-24 where they are subnormal.
o: each p moves by a factor within e^(2 dsum) (its own error and the sum's, dsum with the fp32 sum's n 2^-23),
P is rounded to fp16 (2^-11, or 2^-25 absolute against a sum of at least 1), PV's fp32 sum of n terms errs by n 2^-22,
the output is rounded (2^-11, or 2^-25).
"""
import math
import threading

import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from oracle import pseudo_average as pa

pytestmark = pytest.mark.gpu


def pasa():
    import precision_flashattention_numerics_gb300 as p

    return p


def cu(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def make(seed, lens_q, lens_k, Hq, Hkv, D, bias=True, front=0, tail=3):
    rng = np.random.default_rng(seed)
    Tq, Tk = front + sum(lens_q) + tail, front + sum(lens_k) + tail
    q = rng.standard_normal((Tq, Hq, D)).astype(np.float16)
    k = rng.standard_normal((Tk, Hkv, D)) + (10 * rng.standard_normal((1, Hkv, D)) if bias else 0)
    v = rng.standard_normal((Tk, Hkv, D)).astype(np.float16)
    return q, k.astype(np.float16), v, cu(lens_q, front), cu(lens_k, front)


def reference(q, k, v, causal, mode, scale):
    """o, lse and bounds on their errors of one sequence: q [n, Hq, D], k and v [m, Hkv, D]."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.full((Hq, n), -np.inf), np.zeros((Hq, n))
    if m == 0:
        return o, lse, bo, bl
    shift = mode in (0, 1)
    if shift:
        ks, means = pa.kshift_fast(np.ascontiguousarray(k.transpose(1, 0, 2))[None])
        ks, ms = ks[0].astype(np.float64), np.repeat(means[0].astype(np.float64), 128, axis=1)[:, :m]
    else:
        ks, ms = k.transpose(1, 0, 2).astype(np.float64), np.zeros((Hkv, m, D))
    see = np.arange(m) <= np.arange(n)[:, None] + m - n if causal else np.ones((n, m), bool)
    some = see.any(1)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        qh, vh = q[:, h].astype(np.float64), v[:, g].astype(np.float64)
        x = np.where(see, scale * (qh @ (ks[g] + ms[g]).T), -np.inf)
        top = np.where(some, x.max(1), 0.0)
        p = np.exp(x - top[:, None])
        total = np.where(some, p.sum(1), 1.0)
        lse[h] = np.where(some, top + np.log(total), -np.inf)
        p /= total[:, None]
        o[:, h] = p @ vh
        mag_k = scale * np.where(see, np.abs(qh) @ np.abs(ks[g]).T, 0).max(1)
        mag = mag_k + scale * np.where(see, np.abs(qh) @ np.abs(ms[g]).T, 0).max(1)
        ds = mag * (D * 2.0 ** -22 + 2.0 ** -20) + 2.0 ** -18
        if mode in (0, 2):
            ds = ds + (D // 16) * (mag_k * 2.0 ** -11 + scale * 2.0 ** -24)
        count = see.sum(1)
        dsum = ds + (count + 2) * 2.0 ** -23
        bl[h] = dsum + np.abs(np.where(some, lse[h], 0)) * 2.0 ** -21 + 2.0 ** -20
        bo[:, h] = ((p @ np.abs(vh)) * (2.0 ** -11 + np.expm1(2 * dsum) + count * 2.0 ** -22)[:, None]
                    + (see @ np.abs(vh)) * 2.0 ** -25 + np.abs(o[:, h]) * 2.0 ** -11 + 2.0 ** -25)
    return o, lse, bo, bl


def check(o, lse, q, k, v, cq, ck, causal, mode, scale=None):
    scale = scale or 1 / math.sqrt(q.shape[2])
    o, lse = o.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    inside = np.zeros(len(q), bool)
    for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
        inside[a:b] = True
        if a == b:
            continue
        ro, rl, bo, bl = reference(q[a:b], k[c:d], v[c:d], causal, mode, scale)
        off = np.abs(o[a:b] - ro)
        assert (off <= bo).all(), (a, b, float(np.nanmax(off / np.maximum(bo, 1e-300))), np.isnan(off).any())
        fin = np.isfinite(rl)
        assert np.array_equal(np.isneginf(lse[:, a:b]), ~fin)
        off = np.abs(lse[:, a:b][fin] - rl[fin])
        assert (off <= bl[fin]).all(), (a, b, float((off / bl[fin]).max()))
    return inside


def run(q, k, v, cq, ck, **kw):
    qt, kt, vt, a, b = to_dev(q, k, v, cq, ck)
    out = torch.full_like(qt, 7)
    lse = torch.full((q.shape[1], len(q)), 7.0, device="cuda")
    pasa().attn_fwd_packed(qt, kt, vt, a, b, out=out, lse=lse, **kw)
    pasa().check_device_error()
    return out, lse


CASES = [
    # lens_q, lens_k (None: the same), Hq, Hkv, D, causal
    ([1], None, 1, 1, 128, True),
    ([1], None, 28, 4, 64, True),
    ([128], None, 2, 2, 128, True),
    ([129, 127, 1, 256], None, 2, 1, 128, True),
    ([300, 0, 5, 77], None, 7, 1, 128, True),
    ([300, 0, 5, 77], None, 10, 2, 64, False),
    ([3, 1, 0, 0, 2, 18, 19, 17], None, 14, 2, 128, True),
    ([33, 200, 64], None, 12, 4, 64, True),
    ([40, 1, 9], [300, 257, 0], 16, 2, 128, True),            # chunks of prompts; queries without keys
    ([40, 1, 9, 130], [300, 257, 5, 131], 16, 1, 64, True),   # more queries than keys: the first see none
    ([50, 20], [1, 700], 5, 5, 128, False),
    ([130] * 5, None, 6, 2, 128, True),
    ([21, 100], None, 40, 1, 64, True),                       # 40 heads to a kv head
    ([5, 300], None, 130, 1, 128, True),                      # more heads than a tile has rows
    ([2500], None, 1, 1, 128, True),                          # more than one chunk of offsets
    ([1, 1, 1], [2500, 2049, 2048], 4, 2, 64, True),          # single tokens on long keys
]


@pytest.mark.parametrize("mode", [0, 1, 2, 3])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_parity(case, mode):
    lens_q, lens_k, Hq, Hkv, D, causal = CASES[case]
    q, k, v, cq, ck = make(400 + case, lens_q, lens_k or lens_q, Hq, Hkv, D, bias=mode != 2, front=case % 3 * 2)
    out, lse = run(q, k, v, cq, ck, causal=causal, mode=mode)
    inside = check(out, lse, q, k, v, cq, ck, causal, mode)
    assert (out[~torch.from_numpy(inside)] == 7).all() and (lse[:, ~torch.from_numpy(inside)] == 7).all()
    if case < 4:
        out, lse = run(q, k, v, cq, ck, causal=causal, mode=mode, scale=0.2)
        check(out, lse, q, k, v, cq, ck, causal, mode, 0.2)


LONG = [
    # tiles whose key blocks several CTAs share
    ([64], [6000], 4, 1, 128, True),
    ([64], [6001], 8, 2, 64, True),
    ([1], [20000], 1, 1, 128, True),                          # one tile
    ([1], [9000], 7, 1, 64, True),
    ([4000], None, 1, 1, 64, True),                           # the long tiles of a prompt
    ([3100], None, 2, 1, 128, True),
    ([300, 0, 5, 20], [5000, 7, 2100, 20], 14, 2, 128, True), # divided and whole tiles
    ([100, 1], [4099, 2049], 5, 5, 64, False),
    ([2500], [2200], 1, 1, 128, True),                        # the first 300 see nothing, and few the last pieces
    ([130, 7], [2048, 2176], 130, 1, 128, True),
]


@pytest.mark.parametrize("mode", [0, 1, 2, 3])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_shared_keys(case, mode):
    lens_q, lens_k, Hq, Hkv, D, causal = LONG[case]
    q, k, v, cq, ck = make(500 + case, lens_q, lens_k or lens_q, Hq, Hkv, D, bias=mode != 2, front=case % 3 * 2)
    out, lse = run(q, k, v, cq, ck, causal=causal, mode=mode)
    inside = check(out, lse, q, k, v, cq, ck, causal, mode)
    assert (out[~torch.from_numpy(inside)] == 7).all() and (lse[:, ~torch.from_numpy(inside)] == 7).all()


@pytest.mark.parametrize("D", [64, 128])
def test_shared_keys_among_others(D):
    """Queries of which the first pieces hold nothing that weighs, neighbours of NaN, strided views, in place of q, and no
    result that changes from call to call."""
    q, k, v, cq, ck = make(520 + D, [50, 40], [700, 3500], 4, 2, D, bias=False, front=9, tail=9)
    k[ck[1] + 3000:ck[2]] *= 4                                # the maximum moves up in the last piece
    want, lse = run(q, k, v, cq, ck, mode=1)
    check(want, lse, q, k, v, cq, ck, True, 1)
    foul = [x.copy() for x in (q, k, v)]
    for x, c in zip(foul, (cq, ck, ck)):
        x[:c[0]], x[c[2]:] = np.nan, np.inf
    T = max(len(q), len(k))
    fused = torch.full((T, 8, D), float("nan"), dtype=torch.float16, device="cuda")
    qt, kt, vt, a, b = to_dev(*foul, cq, ck)
    fused[:len(q), :4], fused[:len(k), 4:6], fused[:len(k), 6:] = qt, kt, vt
    views = fused[:len(q), :4], fused[:len(k), 4:6], fused[:len(k), 6:]
    ws = torch.full((pasa().packed_workspace_bytes(2, 4, 2, len(q), len(k), D, 1) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for i in range(3):
        out, other = torch.full_like(want, 7), torch.full_like(lse, 7)
        pasa().attn_fwd_packed(*views, a, b, mode=1, out=out, lse=other, workspace=ws)
        assert torch.equal(out, want) and torch.equal(other, lse)
    assert (ws[-256:] == 0xFF).all()
    pasa().attn_fwd_packed(*views, a, b, mode=1, out=views[0], return_lse=False)
    inside = slice(int(cq[0]), int(cq[-1]))
    assert torch.equal(fused[inside, :4], want[inside]) and fused[:9, :4].isnan().all()


def test_captured_call_divides_by_the_lengths():
    """One graph: keys that are shared among CTAs, then lengths that need none of it, and none at all."""
    q, k, v, _, _ = make(530, [200], [5000], 4, 1, 128, tail=0)
    qt, kt, vt = to_dev(q, k, v)
    a, b = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(qt), torch.zeros((4, 200), device="cuda")
    ws = torch.empty(pasa().packed_workspace_bytes(3, 4, 1, 200, 5000, 128, 1), dtype=torch.uint8, device="cuda")
    call = lambda: pasa().attn_fwd_packed(qt, kt, vt, a, b, out=out, lse=lse, workspace=ws, mode=1)   # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for lens_q, lens_k in (([0, 70, 1], [9, 4800, 130]), ([200, 0, 0], [200, 0, 0]), ([0] * 3, [0] * 3), ([1, 1, 1], [2000, 900, 2100])):
        cq, ck = cu(lens_q), cu(lens_k)
        a.copy_(torch.from_numpy(cq)), b.copy_(torch.from_numpy(ck))
        out.fill_(7), lse.fill_(7)
        graph.replay()
        inside = check(out, lse, q, k, v, cq, ck, True, 1)
        assert (out[~torch.from_numpy(inside)] == 7).all()
    pasa().check_device_error()


@pytest.mark.parametrize("mode", [0, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_a_sequence_does_not_depend_on_its_batch(D, mode):
    """Bit for bit what the sequence gives alone, among sequences that hold NaN and infinities, in views of a fused
    projection, and in place of q."""
    lens_q, lens_k = [70, 18, 0, 333, 1, 128, 45], [70, 400, 9, 333, 129, 128, 45]
    q, k, v, cq, ck = make(7, lens_q, lens_k, 14, 2, D, front=1)
    want, lse = run(q, k, v, cq, ck, mode=mode)
    for s, (n, m) in enumerate(zip(lens_q, lens_k)):
        if n == 0:
            continue
        a, c = cq[s], ck[s]
        one, one_lse = run(q[a:a + n], k[c:c + m], v[c:c + m], cu([n]), cu([m]), mode=mode)
        assert torch.equal(one, want[a:a + n]) and torch.equal(one_lse, lse[:, a:a + n])
        foul = [x.copy() for x in (q, k, v)]
        for x, lo, hi in zip(foul, (a, c, c), (a + n, c + m, c + m)):
            x[:lo], x[hi:] = np.nan, np.inf
        other, other_lse = run(*foul, cq, ck, mode=mode)
        assert torch.equal(other[a:a + n], want[a:a + n]) and torch.equal(other_lse[:, a:a + n], lse[:, a:a + n])
    T = max(len(q), len(k))
    fused = torch.full((T, 18, D), float("nan"), dtype=torch.float16, device="cuda")
    qt, kt, vt, a, b = to_dev(q, k, v, cq, ck)
    fused[:len(q), :14], fused[:len(k), 14:16], fused[:len(k), 16:] = qt, kt, vt
    views = fused[:len(q), :14], fused[:len(k), 14:16], fused[:len(k), 16:]
    held = fused.clone()
    out = torch.full((len(q), 15, D), 7.0, dtype=torch.float16, device="cuda")
    pasa().attn_fwd_packed(*views, a, b, mode=mode, out=out[:, 1:], lse=torch.empty_like(lse))
    inside = slice(int(cq[0]), int(cq[-1]))
    assert torch.equal(out[inside, 1:], want[inside]) and (out[:, 0] == 7).all() and torch.equal(fused.nan_to_num(), held.nan_to_num())
    o, none = pasa().attn_fwd_packed(*views, a, b, mode=mode, out=views[0], return_lse=False)
    assert none is None and torch.equal(fused[inside, :14], want[inside])
    held[inside, :14] = want[inside]
    assert torch.equal(fused.nan_to_num(), held.nan_to_num())


def test_one_sequence_equals_the_dense_call():
    q, k, v, cq, ck = make(8, [777], [777], 8, 2, 128, tail=0)
    qt, kt, vt = to_dev(*(np.ascontiguousarray(x.transpose(1, 0, 2))[None] for x in (q, k, v)))
    for mode in range(4):
        o, lse = run(q, k, v, cq, ck, mode=mode)
        dense, dense_lse = pasa().attn_fwd(qt, kt, vt, causal=True, mode=mode)
        assert torch.equal(o.nan_to_num(), dense[0].transpose(0, 1).nan_to_num()) and torch.equal(lse.nan_to_num(), dense_lse[0].nan_to_num())


def test_many_sequences():
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 9, 3000).tolist()
    q, k, v, cq, ck = make(9, lens, lens, 4, 2, 64)
    out, lse = run(q, k, v, cq, ck, mode=1)
    check(out, lse, q, k, v, cq, ck, True, 1)


def test_large_growing_scores():
    """Scores that grow along the keys, so that the running maximum moves at every block and the output is rescaled."""
    q, k, v, cq, ck = make(10, [600, 300], [600, 900], 4, 1, 128, bias=False)
    q = np.abs(q)
    k = (np.arange(len(k))[:, None, None] / 300 + 0.1 * k.astype(np.float64)).astype(np.float16)
    for mode in (0, 1, 3):
        out, lse = run(q, k, v, cq, ck, mode=mode)
        check(out, lse, q, k, v, cq, ck, True, mode)


def test_offsets_past_32_bits():
    """The sequences lie behind 2^31 elements of rows that belong to none."""
    Hq, Hkv, D = 32, 1, 128
    front = 2 ** 31 // (Hq * D) + 100
    q, k, v, cq, ck = make(11, [200, 77], [200, 77], Hq, Hkv, D, tail=0)
    big = torch.empty((front + len(q), Hq, D), dtype=torch.float16, device="cuda")
    out = torch.empty_like(big)
    out[:front] = 7
    big[front:] = to_dev(q)[0]
    kt, vt, a, b = to_dev(k, v, cq + front, ck)
    _, lse = pasa().attn_fwd_packed(big, kt, vt, a.int(), b, out=out, mode=1)
    check(out[front:], lse[:, front:], q, k, v, cq, ck, True, 1)
    assert bool((out[:front] == 7).all())


def test_offsets_that_do_not_grow_stay_inside():
    """Unspecified results, but nothing outside the tensors is written: guard rows on both sides stay."""
    q, k, v, _, _ = make(12, [300], [300], 4, 2, 64, tail=0)
    qt, kt, vt = to_dev(q, k, v)
    for bad in ([0, 200, 100, 300], [-5, 400, 7, 1000], [300, 200, 100, 0], [0, 2 ** 31 - 1, -2 ** 31, 300], [299, 299, 299, 299]):
        c = torch.tensor(bad, dtype=torch.int32, device="cuda")
        room = torch.full((500, 4, 64), 7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((6, 300), 7.0, device="cuda")
        pasa().attn_fwd_packed(qt, kt, vt, c, mode=1, out=room[100:400], lse=lse[1:5])
        pasa().check_device_error()
        assert (room[:100] == 7).all() and (room[400:] == 7).all() and (lse[0] == 7).all() and (lse[5] == 7).all()


def test_captured_call_follows_the_lengths():
    q, k, v, _, _ = make(13, [500], [700], 8, 2, 128, tail=0)
    qt, kt, vt = to_dev(q, k, v)
    a, b = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    ws = torch.empty(pasa().packed_workspace_bytes(4, 8, 2, 500, 700, 128, 0), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(qt), torch.zeros((8, 500), device="cuda")
    call = lambda: pasa().attn_fwd_packed(qt, kt, vt, a, b, out=out, lse=lse, workspace=ws)   # noqa: E731
    call()
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    with torch.cuda.graph(second):   # another graph on the same workspace
        call()
        call()
    for lens_q, lens_k in (([500, 0, 0, 0], [700, 0, 0, 0]), ([1, 2, 300, 7], [300, 2, 301, 90]), ([0] * 4, [5] * 4)):
        cq, ck = cu(lens_q), cu(lens_k)
        a.copy_(torch.from_numpy(cq)), b.copy_(torch.from_numpy(ck))
        out.fill_(7), lse.fill_(7)
        graph.replay()
        second.replay()
        graph.replay()
        inside = check(out, lse, q, k, v, cq, ck, True, 0)
        assert (out[~torch.from_numpy(inside)] == 7).all()
    pasa().check_device_error()


def test_two_threads_on_two_streams():
    q, k, v, cq, ck = make(14, [300, 40, 128], [300, 40, 128], 8, 2, 64)
    want = run(q, k, v, cq, ck, mode=1)[0]
    got = [None, None]

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            t = to_dev(q, k, v, cq, ck)
            for _ in range(20):
                out = torch.full_like(t[0], 7)
                pasa().attn_fwd_packed(*t, mode=1, out=out)
            got[i] = out
        st.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert torch.equal(got[0], want) and torch.equal(got[1], want)


def test_binding_refusals():
    p = pasa()
    q, k, v, cq, ck = make(15, [30], [30], 4, 2, 64, tail=0)
    qt, kt, vt, a, b = to_dev(q, k, v, cq, ck)
    for args, kw in (((qt.float(), kt, vt, a), {}), ((qt, kt.cpu(), vt, a), {}), ((qt, kt, vt, a.long()), {}), ((qt, kt, vt, a), {"out": qt.float()}),
                     ((qt, kt, vt, a), {"lse": torch.zeros((4, 30), device="cuda").half()})):
        with pytest.raises(TypeError):
            p.attn_fwd_packed(*args, **kw)
    for args, kw in (((qt[None], kt, vt, a), {}), ((qt, kt, vt[:-1], a), {}), ((qt, kt[..., :32], vt[..., :32], a), {}), ((qt, kt, vt, a[:1]), {}),
                     ((qt, kt, vt, a, torch.cat([b, b])), {}), ((qt.transpose(0, 2).contiguous().transpose(0, 2), kt, vt, a), {}),
                     ((qt, kt, vt, a), {"lse": torch.zeros((30, 4), device="cuda")})):
        with pytest.raises(ValueError):
            p.attn_fwd_packed(*args, **kw)
    for args, kw in (((qt, kt, vt, a), {"mode": 4}), ((qt, kt, vt, a), {"out": kt.repeat(1, 2, 1)[:, :1].expand(-1, 4, -1)}),
                     ((torch.cat([qt, qt], 1)[:, 1:5][..., :64], kt, vt, a), {"mode": 7})):
        with pytest.raises(p.PasaError):
            p.attn_fwd_packed(*args, **kw)


@pytest.mark.parametrize("mode", [0, 1, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_up_to_1920_keys_beside_long_ones_nothing_depends_on_the_batch(D, mode):
    """The long sequence's keys are divided among CTAs; those of up to 1920 keys are not, and give bit for bit what they give
    alone. The others stay within their bounds."""
    lens_q, lens_k = [1, 2, 1, 1, 3, 1, 1], [1024, 1025, 1100, 1500, 1920, 1921, 20000]
    q, k, v, cq, ck = make(540 + D, lens_q, lens_k, 28, 4, D, bias=mode != 3)
    want, lse = run(q, k, v, cq, ck, mode=mode)
    check(want, lse, q, k, v, cq, ck, True, mode)
    for s, (n, m) in enumerate(zip(lens_q, lens_k)):
        a, c = cq[s], ck[s]
        if m <= 1920:
            one, one_lse = run(q[a:a + n], k[c:c + m], v[c:c + m], cu([n]), cu([m]), mode=mode)
            assert torch.equal(one, want[a:a + n]) and torch.equal(one_lse, lse[:, a:a + n]), m


@pytest.mark.parametrize("D", [64, 128])
def test_offsets_that_do_not_grow_stay_inside_where_keys_are_divided(D):
    """As test_offsets_that_do_not_grow_stay_inside, with keys enough that tiles come in pieces, offsets of q and k that are bad by
    themselves, and a guard behind the workspace, where the pieces' lists and partial results lie."""
    Tq, Tk, lo, hi = 200, 6000, -2 ** 31, 2 ** 31 - 1
    q, k, v, _, _ = make(550, [Tq], [Tk], 4, 2, D, tail=0)
    qt, kt, vt = to_dev(q, k, v)
    lists_q = [0, 70, 200, 200], [0, 200, 100, 300], [-5, 400, 7, 1000], [200, 150, 100, 0], [0, hi, lo, 200], [199, 199, 199, 199], [lo, hi, lo, hi]
    lists_k = [0, 3000, 5000, 6000], [0, 6000, 2500, 6000], [-5, 9000, 7, 8000], [6000, 4000, 2000, 0], [0, hi, lo, 6000], [lo, hi, lo, hi]
    size = pasa().packed_workspace_bytes(3, 4, 2, Tq, Tk, D, 1)
    for a in lists_q:
        for b in lists_k:
            cq, ck = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (a, b))
            room = torch.full((Tq + 200, 4, D), 7.0, dtype=torch.float16, device="cuda")
            lse = torch.full((6, Tq), 7.0, device="cuda")
            ws = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
            for mode in (1, 3):
                pasa().attn_fwd_packed(qt, kt, vt, cq, ck, mode=mode, out=room[100:100 + Tq], lse=lse[1:5], workspace=ws)
                pasa().check_device_error()
            assert (room[:100] == 7).all() and (room[100 + Tq:] == 7).all() and (lse[0] == 7).all() and (lse[5] == 7).all(), (a, b)
            assert (ws[size:] == 0xFF).all(), (a, b)


@pytest.mark.parametrize("mode", [0, 1, 2, 3])
@pytest.mark.parametrize("lens_q,lens_k", [([70, 40], [70, 300]), ([9, 64], [200, 9000])])
@pytest.mark.parametrize("D", [64, 128])
def test_a_nan_query_stays_in_its_row(D, lens_q, lens_k, mode):
    """An output and an LSE of NaN, not those of a query without keys, and the other rows as they were; with whole tiles, and where
    CTAs share the keys."""
    q, k, v, cq, ck = make(560 + D, lens_q, lens_k, 4, 2, D, bias=False, tail=0)
    want, lse = run(q, k, v, cq, ck, mode=mode)
    assert want.isfinite().all() and lse.isfinite().all()
    bad = torch.zeros(want.shape[:2], dtype=torch.bool, device="cuda")
    for t, h, ch in ((3, 0, 0), (len(q) - 1, 3, D - 1), (lens_q[0], 2, 7)):
        q[t, h, ch] = np.nan
        bad[t, h] = True
    o, other = run(q, k, v, cq, ck, mode=mode)
    assert o[bad].isnan().all() and other.T[bad].isnan().all()
    assert torch.equal(o[~bad], want[~bad]) and torch.equal(other.T[~bad], lse.T[~bad])
