"""GPU parity of the 4-bit key/value cache: storing and reading rows, and decode attention with
the rows' gathered weights, against the exact numpy arithmetic of oracle/kv4.py.

Codes, scales and read-back values are compared bit for bit. Attention is compared with bounds
from the arithmetic (decode_bounds): the cache's values are exact in fp16, so what rounds is
the scores' fp32 sum, the exponential, P in fp16 and the output.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from oracle import kv4

pytestmark = pytest.mark.gpu


def pasa():
    import precision_flashattention_numerics_gb300 as p

    return p


def new_cache(B, H, cap, D, fill=0):
    f16 = torch.float16
    return (torch.full((B, H, cap, D // 2), fill, dtype=torch.uint8, device="cuda"),
            torch.full((B, H, cap, D // 32), fill, dtype=f16, device="cuda"),
            torch.full((B, H, cap, D // 2), fill, dtype=torch.uint8, device="cuda"),
            torch.full((B, H, cap, D // 32), fill, dtype=f16, device="cuda"))


def host(*xs):
    return [x.cpu().numpy() for x in xs]


def rows(rng, B, H, n, D, kind):
    k = rng.standard_normal((B, H, n, D))
    if kind == "bias":
        k = k + 20 * rng.standard_normal((B, H, 1, D))
    elif kind == "wide":      # every magnitude of fp16, subnormals included
        k = k * 2.0 ** rng.uniform(-26, 15, (B, H, n, D // 32)).repeat(32, -1)
    elif kind == "grid":      # small integers and halves: quotients that are ties
        k = rng.integers(-14, 15, (B, H, n, D)) / 2
        k[..., ::32] = 7
    elif kind == "odd":       # not finite, zeros and the largest values among them
        k = k * 100
        k[rng.random(k.shape) < 0.01] = np.nan
        k[rng.random(k.shape) < 0.01] = np.inf
        k[rng.random(k.shape) < 0.01] = -np.inf
        k[rng.random(k.shape) < 0.01] = 65504
        k[:, :, ::3, :32] = 0
    with np.errstate(over="ignore"):
        return k.astype(np.float16)


# ---- storing and reading ----

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,n,shifted", [("bias", 1, True), ("wide", 77, False), ("grid", 130, False), ("odd", 33, True),
                                            ("bias", 1001, True)])
def test_append_and_read_are_exact(kind, n, shifted, D):
    rng = np.random.default_rng(n + D)
    B, H, cap = 3, 2, n + 5
    k, v = rows(rng, B, H, n, D, kind), rows(rng, B, H, n, D, kind)
    shift = k[:, :, 0].copy() if shifted and kind == "bias" else rng.standard_normal((B, H, D)).astype(np.float16)
    kt, vt, st = to_dev(k, v, shift)
    st = st if shifted else None
    cache = new_cache(B, H, cap, D, fill=3)
    pasa().kv4_append(kt, vt, *cache, start=2, shift=st)
    k4, ks, v4, vs = host(*cache)
    ek, es = kv4.quantise(k, shift if shifted else None)
    fk, fs = kv4.quantise(v)
    for got, want in ((k4, ek), (ks, es), (v4, fk), (vs, fs)):
        assert np.array_equal(got[:, :, 2:n + 2], want)
        assert (got[:, :, :2] == 3).all() and (got[:, :, n + 2:] == 3).all()   # the other rows are as they were
    rk, rv = host(*pasa().kv4_read(*cache, n, start=2, shift=st))
    wk = kv4.values(ek, es) + (shift.astype(np.float64)[:, :, None] if shifted else 0.0)
    with np.errstate(over="ignore"):
        assert np.array_equal(rk, wk.astype(np.float16))
    assert np.array_equal(rv.astype(np.float64), kv4.values(fk, fs))


@pytest.mark.parametrize("D", [64, 128])
def test_uneven_starts_and_counts(D):
    """Rows past a sequence's count are neither stored nor read (its padding is NaN), rows outside
    the cache are skipped, and all else stays."""
    rng = np.random.default_rng(7)
    B, H, n, cap = 6, 3, 21, 40
    k, v = rows(rng, B, H, n, D, "bias"), rows(rng, B, H, n, D, "bias")
    starts, counts = [0, 19, 30, -4, 2 ** 31 - 3, 7], [21, 21, 21, 21, 21, 0]
    counts[1] = 5
    k[1, :, 5:] = np.nan
    kt, vt = to_dev(k, v)
    st, ct = torch.tensor(starts).int().cuda(), torch.tensor(counts).int().cuda()
    cache = new_cache(B, H, cap, D, fill=9)
    pasa().kv4_append(kt, vt, *cache, start=st, counts=ct)
    ek, es = kv4.quantise(k)
    k4, ks, _, _ = host(*cache)
    want4, wants = np.full(k4.shape, 9, np.uint8), np.full(ks.shape, 9, np.float16)
    there = [[(i, starts[b] + i) for i in range(counts[b]) if 0 <= starts[b] + i < cap] for b in range(B)]
    for b in range(B):
        for i, r in there[b]:
            want4[b, :, r], wants[b, :, r] = ek[b, :, i], es[b, :, i]
    assert np.array_equal(k4, want4) and np.array_equal(ks, wants)
    ok, ov = torch.full_like(kt, 5), torch.full_like(vt, 5)
    pasa().kv4_read(*cache, n, start=st, counts=ct, out_k=ok, out_v=ov)
    want = np.full(k.shape, 5.0)
    for b in range(B):
        for i, r in there[b]:
            want[b, :, i] = kv4.values(ek, es)[b, :, i]
    assert np.array_equal(ok.cpu().numpy().astype(np.float64), want)
    fresh, _ = pasa().kv4_read(*cache, n, start=st, counts=ct)
    want[want == 5.0] = 0
    assert (fresh[5] == 0).all() and (fresh[4, :, 3:] == 0).all()


# ---- decode ----

def decode_bounds(ref, scale, D, g, Sq, q, shift):
    """Bounds on |o - ref|, |lse - ref| and |weights - ref| (of values starting at 0).

    ds: a score's absolute error. A group of 32 channels is the fp32 sum, in two MMAs, of 32
        products n q (n = code + 8, up to 15) and of -8 sum q: 17 terms at a time, each cut at
        2^-24 of at most 23 sum|q|, together 2 * 17 * 23 2^-24 sum|q| s, and max|k| of a group is
        7 s: at most 56 2^-23 sum|q| max|k|, within D 2^-23 of sabs. Joining the groups, the product
        with scale log2(e) and the difference from the running reference add 2^-21 of
        |x| <= sabs, and 2^-19 numbers within 8 of it and ex2.approx (2^-22 relative).
    o:  each p moves by a factor within e^(2 ds) (its own error and the sum's), P is rounded to
        fp16 (2^-11 relative, or 2^-25 absolute against a sum of at least 1), the sum of n terms
        in fp32 errs by (n / 16 + 2) 2^-23, and the output is rounded (2^-11, or 2^-25)."""
    ds = ref["sabs"] * (D * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -19
    dsum = ds + (ref["n"] + 2) * 2.0 ** -24
    o = (ref["pv"] * (2.0 ** -11 + 2 * dsum[..., None] * 1.01 + ref["n"][..., None] * 2.0 ** -23)
         + ref["vabs"] * 2.0 ** -25 + np.abs(ref["o"]) * 2.0 ** -11 + 2.0 ** -25)
    off = 0.0
    if shift is not None:
        off = scale * np.einsum("bhid,bhd->bhi", np.abs(q.astype(np.float64)),
                                np.repeat(np.abs(shift.astype(np.float64)), g, 1)) * D * 2.0 ** -23
    lse = dsum + off + np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0) * 2.0 ** -21 + 2.0 ** -20
    B, Hq, _ = ref["n"].shape
    worst = (ds + dsum).reshape(B, Hq // g, g * Sq).max(-1)[..., None]
    w = ref["weights"] * (worst * 1.01 + 2.0 ** -20) + 2.0 ** -40
    return o, lse, w


def check(got, ref, bounds, weights=None):
    (o, lse), (bo, bl, bw) = host(*got), bounds
    assert np.isfinite(o).all()
    d = np.abs(o.astype(np.float64) - ref["o"])
    assert (d <= bo).all(), (d / bo).max()
    dead = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), dead) and (o[dead] == 0).all()
    d = np.abs(lse[~dead].astype(np.float64) - ref["lse"][~dead])
    assert (d <= bl[~dead]).all(), (d / bl[~dead]).max()
    if weights is not None:
        d = np.abs(weights.cpu().numpy().astype(np.float64) - ref["weights"])
        assert (d <= bw).all(), (d / bw).max()


DECODE = [
    # B, Hq, Hkv, Sq, Sk, cap, D, causal, lengths (None: Sk), shifted
    (1, 1, 1, 1, 1, 1, 128, True, None, False),
    (2, 8, 1, 1, 300, 300, 128, True, None, True),           # 8 rows, a CTA per head
    (1, 28, 4, 1, 512, 600, 128, True, None, True),          # the longest that a CTA takes whole
    (1, 28, 4, 1, 513, 600, 64, True, None, True),
    (3, 14, 2, 1, 5001, 5003, 128, False, None, True),       # shared by many CTAs
    (2, 32, 2, 1, 2049, 2049, 64, True, None, False),        # 16 rows
    (5, 8, 2, 1, 1500, 1500, 128, True, [0, 1, 1500, 31, 700], True),
    (5, 8, 2, 1, 333, 400, 64, True, [0, 1, 333, 32, 33], True),
    (4, 8, 2, 5, 1500, 1501, 128, True, [0, 3, 1500, 5], True),   # more rows than keys: some see none
    (4, 8, 2, 5, 90, 90, 64, True, [0, 3, 90, 5], False),
    (2, 14, 2, 18, 777, 780, 128, True, [777, 100], True),   # 126 rows: 8 row tiles
    (1, 2, 1, 64, 70, 70, 64, True, None, False),            # 128 rows
    (1, 4, 4, 1, 40000, 40000, 64, False, None, False),
    (1, 7, 1, 1, 90001, 90001, 64, True, None, True),        # shared through the workspace, 7 rows
    (2, 12, 1, 1, 40001, 40001, 64, True, [40001, 33], True),  # and 12
    (1, 14, 1, 3, 40001, 40001, 64, True, None, False),      # 42: three row tiles
    (2, 4, 2, 2, 60000, 60000, 64, True, [0, 0], True),      # nothing to share
    (70, 2, 1, 1, 9000, 9000, 64, True, [(613 * i) % 9001 if i % 3 == 0 else i % 5 for i in range(70)], True),
    (3, 5, 5, 3, 4000, 4100, 64, False, [4100, -5, 2222], True),  # lengths past Sk and below 0
    (70, 2, 1, 1, 600, 600, 64, True, [(37 * i) % 601 for i in range(70)], True),   # many short sequences
    (6, 36, 6, 2, 2500, 2600, 128, True, [2500, 0, 700, 2499, 1, 1800], True),      # 12 rows, more rounds than SMs
    (1, 28, 4, 16, 3800, 3801, 128, True, None, True),       # 112 rows, clusters of 5
    (2, 16, 2, 4, 4100, 4100, 64, True, [4100, 77], True),   # of 6
    (1, 7, 1, 1, 1700, 1700, 128, True, None, True),         # of 7
    (1, 10, 10, 1, 600, 600, 64, False, [555], False),       # of 3
]


@pytest.mark.parametrize("weights", [False, True], ids=["", "weights"])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_parity(case, weights):
    B, Hq, H, Sq, Sk, cap, D, causal, lengths, shifted = DECODE[case]
    rng = np.random.default_rng(100 + case)
    k, v = rows(rng, B, H, cap, D, "bias" if shifted else "plain"), rows(rng, B, H, cap, D, "plain")
    q = rng.standard_normal((B, Hq, Sq, D)).astype(np.float16)
    shift = k[:, :, 0].copy() if shifted else None
    kt, vt, qt = to_dev(k, v, q)
    st = None if shift is None else to_dev(shift)[0]
    cache = new_cache(B, H, cap, D)
    p = pasa()
    p.kv4_append(kt, vt, *cache, shift=st)
    n = np.clip(lengths if lengths else [Sk] * B, 0, Sk)
    for b in range(B):   # rows past the last: whatever was there
        for x, fill in zip(cache, (255, float("nan"), 255, float("inf"))):
            x[b, :, n[b]:] = fill
    ek, es = kv4.quantise(k, shift)
    ref = kv4.decode(q, kv4.values(ek, es), kv4.values(*kv4.quantise(v)), n, causal, D ** -0.5, shift)
    acc = torch.zeros((B, H, cap), device="cuda") if weights else None
    if weights:
        for b in range(B):
            acc[b, :, n[b]:] = -7
            ref["weights"][b, :, n[b]:] = -7
    lt = torch.tensor(lengths).int().cuda() if lengths else None
    got = p.attn_fwd_decode_kv4(qt, *cache, causal=causal, shift=st, length=Sk, lengths=lt, weights=acc)
    bounds = decode_bounds(ref, D ** -0.5, D, Hq // H, Sq, q, shift)
    bounds[2][ref["weights"] < 0] = 0
    check(got, ref, bounds, acc)
    # the same bits again, and with a scale of the caller's
    again = p.attn_fwd_decode_kv4(qt, *cache, causal=causal, shift=st, length=Sk, lengths=lt)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    ref = kv4.decode(q, kv4.values(ek, es), kv4.values(*kv4.quantise(v)), n, causal, 0.25, shift)
    got = p.attn_fwd_decode_kv4(qt, *cache, causal=causal, shift=st, length=Sk, lengths=lt, scale=0.25)
    check(got, ref, decode_bounds(ref, 0.25, D, Hq // H, Sq, q, shift))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sk", [400, 3001])
def test_peaked_scores_and_growing_maxima(Sk, D):
    """Scores that grow along the sequence (the running reference moves again and again), reach
    hundreds, and one row whose query is huge."""
    rng = np.random.default_rng(Sk)
    B, H, g = 1, 2, 4
    k = rows(rng, B, H, Sk, D, "plain").astype(np.float64)
    q = rng.standard_normal((B, H * g, 1, D))
    k += np.linspace(0, 12, Sk)[None, None, :, None] * np.sign(q[:, ::g])
    q[:, 1] *= 300
    k, q = k.astype(np.float16), q.astype(np.float16)
    v = rows(rng, B, H, Sk, D, "plain")
    cache = new_cache(B, H, Sk, D)
    kt, vt, qt = to_dev(k, v, q)
    pasa().kv4_append(kt, vt, *cache)
    acc = torch.zeros((B, H, Sk), device="cuda")
    got = pasa().attn_fwd_decode_kv4(qt, *cache, weights=acc)
    ref = kv4.decode(q, kv4.values(*kv4.quantise(k)), kv4.values(*kv4.quantise(v)), [Sk], False, D ** -0.5)
    check(got, ref, decode_bounds(ref, D ** -0.5, D, g, 1, q, None), acc)


@pytest.mark.parametrize("Sk", [100, 2000])
def test_a_nan_query_stays_in_its_row(Sk):
    rng = np.random.default_rng(3)
    B, H, g, D = 1, 2, 8, 128
    k, v = rows(rng, B, H, Sk, D, "plain"), rows(rng, B, H, Sk, D, "plain")
    q = rng.standard_normal((B, H * g, 1, D)).astype(np.float16)
    cache = new_cache(B, H, Sk, D)
    kt, vt, qt = to_dev(k, v, q)
    p = pasa()
    p.kv4_append(kt, vt, *cache)
    o, lse = p.attn_fwd_decode_kv4(qt, *cache)
    qt[0, 3, 0, 5] = float("nan")
    o2, lse2 = p.attn_fwd_decode_kv4(qt, *cache)
    assert torch.isnan(o2[0, 3]).all() and torch.isnan(lse2[0, 3]).all()
    keep = [h for h in range(H * g) if h != 3]
    assert torch.equal(o[0, keep], o2[0, keep]) and torch.equal(lse[0, keep], lse2[0, keep])


def test_offsets_past_32_bits():
    """One head of 70 million rows: its codes span 4.5 GB, its rows' byte offsets pass 2^32. All keys
    and values are 0 but for three rows, so the result has a closed form."""
    cap, D = 70_000_001, 128
    cache = new_cache(1, 1, cap, D, fill=0)
    p = pasa()
    at = [5, 68_000_003, cap - 1]
    k, v = np.zeros((3, D)), np.zeros((3, D))
    k[:, 0], v[:, 1] = [210, 217, 224], [7, 14, 28]
    for i, r in enumerate(at):
        kt, vt = to_dev(k[i].astype(np.float16)[None, None, None], v[i].astype(np.float16)[None, None, None])
        p.kv4_append(kt, vt, *cache, start=r)
    kr, _ = p.kv4_read(*cache, 1, start=at[2])
    assert kr[0, 0, 0, 0].item() == 224
    q = torch.zeros((1, 2, 1, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 1
    w = torch.zeros((1, 1, cap), device="cuda")
    o, lse = p.attn_fwd_decode_kv4(q, *cache, scale=0.125, weights=w)
    x = k[:, 0] * 0.125
    total = (cap - 3) + np.exp(x).sum()
    pr = np.exp(x) / total
    want = (pr * v[:, 1]).sum()
    # bounds as in decode_bounds with scores up to 28 and 7e7 equal terms summed by 2432 warps
    assert abs(o[0, 0, 0, 1].item() - want) <= want * (2.0 ** -10 + 2.0 ** -9)
    assert abs(lse[0, 0, 0].item() - np.log(total)) <= 2e-3
    got = w[0, 0, torch.tensor(at, device="cuda")].double().cpu().numpy()
    assert np.allclose(got, 2 * pr, rtol=5e-3)
    assert w[0, 0, at[1] - 1].item() == pytest.approx(2 / total, rel=5e-3)
    del cache, w


def test_more_heads_than_a_grid_dimension_and_no_lse():
    """70000 sequences of two rows, their outputs without a log-sum-exp (the C ABI's NULL)."""
    B, D = 70000, 64
    rng = np.random.default_rng(4)
    k, v = rows(rng, B, 1, 2, D, "plain"), rows(rng, B, 1, 2, D, "plain")
    q = rng.standard_normal((B, 1, 1, D)).astype(np.float16)
    cache = new_cache(B, 1, 2, D)
    kt, vt, qt = to_dev(k, v, q)
    p = pasa()
    p.kv4_append(kt, vt, *cache)
    kr, vr = (x.cpu().numpy().astype(np.float64) for x in p.kv4_read(*cache, 2))
    assert np.array_equal(kr, kv4.values(*kv4.quantise(k))) and np.array_equal(vr, kv4.values(*kv4.quantise(v)))
    o = torch.full_like(qt, 9)
    rc = p.library().pasa_attn_fwd_decode_kv4(qt.data_ptr(), *(c.data_ptr() for c in cache), None, None, o.data_ptr(), None,
                                              None, B, 1, 1, 1, 2, 2, D, 1, 0.0, None, 0,
                                              torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    x = np.einsum("bid,bjd->bj", q[:, 0].astype(np.float64), kr[:, 0]) / 8
    w = np.exp(x - x.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    want = np.einsum("bj,bjd->bd", w, vr[:, 0])
    # P's and the output's rounding (2^-11 each of at most max|v|), scores within 2^-16 of |x| < 40
    bound = np.abs(vr[:, 0]).max(1) * (2.0 ** -10 + 40 * 2.0 ** -15)
    assert (np.abs(o[:, 0, 0].cpu().numpy() - want) <= bound).all()


# ---- streams, graphs, workspaces ----

def small(B=3, Hq=14, H=2, Sk=2600, D=128, seed=0):
    rng = np.random.default_rng(seed)
    k, v = rows(rng, B, H, Sk, D, "bias"), rows(rng, B, H, Sk, D, "plain")
    q = rng.standard_normal((B, Hq, 1, D)).astype(np.float16)
    kt, vt, qt = to_dev(k, v, q)
    cache = new_cache(B, H, Sk, D)
    shift = kt[:, :, 0].contiguous()
    pasa().kv4_append(kt, vt, *cache, shift=shift)
    return qt, cache, shift


def test_calls_in_a_row_on_one_workspace_and_on_another_stream():
    p = pasa()
    sets = [small(seed=s, Sk=Sk) for s, Sk in ((0, 2600), (1, 900), (2, 5000))]
    want = [p.attn_fwd_decode_kv4(q, *c, shift=s) for q, c, s in sets]
    nbytes = max(p.decode_kv4_workspace_bytes(3, 14, 2, 1, Sk, 128) for Sk in (2600, 900, 5000))
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [p.attn_fwd_decode_kv4(q, *c, shift=s, workspace=ws) for _ in range(5) for q, c, s in sets]
    side.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])


def test_two_threads_on_two_streams():
    """Calls of all kinds at once, each thread on a stream of its own: equal to calls one by one."""
    import threading

    p = pasa()
    sets = [small(seed=7, Sk=30000, B=2, D=64), small(seed=8, Sk=1500)]
    want = [p.attn_fwd_decode_kv4(q, *c, shift=s) for q, c, s in sets]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            q, c, s = sets[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i].append(p.attn_fwd_decode_kv4(q, *c, shift=s))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,per_sequence,weights", [(1, True, False), (1, False, True), (3, True, True), (200, True, False)])
def test_step_equals_append_and_decode(n, per_sequence, weights, D):
    """Bit for bit, again and again on one stream (the decode kernel starts while rows are stored)."""
    p = pasa()
    B, Hq, H, cap = 3, 8, 2, 3000
    rng = np.random.default_rng(n)
    kt, vt = to_dev(rows(rng, B, H, cap, D, "bias"), rows(rng, B, H, cap, D, "plain"))
    qs = to_dev(rng.standard_normal((6, B, Hq, min(n, 5), D)).astype(np.float16))[0]
    shift = kt[:, :, 0].contiguous()
    first = torch.tensor([1234, 0, 2100] if per_sequence else [700] * 3).int().cuda()
    caches = [new_cache(B, H, cap, D) for _ in range(2)]
    accs = [torch.zeros((B, H, cap), device="cuda") if weights else None for _ in range(2)]
    for c in caches:
        p.kv4_append(kt, vt, *c, counts=first, shift=shift)
    pos = first.clone()
    outs = []
    for i in range(4):   # no synchronisation in between
        a = i * n
        k1, v1 = kt[:, :, a:a + n].contiguous(), vt[:, :, a:a + n].contiguous()
        start = pos.clone() if per_sequence else 700 + a
        got = p.attn_fwd_decode_step_kv4(qs[i], k1, v1, *caches[0], start, causal=True, shift=shift, weights=accs[0])
        p.kv4_append(k1, v1, *caches[1], start=start, shift=shift)
        want = p.attn_fwd_decode_kv4(qs[i], *caches[1], causal=True, shift=shift, weights=accs[1],
                                     **({"lengths": pos + n} if per_sequence else {"length": 700 + a + n}))
        outs.append((got, want))
        pos = pos + n
    for got, want in outs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for a, b in zip(caches[0], caches[1]):
        assert torch.equal(a, b)
    if weights:
        assert torch.equal(accs[0], accs[1])


@pytest.mark.parametrize("cap,weights", [(2000, True), (40000, True), (40000, False)], ids=["clusters", "stream_k", "plain"])
def test_captured_steps_follow_the_lengths_and_share_a_workspace(cap, weights):
    """A decode step (append one row, attend, gather weights) captured once and replayed as the
    sequences grow, twice in two graphs that share a workspace: equal to eager calls."""
    p = pasa()
    B, Hq, H, D = 3, 14, 2, 64
    rng = np.random.default_rng(11)
    kt, vt = to_dev(rows(rng, B, H, cap, D, "bias"), rows(rng, B, H, cap, D, "plain"))
    qs = to_dev(rng.standard_normal((4, B, Hq, 1, D)).astype(np.float16))[0]
    first = torch.tensor([cap - 500, 0, 700]).int().cuda()
    shift = kt[:, :, 0].contiguous()

    def state():
        cache = new_cache(B, H, cap, D)
        p.kv4_append(kt, vt, *cache, counts=first, shift=shift)
        return cache, torch.zeros((B, H, cap), device="cuda") if weights else None, first.clone(), first.clone()

    ws = torch.empty(max(1, p.decode_kv4_workspace_bytes(B, Hq, H, 1, cap, D, weights)), dtype=torch.uint8, device="cuda")

    def step(cache, acc, pos, lengths, q, k1, v1):
        p.kv4_append(k1, v1, *cache, start=pos, shift=shift)
        lengths.add_(1)
        out = p.attn_fwd_decode_kv4(q, *cache, causal=True, shift=shift, lengths=lengths, weights=acc, workspace=ws)
        pos.add_(1)
        return out

    new = [(kt[:, :, i:i + 1].contiguous(), vt[:, :, i:i + 1].contiguous()) for i in range(4)]
    eager = state()
    want = [step(*eager, qs[i], *new[i]) for i in range(4)]
    torch.cuda.synchronize()
    states, graphs, ins, outs = [state(), state()], [], [], []
    side = torch.cuda.Stream()
    for s in states:
        q, k1, v1 = qs[0].clone(), new[0][0].clone(), new[0][1].clone()
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            outs.append(step(*s, q, k1, v1))
        graphs.append(g), ins.append((q, k1, v1))
    for i in range(4):
        for g, x, out, s in zip(graphs, ins, outs, states):
            x[0].copy_(qs[i]), x[1].copy_(new[i][0]), x[2].copy_(new[i][1])
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])
    for s in states:
        for a, b in zip(s[0], eager[0]):
            assert torch.equal(a, b)
        assert s[1] is None or torch.equal(s[1], eager[1])


def test_binding_refusals():
    p = pasa()
    q, cache, shift = small()
    k1 = torch.zeros((3, 2, 1, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        p.attn_fwd_decode_kv4(q.float(), *cache)
    with pytest.raises(TypeError):
        p.attn_fwd_decode_kv4(q, *cache, lengths=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        p.attn_fwd_decode_kv4(q, *cache, lengths=torch.zeros(3, dtype=torch.int32))       # a host tensor
    with pytest.raises(ValueError):
        p.attn_fwd_decode_kv4(q, *cache, lengths=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        p.attn_fwd_decode_kv4(q, *cache, workspace=torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError):
        p.attn_fwd_decode_kv4(q, *cache, weights=torch.zeros((3, 2, 7), device="cuda"))
    with pytest.raises(ValueError):
        p.attn_fwd_decode_kv4(q, *cache, shift=shift[:, :1].contiguous())
    with pytest.raises(p.PasaError):
        p.attn_fwd_decode_kv4(q, *cache, length=2601)
    with pytest.raises(TypeError):
        p.attn_fwd_decode_kv4(q[:, :, :, ::2], *cache)
    with pytest.raises(p.PasaError):
        p.kv4_append(k1, k1, *cache, start=2600)
    with pytest.raises(ValueError):
        p.kv4_append(k1, k1[:, :1].contiguous().expand(3, 1, 1, 128).contiguous(), *cache)
    with pytest.raises(TypeError):
        p.kv4_append(k1.expand(3, 2, 4, 128), k1, *cache)
    with pytest.raises(ValueError):
        p.kv4_read(*cache, 4, out_k=k1)
    with pytest.raises(ValueError):
        p.kv4_append(k1, k1, *cache, start=2 ** 40)
    with pytest.raises(ValueError, match="current device is 1"):
        p._check_cuda(k1, "k", torch.float16, k1.shape, 1)     # a tensor of another device than the current one


@pytest.mark.parametrize("Sk,D", [(900, 128), (40000, 64), (40000, 128)])
def test_output_over_the_queries(Sk, D):
    """out = q gives the same bits, in clusters and shared out; with weights it is refused, as is one tensor
    for two outputs."""
    p = pasa()
    q, cache, shift = small(Sk=Sk, D=D, seed=9)
    o, lse = p.attn_fwd_decode_kv4(q, *cache, shift=shift)
    with pytest.raises(p.PasaError):
        p.attn_fwd_decode_kv4(q, *cache, shift=shift, out=q, weights=torch.zeros((3, 2, Sk), device="cuda"))
    x = torch.zeros((3, 2, 8, D), dtype=torch.float16, device="cuda")
    with pytest.raises(p.PasaError):
        p.kv4_read(*cache, 8, shift=shift, out_k=x, out_v=x)
    with pytest.raises(p.PasaError):
        p.kv4_append(x, x, cache[0], cache[1], cache[0], cache[3], shift=shift)
    got, lse2 = p.attn_fwd_decode_kv4(q, *cache, shift=shift, out=q)
    assert got is q and torch.equal(q, o) and torch.equal(lse2, lse)
