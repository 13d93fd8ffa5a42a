"""The 4-bit cache without a GPU: the oracle's pins, and the refusals of the C ABI (every call
below is rejected by host-side checks, so no pointer is dereferenced) and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4

P = ctypes.c_void_p
FAKE = 1 << 20
MIS4, MIS16, MIS256 = FAKE + 2, FAKE + 8, FAKE + 16


@pytest.fixture(scope="module")
def lib():
    from precision_flashattention_numerics_gb300 import build

    build.build()
    import precision_flashattention_numerics_gb300 as pasa

    return pasa.library()


# ---- the oracle ----

def test_hand_worked_group():
    """max|x| = 7: scale 1, so codes are the rounded values; ties go to the even code."""
    x = np.zeros((1, 1, 1, 32), np.float16)
    x[0, 0, 0, :8] = [7, -7, 0.5, 1.5, 2.5, -0.5, -1.5, 3.25]
    codes, s = kv4.quantise(x)
    assert s.tolist() == [[[[1.0]]]]
    want = [7, -7, 0, 2, 2, 0, -2, 3] + [0] * 24
    assert kv4.values(codes, s)[0, 0, 0].tolist() == want
    assert codes[0, 0, 0, 0] == (7 + 8) | ((-7 + 8) << 4)


def test_scale_has_eight_bits_and_products_are_exact_in_fp16():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((1, 1, 4000, 64)) * 10.0 ** rng.uniform(-7, 4, (1, 1, 4000, 1))).astype(np.float16)
    codes, s = kv4.quantise(x)
    assert np.array_equal(kv4.round_bits(s, 8), s.astype(np.float64))
    v = kv4.values(codes, s)
    assert np.array_equal(kv4.to_fp16(v), v)
    # within half a step of the input, where the scale is not an fp16 subnormal
    step = np.repeat(s.astype(np.float64), 32, -1)
    fine = step >= 2.0 ** -14
    assert (np.abs(v - x.astype(np.float64)) <= 0.5 * step * (1 + 1e-12))[fine].all()


def test_what_is_not_finite_or_zero():
    x = np.zeros((1, 1, 1, 64), np.float16)
    x[0, 0, 0, :4] = [np.nan, np.inf, -np.inf, 65504]
    codes, s = kv4.quantise(x)
    v = kv4.values(codes, s)[0, 0, 0]
    assert v[0] == 0 and v[1] == v[3] == -v[2] == 7 * 9344.0 and np.isfinite(v).all()
    assert (v[32:] == 0).all() and s[0, 0, 0, 1] == 0


def test_fp32_route_gives_the_same_scales_and_codes():
    """The kernel takes both quotients as products with reciprocals in fp32. Scales: max|x| * (1 / 7),
    rounded to 16 bits and then to 8, for every fp16 value. Codes: x * (1 / s) (the reciprocal off by
    up to 2^-22), rounded to a multiple of 2^-14 by adding 768 in one fma and then to an
    integer, for every fp16 value against every 8-bit scale of one binade (other binades are the
    same numbers times a power of two). Both equal the rounding of the exact quotient."""
    a = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float32)
    bits = (a * np.float32(1 / 7)).view(np.uint32)
    s16 = ((bits + np.uint32(0x80)) & np.uint32(0xFFFFFF00)).view(np.float32)
    assert np.array_equal(kv4.round_bits(s16, 8), kv4.round_bits(a.astype(np.float64) / 7, 8))
    x = np.arange(0, 0x4C01, dtype=np.uint16).view(np.float16).astype(np.float64)   # 0 .. 16
    for sv in np.arange(128, 256) * 2.0 ** -7:          # 1 .. 2
        xs = x[x <= 7.04 * sv]
        for off in (-2.0 ** -22, 0.0, 2.0 ** -22):
            r = float(np.float32((1 + off) / sv))
            snapped = np.rint((xs * r + 768.0) * 2.0 ** 14) * 2.0 ** -14
            assert np.array_equal(np.rint(snapped - 768.0), np.rint(xs / sv))


def test_select_order_and_ties():
    w = np.array([3, 1, 3, np.nan, 2, -0.0, 0.0, 9], np.float32)
    assert kv4.select(w, 8, 3, 1) == [0, 2, 7]
    assert kv4.select(w, 8, 2, 1) == [0, 7]
    assert kv4.select(w, 7, 6, 0) == [0, 1, 2, 4, 5, 6]
    assert kv4.select(w, 4, 3, 0) == [0, 1, 2] and kv4.select(w, 3, 3, 0) == [0, 1, 2] and kv4.select(w, 0, 3, 0) == []


# ---- the C ABI ----

def test_store_refusals(lib):
    def store(fn, k=FAKE, v=FAKE, shift=FAKE, k4=FAKE, ks=FAKE, v4=FAKE, vs=FAKE, starts=0, start=0, counts=0, B=1, H=2,
              n=5, cap=16, D=128):
        p = lambda x: P(x) if x else None   # noqa: E731
        if fn is lib.pasa_kv4_append:
            t = [p(k), p(v), p(shift), p(k4), p(ks), p(v4), p(vs)]
        else:
            t = [p(k4), p(ks), p(v4), p(vs), p(shift), p(k), p(v)]
        return fn(*t, p(starts), start, p(counts), B, H, n, cap, D, None)

    for fn in (lib.pasa_kv4_append, lib.pasa_kv4_read):
        for name in ("k", "v", "k4", "ks", "v4", "vs"):
            assert store(fn, **{name: 0}) == -1
            assert store(fn, **{name: MIS16}) == -4
        assert store(fn, shift=MIS16) == -4
        assert store(fn, starts=MIS4) == -4 and store(fn, counts=MIS4) == -4
        for bad in ({"B": 0}, {"H": -1}, {"n": 0}, {"cap": 0}, {"start": -1}, {"start": 12}, {"n": 17}):
            assert store(fn, **bad) == -2, bad
        assert store(fn, start=2 ** 31 - 1, n=2 ** 31 - 1) == -2
        assert store(fn, B=65536, H=65536) == -2                      # B * Hkv overflows
        assert store(fn, n=2 ** 31 - 1, cap=2 ** 31 - 1) == -2        # so do a block's last row numbers
        assert store(fn, D=96) == -3 and store(fn, D=32) == -3


def test_decode_refusals(lib):
    def dec(q=FAKE, k4=FAKE, ks=FAKE, v4=FAKE, vs=FAKE, shift=0, lengths=0, o=FAKE, lse=FAKE, weights=0, B=1, Hq=8,
            Hkv=2, Sq=1, Sk=50000, cap=50000, D=128, ws=FAKE, nbytes=None):
        p = lambda x: P(x) if x else None   # noqa: E731
        if nbytes is None:
            nbytes = lib.pasa_attn_fwd_decode_kv4_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, int(bool(weights)))
        return lib.pasa_attn_fwd_decode_kv4(p(q), p(k4), p(ks), p(v4), p(vs), p(shift), p(lengths), p(o), p(lse),
                                            p(weights), B, Hq, Hkv, Sq, Sk, cap, D, 1, 0.0, p(ws), nbytes, None)

    for name in ("q", "k4", "ks", "v4", "vs", "o"):
        assert dec(**{name: 0}) == -1
    for name in ("q", "k4", "ks", "v4", "vs", "o", "lse", "shift", "weights"):
        assert dec(**{name: MIS16}) == -4
    assert dec(lengths=MIS4) == -4
    for bad in ({"B": 0}, {"Hq": 0}, {"Hkv": 0}, {"Hq": 7}, {"Sq": 0}, {"Sk": 0}, {"cap": 49999}, {"Sk": 2 ** 31 - 1, "cap": 2 ** 31 - 1}):
        assert dec(**bad, nbytes=1 << 30) == -2, bad
    assert dec(D=96, nbytes=1 << 30) == -3
    assert dec(Sq=33, nbytes=1 << 30) == -3                           # 4 heads x 33 rows
    assert dec(ws=0) == -7 and dec(ws=MIS256) == -4
    need = lib.pasa_attn_fwd_decode_kv4_workspace_bytes(1, 8, 2, 1, 50000, 128, 0)
    assert need > 0 and dec(nbytes=need - 1) == -7
    more = lib.pasa_attn_fwd_decode_kv4_workspace_bytes(1, 8, 2, 1, 50000, 128, 1)
    assert more > need and dec(weights=FAKE, nbytes=need) == -7
    assert lib.pasa_attn_fwd_decode_kv4_workspace_bytes(1, 8, 2, 1, 100, 128, 0) == 0   # a CTA per kv head
    assert lib.pasa_attn_fwd_decode_kv4_workspace_bytes(1, 7, 2, 1, 100, 128, 0) == 0
    assert lib.pasa_attn_fwd_decode_kv4_workspace_bytes(1, 8, 2, 33, 5000, 128, 0) == 0


def test_step_refusals(lib):
    def step(k=FAKE, v=FAKE, starts=0, start=49999, n=1, Sq=1, Sk=1, cap=50000, D=128, o=FAKE, ws=FAKE, nbytes=1 << 30):
        p = lambda x: P(x) if x else None   # noqa: E731
        c = [P(FAKE)] * 4
        return lib.pasa_attn_fwd_decode_step_kv4(P(FAKE), p(k), p(v), *c, None, p(starts), start, p(o), P(FAKE), None, 1, 8,
                                                 2, Sq, n, Sk, cap, D, 1, 0.0, p(ws), nbytes, None)

    assert step(o=0) == -1
    for bad in ({"n": 0}, {"start": 50000}, {"start": -1}, {"starts": FAKE, "Sk": 50001}, {"starts": FAKE, "Sk": 0}):
        assert step(**bad) == -2, bad
    assert step(Sq=33) == -3 and step(D=32) == -3
    assert step(ws=0) == -7 and step(nbytes=16) == -7             # 50000 rows, whatever Sk says
    assert step(starts=MIS4, Sk=50000) == -4
    # what the append refuses is refused before anything is enqueued: the decode's checks passed
    assert step(k=0) == -1 and step(v=MIS16) == -4


def test_evict_refusals(lib):
    def evict(planes=(FAKE, FAKE * 3), out=(FAKE * 2, FAKE * 4), rb=(64, 8), n=None, w=FAKE * 5, ow=FAKE * 6, lengths=0,
              index=FAKE, new=0, B=1, H=2, Sk=64, cap=64, out_cap=32, budget=32, recent=4):
        p = lambda x: P(x) if x else None   # noqa: E731
        k = max(len(planes), len(out))
        arr = lambda t, x: (t * k)(*x)      # noqa: E731
        return lib.pasa_cache_evict(arr(P, planes) if planes else None, arr(P, out), arr(ctypes.c_int, rb),
                                    len(planes) if n is None else n, p(w), p(ow), p(lengths), p(index), p(new), B, H, Sk,
                                    cap, out_cap, budget, recent, None)

    assert evict(planes=()) == -1 and evict(w=0) == -1 and evict(ow=0) == -1 and evict(index=0) == -1
    assert evict(planes=(FAKE, 0)) == -1 and evict(out=(FAKE * 2, 0)) == -1
    for bad in ({"B": 0}, {"H": 0}, {"Sk": 0}, {"cap": 63}, {"budget": 0}, {"recent": -1}, {"recent": 33},
                {"out_cap": 31}, {"rb": (64, 0)}, {"rb": (64, 65540)}):
        assert evict(**bad) == -2, bad
    assert evict(n=0) == -3 and evict(n=9) == -3 and evict(rb=(64, 6)) == -3
    for bad in ({"planes": (FAKE, MIS16)}, {"out": (FAKE * 2, MIS16)}, {"w": MIS16}, {"ow": MIS16}, {"index": MIS16},
                {"lengths": MIS4}, {"new": MIS4}):
        assert evict(**bad) == -4, bad
    # in place: everything, and in a cache of the same size
    same = {"out": (FAKE, FAKE * 3), "ow": FAKE * 5, "out_cap": 64}
    assert evict(**{**same, "out_cap": 32}) == -2
    assert evict(**{**same, "ow": FAKE * 2}) == -2
    assert evict(**{**same, "out": (FAKE, FAKE * 2)}) == -2
    # two outputs in one place
    assert evict(out=(FAKE * 2, FAKE * 2)) == -2 and evict(out=(FAKE * 2, FAKE * 6)) == -2
    assert evict(**{**same, "planes": (FAKE, FAKE), "out": (FAKE, FAKE)}) == -2
    if not torch.cuda.is_available():
        assert evict(**same) in (-3, -5) and evict() in (-3, -5)   # nothing wrong but the device


# ---- the binding ----

def test_binding_refuses_host_tensors_and_large_ints():
    import precision_flashattention_numerics_gb300 as pasa

    with pytest.raises(ValueError):
        pasa._int32(2 ** 31, "start")
    with pytest.raises(TypeError):
        pasa._check_cuda(torch.zeros(4), "x", torch.float32, (4,), 0)


# ---- sizes that no GPU holds ----

HUGE = """
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
P, I = ctypes.c_void_p, ctypes.c_int
size = lib.pasa_attn_fwd_decode_kv4_workspace_bytes
size.restype = ctypes.c_size_t
bad = []
# B, Hq, Hkv, Sq, Sk: B * Hkv passes an int; B * Hkv * row tiles does; the segments' rounds do
for B, Hq, Hkv, Sq, Sk, want in ((65536, 32768, 32768, 1, 100, -2), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1, 1, -2),
                                 (32768, 131072, 8192, 8, 100, -2), (2 ** 31 - 1, 128, 1, 1, 1, -2),
                                 (65536, 4096, 4096, 1, 1000, -2), (1024, 1024, 1024, 1, 2 ** 31 - 70000, -2)):
    for weights in (0, 1):
        got = size(B, Hq, Hkv, Sq, Sk, 64, weights)
        if got != 0:
            bad.append((B, Hq, Hkv, Sq, Sk, weights, got))
    f = P(1 << 20)
    for w in (None, f):
        rc = lib.pasa_attn_fwd_decode_kv4(f, f, f, f, f, None, None, f, None, w, B, Hq, Hkv, Sq, Sk, Sk, 64, 1,
                                          ctypes.c_float(0), f, ctypes.c_size_t(1 << 40), None)
        step = lib.pasa_attn_fwd_decode_step_kv4(f, f, f, f, f, f, f, None, f, 0, f, None, w, B, Hq, Hkv, Sq, 1, Sk, Sk, 64,
                                                 1, ctypes.c_float(0), f, ctypes.c_size_t(1 << 40), None)
        if (rc, step) != (want, want):
            bad.append((B, Hq, Hkv, Sq, Sk, rc, step))
print("bad", bad)
"""


def test_more_segments_than_an_int_are_refused(lib):
    """In a process of its own: a size that gets past the checks can end it."""
    import subprocess
    import sys

    from precision_flashattention_numerics_gb300 import library_path

    r = subprocess.run([sys.executable, "-c", HUGE, library_path], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "bad []", (r.returncode, r.stdout, r.stderr)
    # the last size before an int's end has a layout, and only then the device is asked for
    assert lib.pasa_attn_fwd_decode_kv4_workspace_bytes(8192, 8192, 8192, 1, 64, 64, 0) == 0
    assert lib.pasa_attn_fwd_decode_kv4_workspace_bytes(8192, 8192, 8192, 1, 300, 64, 1) == 8192 * 8192 * 8 * 4


def test_evict_refuses_what_overlaps(lib):
    """Tensors that share bytes without being the same one in place: a CTA could write a row before another reads it."""
    M = 1 << 20

    def evict(planes, out, rb, w, ow, B=2, H=4, cap=1024, out_cap=512, budget=512):
        n = len(planes)
        arr = lambda t, x: (t * n)(*x)   # noqa: E731
        return lib.pasa_cache_evict(arr(P, planes), arr(P, out), arr(ctypes.c_int, rb), n, P(w), P(ow), None, P(100 * M), None,
                                    B, H, cap, cap, out_cap, budget, 4, None)

    rb = (64, 8)                      # planes of 512 KB and 64 KB, weights of 32 KB; half of that when out_cap is 512
    fine = dict(planes=(M, 2 * M), out=(3 * M, 4 * M), rb=rb, w=5 * M, ow=6 * M)
    size, half = 2 * 4 * 1024, 2 * 4 * 512
    if not torch.cuda.is_available():
        assert evict(**fine) in (-3, -5)
        # end to end, with no byte shared
        assert evict(**{**fine, "out": (M + 64 * size, 2 * M - 8 * half)}) in (-3, -5)
        assert evict(**{**fine, "out": fine["planes"], "ow": 5 * M, "out_cap": 1024}) in (-3, -5)
    for bad in ({"out": (M + 64 * size - 16, 4 * M)}, {"out": (M - 64 * half + 16, 4 * M)},   # a plane's own source
                {"out": (2 * M, M)},                                                         # each other's place
                {"out": (3 * M, M + 16)}, {"out": (5 * M, 4 * M)}, {"out": (3 * M, 5 * M + 4 * size - 16)},
                {"ow": M}, {"ow": 2 * M + 8 * size - 16}, {"ow": 5 * M + 16},
                {"out": (3 * M, 3 * M + 64 * half - 16)}, {"ow": 4 * M + 16}):              # another output
        assert evict(**{**fine, **bad}) == -2, bad
    # in place, planes that overlap each other or the weights
    for planes, w in (((M, M + 16), 5 * M), ((M, 2 * M), M + 64 * size - 16), ((M, 2 * M), 2 * M + 16)):
        assert evict(planes=planes, out=planes, rb=rb, w=w, ow=w, out_cap=1024) == -2
    # sizes whose bytes pass 64 bits
    assert evict(planes=(M, 1 << 40), out=(1 << 41, 1 << 42), rb=(65536, 65536), w=1 << 43, ow=1 << 44, B=1 << 14, H=1 << 14,
                 cap=2 ** 31 - 1, out_cap=2 ** 31 - 1, budget=64) == -2


@pytest.mark.parametrize("rb,most", [((64, 8, 64, 8), 6_100_480), ((32, 4, 32, 4), 9_586_688), ((256, 256), 2_033_536)])
def test_largest_budget_of_an_eviction(lib, rb, most):
    """CTAs of a budget: 256 threads move 4 words each (16, 8 or 4 bytes, as a row's bytes allow) of columns of up to
    128 bytes, one grid row per CTA, 65535 in all. In place, where a CTA has all rows, no budget is refused."""
    def ctas(budget):
        n = 0
        for b in (*rb, 4):
            word = 16 if b % 16 == 0 else 8 if b % 8 == 0 else 4
            rows = 256 // (min(b, 128) // word) * 4
            n += -(-budget // rows) * -(-b // 128)
        return n

    def evict(budget, in_place=False):
        k, M = len(rb), 1 << 40
        src, dst = [M * (i + 1) for i in range(k)], [M * (20 + i) for i in range(k)]
        dst = src if in_place else dst
        arr = lambda t, x: (t * k)(*x)   # noqa: E731
        return lib.pasa_cache_evict(arr(P, src), arr(P, dst), arr(ctypes.c_int, rb), k, P(M * 10), P(M * (10 if in_place else 30)),
                                    None, P(M * 40), None, 1, 1, budget + 9, budget + 9, budget + (9 if in_place else 0), budget,
                                    4, None)

    assert ctas(most) <= 65535 < ctas(most + 1)
    assert evict(most + 1) == -2
    if not torch.cuda.is_available():
        assert evict(most) in (-3, -5) and evict(most + 1, in_place=True) in (-3, -5)


def test_store_and_decode_refuse_what_overlaps(lib):
    """Outputs that share memory with an input or with each other. (o = q with weights: the weights pass would read the
    output as queries. Two cache tensors in one place: rows of one over rows of the other.)"""
    M = 1 << 20
    B, Hq, H, Sq, n, cap, D = 2, 8, 2, 3, 5, 50000, 128      # 50000 rows: with a workspace
    names = ("q", "k", "v", "k4", "ks", "v4", "vs", "shift", "starts", "counts", "o", "lse", "weights", "ws")
    need = lib.pasa_attn_fwd_decode_kv4_workspace_bytes(B, Hq, H, Sq, cap, D, 1)
    assert need > 0
    size = {"q": B * Hq * Sq * 2 * D, "k": B * H * n * 2 * D, "k4": B * H * cap * D // 2, "ks": B * H * cap * D // 16,
            "shift": B * H * 2 * D, "starts": 4 * B, "lse": B * Hq * Sq * 4, "weights": B * H * cap * 4, "ws": need}
    size.update(v=size["k"], v4=size["k4"], vs=size["ks"], o=size["q"], counts=size["starts"])
    at0 = {name: 64 * M * (i + 1) for i, name in enumerate(names)}

    def calls(at):
        p = {x: P(a) if a else None for x, a in at.items()}
        c = [p[x] for x in ("k4", "ks", "v4", "vs")]
        return {
            "append": lambda: lib.pasa_kv4_append(p["k"], p["v"], p["shift"], *c, p["starts"], 0, p["counts"], B, H, n, cap, D, None),
            "read": lambda: lib.pasa_kv4_read(*c, p["shift"], p["k"], p["v"], p["starts"], 0, p["counts"], B, H, n, cap, D, None),
            "decode": lambda: lib.pasa_attn_fwd_decode_kv4(p["q"], *c, p["shift"], p["starts"], p["o"], p["lse"], p["weights"], B, Hq,
                                                           H, Sq, cap, cap, D, 1, 0.0, p["ws"], need, None),
            "step": lambda: lib.pasa_attn_fwd_decode_step_kv4(p["q"], p["k"], p["v"], *c, p["shift"], p["starts"], 0, p["o"], p["lse"],
                                                              p["weights"], B, Hq, H, Sq, n, cap, cap, D, 1, 0.0, p["ws"], need, None),
        }

    cache = ["k4", "ks", "v4", "vs"]
    # what each writes, and what it reads
    writes = {"append": cache, "read": ["k", "v"], "decode": ["o", "lse", "weights", "ws"], "step": cache + ["o", "lse", "weights", "ws"]}
    reads = {"append": ["k", "v", "shift", "starts", "counts"], "read": cache + ["shift", "starts", "counts"],
             "decode": ["q"] + cache + ["shift", "starts"], "step": ["q", "shift", "starts"]}
    fine = (-3, -5)
    for call in writes:
        if not torch.cuda.is_available():
            assert calls(at0)[call]() in fine, call
        for w in writes[call]:
            for x in writes[call] + reads[call]:
                if x == w:
                    continue
                step = 256 if w == "ws" else 16
                at = dict(at0)
                at[w] = at[x] + (size[x] - 1) // step * step       # w begins in x's last bytes
                assert calls(at)[call]() == -2, (call, w, x)
                at[w] = at[x] - (size[w] - 1) // step * step       # and ends in its first
                assert calls(at)[call]() == -2, (call, w, x)
                at[w] = at[x]
                assert calls(at)[call]() == -2, (call, w, x)
                if not torch.cuda.is_available():
                    at[w] = at[x] + -(-size[x] // step) * step     # behind it
                    assert calls(at)[call]() in fine, (call, w, x)
    for call in ("decode", "step"):
        same = {**at0, "o": at0["q"], "weights": 0}
        assert calls({**same, "o": at0["q"] + 256})[call]() == -2
        if not torch.cuda.is_available():
            assert calls(same)[call]() in fine                    # without weights o may be q
