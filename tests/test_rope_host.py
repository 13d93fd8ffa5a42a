"""Rotary positions without a GPU: the frequencies, and the refusals of the C ABI (every call below is
rejected by host-side checks, so no pointer is dereferenced) and of the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

P = ctypes.c_void_p
FAKE = 1 << 20


@pytest.fixture(scope="module")
def pasa():
    from precision_flashattention_numerics_gb300 import build

    build.build()
    import precision_flashattention_numerics_gb300 as p

    return p


def freq(p, *a, **kw):
    f, m = p.rope_frequencies(*a, device="cpu", **kw)
    return f.numpy(), m


@pytest.mark.parametrize("R", [2, 24, 64, 128, 256])
def test_plain_and_linear_frequencies(pasa, R):
    f, m = freq(pasa, R, base=5e5)
    want = np.array([5e5 ** (-2.0 * i / R) for i in range(R // 2)])
    assert m == 1.0 and np.allclose(f, want, rtol=1e-15, atol=0)
    g, m = freq(pasa, R, base=5e5, scaling=pasa.ROPE_LINEAR, factor=8)
    assert m == 1.0 and np.array_equal(g, f / 8)


def test_changed_base_squeezes_the_slowest_pair_only(pasa):
    f, _ = freq(pasa, 64)
    g, m = freq(pasa, 64, scaling=pasa.ROPE_BASE, factor=4)
    assert m == 1.0 and g[0] == 1.0 and abs(g[-1] * 4 / f[-1] - 1) < 1e-14


def test_by_parts_blends_between_low_and_high(pasa):
    f, _ = freq(pasa, 128)
    g, m = freq(pasa, 128, scaling=pasa.ROPE_BY_PARTS, factor=16, original_length=4096, low=1, high=32)
    assert m == np.float32(0.1 * math.log(16) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert (g[turns > 32] == f[turns > 32]).all() and np.allclose(g[turns < 1], f[turns < 1] / 16, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    keep = (turns[mid] - 1) / 31
    assert mid.sum() > 5 and np.allclose(g[mid], f[mid] * (keep + (1 - keep) / 16), rtol=1e-13)


def test_frequency_refusals(pasa):
    lib = pasa.library()
    buf = (ctypes.c_double * 256)()

    def call(out=buf, R=64, base=1e4, scaling=0, factor=1.0, length=4096.0, low=1.0, high=32.0):
        return lib.pasa_rope_frequencies(ctypes.cast(out, P) if out else None, None, R, base, scaling, factor, length, low, high)

    assert call() == 0 and call(out=None) == -1
    for R in (0, 1, 63, 258, -2):
        assert call(R=R) == -2
    for base in (1.0, 0.0, -3.0, math.inf, math.nan):
        assert call(base=base) == -2
    assert call(scaling=4) == -3 and call(scaling=-1) == -3
    for s in (1, 2, 3):
        for factor in (0.5, math.nan, math.inf):
            assert call(scaling=s, factor=factor) == -2
    assert call(scaling=0, factor=math.nan) == 0      # not looked at
    assert call(R=2, scaling=2) == -2
    for bad in ({"length": 0.0}, {"low": -1.0}, {"low": 32.0}, {"high": math.inf}, {"low": math.nan}):
        assert call(scaling=3, **bad) == -2, bad


def test_rope_refusals(pasa):
    lib = pasa.library()

    def call(q=FAKE, qo=2 * FAKE, k=3 * FAKE, ko=4 * FAKE, Hq=4, Hkv=2, f=5 * FAKE, pos=6 * FAKE, starts=0, B=1, S=16, D=64, R=64,
             m=1.0, tin=0, tout=0, qs=None, ks=None, no_strides=False):
        q_st = (ctypes.c_longlong * 6)(*(qs or (Hq * S * D, S * D, D) * 2))
        k_st = (ctypes.c_longlong * 6)(*(ks or (Hkv * S * D, S * D, D) * 2))
        p = lambda x: P(x) if x else None   # noqa: E731
        st = lambda x: None if no_strides else ctypes.cast(x, P)   # noqa: E731
        return lib.pasa_rope(p(q), p(qo), st(q_st), Hq, p(k), p(ko), st(k_st), Hkv, p(f), p(pos), p(starts), 0, B, S, D, R, 0, 0,
                             m, tin, tout, None)

    good = call()      # everything but the device is fine
    assert good in (0, -3, -5) or torch.cuda.is_available()
    for name in ("q", "qo", "k", "ko", "f"):
        assert call(**{name: 0}) == -1
    assert call(no_strides=True) == -1
    for bad in ({"B": 0}, {"S": 0}, {"Hq": 0}, {"Hkv": -1}, {"D": 0}, {"D": 258, "R": 64}, {"D": 65}, {"R": 0}, {"R": 66}, {"R": 33},
                {"m": math.nan}, {"m": math.inf}, {"B": 65536, "S": 65536}):
        assert call(**bad) == -2, bad
    assert call(tin=3) == -3 and call(tout=3) == -3 and call(tin=0, tout=1) == -3 and call(tin=0, tout=2) == -3 and call(tin=1, tout=2) == -3
    assert call(q=FAKE + 1) == -4 and call(qo=2 * FAKE + 1) == -4 and call(tin=2, tout=2, k=3 * FAKE + 2) == -4
    assert call(f=5 * FAKE + 4) == -4 and call(pos=6 * FAKE + 2) == -4 and call(starts=FAKE + 2) == -4
    assert call(qs=(1024, 1024, -64) + (4096, 1024, 64)) == -2
    assert call(qs=(2 ** 60, 2 ** 60, 64) + (4096, 1024, 64), B=2) == -2


def test_rope_refuses_shared_memory(pasa):
    lib = pasa.library()
    S, D = 16, 64

    def call(q, qs, qo, qos, k, ks, ko, kos, Hq=4, Hkv=2, S=S, f=1 << 30, pos=1 << 31, tin=0, tout=0):
        a, b = (ctypes.c_longlong * 6)(*qs, *qos), (ctypes.c_longlong * 6)(*ks, *kos)
        return lib.pasa_rope(P(q), P(qo), ctypes.cast(a, P), Hq, P(k), P(ko), ctypes.cast(b, P), Hkv, P(f), P(pos), None, 0, 1, S, D,
                             D, 0, 0, 1.0, tin, tout, None)

    W = 8 * D                                   # q, k and v side by side in a row of 8 heads
    view = (0, D, W)
    q, k = FAKE, FAKE + 4 * D * 2
    fine = call(q, view, q, view, k, view, k, view)               # both in place
    assert fine != -2
    assert call(q, view, 2 * FAKE, view, k, view, 2 * FAKE + 4 * D * 2, view) != -2     # into another fused buffer
    assert call(q, view, 2 * FAKE, view, k, view, 2 * FAKE + 3 * D * 2, view) == -2     # k over q's last head
    assert call(q, view, q + D * 2, view, k, view, 2 * FAKE, view) == -2                # q over itself, one head on
    assert call(q, view, k, view, k, view, 2 * FAKE, view) == -2                        # q's output over k
    assert call(q, view, q, view, k, view, q, view) == -2                               # one output twice
    assert call(q, view, q, (0, D, W // 2), k, view, 2 * FAKE, view) == -2              # in place, other strides
    assert call(q, view, q, view, k, view, k, view, tin=1, tout=0) == -2                # in place, another type
    assert call(q, view, 2 * FAKE, (0, 0, W), k, view, 3 * FAKE, view) == -2            # rows of an output one over the other
    assert call(q, view, 2 * FAKE, (0, D, 2 * D), k, view, 3 * FAKE, view) == -2
    assert call(q, view, q, view, k, view, k, view, pos=q + 64) == -2
    assert call(q, view, q, view, k, view, k, view, f=k + 64) == -2
    assert call(q, (0, 0, 0), 2 * FAKE, view, k, view, 3 * FAKE, view) != -2            # a broadcast input is fine


def test_binding_refusals(pasa):
    x = torch.zeros((2, 4, 8, 64), dtype=torch.float16)
    if not torch.cuda.is_available():
        with pytest.raises((TypeError, ValueError, RuntimeError, AssertionError)):
            pasa.rope(x, x, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(pasa.PasaError):
        pasa.rope_frequencies(63, device="cpu")


def test_rope_in_place_is_the_same_order_of_dimensions(pasa):
    """A transposed view of q with as many heads as tokens (or sequences) has q's memory, sizes and set of strides, but
    other elements in its places: it shares q's memory and is no rotation in place."""
    lib = pasa.library()
    n, D = 8, 64

    def call(ins, outs, B=1, H=n, S=n, R=D, f=1 << 30, pos=1 << 31):
        st = (ctypes.c_longlong * 6)(*ins, *outs)
        return lib.pasa_rope(P(FAKE), P(FAKE), ctypes.cast(st, P), H, None, None, None, 0, P(f), P(pos), None, 0, B, S, D, R, 0, 0, 1.0, 0,
                             0, None)

    rows, turned = (0, D, n * D), (0, n * D, D)              # [T, H, D], and its transpose
    assert call(rows, rows) != -2 and call(turned, turned) != -2
    for R in (D, 32):
        assert call(rows, turned, R=R) == -2 and call(turned, rows, R=R) == -2
    whole = (n * n * D, n * D, D)                            # [B, H, S, D]
    assert call(whole, whole, B=n) != -2
    for other in ((n * D, n * n * D, D), (D, n * D, n * n * D), (n * n * D, D, n * D)):
        assert call(whole, other, B=n) == -2, other
    assert call((7, D, n * D), (9, D, n * D)) != -2          # the stride of a dimension of one says nothing
    assert call((7, D, 5), (9, D, 3), S=1) != -2


def test_rope_takes_calls_of_more_than_32_bits_of_pairs(pasa):
    """B * S and the heads fit 31 bits, the pairs of one token 32 bits; those of a call may be more, also where rows are not on
    16-byte boundaries."""
    lib = pasa.library()

    def call(H, S, D, R, B=1, Hkv=0):
        # q and k in place, 2^50 bytes apart
        st = (ctypes.c_longlong * 6)(*(H * S * D, D, H * D) * 2)
        kt = (ctypes.c_longlong * 6)(*(Hkv * S * D, D, Hkv * D) * 2)
        k = P(FAKE + (1 << 50)) if Hkv else None
        return lib.pasa_rope(P(FAKE), P(FAKE), ctypes.cast(st, P), H, k, k, ctypes.cast(kt, P) if Hkv else None, Hkv, P(1 << 60), None, None,
                             0, B, S, D, R, 0, 0, 1.0, 0, 0, None)

    for good in ((65536, 65600, 2, 2), (40, 1 << 26, 128, 24), (1, 2 ** 31 - 1, 128, 6), (32, 1 << 27, 256, 250), (1 << 25, 1, 256, 254)):
        assert call(*good) in (0, -3, -5), good
    assert call(1 << 26, 1, 256, 254) == -2                                      # 2^32 pairs and more in one token
    assert call(2 ** 31 - 1, 1, 16, 16) == -2 and call(2 ** 31 - 1, 1, 2, 2) in (0, -3, -5) and call(1 << 30, 1, 2, 2, Hkv=1 << 30) == -2
