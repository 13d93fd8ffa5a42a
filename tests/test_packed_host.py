"""Attention over packed sequences without a GPU: the workspace's size and the refusals of the C ABI (every
call below is rejected by host-side checks, so no pointer is dereferenced)."""
import ctypes

import pytest

P = ctypes.c_void_p
BIG = 1 << 32
Q, K, V, O, LSE, CQ, CK, WS = (BIG * i for i in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    from precision_flashattention_numerics_gb300 import build

    build.build()
    import precision_flashattention_numerics_gb300 as pasa

    return pasa.library()


def call(lib, q=Q, k=K, v=V, o=O, lse=LSE, cq=CQ, ck=CK, ws=WS, nbytes=None, N=3, Hq=8, Hkv=2, Tq=100, Tk=120, D=128, mode=1, strides=None,
         no_strides=False):
    st = strides or [Hq * D, D, Hkv * D, D, Hkv * D, D, Hq * D, D]
    a = (ctypes.c_longlong * 8)(*st)
    if nbytes is None:
        nbytes = lib.pasa_attn_fwd_packed_workspace_bytes(N, Hq, Hkv, Tq, Tk, D, mode)
    p = lambda x: P(x) if x else None   # noqa: E731
    return lib.pasa_attn_fwd_packed(p(q), p(k), p(v), p(o), None if no_strides else ctypes.cast(a, P), p(lse), p(cq), p(ck), N, Hq,
                                    Hkv, Tq, Tk, D, 1, 0.0, mode, p(ws), nbytes, None)


def test_workspace_bytes(lib):
    f = lib.pasa_attn_fwd_packed_workspace_bytes
    shifted, raw = f(3, 8, 2, 100, 120, 128, 1), f(3, 8, 2, 100, 120, 128, 3)
    assert shifted - raw >= 2 * 120 * 128 * 2 + 2 * 3 * 128 * 2 and raw > 0
    assert f(3, 8, 2, 100, 120, 128, 0) == shifted and f(3, 8, 2, 100, 120, 128, 2) == raw
    for bad in ((0, 8, 2, 100, 120, 128, 1), (3, 8, 3, 100, 120, 128, 1), (3, 8, 2, 0, 120, 128, 1), (3, 8, 2, 100, 0, 128, 1),
                (3, 8, 2, 100, 120, 96, 1), (3, 8, 2, 100, 120, 128, 4), (3, 8, 2, 100, 120, 128, -1),
                (3, 1 << 20, 1, 1 << 20, 120, 128, 1)):
        assert f(*bad) == 0, bad


def test_refusals(lib):
    for name in ("q", "k", "v", "o", "cq", "ck"):
        assert call(lib, **{name: 0}) == -1
    assert call(lib, no_strides=True) == -1
    for bad in ({"N": 0}, {"Hq": 0}, {"Hkv": -1}, {"Tq": 0}, {"Tk": 0}, {"Hkv": 3}, {"Tq": 2 ** 31 - 1}, {"Tk": 2 ** 31 - 1},
                {"Hq": 1 << 20, "Hkv": 1, "Tq": 1 << 20}):
        assert call(lib, nbytes=1 << 30, **bad) == -2, bad
    assert call(lib, D=96, nbytes=1 << 30) == -3
    for mode in (-1, 4, 5, 6):
        assert call(lib, mode=mode, nbytes=1 << 30) == -3
    for name, at in (("q", Q), ("k", K), ("v", V), ("o", O)):
        assert call(lib, **{name: at + 8}) == -4
    assert call(lib, lse=LSE + 2) == -4 and call(lib, cq=CQ + 1) == -4 and call(lib, ck=CK + 2) == -4 and call(lib, ws=WS + 16) == -4
    assert call(lib, ws=0) == -7 and call(lib, nbytes=100) == -7
    good = [8 * 128, 128, 2 * 128, 128, 2 * 128, 128, 8 * 128, 128]
    for i in range(8):
        assert call(lib, strides=good[:i] + [good[i] + 4] + good[i + 1:]) == -4
        assert call(lib, strides=good[:i] + [0] + good[i + 1:]) == -2
        assert call(lib, strides=good[:i] + [-8] + good[i + 1:]) == -2
        assert call(lib, strides=good[:i] + [1 << 40] + good[i + 1:]) == -2


def test_refuses_shared_memory(lib):
    fused = [12 * 128, 128] * 4
    views = dict(k=Q + 8 * 256, v=Q + 10 * 256, strides=fused)
    fine = (0, -3, -5)      # every host check but the device's passed
    assert call(lib, o=Q, **views) in fine and call(lib, **views) in fine               # over q itself, or elsewhere
    assert call(lib, o=Q + 256, **views) == -2                                           # over q, one head on
    assert call(lib, o=Q + 8 * 256, **views) == -2                                       # over k and v
    assert call(lib, o=Q + 4 * 256, **views) == -2
    assert call(lib, o=Q, strides=[8 * 128, 128, 256, 128, 256, 128, 16 * 128, 128]) == -2   # over q, other strides
    assert call(lib, strides=[8 * 128, 128, 256, 128, 256, 128, 128, 128]) == -2         # rows of o one over the other
    for at in (Q, K, V, O, CQ, CK):
        assert call(lib, lse=at) == -2 and call(lib, ws=at) == -2
    assert call(lib, lse=WS + 1024) == -2 and call(lib, o=CQ) == -2


def test_in_place_of_q_is_the_same_order_of_dimensions(lib):
    """o as a transposed view of q, with as many heads as tokens, is not q itself."""
    n, D = 8, 128
    rows, turned, keys = [n * D, D], [D, n * D], [2 * D, D] * 2
    for a, b in ((rows, turned), (turned, rows)):
        assert call(lib, o=Q, Hq=n, Tq=n, strides=a + keys + a) in (0, -3, -5)
        assert call(lib, o=Q, Hq=n, Tq=n, strides=a + keys + b) == -2
