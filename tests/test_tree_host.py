"""Tree attention on the 4-bit cache without a GPU: the workspace's size and the refusals of the C ABI (every call
below is rejected by host-side checks, so no pointer is dereferenced)."""
import ctypes

import pytest

P = ctypes.c_void_p
BIG = 1 << 32
NAMES = ("q", "k", "v", "parents", "counts", "k4", "ks", "v4", "vs", "shift", "lengths", "o", "lse")
AT = {name: BIG * (i + 1) for i, name in enumerate(NAMES)}
WS = BIG * 20


@pytest.fixture(scope="module")
def lib():
    from precision_flashattention_numerics_gb300 import build

    build.build()
    import precision_flashattention_numerics_gb300 as pasa

    return pasa.library()


def call(lib, ws=WS, nbytes=None, B=2, Hq=8, Hkv=2, Sq=5, Sk=5000, cap=5003, D=128, **at):
    if nbytes is None:
        nbytes = lib.pasa_attn_fwd_tree_kv4_workspace_bytes(B, Hq, Hkv, Sq, Sk, D)
    ptr = [P(at.get(n, AT[n])) if at.get(n, AT[n]) else None for n in NAMES]
    return lib.pasa_attn_fwd_tree_kv4(*ptr, B, Hq, Hkv, Sq, Sk, cap, D, 0.0, P(ws) if ws else None, nbytes, None)


def test_workspace_bytes(lib):
    f = lib.pasa_attn_fwd_tree_kv4_workspace_bytes
    assert f(2, 8, 2, 5, 5000, 128) >= 2 * 152 * 128 * (128 * 4 + 8) and f(2, 8, 2, 5, 5000, 64) > 0
    assert f(2, 8, 2, 5, 100, 128) == 0 and f(2, 8, 2, 5, 0, 64) == 0      # a CTA takes each segment whole
    for bad in ((0, 8, 2, 5, 100, 128), (2, 8, 3, 5, 100, 128), (2, 8, 2, 0, 100, 128), (2, 8, 2, 129, 100, 128), (2, 8, 2, 5, -1, 128),
                (2, 8, 2, 5, 100, 96), (1 << 20, 1 << 10, 1 << 10, 5, 1 << 20, 128), (2, 8, 2, 5, 2 ** 31 - 1, 128)):
        assert f(*bad) == 0, bad


def test_refusals(lib):
    for name in ("q", "k", "v", "k4", "ks", "v4", "vs", "o"):
        assert call(lib, **{name: 0}) == -1
    for name in ("q", "k", "v", "k4", "ks", "v4", "vs", "o", "shift", "lse"):
        assert call(lib, **{name: AT[name] + 8}) == -4
    for name in ("parents", "counts", "lengths"):
        assert call(lib, **{name: AT[name] + 2}) == -4
    for bad in ({"B": 0}, {"Hq": 0}, {"Hkv": 3}, {"Sq": 0}, {"Sk": -1}, {"cap": 4999}, {"cap": 0}, {"B": 65536, "Hkv": 65536, "Hq": 65536},
                {"B": 1 << 20, "Hq": 1 << 10, "Hkv": 1 << 10, "Sk": 1 << 20, "cap": 1 << 20}, {"Sk": 2 ** 31 - 1, "cap": 2 ** 31 - 1}):
        assert call(lib, nbytes=1 << 30, **bad) == -2, bad
    assert call(lib, D=96, nbytes=1 << 30) == -3 and call(lib, Sq=129, nbytes=1 << 30) == -3
    assert call(lib, ws=0) == -7 and call(lib, nbytes=1000) == -7 and call(lib, ws=WS + 128) == -4


def test_refuses_shared_memory(lib):
    for name in NAMES[:-2]:
        for out in ("o", "lse"):
            assert call(lib, **{out: AT[name]}) == -2, (out, name)
        assert call(lib, ws=AT[name]) == -2
    assert call(lib, lse=AT["o"]) == -2 and call(lib, ws=AT["o"]) == -2 and call(lib, ws=AT["lse"]) == -2
