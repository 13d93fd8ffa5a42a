"""Storing picked rows in the 4-bit cache without a GPU: the refusals of the C ABI (every call below is
rejected by host-side checks, so no pointer is dereferenced)."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE = 1 << 28


@pytest.fixture(scope="module")
def lib():
    from precision_flashattention_numerics_gb300 import build

    build.build()
    import precision_flashattention_numerics_gb300 as pasa

    return pasa.library()


def test_refusals(lib):
    t = [FAKE * i for i in range(1, 11)]

    def store(k=t[0], v=t[1], shift=t[2], k4=t[3], ks=t[4], v4=t[5], vs=t[6], rows=t[7], starts=0, start=0, counts=0, B=1, H=2, n=5,
              n_src=9, cap=16, D=128):
        p = lambda x: P(x) if x else None   # noqa: E731
        return lib.pasa_kv4_append_rows(p(k), p(v), p(shift), p(k4), p(ks), p(v4), p(vs), p(rows), p(starts), start, p(counts), B, H,
                                        n, n_src, cap, D, None)

    for name in ("k", "v", "k4", "ks", "v4", "vs", "rows"):
        assert store(**{name: 0}) == -1
    for name in ("k", "v", "k4", "ks", "v4", "vs", "shift"):
        assert store(**{name: FAKE + 8}) == -4
    for name in ("rows", "starts", "counts"):
        assert store(**{name: FAKE * 9 + 2}) == -4
    for bad in ({"B": 0}, {"H": -1}, {"n": 0}, {"n_src": 0}, {"cap": 0}, {"start": -1}, {"start": 12}, {"n": 17}, {"B": 65536, "H": 65536}):
        assert store(**bad) == -2, bad
    assert store(D=96) == -3
    # the cache's tensors share no memory with what is read, all n_src rows of k and v among it
    for name in ("k4", "ks", "v4", "vs"):
        assert store(**{name: t[7]}) == -2                               # the row numbers
        assert store(**{name: t[0] + 2 * 9 * 256 - 16}) == -2            # k's last bytes
        assert store(**{name: t[1] + 1024}) == -2
    assert store(k4=t[4]) == -2
