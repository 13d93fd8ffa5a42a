"""GPU parity of storing picked rows in the 4-bit cache (the accepted ones of drafted tokens): bit for bit
against the exact arithmetic of oracle/kv4.py on the rows picked."""
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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,n_src,n,cap,shifted", [(1, 1, 1, 1, 1, False), (3, 2, 8, 5, 20, True), (4, 5, 64, 64, 300, True),
                                                   (2, 1, 700, 33, 40, False), (2, 3, 5, 70, 99, True)])
def test_picked_rows_are_stored_exactly(B, H, n_src, n, cap, shifted, D):
    rng = np.random.default_rng(n + D + n_src)
    k, v = rows(rng, B, H, n_src, D, "bias"), rows(rng, B, H, n_src, D, "wide")
    shift = k[:, :, 0].copy()
    pick = rng.integers(-1, n_src + 1, (B, n)).astype(np.int32)      # some outside, some twice
    pick[0, 0] = n_src - 1
    if n > 2:
        pick[:, 1], pick[:, 2] = -2 ** 31, 2 ** 31 - 1
    counts = rng.integers(0, n + 3, B).astype(np.int32)
    counts[0] = n
    starts = rng.integers(-2, cap, B).astype(np.int32)               # some rows fall outside the cache
    starts[0] = cap - n
    kt, vt, st, pt, ct, at = to_dev(k, v, shift, pick, counts, starts)
    cache = new_cache(B, H, cap, D, fill=3)
    pasa().kv4_append(kt, vt, *cache, start=at, counts=ct, shift=st if shifted else None, rows=pt)
    new = (*kv4.quantise(k, shift if shifted else None), *kv4.quantise(v))
    want = host(*new_cache(B, H, cap, D, fill=3))
    for b in range(B):
        for i in range(min(n, counts[b])):
            row = starts[b] + i
            if 0 <= pick[b, i] < n_src and 0 <= row < cap:
                for w, x in zip(want, new):
                    w[b, :, row] = x[b, :, pick[b, i]]
    for got, w in zip(host(*cache), want):
        assert np.array_equal(got, w)


def test_all_rows_in_order_equal_the_plain_append():
    rng = np.random.default_rng(5)
    k, v = rows(rng, 2, 3, 77, 128, "odd"), rows(rng, 2, 3, 77, 128, "odd")
    kt, vt = to_dev(k, v)
    a, b = new_cache(2, 3, 90, 128), new_cache(2, 3, 90, 128)
    order = torch.arange(77, dtype=torch.int32, device="cuda").expand(2, 77).contiguous()
    pasa().kv4_append(kt, vt, *a, start=4)
    pasa().kv4_append(kt, vt, *b, start=4, rows=order)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_binding_refusals():
    p = pasa()
    k = torch.zeros((2, 1, 4, 64), dtype=torch.float16, device="cuda")
    c = new_cache(2, 1, 8, 64)
    pick = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    for bad in (pick.long(), pick.cpu(), pick.t()):
        with pytest.raises((TypeError, ValueError)):
            p.kv4_append(k, k, *c, rows=bad)
    with pytest.raises(ValueError):
        p.kv4_append(k, k, *c, rows=pick[:1])
    with pytest.raises(ValueError):
        p.kv4_append(k, k, *c, rows=pick[0])
    with pytest.raises(p.PasaError):
        p.kv4_append(k, k, *c, start=6, rows=pick)                       # 3 rows from row 6 of 8
