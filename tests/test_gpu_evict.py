"""GPU parity of cache eviction: the rows kept (whole numbers) and everything that moves with
them, bit for bit against oracle/kv4.py's selection; and the 4-bit cache's operators used
together, prompt to decode."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import rel_errors, to_dev
from oracle import kv4
from test_gpu_kv4 import check, decode_bounds, new_cache, rows

pytestmark = pytest.mark.gpu


def pasa():
    import precision_flashattention_numerics_gb300 as p

    return p


def make_weights(rng, B, H, cap, kind):
    w = rng.random((B, H, cap)).astype(np.float32) ** 8
    if kind == "ties":
        w = rng.integers(0, 4, (B, H, cap)).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":
        w -= 0.01
        w[rng.random(w.shape) < 0.2] = 0.0
        w[rng.random(w.shape) < 0.1] = -0.0
        w[rng.random(w.shape) < 0.1] = np.nan
        w[rng.random(w.shape) < 0.1] = np.inf
        w[rng.random(w.shape) < 0.1] = -np.inf
        w[rng.random(w.shape) < 0.1] = 1e-42
    return w


CASES = [
    # B, H, Sk, cap, out_cap, budget, recent, lengths, kind
    (1, 1, 2, 2, 1, 1, 0, None, "plain"),
    (1, 1, 2, 2, 1, 1, 1, None, "plain"),
    (2, 3, 1000, 1100, 700, 512, 32, None, "plain"),
    (2, 3, 1000, 1100, 700, 512, 0, None, "ties"),
    (2, 3, 1025, 1025, 512, 512, 512, None, "plain"),        # the recent rows only
    (5, 2, 3000, 3001, 1500, 1024, 7, [0, 1, 3000, 1024, 1025], "odd"),
    (4, 1, 5000, 5000, 5000, 4999, 100, [5000, 9999, -3, 4998], "equal"),
    (1, 2, 40000, 40000, 4200, 4096, 128, None, "ties"),
    (1, 1, 70001, 70001, 70001, 30011, 1, None, "plain"),
    (2, 2, 50, 60, 200, 100, 3, [50, 20], "plain"),          # a budget that nothing reaches
    (20, 4, 8300, 8300, 700, 512, 30, None, "ties"),         # many heads: a CTA for each, in two chunks
]


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_evict_parity(case, in_place):
    B, H, Sk, cap, out_cap, budget, recent, lengths, kind = CASES[case]
    if in_place and budget > cap:
        pytest.skip("in place the budget is at most the cache's size")
    rng = np.random.default_rng(case)
    w = make_weights(rng, B, H, cap, kind)
    # planes of every row width: 64 + 8 bytes (a 4-bit cache), fp16 rows, 4, 12 and 48 bytes
    planes = [rng.integers(0, 256, (B, H, cap, n)).astype(np.uint8) for n in (64, 8, 256, 4, 12, 48, 32)]
    n = np.clip(lengths if lengths else [Sk] * B, 0, Sk)
    lt = torch.tensor(lengths).int().cuda() if lengths else None
    wt, *pt = to_dev(w, *planes)
    oc = cap if in_place else out_cap
    out = pt if in_place else [torch.full((B, H, oc, p.shape[-1]), 77, dtype=torch.uint8, device="cuda") for p in pt]
    ow = wt if in_place else torch.full((B, H, oc), 77.0, device="cuda")
    before = [o.cpu().numpy() for o in out]
    index, new = pasa().cache_evict(pt, wt, budget, recent, length=Sk, lengths=lt, out=None if in_place else out,
                                    out_weights=None if in_place else ow)
    index, new, ow = index.cpu().numpy(), new.cpu().numpy(), ow.cpu().numpy()
    assert np.array_equal(new, np.minimum(n, budget))
    got = [o.cpu().numpy() for o in out]
    for b in range(B):
        for h in range(H):
            keep = kv4.select(w[b, h], n[b], budget, recent)
            m = len(keep)
            assert index[b, h, :m].tolist() == keep and (index[b, h, m:] == -1).all()
            assert np.array_equal(ow[b, h, :m], w[b, h, keep], equal_nan=True) and (ow[b, h, m:] == 0).all()
            for g, p, old in zip(got, planes, before):
                assert np.array_equal(g[b, h, :m], p[b, h, keep]) and np.array_equal(g[b, h, m:], old[b, h, m:])


def test_lengths_updated_in_place_on_another_stream_and_in_a_graph():
    """new_lengths may be lengths itself; captured and replayed on fresh contents."""
    p = pasa()
    rng = np.random.default_rng(5)
    B, H, cap, budget = 3, 2, 900, 300
    planes = [rng.integers(0, 256, (B, H, cap, n)).astype(np.uint8) for n in (32, 4)]
    w = make_weights(rng, B, H, cap, "ties")
    lengths = [900, 301, 12]
    lt = torch.tensor(lengths).int().cuda()
    pt, wt = to_dev(*planes), to_dev(w)[0]
    index = torch.empty((B, H, budget), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        p.cache_evict(pt, wt, budget, 10, lengths=lt, index=index, new_lengths=lt)
    for _ in range(2):
        lt.copy_(torch.tensor(lengths)), wt.copy_(torch.from_numpy(w))
        for a, b in zip(pt, planes):
            a.copy_(torch.from_numpy(b))
        g.replay()
        torch.cuda.synchronize()
        assert lt.tolist() == [300, 300, 12]
        for b in range(B):
            for h in range(H):
                keep = kv4.select(w[b, h], lengths[b], budget, 10)
                assert index[b, h].tolist()[:len(keep)] == keep
                assert np.array_equal(pt[0][b, h, :len(keep)].cpu().numpy(), planes[0][b, h, keep])


def test_evict_refusals():
    p = pasa()
    k = torch.zeros((1, 2, 64, 128), dtype=torch.float16, device="cuda")
    w = torch.zeros((1, 2, 64), device="cuda")
    with pytest.raises(p.PasaError):
        p.cache_evict([k, k.clone()], w, 32, 33)
    with pytest.raises(p.PasaError):
        p.cache_evict([k], w, 0)
    with pytest.raises(p.PasaError):
        p.cache_evict([k], w, -1)
    with pytest.raises(ValueError):
        p.cache_evict([k], w, 32, out=[k.clone()])
    with pytest.raises(p.PasaError):
        p.cache_evict([k], w, 32, out=[k], out_weights=w.clone())     # half in place
    with pytest.raises(TypeError):
        p.cache_evict([k], w, 32, out=[k.float()], out_weights=w.clone())
    with pytest.raises(TypeError):
        p.cache_evict([k.transpose(1, 2)], w, 32)
    with pytest.raises(ValueError):
        p.cache_evict([k], w[:, :1].contiguous(), 32)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_score_evict_decode(D):
    """A serving run. The prompt's attention by attn_fwd; its keys and values into a 4-bit cache; the
    last 8 rows score the cache; it is cut down in place; then steps that append a row and
    attend, gathering weights, with a second cut on the way. Checked step by step."""
    p = pasa()
    B, Hq, H, S, W, budget, recent, cap = 2, 8, 2, 700, 8, 300, 40, 800
    g, scale = Hq // H, D ** -0.5
    rng = np.random.default_rng(D)
    k, v = rows(rng, B, H, S + 6, D, "bias"), rows(rng, B, H, S + 6, D, "plain")
    q = rng.standard_normal((B, Hq, S + 6, D)).astype(np.float16)
    kt, vt, qt = to_dev(k, v, q)
    part = lambda x, a, b: x[:, :, a:b].contiguous()   # noqa: E731
    kp, vp, qp = part(kt, 0, S), part(vt, 0, S), part(qt, 0, S)
    o, _ = p.attn_fwd(qp, kp, vp, causal=True, mode=p.MODE_SHIFT_F32ACC)
    o_ref, _ = oracle.attention(q[:, :, :S], k[:, :, :S], v[:, :, :S], causal=True)
    assert rel_errors(o.cpu().numpy(), o_ref)[0] < 5e-3
    # the shift: the pseudo-average of the prompt's first block
    _, means = p.kshift(kp)
    shift = means[:, :, 0].contiguous()
    hs = shift.cpu().numpy()
    cache = new_cache(B, H, cap, D)
    p.kv4_append(kp, vp, *cache, shift=shift)
    # a prefill on the cache: its values through attn_fwd, against the oracle on the same values
    kc, vc = p.kv4_read(*cache, S, shift=shift)
    o, _ = p.attn_fwd(part(qp, S - 64, S), kc, vc, causal=True, mode=p.MODE_SHIFT_F32ACC)
    o_ref, _ = oracle.attention(np.ascontiguousarray(q[:, :, S - 64:S]), kc.cpu().numpy(), vc.cpu().numpy(), causal=True)
    assert rel_errors(o.cpu().numpy(), o_ref)[0] < 5e-3

    acc = torch.zeros((B, H, cap), device="cuda")
    lengths = torch.tensor([S, S]).int().cuda()
    vals = [kv4.values(*kv4.quantise(k[:, :, :S], hs)), kv4.values(*kv4.quantise(v[:, :, :S]))]
    total = np.zeros((B, H, S))

    def attend(a, b):
        n = [vals[0].shape[2]] * B
        qh = np.ascontiguousarray(q[:, :, a:b])
        got = p.attn_fwd_decode_kv4(part(qt, a, b), *cache, causal=True, shift=shift, lengths=lengths, weights=acc)
        ref = kv4.decode(qh, *vals, n, True, scale, hs)
        bounds = decode_bounds(ref, scale, D, g, b - a, qh, hs)
        check(got, ref, bounds)
        bound = bounds[2] + 2.0 ** -23 * total
        total[:] += ref["weights"]
        return bound

    def cut():
        """The oracle selects by the kernel's own weights (their order is theirs to a rounding)."""
        w = acc.cpu().numpy()
        index, _ = p.cache_evict(cache, acc, budget, recent, lengths=lengths, new_lengths=lengths)
        keep = np.array([[kv4.select(w[b, h], n_before, budget, recent) for h in range(H)] for b in range(B)])
        assert np.array_equal(index.cpu().numpy(), keep)
        for i in (0, 1):
            vals[i] = np.take_along_axis(vals[i], keep[..., None], 2)
        assert lengths.tolist() == [budget] * B
        return np.take_along_axis(total, keep, 2)

    bound = attend(S - W, S)
    assert (np.abs(acc[:, :, :S].cpu().numpy() - total) <= bound).all()
    n_before = S
    total = cut()
    for i in range(6):
        k1, v1 = part(kt, S + i, S + i + 1), part(vt, S + i, S + i + 1)
        p.kv4_append(k1, v1, *cache, start=lengths, shift=shift)
        lengths += 1
        vals = [np.concatenate([vals[0], kv4.values(*kv4.quantise(k[:, :, S + i:S + i + 1], hs))], 2),
                np.concatenate([vals[1], kv4.values(*kv4.quantise(v[:, :, S + i:S + i + 1]))], 2)]
        total = np.concatenate([total, np.zeros((B, H, 1))], 2)
        attend(S + i, S + i + 1)
        if i == 3:
            n_before = budget + 4
            total = cut()
    p.check_device_error()


def test_calls_in_a_row_share_index_and_outputs():
    """Twenty evictions of other weights behind one another into the same index, lengths and outputs, each result
    copied on the stream: every move goes by the rows that its own selection, just ahead of it, wrote."""
    p = pasa()
    rng = np.random.default_rng(23)
    B, H, cap, budget, recent = 4, 3, 1300, 700, 20
    planes = [rng.integers(0, 256, (B, H, cap, n)).astype(np.uint8) for n in (64, 8)]
    pt = to_dev(*planes)
    ws = [make_weights(rng, B, H, cap, kind) for kind in ("plain", "ties", "odd", "equal") * 5]
    wt = to_dev(*ws)
    out = [torch.zeros((B, H, budget, x.shape[-1]), dtype=torch.uint8, device="cuda") for x in planes]
    ow = torch.zeros((B, H, budget), device="cuda")
    index = torch.zeros((B, H, budget), dtype=torch.int32, device="cuda")
    new = torch.zeros((B,), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = []
    for w in wt:
        p.cache_evict(pt, w, budget, recent, out=out, out_weights=ow, index=index, new_lengths=new)
        got.append([x.clone() for x in (index, *out, ow)])
    for w, (idx, *moved, kept) in zip(ws, got):
        keep = np.array([[kv4.select(w[b, h], cap, budget, recent) for h in range(H)] for b in range(B)])
        assert np.array_equal(idx.cpu().numpy(), keep)
        for m, x in zip(moved, planes):
            assert np.array_equal(m.cpu().numpy(), np.take_along_axis(x, keep[..., None], 2))
        assert np.array_equal(kept.cpu().numpy(), np.take_along_axis(w, keep, 2), equal_nan=True)
