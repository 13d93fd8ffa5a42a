"""GPU parity of rotary positions against their definition in 64 bits.

The tolerance of an output y = u c - v s. The angle's fraction of a turn is kept to 2^-32 turns and
rounded to fp32 in half turns: at most 2^-25 half turns, pi 2^-25 < 2^-23 radians; sincospif is off by at most
2 units in the last place (2^-23 at 1) and the product with mscale by 2^-24. Two products and a sum (one fused) are off
by at most 3 * 2^-24 of |u| + |v|. Together less than (|u| + |v|) mscale 2^-21. The 64-bit angle of the check
itself, and inv_freq / 2 pi in 64 bits, are off by position * inv_freq * 2^-52 each. Then half a
step of the output's type.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 2.0 ** -149}


def pasa():
    import precision_flashattention_numerics_gb300 as p

    return p


def pairs(R, interleaved):
    i = torch.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def definition(x, pos, f, interleaved, mscale, inverse):
    """(y, |u| + |v| of each output's pair, angle) of x [B, H, S, D] in 64 bits; pos [B, S]."""
    x, f = x.double().cpu(), f.double().cpu()
    a = pos.double().cpu()[:, None, :, None] * f * (-1 if inverse else 1)
    first, second = pairs(2 * len(f), interleaved)
    u, v = x[..., first], x[..., second]
    y, size, angle = x.clone(), torch.zeros_like(x), torch.zeros_like(x)
    y[..., first], y[..., second] = mscale * (u * a.cos() - v * a.sin()), mscale * (u * a.sin() + v * a.cos())
    size[..., first] = size[..., second] = u.abs() + v.abs()
    angle[..., first] = angle[..., second] = a.abs().expand(u.shape)
    return y, size, angle


def close(got, x, pos, f, interleaved=False, mscale=1.0, inverse=False):
    y, size, angle = definition(x, pos, f, interleaved, mscale, inverse)
    turned = size > 0
    tol = size * abs(mscale) * (2.0 ** -21 + angle * 2.0 ** -51) + y.abs() * HALF_STEP[got.dtype] * 1.001 + TINY[got.dtype]
    off = (got.double().cpu() - y).abs()
    assert (off <= tol)[turned].all(), float((off / tol)[turned].max())
    rest = ~turned                    # not turned: copied, rounded to the output's type
    assert torch.equal(got.cpu()[rest], x.cpu()[rest].to(got.dtype))


def inputs(B, H, S, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, H, S, D), generator=g).to(dtype).cuda()


def places(B, S, far, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (B, S), generator=g).int().cuda()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,S,D,R", [(1, 1, 1, 1, 64, 64), (3, 28, 4, 1, 128, 128), (2, 5, 5, 77, 64, 32), (1, 7, 1, 130, 128, 96),
                                           (2, 4, 2, 33, 64, 24), (1, 3, 1, 9, 80, 48), (1, 2, 2, 5, 256, 256), (2, 2, 1, 17, 6, 2),
                                           (1, 9, 3, 1000, 72, 64)])
def test_layouts_and_sizes(B, Hq, Hkv, S, D, R, interleaved):
    q, k, pos = inputs(B, Hq, S, D, torch.float16, 1), inputs(B, Hkv, S, D, torch.float16, 2), places(B, S, 40000, 3)
    f, m = pasa().rope_frequencies(R)
    oq, ok = pasa().rope(q, k, f, positions=pos, interleaved=interleaved)
    close(oq, q, pos, f, interleaved)
    close(ok, k, pos, f, interleaved)


@pytest.mark.parametrize("src,dst", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float16),
                                     (torch.float32, torch.float32), (torch.float32, torch.float16)])
@pytest.mark.parametrize("R", [64, 48, 20])
def test_types_scale_and_inverse(src, dst, R):
    B, S, D = 2, 50, 64
    q, k, pos = inputs(B, 6, S, D, src, 4), inputs(B, 2, S, D, src, 5), places(B, S, 1 << 20, 6)
    f, m = pasa().rope_frequencies(R, base=5e5, scaling=3, factor=8, original_length=8192, low=1, high=4)
    for inverse in (False, True):
        oq, ok = torch.empty_like(q, dtype=dst), torch.empty_like(k, dtype=dst)
        pasa().rope(q, k, f, positions=pos, interleaved=inverse, mscale=m, inverse=inverse, out_q=oq, out_k=ok)
        close(oq, q, pos, f, inverse, m, inverse)
        close(ok, k, pos, f, inverse, m, inverse)


def test_far_and_negative_positions():
    q = inputs(1, 2, 8, 128, torch.float32, 7)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9, 2 ** 24 + 1, -12345]], dtype=torch.int32).cuda()
    f, _ = pasa().rope_frequencies(128)
    out, none = pasa().rope(q, None, f, positions=pos, out_q=torch.empty_like(q))
    assert none is None
    close(out, q, pos, f)


@pytest.mark.parametrize("start", [0, 31000, "tensor"])
def test_positions_from_starts(start):
    B, S = 3, 19
    q, k = inputs(B, 4, S, 64, torch.float16, 8), inputs(B, 4, S, 64, torch.float16, 9)
    st = torch.tensor([5, 0, 32000], dtype=torch.int32).cuda() if start == "tensor" else start
    f, _ = pasa().rope_frequencies(64)
    oq, ok = pasa().rope(q, k, f, start=st)
    pos = (st[:, None] if start == "tensor" else st) + torch.arange(S, dtype=torch.int32).cuda().expand(B, S)
    close(oq, q, pos, f)
    close(ok, k, pos, f)


@pytest.mark.parametrize("R,D", [(64, 64), (32, 64), (24, 64)])
def test_packed_views_in_place_equal_new_tensors(R, D):
    """q and k as views of a fused projection's rows, turned in place; v is left alone."""
    T, Hq, Hkv = 301, 6, 2
    qkv = inputs(1, T, Hq + 2 * Hkv, D, torch.float16, 10)[0]
    pos, (f, _) = places(1, T, 9000, 11)[0], pasa().rope_frequencies(R)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    before = qkv.clone()
    oq, ok = pasa().rope(q, k, f, positions=pos)
    assert torch.equal(qkv, before)
    close(oq.transpose(0, 1)[None], before[:, :Hq].transpose(0, 1)[None], pos[None], f)
    pasa().rope(q, k, f, positions=pos, out_q=q, out_k=k)
    assert torch.equal(q, oq) and torch.equal(k, ok) and torch.equal(qkv[:, Hq + Hkv:], before[:, Hq + Hkv:])
    # [B, H, S, D] views of the same rows, unaligned ones too
    wide = torch.zeros((T, Hq + 2 * Hkv, D + 1), dtype=torch.float16, device="cuda")
    wide[..., 1:] = before
    odd = wide[:, :Hq, 1:].transpose(0, 1)[None]
    out = pasa().rope(odd, None, f, positions=pos[None])[0]
    assert torch.equal(out[0].transpose(0, 1), oq)


def test_broadcast_input_and_spoiled_pairs():
    q = inputs(1, 1, 4, 64, torch.float16, 12).expand(3, 5, 4, 64)
    f, _ = pasa().rope_frequencies(64)
    out = pasa().rope(q, None, f, start=7)[0]
    assert torch.equal(out, pasa().rope(q.contiguous(), None, f, start=7)[0])
    x = inputs(1, 1, 1, 64, torch.float16, 13)
    clean = pasa().rope(x, None, f, start=7)[0]
    x[..., 3], x[..., 40] = float("nan"), float("inf")
    y = pasa().rope(x, None, f, start=7)[0]
    spoiled = torch.zeros(64, dtype=torch.bool)
    spoiled[[3, 35, 8, 40]] = True
    assert torch.equal(y[..., ~spoiled], clean[..., ~spoiled]) and not y[..., spoiled].isfinite().any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """Against the formula (the transpose of the rotation, by autograd in 64 bits) and against differences of
    the kernel's own forward pass, which is linear: <g, rope(x + h d) - rope(x)> = h <rope_inverse(g), d>."""
    B, H, S, D, R, m = 2, 3, 11, 64, 48, 1.2
    x, g = inputs(B, H, S, D, torch.float32, 14), inputs(B, H, S, D, torch.float32, 15)
    pos = places(B, S, 5000, 16)
    f, _ = pasa().rope_frequencies(R)
    grad = pasa().rope(g, None, f, positions=pos, interleaved=interleaved, mscale=m, inverse=True, out_q=torch.empty_like(g))[0]
    leaf = x.double().cpu().requires_grad_()
    a = pos.double().cpu()[:, None, :, None] * f.cpu()
    first, second = pairs(R, interleaved)
    u, v = leaf[..., first], leaf[..., second]
    y = leaf.clone()
    y[..., first], y[..., second] = m * (u * a.cos() - v * a.sin()), m * (u * a.sin() + v * a.cos())
    (y * g.double().cpu()).sum().backward()
    close(grad, g, pos, f, interleaved, m, True)
    assert (grad.double().cpu() - leaf.grad).abs().max() <= 2 * m * g.abs().max().item() * 2.0 ** -20
    d = inputs(B, H, S, D, torch.float32, 17)
    run = lambda t: pasa().rope(t, None, f, positions=pos, interleaved=interleaved, mscale=m,    # noqa: E731
                                out_q=torch.empty_like(t))[0].double()
    left, right = (g.double() * (run(x + d) - run(x))).sum(), (grad.double() * d.double()).sum()
    # each of the n outputs is off by at most (|u| + |v|) m 2^-21 and x + d by 2^-24 of it, |.| <= 8 here
    assert (left - right).abs() <= (g.double().abs().sum() + d.double().abs().sum()) * 64 * m * 2.0 ** -21


def test_refusals_on_the_device():
    p = pasa()
    q = inputs(1, 4, 8, 64, torch.float16, 18)
    f, _ = p.rope_frequencies(64)
    with pytest.raises(ValueError):
        p.rope(q.transpose(2, 3), None, f)                           # channels not contiguous
    with pytest.raises(TypeError):
        p.rope(q.double(), None, f)
    with pytest.raises(TypeError):
        p.rope(q, None, f.float())
    with pytest.raises(TypeError):
        p.rope(q, None, f, positions=torch.zeros((1, 8), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        p.rope(q, None, f, positions=torch.zeros((1, 7), dtype=torch.int32, device="cuda"))
    with pytest.raises(p.PasaError):
        p.rope(q, None, p.rope_frequencies(128)[0])                  # more channels than the head has
    with pytest.raises(p.PasaError):
        p.rope(q[:, :2], q[:, 2:], f, out_q=q[:, 1:3], out_k=torch.empty_like(q[:, 2:]))
    with pytest.raises(p.PasaError):
        p.rope(q, None, f, out_q=torch.empty_like(q, dtype=torch.bfloat16))


def test_captured_on_a_side_stream():
    q, k = inputs(1, 8, 64, 128, torch.float16, 19), inputs(1, 2, 64, 128, torch.float16, 20)
    f, _ = pasa().rope_frequencies(128)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    pasa().rope(q, k, f, start=start, out_q=oq, out_k=ok)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pasa().rope(q, k, f, start=start, out_q=oq, out_k=ok)
    for at in (0, 77):
        start.fill_(at)
        graph.replay()
        want = pasa().rope(q, k, f, start=at)
        assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_gradients_have_the_type_of_what_they_come_from(dtype):
    """A gradient that fp16 cannot hold is not lost where no output is given: turned back, it keeps its type. Forward, the outputs are
    fp16, which the attention takes."""
    g = inputs(2, 3, 9, 64, dtype, 21) * (1.0 if dtype is torch.float16 else 1e6)
    pos, (f, _) = places(2, 9, 5000, 22), pasa().rope_frequencies(64)
    for k in (None, g[:, :1]):
        dq, dk = pasa().rope(g, k, f, positions=pos, inverse=True)
        assert dq.dtype is dtype and (k is None or dk.dtype is dtype)
        close(dq, g, pos, f, inverse=True)
        if k is not None:
            close(dk, k, pos, f, inverse=True)
    packed, _ = pasa().rope(g[0].transpose(0, 1), None, f, positions=pos[0], inverse=True)
    assert torch.equal(packed.transpose(0, 1), dq[0])
    assert pasa().rope(g, None, f, positions=pos)[0].dtype is torch.float16
    half = torch.empty((2, 1, 9, 64), dtype=torch.float16, device="cuda")
    assert pasa().rope(g, g[:, :1], f, positions=pos, inverse=True, out_k=half)[0].dtype is torch.float16


def test_more_than_32_bits_of_pairs():
    """2^32 pairs and more, in place, which takes more than one launch: each token's heads hold the same pair and turn alike, once."""
    T, H = 65600, 65536
    x = torch.empty((T, H, 2), dtype=torch.float16, device="cuda")
    x[..., 0], x[..., 1] = 1, 0.5
    f = torch.tensor([0.01], dtype=torch.float64, device="cuda")
    pasa().rope(x, None, f, out_q=x)
    first = x[:, :1].clone()
    for part in x.split(8192):
        lead = part[:, :1]
        assert bool((part == lead).all())
    want = torch.tensor([1, 0.5], dtype=torch.float16).expand(1, 1, T, 2)
    close(first.transpose(0, 1)[None], want, torch.arange(T)[None], f)


@pytest.mark.parametrize("R", [128, 24])
def test_angles_of_fast_pairs_far_away(R):
    """Against exact arithmetic (integers and fractions, 1 / 2 pi to 80 places): frequencies of many radians a position at the farthest
    positions, where 64-bit products would be off by up to position * frequency * 2^-52 radians. Only what close() allows at
    position 0 is allowed: an angle is off by at most 2^-64 of a turn for each position, 2^-33 turns in all, besides its rounding."""
    from fractions import Fraction

    turn = Fraction("0.15915494309189533576888376337251436203445964574045644874766734405889679763422653509")
    rng = np.random.default_rng(23)
    f = np.concatenate([[1.0, 12.5, 1000.7, 12345.678, 3e9, 0.5, 1e-9], 10.0 ** rng.uniform(-6, 6, R // 2 - 7)])
    pos = np.array([2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, -123456789, 10 ** 6, 1, 0, -1], np.int32)
    x = inputs(1, 2, len(pos), 128, torch.float32, 24)
    out, _ = pasa().rope(x, None, torch.tensor(f).cuda(), positions=torch.tensor(pos)[None].cuda(), out_q=torch.empty_like(x))
    a = 2 * np.pi * np.array([[float((Fraction(float(w)) * turn * int(p) + Fraction(1, 2)) % 1 - Fraction(1, 2)) for w in f] for p in pos])
    u, v = (x.double().cpu().numpy()[0, :, :, s] for s in (slice(0, R // 2), slice(R // 2, R)))
    got = out.double().cpu().numpy()[0]
    for y, want in ((got[..., :R // 2], u * np.cos(a) - v * np.sin(a)), (got[..., R // 2:R], u * np.sin(a) + v * np.cos(a))):
        off = np.abs(y - want)
        tol = (np.abs(u) + np.abs(v)) * 2.0 ** -21 + np.abs(want) * 2.0 ** -24
        assert (off <= tol).all(), (float((off / tol).max()), np.argwhere(off > tol)[:5])
    assert np.array_equal(got[..., R:], x.double().cpu().numpy()[0, ..., R:])


@pytest.mark.parametrize("R,D", [(64, 64), (24, 64)])
def test_starts_whose_tokens_pass_32_bits(R, D):
    """start + s is not cut to 32 bits: the tokens behind position 2^31 - 1 go on turning forwards."""
    q, k = inputs(2, 3, 40, D, torch.float32, 25), inputs(2, 1, 40, D, torch.float32, 26)
    f, _ = pasa().rope_frequencies(R)
    for start in (2 ** 31 - 7, torch.tensor([2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")):
        oq, ok = torch.empty_like(q), torch.empty_like(k)
        pasa().rope(q, k, f, start=start, out_q=oq, out_k=ok)
        first = start.long()[:, None] if isinstance(start, torch.Tensor) else start
        pos = (first + torch.arange(40, device="cuda")).expand(2, 40)
        close(oq, q, pos, f)
        close(ok, k, pos, f)
