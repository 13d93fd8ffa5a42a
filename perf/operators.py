"""What is measured of the operators around a key/value cache held in 4 bits: storing rows and
reading them back, decode attention on the cache (with the attention weight each cached row
has gathered), and eviction of the rows that gathered the least.

``run`` computes a pass in plain torch operations, or, where ``own`` is set, through the
framework's entry points. ``exact`` gives the same outputs from the definition in 64 bits.

The cache. A row of D channels is held in groups of 32. With x the fp16 value (for keys
x = fp16(K - shift), one shift per kv head and channel; NaN counts as 0, an infinity as the
largest finite value), a group's scale is max|x| / 7 rounded to 8 significant bits and then
to fp16, its codes are x / scale rounded to the nearest integer (ties to even) in -7 .. 7,
stored as code + 8 in a nibble: byte i of a row holds channel 2i low and 2i + 1 high.
"""
import math
import random

import torch

own = False

GROUP = 32


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------

def listed():
    return [
        # one generated token of each of 8 sequences goes into a 32K-row cache and is read back:
        # the smallest call, where latency counts
        {"name": "store_token_b8", "op": "store", "B": 8, "Hkv": 4, "n": 1, "cap": 32768, "D": 128, "ragged": True},
        # a padded batch of prompt chunks of uneven length, D = 64, one query head per kv head
        {"name": "store_chunk_d64", "op": "store", "B": 2, "Hkv": 5, "n": 577, "cap": 9216, "D": 64, "ragged": True},
        # the prompts of the 8K workload (4 sequences, 8 kv heads) stored whole, read for a prefill
        {"name": "store_prompt_8k", "op": "store", "B": 4, "Hkv": 8, "n": 8192, "cap": 8192, "D": 128, "ragged": False},
        # one decode step of a short conversation: a few hundred keys, latency again
        {"name": "decode_short", "op": "decode", "B": 1, "Hq": 28, "Hkv": 4, "Sq": 1, "Sk": 300, "D": 128,
         "causal": True, "ragged": False, "weights": False},
        # one decode step at the 4K workload's length
        {"name": "decode_4k", "op": "decode", "B": 1, "Hq": 28, "Hkv": 4, "Sq": 1, "Sk": 4096, "D": 128,
         "causal": True, "ragged": False, "weights": False},
        # the decode workload: 8 sequences of 32K keys
        {"name": "decode_32k_b8", "op": "decode", "B": 8, "Hq": 28, "Hkv": 4, "Sq": 1, "Sk": 32768, "D": 128,
         "causal": True, "ragged": False, "weights": False},
        # a batch in service: uneven lengths, an empty and a one-row sequence among them, D = 64
        {"name": "decode_ragged_d64", "op": "decode", "B": 6, "Hq": 16, "Hkv": 2, "Sq": 1, "Sk": 9216, "D": 64,
         "causal": True, "ragged": True, "weights": False},
        # four drafted tokens of each sequence are checked at once
        {"name": "decode_draft4", "op": "decode", "B": 4, "Hq": 32, "Hkv": 8, "Sq": 4, "Sk": 8191, "D": 128,
         "causal": True, "ragged": False, "weights": False},
        # a decode step that also adds up each cached row's attention weight
        {"name": "weights_32k_b4", "op": "decode", "B": 4, "Hq": 28, "Hkv": 4, "Sq": 1, "Sk": 32768, "D": 128,
         "causal": True, "ragged": True, "weights": True},
        # the last 16 prompt rows score the prompt's cache before it is cut down
        {"name": "weights_window16", "op": "decode", "B": 1, "Hq": 28, "Hkv": 4, "Sq": 16, "Sk": 8192, "D": 128,
         "causal": True, "ragged": False, "weights": True},
        # the 32K caches of 8 sequences cut down to 4096 rows each, into new caches
        {"name": "evict_32k_b8", "op": "evict", "B": 8, "Hkv": 4, "Sk": 32768, "D": 128, "budget": 4096, "recent": 256,
         "ragged": False},
        # a small cache cut by a third, uneven lengths, one below the budget
        {"name": "evict_small_d64", "op": "evict", "B": 3, "Hkv": 5, "Sk": 1537, "D": 64, "budget": 1024, "recent": 33,
         "ragged": True},
    ]


def _size(rng, lo, hi):
    """A size spread evenly over the logarithm of its range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["store", "decode", "decode", "weights", "evict"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    B = _size(rng, 1, 12)
    ragged = rng.random() < 0.5
    room = (1 << 20) // (B * Hkv)   # rows of the largest listed cache: 8 x 4 x 32768
    if op == "store":
        n = _size(rng, 1, min(8192, room // 4))
        return {"op": "store", "B": B, "Hkv": Hkv, "n": n, "cap": n + _size(rng, 1, 9000), "D": D, "ragged": ragged}
    Sk = _size(rng, 1 if op != "evict" else 16, min(32768, room))
    if op == "evict":
        budget = _size(rng, 1, Sk)
        return {"op": "evict", "B": B, "Hkv": Hkv, "Sk": Sk, "D": D, "budget": budget,
                "recent": rng.randint(0, budget), "ragged": ragged}
    g = rng.choice([1, 2, 4, 5, 7, 8, 16])
    Sq = rng.choice([1, 1, 1, 2, 3, 5, 8])
    Sk = min(Sk, (7 << 20) // (B * Hkv * g * Sq))   # pairs of the largest listed decode: 8 x 28 x 32768
    Sq = min(Sk, Sq)
    return {"op": "decode", "B": B, "Hq": Hkv * g, "Hkv": Hkv, "Sq": Sq, "Sk": Sk, "D": D, "causal": rng.random() < 0.8,
            "ragged": ragged, "weights": op == "weights"}


def _lengths(case, most):
    """Rows of each sequence, up to `most`, by the case's sizes alone: uneven ones with a full,
    an empty and a one-row sequence first."""
    B = case["B"]
    if not case["ragged"]:
        return [most] * B
    r = random.Random(1000003 * B + most)
    return ([most, 0, min(1, most)] + [r.randint(most // 4, most) for _ in range(B)])[:B]


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------

def _keys(gen, B, H, S, D):
    """Keys with a bias of each kv head and channel along the sequence, and that bias as a
    program has it: the mean of the first rows."""
    bias = 10.0 * torch.randn((B, H, 1, D), generator=gen, device="cuda")
    k = (bias + torch.randn((B, H, S, D), generator=gen, device="cuda")).half()
    return k, k[:, :, :128].float().mean(2).half()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    B, H, D = case["B"], case["Hkv"], case["D"]
    st = dict(case)
    if case["op"] == "store":
        n, cap = case["n"], case["cap"]
        counts = _lengths(case, n)
        k, shift = _keys(gen, B, H, n, D)
        st.update(k=k, v=torch.randn((B, H, n, D), generator=gen, device="cuda").half(), shift=shift,
                  counts=torch.tensor(counts, dtype=torch.int32, device="cuda"),
                  start=torch.randint(0, cap - n + 1, (B,), generator=gen, device="cuda").int(),
                  cache=_cache(B, H, cap, D), out_k=torch.zeros_like(k), out_v=torch.zeros_like(k))
        return st
    S = case["Sk"]
    lengths = torch.tensor(_lengths(case, S), dtype=torch.int32, device="cuda")
    k, shift = _keys(gen, B, H, S, D)
    k4, ks = _quantise(k, shift)
    del k
    v4, vs = _quantise(torch.randn((B, H, S, D), generator=gen, device="cuda").half(), None)
    past = torch.arange(S, device="cuda")[None, None, :, None] >= lengths[:, None, None, None]
    ks.masked_fill_(past, float("nan"))   # rows past a sequence's last hold whatever was there
    vs.masked_fill_(past, float("inf"))
    weights = torch.rand((B, H, S), generator=gen, device="cuda").pow(8) / 64
    weights = torch.where(past[..., 0], torch.zeros_like(weights), weights)
    st.update(cache=(k4, ks, v4, vs), lengths=lengths, shift=shift, acc=weights)
    if case["op"] == "decode":
        q = torch.randn((B, case["Hq"], case["Sq"], D), generator=gen, device="cuda").half()
        st.update(q=q, out=torch.empty_like(q), lse=torch.empty(q.shape[:3], device="cuda"))
        return st
    # weights of rows that were never looked at are equal (0), and some come in equal pairs
    weights[:, :, 1::7] = 0
    weights[:, :, 3::11] = weights[:, :, 2:-1:11][:, :, :weights[:, :, 3::11].shape[2]]
    N = case["budget"]
    st.update(dst=_cache(B, H, N, D), dst_acc=torch.zeros((B, H, N), device="cuda"),
              out_k=torch.zeros((B, H, N, D), device="cuda", dtype=torch.float16),
              out_v=torch.zeros((B, H, N, D), device="cuda", dtype=torch.float16))
    return st


def _cache(B, H, cap, D):
    codes = lambda: torch.zeros((B, H, cap, D // 2), dtype=torch.uint8, device="cuda")               # noqa: E731
    scales = lambda: torch.zeros((B, H, cap, D // GROUP), dtype=torch.float16, device="cuda")        # noqa: E731
    return codes(), scales(), codes(), scales()


# --------------------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------------------

def _quantise(x, shift):
    """(codes, scales) of fp16 rows [B, H, S, D]."""
    if shift is not None:
        x = (x.float() - shift.float()[:, :, None]).half()
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=65504.0, neginf=-65504.0)
    x = x.unflatten(-1, (-1, GROUP))
    s = x.abs().amax(-1, keepdim=True) / 7
    m, e = torch.frexp(s)
    s = torch.ldexp(torch.round(m * 256), e - 8).half().float()
    c = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, 1.0)).clamp(-7, 7), 0.0)
    c = (c.flatten(-2) + 8).to(torch.uint8).unflatten(-1, (-1, 2))
    return c[..., 0] | (c[..., 1] << 4), s[..., 0].half()


def _values(codes, scales):
    """fp32 values of cache rows."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    return (c.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _read(k4, ks, v4, vs, shift):
    return (_values(k4, ks) + shift.float()[:, :, None]).half(), _values(v4, vs).half()


def _plain_store(st):
    n = st["n"]
    row = torch.arange(n, device="cuda")
    at = (st["start"].long()[:, None] + row)[:, None, :, None]
    there = (row < st["counts"][:, None])[:, None, :, None]
    rows = lambda x: at.expand(-1, st["Hkv"], -1, x.shape[-1])                                       # noqa: E731
    k4, ks = _quantise(st["k"], st["shift"])
    v4, vs = _quantise(st["v"], None)
    k4, ks, v4, vs = (c.scatter_(2, rows(c), torch.where(there, x, c.gather(2, rows(c))))
                      for c, x in zip(st["cache"], (k4, ks, v4, vs)))
    k, v = _read(*(c.gather(2, rows(c)) for c in st["cache"]), st["shift"])
    return torch.where(there, k, st["out_k"]), torch.where(there, v, st["out_v"])


def _plain_decode(st):
    B, Hq, H, Sq, S, D = (st[x] for x in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
    k4, ks, v4, vs = st["cache"]
    scale = 1 / math.sqrt(D)
    q = st["q"].float().view(B, H, Hq // H * Sq, D)
    j = torch.arange(S, device="cuda")
    length = st["lengths"][:, None, None]
    seen = (j < length).expand(B, Sq, S)
    if st["causal"]:
        seen = seen & (j <= torch.arange(Sq, device="cuda")[:, None] + length - Sq)
    seen = seen.repeat(1, Hq // H, 1)[:, None]                       # [B, 1, g * Sq, S]
    x = (scale * (q @ _values(k4, ks).transpose(2, 3))).masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    v = _values(v4, vs).masked_fill((j >= length)[..., None], 0.0)
    lse = (m + torch.log(total))[..., 0] + scale * (q @ st["shift"].float()[..., None])[..., 0]
    out = {"o": (p @ v).half().view(B, Hq, Sq, D), "lse": lse.view(B, Hq, Sq)}
    if st["weights"]:
        out["weights"] = st["acc"].add_(p.sum(2))
    return out


def _plain_evict(st):
    S, N = st["Sk"], st["budget"]
    w = st["acc"]
    j = torch.arange(S, device="cuda")
    length = st["lengths"][:, None, None]
    rank = ((j < length).int() + (j >= length - st["recent"]).int() * (j < length).int()).expand(w.shape)
    order = torch.sort(torch.nan_to_num(w, nan=-math.inf, posinf=math.inf), dim=2, descending=True, stable=True)[1]
    again = torch.sort(rank.gather(2, order), dim=2, descending=True, stable=True)[1]
    kept = order.gather(2, again)[:, :, :N]
    kept = torch.where(rank.gather(2, kept) > 0, kept, S).sort(dim=2)[0]
    there = kept < S
    at = torch.where(there, kept, 0)
    rows = [torch.where(there[..., None], c.gather(2, at[..., None].expand(-1, -1, -1, c.shape[-1])), d)
            for c, d in zip(st["cache"], st["dst"])]
    k, v = _read(*rows, st["shift"])
    return {"index": torch.where(there, kept, -1).int(), "lengths": st["lengths"].clamp(max=N),
            "weights": torch.where(there, w.gather(2, at), 0.0),
            "k": torch.where(there[..., None], k, st["out_k"]), "v": torch.where(there[..., None], v, st["out_v"])}


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------

def run(st):
    if not own:
        return {"store": _plain_store, "decode": _plain_decode, "evict": _plain_evict}[st["op"]](st)
    import precision_flashattention_numerics_gb300 as pasa

    if st["op"] == "store":
        pasa.kv4_append(st["k"], st["v"], *st["cache"], start=st["start"], counts=st["counts"], shift=st["shift"])
        return pasa.kv4_read(*st["cache"], st["n"], start=st["start"], counts=st["counts"], shift=st["shift"],
                             out_k=st["out_k"], out_v=st["out_v"])
    if st["op"] == "decode":
        acc = st["acc"] if st["weights"] else None
        o, lse = pasa.attn_fwd_decode_kv4(st["q"], *st["cache"], causal=st["causal"], shift=st["shift"],
                                          lengths=st["lengths"], weights=acc, out=st["out"], lse=st["lse"])
        return {"o": o, "lse": lse} if acc is None else {"o": o, "lse": lse, "weights": acc}
    index, lengths = pasa.cache_evict(st["cache"], st["acc"], st["budget"], st["recent"], lengths=st["lengths"],
                                      out=st["dst"], out_weights=st["dst_acc"])
    k, v = pasa.kv4_read(*st["dst"], st["budget"], counts=lengths, shift=st["shift"], out_k=st["out_k"],
                         out_v=st["out_v"])
    return {"index": index, "lengths": lengths, "weights": st["dst_acc"], "k": k, "v": v}


def work(case):
    """Each input once and each output once: a cache row is D / 2 bytes of codes and D / 16 of
    scales, for keys and for values."""
    B, H, D = case["B"], case["Hkv"], case["D"]
    row = 2 * (D // 2 + D // 16)
    if case["op"] == "store":
        rows = H * sum(_lengths(case, case["n"]))
        return {"bytes": rows * (4 * D + row + 4 * D) + B * H * 2 * D, "flops": rows * 2 * D * 6}
    rows = H * sum(_lengths(case, case["Sk"]))
    if case["op"] == "decode":
        g, Sq = case["Hq"] // H, case["Sq"]
        some = B * case["Hq"] * Sq * (4 * D + 4) + B * H * 2 * D
        return {"bytes": rows * (row + (8 if case["weights"] else 0)) + some, "flops": rows * g * Sq * 4 * D}
    kept = H * sum(min(x, case["budget"]) for x in _lengths(case, case["Sk"]))
    return {"bytes": rows * 4 + kept * (2 * row + 4 + 4 + 4 * D), "flops": rows * 4 + kept * 4 * D}


# --------------------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------------------

def _to_bits(x, bits, floor):
    """x rounded (ties to even) to `bits` significant bits, and to multiples of `floor`."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1e-30))) + 1 - bits)
    step = torch.where(x.abs() >= step * 2.0 ** bits, step * 2, torch.where(x.abs() < step * 2.0 ** (bits - 1), step / 2, step))
    x = torch.round(x / step) * step
    return torch.where(x.abs() < floor * 2.0 ** bits, torch.round(x / floor) * floor, x)


def _exact_held(x, shift):
    """What the cache holds of fp16 rows, as 64-bit values."""
    x = x.double()
    if shift is not None:
        x = _to_bits(x - shift.double()[:, :, None], 11, 2.0 ** -24)
    x = torch.nan_to_num(x, nan=0.0).clamp(-65504.0, 65504.0)
    x = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    s = x.abs().max(-1, keepdim=True).values / 7
    s = _to_bits(_to_bits(s, 8, 2.0 ** -100), 11, 2.0 ** -24)
    c = torch.where(s > 0, torch.round(x / s.clamp(min=2.0 ** -25)), torch.zeros_like(x)).clamp(-7, 7)
    return (c * s).reshape(*x.shape[:-2], -1)


def _exact_values(codes, scales):
    c = codes.to(torch.int64)
    low, high = c % 16, c // 16
    c = torch.empty((*c.shape[:-1], 2 * c.shape[-1]), dtype=torch.float64, device=c.device)
    c[..., 0::2], c[..., 1::2] = low - 8, high - 8
    return c * scales.double().repeat_interleave(GROUP, dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    B, H, D = case["B"], case["Hkv"], case["D"]
    if case["op"] == "store":
        k = _exact_held(st["k"], st["shift"]) + st["shift"].double()[:, :, None]
        v = _exact_held(st["v"], None)
        for b, n in enumerate(_lengths(case, case["n"])):
            k[b, :, n:] = 0
            v[b, :, n:] = 0
        return k, v
    lengths = _lengths(case, case["Sk"])
    k4, ks, v4, vs = st["cache"]
    if case["op"] == "decode":
        Sq, g = case["Sq"], case["Hq"] // H
        o = torch.zeros((B, H, g, Sq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, H, g, Sq), -math.inf, dtype=torch.float64, device="cuda")
        acc = st["acc"].double()
        for b, n in enumerate(lengths):
            for i in range(Sq):
                see = min(n, i + n - Sq + 1) if case["causal"] else n
                if see <= 0:
                    continue
                q = st["q"][b].double().view(H, g, Sq, D)[:, :, i]
                x = torch.einsum("hgd,hjd->hgj", q, _exact_values(k4[b, :, :see], ks[b, :, :see])) / math.sqrt(D)
                total = torch.logsumexp(x, -1)
                p = torch.exp(x - total[..., None])
                o[b, :, :, i] = torch.einsum("hgj,hjd->hgd", p, _exact_values(v4[b, :, :see], vs[b, :, :see]))
                lse[b, :, :, i] = total + torch.einsum("hgd,hd->hg", q, st["shift"][b].double()) / math.sqrt(D)
                acc[b, :, :see] += p.sum(1)
        got = {"o": o.view(B, H * g, Sq, D), "lse": lse.view(B, H * g, Sq)}
        return {**got, "weights": acc} if case["weights"] else got
    N, recent = case["budget"], case["recent"]
    k = torch.zeros((B, H, N, D), dtype=torch.float64, device="cuda")
    v, w = torch.zeros_like(k), torch.zeros((B, H, N), dtype=torch.float64, device="cuda")
    index = torch.full((B, H, N), -1, dtype=torch.int32)
    acc = st["acc"].double().cpu().numpy()
    for b, n in enumerate(lengths):
        old = max(0, n - recent)
        for h in range(H):
            if n <= N:
                keep = list(range(n))
            else:
                best = sorted(range(old), key=lambda j, a=acc[b, h]: (-a[j], j))[:N - (n - old)]
                keep = sorted(best) + list(range(old, n))
            at = torch.tensor(keep, dtype=torch.long)
            index[b, h, :len(keep)] = at.int()
            at = at.cuda()
            k[b, h, :len(keep)] = _exact_values(k4[b, h, at], ks[b, h, at]) + st["shift"][b, h].double()
            v[b, h, :len(keep)] = _exact_values(v4[b, h, at], vs[b, h, at])
            w[b, h, :len(keep)] = st["acc"][b, h, at].double()
    return {"index": index.cuda(), "lengths": torch.tensor([min(n, N) for n in lengths], dtype=torch.int32),
            "weights": w, "k": k, "v": v}
