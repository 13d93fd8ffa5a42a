"""What is measured of the operators that a serving loop runs around the attention kernels: rotary
positions, attention over packed prompts of uneven lengths, attention for a tree of drafted tokens
over the 4-bit cache, and storing the drafted rows that were accepted.

``run`` computes a pass in plain torch operations, or, where ``own`` is set, through the
framework's entry points. ``exact`` gives the same outputs from the definition in 64 bits.

Rotary positions. Channels are paired, (i, i + R/2) in the half layout and (2i, 2i + 1) in the
interleaved one, for the first R of D channels; a pair (x, y) of a token at position p becomes
(x cos a - y sin a, x sin a + y cos a) * mscale with a = p * inv_freq[i]; the other channels stay.

Packed prompts. Sequence s has the query rows cu_q[s] .. cu_q[s + 1] and the key rows cu_k[s] ..
cu_k[s + 1] of token-major tensors; query i of n sees keys j <= i + m - n of its m (causal).

Tree. Node i of a sequence sees the cache's rows, its ancestors (parents[i], and so on up to -1)
and itself. The cache holds a row of D channels in groups of 32: with x = fp16(K - shift) (values:
V), a group's scale is max|x| / 7 rounded to 8 significant bits and then to fp16, its codes are
x / scale rounded to the nearest integer (ties to even) in -7 .. 7, stored as code + 8 in a nibble.
"""
import math
import random

import torch

own = False

GROUP = 32
HALF = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------

def listed():
    return [
        # the new token of each of 8 sequences, somewhere in a 32K context: the smallest call
        {"name": "rope_token_b8", "op": "rope", "T": 8, "Hq": 28, "Hkv": 4, "D": 128, "R": 128, "interleaved": False,
         "src": "f16", "dst": "f16", "far": 32768, "mscale": 1.0, "inverse": False},
        # q and k of a 32K prompt, views of the projection's one output
        {"name": "rope_prompt_32k", "op": "rope", "T": 32768, "Hq": 28, "Hkv": 4, "D": 128, "R": 128, "interleaved": False,
         "src": "f16", "dst": "f16", "far": 32768, "mscale": 1.0, "inverse": False},
        # half of the channels turn, pairs side by side, far positions, projections in bf16
        {"name": "rope_partial_d64", "op": "rope", "T": 9217, "Hq": 10, "Hkv": 5, "D": 64, "R": 32, "interleaved": True,
         "src": "bf16", "dst": "f16", "far": 1000000, "mscale": 1.1386, "inverse": False},
        # many short prompts at once, some of one token, one empty
        {"name": "packed_short", "op": "packed", "Hq": 28, "Hkv": 4, "D": 128, "mode": 1, "causal": True, "tail": 7,
         "lens_q": "33,1,200,17,64,0,128,5,90,150,3,41,77,129,12,1,180,60,25,110", "lens_k": ""},
        # prompts of a mixed batch, a long one among them, 32K tokens in all
        {"name": "packed_32k", "op": "packed", "Hq": 28, "Hkv": 4, "D": 128, "mode": 1, "causal": True, "tail": 1,
         "lens_q": "2048,16384,4097,1,9000,577,660,0", "lens_k": ""},
        # D = 64, a query head for each kv head, scores in fp16 (the library's default)
        {"name": "packed_d64", "op": "packed", "Hq": 5, "Hkv": 5, "D": 64, "mode": 0, "causal": True, "tail": 0,
         "lens_q": "9216,577,4097,2300", "lens_k": ""},
        # chunks of prompts on the keys of what went before, one generated token among them
        {"name": "packed_chunks", "op": "packed", "Hq": 32, "Hkv": 8, "D": 128, "mode": 1, "causal": True, "tail": 0,
         "lens_q": "512,1,512,300", "lens_k": "8191,2049,512,4396"},
        # eight drafted tokens of a short conversation: latency
        {"name": "tree_short", "op": "tree", "B": 1, "Hq": 28, "Hkv": 4, "Sq": 8, "Sk": 300, "D": 128, "ragged": False},
        # 16 drafted tokens of each of 8 sequences of 32K keys
        {"name": "tree_32k_b8", "op": "tree", "B": 8, "Hq": 28, "Hkv": 4, "Sq": 16, "Sk": 32768, "D": 128, "ragged": False},
        # wide trees of a batch in service, uneven lengths and node counts, D = 64
        {"name": "tree_ragged_d64", "op": "tree", "B": 6, "Hq": 16, "Hkv": 2, "Sq": 61, "Sk": 9216, "D": 64, "ragged": True},
        # the accepted rows of 8 drafted tokens of one sequence go into its cache: latency
        {"name": "accept_b1", "op": "accept", "B": 1, "Hkv": 4, "Sq": 8, "P": 5, "cap": 32768, "D": 128, "ragged": False},
        # a large batch, uneven numbers of accepted rows
        {"name": "accept_b64", "op": "accept", "B": 64, "Hkv": 8, "Sq": 64, "P": 33, "cap": 1100, "D": 128, "ragged": True},
    ]


def _size(rng, lo, hi):
    """A size spread evenly over the logarithm of its range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "packed", "packed", "tree", "tree", "accept"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 4, 5, 7, 8, 16])
    if op == "rope":
        src = rng.choice(["f16", "f16", "bf16", "f32"])
        far = _size(rng, 64, 4000000)
        return {"op": "rope", "T": _size(rng, 1, 32768 * 32 // (Hkv * (g + 1)) // (2 if src == "f32" else 1)), "Hq": Hkv * g,
                "Hkv": Hkv, "D": D, "R": rng.choice([D, D, D // 2, D // 4, 24]), "interleaved": rng.random() < 0.5, "src": src,
                "dst": rng.choice([src, "f16"]), "far": far, "mscale": rng.choice([1.0, 1.0, 0.9, 1.2079]),
                "inverse": rng.random() < 0.3}
    if op == "packed":
        chunks = rng.random() < 0.4
        longest = _size(rng, 1, 16384)
        lens_q, lens_k, room = [], [], (5 << 30) // (Hkv * g)   # pairs of the largest listed case
        for _ in range(_size(rng, 1, 40)):
            n = 0 if rng.random() < 0.05 else _size(rng, 1, longest)
            m = n + _size(rng, 1, longest) if chunks and rng.random() < 0.8 else n
            if n * (2 * m - n) // 2 > room or sum(lens_k) + m > 40000:
                continue
            room -= n * (2 * m - n) // 2
            lens_q.append(n), lens_k.append(m)
        if not sum(lens_q):
            lens_q, lens_k = lens_q + [5], lens_k + [9 if chunks else 5]
        causal = rng.random() < 0.8
        mode = rng.choice([0, 1, 1, 3])
        if not causal and 2 * sum(n * m for n, m in zip(lens_q, lens_k)) * Hkv * g > 5 << 30:
            causal = True
        return {"op": "packed", "Hq": Hkv * g, "Hkv": Hkv, "D": D, "mode": mode, "causal": causal, "tail": rng.randint(0, 40),
                "lens_q": ",".join(map(str, lens_q)), "lens_k": ",".join(map(str, lens_k)) if chunks else ""}
    B = _size(rng, 1, 12)
    Sq = _size(rng, 1, 64)
    ragged = rng.random() < 0.5
    if op == "accept":
        return {"op": "accept", "B": _size(rng, 1, 64), "Hkv": Hkv, "Sq": Sq, "P": rng.randint(1, Sq), "cap": _size(rng, 64, 2000),
                "D": D, "ragged": ragged}
    rows = g * Sq
    Sk = _size(rng, 1, max(1, min(32768, (1 << 20) // (B * Hkv), (1 << 20) * 112 // (B * Hkv * rows))))
    return {"op": "tree", "B": B, "Hq": Hkv * g, "Hkv": Hkv, "Sq": Sq, "Sk": Sk, "D": D, "ragged": ragged}


def _uneven(case, most):
    """`most` for each sequence or, by the case's sizes alone, uneven numbers with a full one, none
    and 1 first."""
    B = case["B"]
    if not case["ragged"]:
        return [most] * B
    r = random.Random(1000003 * B + most)
    return ([most, 0, min(1, most)] + [r.randint(most // 4, most) for _ in range(B)])[:B]


def _accepted(case):
    return _uneven(case, case["P"])


def _counts(case):
    """Nodes of each sequence's tree, the full one last."""
    return _uneven(case, case["Sq"])[::-1]


def _lens(case):
    q = [int(x) for x in case["lens_q"].split(",")]
    return q, [int(x) for x in case["lens_k"].split(",")] if case["lens_k"] else q


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------

def _keys(gen, B, H, S, D, bias=None):
    """Keys with a bias of each kv head and channel along the sequence, and that bias."""
    if bias is None:
        bias = 10.0 * torch.randn((B, H, 1, D), generator=gen, device="cuda")
    return (bias + torch.randn((B, H, S, D), generator=gen, device="cuda")).half(), bias


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _cache(B, H, cap, D):
    codes = lambda: torch.zeros((B, H, cap, D // 2), dtype=torch.uint8, device="cuda")               # noqa: E731
    scales = lambda: torch.zeros((B, H, cap, D // GROUP), dtype=torch.float16, device="cuda")        # noqa: E731
    return codes(), scales(), codes(), scales()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")                         # noqa: E731
    H, D = case["Hkv"], case["D"]
    st = dict(case)
    if case["op"] == "rope":
        T, Hq, R = case["T"], case["Hq"], case["R"]
        qkv = normal(T, Hq + 2 * H, D).to(HALF[case["src"]])   # a projection's output: q, k and v side by side
        inv_freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        positions = torch.randint(0, case["far"], (T,), generator=gen, device="cuda").int()
        st.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], inv_freq=inv_freq, positions=positions,
                  out_q=torch.empty((T, Hq, D), device="cuda", dtype=HALF[case["dst"]]),
                  out_k=torch.empty((T, H, D), device="cuda", dtype=HALF[case["dst"]]))
        return st
    if case["op"] == "packed":
        lens_q, lens_k = _lens(case)
        at_q, at_k = _offsets(lens_q), _offsets(lens_k)
        Tq, Tk = at_q[-1] + case["tail"], at_k[-1] + case["tail"]
        q = normal(Tq, case["Hq"], D).half()
        kv = torch.empty((Tk, 2 * H, D), dtype=torch.float16, device="cuda")   # k and v side by side
        kv[:, :H] = 10.0 * normal(1, H, D) + normal(Tk, H, D)
        kv[:, H:] = normal(Tk, H, D)
        kv[at_k[-1]:] = float("nan")   # rows behind the last sequence hold whatever was there
        cu = lambda at: torch.tensor(at, dtype=torch.int32, device="cuda")                           # noqa: E731
        st.update(q=q, k=kv[:, :H], v=kv[:, H:], cu_q=cu(at_q), cu_k=cu(at_k), at_q=at_q, at_k=at_k,
                  out=torch.zeros_like(q), lse=torch.zeros((case["Hq"], Tq), device="cuda"))
        return st
    B, Sq = case["B"], case["Sq"]
    if case["op"] == "accept":
        cap, P = case["cap"], case["P"]
        k, bias = _keys(gen, B, H, Sq, D)
        # the accepted nodes of a tree, in order of depth
        path = torch.rand((B, Sq), generator=gen, device="cuda").argsort(1)[:, :P].sort(1)[0].int()
        st.update(k=k, v=normal(B, H, Sq, D).half(), shift=bias[:, :, 0].half(), path=path,
                  counts=torch.tensor(_accepted(case), dtype=torch.int32, device="cuda"),
                  start=torch.randint(0, cap - P + 1, (B,), generator=gen, device="cuda").int(), cache=_cache(B, H, cap, D),
                  out_k=torch.zeros((B, H, P, D), dtype=torch.float16, device="cuda"),
                  out_v=torch.zeros((B, H, P, D), dtype=torch.float16, device="cuda"))
        return st
    S = case["Sk"]
    lengths = torch.tensor(_uneven(case, S), dtype=torch.int32, device="cuda")
    k, bias = _keys(gen, B, H, S, D)
    shift = bias[:, :, 0].half()
    k4, ks = _quantise(k, shift)
    del k
    v4, vs = _quantise(normal(B, H, S, D).half(), None)
    past = torch.arange(S, device="cuda")[None, None, :, None] >= lengths[:, None, None, None]
    ks.masked_fill_(past, float("nan"))   # rows past a sequence's last hold whatever was there
    vs.masked_fill_(past, float("inf"))
    knew, _ = _keys(gen, B, H, Sq, D, bias)
    i = torch.arange(Sq, device="cuda")
    parents = (torch.rand((B, Sq), generator=gen, device="cuda") * (i + 1)).int().clamp(max=i) - 1
    q = normal(B, case["Hq"], Sq, D).half()
    st.update(q=q, k=knew, v=normal(B, H, Sq, D).half(), cache=(k4, ks, v4, vs), shift=shift, lengths=lengths,
              parents=parents.int(), counts=torch.tensor(_counts(case), dtype=torch.int32, device="cuda"),
              out=torch.empty_like(q), lse=torch.empty(q.shape[:3], device="cuda"))
    return st


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


def _plain_rope(st):
    R = st["R"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]           # 64 bits: a far position's angle
    sign = -1.0 if st["inverse"] else 1.0
    cos = (torch.cos(angle) * st["mscale"]).float()[:, None]
    sin = (torch.sin(angle) * st["mscale"] * sign).float()[:, None]

    def turn(x, to):
        x = x.float()
        turned, rest = x[..., :R], x[..., R:]
        x0, x1 = (turned[..., 0::2], turned[..., 1::2]) if st["interleaved"] else turned.chunk(2, -1)
        y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
        y = torch.stack([y0, y1], -1).flatten(-2) if st["interleaved"] else torch.cat([y0, y1], -1)
        return to.copy_(torch.cat([y, rest], -1))

    return turn(st["q"], st["out_q"]), turn(st["k"], st["out_k"])


def _plain_packed(st):
    Hq, H, D = st["Hq"], st["Hkv"], st["D"]
    g, scale = Hq // H, 1 / math.sqrt(D)
    # a sequence at a time, and as many of its queries as 2^29 scores allow: a batch padded to its
    # longest prompt would not fit
    for a, b, c, d in zip(st["at_q"], st["at_q"][1:], st["at_k"], st["at_k"][1:]):
        m, n = d - c, b - a
        if n == 0:
            continue
        k = st["k"][c:d].float().permute(1, 2, 0)[:, None]                # [H, 1, D, m]
        v = st["v"][c:d].float().transpose(0, 1)[:, None]
        rows = max(1, (1 << 29) // (Hq * max(1, m)))
        for i0 in range(0, n, rows):
            i1 = min(n, i0 + rows)
            q = st["q"][a + i0:a + i1].float().transpose(0, 1).unflatten(0, (H, g))
            x = scale * (q @ k)                                           # [H, g, rows, m]
            if st["causal"]:
                i = torch.arange(i0, i1, device="cuda")[:, None]
                x = x.masked_fill(torch.arange(m, device="cuda") > i + m - n, -math.inf)
            total = torch.logsumexp(x, -1) if m else torch.full(x.shape[:3], -math.inf, device="cuda")
            p = torch.exp(x - torch.where(total == -math.inf, 0.0, total)[..., None])
            st["out"][a + i0:a + i1] = (p @ v).flatten(0, 1).transpose(0, 1).half()
            st["lse"][:, a + i0:a + i1] = total.flatten(0, 1)
    # with scores held in fp16 the log-sum-exp is as good as they are, and not asked for
    return {"o": st["out"], "lse": st["lse"]} if st["mode"] != 0 else {"o": st["out"]}


def _ancestors(parents, counts):
    """[B, Sq, Sq]: whether node i sees node j, its ancestor or itself."""
    B, Sq = parents.shape
    i = torch.arange(Sq, device="cuda")
    see = (i[:, None] == i).float() + (parents[..., None] == i).float()
    for _ in range(max(1, (Sq - 1).bit_length())):                        # paths of 1, 2, 4 ... steps
        see = ((see @ see) > 0).float()
    there = i < counts[:, None]
    return (see > 0) & there[:, :, None] & there[:, None]


def _plain_tree(st):
    B, Hq, H, Sq, S, D = (st[x] for x in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
    g, scale = Hq // H, 1 / math.sqrt(D)
    k4, ks, v4, vs = st["cache"]
    shift = st["shift"].float()[:, :, None]
    past = (torch.arange(S, device="cuda") >= st["lengths"][:, None])[:, None, None]
    there = (torch.arange(Sq, device="cuda") < st["counts"][:, None]).repeat(1, g)[:, None, :, None]
    q = st["q"].float().view(B, H, g * Sq, D)
    seen = _ancestors(st["parents"], st["counts"]).repeat(1, g, 1)[:, None]
    x = torch.cat([(scale * (q @ _values(k4, ks).transpose(2, 3))).masked_fill(past, -math.inf),
                   (scale * (q @ (st["k"].float() - shift).transpose(2, 3))).masked_fill(~seen, -math.inf)], -1)
    x = x.masked_fill(~there, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    v = torch.cat([_values(v4, vs).masked_fill(past.transpose(2, 3), 0.0), st["v"].float()], 2)
    lse = (m + torch.log(total))[..., 0] + scale * (q @ shift.transpose(2, 3))[..., 0]
    return {"o": (p @ v).half().view(B, Hq, Sq, D), "lse": lse.view(B, Hq, Sq)}


def _plain_accept(st):
    P, H = st["P"], st["Hkv"]
    i = torch.arange(P, device="cuda")
    there = (i < st["counts"][:, None])[:, None, :, None]
    at = (st["start"].long()[:, None] + i)[:, None, :, None]
    rows = lambda x: at.expand(-1, H, -1, x.shape[-1])                                               # noqa: E731
    path = st["path"].long()[:, None, :, None].expand(-1, H, -1, st["D"])
    new = (*_quantise(st["k"].gather(2, path), st["shift"]), *_quantise(st["v"].gather(2, path), None))
    k4, ks, v4, vs = (c.scatter_(2, rows(c), torch.where(there, x, c.gather(2, rows(c)))).gather(2, rows(c))
                      for c, x in zip(st["cache"], new))
    k = (_values(k4, ks) + st["shift"].float()[:, :, None]).half()
    return torch.where(there, k, st["out_k"]), torch.where(there, _values(v4, vs).half(), st["out_v"])


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------

def run(st):
    if not own:
        return {"rope": _plain_rope, "packed": _plain_packed, "tree": _plain_tree, "accept": _plain_accept}[st["op"]](st)
    import precision_flashattention_numerics_gb300 as pasa

    if st["op"] == "rope":
        return pasa.rope(st["q"], st["k"], st["inv_freq"], positions=st["positions"], interleaved=st["interleaved"],
                         mscale=st["mscale"], inverse=st["inverse"], out_q=st["out_q"], out_k=st["out_k"])
    if st["op"] == "packed":
        want = st["mode"] != 0
        o, lse = pasa.attn_fwd_packed(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], causal=st["causal"], mode=st["mode"],
                                      out=st["out"], lse=st["lse"] if want else None, return_lse=want)
        return {"o": o, "lse": lse} if want else {"o": o}
    if st["op"] == "tree":
        o, lse = pasa.attn_fwd_tree_kv4(st["q"], st["k"], st["v"], *st["cache"], st["parents"], lengths=st["lengths"],
                                        counts=st["counts"], shift=st["shift"], out=st["out"], lse=st["lse"])
        return {"o": o, "lse": lse}
    pasa.kv4_append(st["k"], st["v"], *st["cache"], start=st["start"], counts=st["counts"], shift=st["shift"], rows=st["path"])
    return pasa.kv4_read(*st["cache"], st["P"], start=st["start"], counts=st["counts"], shift=st["shift"], out_k=st["out_k"],
                         out_v=st["out_v"])


def work(case):
    """Each input once and each output once: a cache row is D / 2 bytes of codes and D / 16 of
    scales, for keys and for values."""
    H, D = case["Hkv"], case["D"]
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if case["op"] == "rope":
        rows = case["T"] * (case["Hq"] + H)
        return {"bytes": rows * D * (size[case["src"]] + size[case["dst"]]) + case["T"] * 4 + case["R"] * 4,
                "flops": rows * case["R"] * 3}
    if case["op"] == "packed":
        lens_q, lens_k = _lens(case)
        pairs = sum(n * m if not case["causal"] else sum(max(0, i + m - n + 1) for i in range(n)) for n, m in zip(lens_q, lens_k))
        lse = 4 if case["mode"] != 0 else 0
        return {"bytes": sum(lens_q) * case["Hq"] * (4 * D + lse) + sum(m for n, m in zip(lens_q, lens_k) if n) * H * 4 * D,
                "flops": pairs * case["Hq"] * 4 * D}
    row = 2 * (D // 2 + D // 16)
    if case["op"] == "accept":
        rows = H * sum(_accepted(case))
        return {"bytes": rows * (4 * D + row + 4 * D) + case["B"] * H * 2 * D, "flops": rows * 2 * D * 6}
    counts, g = _counts(case), case["Hq"] // H
    keys = [n if c else 0 for n, c in zip(_uneven(case, case["Sk"]), counts)]
    some = case["B"] * case["Hq"] * case["Sq"] * (4 * D + 4) + case["B"] * H * 2 * D
    pairs = sum(g * c * (n + (c + 1) // 2) for n, c in zip(keys, counts))
    return {"bytes": H * (sum(keys) * row + sum(counts) * 4 * D) + some, "flops": H * pairs * 4 * D}


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


def _exact_rope(x, st):
    """A rotation by the complex exponential."""
    R = st["R"]
    i = torch.arange(R // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + R // 2)
    turn = torch.polar(torch.full((st["T"], R // 2), float(st["mscale"]), dtype=torch.float64, device="cuda"),
                       st["positions"].double()[:, None] * st["inv_freq"] * (-1 if st["inverse"] else 1))
    y = x.double().clone()
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    H, D = case["Hkv"], case["D"]
    if case["op"] == "rope":
        return _exact_rope(st["q"], st), _exact_rope(st["k"], st)
    if case["op"] == "packed":
        lens_q, lens_k = _lens(case)
        g = case["Hq"] // H
        if sum(n * m for n, m in zip(lens_q, lens_k)) * case["Hq"] * 4 * D > 1.2e13:
            return None
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
        for s, (n, m) in enumerate(zip(lens_q, lens_k)):
            a, c = st["at_q"][s], st["at_k"][s]
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                last = min(m, i1 + m - n) if case["causal"] else m
                for h in range(H):
                    q = st["q"][a + i0:a + i1, h * g:(h + 1) * g].double()
                    if last <= 0:
                        lse[h * g:(h + 1) * g, a + i0:a + i1] = -math.inf
                        continue
                    k, v = st["k"][c:c + last, h].double(), st["v"][c:c + last, h].double()
                    x = (q.reshape(-1, D) @ k.T).view(i1 - i0, g, last) / math.sqrt(D)
                    if case["causal"]:
                        i = torch.arange(i0, i1, device="cuda")[:, None, None]
                        x = torch.where(torch.arange(last, device="cuda") <= i + m - n, x, -math.inf)
                    total = torch.logsumexp(x, -1)
                    p = torch.exp(x - torch.where(total == -math.inf, 0.0, total)[..., None])
                    o[a + i0:a + i1, h * g:(h + 1) * g] = (p.view(-1, last) @ v).view(i1 - i0, g, D)
                    lse[h * g:(h + 1) * g, a + i0:a + i1] = total.T
        return {"o": o, "lse": lse} if case["mode"] != 0 else {"o": o}
    B, Sq = case["B"], case["Sq"]
    if case["op"] == "accept":
        k = torch.zeros((B, H, case["P"], D), dtype=torch.float64, device="cuda")
        v = torch.zeros_like(k)
        kept_k, kept_v = _exact_held(st["k"], st["shift"]) + st["shift"].double()[:, :, None], _exact_held(st["v"], None)
        path = st["path"].tolist()
        for b, n in enumerate(_accepted(case)):
            for i in range(n):
                k[b, :, i], v[b, :, i] = kept_k[b, :, path[b][i]], kept_v[b, :, path[b][i]]
        return k, v
    g = case["Hq"] // H
    o = torch.zeros((B, H, g, Sq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, g, Sq), -math.inf, dtype=torch.float64, device="cuda")
    k4, ks, v4, vs = st["cache"]
    parents = st["parents"].tolist()
    for b, (n, c) in enumerate(zip(_uneven(case, case["Sk"]), _counts(case))):
        if c == 0:
            continue
        see = torch.zeros((c, n + c), dtype=torch.bool)
        see[:, :n] = True
        for i in range(c):
            j = i
            while j >= 0:
                see[i, n + j] = True
                j = parents[b][j]
        see = see.cuda()
        for h in range(H):
            shift = st["shift"][b, h].double()
            k = torch.cat([_exact_values(k4[b, h, :n], ks[b, h, :n]) + shift, st["k"][b, h, :c].double()])
            v = torch.cat([_exact_values(v4[b, h, :n], vs[b, h, :n]), st["v"][b, h, :c].double()])
            x = torch.einsum("gid,jd->gij", st["q"][b].double().view(H, g, Sq, D)[h, :, :c], k) / math.sqrt(D)
            x = torch.where(see, x, -math.inf)
            lse[b, h, :, :c] = torch.logsumexp(x, -1)
            o[b, h, :, :c] = torch.softmax(x, -1) @ v
    return {"o": o.view(B, H * g, Sq, D), "lse": lse.view(B, H * g, Sq)}
