"""Cases for the operators that prepare and read a paged KV cache when serving.

Four operators, in the order in which one layer of a serving step calls them:

  rope   norms of queries and keys for each head, with the rotation by position in the same pass
  write  keys and values quantised to e4m3 (a power-of-two scale for each key of each head) into a paged cache
  read   the same cache read back as bf16
  tree   attention of drafted tokens (a tree, a chain, or one token) over a paged cache, bf16 or e4m3

``listed`` names fixed cases, ``draw`` gives more of the same ranges, ``prepare`` makes a case's inputs on the GPU,
``run`` is one pass: elementary torch operations in 32 bits, or with ``own`` set the package's calls.
``exact`` is the definition in 64 bits, and ``work`` counts what a pass cannot do without.
"""
import math

import torch

own = False

PAGE = 64  # keys of a page


def listed():
    return [
        # one decode step of 16 sequences: Q and K are slices of the fused projection's output, norms on both
        {"name": "rope decode 16", "op": "rope", "B": 0, "N": 16, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "norm": True, "far": 131072},
        # the 8B layer's prompt of 8192 tokens: no norms, [B, N, H, d] in and [B, H, N, d] out
        {"name": "rope prompt 8192", "op": "rope", "B": 1, "N": 8192, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "norm": False, "far": 8192},
        # a packed batch of odd size with small heads, a part of the head rotated in adjacent pairs
        {"name": "rope packed 30011 d64", "op": "rope", "B": 0, "N": 30011, "Hq": 16, "Hkv": 4, "d": 64, "rot": 32,
         "interleaved": True, "norm": True, "far": 1000000},
        # one decode step of 16 sequences
        {"name": "write decode 16", "op": "write", "B": 0, "N": 16, "Hkv": 8, "d": 128, "pages": 512},
        # the prompt of an 8B layer, four sequences of odd length in the prefill layout
        {"name": "write prompts 4x4099", "op": "write", "B": 4, "N": 4099, "Hkv": 8, "d": 128, "pages": 300},
        # a prefix of a packed batch taken back out of the cache
        {"name": "read packed 1000 d64", "op": "read", "B": 0, "N": 1000, "Hkv": 8, "d": 64, "pages": 64},
        # a long cached prefix in the layout of the contiguous decode
        {"name": "read prefix 2x32768", "op": "read", "B": 2, "N": 32768, "Hkv": 8, "d": 128, "pages": 1100},
        # the smallest: a chain of 5 drafted tokens of one short sequence, odd length, e4m3
        {"name": "tree e4m3 1x5 L1001", "op": "tree", "cache": "e4m3", "B": 1, "T": 5, "Hq": 8, "Hkv": 8, "d": 64,
         "L": 1001, "ragged": False, "chain": True},
        # single tokens over the e4m3 cache: the GQA decode workload's shape
        {"name": "tree e4m3 16x1 L32768", "op": "tree", "cache": "e4m3", "B": 16, "T": 1, "Hq": 32, "Hkv": 8, "d": 128,
         "L": 32768, "ragged": False, "chain": True},
        # drafted trees of up to 16 tokens in a ragged batch, e4m3
        {"name": "tree e4m3 16x16 ragged", "op": "tree", "cache": "e4m3", "B": 16, "T": 16, "Hq": 32, "Hkv": 8,
         "d": 128, "L": 16384, "ragged": True, "chain": False},
        # drafted trees of 8 tokens over the bf16 cache, ragged
        {"name": "tree bf16 16x8 ragged", "op": "tree", "cache": "bf16", "B": 16, "T": 8, "Hq": 32, "Hkv": 8, "d": 128,
         "L": 32768, "ragged": True, "chain": False},
        # large trees with the 70B layer's heads over a few long sequences, bf16
        {"name": "tree bf16 4x64 64q", "op": "tree", "cache": "bf16", "B": 4, "T": 64, "Hq": 64, "Hkv": 8, "d": 128,
         "L": 16384, "ragged": False, "chain": False},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "tree", "tree"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "rope":
        B = rng.choice([0, 0, 1, 2, 3])
        return {"op": "rope", "B": B, "N": _spread(rng, 1, 16000 // max(1, B)), "Hq": Hkv * rng.choice([1, 2, 4, 8]),
                "Hkv": Hkv, "d": d, "rot": rng.choice([d, d, d // 2]), "interleaved": rng.random() < 0.5,
                "norm": rng.random() < 0.5, "far": _spread(rng, 100, 2000000)}
    if op in ("write", "read"):
        B = rng.choice([0, 0, 1, 2, 3])
        N = _spread(rng, 1, 16000 // max(1, B))
        return {"op": op, "B": B, "N": N, "Hkv": Hkv, "d": d, "pages": N * max(1, B) // PAGE + rng.randint(1, 40)}
    B, T, Hq = _spread(rng, 1, 16), _spread(rng, 1, 64), Hkv * rng.choice([1, 2, 4, 8])
    most = min(200000 // B, 32768 * 8192 // (B * T * Hq))  # keys, and pairs of a query and a key
    return {"op": "tree", "cache": rng.choice(["bf16", "e4m3"]), "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "d": d,
            "L": _spread(rng, 70, max(80, most)), "ragged": rng.random() < 0.6, "chain": rng.random() < 0.4}


# ------------------------------------------------------------------ sizes that follow from a case

def _lens(case):
    """Keys of each sequence, its drafted tokens among them: a ragged batch runs from about half of L up to L."""
    B, L = case["B"], case["L"]
    return [L - (b * (L // 2)) // B if case["ragged"] else L for b in range(B)]


def _drafted(case):
    """Drafted tokens of each sequence: in a ragged batch some have fewer."""
    return [max(1, case["T"] - (b % 3) * (case["T"] // 4)) if case["ragged"] else case["T"] for b in range(case["B"])]


def work(case):
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "tree":
        rows = sum(_drafted(case)) * case["Hq"]
        keys = sum(_lens(case)) * Hkv
        element = 2 * d if case["cache"] == "bf16" else d + 4  # one key's bytes: values, or codes and a scale
        pairs = sum(t * n for t, n in zip(_drafted(case), _lens(case))) * case["Hq"]
        return {"bytes": 2 * keys * element + 4 * rows * d, "flops": 4 * pairs * d}
    tokens = max(1, case["B"]) * case["N"]
    if op == "rope":
        values = tokens * (case["Hq"] + Hkv) * d
        return {"bytes": 4 * values + 4 * tokens, "flops": 8 * values}
    values = tokens * Hkv * d * 2
    return {"bytes": 3 * values + 8 * tokens * Hkv + 8 * tokens, "flops": 3 * values}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


def _quantised(x):
    """e4m3 codes and a power-of-two scale for each vector along the last axis."""
    amax = x.float().abs().amax(-1, keepdim=True)
    mantissa, exponent = torch.frexp(amax)
    exponent = torch.where(mantissa <= 0.875, exponent - 9, exponent - 8).clamp_min(-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), exponent), torch.ones_like(amax))
    return (x.float() / scale).to(torch.float8_e4m3fn).view(torch.uint8), scale.squeeze(-1)


def _pool(gen, pages, Hkv, d):
    """A page pool with keys and values as layers give them: values of about 1, some heads and keys larger."""
    K = torch.randn(pages, Hkv, PAGE, d, generator=gen, device="cuda")
    V = torch.randn(pages, Hkv, PAGE, d, generator=gen, device="cuda")
    K *= 1 + 0.5 * torch.rand(pages, Hkv, PAGE, 1, generator=gen, device="cuda")
    V *= 0.25 + torch.rand(pages, Hkv, PAGE, 1, generator=gen, device="cuda")
    return K.to(torch.bfloat16), V.to(torch.bfloat16)


def _tree_bits(T, rng):
    """Ancestors (and itself) of each token of a random tree, as 64 bits in an int64."""
    bits = [1]
    for i in range(1, T):
        bits.append(bits[int(torch.randint(0, i, (1,), generator=rng))] | (1 << i))
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def prepare(case, seed):
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    gen = _gen(seed)
    s = {"case": case}
    if op == "tree":
        B, Hq = case["B"], case["Hq"]
        lens, drafted = _lens(case), _drafted(case)
        used = [-(-n // PAGE) for n in lens]
        pool = sum(used) + 3
        K, V = _pool(gen, pool, Hkv, d)
        order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))
        table = torch.full((B, max(used)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = order[at: at + n]
            at += n
        total = sum(drafted) + (2 if case["ragged"] else 0)  # a padded batch ends in rows of no sequence
        rng = torch.Generator().manual_seed(seed + 1)
        bits = sum((_tree_bits(t, rng) for t in drafted), []) + [0] * (total - sum(drafted))
        s["q"] = (2 * torch.randn(total, Hq, d, generator=gen, device="cuda")).to(torch.bfloat16)
        s["o"] = torch.zeros(total, Hq, d, dtype=torch.bfloat16, device="cuda")
        s["table"] = table.cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["cu_q"] = torch.tensor([0] + torch.tensor(drafted).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        s["bits"] = None if case["chain"] else torch.tensor(bits, dtype=torch.int64, device="cuda")
        if case["cache"] == "bf16":
            s["K"], s["V"] = K, V
        else:
            (s["K"], s["Ks"]), (s["V"], s["Vs"]) = _quantised(K), _quantised(V)
        return s
    B, N = case["B"], case["N"]
    tokens = max(1, B) * N
    if op == "rope":
        Hq = case["Hq"]
        fused = torch.randn(tokens, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
        q, k = fused[:, :Hq], fused[:, Hq: Hq + Hkv]
        if B:
            q, k = (x.unflatten(0, (B, N)).transpose(1, 2) for x in (q, k))
        rot = case["rot"]
        s["q"], s["k"] = q, k
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        if B:  # prompts: consecutive positions, from another start for each sequence
            start = torch.randint(0, case["far"], (B, 1), generator=gen, device="cuda")
            s["pos"] = (start + torch.arange(N, device="cuda")).to(torch.int32)
        else:
            s["pos"] = torch.randint(0, case["far"], (N,), generator=gen, device="cuda").to(torch.int32)
        s["wq"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        s["wk"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        return s
    pages = case["pages"]
    s["slots"] = torch.randperm(pages * PAGE, generator=gen, device="cuda")[:tokens]
    if B:
        s["slots"] = s["slots"].view(B, N)
    if op == "write":
        spread = 0.1 + 4 * torch.rand(tokens, Hkv, 1, generator=gen, device="cuda")
        fused = torch.randn(tokens, 2 * Hkv, d, generator=gen, device="cuda") * spread.repeat(1, 2, 1)
        fused = fused.to(torch.bfloat16)
        k, v = fused[:, :Hkv], fused[:, Hkv:]
        if B:  # the prefill layout
            k, v = (x.unflatten(0, (B, N)).transpose(1, 2).contiguous() for x in (k, v))
        s["k"], s["v"] = k, v
        s["K"], s["V"] = (torch.zeros(pages, Hkv, PAGE, d, dtype=torch.uint8, device="cuda") for _ in range(2))
        s["Ks"], s["Vs"] = (torch.zeros(pages, Hkv, PAGE, dtype=torch.float32, device="cuda") for _ in range(2))
    else:
        K, V = _pool(gen, pages, Hkv, d)
        (s["K"], s["Ks"]), (s["V"], s["Vs"]) = _quantised(K), _quantised(V)
    return s


# ------------------------------------------------------------------ one pass

def _by_token(x, B):
    """[B, H, N, d] as [B * N, H, d]; a packed [T, H, d] as it is."""
    return x.transpose(1, 2).flatten(0, 1) if B else x


def _as_given(x, B):
    """[B * N, H, d] back as contiguous [B, H, N, d]; a packed tensor as it is."""
    return x.unflatten(0, (B, -1)).transpose(1, 2).contiguous() if B else x


def _norm_rope(x, w, cos, sin, rot, interleaved, eps=1e-6):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1).to(torch.bfloat16)


def _run_rope(s, c):
    if own:
        import block_skipping_softmax_b200 as bss

        return bss.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["wq"], s["wk"],
                                interleaved=c["interleaved"])
    angle = s["pos"].flatten().double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    return tuple(_as_given(_norm_rope(_by_token(x, c["B"]), w, cos, sin, c["rot"], c["interleaved"]), c["B"])
                 for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))


def _pool_values(s):
    return {"K": s["K"].view(torch.float8_e4m3fn), "V": s["V"].view(torch.float8_e4m3fn), "Ks": s["Ks"], "Vs": s["Vs"]}


def _run_write(s, c):
    if own:
        import block_skipping_softmax_b200 as bss

        bss.cache_write_e4m3(s["k"], s["v"], s["slots"], s["K"], s["V"], s["Ks"], s["Vs"])
        return _pool_values(s)
    slots = s["slots"].flatten()[:, None]
    at = (slots // PAGE, torch.arange(c["Hkv"], device="cuda")[None], slots % PAGE)
    for x, codes, scales in ((s["k"], s["K"], s["Ks"]), (s["v"], s["V"], s["Vs"])):
        new, scale = _quantised(_by_token(x, c["B"]))
        codes[at] = new
        scales[at] = scale
    return _pool_values(s)


def _run_read(s, c):
    if own:
        import block_skipping_softmax_b200 as bss

        return bss.cache_read_e4m3(s["K"], s["V"], s["Ks"], s["Vs"], s["slots"])
    slots = s["slots"].flatten()[:, None]
    at = (slots // PAGE, torch.arange(c["Hkv"], device="cuda")[None], slots % PAGE)
    return tuple(_as_given((codes[at].view(torch.float8_e4m3fn).float() * scales[at][..., None]).to(torch.bfloat16),
                           c["B"]) for codes, scales in ((s["K"], s["Ks"]), (s["V"], s["Vs"])))


def _run_tree(s, c):
    if own:
        import block_skipping_softmax_b200 as bss

        if c["cache"] == "bf16":
            return bss.tree_paged(s["q"], s["K"], s["V"], s["table"], s["lens"], s["cu_q"], c["T"], c["L"], s["bits"],
                                  out=s["o"])
        return bss.tree_paged_e4m3(s["q"], s["K"], s["V"], s["Ks"], s["Vs"], s["table"], s["lens"], s["cu_q"], c["T"],
                                   c["L"], s["bits"], out=s["o"])
    B, T, Hq, Hkv, d = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"]
    g, total = Hq // Hkv, s["q"].shape[0]
    page = s["table"].clamp_min(0).long()

    def gathered(values, scales):  # [B, Hkv, keys, d] in 32 bits
        x = values[page].float() if scales is None else \
            values[page].view(torch.float8_e4m3fn).float() * scales[page][..., None]
        return x.transpose(1, 2).flatten(2, 3)

    K, V = gathered(s["K"], s.get("Ks")), gathered(s["V"], s.get("Vs"))
    n = K.shape[2]
    t = torch.arange(T, device="cuda")
    first, count = s["cu_q"][:-1, None], s["cu_q"][1:, None] - s["cu_q"][:-1, None]
    valid = t < count  # [B, T]
    token = (first + t).clamp_max(total - 1).long()
    q = s["q"][token].float().unflatten(2, (Hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, Hkv, T * g, d]
    x = (q @ K.transpose(2, 3)) / math.sqrt(d)
    key = torch.arange(n, device="cuda")
    prefix = (s["lens"][:, None] - count).clamp_min(0)  # [B, 1]
    draft = key - prefix  # [B, keys]: which drafted token a key is
    if c["chain"]:
        sees = draft[:, None] <= t[:, None]
    else:
        bits = s["bits"][token]  # [B, T]
        sees = (draft[:, None] < 0) | ((bits[:, :, None] >> draft[:, None].clamp(0, 63)) & 1).bool()
    sees = sees & (key < s["lens"][:, None])[:, None] & valid[:, :, None]  # [B, T, keys]
    sees = sees[:, None, :, None].expand(B, 1, T, g, n).flatten(2, 3)
    x = torch.where(sees, x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(x - top)
    sums = p.sum(-1, keepdim=True)
    V = torch.where((key < s["lens"][:, None])[:, None, :, None], V, 0)
    o = (p @ V) / torch.where(sums > 0, sums, 1)
    o = o.unflatten(2, (T, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, T, Hq, d]
    out = torch.zeros(total + 1, Hq, d, device="cuda")
    out[torch.where(valid, token, total)] = o  # rows of no sequence stay as they were
    return out[:total].to(torch.bfloat16)


def run(state):
    c = state["case"]
    return {"rope": _run_rope, "write": _run_write, "read": _run_read, "tree": _run_tree}[c["op"]](state, c)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read, "tree": _exact_tree}[case["op"]](s, case)


def _exact_rope(s, c):
    d, rot = c["d"], c["rot"]
    outs = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
        pos = s["pos"].double()
        pos = pos[:, None, :] if c["B"] else pos[:, None]  # [B, 1, N] or [T, 1]
        y = x.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
            turn = torch.polar(torch.ones_like(pos), pos * s["inv_freq"][i].double())
            z = torch.complex(x[..., a], x[..., b]) * turn
            y[..., a], y[..., b] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_write(s, c):
    pool = {"K": s["K"], "V": s["V"]}
    out = {n: torch.zeros(p.transpose(1, 2).shape, dtype=torch.float64, device="cuda") for n, p in pool.items()}
    out |= {n + "s": torch.zeros(out[n].shape[:3], dtype=torch.float64, device="cuda") for n in pool}
    for n, x in (("K", s["k"]), ("V", s["v"])):
        x = x.transpose(1, 2).double() if c["B"] else x.double()  # heads behind tokens, as the slots are
        k = torch.floor(torch.log2(x.abs().amax(-1) / 448)).clamp_min(-126)
        k = torch.where(x.abs().amax(-1) <= 448 * torch.exp2(k), k, k + 1)
        y = x / torch.exp2(k)[..., None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        out[n].flatten(0, 1)[s["slots"]] = torch.round(y / step) * step
        out[n + "s"].flatten(0, 1)[s["slots"]] = torch.exp2(k)
    return {n: x.transpose(1, 2) for n, x in out.items()}


def _dequantised(codes, scales):
    code = codes.long()
    e, m = (code >> 3) & 15, (code & 7).double()
    value = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(code >= 128, -value, value) * scales.double()[..., None]


def _exact_read(s, c):
    outs = []
    for codes, scales in ((s["K"], s["Ks"]), (s["V"], s["Vs"])):
        flat = codes.transpose(1, 2).flatten(0, 1)[s["slots"]], scales.transpose(1, 2).flatten(0, 1)[s["slots"]]
        x = _dequantised(*flat)
        outs.append(x.transpose(1, 2) if c["B"] else x)
    return tuple(outs)


def _exact_tree(s, c):
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    lens, drafted = _lens(c), _drafted(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, T) in enumerate(zip(lens, drafted)):
        page = s["table"][b, : -(-n // PAGE)].long()
        if c["cache"] == "bf16":
            K, V = s["K"][page].double(), s["V"][page].double()
        else:
            K, V = _dequantised(s["K"][page], s["Ks"][page]), _dequantised(s["V"][page], s["Vs"][page])
        K, V = (x.permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n] for x in (K, V))
        sees = torch.ones(T, n, dtype=torch.bool, device="cuda")
        prefix = max(0, n - T)
        for i in range(T):
            own_bits = ((1 << (i + 1)) - 1) if c["chain"] else int(s["bits"][at + i])
            for j in range(n - prefix):
                if not (own_bits >> j) & 1:
                    sees[i, prefix + j] = False
        for h in range(Hq):
            x = s["q"][at: at + T, h].double() @ K[h // (Hq // Hkv)].T / math.sqrt(d)
            x = x.masked_fill(~sees, -math.inf)
            some = sees.any(1, keepdim=True)
            p = torch.where(some, torch.softmax(x.masked_fill(~some, 0), -1), 0)
            out[at: at + T, h] = p @ V[h // (Hq // Hkv)]
        at += T
    return out
