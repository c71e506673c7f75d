"""Workloads of the 4-bit cache, of norm with rotation, and of the page plan.

Five operators of a serving path, each as real programs call it:

  store   quantises new key and value vectors into the paged 4-bit cache
          (4-bit integers, one scale byte for 16 of them, one exponent byte for
          a vector)
  load    reads sequences of that cache back into packed rows
  decode  attention of one new token per sequence over that cache
  rotate  norms each query and key head, rotates it by its position, and puts
          keys and values where attention wants them
  plan    block-table entries, slots, positions and row starts of a step's new
          tokens, from the lengths of the requests and a list of free blocks

``run`` computes them in elementary torch operations, or, where ``own`` is
true, with the library's calls.  ``exact`` gives the same outputs from the
definitions in 64 bits.

A page of the cache holds 16 tokens of one KV head: 16 x d/2 bytes of key
codes, as many of value codes, 16 x d/16 key scales, 16 x d/16 value scales, 16
key and 16 value exponents; the cache is [blocks][KV heads][page].  Byte j of a
vector's codes holds elements 2j (low half) and 2j + 1; a code n stands for
n - 8.  A scale byte u stands for S(u), the fp16 number with the bits u << 7,
an exponent byte E for 2^(E - 127), 255 for NaN.  Every decision of the store
is exact, so its bytes are equal or wrong: they are returned as they are.
"""

import math
import random

import torch

own = False

BLOCK = 16
GROUP = 16
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's new tokens, 16 sequences of a model with 8 KV heads: latency
        _store("store4_step16_d128", 16, 8, 128, "bf16", "step"),
        # the prompts of 64 requests written at once
        _store("store4_prefill65536_d128", 65536, 8, 128, "bf16", "prefill"),
        # a short prefix read back before the next chunk of its prompt
        _load("load4_1x700_d128", 1, 700, "equal", 1, 8, 128, "bf16", 64),
        # the prefixes of a batch of requests, different lengths, room for a chunk behind each
        _load("load4_16xragged16384_d128", 16, 16384, "ragged", 2, 8, 128, "bf16", 256),
        # one short conversation: latency
        _decode("decode4_1x130_d128", 1, 130, "equal", 3, 32, 8, 128, "bf16", "bf16"),
        # a batch of chats at 8192 tokens
        _decode("decode4_16x8192_d128", 16, 8192, "equal", 4, 32, 8, 128, "bf16", "bf16"),
        # long documents of different lengths, 64 query heads
        _decode("decode4_4xragged131072_d128", 4, 131072, "ragged", 5, 64, 8, 128, "bf16", "bf16"),
        # wide heads, float queries and outputs
        _decode("decode4_8xragged32768_d256_f32", 8, 32768, "ragged", 6, 32, 4, 256, "f32", "f32"),
        # the queries and keys of a decode step, far positions: latency
        _rotate("rotate_step16_d128", 16, 32, 8, 128, 128, "bf16", False, 1.0e6, True, False, 131072),
        # a prefill's rows out of the fused projection, keys and values to their places behind stored prefixes
        _rotate("rotate_prefill8192_d128", 8192, 32, 8, 128, 128, "bf16", False, 5.0e5, True, True, 32768),
        # a decode step of 256 requests
        _plan("plan_step256", 256, 16384, 0, 7, 0),
        # chunks of 64 requests, of different lengths, behind stored prefixes of different lengths
        _plan("plan_chunks64", 64, 8192, 2048, 8, 100),
    ]


def _store(name, tokens, kv_heads, d, dtype, kind):
    return dict(name=name, op="store", tokens=tokens, kv_heads=kv_heads, d=d, dtype=dtype, kind=kind)


def _load(name, batch, longest, spread, mix, kv_heads, d, dtype, room):
    return dict(name=name, op="load", batch=batch, longest=longest, spread=spread, mix=mix, kv_heads=kv_heads, d=d,
                dtype=dtype, room=room)


def _decode(name, batch, longest, spread, mix, q_heads, kv_heads, d, dtype, out_dtype):
    return dict(name=name, op="decode", batch=batch, longest=longest, spread=spread, mix=mix, q_heads=q_heads,
                kv_heads=kv_heads, d=d, dtype=dtype, out_dtype=out_dtype)


def _rotate(name, tokens, q_heads, kv_heads, d, rot_dim, dtype, interleaved, base, fused, place, farthest):
    """fused: rows of one projection; place: keys and values go to rows of a longer buffer."""
    return dict(name=name, op="rotate", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, d=d, rot_dim=rot_dim,
                dtype=dtype, interleaved=interleaved, base=base, fused=fused, place=place, farthest=farthest)


def _plan(name, batch, longest, chunk, mix, pad):
    """chunk: most new tokens of a request, 0 for a decode step (one each); pad: rows behind the last token."""
    return dict(name=name, op="plan", batch=batch, longest=longest, chunk=chunk, mix=mix, pad=pad)


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["store", "load", "decode", "decode", "rotate", "rotate", "plan"])
    d = rng.choice([128, 128, 256])
    mix = rng.randrange(1 << 20)
    spread = rng.choice(["equal", "ragged", "ragged"])
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    if op == "store":
        c = _store("", _log(rng, 1, 65536), kv_heads, d, rng.choice(["bf16", "bf16", "f32", "f16"]),
                   rng.choice(["step", "prefill"]))
        if c["kind"] == "step":
            c["tokens"] = min(c["tokens"], 1024)
        while c["tokens"] * c["kv_heads"] * d > 65536 * 8 * 128:
            c["tokens"] //= 2
    elif op == "load":
        c = _load("", _log(rng, 1, 64), _log(rng, 1, 32768), spread, mix, kv_heads, d,
                  rng.choice(["bf16", "f16", "f32"]), rng.choice([0, 1, 37, 512]))
        while c["batch"] * c["longest"] * kv_heads * d > 8 * 16384 * 8 * 128:
            c["longest"] = max(1, c["longest"] // 2)
    elif op == "decode":
        group = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        c = _decode("", _log(rng, 1, 256), _log(rng, 1, 131072), spread, mix, group * kv_heads, kv_heads, d,
                    rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice(["bf16", "bf16", "f16", "f32"]))
        while c["batch"] * c["longest"] * kv_heads * d > 2 * 131072 * 8 * 128:
            c["longest"] = max(1, c["longest"] // 2)
    elif op == "rotate":
        group = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        c = _rotate("", _log(rng, 1, 32768), group * kv_heads, kv_heads, d, rng.choice([d, d, d // 2, d // 4, 96, 16]),
                    rng.choice(["bf16", "bf16", "f16", "f32"]), rng.random() < 0.4, rng.choice([1.0e4, 5.0e5, 1.0e6]),
                    rng.random() < 0.6, rng.random() < 0.4, _log(rng, 1, 1 << 20))
        while c["tokens"] * (c["q_heads"] + 2 * kv_heads) * d > 8192 * 48 * 128:
            c["tokens"] //= 2
    else:
        c = _plan("", _log(rng, 1, 1024), _log(rng, 1, 131072), rng.choice([0, 0, _log(rng, 1, 8192)]), mix,
                  rng.choice([0, 0, 1, 45]))
        while c["batch"] * c["chunk"] > 2 * 65536:
            c["chunk"] //= 2
        while c["batch"] * c["longest"] > 1024 * 16384:
            c["longest"] //= 2
    del c["name"]
    return c


def _lengths(case):
    """Tokens per sequence: all `longest`, or spread between 1 and it with one that reaches it."""
    n, b = case["longest"], case["batch"]
    if case["spread"] == "equal":
        return [n] * b
    rng = random.Random(case["mix"])
    lens = [rng.randint(1, n) for _ in range(b)]
    lens[rng.randrange(b)] = n
    return lens


def _requests(case):
    """Stored and new tokens of a plan's requests; some have nothing stored yet, some nothing new."""
    rng = random.Random(case["mix"])
    lens = [rng.randint(1, case["longest"]) for _ in range(case["batch"])]
    if case["chunk"] == 0:
        return lens, [1] * len(lens)
    lens = [0 if rng.random() < 0.3 else n for n in lens]
    new = [0 if rng.random() < 0.1 else rng.randint(1, case["chunk"]) for _ in lens]
    new[rng.randrange(len(new))] = case["chunk"]
    return lens, new


def _blocks(tokens):
    return (tokens + BLOCK - 1) // BLOCK


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] == "plan":
        lens, new = _requests(case)
        taken = sum(_blocks(a + n) - _blocks(a) for a, n in zip(lens, new))
        return {"bytes": 20 * len(lens) + 8 * taken + 16 * (sum(new) + case["pad"]), "flops": 0}
    d = case["d"]
    if case["op"] == "rotate":
        heads = case["q_heads"] + case["kv_heads"] * (2 if case["place"] else 1)
        return {"bytes": case["tokens"] * (2 * heads * d * size[case["dtype"]] + (8 if case["place"] else 4)), "flops": 0}
    vector = d // 2 + d // GROUP + 1
    if case["op"] == "store":
        vec = case["tokens"] * case["kv_heads"] * 2
        return {"bytes": vec * (d * size[case["dtype"]] + vector) + 8 * case["tokens"], "flops": 0}
    lens = _lengths(case)
    n = sum(lens)
    if case["op"] == "load":
        return {"bytes": n * case["kv_heads"] * 2 * (vector + d * size[case["dtype"]]), "flops": 0}
    rows = case["batch"] * case["q_heads"]
    return {"bytes": n * case["kv_heads"] * 2 * vector + rows * d * (size[case["dtype"]] + size[case["out_dtype"]]),
            "flops": 4 * d * n * case["q_heads"]}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _vectors(g, rows, heads, d, dtype, gains):
    """Normal vectors; keys have channels of different strength, as projected keys do."""
    x = torch.randn((rows, heads, d), generator=g, device="cuda")
    if gains:
        x *= torch.exp(0.5 * torch.randn((heads, d), generator=g, device="cuda"))
    return x.to(dtype)


def _page_bytes(d):
    return 2 * BLOCK * (d // 2 + d // GROUP + 1)


def _page_parts(cache, blocks, heads, d):
    """Key and value codes [.., 16, d/2], their scales [.., 16, d/16] and exponents [.., 16], as views of the pages."""
    p = cache.view(blocks, heads, _page_bytes(d))
    parts, at = [], 0
    for width in (d // 2, d // 2, d // GROUP, d // GROUP, 1, 1):
        part = p[:, :, at:at + BLOCK * width]
        parts.append(part.unflatten(2, (BLOCK, width)) if width > 1 else part)
        at += BLOCK * width
    return parts


def _filled_cache(g, blocks, heads, d):
    """A cache whose every slot holds a quantised vector."""
    cache = torch.empty(blocks * heads * _page_bytes(d), dtype=torch.uint8, device="cuda")
    parts = _page_parts(cache, blocks, heads, d)
    for i in (0, 1):
        gain = torch.exp(0.5 * torch.randn((heads, d), generator=g, device="cuda")) if i == 0 else 1.0
        for at in range(0, blocks, 4096):
            n = min(4096, blocks - at)
            made = _quantise(torch.randn((n, heads, BLOCK, d), generator=g, device="cuda") * gain.unsqueeze(1)
                             if i == 0 else torch.randn((n, heads, BLOCK, d), generator=g, device="cuda"))
            for j in range(3):
                parts[2 * j + i][at:at + n] = made[j]
    return cache


def _table(g, lens):
    """Each sequence's blocks: a permutation of the pool, as after some hours of serving."""
    need = [_blocks(n) for n in lens]
    blocks = max(1, sum(need))
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, blocks


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _handle(case, blocks, columns, cache):
    import turboquant_bit_kv_tq_gb300 as tq

    heads = case["kv_heads"]
    return tq.TQI4Cache(head_dim=case["d"], num_kv_heads=heads, num_q_heads=case.get("q_heads", heads),
                        num_blocks=blocks, max_batch=case.get("batch", 1), max_blocks_per_seq=columns, cache=cache)


def _prepare_rotate(case, g):
    n, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["d"]
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    q, k = _vectors(g, n, hq, d, dtype, True), _vectors(g, n, hk, d, dtype, True)
    v = _vectors(g, n, hk, d, dtype, False)
    if case["fused"]:
        s["qkv"] = torch.cat([q, k, v], dim=1)
        q, k, v = s["qkv"].split([hq, hk, hk], dim=1)
    s["q"], s["k"], s["v"] = q, k, v
    s["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    s["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    far = case["farthest"]
    start = torch.randint(0, max(1, far - n + 1), (1,), generator=g, device="cuda")
    if case["place"]:  # consecutive positions of one chunk
        s["positions"] = (start + torch.arange(n, device="cuda")).to(torch.int32)
    else:  # a position for each of many sequences
        s["positions"] = torch.randint(0, far, (n,), generator=g, device="cuda").to(torch.int32)
    rows = n
    if case["place"]:  # behind prefixes of several prompts: rows in order, with gaps
        rows = 2 * n
        s["rows"] = (torch.randperm(rows, generator=g, device="cuda")[:n].sort().values).to(torch.int32)
    s["q_out"] = torch.zeros((n, hq, d), dtype=dtype, device="cuda")
    s["k_out"] = torch.zeros((rows, hk, d), dtype=dtype, device="cuda")
    s["v_out"] = torch.zeros((rows, hk, d), dtype=dtype, device="cuda") if case["place"] else None
    s["inv_freq"] = torch.tensor([case["base"] ** (-2.0 * i / case["rot_dim"]) for i in range(case["rot_dim"] // 2)],
                                 dtype=torch.float64, device="cuda")
    s["eps"] = 1.0e-6
    if own:
        import turboquant_bit_kv_tq_gb300 as tq

        s["handle"] = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=hk, rot_dim=case["rot_dim"],
                                    base=case["base"], eps=s["eps"], interleaved=case["interleaved"])
    return s


def _prepare_plan(case, g):
    lens, new = _requests(case)
    s = {"case": case, "lens": _ints(lens), "new": _ints(new) if case["chunk"] else None,
         "tokens": sum(new) + case["pad"]}
    have = [_blocks(n) for n in lens]
    taken = sum(_blocks(a + n) for a, n in zip(lens, new)) - sum(have)
    columns = max(1, max(_blocks(a + n) for a, n in zip(lens, new)))
    skip, spare = 5, 11  # blocks of the list that earlier steps took, blocks that stay free
    perm = torch.randperm(sum(have) + skip + taken + spare, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.full((len(lens), columns), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(have):
        s["table"][b, :n] = perm[at:at + n]
        at += n
    s["free"] = perm[at:].clone()
    s["next"] = _ints([skip])
    if own:
        import turboquant_bit_kv_tq_gb300 as tq

        s["handle"] = tq.TQPlan(max_batch=len(lens), max_blocks_per_seq=columns)
        s["out"] = s["handle"].outputs(len(lens), s["tokens"])
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "rotate":
        return _prepare_rotate(case, g)
    if case["op"] == "plan":
        return _prepare_plan(case, g)
    d, heads = case["d"], case["kv_heads"]
    s = {"case": case}
    if case["op"] == "store":
        n = case["tokens"]
        s["k"] = _vectors(g, n, heads, d, DTYPES[case["dtype"]], True)
        s["v"] = _vectors(g, n, heads, d, DTYPES[case["dtype"]], False)
        if case["kind"] == "prefill":  # consecutive positions in blocks from all over the pool
            blocks = _blocks(n)
            perm = torch.randperm(blocks, generator=g, device="cuda")
            t = torch.arange(n, device="cuda")
            s["slots"] = perm[t // BLOCK] * BLOCK + t % BLOCK
        else:  # one token of each sequence, each in a block of its own
            blocks = n
            s["slots"] = torch.randperm(n, generator=g, device="cuda") * BLOCK + torch.randint(
                0, BLOCK, (n,), generator=g, device="cuda")
        s["blocks"] = blocks
        s["cache"] = torch.zeros(blocks * heads * _page_bytes(d), dtype=torch.uint8, device="cuda")
        s["parts"] = _page_parts(s["cache"], blocks, heads, d)
        if own:
            s["handle"] = _handle(case, blocks, 1, s["cache"])
        return s
    lens = _lengths(case)
    s["longest"] = max(lens)
    s["table"], s["blocks"] = _table(g, lens)
    s["lens"] = _ints(lens)
    s["cache"] = _filled_cache(g, s["blocks"], heads, d)
    if own:
        s["handle"] = _handle(case, s["blocks"], s["table"].shape[1], s["cache"])
    if case["op"] == "load":
        starts = _starts([n + case["room"] for n in lens])
        s["starts"] = _ints(starts)
        s["k"] = torch.zeros((starts[-1], heads, d), dtype=DTYPES[case["dtype"]], device="cuda")
        s["v"] = torch.zeros_like(s["k"])
    else:
        s["q"] = _vectors(g, case["batch"], case["q_heads"], d, DTYPES[case["dtype"]], False)
        s["out"] = torch.zeros(s["q"].shape, dtype=DTYPES[case["out_dtype"]], device="cuda")
    return s


# -------------------------------------------------------------- plain forms
def _scales(u):
    """What scale bytes stand for: fp16 numbers without sign, cut to three bits behind the point."""
    return (u.to(torch.int16) << 7).view(torch.float16).float()


def _quantise(x):
    """x [..., d] -> (packed codes [..., d/2], scale bytes [..., d/16], exponent bytes [...]), as uint8."""
    x = x.float()
    top = x.abs().amax(dim=-1)
    bad = ~torch.isfinite(top)
    bits = torch.where(bad, torch.zeros_like(top), top).view(torch.int32)
    # smallest e with top <= 240 * 2^e = 1.875 * 2^(e + 7)
    byte = ((bits >> 23) - 7 + ((bits & 0x7FFFFF) > 0x700000).int()).clamp(1, 254)
    y = torch.ldexp(x, (127 - byte).unsqueeze(-1))
    y = torch.where(bad.unsqueeze(-1), torch.zeros_like(y), y).unflatten(-1, (-1, GROUP))
    g = y.abs().amax(dim=-1)
    # the byte below g / 7.5 by bits (steps of 2^-17 below 2^-14), then up to the first that is not too small
    t = g * (2.0 / 15.0)
    normal = (t.view(torch.int32) >> 20) - ((127 - 15) << 3)
    u = torch.where(t < 2.0 ** -14, (t * 2.0 ** 17).int(), normal).clamp(min=1)
    for _ in (0, 1):
        u = u + (_scales(u) * 7.5 < g).int()
    u = torch.where(g <= 2.0 ** -18, torch.zeros_like(u), u)
    s = _scales(u).unsqueeze(-1)
    # quotients next to a border between two codes: 64 bits
    n = torch.where(s > 0, y.double() / torch.where(s > 0, s, torch.ones_like(s)).double(), 0.0)
    n = (n.round().clamp(-7, 7) + 8).to(torch.uint8).flatten(-2)
    exps = torch.where(bad, torch.full_like(byte, 255), byte).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), u.to(torch.uint8), exps


def _values(codes, scales, exps):
    n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8.0
    x = (n.unflatten(-1, (-1, GROUP)) * _scales(scales).unsqueeze(-1)).flatten(-2)
    x = torch.ldexp(x, (exps.int() - 127).unsqueeze(-1))
    return torch.where((exps == 255).unsqueeze(-1), torch.full_like(x, math.nan), x)


def _read_rows(s, heads, d):
    """Keys and values [batch, longest, heads, d] as float, and which rows are tokens."""
    parts = _page_parts(s["cache"], s["blocks"], heads, d)
    t = torch.arange(s["longest"], device="cuda")
    live = t < s["lens"].unsqueeze(1)
    block = s["table"].long()[:, t // BLOCK]
    row = (t % BLOCK).expand_as(block)
    get = lambda p: p.transpose(1, 2)[block, row]  # noqa: E731
    k, v = (_values(get(parts[i]), get(parts[2 + i]), get(parts[4 + i])) for i in (0, 1))
    return k, v, live


def _plain_store(s):
    block, row = s["slots"] // BLOCK, s["slots"] % BLOCK
    for i, x in enumerate((s["k"], s["v"])):
        for j, made in enumerate(_quantise(x)):
            s["parts"][2 * j + i].transpose(1, 2)[block, row] = made


def _plain_load(s):
    c = s["case"]
    k, v, live = _read_rows(s, c["kv_heads"], c["d"])
    b, t = live.nonzero(as_tuple=True)
    rows = s["starts"].long()[b] + t
    s["k"][rows] = k[b, t].to(s["k"].dtype)
    s["v"][rows] = v[b, t].to(s["v"].dtype)


def _plain_decode(s):
    c = s["case"]
    d, heads = c["d"], c["kv_heads"]
    k, v, live = _read_rows(s, heads, d)
    k.masked_fill_(~live[:, :, None, None], 0.0)
    v.masked_fill_(~live[:, :, None, None], 0.0)
    q = s["q"].float().unflatten(1, (heads, -1))
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    scores.masked_fill_(~live[:, None, None, :], -math.inf)
    p = scores.sub_(scores.amax(dim=-1, keepdim=True)).exp_()
    out = torch.matmul(p, v.transpose(1, 2)) / p.sum(dim=-1, keepdim=True)
    return out.flatten(1, 2).to(s["out"].dtype)


def _plain_head(s, x, weight, cos, sin):
    """Norm of each head, then rotation of its first rot_dim elements."""
    c = s["case"]
    rot = c["rot_dim"]
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + s["eps"]) * weight.float()
    if c["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, y[..., rot:]], dim=-1).to(s["q"].dtype)


def _plain_rotate(s):
    # the angles of far positions: 64 bits
    angle = s["positions"].double().unsqueeze(1) * s["inv_freq"]
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    q = _plain_head(s, s["q"], s["q_weight"], cos, sin)
    k = _plain_head(s, s["k"], s["k_weight"], cos, sin)
    if s["v_out"] is None:
        return q, k
    at = s["rows"].long()
    s["k_out"][at] = k
    s["v_out"][at] = s["v"]
    return q, s["k_out"], s["v_out"]


def _plain_plan(s):
    lens, free = s["lens"].long(), s["free"]
    new = torch.ones_like(lens) if s["new"] is None else s["new"].long()
    table = s["table"]
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    have, want = (lens + BLOCK - 1) // BLOCK, (lens + new + BLOCK - 1) // BLOCK
    cu_q = torch.cat([zero, new.cumsum(0)])
    cu_k = torch.cat([zero, (lens + new).cumsum(0)])
    off = torch.cat([zero, (want - have).cumsum(0)])
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu_q[1:], t, right=True)
    real = b < lens.shape[0]
    b = b.clamp(max=lens.shape[0] - 1)
    pos = lens[b] + t - cu_q[b]
    column = pos // BLOCK
    fresh = column >= have[b]
    at = (s["next"].long() + off[b] + column - have[b]).clamp(0, free.shape[0] - 1)
    block = torch.where(fresh, free[at], table[b, column.clamp(max=table.shape[1] - 1)])
    first = real & fresh & (pos % BLOCK == 0)
    table[b[first], column[first]] = block[first]
    slots = torch.where(real, block.long() * BLOCK + pos % BLOCK, -1)
    rows = torch.where(real, cu_k[b] + pos, -1).int()
    pos = torch.where(real, pos, 0).int()
    return (table, slots, pos, rows, (lens + new).int(), cu_q.int(), cu_k.int(), s["next"] + off[-1:].int())


def run(s):
    c = s["case"]
    if c["op"] == "store":
        if own:
            s["handle"].store(s["k"], s["v"], s["slots"])
        else:
            _plain_store(s)
        return s["parts"]
    if c["op"] == "load":
        if own:
            s["handle"].load(s["table"], s["lens"], s["starts"], s["k"], s["v"])
        else:
            _plain_load(s)
        return s["k"], s["v"]
    if c["op"] == "decode":
        return s["handle"].decode(s["q"], s["table"], s["lens"], out=s["out"]) if own else _plain_decode(s)
    if c["op"] == "rotate":
        if not own:
            return _plain_rotate(s)
        if not c["place"]:
            return s["handle"].apply(s["q"], s["k"], s["positions"], s["q_weight"], s["k_weight"], q_out=s["q_out"],
                                     k_out=s["k_out"])
        return s["handle"].apply(s["q"], s["k"], s["positions"], s["q_weight"], s["k_weight"], q_out=s["q_out"],
                                 k_out=s["k_out"], v=s["v"], v_out=s["v_out"], kv_rows=s["rows"])
    if not own:
        return _plain_plan(s)
    o = s["handle"].step(s["lens"], s["new"], s["table"], s["free"], s["next"], s["out"])
    return (s["table"], o.slot_mapping, o.positions, o.kv_rows, o.seq_lens, o.cu_q, o.cu_k, o.next_free)


# ----------------------------------------------------------- 64-bit answers
def _scale_table():
    """Values of the scale bytes: five bits of exponent, three behind the point."""
    return torch.tensor([(u & 7) * 2.0 ** -17 if u < 8 else (8 + (u & 7)) * 2.0 ** ((u >> 3) - 18) for u in range(256)],
                        dtype=torch.float64, device="cuda")


def _exact_bytes(x):
    """Packed codes, scale bytes and exponent bytes of finite vectors."""
    x = x.double()
    top = x.abs().amax(dim=-1, keepdim=True)
    frac, e = torch.frexp(top / 240.0)  # top / 240 = frac * 2^e, 0.5 <= frac < 1
    e = torch.where(frac == 0.5, e - 1, e).double()
    e = torch.where(top > 0, e, torch.full_like(e, -126.0)).clamp(min=-126.0)
    y = (x * torch.exp2(-e)).unflatten(-1, (-1, GROUP))
    g = y.abs().amax(dim=-1)
    table = _scale_table()
    u = 1 + torch.searchsorted(7.5 * table[1:], g.contiguous(), right=False)
    u = torch.where(g <= 2.0 ** -18, torch.zeros_like(u), u)
    q = torch.round(y / table[u].clamp(min=2.0 ** -17).unsqueeze(-1)).clamp(-7, 7)
    q = torch.where((u == 0).unsqueeze(-1), torch.zeros_like(q), q).flatten(-2).long() + 8
    return (q[..., 0::2] + 16 * q[..., 1::2]).to(torch.uint8), u.to(torch.uint8), (e + 127).squeeze(-1).to(torch.uint8)


def _exact_rows(s, b, n, heads, d):
    """Sequence b's keys and values [heads, n, d] in 64 bits."""
    page = s["cache"].view(s["blocks"], heads, -1)[s["table"][b, : _blocks(n)].long()].long()
    table = _scale_table()
    both = []
    for i in (0, 1):
        codes = page[:, :, 8 * d * i: 8 * d * (i + 1)].unflatten(2, (16, d // 2))
        at = 16 * d + d * i
        scales = table[page[:, :, at: at + d].unflatten(2, (16, d // 16))]
        exps = torch.exp2(page[:, :, 18 * d + 16 * i: 18 * d + 16 * i + 16].double() - 127.0)
        x = torch.empty(codes.shape[:3] + (d,), dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = codes % 16 - 8, codes // 16 - 8
        x *= scales.repeat_interleave(16, dim=-1) * exps.unsqueeze(-1)
        both.append(x.transpose(0, 1).flatten(1, 2)[:, :n])
    return both


def _exact_rotate(s):
    c = s["case"]
    rot, half = c["rot_dim"], c["rot_dim"] // 2
    i = torch.arange(half, device="cuda")
    first = 2 * i if c["interleaved"] else i
    second = 2 * i + 1 if c["interleaved"] else i + half
    turn = s["positions"].double()[:, None, None] * torch.pow(
        torch.tensor(c["base"], dtype=torch.float64, device="cuda"), -i.double() / half)
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        y = y / torch.sqrt((y * y).sum(dim=-1, keepdim=True) / c["d"] + s["eps"]) * w.double()
        z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(turn), turn)
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    if not c["place"]:
        return tuple(out)
    rows = s["rows"].long()
    k, v = torch.zeros_like(s["k_out"], dtype=torch.float64), torch.zeros_like(s["v_out"], dtype=torch.float64)
    k[rows], v[rows] = out[1], s["v"].double()
    return out[0], k, v


def _exact_plan(s):
    """Request by request, token by token in pieces of a block."""
    lens, new = _requests(s["case"])
    table, free, at = s["table"].tolist(), s["free"].tolist(), int(s["next"])
    slots, positions, rows = [], [], []
    ends, cu_q, cu_k = [], [0], [0]
    for b, (have, n) in enumerate(zip(lens, new)):
        p = have
        while p < have + n:
            if p % BLOCK == 0:
                table[b][p // BLOCK] = free[at]
                at += 1
            stop = min(have + n, p - p % BLOCK + BLOCK)
            start = table[b][p // BLOCK] * BLOCK
            slots.extend(range(start + p % BLOCK, start + p % BLOCK + stop - p))
            positions.extend(range(p, stop))
            rows.extend(range(cu_k[-1] + p, cu_k[-1] + stop))
            p = stop
        ends.append(have + n)
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + have + n)
    behind = s["tokens"] - len(slots)
    return (_ints(table), torch.tensor(slots + [-1] * behind, dtype=torch.int64, device="cuda"),
            _ints(positions + [0] * behind), _ints(rows + [-1] * behind), _ints(ends), _ints(cu_q), _ints(cu_k),
            _ints([at]))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s)
    if case["op"] == "plan":
        return _exact_plan(s)
    d, heads = case["d"], case["kv_heads"]
    if case["op"] == "store":
        parts = []
        for made in zip(*(_exact_bytes(x) for x in (s["k"], s["v"]))):
            for x in made:
                to = torch.zeros((s["blocks"] * BLOCK,) + x.shape[1:], dtype=torch.uint8, device="cuda")
                to[s["slots"]] = x
                parts.append(to.unflatten(0, (-1, BLOCK)).transpose(1, 2))
        return parts
    lens = _lengths(case)
    if case["op"] == "load":
        k, v = torch.zeros_like(s["k"], dtype=torch.float64), torch.zeros_like(s["v"], dtype=torch.float64)
        for b, n in enumerate(lens):
            at = int(s["starts"][b])
            kk, vv = _exact_rows(s, b, n, heads, d)
            k[at:at + n], v[at:at + n] = kk.transpose(0, 1), vv.transpose(0, 1)
        return k, v
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        k, v = _exact_rows(s, b, n, heads, d)
        q = s["q"][b].double().view(heads, -1, d)
        z = torch.einsum("hgd,hmd->hgm", q, k) / math.sqrt(d)
        out[b] = torch.einsum("hgm,hmd->hgd", torch.softmax(z, dim=-1), v).reshape(-1, d)
    return out
