"""Workloads of the 8-bit cache and prompt-attention operators.

Four operators of a serving path, each as real programs call it:

  store   quantises new key and value vectors into the paged 8-bit cache
          (e4m3 codes, one power-of-two scale per vector)
  load    reads sequences of that cache back into packed rows
  decode  attention of one new token per sequence over that cache
  prompt  attention of packed prompt rows over packed keys and values,
          causal against the end of each sequence's keys

``run`` computes them in elementary torch operations, or, where ``own`` is
true, with the library's calls.  ``exact`` gives the same outputs from the
definitions in 64 bits.

A page of the cache holds 16 tokens of one KV head: 16 x d key codes, 16 x d
value codes, 16 key exponent bytes, 16 value exponent bytes; the cache is
[blocks][KV heads][page].  An exponent byte E stands for 2^(E - 127), 255 for
NaN.
"""

import math
import random

import torch

own = False

BLOCK = 16
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's new tokens, 16 sequences of a model with 8 KV heads: latency
        _store("store_step16_d128", 16, 8, 128, "bf16", "step"),
        # the prompts of 64 requests written at once
        _store("store_prefill65536_d128", 65536, 8, 128, "bf16", "prefill"),
        # a prompt of odd length, float inputs, wide heads
        _store("store_prefill9001_d256_f32", 9001, 4, 256, "f32", "prefill"),
        # a short prefix read back before the next chunk of its prompt
        _load("load_1x700_d128", 1, 700, "equal", 1, 8, 128, "bf16", 64),
        # the prefixes of a batch of requests, different lengths, room for a chunk behind each
        _load("load_16xragged16384_d128", 16, 16384, "ragged", 2, 8, 128, "bf16", 256),
        # one short conversation: latency
        _decode("decode_1x130_d128", 1, 130, "equal", 3, 32, 8, 128, "bf16", "bf16"),
        # a batch of chats at 8192 tokens
        _decode("decode_16x8192_d128", 16, 8192, "equal", 4, 32, 8, 128, "bf16", "bf16"),
        # long documents of different lengths, 64 query heads
        _decode("decode_4xragged131072_d128", 4, 131072, "ragged", 5, 64, 8, 128, "bf16", "bf16"),
        # wide heads, float queries and outputs
        _decode("decode_8xragged32768_d256_f32", 8, 32768, "ragged", 6, 32, 4, 256, "f32", "f32"),
        # one long prompt (the largest case)
        _prompt("prompt_1x8192_d128", 1, 8192, 0, "equal", 7, 32, 8, 128, "bf16", True, False),
        # a packed batch of prompts of 1 to 2048 tokens, rows of a fused projection
        _prompt("prompt_16xragged2048_d128", 16, 2048, 0, "ragged", 8, 32, 8, 128, "bf16", True, True),
        # a small chunk behind a long prefix, wide heads
        _prompt("prompt_1x96_after16384_d256", 1, 96, 16384, "equal", 9, 32, 4, 256, "f16", True, False),
    ]


def _store(name, tokens, kv_heads, d, dtype, kind):
    return dict(name=name, op="store", tokens=tokens, kv_heads=kv_heads, d=d, dtype=dtype, kind=kind)


def _load(name, batch, longest, spread, mix, kv_heads, d, dtype, room):
    return dict(name=name, op="load", batch=batch, longest=longest, spread=spread, mix=mix, kv_heads=kv_heads, d=d,
                dtype=dtype, room=room)


def _decode(name, batch, longest, spread, mix, q_heads, kv_heads, d, dtype, out_dtype):
    return dict(name=name, op="decode", batch=batch, longest=longest, spread=spread, mix=mix, q_heads=q_heads,
                kv_heads=kv_heads, d=d, dtype=dtype, out_dtype=out_dtype)


def _prompt(name, batch, longest, prefix, spread, mix, q_heads, kv_heads, d, dtype, causal, fused):
    return dict(name=name, op="prompt", batch=batch, longest=longest, prefix=prefix, spread=spread, mix=mix,
                q_heads=q_heads, kv_heads=kv_heads, d=d, dtype=dtype, causal=causal, fused=fused)


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["store", "load", "decode", "decode", "prompt", "prompt"])
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
    else:
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        c = _prompt("", _log(rng, 1, 24), _log(rng, 1, 8192), rng.choice([0, 0, _log(rng, 1, 32768)]), spread, mix,
                    group * kv_heads, kv_heads, d, rng.choice(["bf16", "bf16", "f16"]), rng.random() < 0.8,
                    rng.random() < 0.4)
        if c["prefix"]:
            c["fused"] = False  # keys that come from a cache are no rows of the projection
        # the largest listed case's rows x keys x width
        while c["batch"] * c["q_heads"] * c["longest"] * (c["longest"] + c["prefix"]) * d > 32 * 8192 * 8192 * 128 // 2:
            if c["longest"] >= c["prefix"]:
                c["longest"] //= 2
            else:
                c["prefix"] //= 2
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


def _prefixes(case):
    p, b = case["prefix"], case["batch"]
    if p == 0 or case["spread"] == "equal":
        return [p] * b
    rng = random.Random(case["mix"] + 1)
    return [rng.randint(0, p) for _ in range(b)]


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    d = case["d"]
    if case["op"] == "store":
        vec = case["tokens"] * case["kv_heads"] * 2
        return {"bytes": vec * (d * size[case["dtype"]] + d + 1) + 8 * case["tokens"], "flops": 0}
    lens = _lengths(case)
    n = sum(lens)
    if case["op"] == "load":
        return {"bytes": n * case["kv_heads"] * 2 * (d + 1 + d * size[case["dtype"]]), "flops": 0}
    if case["op"] == "decode":
        rows = case["batch"] * case["q_heads"]
        return {"bytes": n * case["kv_heads"] * 2 * (d + 1) + rows * d * (size[case["dtype"]] + size[case["out_dtype"]]),
                "flops": 4 * d * n * (case["q_heads"])}
    pre = _prefixes(case)
    keys = n + sum(pre)
    pairs = sum(a * p + (a * (a + 1) // 2 if case["causal"] else a * a) for a, p in zip(lens, pre))
    return {"bytes": 2 * d * (2 * n * case["q_heads"] + 2 * keys * case["kv_heads"]) + 4 * n * case["q_heads"],
            "flops": 4 * d * case["q_heads"] * pairs}


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


def _page_parts(cache, blocks, heads, d):
    """The cache's key codes, value codes (as e4m3), key and value exponent bytes, as views."""
    p = cache.view(blocks, heads, 32 * d + 32)
    codes = p[:, :, : 32 * d].view(torch.float8_e4m3fn)
    return (codes[:, :, : 16 * d].unflatten(2, (16, d)), codes[:, :, 16 * d:].unflatten(2, (16, d)),
            p[:, :, 32 * d: 32 * d + 16], p[:, :, 32 * d + 16:])


def _filled_cache(g, blocks, heads, d):
    """A cache whose every slot holds a quantised vector."""
    cache = torch.empty(blocks * heads * (32 * d + 32), dtype=torch.uint8, device="cuda")
    parts = _page_parts(cache, blocks, heads, d)
    for i in (0, 1):
        gain = torch.exp(0.5 * torch.randn((heads, d), generator=g, device="cuda")) if i == 0 else 1.0
        for at in range(0, blocks, 4096):
            n = min(4096, blocks - at)
            x = torch.randn((n, BLOCK, heads, d), generator=g, device="cuda") * gain
            codes, exps = _quantise(x)
            parts[i][at:at + n].view(torch.uint8).copy_(codes.view(torch.uint8).transpose(1, 2))
            parts[2 + i][at:at + n] = exps.transpose(1, 2)
    return cache


def _table(g, lens):
    """Each sequence's blocks: a permutation of the pool, as after some hours of serving."""
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
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
    return tq.TQF8Cache(head_dim=case["d"], num_kv_heads=heads, num_q_heads=case.get("q_heads", heads),
                        num_blocks=blocks, max_batch=case.get("batch", 1), max_blocks_per_seq=columns, cache=cache)


def prepare(case, seed):
    g = _generator(seed)
    d, heads = case["d"], case["kv_heads"]
    s = {"case": case}
    if case["op"] == "store":
        n = case["tokens"]
        s["k"] = _vectors(g, n, heads, d, DTYPES[case["dtype"]], True)
        s["v"] = _vectors(g, n, heads, d, DTYPES[case["dtype"]], False)
        if case["kind"] == "prefill":  # consecutive positions in blocks from all over the pool
            blocks = (n + BLOCK - 1) // BLOCK
            perm = torch.randperm(blocks, generator=g, device="cuda")
            t = torch.arange(n, device="cuda")
            s["slots"] = perm[t // BLOCK] * BLOCK + t % BLOCK
        else:  # one token of each sequence, each in a block of its own
            blocks = n
            s["slots"] = torch.randperm(n, generator=g, device="cuda") * BLOCK + torch.randint(
                0, BLOCK, (n,), generator=g, device="cuda")
        s["blocks"] = blocks
        s["cache"] = torch.zeros(blocks * heads * (32 * d + 32), dtype=torch.uint8, device="cuda")
        if own:
            s["handle"] = _handle(case, blocks, 1, s["cache"])
        return s
    lens = _lengths(case)
    if case["op"] in ("load", "decode"):
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
    pre = _prefixes(case)
    dtype = DTYPES[case["dtype"]]
    n, m, hq = sum(lens), sum(lens) + sum(pre), case["q_heads"]
    s["longest"], s["longest_k"] = max(lens), max(a + p for a, p in zip(lens, pre))
    s["cu_q"] = _ints(_starts(lens))
    s["cu_k"] = _ints(_starts([a + p for a, p in zip(lens, pre)]))
    q, k = _vectors(g, n, hq, d, dtype, False), _vectors(g, m, heads, d, dtype, True)
    v = _vectors(g, m, heads, d, dtype, False)
    if case["fused"]:
        s["qkv"] = torch.cat([q, k, v], dim=1)
        q, k, v = s["qkv"].split([hq, heads, heads], dim=1)
    s["q"], s["k"], s["v"] = q, k, v
    s["out"] = torch.zeros((n, hq, d), dtype=dtype, device="cuda")
    s["lse"] = torch.zeros((n, hq), dtype=torch.float32, device="cuda")
    if own:
        import turboquant_bit_kv_tq_gb300 as tq

        s["plan"] = tq.TQPrompt(head_dim=d, num_kv_heads=heads, num_q_heads=hq, dtype=dtype, max_batch=case["batch"],
                                max_tokens=n)
    return s


# -------------------------------------------------------------- plain forms
def _quantise(x):
    """x [..., d] -> (e4m3 codes, exponent bytes [...])."""
    x = x.float()
    top = x.abs().amax(dim=-1)
    bad = ~torch.isfinite(top)
    bits = torch.where(bad, torch.zeros_like(top), top).view(torch.int32)
    # smallest e with top <= 448 * 2^e = 1.75 * 2^(e + 8)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(1, 254)
    codes = torch.ldexp(x, (127 - byte).unsqueeze(-1))
    codes = torch.where(bad.unsqueeze(-1), torch.zeros_like(codes), codes).to(torch.float8_e4m3fn)
    return codes, torch.where(bad, torch.full_like(byte, 255), byte).to(torch.uint8)


def _values(codes, exps):
    e = exps.int() - 127
    x = torch.ldexp(codes.float(), e.unsqueeze(-1))
    return torch.where((exps == 255).unsqueeze(-1), torch.full_like(x, math.nan), x)


def _read_rows(s, heads, d):
    """Keys and values [batch, longest, heads, d] as float, and which rows are tokens."""
    parts = _page_parts(s["cache"], s["blocks"], heads, d)
    t = torch.arange(s["longest"], device="cuda")
    live = t < s["lens"].unsqueeze(1)
    block = s["table"].long()[:, t // BLOCK]
    row = (t % BLOCK).expand_as(block)
    get = lambda p: p.view(torch.uint8).transpose(1, 2)[block, row]  # noqa: E731
    kv = [_values(get(parts[i]).view(torch.float8_e4m3fn), get(parts[2 + i])) for i in (0, 1)]
    return kv[0], kv[1], live


def _softmax_values(scores, live, values):
    """softmax over the last axis of the live scores, times values; a row with no live score gets 0.  Also the
    logarithm of the sum of exponentials."""
    scores.masked_fill_(~live, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, values) / torch.where(total == 0, torch.ones_like(total), total)
    return out, (total.log() + top).squeeze(-1)


def _plain_store(s):
    c = s["case"]
    parts = _page_parts(s["cache"], s["blocks"], c["kv_heads"], c["d"])
    block, row = s["slots"] // BLOCK, s["slots"] % BLOCK
    for i, x in enumerate((s["k"], s["v"])):
        codes, exps = _quantise(x)
        parts[i].view(torch.uint8).transpose(1, 2)[block, row] = codes.view(torch.uint8)
        parts[2 + i].transpose(1, 2)[block, row] = exps


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
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    out, _ = _softmax_values(scores, live[:, None, None, :], v.transpose(1, 2))
    return out.flatten(1, 2).to(s["out"].dtype)


def _plain_prompt(s):
    c = s["case"]
    d, heads = c["d"], c["kv_heads"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cu_q.diff(), cu_k.diff()
    i = torch.arange(s["longest"], device="cuda")
    j = torch.arange(s["longest_k"], device="cuda")
    here_q, here_k = i < lq.unsqueeze(1), j < lk.unsqueeze(1)
    at_q = (cu_q[:-1].unsqueeze(1) + i).clamp(max=s["q"].shape[0] - 1)
    at_k = (cu_k[:-1].unsqueeze(1) + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"].float()[at_q].unflatten(2, (heads, -1)).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, Lq, d]
    k = s["k"].float()[at_k].permute(0, 2, 3, 1).unsqueeze(2)  # [B, Hkv, 1, d, Lk]
    v = s["v"].float()[at_k].masked_fill_(~here_k[:, :, None, None], 0.0).permute(0, 2, 1, 3)  # [B, Hkv, Lk, d]
    shape = q.shape[:4]
    scores = torch.matmul(q.flatten(2, 3), k.squeeze(2)).unflatten(2, shape[2:4]).mul_(1.0 / math.sqrt(d))
    live = here_k[:, None, :]
    if c["causal"]:
        live = live & (j <= i.unsqueeze(1) + (lk - lq)[:, None, None])
    out, lse = _softmax_values(scores, live[:, None, None], v.unsqueeze(2))
    b, t = here_q.nonzero(as_tuple=True)
    out = out.permute(0, 3, 1, 2, 4)[b, t].flatten(1, 2)
    lse = lse.permute(0, 3, 1, 2)[b, t].flatten(1, 2)
    return out.to(s["out"].dtype), lse


def run(s):
    c = s["case"]
    if c["op"] == "store":
        if own:
            s["handle"].store(s["k"], s["v"], s["slots"])
        else:
            _plain_store(s)
        return _page_parts(s["cache"], s["blocks"], c["kv_heads"], c["d"])
    if c["op"] == "load":
        if own:
            s["handle"].load(s["table"], s["lens"], s["starts"], s["k"], s["v"])
        else:
            _plain_load(s)
        return s["k"], s["v"]
    if c["op"] == "decode":
        return s["handle"].decode(s["q"], s["table"], s["lens"], out=s["out"]) if own else _plain_decode(s)
    if own:
        s["plan"].attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out=s["out"], lse=s["lse"],
                            causal=c["causal"])
        return s["out"], s["lse"]
    return _plain_prompt(s)


# ----------------------------------------------------------- 64-bit answers
def _exact_codes(x):
    """x * 2^-e for the smallest e in [-126, 127] with max |x| <= 448 * 2^e, and e + 127."""
    x = x.double()
    top = x.abs().amax(dim=-1, keepdim=True)
    frac, e = torch.frexp(top / 448.0)  # top / 448 = frac * 2^e, 0.5 <= frac < 1
    e = torch.where(frac == 0.5, e - 1, e).double()
    e = torch.where(top > 0, e, torch.full_like(e, -126.0)).clamp(min=-126.0)
    return x * torch.exp2(-e), (e + 127).squeeze(-1).to(torch.uint8)


def _e4m3_table():
    """The 256 values of the 8-bit codes."""
    vals = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        vals.append(-x if c >> 7 else x)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _exact_rows(s, b, n, heads, d):
    """Sequence b's keys and values [heads, n, d] in 64 bits."""
    page = s["cache"].view(s["blocks"], heads, -1)[s["table"][b, : (n + BLOCK - 1) // BLOCK].long()]
    table = _e4m3_table()
    both = []
    for i in (0, 1):
        codes = table[page[:, :, 16 * d * i: 16 * d * (i + 1)].int()].unflatten(2, (16, d))
        scale = torch.exp2(page[:, :, 32 * d + 16 * i: 32 * d + 16 * (i + 1)].double() - 127.0)
        both.append((codes * scale.unsqueeze(-1)).transpose(0, 1).flatten(1, 2)[:, :n])
    return both


def _exact_attention(q, k, v, d, offset):
    """q [heads, G, n, d], k and v [heads, m, d]; row i sees keys 0 .. i + offset (all keys where offset is None)."""
    out, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    if k.shape[1] == 0:
        return out, lse
    for h in range(q.shape[0]):
        z = torch.einsum("gnd,md->gnm", q[h], k[h]) / math.sqrt(d)
        if offset is not None:
            i = torch.arange(q.shape[2], device="cuda").unsqueeze(1)
            z = torch.where(torch.arange(k.shape[1], device="cuda") <= i + offset, z, -math.inf)
        lse[h] = torch.logsumexp(z, dim=-1)
        out[h] = torch.einsum("gnm,md->gnd", torch.softmax(z, dim=-1).nan_to_num_(0.0), v[h])
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    d, heads = case["d"], case["kv_heads"]
    if case["op"] == "store":
        slots, parts = s["slots"], []
        made = [_exact_codes(x) for x in (s["k"], s["v"])]
        for codes, _ in made:
            to = torch.zeros((s["blocks"] * BLOCK, heads, d), dtype=torch.float64, device="cuda")
            to[slots] = codes
            parts.append(to.view(s["blocks"], BLOCK, heads, d).transpose(1, 2))
        for _, exps in made:
            to = torch.zeros((s["blocks"] * BLOCK, heads), dtype=torch.uint8, device="cuda")
            to[slots] = exps
            parts.append(to.view(s["blocks"], BLOCK, heads).transpose(1, 2))
        return tuple(parts)
    lens = _lengths(case)
    if case["op"] == "load":
        k, v = torch.zeros_like(s["k"], dtype=torch.float64), torch.zeros_like(s["v"], dtype=torch.float64)
        for b, n in enumerate(lens):
            at = int(s["starts"][b])
            kk, vv = _exact_rows(s, b, n, heads, d)
            k[at:at + n], v[at:at + n] = kk.transpose(0, 1), vv.transpose(0, 1)
        return k, v
    if case["op"] == "decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            k, v = _exact_rows(s, b, n, heads, d)
            q = s["q"][b].double().view(heads, -1, 1, d)
            out[b] = _exact_attention(q, k, v, d, None)[0].reshape(-1, d)
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(case["batch"]):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        q = s["q"][cu_q[b]:cu_q[b + 1]].double().view(n, heads, -1, d).permute(1, 2, 0, 3)
        k, v = (s[x][cu_k[b]:cu_k[b + 1]].double().transpose(0, 1) for x in ("k", "v"))
        o, z = _exact_attention(q, k, v, d, m - n if case["causal"] else None)
        out[cu_q[b]:cu_q[b + 1]] = o.permute(2, 0, 1, 3).flatten(1, 2)
        lse[cu_q[b]:cu_q[b + 1]] = z.permute(2, 0, 1).flatten(1, 2)
    return out, lse
