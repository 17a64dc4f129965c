"""Cases of the cache operators: appending keys and values to a paged cache with the position rotation applied on
the way (16-bit caches, and 8-bit caches with a scale for each block of tokens and head), and attention over the
8-bit cache, for one or several new tokens per sequence.

``run`` computes each operator in plain fp32 torch operations, or, with ``own`` set, through the package's entry
points; ``exact`` computes the same results in 64 bits.

The 8-bit cache: e4m3 values, laid out as the 16-bit caches are ([num_blocks, kv_heads, block_size, head_dim]), and
one fp32 scale per (block, KV head) for K and one for V; a stored value stands for value * scale.  The append writes
scales that are powers of two: the smallest one under which the largest magnitude among the block's new tokens fits
e4m3's 448, and never below the scale that the block's earlier tokens already have (those are then re-quantised).
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126


def _attend(name, dtype, seqs, heads, kv_heads, head_dim, block_size, q_len, partition, lens, len_min, len_max, pool=1.25, **more):
    return dict(name=name, op="attend_q8", dtype=dtype, seqs=seqs, heads=heads, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size,
                q_len=q_len, partition=partition, lens=lens, len_min=len_min, len_max=len_max, pool=pool, **more)


def _append(name, op, dtype, seqs, heads, kv_heads, head_dim, block_size, new, new_min, past_max, rotary, interleaved, padding=0):
    return dict(name=name, op=op, dtype=dtype, seqs=seqs, heads=heads, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size,
                new=new, new_min=new_min, past_max=past_max, rotary=rotary, interleaved=interleaved, padding=padding)


def listed():
    return [
        # One request's next token: the smallest append there is; its launch and its chain of dependent loads are its time.
        _append("append_one_token", "append", "f16", 1, 8, 2, 128, 16, 1, 1, 1000, 128, False),
        # A serving step that mixes prompts and running requests: ragged counts of new tokens, empty slots, padding rows behind the last one.
        _append("append_ragged_prompts", "append", "bf16", 64, 64, 8, 128, 32, 2048, 0, 4096, 128, False, padding=37),
        # The next token of every request of a batch, into blocks that are partly filled.
        _append("append_q8_batch_decode", "append_q8", "bf16", 32, 32, 8, 128, 16, 1, 1, 8191, 128, False),
        # A prompt's chunk for two requests, into an 8-bit cache.
        _append("append_q8_chunk", "append_q8", "f16", 2, 32, 8, 128, 16, 2048, 2048, 28000, 64, True),
        # Ragged prompts into an 8-bit cache: the largest append.
        _append("append_q8_ragged_prompts", "append_q8", "bf16", 64, 64, 8, 128, 32, 2048, 0, 4096, 128, False, padding=37),
        # One short request: the call's latency.
        _attend("attend_q8_tiny", "f16", 1, 8, 2, 128, 16, 1, 512, "fixed", 1000, 1000),
        # A batch of requests at all stages of their answers.
        _attend("attend_q8_batch_decode", "bf16", 32, 32, 8, 128, 16, 1, 512, "uniform", 1, 8192),
        # One request with a long document.
        _attend("attend_q8_long_100k", "bf16", 1, 32, 4, 128, 16, 1, 512, "fixed", 100000, 100000),
        # A serving batch with a long tail of lengths.
        _attend("attend_q8_ragged_serving", "bf16", 64, 64, 8, 128, 32, 1, 512, "lognormal", 16, 32768),
        # The whole card's worth of long requests: the largest read.
        _attend("attend_q8_stress", "f16", 8, 64, 8, 128, 16, 1, 1024, "fixed", 131072, 131072, pool=1.07),
        # Checking 16 guessed tokens for each request of a batch.
        _attend("attend_q8_verify_16", "bf16", 32, 32, 8, 128, 16, 16, 512, "uniform", 16, 8192),
        # A prompt's chunk for two requests, over the chunk itself and what came before it.
        _attend("attend_q8_chunk", "bf16", 2, 32, 8, 128, 16, 1024, 512, "uniform", 8192, 9216),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["append", "append_q8", "attend_q8", "attend_q8", "attend_q8"])
    dtype = rng.choice(["bf16", "f16"])
    head_dim = rng.choice([64, 128, 128, 256])
    block_size = rng.choice([8, 16, 16, 32, 64])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    heads = kv_heads * group
    if op != "attend_q8":
        seqs = log(1, 96)
        most = max(1, min(2048, (64 * 1024 * 80 * 128) // (seqs * (heads + 2 * kv_heads) * head_dim)))
        new = rng.choice([1, rng.randint(1, 16), log(1, most)])
        new = min(new, most)
        new_min = rng.choice([0, new])
        rotary = rng.choice([head_dim, head_dim // 2, 32])
        c = _append("", op, dtype, seqs, heads, kv_heads, head_dim, block_size, new, new_min, log(1, 9000), rotary, rng.random() < 0.3, rng.choice([0, 0, 5]))
    else:
        seqs = log(1, 96)
        q_len = rng.choice([1, 1, 1, rng.randint(2, 9), rng.randint(10, 64), log(16, 1024)])
        # Neither more to read nor more to compute than the largest listed cases.
        by_read = 10 ** 9 // (seqs * kv_heads * head_dim)
        by_work = 290 * 10 ** 9 // (4 * seqs * q_len * heads * head_dim)
        # Plain scores of the padded batch stay within a few GB.
        by_room = 600 * 10 ** 6 // (seqs * q_len * heads)
        hi = min(140000, by_read, by_work, by_room)
        if hi < q_len:
            q_len, hi = 1, max(1, min(by_read, 600 * 10 ** 6 // (seqs * heads)))
        len_max = log(max(q_len, 1), max(q_len, hi))
        lens = rng.choice(["uniform", "uniform", "fixed", "lognormal"])
        len_min = rng.choice([0, min(1, len_max), min(q_len, len_max)]) if lens != "fixed" else len_max
        c = _attend("", dtype, seqs, heads, kv_heads, head_dim, block_size, q_len, rng.choice([256, 512, 1024, 1000]), lens, len_min, len_max)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------------ inputs


def _lengths(case, rand):
    """Each sequence's length, on the host: a program that schedules requests knows them."""
    lo, hi, n = case["len_min"], case["len_max"], case["seqs"]
    if case["lens"] == "fixed":
        return [hi] * n
    if case["lens"] == "uniform":
        return torch.randint(lo, hi + 1, (n,), generator=rand).tolist()
    median = max(1.0, hi / 16)
    z = torch.randn(n, generator=rand, dtype=torch.float64)
    return [int(v) for v in torch.exp(math.log(median) + z).round().clamp(max(lo, 0), hi).tolist()]


def _counts(case, rand):
    """Each sequence's new tokens, new_min to new of them, tokens(case) in all: the rows of a batch that a scheduler fills up."""
    lo, hi, n = case["new_min"], case["new"], case["seqs"]
    new = torch.randint(lo, hi + 1, (n,), generator=rand).tolist()
    over = sum(new) - _tokens(case)
    for b in range(n):
        step = min(over, new[b] - lo) if over > 0 else max(over, new[b] - hi)
        new[b] -= step
        over -= step
    return new


def _tokens(case):
    return case["seqs"] * (case["new"] + case["new_min"]) // 2


def _tables(used, pool, width, rand):
    """Block tables over a shuffled pool; entries past a sequence's last block hold -1."""
    perm = torch.randperm(pool, generator=rand).to(torch.int32)
    table = torch.full((len(used), max(1, width)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.to(DEVICE)


def _scale_of(amax):
    """The smallest power of two s (from 2^-126 up) with amax <= 448 s."""
    mantissa, exponent = torch.frexp(amax)  # amax = mantissa * 2^exponent, and 448 = 0.875 * 2^9
    exponent = exponent - 9 + (mantissa > 0.875).to(exponent.dtype)
    power = ((exponent.clamp(-126, 127) + 127).to(torch.int32) << 23).view(torch.float32)  # 2^exponent, from its bits
    return torch.where(amax > 0, power, torch.full_like(amax, MIN_SCALE))


def _filled(pool, case, gen):
    """An 8-bit cache with every row written: N(0, 1) values; K with some channels eight times as large, block scales as the append leaves them."""
    kv, bs, d = case["kv_heads"], case["block_size"], case["head_dim"]
    caches, scales = [], []
    for which in range(2):
        cache = torch.empty((pool, kv, bs, d), dtype=torch.uint8, device=DEVICE).view(E4M3)
        scale = torch.empty((pool, kv), dtype=torch.float32, device=DEVICE)
        step = max(1, (64 << 20) // (kv * bs * d))
        for at in range(0, pool, step):
            x = torch.randn((min(step, pool - at), kv, bs, d), generator=gen, device=DEVICE)
            if which == 0:
                x[..., ::21] *= 8.0
            s = _scale_of(x.abs().amax(dim=(2, 3)))
            scale[at:at + step] = s
            cache[at:at + step] = (x / s[:, :, None, None]).to(E4M3)
        caches.append(cache)
        scales.append(scale)
    return caches, scales


def prepare(case, seed):
    rand = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(seed + 1)
    dt = DTYPE[case["dtype"]]
    bs, kv, d, heads, n = case["block_size"], case["kv_heads"], case["head_dim"], case["heads"], case["seqs"]
    s = {"case": case}
    if case["op"] == "attend_q8":
        lens = _lengths(case, rand)
        used = [-(-x // bs) for x in lens]
        pool = max(1, math.ceil(case["pool"] * sum(used)))
        (s["key_cache"], s["value_cache"]), (s["k_scales"], s["v_scales"]) = _filled(pool, case, gen)
        s["tables"] = _tables(used, pool, -(-case["len_max"] // bs), rand)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
        s["hint"] = max(1, max(lens))
        shape = (n, heads, d) if case["q_len"] == 1 else (n, case["q_len"], heads, d)
        s["query"] = torch.randn(shape, generator=gen, device=DEVICE).to(dt)
        s["scale"] = 1.0 / math.sqrt(d)
        if own:
            import paged_kv_decode_v2_gb300 as pa
            s["out"] = torch.empty_like(s["query"])
            parts = pa.num_partitions(s["hint"], case["partition"])
            s["workspace"] = pa.alloc_workspace(n, heads, d, max(1, parts), device=DEVICE, q_len=case["q_len"])
        return s
    new = _counts(case, rand)
    past = torch.randint(0, case["past_max"] + 1, (n,), generator=rand).tolist()
    lens = [a + b for a, b in zip(past, new)]
    width = -(-(case["past_max"] + case["new"]) // bs)
    pool = n * width
    s["tables"] = _tables([-(-x // bs) for x in lens], pool, width, rand)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEVICE)
    rows = max(1, starts[-1] + case["padding"])
    # One projection's output, of which the query, key and value are parts.
    qkv = torch.randn((rows, heads + 2 * kv, d), generator=gen, device=DEVICE).to(dt)
    s["query"], s["key"], s["value"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    s["query_out"] = torch.zeros((rows, heads, d), dtype=dt, device=DEVICE)
    # Cosines and sines of every position, computed in 64 bits: [positions, rotary], the cosines first.
    half = case["rotary"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEVICE) / half)
    angle = torch.arange(case["past_max"] + case["new"] + 1, dtype=torch.float64, device=DEVICE)[:, None] * inv
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    if case["op"] == "append":
        shape = (pool, kv, bs, d)
        s["key_cache"] = torch.randn(shape, generator=gen, device=DEVICE).to(dt)
        s["value_cache"] = torch.randn(shape, generator=gen, device=DEVICE).to(dt)
    else:
        (s["key_cache"], s["value_cache"]), (s["k_scales"], s["v_scales"]) = _filled(pool, case, gen)
    return s


# ------------------------------------------------------------------------------------------- one pass, plain form


def _rotated(x, cos, sin, interleaved):
    """x [tokens, heads, d] in fp32 with its first 2 * cos.shape[1] dims rotated; cos, sin [tokens, half]."""
    half = cos.shape[1]
    c, s = cos[:, None, :], sin[:, None, :]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    lo, hi = a * c - b * s, b * c + a * s
    turned = torch.stack([lo, hi], dim=-1).flatten(-2) if interleaved else torch.cat([lo, hi], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _places(s):
    """For each new token: its row, sequence, position, physical block and row in the block."""
    case, rows = s["case"], s["key"].shape[0]
    bs, starts = case["block_size"], s["starts"].long()
    row = torch.arange(rows, device=DEVICE)
    seq = torch.searchsorted(starts, row, right=True) - 1
    live = row < starts[-1]
    row, seq = row[live], seq[live]
    pos = s["lens"].long()[seq] - starts[seq + 1] + row
    return row, seq, pos, s["tables"].long()[seq, pos // bs], pos % bs


def _append_plain(s):
    case = s["case"]
    row, seq, pos, block, at = _places(s)
    half = case["rotary"] // 2
    cos, sin = s["cos_sin"][pos, :half], s["cos_sin"][pos, half:]
    q = _rotated(s["query"][row].float(), cos, sin, case["interleaved"])
    k = _rotated(s["key"][row].float(), cos, sin, case["interleaved"])
    s["query_out"][row] = q.to(s["query_out"].dtype)
    if case["op"] == "append":
        s["key_cache"][block, :, at] = k.to(s["key_cache"].dtype)
        s["value_cache"][block, :, at] = s["value"][row]
        return {"query": s["query_out"], "key_cache": s["key_cache"], "value_cache": s["value_cache"]}
    bs = case["block_size"]
    starts = s["starts"].long()
    past = (s["lens"].long() - (starts[1:] - starts[:-1]))[seq]
    kept = (past - pos // bs * bs).clamp(0, bs)  # rows of the token's block that earlier tokens fill
    v = s["value"][row].float()
    for x, cache, scales in ((k, "key_cache", "k_scales"), (v, "value_cache", "v_scales")):
        old = s[scales]
        amax = torch.zeros_like(old).index_reduce_(0, block, x.abs().amax(dim=-1), "amax")
        fresh = torch.zeros_like(old[:, 0], dtype=torch.bool).index_fill_(0, block[kept == 0], True)
        touched = torch.zeros_like(fresh).index_fill_(0, block, True)
        scale = _scale_of(amax)
        scale = torch.where(fresh[:, None], scale, torch.maximum(scale, old))
        scale = torch.where(touched[:, None], scale, old)
        held = s[cache].view(torch.uint8)
        first = (pos == past) & (kept > 0)  # one token of each partly filled block: its kept rows take the new scale
        again = held[block[first]].view(E4M3).float() * (old / scale)[block[first]][:, :, None, None]
        keep = torch.arange(bs, device=DEVICE) < kept[first][:, None]
        held[block[first]] = torch.where(keep[:, None, :, None], again.to(E4M3).view(torch.uint8), held[block[first]])
        held[block, :, at] = (x / scale[block][:, :, None]).to(E4M3).view(torch.uint8)
        s[scales].copy_(scale)
    return {"query": s["query_out"], "key_cache": s["key_cache"], "value_cache": s["value_cache"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _gathered(s, cache, scales):
    """[seqs, kv_heads, tokens, head_dim] in fp32."""
    ids = s["tables"].clamp(min=0).long()
    x = s[cache].view(torch.uint8)[ids].view(E4M3).float() * s[scales][ids][..., None, None]
    n, blocks, kv, bs, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, kv, blocks * bs, d)


def _attend_plain(s):
    case, q = s["case"], s["query"]
    n, q_len, kv, d = case["seqs"], case["q_len"], case["kv_heads"], case["head_dim"]
    group = case["heads"] // kv
    q = q.view(n, q_len, kv, group, d).permute(0, 2, 1, 3, 4).reshape(n, kv, q_len * group, d).float()
    scores = torch.matmul(q, _gathered(s, "key_cache", "k_scales").transpose(2, 3)).mul_(s["scale"])
    tokens = torch.arange(scores.shape[-1], device=DEVICE)
    # New token i sits at position length - q_len + i and sees the positions up to its own.
    end = s["lens"][:, None] - q_len + 1 + torch.arange(q_len, device=DEVICE)
    hidden = tokens >= end.repeat_interleave(group, dim=1)[:, None, :, None]
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, _gathered(s, "value_cache", "v_scales")) / torch.where(total > 0, total, torch.ones_like(total))
    return out.view(n, kv, q_len, group, d).permute(0, 2, 1, 3, 4).reshape(s["query"].shape).to(s["query"].dtype)


def run(state):
    s, case = state, state["case"]
    if not own:
        return _attend_plain(s) if case["op"] == "attend_q8" else _append_plain(s)
    import paged_kv_decode_v2_gb300 as pa
    if case["op"] == "attend_q8":
        return pa.pa_decode_q8(s["query"], s["key_cache"], s["value_cache"], s["k_scales"], s["v_scales"], s["tables"], s["lens"], s["scale"],
                               case["partition"], s["out"], *s["workspace"], max_seq_len_hint=s["hint"])
    if case["op"] == "append":
        pa.pa_kv_append(s["key"], s["value"], s["tables"], s["lens"], s["key_cache"], s["value_cache"], cos_sin=s["cos_sin"],
                        interleaved=case["interleaved"], query=s["query"], query_out=s["query_out"], token_starts=s["starts"])
        return {"query": s["query_out"], "key_cache": s["key_cache"], "value_cache": s["value_cache"]}
    pa.pa_kv_append_q8(s["key"], s["value"], s["tables"], s["lens"], s["key_cache"], s["value_cache"], s["k_scales"], s["v_scales"],
                       cos_sin=s["cos_sin"], interleaved=case["interleaved"], query=s["query"], query_out=s["query_out"], token_starts=s["starts"])
    return {"query": s["query_out"], "key_cache": s["key_cache"], "value_cache": s["value_cache"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def work(case):
    kv, d, heads, n = case["kv_heads"], case["head_dim"], case["heads"], case["seqs"]
    if case["op"] == "attend_q8":
        lens = {"fixed": case["len_max"], "uniform": (case["len_min"] + case["len_max"]) / 2, "lognormal": case["len_max"] / 16 * 1.5}[case["lens"]]
        tokens = n * lens
        q = case["q_len"]
        # Of q new tokens, the i-th sees q - 1 - i tokens fewer than the last.
        seen = n * q * max(lens - (q - 1) / 2, lens / 2)
        read = tokens * kv * d * 2 + tokens / case["block_size"] * (kv * 8 + 4)
        return {"bytes": read + 2 * n * q * heads * d * 2, "flops": 4 * seen * heads * d}
    tokens = _tokens(case)
    elem = 2 if case["op"] == "append" else 1
    read = tokens * (heads + 2 * kv) * d * 2
    written = tokens * (heads * d * 2 + 2 * kv * d * elem)
    # The cosines and sines of each token's position, 3 operations for each rotated value.
    return {"bytes": max(1.0, read + written + tokens * case["rotary"] * 4), "flops": max(1.0, tokens * (heads + kv) * case["rotary"] * 3)}


# ----------------------------------------------------------------------------------------------- in 64 bits


def _two_to(exponent):
    """2^exponent in 64 bits, exactly, for exponents from -200 to 200."""
    return torch.tensor([2.0 ** e for e in range(-200, 201)], dtype=torch.float64, device=DEVICE)[exponent.long() + 200]


def _nearest_e4m3(x):
    """The nearest e4m3 value to each x of at most 448 in magnitude, ties to even, in 64 bits."""
    step = _two_to((torch.frexp(x.abs())[1] - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_attend(s):
    case, out = s["case"], []
    bs, kv, d, q_len = case["block_size"], case["kv_heads"], case["head_dim"], case["q_len"]
    group = case["heads"] // kv
    for b, length in enumerate(s["lens"].tolist()):
        q = s["query"][b].double().view(q_len, kv, group, d)
        ids = s["tables"][b, :-(-length // bs)].long()
        o = torch.zeros_like(q)
        for h in range(kv if length else 0):
            k = (s["key_cache"][:, h].view(torch.uint8)[ids].view(E4M3).double() * s["k_scales"][ids, h].double()[:, None, None]).reshape(-1, d)[:length]
            v = (s["value_cache"][:, h].view(torch.uint8)[ids].view(E4M3).double() * s["v_scales"][ids, h].double()[:, None, None]).reshape(-1, d)[:length]
            last = torch.arange(q_len, device=DEVICE) + length - q_len
            sees = torch.arange(length, device=DEVICE)[None, :] <= last[:, None]
            w = torch.einsum("qgd,td->qgt", q[:, h], k) * s["scale"]
            w = torch.softmax(w.masked_fill(~sees[:, None, :], -math.inf), dim=-1)
            o[:, h] = torch.einsum("qgt,td->qgd", torch.nan_to_num(w, nan=0.0), v)
        out.append(o.reshape(s["query"].shape[1:]))
    return torch.stack(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend_q8":
        return _exact_attend(s)
    eight = case["op"] == "append_q8"
    bs = case["block_size"]
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    query = s["query_out"].double()
    names = ("key_cache", "value_cache")
    caches = [s[x].double() for x in names]
    scales = [s[x].double() for x in ("k_scales", "v_scales")] if eight else None
    for b, length in enumerate(lens):
        rows = range(starts[b], starts[b + 1])
        if not rows:
            continue
        first = length - len(rows)
        pairs = s["cos_sin"][first:length].double()[:, None, :]
        half = case["rotary"] // 2
        a, z = rows[0], rows[-1] + 1
        idx = torch.arange(half, device=DEVICE) * (2 if case["interleaved"] else 1)
        jdx = idx + (1 if case["interleaved"] else half)
        turned = []
        for x in (s["query"], s["key"]):
            x = x[a:z].double()
            w = torch.complex(x[..., idx], x[..., jdx]) * torch.complex(pairs[..., :half].contiguous(), pairs[..., half:].contiguous())
            x[..., idx], x[..., jdx] = w.real, w.imag
            turned.append(x)
        query[a:z] = turned[0]
        new = (turned[1], s["value"][a:z].double())
        for j in range(first // bs, -(-length // bs)):
            block = int(s["tables"][b, j])
            lo, hi = max(first, j * bs), min(length, (j + 1) * bs)
            for i in range(2):
                x = new[i][lo - first:hi - first].transpose(0, 1)  # [kv_heads, tokens, d]
                if eight:
                    # The scale times 448 covers the largest; halved, it would not.
                    most = x.abs().amax(dim=(1, 2))
                    scale = _two_to(torch.ceil(torch.log2(most / E4M3_MAX)).clamp(min=-126.0))
                    scale = torch.where(scale * E4M3_MAX < most, scale * 2, scale)
                    scale = torch.where((scale * E4M3_MAX / 2 >= most) & (scale > MIN_SCALE), scale / 2, scale)
                    if lo > j * bs:
                        before = scales[i][block]
                        scale = torch.maximum(scale, before)
                        kept = caches[i][block, :, :lo - j * bs]
                        caches[i][block, :, :lo - j * bs] = _nearest_e4m3(kept * (before / scale)[:, None, None])
                    scales[i][block] = scale
                    x = _nearest_e4m3(x / scale[:, None, None])
                caches[i][block, :, lo - j * bs:hi - j * bs] = x
    got = {"query": query, "key_cache": caches[0], "value_cache": caches[1]}
    if eight:
        got.update(k_scales=scales[0], v_scales=scales[1])
    return got
