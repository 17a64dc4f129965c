"""Plain 64-bit references of the cache operators (on the CPU, sharing no code with the library),
and the inputs their tests draw."""
from __future__ import annotations

import dataclasses
import math

import torch

E4M3 = torch.float8_e4m3fn
MAX = 448.0
# Half a step of rounding to nearest, relative to the value.
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, E4M3: 2.0 ** -4}
# Half the spacing of the smallest values.
HALF_TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, E4M3: 2.0 ** -10}


def scale_of(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while amax > MAX * s:
        s *= 2.0
    return s


@dataclasses.dataclass
class Batch:
    """New tokens of a ragged batch, the cache before them, and where they go (CPU tensors)."""
    key: torch.Tensor
    value: torch.Tensor
    query: torch.Tensor
    starts: torch.Tensor
    lens: torch.Tensor
    tables: torch.Tensor
    key_cache: torch.Tensor
    value_cache: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor
    cos_sin: torch.Tensor
    interleaved: bool

    def cuda(self) -> "Batch":
        return Batch(*[v.cuda() if isinstance(v, torch.Tensor) else v
                       for v in (getattr(self, f.name) for f in dataclasses.fields(self))])


def codes(shape, gen):
    """Random finite e4m3 codes (all signs and exponents)."""
    c = torch.randint(0, 256, shape, generator=gen, dtype=torch.int32)
    return torch.where((c & 127) == 127, c - 1, c).to(torch.uint8).view(E4M3)


def batch(new, past, H=4, KV=2, D=64, bs=16, dtype=torch.bfloat16, rotary=None, interleaved=False,
          padding=0, q8=True, seed=0, spread=0, extra_positions=0):
    """new[b] new tokens after past[b] earlier ones; values N(0, 1), times 2^U{-spread..spread}
    per token."""
    g = torch.Generator().manual_seed(seed)
    S, lens = len(new), [a + b for a, b in zip(new, past)]
    used = [-(-x // bs) for x in lens]
    width = max(max(used), 1)
    pool = sum(used) + 3
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    tables = torch.full((S, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        tables[b, :n] = perm[at:at + n]
        at += n
    T = sum(new) + padding
    qkv = torch.randn((T, H + 2 * KV, D), generator=g)
    if spread:
        qkv *= torch.exp2(torch.randint(-spread, spread + 1, (T, 1, 1), generator=g).float())
    qkv = qkv.to(dtype)
    starts = torch.zeros(S + 1, dtype=torch.int32)
    starts[1:] = torch.cumsum(torch.tensor(new), 0)
    shape = (pool, KV, bs, D)
    if q8:
        kc, vc = codes(shape, g), codes(shape, g)
        ks = torch.exp2(torch.randint(-10, -5, (pool, KV), generator=g).float())
        vs = torch.exp2(torch.randint(-10, -5, (pool, KV), generator=g).float())
    else:
        kc, vc = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
        ks = vs = torch.zeros(0)
    r = D if rotary is None else rotary
    half = max(r // 2, 1)
    angle = torch.arange(max(lens) + 1 + extra_positions, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    return Batch(qkv[:, H:H + KV], qkv[:, H + KV:], qkv[:, :H], starts,
                 torch.tensor(lens, dtype=torch.int32), tables, kc, vc, ks, vs, cos_sin, interleaved)


def rotate(x, pair, interleaved):
    """(rotated x, |a| + |b| of each value's pair); x [heads, D] float64, pair = [cos, sin]."""
    half = pair.numel() // 2
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = pair[:half].double(), pair[half:].double()
    out, size = x.clone(), torch.zeros_like(x)
    out[:, a] = x[:, a] * c - x[:, b] * s
    out[:, b] = x[:, b] * c + x[:, a] * s
    size[:, a] = size[:, b] = x[:, a].abs() + x[:, b].abs()
    return out, size


def append_reference(t: Batch, rotated=True):
    """Per new token row: (row, sequence, position, block, slot, k, size of k's pairs, v, q, size of q's)."""
    bs = t.key_cache.shape[2]
    for b in range(t.lens.numel()):
        first, last = int(t.starts[b]), int(t.starts[b + 1])
        for row in range(first, last):
            pos = int(t.lens[b]) - last + row
            block = int(t.tables[b, pos // bs])
            k, q = t.key[row].double(), t.query[row].double()
            ksize, qsize = torch.zeros_like(k), torch.zeros_like(q)
            if rotated:
                k, ksize = rotate(k, t.cos_sin[pos], t.interleaved)
                q, qsize = rotate(q, t.cos_sin[pos], t.interleaved)
            yield row, b, pos, block, pos % bs, k, ksize, t.value[row].double(), q, qsize


def attend_reference(q, kc, vc, ks, vs, tables, lens, scale, held=0.0):
    """(out, tolerance but for the output's own rounding) in 64 bits.  q [S, Q, H, D].

    The tolerance: P is rounded to binary16 (2^-11 of each term, doubled for fp32 sums and exp2),
    a score is off by at most D 2^-23 sum |q k| scale (fp32 accumulation) and P by that factor, and
    P below binary16's normals by at most 2^-25.
    """
    S, Q, H, D = q.shape
    KV, bs = kc.shape[1], kc.shape[2]
    G = H // KV
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    for b in range(S):
        L = int(lens[b])
        ids = tables[b, :-(-L // bs)].long()
        for h in range(KV if L > 0 else 0):
            def rows(c, s):
                x = c.view(torch.uint8)[ids, h].view(E4M3).double() * s[ids, h].double()[:, None, None]
                return x.reshape(-1, D)[:L]
            k, v = rows(kc, ks), rows(vc, vs)
            for i in range(Q):
                n = L - Q + i + 1
                if n <= 0:
                    continue
                qq = q[b, i, h * G:(h + 1) * G].double()
                w = qq @ k[:n].T * scale
                p = torch.softmax(w, dim=1)
                out[b, i, h * G:(h + 1) * G] = p @ v[:n]
                off = abs(scale) * (D * 2.0 ** -23 * (qq.abs() @ k[:n].abs().T).amax(1, keepdim=True) +
                                    held * (qq.abs() @ k[:n].abs().T).amax(1, keepdim=True) +
                                    2.0 ** -17 * qq.abs().amax(1, keepdim=True) * k[:n].abs().sum(1).max())
                tol[b, i, h * G:(h + 1) * G] = (2.0 ** -11 + held + 4 * off) * (p @ v[:n].abs()) + \
                    2.0 ** -25 * v[:n].abs().sum(0) + 448 * 2.0 ** -60 * float(vs[ids, h].max())
    return out, tol


def rounding(ref, dtype):
    return HALF_STEP[dtype] * ref.abs() + HALF_TINY[dtype]


def cache8(lens, KV=2, D=64, bs=16, seed=0, scales="blocks", poison=False):
    """An 8-bit cache of N(0, 1) values with block scales, its tables and lengths (CPU).

    scales: "blocks" powers of two that fit each block; "any" those times U(1, 2); "wild" blocks
    whose values differ by factors up to 2^40; "zero" some blocks with scale 0.
    poison: NaN codes in rows past the lengths and in blocks no sequence uses.
    """
    g = torch.Generator().manual_seed(seed)
    used = [-(-x // bs) for x in lens]
    pool = sum(used) + 5
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    tables = torch.full((len(lens), max(max(used), 1) + 2), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        tables[b, :n] = perm[at:at + n]
        at += n
    got = []
    for which in range(2):
        x = torch.randn((pool, KV, bs, D), generator=g)
        if scales == "wild" and which == 1:
            x *= torch.exp2(torch.randint(-20, 21, (pool, KV, 1, 1), generator=g).float())
        s = torch.tensor([scale_of(float(v)) for v in x.abs().amax(dim=(2, 3)).flatten()]).view(pool, KV)
        if scales == "any":
            s = s * (1 + torch.rand((pool, KV), generator=g))
        c = (x / s[:, :, None, None]).to(E4M3)
        if scales == "zero":
            s = torch.where(torch.rand((pool, KV), generator=g) < 0.3, torch.zeros_like(s), s)
        if poison:
            raw = c.view(torch.uint8)
            alive = torch.zeros(pool, bs, dtype=torch.bool)
            for b, L in enumerate(lens):
                for j in range(used[b]):
                    alive[tables[b, j], :max(0, min(bs, L - j * bs))] = True
            raw.masked_fill_(~alive[:, None, :, None], 0x7f)
            s = torch.where(alive.any(1)[:, None], s, torch.full_like(s, math.nan))
        got += [c, s]
    kc, ks, vc, vs = got
    return kc, vc, ks, vs, tables, torch.tensor(lens, dtype=torch.int32)
