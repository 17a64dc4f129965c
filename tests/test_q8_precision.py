"""What pa_decode_q8 keeps of its operands: directed inputs on which a bit that is lost, or a value
that is held in fewer bits, moves the result by many times the tolerance."""
import math

import pytest
import torch

import cache_util as cu
from cache_util import E4M3
from test_decode_q8 import run

F16, BF16 = torch.float16, torch.bfloat16
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return cuda_lib


def cache_of(k, v, k_scales, v_scales, bs):
    """(key_cache, value_cache, k_scales, v_scales, tables, lens) of one sequence and one KV head, blocks in order;
    k and v [tokens, D] are values that e4m3 holds."""
    L, D = k.shape
    n = -(-L // bs)
    caches = []
    for x in (k, v):
        c = torch.zeros(n * bs, D)
        c[:L] = x
        code = c.to(E4M3)
        assert torch.equal(code.float(), c)
        caches.append(code.view(torch.uint8).view(n, 1, bs, D).contiguous().view(E4M3))
    return (*caches, torch.as_tensor(k_scales).float().view(n, 1).contiguous(),
            torch.as_tensor(v_scales).float().view(n, 1).contiguous(), torch.arange(n, dtype=torch.int32).view(1, n),
            torch.tensor([L], dtype=torch.int32))


# ---------------------------------------------------------------- scales that are no powers of two


def odd_scales(D, bs, L, dtype):
    """Keys of one code under block scales that rounding the product to `dtype` moves by all but half a step, up in even
    blocks and down in odd ones: nearly equal scores, and V of +1 and -1 shows which is larger."""
    bits = 8 if dtype == BF16 else 11
    code = 1.875
    up, down = [], []
    for m in range(2 ** 16, 2 ** 16 * 2):
        x = code * m / 2 ** 16
        step = 2.0 ** (math.floor(math.log2(x)) + 1 - bits)
        part = x / step - math.floor(x / step)
        if 0.5 < part < 0.51:
            up.append(m / 2 ** 16)
        elif 0.49 < part < 0.5:
            down.append(m / 2 ** 16)
    near = min(up, key=lambda s: abs(s - 1.2)), min(down, key=lambda s: abs(s - 1.2))
    n = -(-L // bs)
    block = torch.arange(L) // bs
    k = torch.full((L, D), code)
    v = torch.where(block % 2 == 0, 1.0, -1.0)[:, None].expand(L, D)
    return cache_of(k, v, [near[i % 2] for i in range(n)], [1.0] * n, bs)


@gpu
@pytest.mark.parametrize("Q,G", [(70, 4), (900, 4), (1300, 3)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scales_are_kept_whatever_the_rows_and_the_workspace(pa, D, dtype, Q, G):
    """From 256 rows on, with room for it, the call may work on a 16-bit copy of its blocks, where a value under such a scale
    would be rounded: a score of 100 is then off by 2^-9 or 2^-12 of it, more than any other error of the call."""
    L, bs = 4800, 16
    c = odd_scales(D, bs, L, dtype)
    q = torch.ones((1, Q, G, D), dtype=dtype)
    scale = 100.0 / (1.875 * 1.2 * D)
    ref, tol = cu.attend_reference(q[:, -2:], *c, scale)
    for P in (32, 128, 4096):  # the intermediates' size grows as P falls
        out, status = run(pa, q, c, scale, P)
        assert status == 0
        out = out[:, -2:].double()
        assert ((out - ref).abs() <= tol + cu.rounding(ref.abs() + tol, dtype)).all(), float((out - ref).abs().max())


@gpu
@pytest.mark.parametrize("up", [105, -100])
@pytest.mark.parametrize("Q", [70, 900])
@pytest.mark.parametrize("D", [64, 256])
def test_extreme_scales_are_kept_whatever_the_rows(pa, D, Q, up):
    """bf16 queries and K scales whose sums of products leave fp32's range, and a softmax scale that brings the scores back
    to a size of 4: the 8-bit kernel's sums are of codes, those over a 16-bit copy would be infinite."""
    c = list(cu.cache8([4800], KV=1, D=D, bs=16, seed=up))
    c[2] = c[2] * 2.0 ** up
    g = torch.Generator().manual_seed(9)
    few = 125 - up if up > 0 else -140 - up
    q = (torch.randn((1, Q, 4, D), generator=g) * 2.0 ** few).to(BF16)
    scale = 2.0 ** -126 if up > 0 else 2.0 ** 127
    ref, tol = cu.attend_reference(q[:, -2:], *c, scale)
    assert torch.isfinite(ref).all()
    out, status = run(pa, q, c, scale, 128)
    out = out[:, -2:].double()
    assert status == 0
    assert ((out - ref).abs() <= tol + cu.rounding(ref.abs() + tol, BF16)).all(), float((out - ref).abs().max())


# ---------------------------------------------------------------- scores of any finite size


@gpu
@pytest.mark.parametrize("lens,P,Q", [([130], 2048, 1), ([1100, 40], 2048, 1), ([6000, 300], 64, 3), ([300, 700], 2048, 70)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_very_negative_scores(pa, lens, P, Q, dtype):
    """Every score below -1e30: the softmax is all on the largest of them, as for any others."""
    D, bs = 64, 16
    n = [-(-x // bs) for x in lens]
    tables = torch.full((len(lens), max(n)), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(n):
        tables[b, :x] = torch.arange(at, at + x, dtype=torch.int32)
        at += x
    g = torch.Generator().manual_seed(2)
    k = torch.ones(at, 1, bs, D)
    v = torch.randint(-8, 9, (at, 1, bs, D), generator=g).float()
    q = torch.full((len(lens), Q, 4, D), -1.0, dtype=dtype)
    best = [5, 17]
    for b in range(len(lens)):
        k[tables[b, best[b] // bs], 0, best[b] % bs] = 0.5
    c = (k.to(E4M3), v.to(E4M3), torch.full((at, 1), 2.0 ** 104), torch.ones(at, 1), tables, torch.tensor(lens, dtype=torch.int32))
    out, status = run(pa, q, c, 0.125, P)
    assert status == 0
    for b in range(len(lens)):
        assert (out[b].float() == v[tables[b, best[b] // bs], 0, best[b] % bs]).all()


# ---------------------------------------------------------------- the parts of Q and P


def parts_of(x, count):
    """Rows of x as `count` e4m3 parts, part j standing for 16^-j of its value, of the row scaled to [2^7, 2^8)."""
    x = x.double()
    f = torch.exp2(7 - torch.floor(torch.log2(x.abs().amax(-1, keepdim=True))))
    rest, got = x * f, []
    for _ in range(count):
        p = rest.float().to(E4M3).double()
        got.append(p)
        rest = (rest - p) * 16
    return sum(p / 16.0 ** j for j, p in enumerate(got)) / f


def low_bits(D, bs, L, dtype, G, seed=3):
    """Query rows c + d, -c on pairs of dims with equal keys: the scores are sum d k, and d lies in the bits that only the
    last part of a query holds (fp16's low 3, bf16's low 4)."""
    g = torch.Generator().manual_seed(seed)
    step, high = (2.0 ** -10, 128) if dtype == F16 else (2.0 ** -7, 8)
    top = 7 if dtype == F16 else 15
    c = 1 + torch.randint(0, high - 1, (1, 1, G, D // 2), generator=g).double() / high
    d = step * torch.randint(1, top + 1, (1, 1, G, D // 2), generator=g).double()
    q = torch.stack([c + d, -c], -1).flatten(-2)
    assert torch.equal(q.to(dtype).double(), q)
    k = torch.randint(-15, 16, (L, D // 2), generator=g).double() / 8
    scores = k @ d[0, 0, 0]
    scale = 3.0 / float(scores.std())
    v = torch.randint(-15, 16, (L, D), generator=g).float() / 8
    n = -(-L // bs)
    return q.to(dtype), cache_of(k.repeat_interleave(2, 1).float(), v, [1.0] * n, [1.0] * n, bs), scale


def exact_with(q, c, scale):
    """(out, tolerance) in 64 bits for queries q (64 bits).  Parts of a query are whole multiples of 2^-3 up to 2^8, keys of
    2^-3 below 2: the sums over a row are multiples of 2^-6 below 2^17, exact in fp32.  A score (below 40 in log2 units)
    is then off by some 3 roundings of 2^-24 of it and exp2 by 2^-22: together below 2^-16.  A weight is rounded to binary16
    (2^-11 of it), and what lies below 2^-27 of the largest is lost."""
    k, v = (x.view(torch.uint8).view(E4M3).float().double().flatten(0, 2)[:int(c[5])] for x in c[:2])
    p = torch.softmax(q[0, 0] @ k.T * scale, 1)
    out = p @ v
    return out, (2.0 ** -11 + 2.0 ** -15) * (p @ v.abs()) + 2.0 ** -27 * p.amax(1, keepdim=True) * v.abs().sum(0)


@pytest.mark.parametrize("dtype,parts", [(F16, 3), (BF16, 2)])
def test_a_lost_part_of_q_is_seen(dtype, parts):
    q, c, scale = low_bits(128, 16, 1000, dtype, 4)
    ref, tol = exact_with(q.double(), c, scale)
    tol = tol + cu.rounding(ref.abs() + tol, dtype)
    assert torch.equal(parts_of(q, parts), q.double())
    lost, _ = exact_with(parts_of(q, parts - 1), c, scale)
    assert ((lost - ref).abs() > 20 * tol).double().mean() > 0.5


@gpu
@pytest.mark.parametrize("G", [1, 6, 12, 24, 64])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32), (256, 8)])
@pytest.mark.parametrize("L,P", [(100, 512), (1000, 512), (7000, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_part_of_q(pa, dtype, L, P, D, bs, G):
    q, c, scale = low_bits(D, bs, L, dtype, G)
    ref, tol = exact_with(q.double(), c, scale)
    out, status = run(pa, q, c, scale, P)
    assert status == 0
    assert ((out[0, 0].double() - ref).abs() <= tol + cu.rounding(ref.abs() + tol, dtype)).all()


def even_weights(D, bs, L, dtype):
    """Weights of 2047/2048 of the largest (eleven ones: every part of P is needed, and what is lost of it adds up), in all
    blocks but the first of every 128 tokens, whose weight is 1.  V is one value, just above the middle between two values of the
    output's type: the exact result is that value, and one that is smaller by 2^-11 rounds down."""
    n = -(-L // bs)
    x = -math.log(2047 / 2048)
    k = torch.zeros(L, D)
    k[:, 0] = -1.0
    k[(torch.arange(L) % 128) < bs] = 0.0
    middle = 1 + cu.HALF_STEP[dtype]
    value = float(torch.tensor(middle * (1 + 2.0 ** -12)).float())
    return cache_of(k, torch.ones(L, D), [x] * n, [value] * n, bs), value


def rounded_up(dtype):
    return 1 + 2 * cu.HALF_STEP[dtype]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bs", [8, 64])
def test_a_lost_part_of_p_is_seen(dtype, bs):
    c, value = even_weights(64, bs, 1280, dtype)
    w = torch.where((torch.arange(1280) % 128) < bs, 2048.0, 2047.0).double()
    lost = torch.where(w == 2047, 2044.0, w)  # without the fourth part: 3 + 3 + 3 bits
    assert float((torch.tensor(value).double() * lost.sum() / w.sum()).to(dtype)) < rounded_up(dtype)
    assert float(torch.tensor(value).to(dtype)) == rounded_up(dtype)


@gpu
@pytest.mark.parametrize("G", [1, 6, 12, 24, 64])
@pytest.mark.parametrize("D,bs", [(64, 64), (128, 32), (256, 8)])
@pytest.mark.parametrize("L,P", [(100, 512), (1000, 512), (7000, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_part_of_p(pa, dtype, L, P, D, bs, G):
    """(exp2, the sums and the quotient are off by less than 2^-19: no weight's rounding moves, and the result rounds up.)"""
    c, value = even_weights(D, bs, L, dtype)
    q = torch.zeros((1, 1, G, D), dtype=dtype)
    q[..., 0] = 1.0
    out, status = run(pa, q, c, 1.0, P)
    assert status == 0 and (out.float() == rounded_up(dtype)).all()


# ---------------------------------------------------------------- small weights beside a large one


def sink(D, bs, L, exponent):
    """One token of weight 1 whose V is 0, and L - 1 of weight 2047 * 2^exponent (eleven ones) whose V is 1: the result is
    what the small ones add up to."""
    n = -(-L // bs)
    w = 2047 * 2.0 ** exponent
    k = torch.zeros(L, D)
    k[1:, 0] = -1.0
    v = torch.ones(L, D)
    v[0] = 0.0
    return cache_of(k, v, [-math.log(w)] * n, [1.0] * n, bs), (L - 1) * w / (1 + (L - 1) * w)


def sink_tolerance(ref, L, dtype):
    """A weight, in units of 2^-11, is rounded to binary16: by 2^-11 of it, or 2^-25 where that is more; exp2 and the sums
    add less than 2^-18."""
    tol = ref * (2.0 ** -11 + 2.0 ** -18) + L * 2.0 ** -36
    return tol + float(cu.rounding(torch.tensor(ref + tol, dtype=torch.float64), dtype))


@pytest.mark.parametrize("exponent", [-31, -34])
def test_truncated_small_weights_are_seen(exponent):
    """Parts that end at 2^-16 of those units (e5m2's smallest step, without a factor between them)."""
    ref = sink(64, 16, 8000, exponent)[1]
    w = 2047 * 2.0 ** (exponent + 11)
    kept = math.floor(w * 2 ** 16) / 2 ** 16
    assert ref * (1 - kept / w) > sink_tolerance(ref, 8000, F16)


@gpu
@pytest.mark.parametrize("exponent", [-31, -34, -37])
@pytest.mark.parametrize("G", [4, 16, 30, 60])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32), (256, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_small_weights_beside_a_large_one(pa, dtype, D, bs, G, exponent):
    """All tokens of a sequence in one CTA."""
    S, L = 200, 8000
    c, ref = sink(D, bs, L, exponent)
    c = c[:4] + (c[4].expand(S, -1).contiguous(), c[5].expand(S).contiguous())
    q = torch.zeros((S, 1, G, D), dtype=dtype)
    q[..., 0] = 1.0
    out, status = run(pa, q, c, 1.0, 8192)
    tol = sink_tolerance(ref, L, dtype)
    assert status == 0
    assert ((out.double() - ref).abs() <= tol).all(), (float((out.double() - ref).abs().max()), ref, tol)
