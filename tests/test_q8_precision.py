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
