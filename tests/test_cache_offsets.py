"""Filling and reading caches whose offsets pass 32 bits: bit for bit what the same calls do in a small cache."""
import pytest
import torch

import cache_util as cu
from cache_util import E4M3

pytestmark = pytest.mark.gpu

KV, D, BS, H = 2, 256, 64, 8


@pytest.fixture(scope="module")
def pa(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    return cuda_lib


def fill_and_attend(pa, t, q8, blocks, ids, dtype, far=False):
    """(rotated query, attention of each sequence's last token, the cache blocks `ids`) of a cache of `blocks` blocks."""
    d = t.cuda()
    tables = torch.tensor(ids, dtype=torch.int32, device="cuda").view(2, 2)
    shape = (blocks, KV, BS, D)
    kc, vc = (torch.empty(shape, dtype=torch.uint8, device="cuda").view(E4M3) if q8 else torch.empty(shape, dtype=dtype, device="cuda")
              for _ in range(2))
    key = d.key
    if far:  # tokens 2^29 elements apart: the last ones beyond 2^31 elements
        room = torch.empty((t.key.shape[0] - 1) * 2 ** 29 + KV * D, dtype=dtype, device="cuda")
        key = room.as_strided(t.key.shape, (2 ** 29, D, 1))
        key.copy_(d.key)
    rotated = torch.empty_like(d.query.contiguous())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    opt = dict(cos_sin=d.cos_sin, query=d.query, query_out=rotated, token_starts=d.starts, status=status)
    last = [int(x) - 1 for x in t.starts[1:]]
    out = torch.empty((2, H, D), dtype=dtype, device="cuda")
    work = pa.alloc_workspace(2, H, D, 4)
    if q8:
        ks, vs = (torch.zeros((blocks, KV), device="cuda") for _ in range(2))  # (some blocks stay unused)
        pa.pa_kv_append_q8(key, d.value, tables, d.lens, kc, vc, ks, vs, **opt)
        pa.pa_decode_q8(rotated[last], kc, vc, ks, vs, tables, d.lens, D ** -0.5, 64, out, *work, status=status)
        scales = [ks[ids], vs[ids]]
    else:
        pa.pa_kv_append(key, d.value, tables, d.lens, kc, vc, **opt)
        pa.pa_decode(rotated[last], kc, vc, tables, d.lens, D ** -0.5, 64, out, *work, status=status)
        scales = []
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    rows = []
    for b, n in enumerate(t.lens.tolist()):
        for p in range(n):
            rows += [c[ids[2 * b + p // BS], :, p % BS].clone() for c in (kc, vc)]
    return [rotated, out] + rows + scales


def differing(a, b):
    """Which of the tensors differ."""
    return [i for i, (x, y) in enumerate(zip(a, b, strict=True)) if not torch.equal(x.view(torch.uint8), y.view(torch.uint8))]


@pytest.mark.parametrize("q8,dtype", [(True, torch.bfloat16), (False, torch.float16)])
def test_blocks_beyond_32_bits(pa, q8, dtype):
    t = cu.batch([70, 66], [0, 0], H=H, KV=KV, D=D, bs=BS, dtype=dtype, q8=q8)
    near = fill_and_attend(pa, t, q8, 4, [3, 1, 0, 2], dtype)
    blocks = 140000  # of 2^15 values: the last ones begin beyond 2^32
    assert (blocks - 2) * KV * BS * D > 2 ** 32
    assert differing(fill_and_attend(pa, t, q8, blocks, [blocks - 1, 5, blocks - 2, 70000], dtype), near) == []


@pytest.mark.parametrize("q8", [True, False])
def test_tokens_beyond_32_bits(pa, q8):
    t = cu.batch([4, 2], [0, 0], H=H, KV=KV, D=D, bs=BS, dtype=torch.bfloat16, q8=q8)
    t.tables = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    near = fill_and_attend(pa, t, q8, 4, [3, 1, 0, 2], torch.bfloat16)
    assert differing(fill_and_attend(pa, t, q8, 4, [3, 1, 0, 2], torch.bfloat16, far=True), near) == []
