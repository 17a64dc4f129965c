"""pa_kv_append and pa_kv_append_q8: what a promise of the language, a tie or an empty argument decides."""
import os
import re

import pytest
import torch

import cache_util as cu

F16, BF16 = torch.float16, torch.bfloat16
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return cuda_lib


def nearest_e4m3(x):
    """The nearest e4m3 value, ties to even, of 64-bit x up to 448 in magnitude."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def ties(scale, dtype, count):
    """Values x of `dtype` with x / scale halfway between two e4m3 values."""
    got = []
    for e in range(-6, 8):
        for m in range(17, 32, 2):
            x = scale * m / 16 * 2.0 ** e
            if m / 16 * 2.0 ** e < 448 and float(torch.tensor(x).to(dtype)) == x:
                got += [x, -x]
    return torch.tensor([got[i % len(got)] for i in range(count)], dtype=torch.float64)


@gpu
@pytest.mark.parametrize("dtype,scale", [(F16, 1.625), (F16, 1.75), (F16, 1.875), (F16, 0.875), (F16, 1.15625), (BF16, 1.625),
                                         (BF16, 1.75), (BF16, 1.875), (BF16, 0.875)])
def test_codes_under_a_scale_that_is_no_power_of_two(pa, dtype, scale):
    """Blocks that another writer began keep its scale where that is the larger (for all values but fp16's at 1.875,
    the largest of which, 465, takes 2): new codes are e4m3(x / s), ties to even."""
    D, KV, bs = 64, 2, 16
    t = cu.batch([7], [3], H=2, KV=KV, D=D, bs=bs, dtype=dtype)
    t.k_scales[:], t.v_scales[:] = scale, scale
    x = ties(scale, dtype, 7 * KV * D).view(7, KV, D).to(dtype)
    t.key[:], t.value[:] = x, x
    d = t.cuda()
    pa.pa_kv_append_q8(d.key, d.value, d.tables, d.lens, d.key_cache, d.value_cache, d.k_scales, d.v_scales)
    torch.cuda.synchronize()
    block = int(t.tables[0, 0])
    s = max(scale, cu.scale_of(float(x.abs().max())))
    want = nearest_e4m3(x.double() / s)
    for cache, scales in ((d.key_cache, d.k_scales), (d.value_cache, d.v_scales)):
        assert (scales[block] == s).all()
        got = cache[block].float().cpu().double()[:, 3:10].transpose(0, 1)
        assert torch.equal(got, want), int((got != want).sum())


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_a_table_of_no_positions_is_refused(pa, q8):
    """(an empty tensor has no address, and a call without a table does not rotate)"""
    d = cu.batch([2, 1], [3, 0], q8=q8).cuda()
    args = (d.key, d.value, d.tables, d.lens, d.key_cache, d.value_cache) + ((d.k_scales, d.v_scales) if q8 else ())
    before = d.key_cache.clone()
    for empty in (d.cos_sin[:0], d.cos_sin[:, :0].contiguous()):
        with pytest.raises(ValueError):
            (pa.pa_kv_append_q8 if q8 else pa.pa_kv_append)(*args, cos_sin=empty, token_starts=d.starts)
    torch.cuda.synchronize()
    assert torch.equal(d.key_cache.view(torch.uint8), before.view(torch.uint8))


def test_what_the_append_writes_is_not_loaded_as_constant(cuda_lib):
    """__ldg promises that its array stays as it is during the launch: none that the appends write is loaded so."""
    csrc = os.path.join(os.path.dirname(cuda_lib.LIB_PATH), "csrc")
    with open(os.path.join(csrc, "pa_append.cu")) as f:
        text = f.read()
    for name in ("k_scales", "v_scales", "key_cache", "value_cache", "query_out"):
        assert not re.search(r"__ldg\([^;]*\b%s\b" % name, text), name
