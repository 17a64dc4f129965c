"""A batch of empty sequences between others, on one stream: the merge of phase 2 ends behind phase 1 even where it has
nothing to merge, so what follows may change the lengths and the intermediates."""
import pytest
import torch

import cache_util as cu

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1, 2])
def pa(cuda_lib, request):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    cuda_lib.pa_set_merge_form(request.param)
    yield cuda_lib
    cuda_lib.pa_set_merge_form(0)


@pytest.mark.parametrize("q8", [False, True])
def test_empty_batches_between_others(pa, q8):
    lens = [9000, 300, 8200, 64]
    kc, vc, ks, vs, tables, real = [x.cuda() for x in cu.cache8(lens, KV=2, D=64, bs=16)]
    if not q8:
        kc, vc = kc.view(torch.uint8).half(), vc.view(torch.uint8).half() / 256
    q = (torch.randn((4, 8, 64), generator=torch.Generator().manual_seed(1)) / 100).half().cuda()
    P = 64
    work = pa.alloc_workspace(4, 8, 64, pa.num_partitions(tables.shape[1] * 16, P))
    seq_lens, out = real.clone(), torch.empty_like(q)

    def call():
        if q8:
            pa.pa_decode_q8(q, kc, vc, ks, vs, tables, seq_lens, 0.125, P, out, *work)
        else:
            pa.pa_decode_v2(q, kc, vc, tables, seq_lens, 0.125, P, out, *work)
        return out.clone()

    want, got = call(), []
    for _ in range(20):
        seq_lens.zero_()
        got.append((call(), torch.zeros_like(want)))
        seq_lens.copy_(real)
        got.append((call(), want))
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and (want != 0).any()
    assert all(torch.equal(a, b) for a, b in got)
