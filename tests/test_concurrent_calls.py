"""Calls of several host threads on streams of their own: bit for bit what each alone returns."""
import threading

import pytest
import torch

import cache_util as cu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return cuda_lib


def worker(pa, which, stream):
    """A function that appends, attends and returns clones of everything written; its tensors are its own."""
    dtype = [torch.float16, torch.bfloat16][which % 2]
    # A cluster's CTAs, partitions with a merge, many rows (the copy under powers of two, and what follows where one is none).
    lens, Q, G, P, odd = [([900, 40], 1, 4, 2048, False), ([9000, 8100, 20], 2, 4, 64, False), ([1800, 700], 300, 4, 64, False),
                          ([1800, 700], 300, 4, 64, True)][which]
    c = [x.cuda() for x in cu.cache8(lens, KV=2, D=128, bs=16, seed=which, scales="any" if odd else "blocks")]
    q = torch.randn((len(lens), Q, 2 * G, 128), generator=torch.Generator().manual_seed(which)).to(dtype).cuda()
    q = q if Q > 1 else q[:, 0].contiguous()
    work = pa.alloc_workspace(len(lens), 2 * G, 128, pa.num_partitions(c[4].shape[1] * 16, P), q_len=Q)
    out = torch.empty_like(q)
    t = cu.batch([40, 3], [7, 0], D=128, H=8, KV=2, dtype=dtype, seed=which).cuda()
    rotated = torch.empty_like(t.query.contiguous())
    first = [x.clone() for x in (t.key_cache, t.value_cache, t.k_scales, t.v_scales)]
    state = [t.key_cache, t.value_cache, t.k_scales, t.v_scales, rotated, out]

    def call(n=1):
        got = []
        with torch.cuda.stream(stream):
            for _ in range(n):
                for x, y in zip(state, first):
                    x.view(torch.uint8).copy_(y.view(torch.uint8))
                pa.pa_kv_append_q8(t.key, t.value, t.tables, t.lens, *state[:4], cos_sin=t.cos_sin, query=t.query, query_out=rotated,
                                   token_starts=t.starts)
                pa.pa_decode_q8(q, *c, 0.088, P, out, *work)
                got.append([x.view(torch.uint8).clone() for x in state])
        return got

    return call


def test_threads_and_streams(pa):
    streams = [torch.cuda.Stream() for _ in range(4)]
    calls = [worker(pa, i, s) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    alone = []
    for call in calls:
        alone.append(call()[0])
        torch.cuda.synchronize()
    together, errors = [None] * 4, []

    def run(i):
        try:
            together[i] = calls[i](15)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(4):
        for n, got in enumerate(together[i]):
            assert [j for j in range(6) if not torch.equal(got[j], alone[i][j])] == [], (i, n)
