"""The queries for a call's variant and partition size refuse, on the host, the sizes that the calls refuse."""
import pytest


@pytest.mark.parametrize("name", ["pa_decode_q8_partition", "pa_decode_mq_partition", "pa_decode_mq_choose"])
@pytest.mark.parametrize("seqs,q_len,heads,kv", [
    (1, 2 ** 29, 64, 8),                      # q_len * G is 2^32: nothing, in 32 bits
    (1, 4097, 32, 8), (17, 4096, 32, 8),      # new tokens a sequence, and in all
    (1, 1, 130, 2),                           # query heads of a KV head
    (65536, 1, 8, 2), (1, 1, 65536, 65536),
    (2 ** 31 - 1, 1, 2 ** 31 - 1, 2 ** 31 - 1),
])
def test_sizes_that_the_calls_refuse(cuda_lib, name, seqs, q_len, heads, kv):
    assert getattr(cuda_lib.load(), name)(seqs, q_len, heads, kv, 128, 100000, 512) == -cuda_lib.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["pa_decode_q8_partition", "pa_decode_mq_partition", "pa_decode_mq_choose"])
@pytest.mark.parametrize("head_dim", [1, 96, 192, 512])
def test_head_dims_that_the_calls_refuse(cuda_lib, name, head_dim):
    assert getattr(cuda_lib.load(), name)(1, 1, 8, 2, head_dim, 100000, 512) == -cuda_lib.PA_ERR_UNSUPPORTED
