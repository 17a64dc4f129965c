"""What slots of attention weights hold beside the call's own sums: another sequence's tokens in a shared block,
contents that must not count, tokens that a row with a score that is not finite does not see."""
import math

import pytest
import torch

import q4_util as q4
from q4_util import BF16, F16
from test_kv_weights import inputs, pa, run  # noqa: F401 (pa: the fixture)

pytestmark = pytest.mark.gpu


def slots(x, tables, b, L):
    """[KV, L]: sequence b's slots of x."""
    bs = x.shape[2]
    return x[tables[b, :-(-L // bs)].long()].transpose(0, 1).reshape(x.shape[1], -1)[:, :L]


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("Q,G", [(1, 1), (1, 4), (2, 8), (3, 16), (5, 8), (16, 2), (20, 1)])
@pytest.mark.parametrize("short,long", [(5, 8), (7, 8), (21, 24), (33, 47), (45, 64)])
def test_a_longer_sequence_in_a_shared_block(pa, short, long, Q, G, bits):  # noqa: F811
    """Pairs whose tables are the same blocks: what the longer one alone has there is its own, every time."""
    n, D, bs, KV = 100, 64, 16, 2
    q, kc, ks, tables, lens, w = inputs([long] * n, Q, G, KV, D, bs, BF16, bits, short)
    both = torch.stack([tables, tables], 1).flatten(0, 1)
    # The shorter ones before and behind the longer ones, in turn.
    lens2 = torch.tensor([x for i in range(n) for x in ((short, long) if i % 2 else (long, short))], dtype=torch.int32)
    own = [2 * i + (1 if i % 2 else 0) for i in range(n)]
    q2 = torch.randn((2 * n,) + q.shape[1:], generator=torch.Generator().manual_seed(1)).to(q.dtype)
    q2[own] = q
    ref, tol = q4.weigh_reference(q, kc, ks, tables, lens, 0.125, w, 1.0)
    for _ in range(10):
        got, status = run(pa, q2, kc, ks, both, lens2, w, 0.125, 1.0)
        assert status == 0
        for i in range(n):
            x, r, t = (slots(y, tables, i, long)[:, short:] for y in (got.double(), ref, tol))
            assert ((x - r).abs() <= t).all(), (i, x, r)
        rest = torch.ones(w.shape, dtype=torch.bool)
        for i in range(n):
            for at in range(long):
                rest[tables[i, at // bs], :, at % bs] = False
        assert torch.equal(got[rest], w[rest])
