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


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("Q,G,D", [(1, 1, 64), (1, 4, 128), (5, 8, 64), (3, 16, 256), (16, 2, 128), (20, 4, 64), (40, 8, 256)])
@pytest.mark.parametrize("held", [math.nan, math.inf, -math.inf])
def test_decay_zero_reads_nothing(pa, held, Q, G, D, bits):  # noqa: F811
    """decay 0 keeps the call's own sums alone, whatever the slots hold."""
    lens = [0, 1, 7, 64, 65, 1300]
    q, kc, ks, tables, n, w = inputs(lens, Q, G, 2, D, 16, F16, bits, Q)
    ref, tol = q4.weigh_reference(q, kc, ks, tables, n, 0.1, torch.zeros_like(w), 0.0)
    got, status = run(pa, q, kc, ks, tables, n, torch.full_like(w, held), 0.1, 0.0)
    assert status == 0
    for b, L in enumerate(lens):
        x, r, t = (slots(y, tables, b, L) for y in (got.double(), ref, tol))
        assert ((x - r).abs() <= t).all(), (L, x, r)
    # With any other decay what they hold counts.
    got, status = run(pa, q, kc, ks, tables, n, torch.full_like(w, held), 0.1, 0.5)
    assert status == 0 and not torch.isfinite(slots(got, tables, 5, 1300 - Q)).any()


def test_a_prompt_longer_than_its_window(pa):  # noqa: F811
    """Into weights that nobody has initialised: a prompt whose last 20 tokens are counted with decay 0, then single
    tokens added up, are the sums from the definition."""
    L, Q, steps, D, bs, KV, G = 200, 20, 6, 64, 16, 2, 3
    q, kc, ks, tables, _, w = inputs([L + steps], Q + steps, G, KV, D, bs, F16, 4, 2)
    kc, ks, tables = kc.cuda(), ks.cuda(), tables.cuda()
    dev = torch.full(w.shape, math.nan, device="cuda")
    ws = pa.alloc_weights_workspace(1, G * KV, tables.shape[1] * bs, q_len=Q)
    calls = [(q[:, :Q], L, 0.0)] + [(q[:, Q + i], L + i + 1, 1.0) for i in range(steps)]
    ref, off = torch.zeros(w.shape, dtype=torch.float64), torch.zeros(w.shape, dtype=torch.float64)
    for x, length, decay in calls:
        n = torch.tensor([length], dtype=torch.int32)
        pa.pa_kv_weights(x.contiguous().cuda(), kc, tables, n.cuda(), 0.125, dev, ws, k_scales=ks, decay=decay)
        got, t = q4.weigh_reference(x if x.dim() == 4 else x[:, None], kc.cpu(), ks.cpu(), tables.cpu(), n, 0.125,
                                    torch.zeros(w.shape), 0.0)
        ref, off = ref + got, off + t
    x, r, t = (slots(y, tables.cpu(), 0, L + steps) for y in (dev.cpu().double(), ref, off))
    assert ((x - r).abs() <= t + steps * 2.0 ** -23 * r).all()


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("Q,G", [(2, 4), (5, 1), (7, 8), (15, 3), (16, 3), (20, 4)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_tokens_hidden_from_a_row_that_is_not_finite(pa, bad, Q, G, bits):  # noqa: F811
    """A row whose scores are not finite makes NaN of the weights of the tokens that it sees, not of later ones."""
    L = 50
    q, kc, ks, tables, n, w = inputs([L, 33], Q, G, 2, 64, 16, F16, bits, Q)
    at = Q // 2 - 1
    q[0, at, G, 9] = bad  # new token `at`, KV head 1: sees L - Q + at + 1 tokens
    got, status = run(pa, q, kc, ks, tables, n, w, 0.1, 1.0)
    of = slots(got, tables, 0, L)
    sees = L - Q + at + 1
    assert status == 0 and torch.isnan(of[1, :sees]).all() and torch.isfinite(of[1, sees:]).all()
    assert torch.isfinite(of[0]).all() and torch.isfinite(slots(got, tables, 1, 33)).all()


@pytest.mark.parametrize("Q,G", [(1, 4), (6, 8), (20, 4)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_score_of_minus_infinity_counts_as_nothing(pa, dtype, Q, G):  # noqa: F811
    """16-bit keys with an infinite value, every score of which is -inf: softmax weight 0, the others' sums as ever."""
    L = 100
    q, kc, ks, tables, n, w = inputs([L, 20], Q, G, 2, 64, 16, dtype, 16, 4)
    q[..., 3] = -q[..., 3].abs() - 1
    for t in (0, 17, 70):
        kc[tables[0, t // 16], :, t % 16, 3] = math.inf
    got, status = run(pa, q, kc, ks, tables, n, w, 0.1, 1.0)
    far, gone = (torch.where(torch.isinf(kc), torch.full_like(kc, x), kc) for x in (2.0 ** 14, 0.0))
    ref, _ = q4.weigh_reference(q, far, ks, tables, n, 0.1, w, 1.0)   # weight e^-1638 and less: 0 in 64 bits too
    _, tol = q4.weigh_reference(q, gone, ks, tables, n, 0.1, w, 1.0)  # (a far key's size is no error of the others')
    x, r, t = (slots(y, tables, 0, L) for y in (got.double(), ref, tol))
    assert status == 0 and ((x - r).abs() <= t).all()


@pytest.mark.parametrize("bits", [4, 16])
def test_steps_without_a_call(pa, bits):  # noqa: F811
    """A call at every third step, for the newest query alone; tokens of the steps between start from slots that
    are cleared as they are appended, whatever those held."""
    D, bs, KV, G, first, steps = 64, 16, 2, 3, (40, 7), 12
    S, H = 2, 6
    lens = [x + steps for x in first]
    q, kc, ks, tables, _, w = inputs(lens, steps, G, KV, D, bs, F16, bits, 7)
    dev = torch.full(w.shape, math.nan, device="cuda")
    c, t, scales = kc.cuda(), tables.cuda(), ks.cuda() if ks is not None else None
    ws = pa.alloc_weights_workspace(S, H, tables.shape[1] * bs)
    ref = off = torch.zeros(w.shape, dtype=torch.float64)
    for step in range(steps):
        n = torch.tensor([x + step + 1 for x in first], dtype=torch.int32)
        p = (n.cuda() - 1).long()
        dev[t[torch.arange(S, device="cuda"), p // bs].long(), :, p % bs] = 0
        if step % 3:
            continue
        pa.pa_kv_weights(q[:, step].contiguous().cuda(), c, t, n.cuda(), 0.125, dev, ws, k_scales=scales,
                         decay=0.0 if step == 0 else 1.0)
        got, tol = q4.weigh_reference(q[:, step:step + 1], kc, ks, tables, n, 0.125, torch.zeros(w.shape), 0.0)
        ref, off = ref + got, off + tol
    for b in range(S):
        x, r, tol = (slots(y, tables, b, lens[b]) for y in (dev.cpu().double(), ref, off))
        assert ((x - r).abs() <= tol + steps * 2.0 ** -23 * r).all()
