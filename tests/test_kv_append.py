"""pa_kv_append and pa_kv_append_q8 against a plain 64-bit reference, and their refusals."""
import pytest
import torch

import cache_util as cu
from cache_util import E4M3

F16, BF16 = torch.float16, torch.bfloat16
FAKE = 0x10000  # never dereferenced: the calls are refused on the host

# ---------------------------------------------------------------- refusals (no GPU)


def _call(lib, q8=False, **kw):
    a = dict(key=FAKE, value=FAKE, ks=1024, vs=1024, query=FAKE, query_out=FAKE, qs=1024, qos=1024,
             cos_sin=FAKE, rotary=128, positions=100, interleaved=0, tables=FAKE, lens=FAKE, starts=FAKE,
             tokens=4, seqs=2, heads=8, kv=2, d=128, blocks=16, bs=16, mb=4, dtype=0, kc=FAKE, vc=FAKE,
             ksc=FAKE, vsc=FAKE, status=None)
    a.update(kw)
    args = [a[k] for k in ("key", "value", "ks", "vs", "query", "query_out", "qs", "qos", "cos_sin", "rotary",
                           "positions", "interleaved", "tables", "lens", "starts", "tokens", "seqs", "heads", "kv",
                           "d", "blocks", "bs", "mb", "dtype", "kc", "vc")]
    if q8:
        return lib.pa_kv_append_q8(*args, a["ksc"], a["vsc"], a["status"], None)
    return lib.pa_kv_append(*args, a["status"], None)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(key=None), 1), (dict(value=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(tables=None), 1),
    (dict(lens=None), 1), (dict(query=None), 1), (dict(query_out=None), 1), (dict(key=FAKE + 8), 1),
    (dict(value=FAKE + 2), 1), (dict(query=FAKE + 4), 1), (dict(kc=FAKE + 8), 1), (dict(ks=1028), 1),
    (dict(vs=248), 1), (dict(qs=1000), 1), (dict(qos=0), 1), (dict(seqs=0), 1), (dict(tokens=-1), 1),
    (dict(starts=None, tokens=3), 1), (dict(starts=FAKE + 2), 1), (dict(heads=7), 1), (dict(heads=0), 1),
    (dict(kv=0), 1), (dict(dtype=2), 1), (dict(rotary=0), 1), (dict(positions=0), 1), (dict(cos_sin=FAKE + 4), 1),
    (dict(rotary=24), 2), (dict(rotary=144), 2), (dict(d=96), 2), (dict(bs=4), 2), (dict(bs=128), 2),
    (dict(blocks=2 ** 30, kv=2, bs=16), 2), (dict(mb=2 ** 28), 2), (dict(seqs=65536), 2), (dict(status=FAKE + 1), 1),
])
def test_refused_before_launch(cuda_lib, q8, kw, code):
    assert _call(cuda_lib.load(), q8, **kw) == code


@pytest.mark.parametrize("kw", [dict(ksc=None), dict(vsc=None), dict(ksc=FAKE + 2)])
def test_scales_refused(cuda_lib, kw):
    assert _call(cuda_lib.load(), True, **kw) == 1


@pytest.mark.parametrize("q8", [False, True])
def test_no_tokens_is_no_launch(cuda_lib, q8):
    assert _call(cuda_lib.load(), q8, tokens=0) == 0
    assert _call(cuda_lib.load(), q8, tokens=0, key=None, value=None, starts=None) == 0


def test_binding_refuses(cuda_lib):
    t = cu.batch([2, 1], [3, 0])
    args = (t.key, t.value, t.tables, t.lens, t.key_cache, t.value_cache)
    with pytest.raises(ValueError):  # CPU tensors
        cuda_lib.pa_kv_append_q8(*args, t.k_scales, t.v_scales, token_starts=t.starts)
    with pytest.raises(ValueError):
        cuda_lib.pa_kv_append_q8(*args, None, t.v_scales, token_starts=t.starts)
    with pytest.raises(TypeError):
        cuda_lib.pa_kv_append(t.key.float(), *args[1:], token_starts=t.starts)


# ---------------------------------------------------------------- on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return cuda_lib


def _run(pa, t, q8, with_query=True, rotated=True, starts=True, **kw):
    """The call on copies of the batch's caches; returns (query_out, caches..., status)."""
    d = t.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.full(t.query.shape, 7.0, dtype=t.query.dtype, device="cuda") if with_query else None
    opt = dict(cos_sin=d.cos_sin if rotated else None, interleaved=t.interleaved,
               query=d.query if with_query else None, query_out=qo, token_starts=d.starts if starts else None,
               status=status, **kw)
    if q8:
        pa.pa_kv_append_q8(d.key, d.value, d.tables, d.lens, d.key_cache, d.value_cache, d.k_scales, d.v_scales, **opt)
    else:
        pa.pa_kv_append(d.key, d.value, d.tables, d.lens, d.key_cache, d.value_cache, **opt)
    torch.cuda.synchronize()
    return (qo.cpu() if with_query else None, d.key_cache.cpu(), d.value_cache.cpu(), d.k_scales.cpu(),
            d.v_scales.cpu(), int(status.item()))


def _near(got, ref, size, dtype):
    """Rounded once from fp32 products and a sum of them (three roundings of at most 2^-24)."""
    tol = cu.rounding(ref, dtype) + 3 * 2.0 ** -24 * size
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), float(((got.double() - ref).abs() - tol).max())


def check(pa, t, q8, with_query=True, rotated=True, starts=True):
    qo, kc, vc, ks, vs, status = _run(pa, t, q8, with_query, rotated, starts)
    assert status == 0
    dtype = t.key.dtype
    want_q = torch.full(t.query.shape, 7.0, dtype=dtype)
    want = [t.key_cache.clone(), t.value_cache.clone()]
    if not q8:
        for row, b, pos, block, at, k, ksize, v, q, qsize in cu.append_reference(t, rotated):
            _near(kc[block, :, at], k, ksize, dtype)
            assert torch.equal(vc[block, :, at], t.value[row])
            want[0][block, :, at] = kc[block, :, at]
            want[1][block, :, at] = t.value[row]
    else:
        check_q8(t, kc, vc, ks, vs, rotated)
    if with_query:
        for row, b, pos, block, at, k, ksize, v, q, qsize in cu.append_reference(t, rotated):
            _near(qo[row], q, qsize, dtype)
            want_q[row] = qo[row]
        assert torch.equal(qo, want_q)  # padding rows untouched
    if not q8:
        assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])  # and every other cache row


def check_q8(t, kc, vc, ks, vs, rotated=True):
    groups = {}
    for row, b, pos, block, at, k, ksize, v, q, qsize in cu.append_reference(t, rotated):
        groups.setdefault(block, []).append((at, k, ksize, v))
    for got, old, got_s, old_s, which in ((kc, t.key_cache, ks, t.k_scales, 1), (vc, t.value_cache, vs, t.v_scales, 3)):
        want, want_s = old.clone(), old_s.clone()
        for block, rows in groups.items():
            kept = min(r[0] for r in rows)
            for h in range(kc.shape[1]):
                x = torch.stack([r[which][h] for r in rows])
                size = torch.stack([r[2][h] for r in rows]) if which == 1 else torch.zeros_like(x)
                s = cu.scale_of(float(x.abs().max()))
                if kept:
                    s = max(s, float(old_s[block, h]))
                    # fp32 quotient and product, then one rounding to e4m3.
                    again = (old[block, h, :kept].float() * (old_s[block, h] / torch.tensor(s))).to(E4M3)
                    want.view(torch.uint8)[block, h, :kept] = again.view(torch.uint8)
                want_s[block, h] = s
                at = torch.tensor([r[0] for r in rows])
                code = got.float()[block, h, at].double()
                tol = cu.rounding(x / s, E4M3) + 3 * 2.0 ** -24 * size / s
                assert ((code - x / s).abs() <= tol).all()
                want.view(torch.uint8)[block, h, at] = got.view(torch.uint8)[block, h, at]
        assert torch.equal(got_s, want_s)
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


SHAPES = [
    dict(new=[1], past=[0]),
    dict(new=[1, 1, 1, 1], past=[0, 15, 16, 40]),
    dict(new=[17, 0, 3, 33, 0], past=[5, 9, 0, 31, 0], padding=4),
    dict(new=[5, 40], past=[11, 2], D=128, H=8, KV=2, bs=8),
    dict(new=[70, 1], past=[100, 63], D=256, H=6, KV=3, bs=64),
    dict(new=[64, 129, 7], past=[0, 3, 60], D=128, H=5, KV=1, bs=32, rotary=32),
    dict(new=[9, 2], past=[0, 7], D=64, H=4, KV=4, bs=8, rotary=16),
    dict(new=[3] * 70, past=list(range(70)), D=64, H=2, KV=1, bs=16),
]


@gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_ragged(pa, shape, dtype, interleaved, q8):
    check(pa, cu.batch(dtype=dtype, interleaved=interleaved, q8=q8, seed=len(shape["new"]), **shape), q8)


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_equal_counts_without_starts(pa, q8):
    check(pa, cu.batch([6] * 5, [0, 9, 10, 11, 30], D=128, q8=q8), q8, starts=False)
    check(pa, cu.batch([1] * 33, list(range(33)), q8=q8), q8, starts=False)


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_no_rotation_and_no_query(pa, q8):
    t = cu.batch([6, 20], [0, 9], D=128, q8=q8)
    check(pa, t, q8, rotated=False)
    check(pa, t, q8, with_query=False)


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_q8_magnitudes(pa, dtype):
    """Tokens whose sizes differ by 2^16: scales grow inside a block and old rows fall to subnormals."""
    for seed in range(4):
        check(pa, cu.batch([1, 9, 30, 2], [6, 3, 0, 14], dtype=dtype, seed=seed, spread=8), True)


@gpu
def test_q8_zeros_and_borders(pa):
    """All-zero tokens take the smallest scale; 448 s itself still fits s, the next value does not."""
    t = cu.batch([4, 4, 4], [0, 0, 3], D=64, KV=1, H=1, dtype=BF16)
    t.key[:4], t.value[:4] = 0.0, 0.0
    t.value[4:8] = 1.75
    t.value[8:12] = 1.7578125  # one bf16 step above 448 * 2^-8
    check(pa, t, True, rotated=False)


@gpu
def test_q8_non_finite(pa):
    t = cu.batch([8], [0], D=64, KV=1, H=1, dtype=BF16)
    t.value[2, 0, 5], t.value[3, 0, 6], t.value[4, 0, 7] = float("inf"), float("-inf"), float("nan")
    _, kc, vc, ks, vs, status = _run(pa, t, True)
    block = int(t.tables[0, 0])
    got = vc[block, 0, :8].float() * vs[block, 0]
    bad = ~torch.isfinite(t.value[:, 0].float())
    assert torch.equal(torch.isnan(got), bad)
    assert float(vs[block, 0]) == cu.scale_of(float(t.value[:, 0].float()[~bad].abs().max()))


@gpu
def test_query_in_place(pa):
    t = cu.batch([5, 3], [0, 4], D=128, q8=False)
    want = _run(pa, t, False)[0]
    d = t.cuda()
    pa.pa_kv_append(d.key, d.value, d.tables, d.lens, d.key_cache, d.value_cache, cos_sin=d.cos_sin,
                    query=d.query, query_out=d.query, token_starts=d.starts)
    torch.cuda.synchronize()
    assert torch.equal(d.query.cpu(), want)
    assert torch.equal(d.key.cpu(), t.key) and torch.equal(d.value.cpu(), t.value)


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_four_dimensional_rows(pa, q8):
    t = cu.batch([4] * 3, [1, 2, 3], q8=q8)
    a = _run(pa, t, q8, starts=False)
    d = t.cuda()
    shape = lambda x: x.unflatten(0, (3, 4))  # noqa: E731
    qo = torch.zeros_like(shape(d.query))
    if q8:
        pa.pa_kv_append_q8(shape(d.key), shape(d.value), d.tables, d.lens, d.key_cache, d.value_cache, d.k_scales,
                           d.v_scales, cos_sin=d.cos_sin, query=shape(d.query), query_out=qo)
    else:
        pa.pa_kv_append(shape(d.key), shape(d.value), d.tables, d.lens, d.key_cache, d.value_cache, cos_sin=d.cos_sin,
                        query=shape(d.query), query_out=qo)
    torch.cuda.synchronize()
    assert torch.equal(qo.flatten(0, 1).cpu(), a[0])
    assert torch.equal(d.key_cache.view(torch.uint8).cpu(), a[1].view(torch.uint8))


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_status(pa, q8):
    """Device-side problems set their bit, write nothing of the token, and leave the others' rows right."""
    base = cu.batch([3, 2], [4, 6], bs=8, q8=q8)
    good = _run(pa, base, q8)

    def rows_of(got, b, n):
        return [got[1].view(torch.uint8)[int(base.tables[b, p // 8]), :, p % 8] for p in range(n)]

    t = cu.batch([3, 2], [4, 6], bs=8, q8=q8)
    t.tables[1, 0] = 999  # block id out of range: sequence 1's tokens are not written
    got = _run(pa, t, q8)
    assert got[5] == pa.PA_STATUS_BAD_BLOCK_ID
    assert all(torch.equal(x, y) for x, y in zip(rows_of(got, 0, 7), rows_of(good, 0, 7)))
    at = int(base.tables[1, 0])
    assert torch.equal(got[1].view(torch.uint8)[at], base.key_cache.view(torch.uint8)[at])

    t = cu.batch([3, 2], [4, 6], bs=8, q8=q8)
    t.lens[1] = 1  # two new tokens, one of them at position -1
    got = _run(pa, t, q8)
    assert got[5] == pa.PA_STATUS_BAD_SEQ_LEN
    assert (got[0][3] == 7).all() and not (got[0][4] == 7).all()

    t = cu.batch([3, 2], [4, 6], bs=8, q8=q8)
    t.lens[1] = 10  # positions 8 and 9, past the one-block table
    t.tables = t.tables[:, :1].contiguous()
    got = _run(pa, t, q8)
    assert got[5] == pa.PA_STATUS_BAD_SEQ_LEN
    assert (got[0][3:5] == 7).all()

    t = cu.batch([3, 2], [4, 6], bs=8, q8=q8)
    t.cos_sin = t.cos_sin[:7].contiguous()  # sequence 1's position 7 has no angles
    got = _run(pa, t, q8)
    assert got[5] == pa.PA_STATUS_BAD_POSITION
    assert not (got[0][3] == 7).all() and (got[0][4] == 7).all()

    t = cu.batch([3, 2], [4, 6], bs=8, q8=q8)
    t.starts[2] = 9  # beyond the rows there are
    got = _run(pa, t, q8)
    assert got[5] == pa.PA_STATUS_BAD_SEQ_LEN
    assert torch.equal(got[0][:3], good[0][:3])


@gpu
def test_q8_token_by_token_equals_one_call(pa):
    """Scales only ever grow by powers of two: the same scales as one call over all tokens, and codes
    that differ only where a value fell among the subnormals of a later, larger scale."""
    t = cu.batch([40], [0], D=64, bs=16, dtype=F16, spread=2, seed=5)
    whole = _run(pa, t, True)
    d = t.cuda()
    for n in range(1, 41):
        pa.pa_kv_append_q8(d.key[n - 1:n], d.value[n - 1:n], d.tables,
                           torch.tensor([n], dtype=torch.int32, device="cuda"), d.key_cache, d.value_cache,
                           d.k_scales, d.v_scales, cos_sin=d.cos_sin)
    torch.cuda.synchronize()
    assert torch.equal(d.k_scales.cpu(), whole[3]) and torch.equal(d.v_scales.cpu(), whole[4])
    for a, b in ((d.key_cache.cpu(), whole[1]), (d.value_cache.cpu(), whole[2])):
        a, b = a.float(), b.float()
        # Two roundings instead of one, each at most half a subnormal step of 2^-9.
        assert ((a - b).abs() <= torch.where(b.abs() < 2.0 ** -6, 2.0 ** -9, 0.0)).all()


@gpu
def test_graph_replay_and_stream(pa):
    t = cu.batch([1, 1, 1], [3, 15, 16], D=128)
    want = _run(pa, t, True)
    d = t.cuda()
    qo = torch.zeros_like(d.query)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fresh = [x.clone() for x in (d.key_cache, d.value_cache, d.k_scales, d.v_scales)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pa.pa_kv_append_q8(d.key, d.value, d.tables, d.lens, d.key_cache, d.value_cache, d.k_scales, d.v_scales,
                           cos_sin=d.cos_sin, query=d.query, query_out=qo, token_starts=d.starts)
    for _ in range(2):
        for x, y in zip((d.key_cache, d.value_cache, d.k_scales, d.v_scales), fresh):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo.cpu(), want[0]) and torch.equal(d.k_scales.cpu(), want[3])
        assert torch.equal(d.key_cache.view(torch.uint8).cpu(), want[1].view(torch.uint8))
    other = t.cuda()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_kv_append_q8(other.key, other.value, other.tables, other.lens, other.key_cache, other.value_cache,
                       other.k_scales, other.v_scales, cos_sin=other.cos_sin, token_starts=other.starts, stream=side)
    side.synchronize()
    assert torch.equal(other.key_cache.view(torch.uint8).cpu(), want[1].view(torch.uint8))


@gpu
@pytest.mark.parametrize("q8", [False, True])
def test_binding_refuses_shapes(pa, q8):
    d = cu.batch([2, 1], [3, 0]).cuda()
    out = torch.empty_like(d.query)
    good = dict(key=d.key, value=d.value, block_tables=d.tables, seq_lens=d.lens, key_cache=d.key_cache, value_cache=d.value_cache,
                cos_sin=d.cos_sin, query=d.query, query_out=out, token_starts=d.starts)
    wrong = [("key", d.key[:2]), ("key", d.key[..., :32]), ("key", d.key[:, :1]), ("key", d.key.transpose(1, 2)), ("value", d.value.float()),
             ("value", d.value[0]), ("query", None), ("query_out", None), ("query", d.query[:1]), ("query_out", out[:, :1]),
             ("token_starts", d.starts[:2]), ("token_starts", d.starts.long()), ("token_starts", None), ("cos_sin", d.cos_sin.double()),
             ("cos_sin", d.cos_sin[0]), ("cos_sin", d.cos_sin.t()), ("seq_lens", d.lens.cpu()), ("key_cache", d.key_cache.double()),
             ("status", d.lens.long())]
    if q8:
        good.update(k_scales=d.k_scales, v_scales=d.v_scales)
        wrong += [("k_scales", d.k_scales[:1]), ("v_scales", d.v_scales.double()), ("k_scales", None)]
    before = d.key_cache.clone()
    for name, value in wrong:
        with pytest.raises((TypeError, ValueError)):
            (pa.pa_kv_append_q8 if q8 else pa.pa_kv_append)(**dict(good, **{name: value}))
    torch.cuda.synchronize()
    assert torch.equal(d.key_cache.view(torch.uint8), before.view(torch.uint8))


@gpu
@pytest.mark.parametrize("S,new,shape", [
    (50, 520, dict(D=64, bs=8, KV=2, H=2, dtype=BF16, interleaved=True)),     # two heads a CTA, queries apart
    (300, 9, dict(D=256, bs=64, KV=8, H=8, dtype=F16)),                       # the same in the widest CTAs
    (30, 900, dict(D=128, bs=16, KV=5, H=10, dtype=BF16, rotary=64)),         # heads that two do not divide
    (700, 3, dict(D=128, bs=32, KV=12, H=12, dtype=BF16)),
])
def test_q8_large_batches_equal_their_sequences(pa, S, new, shape):
    """A batch large enough for CTAs of several heads and a launch of its own for the queries: bit for bit what one call
    per sequence writes."""
    counts = [(new * (b % 3) + b) % (2 * new) for b in range(S)]
    past = [(7 * b) % 61 for b in range(S)]
    t = cu.batch(counts, past, seed=S, padding=3, **shape)
    whole = _run(pa, t, True)
    d = t.cuda()
    query = torch.full(t.query.shape, 7.0, dtype=t.query.dtype, device="cuda")
    for b in range(S):
        a, e = int(t.starts[b]), int(t.starts[b + 1])
        if a < e:
            pa.pa_kv_append_q8(d.key[a:e], d.value[a:e], d.tables[b:b + 1], d.lens[b:b + 1], d.key_cache, d.value_cache,
                               d.k_scales, d.v_scales, cos_sin=d.cos_sin, interleaved=t.interleaved, query=d.query[a:e],
                               query_out=query[a:e])
    torch.cuda.synchronize()
    assert whole[5] == 0
    assert torch.equal(whole[0].view(torch.int16), query.cpu().view(torch.int16))
    for got, ref in zip(whole[1:3], (d.key_cache, d.value_cache)):
        assert torch.equal(got.view(torch.uint8), ref.cpu().view(torch.uint8))
    assert torch.equal(whole[3], d.k_scales.cpu()) and torch.equal(whole[4], d.v_scales.cpu())
