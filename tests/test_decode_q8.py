"""pa_decode_q8 against a plain 64-bit reference, its refusals, and the append + attention path."""
import math

import pytest
import torch

import cache_util as cu
from cache_util import E4M3

F16, BF16 = torch.float16, torch.bfloat16
FAKE = 0x10000  # never dereferenced: the calls are refused on the host

# ---------------------------------------------------------------- refusals (no GPU)


def _call(lib, **kw):
    a = dict(query=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, tables=FAKE, lens=FAKE, seqs=1, q_len=1, heads=8, kv=2,
             d=128, blocks=128, bs=16, mb=63, hint=0, scale=0.088, part=512, dtype=0, out=FAKE, tmp=FAKE, es=FAKE,
             ml=FAKE, np=2, status=None)
    a.update(kw)
    return lib.pa_decode_q8(*[a[k] for k in ("query", "kc", "vc", "ks", "vs", "tables", "lens", "seqs", "q_len", "heads",
                                             "kv", "d", "blocks", "bs", "mb", "hint", "scale", "part", "dtype", "out",
                                             "tmp", "es", "ml", "np", "status")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(query=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
    (dict(tables=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(seqs=0), 1), (dict(q_len=0), 1),
    (dict(heads=0), 1), (dict(heads=7), 1), (dict(kv=0), 1), (dict(blocks=0), 1), (dict(part=0), 1),
    (dict(dtype=2), 1), (dict(scale=math.inf), 1), (dict(kc=FAKE + 8), 1), (dict(query=FAKE + 2), 1),
    (dict(out=FAKE + 1), 1), (dict(ks=FAKE + 2), 1), (dict(status=FAKE + 2), 1), (dict(lens=FAKE + 2), 1),
    (dict(d=96), 2), (dict(bs=48), 2), (dict(heads=130, kv=2), 2), (dict(q_len=4097), 2), (dict(seqs=30, q_len=4000), 2),
    (dict(seqs=65536), 2), (dict(blocks=2 ** 30), 2), (dict(mb=2 ** 28), 2),
])
def test_refused_before_launch(cuda_lib, kw, code):
    assert _call(cuda_lib.load(), **kw) == code


def test_partition_arguments(cuda_lib):
    for bad in ((0, 1, 8, 2, 128, 1000, 512), (1, 0, 8, 2, 128, 1000, 512), (1, 1, 7, 2, 128, 1000, 512),
                (1, 1, 8, 2, 0, 1000, 512), (1, 1, 8, 2, 128, -1, 512), (1, 1, 8, 2, 128, 1000, 0)):
        assert cuda_lib.load().pa_decode_q8_partition(*bad) == -1


def test_binding_refuses(cuda_lib):
    kc, vc, ks, vs, tables, lens = cu.cache8([40, 3])
    q = torch.zeros((2, 4, 64), dtype=F16)
    with pytest.raises(ValueError):  # CPU tensors
        cuda_lib.pa_decode_q8(q, kc, vc, ks, vs, tables, lens, 0.125, 64, torch.empty_like(q), None, None, None)
    with pytest.raises(TypeError):
        cuda_lib.pa_decode_q8(q.float(), kc, vc, ks, vs, tables, lens, 0.125, 64, q.float(), None, None, None)


def test_binding_refuses_what_is_no_tensor(cuda_lib):
    kc, vc, ks, vs, tables, lens = cu.cache8([40, 3])
    q = torch.zeros((2, 4, 64), dtype=F16)
    for args in ((None, kc, vc, ks, vs, tables, lens, 0.125, 64, q), (q, kc, vc, None, vs, tables, lens, 0.125, 64, q),
                 (q, kc, vc, ks, vs, tables, [40, 3], 0.125, 64, q), (q, kc, vc, ks, vs, tables, lens, "x", 64, q),
                 (q, kc, vc, ks, vs, tables, lens, 0.125, 6.5, q)):
        with pytest.raises(TypeError):
            cuda_lib.pa_decode_q8(*args, None, None, None)
    with pytest.raises(ValueError):
        cuda_lib.pa_decode_q8(q, kc, vc, ks, vs, tables, lens, 0.125, 2 ** 40, q, None, None, None)


# ---------------------------------------------------------------- on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return cuda_lib


def run(pa, q, cache, scale, P, hint=0):
    kc, vc, ks, vs, tables, lens = [x.cuda() for x in cache]
    S, Q, H, D = q.shape
    cap = tables.shape[1] * kc.shape[2]
    cap = min(cap, hint) if hint > 0 else cap
    work = pa.alloc_workspace(S, H, D, max(1, pa.num_partitions(cap, P)), q_len=Q)
    for t in work:
        t.fill_(math.nan)
    qq = q.cuda() if Q > 1 else q[:, 0].contiguous().cuda()
    out = torch.full_like(qq, math.nan)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_decode_q8(qq, kc, vc, ks, vs, tables, lens, scale, P, out, *work, max_seq_len_hint=hint, status=status)
    torch.cuda.synchronize()
    return out.view(S, Q, H, D).cpu(), int(status.item())


def check(pa, lens, Q=1, G=4, KV=2, D=64, bs=16, P=64, dtype=BF16, scale=None, seed=0, q=None, hint=0, held=0.0, **cache):
    c = cu.cache8(lens, KV=KV, D=D, bs=bs, seed=seed, **cache)
    g = torch.Generator().manual_seed(seed + 1)
    if q is None:
        q = torch.randn((len(lens), Q, G * KV, D), generator=g).to(dtype)
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, status = run(pa, q, c, scale, P, hint)
    ref, tol = cu.attend_reference(q, c[0], c[1], *[torch.nan_to_num(x) for x in c[2:4]], *c[4:], scale, held)
    assert status == 0
    tol = tol + cu.rounding(ref.abs() + tol, dtype)
    # binary16's largest value is 65504 and its next step would be 65536: results from the middle,
    # 65520, on round to infinity (bfloat16 reaches as far as fp32).
    over = torch.tensor(dtype == F16) & (out.double() == ref.sign() * math.inf) & (ref.abs() + tol >= 65520)
    bad = ~(((out.double() - ref).abs() <= tol) | over)
    assert not bad.any(), (int(bad.sum()), float(((out.double() - ref).abs() / tol).max()))


LENS = [0, 1, 7, 16, 17, 63, 64, 65, 300]


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_shapes(pa, D, bs, dtype):
    check(pa, LENS, D=D, bs=bs, dtype=dtype)                        # several partitions, tails inside blocks
    check(pa, LENS, D=D, bs=bs, dtype=dtype, P=100, G=12, KV=1)     # two n-tiles, partitions across blocks
    check(pa, [40, 0, 33], D=D, bs=bs, dtype=dtype, P=512, G=1)     # one partition


@gpu
@pytest.mark.parametrize("G,Q,D,bs,dtype", [(4, 1, 128, 16, BF16), (16, 1, 64, 8, F16), (1, 6, 256, 64, BF16),
                                            (8, 12, 128, 32, F16), (64, 1, 128, 16, BF16)])
@pytest.mark.parametrize("P", [64, 200, 333])
def test_long_sequences_in_partitions(pa, G, Q, D, bs, dtype, P):
    """V2: partitions of one tile, ends inside blocks and inside tiles, partitions that hold nothing."""
    lens = [6000, 0, 3, 2500]
    assert pa.pa_decode_q8_partition(4, Q, G, 1, D, 6000 // bs * bs, P) > 0
    check(pa, lens, Q=Q, G=G, KV=1, D=D, bs=bs, dtype=dtype, P=P, scales="any")


@gpu
@pytest.mark.parametrize("G,Q,D,bs", [(4, 1, 64, 64), (5, 3, 128, 8), (2, 16, 256, 16), (32, 2, 128, 32)])
@pytest.mark.parametrize("longest", [128, 129, 400, 1000, 1300])
def test_sequences_shared_by_a_cluster(pa, G, Q, D, bs, longest):
    """V1 with 1 to 8 CTAs per sequence and KV head, some without a token."""
    check(pa, [longest, 130, 0, 1], Q=Q, G=G, KV=1, D=D, bs=bs, P=2048, scales="any")
    check(pa, [longest], Q=Q, G=G, KV=2, D=D, bs=bs, P=2048, dtype=F16)


@gpu
@pytest.mark.parametrize("G,Q", [(1, 1), (3, 1), (7, 1), (8, 1), (16, 1), (5, 1), (64, 1), (1, 2), (4, 2), (4, 4), (3, 7),
                                 (8, 5), (1, 33), (4, 16), (2, 64), (5, 27), (8, 40)])
@pytest.mark.parametrize("D,bs", [(64, 8), (128, 16), (128, 32), (256, 64)])
def test_rows(pa, G, Q, D, bs):
    """Every row count: n-tiles, row groups, causal limits inside tiles, new tokens that see no key (lengths below Q)."""
    check(pa, [0, 1, 20, 130, 263], Q=Q, G=G, D=D, bs=bs)
    check(pa, [70, 31], Q=Q, G=G, D=D, bs=bs, P=512, dtype=F16)


@gpu
@pytest.mark.parametrize("Q,G", [(1, 4), (5, 2), (12, 8)])
@pytest.mark.parametrize("bs", [8, 16, 64])
@pytest.mark.parametrize("scales", ["any", "wild", "zero"])
def test_scales(pa, scales, bs, Q, G):
    check(pa, [200, 65, 3], Q=Q, G=G, bs=bs, D=128, scales=scales)
    check(pa, [200, 65, 3], Q=Q, G=G, bs=bs, D=128, scales=scales, P=512, dtype=F16)


@gpu
@pytest.mark.parametrize("Q,G", [(1, 4), (9, 1), (12, 8)])
@pytest.mark.parametrize("D,bs", [(64, 8), (64, 16), (128, 64), (256, 32)])
def test_poisoned_slots_are_not_read(pa, D, bs, Q, G):
    check(pa, [20, 1, 77, 129], Q=Q, G=G, D=D, bs=bs, poison=True)
    check(pa, [20, 1, 77, 129], Q=Q, G=G, D=D, bs=bs, poison=True, P=512)


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,bs,KV", [(64, 16, 2), (128, 16, 2), (128, 64, 1), (256, 32, 1), (64, 8, 3)])
def test_many_rows(pa, D, bs, KV, dtype):
    """Hundreds of rows per KV head, where the call may work on a 16-bit copy: short and long
    sequences, stale NaN rows, scales that are no powers of two, and values no copy can hold."""
    many = dict(Q=90, G=4, D=D, bs=bs, KV=KV, dtype=dtype, P=128)
    check(pa, [1100, 90, 300, 0, 33], poison=True, **many)
    check(pa, [200, 131], poison=True, **many)
    check(pa, [1100, 95], scales="any", held=cu.HALF_STEP[dtype], **many)
    check(pa, [1100, 95], scales="wild", **many)
    check(pa, [1100, 95], scales="zero", **many)


@gpu
@pytest.mark.parametrize("D,bs,dtype", [(64, 16, F16), (64, 8, BF16), (128, 32, BF16), (128, 16, F16), (256, 64, F16)])
def test_many_rows_that_no_copy_can_hold(pa, D, bs, dtype):
    """More units of the 8-bit kernel than the GPU has SMs, after the copy's attention."""
    check(pa, [320, 0, 301, 40], Q=300, G=4, KV=3, D=D, bs=bs, dtype=dtype, P=128, scales="wild")
    check(pa, [1300, 0, 301, 40], Q=300, G=4, KV=3, D=D, bs=bs, dtype=dtype, P=128, scales="wild")


@gpu
@pytest.mark.parametrize("D,bs,dtype", [(64, 16, F16), (64, 8, BF16), (128, 32, BF16), (128, 16, F16), (256, 64, BF16)])
@pytest.mark.parametrize("scales", ["blocks", "any", "zero"])
def test_many_rows_of_long_sequences(pa, D, bs, dtype, scales):
    """Enough of them for the 16-bit copy: stale NaN rows, scales that are no powers of two, a sequence below q_len."""
    held = cu.HALF_STEP[dtype] if scales == "any" else 0.0
    check(pa, [1800, 33, 0, 290, 700], Q=300, G=4, KV=2, D=D, bs=bs, dtype=dtype, P=128, scales=scales, held=held,
          poison=scales == "blocks")


@gpu
@pytest.mark.parametrize("Q", [1, 12])
@pytest.mark.parametrize("scale", [0.0, -0.2, 2.0])
def test_softmax_scales(pa, scale, Q):
    check(pa, [90, 200], Q=Q, D=128, scale=scale)


@gpu
@pytest.mark.parametrize("Q,G", [(1, 4), (12, 4)])
@pytest.mark.parametrize("exponent", [-120, -30, 30, 110])
def test_query_magnitudes(pa, exponent, Q, G):
    """bf16 queries far from binary16's range, with the softmax scale that brings the scores back."""
    g = torch.Generator().manual_seed(3)
    q = (torch.randn((2, Q, 2 * G, 64), generator=g) * 2.0 ** exponent).to(BF16)
    check(pa, [90, 33], Q=Q, G=G, q=q, scale=2.0 ** -exponent / 8)


@gpu
def test_hint_and_long_cache(pa):
    check(pa, [1000, 999, 5], D=128, P=128, hint=1000)
    check(pa, [5000], D=128, P=512, KV=1, G=8)
    check(pa, [5000], D=128, P=512, KV=1, G=8, Q=9, dtype=F16)


@gpu
@pytest.mark.parametrize("what", ["k code", "v code", "k scale", "v scale", "v scale < 0", "v scale inf"])
@pytest.mark.parametrize("lens,P,Q", [([130], 2048, 1), ([300, 90], 64, 2), ([1100, 40], 2048, 1), ([6000, 90], 64, 3),
                                      ([500] * 160, 512, 1), ([120, 700], 2048, 70), ([3600, 400], 64, 300)])
def test_nan_is_not_lost(pa, lens, P, Q, what):
    """V1 on one CTA and on a cluster, V2, sorted units, the 16-bit copy: NaN reaches what sees it, and nothing else."""
    kc, vc, ks, vs, tables, lens = c = cu.cache8(lens, KV=2, D=64, bs=16)
    block = int(tables[0, 2]) # tokens 32 to 47
    target = {"k code": kc, "v code": vc, "k scale": ks}.get(what, vs)
    if "code" in what:
        target.view(torch.uint8)[block, 1, 3, 5] = 0x7f
    else:
        target[block, 1] = {"v scale < 0": -1.0, "v scale inf": math.inf}.get(what, math.nan)
    q = torch.randn((len(lens), Q, 8, 64)).to(BF16)
    out, status = run(pa, q, c, 0.125, P)
    assert status == 0
    bad = torch.isnan(out)
    seen = torch.tensor([int(lens[0]) - Q + i >= 47 for i in range(Q)])
    if what == "v code":  # the one dim; and of new tokens that do not see it as well (0 * NaN)
        assert bad[0, seen][:, 4:, 5].all()
        bad[0, :, 4:, 5] = False
    else:
        assert bad[0, seen][:, 4:].all()
        bad[0, :, 4:] &= ~torch.tensor([int(lens[0]) - Q + i >= 32 for i in range(Q)])[:, None, None]
    assert not bad.any()


@gpu
@pytest.mark.parametrize("lens,P,Q", [([130], 2048, 1), ([1100, 40], 2048, 1), ([6000, 90], 64, 3), ([120, 700], 2048, 70), ([3600, 400], 64, 300)])
def test_scales_of_zero(pa, lens, P, Q):
    """K scales of 0 make the softmax uniform, V scales of 0 the output exactly 0."""
    q = torch.randn((len(lens), Q, 8, 64)).to(BF16)
    c = list(cu.cache8(lens, KV=2, D=64, bs=16))
    c[2] = torch.zeros_like(c[2])
    out, status = run(pa, q, c, 0.125, P)
    ref, tol = cu.attend_reference(q, *c, 0.125)
    assert status == 0 and ((out.double() - ref).abs() <= tol + cu.rounding(ref.abs() + tol, BF16)).all()
    c[3] = torch.zeros_like(c[3])
    out, status = run(pa, q, c, 0.125, P)
    assert status == 0 and (out == 0).all()


@gpu
@pytest.mark.parametrize("dtype,G,Q", [(BF16, 2, 1), (F16, 12, 1), (BF16, 2, 30)])
@pytest.mark.parametrize("S", [150, 256, 257])
def test_many_sequences(pa, S, dtype, G, Q):
    """More units than the GPU holds: sorted by size up to 256 sequences; V1 (short ones) and V2."""
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(0, 70, (S,), generator=g)
    lens[::17] = 0
    lens[5:140:45] = torch.tensor([300, 128, 511])
    check(pa, lens.tolist(), KV=2, G=G, Q=Q, D=64, bs=16, P=512, dtype=dtype)
    lens[7:140:45] = torch.tensor([9000, 8192, 4100])  # (partitions: where a sequence has more than 8192 tokens)
    assert pa.pa_decode_q8_partition(S, Q, 2 * G, 2, 64, 9040, 64) > 0
    check(pa, lens.tolist(), KV=2, G=G, Q=Q, D=64, bs=16, P=64, dtype=dtype)


@gpu
def test_status_of_many_sequences(pa):
    c = list(cu.cache8([33] * 200, bs=16))
    c[4].clamp_(min=0)
    q = torch.randn((200, 1, 8, 64)).to(F16)
    clean, status = run(pa, q, c, 0.125, 512)
    assert status == 0
    for bad in (-1, 10 ** 6):
        c[5][150] = bad
        out, status = run(pa, q, c, 0.125, 512)
        assert status == pa.PA_STATUS_BAD_SEQ_LEN
        rest = [b for b in range(200) if b != 150]
        assert torch.equal(out[rest], clean[rest]) and (bad > 0 or (out[150] == 0).all())


@gpu
@pytest.mark.parametrize("Q", [1, 20])
def test_status(pa, Q):
    c = list(cu.cache8([40, 100], bs=16))
    q = torch.randn((2, Q, 4, 64)).to(F16)
    c[4][1, 2] = 10 ** 6
    out, status = run(pa, q, c, 0.125, 32)
    assert status == pa.PA_STATUS_BAD_BLOCK_ID and torch.isfinite(out).all()
    c = list(cu.cache8([40, 100], bs=16))
    c[5][0] = 10 ** 6
    c[4].clamp_(min=0)
    assert run(pa, q, c, 0.125, 32)[1] == pa.PA_STATUS_BAD_SEQ_LEN
    c[5][0] = -3
    out, status = run(pa, q, c, 0.125, 32)
    assert status == pa.PA_STATUS_BAD_SEQ_LEN and (out[0] == 0).all()


@gpu
@pytest.mark.parametrize("Q,G", [(1, 4), (3, 4), (40, 4)])
def test_same_bits_every_time_and_under_a_graph(pa, Q, G):
    c = [x.cuda() for x in cu.cache8([700, 30, 1500], D=128)]
    q = torch.randn((3, Q, 2 * G, 128), device="cuda").to(BF16)
    q = q if Q > 1 else q[:, 0].contiguous()
    work = pa.alloc_workspace(3, 2 * G, 128, pa.num_partitions(c[4].shape[1] * 16, 256), q_len=Q)
    outs = [torch.empty_like(q) for _ in range(3)]
    call = lambda o: pa.pa_decode_q8(q, *c[:6], 0.088, 256, o, *work)  # noqa: E731
    call(outs[0])
    call(outs[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[2])
    outs[2].fill_(math.nan)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@gpu
def test_binding_refuses_shapes(pa):
    kc, vc, ks, vs, tables, lens = [x.cuda() for x in cu.cache8([40, 3])]
    q = torch.zeros((2, 8, 64), dtype=F16, device="cuda")
    out = torch.empty_like(q)
    work = pa.alloc_workspace(2, 8, 64, 2)
    good = dict(query=q, key_cache=kc, value_cache=vc, k_scales=ks, v_scales=vs, block_tables=tables, seq_lens=lens,
                scale=0.125, partition_size=64, out=out, tmp_output=work[0], exp_sums=work[1], max_logits=work[2])
    pa.pa_decode_q8(**good)
    wrong = [("query", q[:1]), ("query", q[..., :32]), ("query", q.transpose(0, 1)), ("query", q.bfloat16()), ("out", out[:, :4]),
             ("out", out.bfloat16()), ("key_cache", kc[:1]), ("key_cache", kc.view(torch.uint8)), ("value_cache", vc.transpose(1, 2)),
             ("k_scales", ks[:1]), ("k_scales", ks.double()), ("v_scales", vs.t()), ("block_tables", tables.long()),
             ("block_tables", tables[:1]), ("seq_lens", lens.cpu()), ("seq_lens", lens[:0]), ("exp_sums", None),
             ("exp_sums", work[1].flatten()[:3]), ("max_logits", work[2].half()), ("status", lens.long()), ("status", lens[:0])]
    for name, value in wrong:
        with pytest.raises((TypeError, ValueError)):
            pa.pa_decode_q8(**dict(good, **{name: value}))
    torch.cuda.synchronize()


@gpu
def test_partitions_never_finer(pa):
    for S, Q, H, KV, L, P in ((1, 1, 32, 4, 100000, 512), (32, 1, 32, 8, 8192, 512), (32, 16, 32, 8, 8192, 512),
                              (2, 2048, 32, 8, 32768, 512), (1, 1, 8, 2, 1000, 512), (64, 1, 64, 8, 32768, 1000)):
        p = pa.pa_decode_q8_partition(S, Q, H, KV, 128, L, P)
        assert p == 0 or p >= P


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q8", [False, True])
def test_prompt_then_tokens(pa, q8, dtype):
    """The path as it is used: append a ragged prompt, attend to it, then token after token."""
    S, H, KV, D, bs, P = 3, 8, 2, 128, 16, 64
    prompt, steps = [37, 1, 16], 4
    g = torch.Generator().manual_seed(11)
    total = [n + steps for n in prompt]
    width = -(-max(total) // bs)
    tables = torch.randperm(S * width, generator=g).to(torch.int32).view(S, width).cuda()
    kc = torch.zeros((S * width, KV, bs, D), dtype=torch.uint8).view(E4M3).cuda() if q8 else \
        torch.zeros((S * width, KV, bs, D), dtype=dtype).cuda()
    vc = kc.clone()
    ks, vs = (torch.zeros((S * width, KV)).cuda() for _ in range(2))
    t = cu.batch(total, [0] * S, H=H, KV=KV, D=D, bs=bs, dtype=dtype, seed=4)
    cos_sin = t.cos_sin.cuda()
    work = pa.alloc_workspace(S, H, D, pa.num_partitions(width * bs, P))

    def append(rows, lens, starts, query):
        lens = torch.tensor(lens, dtype=torch.int32).cuda()
        out = torch.empty((len(rows), H, D), dtype=dtype).cuda()
        args = (t.key[rows].cuda(), t.value[rows].cuda(), tables, lens, kc, vc)
        opt = dict(cos_sin=cos_sin, query=query.cuda(), query_out=out,
                   token_starts=torch.tensor(starts, dtype=torch.int32).cuda())
        if q8:
            pa.pa_kv_append_q8(*args, ks, vs, **opt)
        else:
            pa.pa_kv_append(*args, **opt)
        return lens, out

    first = [int(x) for x in t.starts[:S]]
    rows = [first[b] + i for b in range(S) for i in range(prompt[b])]
    append(rows, prompt, [0, prompt[0], prompt[0] + prompt[1], sum(prompt)], t.query[rows])
    for n in range(steps):
        rows = [first[b] + prompt[b] + n for b in range(S)]
        lens, q = append(rows, [x + n + 1 for x in prompt], [0, 1, 2, 3], t.query[rows])
        out = torch.empty((S, H, D), dtype=dtype).cuda()
        if q8:
            pa.pa_decode_q8(q, kc, vc, ks, vs, tables, lens, D ** -0.5, P, out, *work)
        else:
            pa.pa_decode(q, kc, vc, tables, lens, D ** -0.5, P, out, *work)
        torch.cuda.synchronize()
        if q8:  # over the codes as they are stored
            ref, tol = cu.attend_reference(q.cpu()[:, None], kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu(), tables.cpu(),
                                           lens.cpu(), D ** -0.5)
            assert ((out.cpu()[:, None].double() - ref).abs() <= tol + cu.rounding(ref.abs() + tol, dtype)).all()
        for b in range(S):
            L = prompt[b] + n + 1
            for h in range(H):
                pairs = [cu.rotate(t.key[first[b] + i].double(), t.cos_sin[i], False)[0][h // 4] for i in range(L)]
                k = torch.stack(pairs)
                v = t.value[first[b]:first[b] + L, h // 4].double()
                qq = cu.rotate(t.query[rows[b]].double(), t.cos_sin[L - 1], False)[0][h]
                w = k @ qq / math.sqrt(D)
                p = torch.softmax(w, 0)
                # K, V and q each off by half a step of their type; a score by at most the sum of the
                # products' errors, P by that factor (at most e^2d - 1), the output by its own rounding.
                ek = cu.HALF_STEP[E4M3 if q8 else dtype]
                tiny = (cu.HALF_TINY[E4M3] * 2 * 2 ** -6 if q8 else 0.0)  # scales here are at most 2^-6
                d = float(((k.abs() * (ek + 2.0 ** -10) + tiny) @ qq.abs() / math.sqrt(D) +
                           k.abs() @ qq.abs() / math.sqrt(D) * cu.HALF_STEP[dtype]).max())
                ref = p @ v
                tol = math.expm1(2 * d) * (p @ (v - ref).abs()) + math.exp(2 * d) * (p @ (v.abs() * (ek + 2.0 ** -10) + tiny))
                tol = tol + cu.rounding(ref.abs() + tol, dtype)
                assert ((out[b, h].double().cpu() - ref).abs() <= tol).all()
    if q8:
        assert float(ks.max()) <= 2.0 ** -6 and float(vs.max()) <= 2.0 ** -6
