"""One token of every sequence over a cache whose first pages the sequences share,
against the definition in 64 bits."""
import ctypes

import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from attn_testutil import rope_table, rotate
from cache_testutil import (DT, FP32, ONE_PART, check_rows, i32, mma, offsets, paged_shared, randn,
                            widen)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()


def _weights(dtype, d):
    return ONE_PART if mma(dtype, d) else FP32


def _lens(seed, n, shared, lo, hi):
    """n lengths behind `shared` tokens."""
    g = torch.Generator().manual_seed(seed)
    return [shared + int(x) for x in torch.randint(lo, hi + 1, (n,), generator=g)]


SHARED = [
    # shared pages, lens, HQ, HKV, d, page
    (1, [17], 1, 1, 64, 16),                                     # a lone sequence
    (1, [16, 16, 16], 2, 1, 128, 16),                            # nothing behind the shared page
    (0, [5, 70, 0], 8, 2, 128, 32),                              # no shared page
    (2, [33, 40, 0, 31, 32, 1, 64], 8, 2, 64, 16),               # some that hold less
    (3, [0, 0, 20], 4, 2, 128, 16),                              # none that holds them
    (8, _lens(1, 9, 128, 0, 40), 8, 8, 128, 16),                 # one tile of keys
    (9, _lens(2, 9, 144, 0, 40), 12, 4, 128, 16),                # a tile and 16 tokens
    (17, _lens(3, 5, 272, 0, 130), 14, 2, 64, 16),
    (5, _lens(4, 3, 1280, 1, 300), 16, 1, 128, 256),             # pages of two tiles
    (4, _lens(5, 11, 512, 1, 30), 8, 2, 64, 128),
    (30, _lens(6, 31, 1920, 0, 200), 32, 8, 128, 64),            # a batch
    (30, _lens(7, 40, 1920, 0, 100), 20, 4, 64, 64),
    (40, _lens(8, 130, 1280, 0, 60), 8, 2, 128, 32),             # more rows than a row tile
    (20, _lens(9, 70, 640, 0, 60), 40, 8, 64, 32),
    (6, _lens(10, 3, 384, 0, 60), 128, 1, 128, 64),              # a row tile per sequence
    (6, _lens(11, 5, 384, 0, 60), 70, 1, 64, 64),
    (7, _lens(12, 90, 448, 0, 60), 3, 1, 128, 64),               # 42 sequences to a row tile
    (300, _lens(13, 4, 19200, 0, 200), 8, 2, 128, 64),           # many tiles of keys
    (500, _lens(14, 2, 8000, 0, 3), 2, 2, 64, 16),
]


@pytest.mark.parametrize("common,lens,HQ,HKV,d,page", SHARED)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wide", [False, True])
def test_shared(common, lens, HQ, HKV, d, page, dtype, wide):
    """NaN behind every length is never used, nor what a shorter sequence leaves of
    its row of the table."""
    N = len(lens)
    ks, vs, kc, vc, table = paged_shared(HQ + d, common, lens, HKV, d, page, dtype)
    if wide:
        table = widen(table)
    q = randn(1, N, HQ, d, dtype=dtype).cuda()
    lse = torch.full((N, HQ), float("nan"), device="cuda")
    args = (q, kc, vc, table, i32(lens), i32([common]), d ** -0.5)
    out, _ = kda.kda_attn_step_shared(*args, None, lse)
    check_rows(q, ks, vs, d ** -0.5, out, lse, _weights(dtype, d))
    assert kda.kda_device_status() == kda.KDA_SUCCESS
    # the same call gives the same bits
    assert torch.equal(kda.kda_attn_step_shared(*args)[0], out)


@pytest.mark.parametrize("d", [16, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_narrow_heads(d, dtype):
    lens = [160, 100, 0, 333, 129]
    ks, vs, kc, vc, table = paged_shared(d, 8, lens, 2, d, 16, dtype)
    q = randn(1, 5, 6, d, dtype=dtype).cuda()
    out, _ = kda.kda_attn_step_shared(q, kc, vc, table, i32(lens), i32([8]), 0.4)
    check_rows(q, ks, vs, 0.4, out, None, FP32)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_shared_strided_q_f32_out_and_negative_lengths(dtype, d):
    lens = [200, 0, 131, 128]
    ks, vs, kc, vc, table = paged_shared(3, 4, lens, 2, d, 32, dtype)
    q = randn(1, 4, 10, d, dtype=dtype).cuda()[:, 2:8]
    out, _ = kda.kda_attn_step_shared(q, kc, vc, table, i32([200, -4, 131, 128]), i32([4]), 0.1,
                                      out_f32=True)
    assert out.dtype == torch.float32
    check_rows(q, ks, vs, 0.1, out, None, _weights(dtype, d))
    assert kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_shared_scores_far_apart(dtype, d):
    """Maxima that move by far more than 2^8 from tile to tile and between the
    shared tokens and a sequence's own."""
    lens = _lens(1, 6, 1280, 0, 300)
    ks, vs, kc, vc, table = paged_shared(4, 20, lens, 2, d, 64, dtype)
    q = randn(1, 6, 8, d, dtype=dtype).cuda()
    q[3] *= 100
    q[4] *= 0
    lse = torch.empty(6, 8, device="cuda")
    out, _ = kda.kda_attn_step_shared(q, kc, vc, table, i32(lens), i32([20]), 2.0, None, lse)
    check_rows(q, ks, vs, 2.0, out, lse, _weights(dtype, d))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_shared_bad_places(dtype, d, page):
    """Shared pages that do not exist are left out for all that share them, and
    reported; so are the step's own places and numbers out of range."""
    common = 768 // page
    lens = [800, 768, 900, 5, 0]
    ks, vs, kc, vc, table = paged_shared(5, common, lens, 2, d, page, dtype)
    q = randn(1, 5, 6, d, dtype=dtype).cuda()
    call = lambda t, n, l=lens: kda.kda_attn_step_shared(q, kc, vc, t, i32(l), i32([n]), 0.1)[0]
    w = _weights(dtype, d)
    for bad, at in ((-1, 0), (kc.shape[0], common - 1), (1 << 30, common // 2)):
        t = table.clone()
        t[:3, at] = bad
        out = call(t, common)
        assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
        left = [[torch.cat((x[s][:at * page], x[s][(at + 1) * page:])) if s < 3 else x[s]
                 for s in range(5)] for x in (ks, vs)]
        check_rows(q, *left, 0.1, out, None, w)
    # no shared page that exists: the sequences' own tokens alone
    t = table.clone()
    t[:3, :common] = -1
    out = call(t, common)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    left = [[x[s][768:] if s < 3 else x[s] for s in range(5)] for x in (ks, vs)]
    check_rows(q, *left, 0.1, out, None, w)
    # a negative number is none; one above the table's width is the width, and with
    # it no sequence here holds them all
    for n in (-3, table.shape[1] + 5):
        out = call(table, n)
        assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
        check_rows(q, ks, vs, 0.1, out, None, w)
    assert torch.equal(call(table, common), call(table, common))
    assert kda.kda_device_status() == kda.KDA_SUCCESS
    # a length past the table
    t = table[:, :-(-900 // page)].contiguous()
    out = call(t, common, [800, 768, 1 << 30, 5, 0])
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    check_rows(q[:2], ks[:2], vs[:2], 0.1, out[:2], None, w)
    # no pages at all
    empty = kc[:0]
    out, _ = kda.kda_attn_step_shared(q, empty, empty, table[:, :0].contiguous(), i32([0] * 5),
                                      i32([0]), 0.1)
    assert (out == 0).all() and kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_shared_rows_of_infinite_scores_and_nan(dtype, d):
    """A key of -infinity in a shared page scores -infinity or NaN for all; a NaN
    in one sequence's own tokens is that sequence's."""
    lens = [300, 280, 256]
    ks, vs, kc, vc, table = paged_shared(6, 4, lens, 1, d, 64, dtype)
    kc[int(table[1, 4]), 0, 3] = float("nan")
    q = randn(1, 3, 2, d, dtype=dtype).cuda()
    out, _ = kda.kda_attn_step_shared(q, kc, vc, table, i32(lens), i32([4]), 0.1)
    assert out[1].isnan().all()
    for s in (0, 2):
        check_rows(q[s:s + 1], ks[s:s + 1], vs[s:s + 1], 0.1, out[s:s + 1], None, _weights(dtype, d))
    # all scores of the shared tokens -infinity: weights of 0
    q = q.abs()
    for j in range(4):
        kc[int(table[0, j])] = -float("inf")
    lse = torch.empty(3, 2, device="cuda")
    out, _ = kda.kda_attn_step_shared(q, kc, vc, table, i32(lens), i32([4]), 0.1, None, lse)
    check_rows(q[:1], [ks[0][256:]], [vs[0][256:]], 0.1, out[:1], lse[:1], _weights(dtype, d))
    # and no others: the formula's 0 / 0
    assert out[2].isnan().all() and (lse[2] == -float("inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_offsets_past_32_bits(dtype):
    """A cache of more than 2^31 elements, all pages among its last."""
    HKV, d, page, lens = 8, 128, 64, [1000, 960, 1100]
    pages = (1 << 31) // (HKV * page * d) + 40
    ks, vs, k, v, table = paged_shared(6, 15, lens, HKV, d, page, dtype, 0.0)
    m = k.shape[0]
    kc = torch.zeros(pages, HKV, page, d, dtype=DT[dtype], device="cuda")
    vc = torch.zeros_like(kc)
    kc[pages - m:], vc[pages - m:] = k, v
    q = randn(1, 3, 16, d, dtype=dtype).cuda()
    shifted = torch.where(table >= 0, table + (pages - m), table)
    out, _ = kda.kda_attn_step_shared(q, kc, vc, shifted, i32(lens), i32([15]), 0.1)
    check_rows(q, ks, vs, 0.1, out, None, _weights(dtype, d))


@pytest.mark.parametrize("HQ,HKV,d,dtype", [(8, 2, 128, "bf16"), (8, 2, 64, "bf16"), (1, 1, 128, "bf16"),
                                            (40, 1, 64, "bf16"), (6, 2, 64, "f32")])
@pytest.mark.parametrize("where", ["shared", "own"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_shared_infinite_values(HQ, HKV, d, dtype, where, value):
    """A non-finite value shows in its channel, however small its weight, and in no
    other channel; in one sequence's own tokens, in that sequence's rows alone."""
    lens = [700, 600, 520, 530, 515]
    _, _, kc, vc, table = paged_shared(8, 8, lens, HKV, d, 64, dtype, 0.0)
    page, row = (int(table[0, 4]), 13) if where == "shared" else (int(table[0, 9]), 21)
    q = torch.zeros(len(lens), HQ, d, dtype=DT[dtype], device="cuda")
    q[..., 0] = 1
    kc[..., 0] = 0
    vc[page, :, row, 5] = value
    for gap in (0.0, 1.0, 30.0, 100.0, 124.0):
        kc[page, :, row, 0] = -gap
        out, _ = kda.kda_attn_step_shared(q, kc, vc, widen(table), i32(lens), i32([8]),
                                          0.6931471805599453)
        seen = out[..., 5].float()
        has = torch.isnan(seen) if value != value else seen == value
        hit = slice(0, None) if where == "shared" else slice(0, 1)
        assert has[hit].all()
        if where == "own":
            assert torch.isfinite(seen[1:]).all()
        rest = torch.cat((out[..., :5], out[..., 6:]), dim=-1)
        assert torch.isfinite(rest).all()


@pytest.mark.parametrize("HQ,HKV", [(2, 2), (4, 2), (3, 1), (9, 1)])
@pytest.mark.parametrize("dtype,d", [("f32", 16), ("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 16),
                                     ("bf16", 32)])
@pytest.mark.parametrize("common,lens", [(4, [2256, 300, 4100, 256, 257, 80]), (0, [3000]), (30, [9000, 1920])])
def test_shared_long_tails_of_few_rows(HQ, HKV, dtype, d, common, lens):
    """Own tokens that many CTAs share, with every number of rows to a CTA."""
    ks, vs, kc, vc, table = paged_shared(d + HQ, common, lens, HKV, d, 64, dtype)
    q = randn(2, len(lens), HQ, d, dtype=dtype).cuda()
    lse = torch.full((len(lens), HQ), float("nan"), device="cuda")
    out, _ = kda.kda_attn_step_shared(q, kc, vc, widen(table), i32(lens), i32([common]), d ** -0.5,
                                      None, lse)
    check_rows(q, ks, vs, d ** -0.5, out, lse, _weights(dtype, d))


@pytest.mark.parametrize("dtype,HQ", [("bf16", 2), ("bf16", 9), ("f32", 2)])
def test_shared_thousands_of_sequences(dtype, HQ):
    """Sequences by the thousand with few tokens of their own, none, or too few to share."""
    N, d, common = 2500, 64, 5
    lens = [80 + (7 * i) % 30 if i % 5 else (11 * i) % 80 for i in range(N)]
    lens[7::50] = [80] * len(lens[7::50])
    ks, vs, kc, vc, table = paged_shared(18, common, lens, 1, d, 16, dtype)
    q = randn(2, N, HQ, d, dtype=dtype).cuda()
    lse = torch.full((N, HQ), float("nan"), device="cuda")
    out, _ = kda.kda_attn_step_shared(q, kc, vc, widen(table, 64), i32(lens), i32([common]), d ** -0.5,
                                      None, lse)
    check_rows(q, ks, vs, d ** -0.5, out, lse, _weights(dtype, d))
    assert kda.kda_device_status() == kda.KDA_SUCCESS


MANY = [
    # shared pages, sequences, own tokens up to, HQ, HKV, d, page
    (32, 96, 900, 32, 8, 128, 64),       # much of both kinds: the SMs divided
    (64, 40, 40, 32, 8, 128, 64),        # nearly all of it shared
    (2, 200, 700, 16, 4, 128, 64),       # nearly none of it
    (16, 300, 300, 12, 2, 64, 128),
    (24, 150, 500, 40, 4, 64, 32),       # 10 query heads to a key-value head
    (40, 64, 300, 32, 2, 128, 32),       # 16
]


@pytest.mark.parametrize("common,n,most,HQ,HKV,d,page", MANY)
def test_shared_many_sequences(common, n, most, HQ, HKV, d, page):
    """Sequences of every length behind the shared tokens, some of none and some that
    hold fewer than those."""
    lens = _lens(20 + n, n, common * page, 0, most)
    lens[3:n:17] = [common * page] * len(lens[3:n:17])
    lens[5:n:29] = _lens(n, len(lens[5:n:29]), 0, 0, common * page - 1)
    ks, vs, kc, vc, table = paged_shared(n, common, lens, HKV, d, page, "bf16")
    q = randn(1, n, HQ, d, dtype="bf16").cuda()
    lse = torch.full((n, HQ), float("nan"), device="cuda")
    args = (q, kc, vc, widen(table), i32(lens), i32([common]), d ** -0.5)
    out, _ = kda.kda_attn_step_shared(*args, None, lse)
    check_rows(q, ks, vs, d ** -0.5, out, lse, ONE_PART)
    assert kda.kda_device_status() == kda.KDA_SUCCESS
    assert torch.equal(kda.kda_attn_step_shared(*args)[0], out)


@pytest.mark.parametrize("dtype,d,HQ", [("bf16", 64, 1), ("bf16", 64, 16), ("f32", 16, 1)])
@pytest.mark.parametrize("left,own", [(65, 1), (32, 1 << 30)])
def test_shared_lengths_up_to_2_31(dtype, d, HQ, left, own):
    """A table of 2^31 - 32 tokens whose entries name one page of 32 over and
    over: nearly all of them shared, or half of them, by two sequences, and a third
    of 70 tokens.

    Bound: as for kda_attn_step's, with at most sixteen additions to an accumulator
    (two to a sum) per 128 tokens and pieces for a quarter of the SMs at least; one bf16 rounding of
    a weight (2^-8) and the output's."""
    page, top = 32, 1 << 31
    width = top // page - 1
    k, v = (randn(i, 1, 1, page, d, dtype=dtype) for i in (1, 2))
    v += 1   # (means that are not near zero)
    q = randn(3, 3, HQ, d, dtype=dtype)
    table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
    lens = [top - left, top - left - 5, 70]
    shared = (top - left - 5 - (own if own > 1 else 0)) // page
    lse = torch.full((3, HQ), float("nan"), device="cuda")
    scale = d ** -0.5
    out, _ = kda.kda_attn_step_shared(q.cuda(), k.cuda(), v.cuda(), table, i32(lens), i32([shared]),
                                      scale, None, lse)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for s, n in enumerate(lens):
        count = n // page + (torch.arange(page) < n % page)
        z = scale * (q[s].double() @ k[0, 0].double().T)
        w = count * torch.exp(z - z.amax(-1, keepdim=True))
        l = w.sum(-1, keepdim=True)
        want, size = (w @ v[0, 0].double()) / l, (w @ v[0, 0].double().abs()) / l
        rel = 16 * (n / 128 / (sms / 4) + 1) * 2.0 ** -23 + 1e-4
        lz = z.amax(-1) + l[:, 0].log()
        assert ((lse[s].cpu().double() - lz).abs() <= rel / 8 + 1e-4).all()
        assert ((out[s].cpu().double() - want).abs() <= (2 * rel + 2.0 ** -7) * size).all()
    assert kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("wide", [False, True])
def test_shared_streams_graphs_and_workspace(dtype, d, wide):
    """Two calls at once, two captured graphs replayed with other lengths and
    another number of shared pages, and a caller's workspace: the bits of a plain
    call."""
    lens, HQ, HKV, page, common = [3000, 517, 900, 0, 564], 8, 2, 16, 32
    ks, vs, kc, vc, table = paged_shared(7, common, lens, HKV, d, page, dtype)
    if wide:
        table = widen(table)
    q = [randn(i, 5, HQ, d, dtype=dtype).cuda() for i in (1, 2)]
    settings = {1: (i32(lens), i32([common])), 2: (i32([600, 0, 512, 0, 3]), i32([5])),
                3: (i32(lens), i32([0]))}
    step = lambda i, l, n, **kw: kda.kda_attn_step_shared(q[i], kc, vc, table, l, n, 0.1, **kw)[0]
    want = {(i, j): step(i, *settings[j]) for i in (0, 1) for j in settings}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [step(i, *settings[1], stream=streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0, 1]) and torch.equal(got[1], want[1, 1])
    cur, now = settings[1][0].clone(), settings[1][1].clone()
    outs, graphs = [torch.empty_like(x) for x in q], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(i, cur, now, out=outs[i])
        graphs.append(g)
    for j in (2, 3, 1):
        cur.copy_(settings[j][0])
        now.copy_(settings[j][1])
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(outs[i], want[i, j])
    code = kda.KDA_DTYPE_BF16 if dtype == "bf16" else kda.KDA_DTYPE_F32
    shape = kda.make_attn_shape(5, 5, HQ, HKV, d, code)
    c = kda.kdaPagedCache_t(kc.data_ptr(), vc.data_ptr(), table.data_ptr(), kc.shape[0], page,
                            table.shape[1])
    need = kda.kda_attn_step_shared_workspace_size(c, shape)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    assert torch.equal(step(0, *settings[1], workspace=ws), want[0, 1])
    assert (need > 0) == wide   # (short tables take none)
    if wide:
        with pytest.raises(kda.KdaError):
            step(0, *settings[1], workspace=ws[:512])
    # the library's own scratch (C entry without a workspace)
    from kimi_delta_attention_chunkwise_gb300 import binding
    out2 = torch.empty_like(want[0, 1])
    rc = binding.load().kda_attn_step_shared(
        q[0].data_ptr(), ctypes.byref(c), settings[1][0].data_ptr(), settings[1][1].data_ptr(),
        0.1, out2.data_ptr(), None, ctypes.byref(shape), torch.cuda.current_stream().cuda_stream)
    assert rc == kda.KDA_SUCCESS and torch.equal(out2, want[0, 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_calls_in_a_row(dtype):
    """Calls of several sizes one after the other on one stream, and a plain step
    between them: what a call starts early never passes what it needs."""
    HQ, HKV, d, page = 8, 2, 128, 32
    jobs = []
    for i, (common, n) in enumerate(((40, 3), (2, 60), (100, 20), (1, 1))):
        lens = _lens(20 + i, n, common * page, 0, 200)
        ks, vs, kc, vc, table = paged_shared(i, common, lens, HKV, d, page, dtype)
        q = randn(i, n, HQ, d, dtype=dtype).cuda()
        jobs.append((q, kc, vc, widen(table), i32(lens), i32([common])))
    run = lambda j: kda.kda_attn_step_shared(*j, 0.1)[0]
    want = []
    for j in jobs:
        torch.cuda.synchronize()
        want.append(run(j))
    torch.cuda.synchronize()
    for _ in range(30):
        got = []
        for j in jobs:
            got.append(run(j))
            kda.kda_attn_step(*j[:5], 0.1)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_a_prompt_and_its_samples_together(dtype, d):
    """A prompt through append and prompt attention; several answers to it, decoded
    behind its whole pages: append, then the shared step and the plain one."""
    HQ, HKV, page, n, T = 6, 2, 16, 5, 83
    rope = rope_table(256, d)
    whole = T // page
    pages = whole + 2 * n
    kc = torch.full((pages, HKV, page, d), float("nan"), dtype=DT[dtype], device="cuda")
    vc = kc.clone()
    table = torch.zeros(n, whole + 2, dtype=torch.int32)
    table[:, :whole] = torch.arange(whole)
    table[:, whole:] = whole + torch.arange(2 * n).view(n, 2)
    table = table.cuda()
    q, k, v = (randn(i, T, h, d, dtype=dtype) for i, h in ((1, HQ), (2, HKV), (3, HKV)))
    pos = torch.arange(T)
    rq, rk = (rotate(x, pos, rope, False) for x in (q, k))
    # the prompt into the first answer's pages, its last, partial one to each of the others
    kda.kda_cache_append(k.cuda(), v.cuda(), kc, vc, table[:1], i32([0]), rope=rope.cuda())
    rest = slice(whole * page, T)
    for s in range(1, n):
        kda.kda_cache_append(k[rest].cuda(), v[rest].cuda(), kc, vc, table[s:s + 1],
                             i32([whole * page]), rope=rope.cuda())
    ks, vs = [rk] * n, [v] * n
    held, common = i32([T] * n), i32([whole])
    for i in range(3):
        q, k, v = (randn(10 * i + j, n, h, d, dtype=dtype) for j, h in ((4, HQ), (5, HKV), (6, HKV)))
        pos = torch.full((n,), T + i)
        q_out, _ = kda.kda_cache_append(k.cuda(), v.cuda(), kc, vc, table, held, q=q.cuda(),
                                        rope=rope.cuda())
        held += 1
        out, _ = kda.kda_attn_step_shared(q_out, kc, vc, table, held, common, d ** -0.5)
        plain, _ = kda.kda_attn_step(q_out, kc, vc, table, held, d ** -0.5)
        rk = rotate(k, pos, rope, False)
        ks = [torch.cat((x, rk[s:s + 1])) for s, x in enumerate(ks)]
        vs = [torch.cat((x, v[s:s + 1])) for s, x in enumerate(vs)]
        for o in (out, plain):
            check_rows(rotate(q, pos, rope, False), ks, vs, d ** -0.5, o, None, _weights(dtype, d))
