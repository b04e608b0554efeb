"""The paged cache on the GPU: append with rotation (bit for bit), and one
token of every sequence over its cache (against the definition in 64 bits)."""
import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from attn_testutil import check, reference, rope_table, rotate, tables

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()


def _randn(seed, *shape, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens, start=0):
    c = [start]
    for n in lens:
        c.append(c[-1] + n)
    return _i32(c)


def _fill(cache, rows, table, held, lens, page):
    """cache [P, HKV, page, d] with rows [sum(lens), HKV, d] put in place."""
    want, t = cache.clone(), 0
    for s, n in enumerate(lens):
        for i in range(n):
            p = held[s] + i
            b = int(table[s, p // page])
            if b >= 0:
                want[b, :, p % page] = rows[t]
            t += 1
    return want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 128, True), (128, 32, False),
                                         (64, 64, True), (64, 48, False), (64, 16, True),
                                         (32, 32, False), (16, 16, True), (16, 16, False), (64, 0, False)])
@pytest.mark.parametrize("lens,held,page", [([1], [0], 16), ([37, 0, 1, 90], [0, 5, 63, 30], 32),
                                            ([130, 5], [1, 511], 256)])
def test_append(dtype, d, rot, inter, lens, held, page):
    HQ, HKV, T, N = 6, 2, sum(lens), len(lens)
    q, k, v = (_randn(i + d, T, h, d, dtype=dtype) for i, h in ((1, HQ), (2, HKV), (3, HKV)))
    need = [(h + n + page - 1) // page for h, n in zip(held, lens)]
    table, pages = tables(need, max(need) + 1)
    kc, vc = (_randn(i, pages, HKV, page, d, dtype=dtype) for i in (7, 8))
    rope = rope_table(700, rot) if rot else None
    pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, lens)])
    want_q, want_k = (rotate(x, pos, rope, inter) if rot else x for x in (q, k))
    gk, gv = kc.cuda(), vc.cuda()
    k_out = torch.empty_like(k, device="cuda")
    q_out, ko = kda.kda_cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), _i32(held),
                                     _cu(lens), q=q.cuda(), k_out=k_out,
                                     rope=rope.cuda() if rot else None, rope_interleaved=inter)
    assert ko is k_out
    # the products and sums are rounded one by one: the same bits
    assert torch.equal(q_out.cpu(), want_q) and torch.equal(k_out.cpu(), want_k)
    assert torch.equal(gk.cpu(), _fill(kc, want_k, table, held, lens, page))
    assert torch.equal(gv.cpu(), _fill(vc, v, table, held, lens, page))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_one_token_each_in_place_and_without_q(dtype):
    N, HQ, HKV, d, page = 9, 4, 4, 64, 16
    held = [0, 1, 15, 16, 17, 31, 32, 47, 3]
    need = [h // page + 1 for h in held]
    table, pages = tables(need, 4)
    q, k, v = (_randn(i, N, HKV, d, dtype=dtype) for i in (1, 2, 3))
    rope = rope_table(64, d)
    pos = torch.tensor(held)
    kc = torch.zeros(pages, HKV, page, d, dtype=DT[dtype])
    want = _fill(kc, rotate(k, pos, rope, False), table, held, [1] * N, page)
    gk, gv = kc.cuda(), kc.cuda()
    assert kda.kda_cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), _i32(held),
                                rope=rope.cuda()) == (None, None)
    assert torch.equal(gk.cpu(), want)
    # q and k rotated in place, twice: two rotations
    gq, gkk = q.cuda(), k.cuda()
    for _ in range(2):
        kda.kda_cache_append(gkk, v.cuda(), gk, gv, table.cuda(), _i32(held), q=gq, q_out=gq,
                             k_out=gkk, rope=rope.cuda())
    assert torch.equal(gq.cpu(), rotate(rotate(q, pos, rope, False), pos, rope, False))
    assert torch.equal(gk.cpu(), _fill(kc, rotate(rotate(k, pos, rope, False), pos, rope, False),
                                       table, held, [1] * N, page))


def test_append_one_sequence_without_offsets():
    T, HKV, d, page, held = 70, 2, 128, 64, 60
    k, v = (_randn(i, T, HKV, d, dtype="bf16") for i in (1, 2))
    table, pages = tables([3], 3)
    kc = _randn(3, pages, HKV, page, d, dtype="bf16")
    gk, gv = kc.cuda(), kc.cuda()
    kda.kda_cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), _i32([held]))
    assert torch.equal(gk.cpu(), _fill(kc, k, table, [held], [T], page))
    assert torch.equal(gv.cpu(), _fill(kc, v, table, [held], [T], page))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_many_tokens_and_graph_replay(dtype):
    """More tokens than take the one-token CTAs, an odd number of them; a
    captured call replayed on other tokens and lengths."""
    HQ, HKV, d, page = 3, 3, 64, 32
    lens, held = [700, 1, 0, 800], [3, 100, 50, 31]
    T = sum(lens)
    need = [(h + n + 40 + page - 1) // page for h, n in zip(held, lens)]
    table, pages = tables(need, max(need))
    rope = rope_table(1000, d)
    x = [_randn(i, T, HKV, d, dtype=dtype) for i in range(6)]
    zero = torch.zeros(pages, HKV, page, d, dtype=DT[dtype])
    gk, gv = zero.cuda(), zero.cuda()
    q, k, v = (t.cuda() for t in x[:3])
    now, q_out, k_out = _i32(held), torch.empty_like(q), torch.empty_like(k)
    cu, gt, gr = _cu(lens), table.cuda(), rope.cuda()

    def call():
        kda.kda_cache_append(k, v, gk, gv, gt, now, cu, q=q, q_out=q_out, k_out=k_out, rope=gr)

    def expect(data, at):
        pos = torch.cat([torch.arange(h, h + n) for h, n in zip(at, lens)])
        rk = rotate(data[1], pos, rope, False)
        assert torch.equal(q_out.cpu(), rotate(data[0], pos, rope, False))
        assert torch.equal(k_out.cpu(), rk)
        assert torch.equal(gk.cpu(), _fill(zero, rk, table, at, lens, page))
        assert torch.equal(gv.cpu(), _fill(zero, data[2], table, at, lens, page))

    call()
    expect(x[:3], held)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    moved = [h + 37 for h in held]
    for t, new in zip((q, k, v), x[3:]):
        t.copy_(new)
    now.copy_(_i32(moved))
    gk.zero_()
    gv.zero_()
    g.replay()
    torch.cuda.synchronize()
    expect(x[3:], moved)


def test_append_views_and_rows_outside_sequences():
    HQ, HKV, d, page, T = 4, 2, 64, 16, 60
    lens, start, held = [20, 13], 9, [3, 40]
    x = _randn(4, T, HQ + 2 * HKV, d, dtype="bf16").cuda()
    q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
    need = [(h + n + page - 1) // page for h, n in zip(held, lens)]
    table, pages = tables(need, max(need))
    kc = torch.zeros(pages, HKV, page, d, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    q_out = torch.full((T, HQ, d), 5.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((T, HKV, d), 5.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_cache_append(k, v, kc, vc, table.cuda(), _i32(held), _cu(lens, start), q=q, q_out=q_out,
                         k_out=k_out)
    a, b = start, start + sum(lens)
    assert torch.equal(q_out[a:b], q[a:b]) and torch.equal(k_out[a:b], k[a:b])
    for o in (q_out, k_out):
        assert (o[:a] == 5).all() and (o[b:] == 5).all()
    zero = torch.zeros(pages, HKV, page, d, dtype=torch.bfloat16)
    assert torch.equal(vc.cpu(), _fill(zero, v[a:b].cpu(), table, held, lens, page))


def test_append_skips_and_reports_bad_places():
    """A negative page keeps the token out of the cache; a position without a
    block-table entry or table row, or a page that does not exist, skips the
    token and is reported."""
    HKV, d, page = 2, 64, 16
    k = _randn(1, 4, HKV, d, dtype="bf16")
    table = torch.tensor([[0, 1], [-1, 2], [3, 9], [-1, -1]], dtype=torch.int32)
    zero = torch.zeros(4, HKV, page, d, dtype=torch.bfloat16)

    def run(held, rope=None):
        kc, vc = zero.cuda(), zero.cuda()
        out = torch.full((4, HKV, d), 5.0, dtype=torch.bfloat16, device="cuda")
        kda.kda_cache_append(k.cuda(), k.cuda(), kc, vc, table.cuda(), _i32(held), k_out=out,
                             rope=rope)
        return kda.kda_device_status(), kc.cpu(), out.cpu()

    st, kc, out = run([0, 3, 15, 20])
    assert st == kda.KDA_SUCCESS
    want = zero.clone()
    want[0, :, 0], want[3, :, 15] = k[0], k[2]
    assert torch.equal(kc, want) and torch.equal(out, k)
    for held, skipped in (([0, 16, 16, 0], 2), ([32, 16, 0, 0], 0), ([-1, 16, 0, 0], 0)):
        st, kc, out = run(held)
        assert st == kda.KDA_ERR_INVALID_ARG
        assert (out[skipped] == 5).all()
        assert torch.equal(out[1], k[1]) and torch.equal(kc[2, :, 0], k[1])
    st, kc, out = run([8, 7, 0, 0], rope_table(8, 64).cuda())   # position 8 of 8
    assert st == kda.KDA_ERR_INVALID_ARG and (out[0] == 5).all() and (out[1] != 5).any()
    assert kda.kda_device_status() == kda.KDA_SUCCESS


# ---------------------------------------------------------------------------
# one token over the cache
# ---------------------------------------------------------------------------
def _paged(seed, lens, HKV, d, page, dtype, garbage=float("nan")):
    """Caches that hold random rows for the lengths and `garbage` elsewhere:
    (k rows, v rows per sequence, k cache, v cache, table)."""
    need = [(n + page - 1) // page for n in lens]
    table, pages = tables(need, max(max(need), 1) + 1, seed=seed)
    kc = torch.full((pages, HKV, page, d), garbage, dtype=DT[dtype])
    vc = kc.clone()
    ks, vs = [], []
    for s, n in enumerate(lens):
        k, v = (_randn(seed + 2 * s + i, n, HKV, d, dtype=dtype) for i in (100, 101))
        ks.append(k)
        vs.append(v)
        for j in range(need[s]):
            m = min(page, n - j * page)
            b = int(table[s, j])
            kc[b, :, :m] = k[j * page:j * page + m].transpose(0, 1)
            vc[b, :, :m] = v[j * page:j * page + m].transpose(0, 1)
    return ks, vs, kc.cuda(), vc.cuda(), table.cuda()


def _widen(table):
    """The table with room for 16384 pages a sequence (none there)."""
    wide = torch.full((table.shape[0], 16384), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    return wide


def _check_step(q, ks, vs, scale, out, lse, weights_bf16):
    for s in range(q.shape[0]):
        n = ks[s].shape[0]
        if n == 0:
            assert (out[s] == 0).all()
            if lse is not None:
                assert (lse[s] == -float("inf")).all()
            continue
        check(out[s:s + 1], None if lse is None else lse[s:s + 1],
              reference(q[s:s + 1], ks[s], vs[s], scale, n - 1), n, q.shape[2], weights_bf16)


def _mma(dtype, d):
    return dtype == "bf16" and d in (64, 128)


STEP = [
    # lens, HQ, HKV, d, page
    ([1], 1, 1, 64, 16), ([0, 0, 0], 2, 1, 128, 16), ([15, 16, 17, 0, 1], 8, 2, 128, 16),
    ([63, 64, 65, 128, 129], 4, 4, 64, 32), ([1000, 3, 0, 260], 8, 1, 128, 64),
    ([4100], 5, 1, 128, 128), ([300, 40], 14, 2, 64, 16), ([500, 20], 16, 1, 128, 256),
    ([90, 1, 777], 12, 4, 64, 64), ([333], 40, 1, 128, 16), ([70, 5], 128, 1, 64, 32),
    ([20000], 2, 2, 64, 64), ([i % 50 for i in range(300)], 4, 2, 64, 16),
]


@pytest.mark.parametrize("lens,HQ,HKV,d,page", STEP)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wide", [False, True])
def test_step(lens, HQ, HKV, d, page, dtype, wide):
    """Rows behind a sequence's length hold NaN and are never used.  Short
    tables and wide ones take different kernels."""
    N = len(lens)
    ks, vs, kc, vc, table = _paged(HQ + d, lens, HKV, d, page, dtype)
    if wide:
        table = _widen(table)
    q = _randn(1, N, HQ, d, dtype=dtype).cuda()
    lse = torch.full((N, HQ), float("nan"), device="cuda")
    out, _ = kda.kda_attn_step(q, kc, vc, table, _i32(lens), d ** -0.5, None, lse)
    _check_step(q, ks, vs, d ** -0.5, out, lse, _mma(dtype, d))


@pytest.mark.parametrize("d", [16, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_narrow_heads(d, dtype):
    lens = [100, 1, 0, 333]
    ks, vs, kc, vc, table = _paged(d, lens, 2, d, 16, dtype)
    q = _randn(1, 4, 6, d, dtype=dtype).cuda()
    out, _ = kda.kda_attn_step(q, kc, vc, table, _i32(lens), 0.4)
    _check_step(q, ks, vs, 0.4, out, None, False)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_step_strided_q_f32_out_and_negative_lengths(dtype, d):
    lens = [200, 0, 31]
    ks, vs, kc, vc, table = _paged(3, lens, 2, d, 32, dtype)
    x = _randn(1, 3, 10, d, dtype=dtype).cuda()
    q = x[:, 2:8]
    given = _i32([200, -4, 31])
    out, _ = kda.kda_attn_step(q, kc, vc, table, given, 0.1, out_f32=True)
    assert out.dtype == torch.float32
    _check_step(q, ks, vs, 0.1, out, None, _mma(dtype, d))
    assert kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_step_scores_far_apart(dtype, d):
    lens = [700]
    ks, vs, kc, vc, table = _paged(4, lens, 1, d, 16, dtype)
    q = _randn(1, 1, 4, d, dtype=dtype).cuda()
    out, _ = kda.kda_attn_step(q, kc, vc, table, _i32(lens), 5.0)
    _check_step(q, ks, vs, 5.0, out, None, _mma(dtype, d))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_step_shared_pages_and_bad_places(dtype, d):
    """Sequences may share pages; lengths past the table and pages that do not
    exist are left out and reported."""
    lens = [96, 96]
    ks, vs, kc, vc, table = _paged(5, lens, 2, d, 32, dtype)
    q = _randn(1, 2, 4, d, dtype=dtype).cuda()
    table[1, 0] = table[0, 0]
    ks[1][:32], vs[1][:32] = ks[0][:32], vs[0][:32]
    out, _ = kda.kda_attn_step(q, kc, vc, table, _i32(lens), 0.1)
    _check_step(q, ks, vs, 0.1, out, None, _mma(dtype, d))
    assert kda.kda_device_status() == kda.KDA_SUCCESS
    good = table[1, 1].item()
    for bad in (-1, kc.shape[0]):
        table[1, 1] = bad
        out, _ = kda.kda_attn_step(q, kc, vc, table, _i32(lens), 0.1)
        assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
        left = [torch.cat((x[1][:32], x[1][64:])) for x in (ks, vs)]
        _check_step(q, [ks[0], left[0]], [vs[0], left[1]], 0.1, out, None, _mma(dtype, d))
    table[1, 1] = good
    table = table[:, :3].contiguous()
    out, _ = kda.kda_attn_step(q, kc, vc, table, _i32([96, 1 << 30]), 0.1)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    _check_step(q, ks, vs, 0.1, out, None, _mma(dtype, d))
    # no pages at all
    empty = kc[:0]
    out, _ = kda.kda_attn_step(q, empty, empty, table[:, :0].contiguous(), _i32([0, 0]), 0.1)
    assert (out == 0).all() and kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_offsets_past_32_bits(dtype):
    """A cache of more than 2^31 elements, the sequence in its last pages."""
    HKV, d, page, n = 8, 128, 64, 1000
    pages = (1 << 31) // (HKV * page * d) + 40
    kc = torch.zeros(pages, HKV, page, d, dtype=DT[dtype], device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs, k, v, table = _paged(6, [n], HKV, d, page, dtype, 0.0)
    m = k.shape[0]
    kc[pages - m:], vc[pages - m:] = k, v
    q = _randn(1, 1, 16, d, dtype=dtype).cuda()
    shifted = torch.where(table >= 0, table + (pages - m), table)
    out, _ = kda.kda_attn_step(q, kc, vc, shifted, _i32([n]), 0.1)
    _check_step(q, ks, vs, 0.1, out, None, _mma(dtype, d))
    new = _randn(9, 1, HKV, d, dtype=dtype).cuda()
    kda.kda_cache_append(new, new, kc, vc, shifted, _i32([n - 1]))
    b, r = int(shifted[0, (n - 1) // page]), (n - 1) % page
    assert torch.equal(kc[b, :, r], new[0]) and torch.equal(vc[b, :, r], new[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wide", [False, True])
def test_step_streams_graphs_and_workspace(dtype, wide):
    """Two calls at once, two captured graphs replayed with other lengths, and
    a caller's workspace all give the bits of a plain call; with a short table
    (no scratch) and with a wide one."""
    lens, HQ, HKV, d, page = [3000, 17, 900, 0, 64], 8, 2, 128, 16
    ks, vs, kc, vc, table = _paged(7, lens, HKV, d, page, dtype)
    if wide:
        table = _widen(table)
    q = [_randn(i, 5, HQ, d, dtype=dtype).cuda() for i in (1, 2)]
    l1, l2 = _i32(lens), _i32([100, 0, 900, 0, 3])
    want = {(i, j): kda.kda_attn_step(q[i], kc, vc, table, l, 0.1)[0]
            for i in (0, 1) for j, l in ((1, l1), (2, l2))}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [kda.kda_attn_step(q[i], kc, vc, table, l1, 0.1, stream=streams[i])[0] for i in (0, 1)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0, 1]) and torch.equal(got[1], want[1, 1])
    cur = l1.clone()
    outs, graphs = [torch.empty_like(x) for x in q], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.kda_attn_step(q[i], kc, vc, table, cur, 0.1, outs[i])
        graphs.append(g)
    for j, l in ((2, l2), (1, l1)):
        cur.copy_(l)
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(outs[i], want[i, j])
    shape = kda.make_attn_shape(5, 5, HQ, HKV, d, kda.KDA_DTYPE_BF16 if dtype == "bf16" else kda.KDA_DTYPE_F32)
    cache = kda.kdaPagedCache_t(kc.data_ptr(), vc.data_ptr(), table.data_ptr(), kc.shape[0], page,
                                table.shape[1])
    need = kda.kda_attn_step_workspace_size(cache, shape)
    assert (need > 0) == wide
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    out, _ = kda.kda_attn_step(q[0], kc, vc, table, l1, 0.1, workspace=ws)
    assert torch.equal(out, want[0, 1])
    if wide:
        with pytest.raises(kda.KdaError):
            kda.kda_attn_step(q[0], kc, vc, table, l1, 0.1, workspace=ws[:1024])
    # the library's own scratch (C entry without a workspace)
    import ctypes
    from kimi_delta_attention_chunkwise_gb300 import binding
    out2 = torch.empty_like(out)
    rc = binding.load().kda_attn_step(q[0].data_ptr(), ctypes.byref(cache), l1.data_ptr(), 0.1,
                                      out2.data_ptr(), None, ctypes.byref(shape),
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == kda.KDA_SUCCESS and torch.equal(out2, want[0, 1])


@pytest.mark.parametrize("dtype,d,inter", [("bf16", 128, False), ("bf16", 64, True), ("f32", 64, False)])
def test_prompt_append_and_steps_together(dtype, d, inter):
    """A served batch: prompts through append and prompt attention, then a few
    decoded tokens through append and step; every output against attention in
    64 bits over the rotated rows."""
    HQ, HKV, page, steps = 6, 2, 16, 3
    lens = [40, 1, 100]
    N, T = 3, 141
    wb = _mma(dtype, d)
    rope = rope_table(256, d)
    need = [(n + steps + page - 1) // page for n in lens]
    table, pages = tables(need, max(need))
    kc = torch.full((pages, HKV, page, d), float("nan"), dtype=DT[dtype], device="cuda")
    vc, table = kc.clone(), table.cuda()
    q, k, v = (_randn(i, T, h, d, dtype=dtype) for i, h in ((1, HQ), (2, HKV), (3, HKV)))
    pos = torch.cat([torch.arange(n) for n in lens])
    rq, rk = (rotate(x, pos, rope, inter) for x in (q, k))
    k_out = torch.empty_like(k, device="cuda")
    cu, held = _cu(lens), _i32([0, 0, 0])
    q_out, _ = kda.kda_cache_append(k.cuda(), v.cuda(), kc, vc, table, held, cu, q=q.cuda(),
                                    k_out=k_out, rope=rope.cuda(), rope_interleaved=inter)
    out, _ = kda.kda_attn_fwd(q_out, k_out, v.cuda(), d ** -0.5, cu)
    a, ks, vs = 0, [], []
    for n in lens:
        check(out[a:a + n], None, reference(rq[a:a + n], rk[a:a + n], v[a:a + n], d ** -0.5, 0), n,
              d, wb)
        ks.append(rk[a:a + n])
        vs.append(v[a:a + n])
        a += n
    held = _i32(lens)
    for i in range(steps):
        q, k, v = (_randn(10 * i + j, N, h, d, dtype=dtype) for j, h in ((4, HQ), (5, HKV), (6, HKV)))
        pos = torch.tensor(lens) + i
        q_out, _ = kda.kda_cache_append(k.cuda(), v.cuda(), kc, vc, table, held, q=q.cuda(),
                                        rope=rope.cuda(), rope_interleaved=inter)
        held += 1
        out, _ = kda.kda_attn_step(q_out, kc, vc, table, held, d ** -0.5)
        rk = rotate(k, pos, rope, inter)
        for s in range(N):
            ks[s], vs[s] = torch.cat((ks[s], rk[s:s + 1])), torch.cat((vs[s], v[s:s + 1]))
        _check_step(rotate(q, pos, rope, inter), ks, vs, d ** -0.5, out, None, wb)
