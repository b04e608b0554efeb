"""The paged cache of 8-bit codes on the GPU: append (codes, scales and what they
stand for, bit for bit), and one token of every sequence over it (against the
definition in 64 bits)."""
import ctypes
import math

import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from attn_testutil import rope_table, rotate, tables
from cache_testutil import (DT, FP32, ONE_PART, SMALLEST, TWO_PARTS, check_rows, encode, i32, mma,
                            offsets, paged_q8, put, randn, widen)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()


def _same(got, want):
    """Bit for bit, but for which NaN a NaN is."""
    got = got.cpu()
    return torch.equal(got.isnan(), want.isnan()) and \
        torch.equal(got.nan_to_num(0.0, float("inf"), -float("inf")),
                    want.nan_to_num(0.0, float("inf"), -float("inf")))


class _Cache:
    """A cache that holds other rows' codes already, and its copy on the CPU."""

    def __init__(self, pages, HKV, page, d, seed=9):
        g = torch.Generator().manual_seed(seed)
        self.codes = [torch.randint(-127, 128, (pages, HKV, page, d), generator=g, dtype=torch.int8)
                      for _ in range(2)]
        self.scales = [torch.rand(pages, HKV, page, generator=g) for _ in range(2)]
        self.gpu = [x.cuda() for x in (*self.codes, *self.scales)]

    def expect(self, k, v, table, held, lens):
        """The rows k, v (fp32, rotated) put in; compares the GPU's, which are to be
        the same everywhere.  Returns what the rows stand for."""
        stood = []
        for i, x in enumerate((k, v)):
            c, f = encode(x)
            put(self.codes[i], c.to(torch.int8), table, held, lens)
            put(self.scales[i], f, table, held, lens)
            assert torch.equal(self.gpu[i].cpu(), self.codes[i])
            assert _same(self.gpu[2 + i], self.scales[i])
            stood.append(c * f[..., None])
        return stood


def _turned(x, pos, rope, inter):
    """x rotated in fp32, and rounded to its type (CPU)."""
    if rope is None:
        return x.float(), x
    y = rotate(x.float(), pos, rope, inter)
    return y, y.to(x.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 128, True), (128, 32, False),
                                         (64, 64, True), (64, 48, False), (64, 16, True),
                                         (32, 32, False), (16, 16, True), (16, 16, False),
                                         (64, 0, False)])
@pytest.mark.parametrize("lens,held,page", [([1], [0], 16), ([37, 0, 1, 90], [0, 5, 63, 30], 32),
                                            ([130, 5], [1, 511], 256)])
def test_append(dtype, d, rot, inter, lens, held, page):
    HQ, HKV, T = 6, 2, sum(lens)
    q, k, v = (randn(i + d, T, h, d, dtype=dtype) for i, h in ((1, HQ), (2, HKV), (3, HKV)))
    need = [(h + n + page - 1) // page for h, n in zip(held, lens)]
    table, pages = tables(need, max(need) + 1)
    c = _Cache(pages, HKV, page, d)
    rope = rope_table(700, rot) if rot else None
    pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, lens)])
    made = [torch.empty_like(x, device="cuda") for x in (k, k, v)]
    q_out, k_out = kda.kda_cache_append_q8(
        k.cuda(), v.cuda(), *c.gpu, table.cuda(), i32(held), offsets(lens), q=q.cuda(),
        k_out=made[0], k_stored=made[1], v_stored=made[2], rope=rope.cuda() if rot else None,
        rope_interleaved=inter)
    assert k_out is made[0]
    rk, rk_out = _turned(k, pos, rope, inter)
    assert torch.equal(q_out.cpu(), _turned(q, pos, rope, inter)[1])
    assert torch.equal(k_out.cpu(), rk_out)
    stood = c.expect(rk, v.float(), table, held, lens)
    for got, want, x in zip(made[1:], stood, (rk, v.float())):
        assert torch.equal(got.cpu(), want.to(DT[dtype]))
        # half a scale, and the roundings of 127 / top, the product and code * scale
        top = x.abs().amax(dim=-1, keepdim=True).double()
        assert ((want.double() - x.double()).abs() <= top / 127 * (0.5 + 127 * 3 * 2.0 ** -24)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_append_rows_at_the_ends_of_the_numbers(dtype, d):
    """Zeros, numbers around the smallest that is held, the largest, infinities
    and NaN: a row's codes and scale are its own whatever its neighbours hold."""
    big = float(torch.finfo(DT[dtype]).max)
    tops = [0.0, 1e-40, SMALLEST * 0.99, SMALLEST, SMALLEST * 1.25, 1e-20, 1.0, 3e30, big,
            float("inf"), -float("inf"), float("nan"), 127.0, -127.0, 126.5]
    N, HKV, page = len(tops), 2, 16
    k, v = (randn(i, N, HKV, d).clamp(-0.9, 0.9) for i in (1, 2))
    for i, t in enumerate(tops):
        size = abs(t) if abs(t) <= big else 1.0
        for x, j in ((k, i), (v, N - 1 - i)):
            x[j] *= size
            x[j, :, (5 * i) % d] = t
    k, v = k.to(DT[dtype]), v.to(DT[dtype])
    table = torch.arange(N, dtype=torch.int32)[:, None].contiguous()
    c = _Cache(N, HKV, page, d)
    ks, vs = torch.empty_like(k, device="cuda"), torch.empty_like(v, device="cuda")
    kda.kda_cache_append_q8(k.cuda(), v.cuda(), *c.gpu, table.cuda(), i32(list(range(N))),
                            k_stored=ks, v_stored=vs)
    stood = c.expect(k.float(), v.float(), table, list(range(N)), [1] * N)
    assert _same(ks, stood[0].to(DT[dtype])) and _same(vs, stood[1].to(DT[dtype]))
    assert (stood[0][0] == 0).all() and (stood[0][2] == 0).all() and (stood[0][3] != 0).any()
    assert stood[0][9:12].isnan().all() and torch.isfinite(stood[0][12:]).all()


def test_append_ties_go_to_the_even_code():
    """A row whose largest is 127 has a scale of 1: halves lie between two codes."""
    d, page = 64, 16
    k = torch.zeros(1, 1, d, dtype=torch.bfloat16)
    k[0, 0, :9] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 63.5, -62.5, 3.25]).bfloat16()
    c = _Cache(1, 1, page, d)
    kda.kda_cache_append_q8(k.cuda(), k.cuda(), *c.gpu, i32([[0]]), i32([3]))
    want = torch.tensor([127, 0, 2, 2, 0, -2, 64, -62, 3], dtype=torch.int8)
    assert torch.equal(c.gpu[0][0, 0, 3, :9].cpu(), want)
    assert c.gpu[2][0, 0, 3].item() == 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_many_tokens_in_place_and_graph_replay(dtype):
    """More tokens than take the one-token CTAs, an odd number of them, q and k
    rotated in place; a captured call replayed on other tokens and lengths."""
    HQ, HKV, d, page = 3, 3, 64, 32
    lens, held = [700, 1, 0, 800], [3, 100, 50, 31]
    T = sum(lens)
    need = [(h + n + 40 + page - 1) // page for h, n in zip(held, lens)]
    table, pages = tables(need, max(need))
    rope = rope_table(1000, d)
    x = [randn(i, T, HKV, d, dtype=dtype) for i in range(6)]
    c = _Cache(pages, HKV, page, d)
    q, k, v = (t.cuda() for t in x[:3])
    now, cu, gt, gr = i32(held), offsets(lens), table.cuda(), rope.cuda()
    stored = torch.empty_like(k)

    def call():
        kda.kda_cache_append_q8(k, v, *c.gpu, gt, now, cu, q=q, q_out=q, k_out=k, v_stored=stored,
                                rope=gr)

    def expect(data, at):
        pos = torch.cat([torch.arange(h, h + n) for h, n in zip(at, lens)])
        rk, rk_out = _turned(data[1], pos, rope, False)
        assert torch.equal(q.cpu(), _turned(data[0], pos, rope, False)[1])
        assert torch.equal(k.cpu(), rk_out)
        stood = c.expect(rk, data[2].float(), table, at, lens)
        assert torch.equal(stored.cpu(), stood[1].to(DT[dtype]))

    call()
    expect(x[:3], held)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    moved = [h + 37 for h in held]
    for t, new in zip((q, k, v), x[3:]):
        t.copy_(new)
    now.copy_(i32(moved))
    g.replay()
    torch.cuda.synchronize()
    expect(x[3:], moved)


def test_append_views_and_rows_outside_sequences():
    HQ, HKV, d, page, T = 4, 2, 64, 16, 60
    lens, start, held = [20, 13], 9, [3, 40]
    x = randn(4, T, HQ + 2 * HKV, d, dtype="bf16")
    gx = x.cuda()
    need = [(h + n + page - 1) // page for h, n in zip(held, lens)]
    table, pages = tables(need, max(need))
    c = _Cache(pages, HKV, page, d)
    full = lambda h: torch.full((T, h, d), 5.0, dtype=torch.bfloat16, device="cuda")
    q_out, k_out, ks, vs = full(HQ), full(HKV), full(HKV), full(HKV)
    kda.kda_cache_append_q8(gx[:, HQ:HQ + HKV], gx[:, HQ + HKV:], *c.gpu, table.cuda(), i32(held),
                            offsets(lens, start), q=gx[:, :HQ], q_out=q_out, k_out=k_out,
                            k_stored=ks, v_stored=vs)
    a, b = start, start + sum(lens)
    k, v = x[a:b, HQ:HQ + HKV], x[a:b, HQ + HKV:]
    assert torch.equal(q_out[a:b].cpu(), x[a:b, :HQ]) and torch.equal(k_out[a:b].cpu(), k)
    stood = c.expect(k.float(), v.float(), table, held, lens)
    assert torch.equal(ks[a:b].cpu(), stood[0].bfloat16())
    assert torch.equal(vs[a:b].cpu(), stood[1].bfloat16())
    for o in (q_out, k_out, ks, vs):
        assert (o[:a] == 5).all() and (o[b:] == 5).all()


def test_append_skips_and_reports_bad_places():
    """As kda_cache_append: a negative page keeps the token out of the cache; a
    position without a block-table entry or table row, or a page that does not
    exist, skips the token and is reported."""
    HKV, d, page = 2, 64, 16
    k = randn(1, 4, HKV, d, dtype="bf16")
    table = torch.tensor([[0, 1], [-1, 2], [3, 9], [-1, -1]], dtype=torch.int32)

    def run(held, rope=None):
        c = _Cache(4, HKV, page, d)
        out = torch.full((2, 4, HKV, d), 5.0, dtype=torch.bfloat16, device="cuda")
        kda.kda_cache_append_q8(k.cuda(), k.cuda(), *c.gpu, table.cuda(), i32(held), k_out=out[0],
                                v_stored=out[1], rope=rope)
        return kda.kda_device_status(), c, out.cpu()

    codes, scales = encode(k)
    stood = (codes * scales[..., None]).bfloat16()
    st, c, out = run([0, 3, 15, 20])
    assert st == kda.KDA_SUCCESS and torch.equal(out[0], k) and torch.equal(out[1], stood)
    c.codes[0][0, :, 0], c.codes[0][3, :, 15] = codes[0].to(torch.int8), codes[2].to(torch.int8)
    c.scales[0][0, :, 0], c.scales[0][3, :, 15] = scales[0], scales[2]
    assert torch.equal(c.gpu[0].cpu(), c.codes[0]) and torch.equal(c.gpu[2].cpu(), c.scales[0])
    for held, skipped in (([0, 16, 16, 0], 2), ([32, 16, 0, 0], 0), ([-1, 16, 0, 0], 0)):
        st, c, out = run(held)
        assert st == kda.KDA_ERR_INVALID_ARG
        assert (out[:, skipped] == 5).all()
        assert torch.equal(out[0, 1], k[1]) and torch.equal(out[1, 1], stood[1])
        assert torch.equal(c.gpu[0][2, :, 0].cpu(), codes[1].to(torch.int8))
    st, c, out = run([8, 7, 0, 0], rope_table(8, 64).cuda())   # position 8 of 8
    assert st == kda.KDA_ERR_INVALID_ARG and (out[:, 0] == 5).all() and (out[:, 1] != 5).any()
    assert kda.kda_device_status() == kda.KDA_SUCCESS


# ---------------------------------------------------------------------------
# one token over the cache
# ---------------------------------------------------------------------------
def _weights(dtype, d):
    return TWO_PARTS if mma(dtype, d) else FP32


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
    """Rows behind a sequence's length hold scales of NaN and are never used.
    Short tables and wide ones take different kernels."""
    N = len(lens)
    ks, vs, cache, table = paged_q8(HQ + d, lens, HKV, d, page)
    if wide:
        table = widen(table)
    q = randn(1, N, HQ, d, dtype=dtype).cuda()
    lse = torch.full((N, HQ), float("nan"), device="cuda")
    out, _ = kda.kda_attn_step_q8(q, *cache, table, i32(lens), d ** -0.5, None, lse)
    check_rows(q, ks, vs, d ** -0.5, out, lse, _weights(dtype, d))


@pytest.mark.parametrize("d", [16, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_narrow_heads(d, dtype):
    lens = [100, 1, 0, 333]
    ks, vs, cache, table = paged_q8(d, lens, 2, d, 16)
    q = randn(1, 4, 6, d, dtype=dtype).cuda()
    out, _ = kda.kda_attn_step_q8(q, *cache, table, i32(lens), 0.4)
    check_rows(q, ks, vs, 0.4, out, None, FP32)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_step_strided_q_f32_out_and_negative_lengths(dtype, d):
    lens = [200, 0, 31]
    ks, vs, cache, table = paged_q8(3, lens, 2, d, 32)
    q = randn(1, 3, 10, d, dtype=dtype).cuda()[:, 2:8]
    out, _ = kda.kda_attn_step_q8(q, *cache, table, i32([200, -4, 31]), 0.1, out_f32=True)
    assert out.dtype == torch.float32
    check_rows(q, ks, vs, 0.1, out, None, _weights(dtype, d))
    assert kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("codes", [-127, 127, "each channel its own"])
def test_step_every_code(dtype, d, codes):
    """Keys and values that hold every code in every channel, and rows of one."""
    n, page = 255, 32
    need = 8
    table = torch.arange(need, dtype=torch.int32)[None].flip(1).contiguous()
    if codes in (-127, 127):
        c = torch.full((n, 1, d), codes, dtype=torch.int8)
    else:
        c = ((torch.arange(n)[:, None] + 3 * torch.arange(d)[None]) % 255 - 127).to(torch.int8)[:, None]
    f = 0.001 * (1 + torch.arange(n) % 7).float()[:, None]
    kc = put(torch.zeros(need, 1, page, d, dtype=torch.int8), c, table, [0], [n])
    fs = put(torch.full((need, 1, page), float("nan")), f, table, [0], [n])
    rows = c.double() * f.double()[..., None]
    q = randn(1, 1, 3, d, dtype=dtype).cuda()
    lse = torch.empty(1, 3, device="cuda")
    out, _ = kda.kda_attn_step_q8(q, kc.cuda(), kc.cuda(), fs.cuda(), fs.cuda(), table.cuda(),
                                  i32([n]), 0.3, None, lse)
    check_rows(q, [rows], [rows], 0.3, out, lse, _weights(dtype, d))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 16)])
@pytest.mark.parametrize("size", [2.0 ** -100, 1e-20, 1e15])
def test_step_scales_far_from_one(dtype, d, size):
    """Values of any size, and keys whose scales differ by 2^60 from row to row."""
    n, page = 70, 16
    ks, vs, (kc, vc, kf, vf), table = paged_q8(4, [n], 2, d, page)
    vf *= size
    kf[:, :, 1::2] *= 2.0 ** -60
    ks[0][1::2] *= 2.0 ** -60
    q = randn(1, 1, 4, d, dtype=dtype).cuda()
    out, _ = kda.kda_attn_step_q8(q, kc, vc, kf, vf, table, i32([n]), 0.2, out_f32=True)
    # (2^-23: the scales' product with size; a weight times a scale may lie among the
    # numbers below 2^-126, whose steps in bf16, 2^-133, times the codes are 2^-24 of
    # values of 2^-100 to a key)
    check_rows(q, ks, vs, 0.2, out.double() / size, None,
               _weights(dtype, d) + 2.0 ** -23 + n * 2.0 ** -24)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("HQ", [2, 8])
@pytest.mark.parametrize("below", [8.0, 17.0, 26.0])
def test_step_small_weights_beside_a_large_one(d, HQ, below):
    """One key takes nearly all the weight and has a value of zero; the result is
    what the others, e^-below of it each, leave.  Weights down to 2^-28 of the
    largest keep 2^-15; below (26 / ln 2 = 37.5 powers of two) they are off by
    2^-43 of it (and at most 4 query heads; with more, by 2^-15 of their own).
    Scores of tens: the roundings of their exponentials are check()'s."""
    n, page, HKV = 300, 16, 1
    g = torch.Generator().manual_seed(d)
    q = torch.ones(1, HQ, d, dtype=torch.bfloat16)
    # scores: token 0 has below more than the others'
    k = torch.randint(-3, 4, (n, HKV, d), generator=g, dtype=torch.int8)
    k[0] = 100
    f = torch.full((n, HKV), below / (100 * d))
    f[1:] *= 0.01
    v = torch.randint(1, 128, (n, HKV, d), generator=g, dtype=torch.int8)
    fv = 0.01 * (1 + torch.rand(n, HKV, generator=g))
    fv[0] = 0.0
    need = -(-n // page)
    t = torch.arange(need, dtype=torch.int32)[None]
    put = lambda shape, x, dt: _put_rows(torch.zeros(shape, dtype=dt), x, t, n)
    cache = (put((need, HKV, page, d), k, torch.int8), put((need, HKV, page, d), v, torch.int8),
             put((need, HKV, page), f, torch.float32), put((need, HKV, page), fv, torch.float32))
    rows = [k.double() * f.double()[..., None], v.double() * fv.double()[..., None]]
    for table_ in (t, widen(t)):
        out, _ = kda.kda_attn_step_q8(q.cuda(), *(x.cuda() for x in cache), table_.cuda(), i32([n]),
                                      1.0, out_f32=True)
        # the small weights' 2^-43 of the largest, over what there is of them
        small = n * 2.0 ** -43 * 2 * 127 * 0.02 / (n * math.exp(-below) * 0.5)
        check_rows(q, [rows[0]], [rows[1]], 1.0, out, None, TWO_PARTS + small)


def _put_rows(cache, rows, table, n):
    return put(cache, rows, table, [0], [n])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_step_rows_that_no_code_stands_for(dtype, d):
    """A NaN scale makes NaN of what attends to it, and of nothing else; a scale
    of 0 is a row of zeros."""
    lens = [100, 100, 90]
    ks, vs, (kc, vc, kf, vf), table = paged_q8(5, lens, 1, d, 32)
    kf[int(table[0, 1]), 0, 3] = float("nan")
    vf[int(table[2, 0]), 0, 30] = 0.0
    kf[int(table[2, 2]), 0, 7] = 0.0
    vs[2][30] = 0.0
    ks[2][71] = 0.0
    q = randn(1, 3, 2, d, dtype=dtype).cuda()
    for table_ in (table, widen(table)):
        out, _ = kda.kda_attn_step_q8(q, kc, vc, kf, vf, table_, i32(lens), 0.1)
        assert out[0].isnan().all()
        check_rows(q[1:], ks[1:], vs[1:], 0.1, out[1:], None, _weights(dtype, d))


@pytest.mark.parametrize("dtype,HQ", [("bf16", 2), ("bf16", 9), ("f32", 2)])
def test_step_thousands_of_sequences(dtype, HQ):
    """Short sequences and empty ones by the thousand, in a table of 1024 tokens."""
    N, d = 2500, 64
    lens = [(7 * i) % 40 if i % 5 else 0 for i in range(N)]
    ks, vs, cache, table = paged_q8(17, lens, 1, d, 16)
    q = randn(2, N, HQ, d, dtype=dtype).cuda()
    lse = torch.full((N, HQ), float("nan"), device="cuda")
    out, _ = kda.kda_attn_step_q8(q, *cache, widen(table, 64), i32(lens), d ** -0.5, None, lse)
    check_rows(q, ks, vs, d ** -0.5, out, lse, _weights(dtype, d))


@pytest.mark.parametrize("HQ,HKV", [(2, 2), (4, 2), (3, 1), (9, 1)])
@pytest.mark.parametrize("dtype,d", [("f32", 16), ("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 16),
                                     ("bf16", 32)])
@pytest.mark.parametrize("lens", [[3000, 0, 17], [700, 1200, 64, 1, 0, 90]])
@pytest.mark.parametrize("wide", [False, True])
def test_step_every_number_of_rows(HQ, HKV, dtype, d, lens, wide):
    """Long sequences, shared by CTAs, with every number of rows to a CTA."""
    ks, vs, cache, table = paged_q8(d + HQ, lens, HKV, d, 64)
    q = randn(2, len(lens), HQ, d, dtype=dtype).cuda()
    lse = torch.full((len(lens), HQ), float("nan"), device="cuda")
    out, _ = kda.kda_attn_step_q8(q, *cache, widen(table) if wide else table, i32(lens), d ** -0.5,
                                  None, lse)
    check_rows(q, ks, vs, d ** -0.5, out, lse, _weights(dtype, d))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("HQ", [2, 8])
@pytest.mark.parametrize("wide", [False, True])
def test_step_scales_below_zero(dtype, d, HQ, wide):
    """A scale may have either sign."""
    lens = [333, 40]
    ks, vs, (kc, vc, kf, vf), table = paged_q8(15, lens, 1, d, 32)
    kf.neg_()
    vf[1:].neg_()
    for s, n in enumerate(lens):
        ks[s].neg_()
        for j in range((n + 31) // 32):
            if int(table[s, j]) > 0:
                vs[s][j * 32:(j + 1) * 32].neg_()
    q = randn(1, 2, HQ, d, dtype=dtype).cuda()
    out, _ = kda.kda_attn_step_q8(q, kc, vc, kf, vf, widen(table) if wide else table, i32(lens), 0.1)
    check_rows(q, ks, vs, 0.1, out, None, _weights(dtype, d))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("wide", [False, True])
def test_step_queries_that_are_no_numbers(dtype, d, value, wide):
    """An infinity or a NaN in a head's query is that head's alone: no code stands
    for an infinity, so that scores of +inf among others leave NaN."""
    lens = [200, 50]
    ks, vs, cache, table = paged_q8(16, lens, 1, d, 16)
    q = randn(1, 2, 3, d, dtype=dtype)
    q[0, 1, d // 2] = value
    out, _ = kda.kda_attn_step_q8(q.cuda(), *cache, widen(table) if wide else table, i32(lens), 0.1)
    assert out[0, 1].isnan().all()
    for s, h in ((0, 0), (0, 2), (1, 0), (1, 1), (1, 2)):
        one = (slice(s, s + 1), slice(h, h + 1))
        check_rows(q[one], ks[s:s + 1], vs[s:s + 1], 0.1, out[one], None, _weights(dtype, d))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16)])
@pytest.mark.parametrize("left", [65, 63, 32])
def test_step_lengths_up_to_2_31(dtype, d, left):
    """A table of 2^31 - 32 tokens whose entries name one page of 32 over and
    over, beside a sequence of 70 tokens.

    Bound: at most four additions to an accumulator per tile of 64 tokens, with a
    whole step of fp32 (2^-23) each; a CTA, or a warp, has its share of the tiles
    (plus the joins', far fewer than a tenth).  The output's own rounding is 2^-8."""
    page, top = 32, 1 << 31
    width, lens = top // page - 1, [top - left, 70]
    g = torch.Generator().manual_seed(d)
    codes = torch.randint(-127, 128, (2, 1, 1, page, d), generator=g, dtype=torch.int8)
    codes[1] = codes[1] // 4 + 90    # (means that are not near zero)
    scales = (0.5 + torch.rand(2, 1, 1, page, generator=g)) / 127
    k, v = (codes[i, 0, 0].double() * scales[i, 0, 0].double()[:, None] for i in (0, 1))
    q = randn(3, 2, 1, d, dtype=dtype)
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    lse = torch.full((2, 1), float("nan"), device="cuda")
    scale = d ** -0.5
    out, _ = kda.kda_attn_step_q8(q.cuda(), *codes.cuda(), *scales.cuda(), table, i32(lens), scale,
                                  None, lse)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for s, n in enumerate(lens):
        count = n // page + (torch.arange(page) < n % page)
        z = scale * (k @ q[s, 0].double())
        w = count * torch.exp(z - z.max())
        want, size = (w @ v) / w.sum(), (w @ v.abs()) / w.sum()
        rel = 4.4 * (n / 64 / sms + 1) * 2.0 ** -23 + 1e-4
        assert abs(lse[s, 0].item() - (z.max() + w.sum().log()).item()) <= rel + 1e-5
        assert ((out[s, 0].cpu().double() - want).abs() <= (2 * rel + 2.0 ** -8) * size).all()
    assert kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_step_bad_places(dtype, d):
    """Lengths past the table and pages that do not exist are left out and reported."""
    lens = [96, 96]
    ks, vs, cache, table = paged_q8(5, lens, 2, d, 32)
    q = randn(1, 2, 4, d, dtype=dtype).cuda()
    good = table[1, 1].item()
    for bad in (-1, cache[0].shape[0]):
        table[1, 1] = bad
        out, _ = kda.kda_attn_step_q8(q, *cache, table, i32(lens), 0.1)
        assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
        left = [torch.cat((x[1][:32], x[1][64:])) for x in (ks, vs)]
        check_rows(q, [ks[0], left[0]], [vs[0], left[1]], 0.1, out, None, _weights(dtype, d))
    table[1, 1] = good
    table = table[:, :3].contiguous()
    out, _ = kda.kda_attn_step_q8(q, *cache, table, i32([96, 1 << 30]), 0.1)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    check_rows(q, ks, vs, 0.1, out, None, _weights(dtype, d))
    empty = [x[:0] for x in cache]
    out, _ = kda.kda_attn_step_q8(q, *empty, table[:, :0].contiguous(), i32([0, 0]), 0.1)
    assert (out == 0).all() and kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_and_append_past_32_bits(dtype):
    """A cache of more than 2^31 codes, the sequence in its last pages."""
    HKV, d, page, n = 8, 128, 64, 1000
    pages = (1 << 31) // (HKV * page * d) + 40
    ks, vs, small, table = paged_q8(6, [n], HKV, d, page)
    m = small[0].shape[0]
    cache = []
    for x in small:
        big = torch.zeros(pages, *x.shape[1:], dtype=x.dtype, device="cuda")
        big[pages - m:] = x
        cache.append(big)
    q = randn(1, 1, 16, d, dtype=dtype).cuda()
    shifted = torch.where(table >= 0, table + (pages - m), table)
    out, _ = kda.kda_attn_step_q8(q, *cache, shifted, i32([n]), 0.1)
    check_rows(q, ks, vs, 0.1, out, None, _weights(dtype, d))
    new = randn(9, 1, HKV, d, dtype=dtype)
    kda.kda_cache_append_q8(new.cuda(), new.cuda(), *cache, shifted, i32([n - 1]))
    b, r = int(shifted[0, (n - 1) // page]), (n - 1) % page
    codes, scales = encode(new)
    for i in range(2):
        assert torch.equal(cache[i][b, :, r].cpu(), codes[0].to(torch.int8))
        assert torch.equal(cache[2 + i][b, :, r].cpu(), scales[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wide", [False, True])
def test_step_streams_graphs_and_workspace(dtype, wide):
    """Two calls at once, two captured graphs replayed with other lengths, and a
    caller's workspace all give the bits of a plain call."""
    lens, HQ, HKV, d, page = [3000, 17, 900, 0, 64], 8, 2, 128, 16
    ks, vs, cache, table = paged_q8(7, lens, HKV, d, page)
    if wide:
        table = widen(table)
    q = [randn(i, 5, HQ, d, dtype=dtype).cuda() for i in (1, 2)]
    l1, l2 = i32(lens), i32([100, 0, 900, 0, 3])
    step = lambda i, l, **kw: kda.kda_attn_step_q8(q[i], *cache, table, l, 0.1, **kw)[0]
    want = {(i, j): step(i, l) for i in (0, 1) for j, l in ((1, l1), (2, l2))}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [step(i, l1, stream=streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0, 1]) and torch.equal(got[1], want[1, 1])
    cur = l1.clone()
    outs, graphs = [torch.empty_like(x) for x in q], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(i, cur, out=outs[i])
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
    code = kda.KDA_DTYPE_BF16 if dtype == "bf16" else kda.KDA_DTYPE_F32
    shape = kda.make_attn_shape(5, 5, HQ, HKV, d, code)
    c = kda.kdaPagedCacheQ8_t(*(x.data_ptr() for x in (*cache, table)), cache[0].shape[0], page,
                              table.shape[1])
    need = kda.kda_attn_step_q8_workspace_size(c, shape)
    assert (need > 0) == wide
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    assert torch.equal(step(0, l1, workspace=ws), want[0, 1])
    if wide:
        with pytest.raises(kda.KdaError):
            step(0, l1, workspace=ws[:1024])
    # the library's own scratch (C entry without a workspace)
    from kimi_delta_attention_chunkwise_gb300 import binding
    out2 = torch.empty_like(want[0, 1])
    rc = binding.load().kda_attn_step_q8(q[0].data_ptr(), ctypes.byref(c), l1.data_ptr(), 0.1,
                                         out2.data_ptr(), None, ctypes.byref(shape),
                                         torch.cuda.current_stream().cuda_stream)
    assert rc == kda.KDA_SUCCESS and torch.equal(out2, want[0, 1])


@pytest.mark.parametrize("dtype,d,inter", [("bf16", 128, False), ("bf16", 64, True),
                                           ("f32", 64, False)])
def test_prompt_append_and_steps_together(dtype, d, inter):
    """A served batch over a cache of codes: prompts through append and prompt
    attention over what the codes stand for, then a few decoded tokens through
    append and step; every output against attention in 64 bits over the codes."""
    HQ, HKV, page, steps = 6, 2, 16, 3
    lens = [40, 1, 100]
    N, T = 3, 141
    rope = rope_table(256, d)
    need = [(n + steps + page - 1) // page for n in lens]
    table, pages = tables(need, max(need))
    kc = torch.full((pages, HKV, page, d), -128, dtype=torch.int8, device="cuda")
    kf = torch.full((pages, HKV, page), float("nan"), device="cuda")
    cache, table = (kc, kc.clone(), kf, kf.clone()), table.cuda()
    q, k, v = (randn(i, T, h, d, dtype=dtype) for i, h in ((1, HQ), (2, HKV), (3, HKV)))
    pos = torch.cat([torch.arange(n) for n in lens])
    ks, vs = torch.empty_like(k, device="cuda"), torch.empty_like(v, device="cuda")
    held, cu = i32([0, 0, 0]), offsets(lens)
    q_out, _ = kda.kda_cache_append_q8(k.cuda(), v.cuda(), *cache, table, held, cu, q=q.cuda(),
                                       k_stored=ks, v_stored=vs, rope=rope.cuda(),
                                       rope_interleaved=inter)
    out, _ = kda.kda_attn_fwd(q_out, ks, vs, d ** -0.5, cu)
    rq = rotate(q, pos, rope, inter)
    last = torch.tensor(lens).cumsum(0) - 1
    # rows of codes as the sequences hold them
    seqs = [[], []]
    a = 0
    for n in lens:
        for i, x in enumerate((rotate(k.float(), pos, rope, inter), v.float())):
            c, f = encode(x[a:a + n])
            seqs[i].append(c.double() * f.double()[..., None])
        a += n
    # a prompt's last token sees what a step would (the prompt reads the codes' values
    # rounded to its type: half a step of each, in the scores and in the values)
    o = out[last.cuda()].cpu().double()
    step_out, _ = kda.kda_attn_step_q8(q_out[last.cuda()].contiguous(), *cache, table, i32(lens),
                                       d ** -0.5, out_f32=True)
    check_rows(rq[last], *seqs, d ** -0.5, step_out, None, _weights(dtype, d))
    half = torch.finfo(DT[dtype]).eps / 2
    for s in range(N):
        big = seqs[1][s].abs().max()
        z = (rq[last[s]].double().abs().sum(dim=-1).max() * seqs[0][s].abs().max()) * d ** -0.5
        tol = big * (math.expm1(2 * half * z) + 3 * half + (ONE_PART if mma(dtype, d) else 0) + 1e-4)
        assert ((o[s] - step_out[s].cpu().double()).abs() <= tol).all()
    held = i32(lens)
    for i in range(steps):
        q, k, v = (randn(10 * i + j, N, h, d, dtype=dtype) for j, h in ((4, HQ), (5, HKV), (6, HKV)))
        pos = torch.tensor(lens) + i
        q_out, _ = kda.kda_cache_append_q8(k.cuda(), v.cuda(), *cache, table, held, q=q.cuda(),
                                           rope=rope.cuda(), rope_interleaved=inter)
        held += 1
        out, _ = kda.kda_attn_step_q8(q_out, *cache, table, held, d ** -0.5)
        for j, x in enumerate((rotate(k.float(), pos, rope, inter), v.float())):
            c, f = encode(x)
            x = c.double() * f.double()[..., None]
            seqs[j] = [torch.cat((y, x[s:s + 1])) for s, y in enumerate(seqs[j])]
        check_rows(rotate(q, pos, rope, inter), *seqs, d ** -0.5, out, None, _weights(dtype, d))
