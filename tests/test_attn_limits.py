"""The full-attention layer at the ends of the sizes it accepts."""
import ctypes

import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from attn_testutil import U, check, reference, rope_table, rotate, tables

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOP = 1 << 31


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()
    torch.cuda.empty_cache()


def test_more_than_2_30_sequences_are_refused():
    """The kernels find a token's sequence, and the sequences' tiles, with sums
    of two sequence indices in 32 bits."""
    from kimi_delta_attention_chunkwise_gb300 import binding, build
    build.build()
    lib, fake, other = binding.load(), 0x10000, 0x20000   # never dereferenced
    cache = kda.kdaPagedCache_t(fake, fake, fake, 4, 16, 2)
    n = ctypes.c_size_t(0)
    for N, T, code in (((1 << 30) + 1, 9, kda.KDA_ERR_UNSUPPORTED),
                       (TOP - 1, 9, kda.KDA_ERR_UNSUPPORTED), (1 << 30, 0, kda.KDA_SUCCESS)):
        s = ctypes.byref(kda.make_attn_shape(N, T, 1, 1, 64, kda.KDA_DTYPE_BF16))
        assert lib.kda_attn_fwd(fake, fake, fake, 0.1, fake, other, None, s, None) == code
        assert lib.kda_cache_append(None, fake, fake, fake, fake, None, None, None,
                                    ctypes.byref(cache), s, None) == code
    s = ctypes.byref(kda.make_attn_shape((1 << 30) + 1, (1 << 30) + 1, 1, 1, 64, kda.KDA_DTYPE_BF16))
    assert lib.kda_attn_step_workspace_size(ctypes.byref(cache), s, ctypes.byref(n)) == \
        kda.KDA_ERR_UNSUPPORTED


def test_grids_past_2_31_blocks_are_refused():
    """One more tile of rows than a grid holds, whichever engine takes it."""
    from kimi_delta_attention_chunkwise_gb300 import binding, build
    build.build()
    lib, fake, other = binding.load(), 0x10000, 0x20000   # never dereferenced
    for dtype in (kda.KDA_DTYPE_F32, kda.KDA_DTYPE_BF16):
        for N, T, H in (((1 << 30) - 1, 40, 2), ((1 << 24) - 1, 1 << 24, 127)):
            assert max(N * H, T * H) < TOP <= T * H // 16 + N * H
            s = ctypes.byref(kda.make_attn_shape(N, T, H, H, 64, dtype))
            assert lib.kda_attn_fwd(fake, fake, fake, 0.1, fake, other, None, s, None) == \
                kda.KDA_ERR_UNSUPPORTED


def test_sizes_past_32_bits_are_refused_not_cut_off():
    """2^32 + 5 of anything would arrive as 5."""
    from kimi_delta_attention_chunkwise_gb300 import binding
    many = (1 << 32) + 5
    for i in range(5):
        sizes = [1, 1, 1, 1, 64]
        sizes[i] = many
        with pytest.raises(ValueError, match="2\\^31"):
            kda.make_attn_shape(*sizes, kda.KDA_DTYPE_BF16)
        with pytest.raises(ValueError, match="2\\^31"):
            binding._shape_ref(*sizes, kda.KDA_DTYPE_BF16, 0, 0, 0, 0, 0)
    meta = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="meta")   # device -1
    for pages, width in ((4, many), (many, 4)):
        cache = meta(pages, 1, 16, 16)
        with pytest.raises(ValueError, match="2\\^31"):
            binding._paged_cache(cache, cache, meta(1, width, dt=torch.int32), -1, torch.bfloat16,
                                 torch.int32, 1, 16)


def _randn(seed, *shape, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 16)])
@pytest.mark.parametrize("length", [TOP - 65, TOP - 63, TOP - 32])
def test_step_lengths_up_to_2_31(gpu, dtype, d, length):
    """A table of 2^31 - 32 tokens whose entries name one page of 32 over and
    over, beside a sequence of 70 tokens.  A row's weight is its number of
    occurrences times its exponential.

    Bound: the accumulators of the sums and of the outputs take at most two
    additions per tile of 64 tokens, with a whole step of fp32 (2^-23) each, and
    a CTA has its share of the tiles (plus the joins', far fewer than a tenth).
    Weights of bf16 values are rounded by 2^-8 at most, and so is the output."""
    page, width = 32, TOP // 32 - 1
    k, v = (_randn(i, 1, 1, page, d, dtype=dtype) for i in (1, 2))
    v += 1   # (means that are not near zero)
    q = _randn(3, 2, 1, d, dtype=dtype)
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    lens = [length, 70]
    lse = torch.full((2, 1), float("nan"), device="cuda")
    out = torch.full((2, 1, d), float("nan"), dtype=DT[dtype], device="cuda")
    scale = d ** -0.5
    kda.kda_attn_step(q.cuda(), k.cuda(), v.cuda(), table,
                      torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, out, lse)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    additions = 2.2 * (length / 64 / sms + 1)
    for s, n in enumerate(lens):
        count = n // page + (torch.arange(page) < n % page)
        z = scale * (k[0, 0].double() @ q[s, 0].double())
        w = count * torch.exp(z - z.max())
        want = (w @ v[0, 0].double()) / w.sum()
        size = (w @ v[0, 0].double().abs()) / w.sum()
        rel = additions * 2.0 ** -23 + 1e-4
        assert abs(lse[s, 0].item() - (z.max() + w.sum().log()).item()) <= rel + 1e-5
        assert ((out[s, 0].cpu().double() - want).abs() <= (2 * rel + 2.0 ** -7) * size).all()
    # the last row of the table, too, takes a new token
    if length == TOP - 32:
        kc, vc = torch.zeros(1, 1, page, d, dtype=DT[dtype], device="cuda"), v.cuda()
        new = _randn(4, 2, 1, d, dtype=dtype).cuda()
        kda.kda_cache_append(new, new, kc, vc, table,
                             torch.tensor([length - 1, 3], dtype=torch.int32, device="cuda"))
        assert torch.equal(kc[0, 0, 31], new[0, 0]) and torch.equal(kc[0, 0, 3], new[1, 0])


@pytest.mark.gpu
def test_append_of_2_31_less_one_tokens(gpu):
    """The largest token count: all but the first and the last few rows lie
    outside every sequence.  (64 GB of keys, which are the values too.)"""
    T, d, page = TOP - 1, 16, 16
    if torch.cuda.mem_get_info()[0] < 3 * T * d:
        pytest.skip("not enough free memory")
    x = torch.empty(T, 1, d, dtype=torch.bfloat16, device="cuda")
    rows = _randn(1, 6, 1, d, dtype="bf16").cuda()
    x[:3], x[T - 3:] = rows[:3], rows[3:]
    kc = torch.zeros(2, 1, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    for cu, page_of in (((0, 3, 3), 0), ((T - 3, T - 3, T), 1)):
        want = torch.zeros_like(kc)
        want[page_of, 0, 5:8] = rows[:3, 0] if page_of == 0 else rows[3:, 0]
        kc.zero_(), vc.zero_()
        kda.kda_cache_append(x, x, kc, vc, table, i32(5, 5), i32(*cu))
        assert torch.equal(kc, want) and torch.equal(vc, want)
    del x
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,HQ,HKV", [("bf16", 128, 8, 2), ("bf16", 64, 12, 1), ("bf16", 32, 4, 2),
                                            ("f32", 64, 6, 2), ("f32", 128, 2, 2)])
@pytest.mark.parametrize("wide", [False, True])
def test_step_scores_of_minus_infinity(gpu, dtype, d, HQ, HKV, wide):
    """Keys whose scores are -inf weigh nothing; a sequence that has no others
    gives the formula's 0 / 0 and ln 0 = -inf, as the prompt attention does.  Out
    = 0 is for sequences without keys."""
    page, pages = 64, 48
    lens = [900, 900, 900, 70, 1, 0, 900]
    dead = [900, 0, 700, 70, 1, 0, 899]     # the first so many tokens score -inf
    N = len(lens)
    q = _randn(1, N, HQ, d, dtype=dtype)
    q[..., 0] = 1
    ks, vs = ([_randn(10 * s + i, n, HKV, d, dtype=dtype) for s, n in enumerate(lens)] for i in (2, 3))
    kc, vc = (torch.zeros(N * 15, HKV, page, d, dtype=DT[dtype]) for _ in range(2))
    table = torch.full((N, 16384 if wide else 15), -1, dtype=torch.int32)
    for s, n in enumerate(lens):
        ks[s][:dead[s], :, 0] = -float("inf")
        table[s, :15] = torch.arange(15) + 15 * s
        for c, x in ((kc, ks[s]), (vc, vs[s])):
            rows = torch.zeros(15 * page, HKV, d, dtype=DT[dtype])
            rows[:n] = x
            c[15 * s:15 * s + 15] = rows.view(15, page, HKV, d).transpose(1, 2)
    lse = torch.zeros(N, HQ, device="cuda")
    out, _ = kda.kda_attn_step(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, None, lse)
    for s, n in enumerate(lens):
        if n == 0:
            assert (out[s] == 0).all() and (lse[s] == -float("inf")).all()
        elif dead[s] == n:
            assert torch.isnan(out[s]).all() and (lse[s] == -float("inf")).all()
        else:
            left = n - dead[s]
            check(out[s:s + 1], lse[s:s + 1], reference(q[s:s + 1], ks[s][dead[s]:], vs[s][dead[s]:],
                                                        0.1, left - 1), n, d, dtype == "bf16" and d >= 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,engine,d", [("bf16", "auto", 128), ("bf16", "auto", 64),
                                            ("bf16", "simt", 64), ("f32", "auto", 64)])
@pytest.mark.parametrize("lens", [[400], [130, 60] + [40] * 20])
def test_prompt_scores_of_minus_infinity(gpu, dtype, engine, d, lens):
    """The same in prompts: a sequence's first tokens see nothing but -inf."""
    HQ, HKV, T = 4, 2, sum(lens)
    q, k, v = (_randn(i, T, h, d, dtype=dtype) for i, h in ((1, HQ), (2, HKV), (3, HKV)))
    q[..., 0] = 1
    cu = [0]
    for n in lens:
        k[cu[-1]:cu[-1] + n // 2, :, 0] = -float("inf")
        cu.append(cu[-1] + n)
    lse = torch.zeros(T, HQ, device="cuda")
    out, _ = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), 0.1,
                              torch.tensor(cu, dtype=torch.int32, device="cuda"), None, lse,
                              engine=engine)
    for a, n in zip(cu, lens):
        m = n // 2
        assert torch.isnan(out[a:a + m]).all() and (lse[a:a + m] == -float("inf")).all()
        b, e = a + m, a + n
        check(out[b:e], lse[b:e], reference(q[b:e], k[b:e], v[b:e], 0.1, 0), n, d,
              dtype == "bf16" and engine == "auto")


def _step_case(seed, lens, HQ, HKV, d, dtype, wide):
    """q, a sequence's keys and values, caches with pages of 32 in order, table."""
    N, page, most = len(lens), 32, (max(lens) + 31) // 32
    q = _randn(seed, N, HQ, d, dtype=dtype)
    ks, vs = ([_randn(seed + 10 * s + i, n, HKV, d, dtype=dtype) for s, n in enumerate(lens)]
              for i in (1, 2))
    table = torch.full((N, 16384 if wide else most), -1, dtype=torch.int32)
    for s in range(N):
        table[s, :most] = torch.arange(most) + most * s

    def cache(rows):
        c = torch.zeros(N * most, HKV, page, d, dtype=DT[dtype])
        for s, n in enumerate(lens):
            x = torch.zeros(most * page, HKV, d, dtype=DT[dtype])
            x[:n] = rows[s]
            c[most * s:most * (s + 1)] = x.view(most, page, HKV, d).transpose(1, 2)
        return c.cuda()

    return q, ks, vs, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


GROUPS = [(1, 1, 64), (3, 1, 128), (8, 2, 128), (8, 2, 64), (5, 1, 128), (16, 2, 64), (12, 1, 128),
          (32, 2, 64), (40, 1, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("HQ,HKV,d", GROUPS)
@pytest.mark.parametrize("wide", [False, True])
def test_step_keeps_its_weights_bits(gpu, HQ, HKV, d, wide):
    """bf16 with float32 results: the weights' two parts leave 2^-15 of them out
    (2^-7 cut off, then rounded by 2^-8) and may add 2^-20, not the 2^-8 of one
    rounded part; a key's two products are two additions."""
    lens = [513, 64, 1, 2000]
    q, ks, vs, cache, table, n32 = _step_case(HQ + d, lens, HQ, HKV, d, "bf16", wide)
    out, _ = kda.kda_attn_step(q.cuda(), cache(ks), cache(vs), table, n32, d ** -0.5, out_f32=True)
    for s, n in enumerate(lens):
        o, A, _, z1 = reference(q[s:s + 1], ks[s], vs[s], d ** -0.5, n - 1)
        rel = 2 * ((d + 8) * U * z1 + 4 * U * (2 * z1 + 2)) + 3 * (n + 16) * U + 2.0 ** -15 + 2.0 ** -20
        assert ((out[s:s + 1].cpu().double() - o).abs() <= rel[..., None] * A + U * o.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("HQ,HKV,d,dtype", [(*g, "bf16") for g in GROUPS] +
                         [(4, 2, 32, "bf16"), (6, 2, 64, "f32"), (8, 1, 128, "f32")])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_step_infinite_values(gpu, HQ, HKV, d, dtype, wide, value):
    """A non-finite value shows in its channel, however small its weight (down
    to the smallest normal number), and in no other channel."""
    lens = [300, 90]
    q, ks, vs, cache, table, n32 = _step_case(HQ, lens, HQ, HKV, d, dtype, wide)
    q[..., 0], q[..., 1:] = 1, 0        # scores: the keys' first channel
    for gap in (0.0, 1.0, 30.0, 100.0, 124.0):
        for s in (0, 1):
            ks[s][..., 0] = 0
            ks[s][77, :, 0] = -gap      # 2^-gap of the largest weight
            vs[s][77, :, 5] = value
        out, _ = kda.kda_attn_step(q.cuda(), cache(ks), cache(vs), table, n32, 0.6931471805599453)
        seen = out[..., 5].float()
        assert (torch.isnan(seen) if value != value else seen == value).all()
        rest = torch.cat((out[..., :5], out[..., 6:]), dim=-1)
        assert torch.isfinite(rest).all()


@pytest.mark.gpu
@pytest.mark.parametrize("HQ,HKV,d", [(4, 2, 128), (8, 2, 64), (3, 3, 64), (7, 1, 128)])
@pytest.mark.parametrize("before", [0, 77])
def test_long_prompts_on_the_tensor_cores(gpu, HQ, HKV, d, before):
    """Rows from a prompt's start, its middle and its end, and a short prompt in
    front of it."""
    n = 9001
    q, k, v = (_randn(i + d, before + n, h, d, dtype="bf16") for i, h in ((1, HQ), (2, HKV), (3, HKV)))
    cu = torch.tensor(([0] if before else []) + [before, before + n], dtype=torch.int32).cuda()
    lse = torch.full((before + n, HQ), float("nan"), device="cuda")
    out, _ = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), d ** -0.5, cu, None, lse, engine="tensor")
    assert not torch.isnan(out).any() and not torch.isnan(lse).any()
    for a, b in ((0, 150), (2490, 2640), (5000, 5130), (n - 300, n)):
        rows = slice(before + a, before + b)
        check(out[rows], lse[rows],
              reference(q[rows], k[before:before + b], v[before:before + b], d ** -0.5, a), b, d, True)
    if before:
        check(out[:before], lse[:before], reference(q[:before], k[:before], v[:before], d ** -0.5, 0),
              before, d, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,inter", [(64, 32, True), (128, 128, True), (32, 32, True), (16, 16, False),
                                         (128, 48, False)])
def test_append_of_more_tokens_than_ctas_of_one_take(gpu, dtype, d, rot, inter):
    """Past 1024 tokens a CTA takes two; both pairings, parts of a head, and
    rows outside every sequence."""
    HQ, HKV, page, lens, held, T = 6, 2, 32, [1100, 0, 403], [500, 7, 31], 1506
    q, k, v = (_randn(i + d, T, h, d, dtype=dtype) for i, h in ((1, HQ), (2, HKV), (3, HKV)))
    need = [(h + n + page - 1) // page for h, n in zip(held, lens)]
    table, pages = tables(need, max(need))
    rope = rope_table(1700, rot)
    pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, lens)])
    want_q, want_k = (torch.full_like(x, 3) for x in (q, k))
    want_q[1:1504], want_k[1:1504] = (rotate(x[1:1504], pos, rope, inter) for x in (q, k))
    kc, vc = (torch.zeros(pages, HKV, page, d, dtype=DT[dtype]) for _ in range(2))
    gk, gv = kc.cuda(), vc.cuda()
    t = 1
    for s, n in enumerate(lens):
        for p in range(held[s], held[s] + n):
            b = int(table[s, p // page])
            kc[b, :, p % page], vc[b, :, p % page] = want_k[t], v[t]
            t += 1
    q_out, k_out = (torch.full_like(x, 3, device="cuda") for x in (q, k))
    kda.kda_cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(),
                         torch.tensor(held, dtype=torch.int32).cuda(),
                         torch.tensor([1, 1101, 1101, 1504], dtype=torch.int32).cuda(), q=q.cuda(),
                         q_out=q_out, k_out=k_out, rope=rope.cuda(), rope_interleaved=inter)
    assert torch.equal(q_out.cpu(), want_q) and torch.equal(k_out.cpu(), want_k)
    assert torch.equal(gk.cpu(), kc) and torch.equal(gv.cpu(), vc)
