"""Prompt attention on the GPU against the definition in 64 bits."""
import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from attn_testutil import check, reference

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()


def _qkv(seed, T, HQ, HKV, d, dtype):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, d, generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV, HKV)]


def _cu(lens, start=0):
    c = [start]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _tensor(dtype, d, engine):
    return engine != "simt" and dtype == "bf16" and d in (64, 128)


def _check_packed(q, k, v, scale, lens, out, lse, weights_bf16, start=0):
    a = start
    for n in lens:
        if n:
            ref = reference(q[a:a + n], k[a:a + n], v[a:a + n], scale, 0)
            check(out[a:a + n], None if lse is None else lse[a:a + n], ref, n, q.shape[2],
                  weights_bf16)
        a += n


CASES = [
    # lens, HQ, HKV, d
    ([1], 1, 1, 64), ([2, 1, 3], 4, 2, 128), ([127, 128, 129], 2, 2, 64), ([0, 5, 0, 64, 0], 6, 2, 128),
    ([255, 257], 3, 1, 128), ([300], 5, 1, 64), ([190, 65], 14, 2, 128), ([513], 8, 8, 128),
    ([33, 400], 16, 1, 64), ([70], 48, 1, 128), ([40, 7], 128, 1, 64), ([900], 4, 2, 128),
    ([1] * 70, 8, 2, 64), ([1300, 5], 2, 1, 64),
]


@pytest.mark.parametrize("lens,HQ,HKV,d", CASES)
@pytest.mark.parametrize("dtype,engine", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_prompt(lens, HQ, HKV, d, dtype, engine):
    q, k, v = _qkv(len(lens) + HQ, sum(lens), HQ, HKV, d, dtype)
    lse = torch.full((sum(lens), HQ), float("nan"), device="cuda")
    out, got = kda.kda_attn_fwd(q, k, v, d ** -0.5, _cu(lens), None, lse, engine=engine)
    assert got is lse and out.dtype == q.dtype
    _check_packed(q, k, v, d ** -0.5, lens, out, lse, _tensor(dtype, d, engine))


@pytest.mark.parametrize("d", [16, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_narrow_heads(d, dtype):
    lens = [77, 1, 130]
    q, k, v = _qkv(3, sum(lens), 6, 3, d, dtype)
    out, none = kda.kda_attn_fwd(q, k, v, 0.3, _cu(lens))
    assert none is None
    _check_packed(q, k, v, 0.3, lens, out, None, False)


@pytest.mark.parametrize("dtype,engine,d", [("bf16", "auto", 128), ("bf16", "simt", 64), ("f32", "auto", 64)])
def test_one_sequence_without_offsets_and_f32_out(dtype, engine, d):
    q, k, v = _qkv(5, 261, 4, 2, d, dtype)
    out, _ = kda.kda_attn_fwd(q, k, v, 0.2, out_f32=True, engine=engine)
    assert out.dtype == torch.float32
    _check_packed(q, k, v, 0.2, [261], out, None, _tensor(dtype, d, engine))


@pytest.mark.parametrize("dtype,engine,d", [("bf16", "auto", 128), ("bf16", "auto", 64),
                                            ("bf16", "simt", 64), ("f32", "auto", 128)])
def test_views_of_a_fused_projection(dtype, engine, d):
    """Token strides other than contiguous, and offsets into the rows."""
    HQ, HKV, lens = 6, 2, [150, 41]
    T = sum(lens)
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, HQ + 2 * HKV + 1, d, generator=g).to(DT[dtype]).cuda()
    q, k, v = x[:, 1:1 + HQ], x[:, 1 + HQ:1 + HQ + HKV], x[:, 1 + HQ + HKV:]
    out, _ = kda.kda_attn_fwd(q, k, v, d ** -0.5, _cu(lens), engine=engine)
    _check_packed(q, k, v, d ** -0.5, lens, out, None, _tensor(dtype, d, engine))
    with pytest.raises(ValueError):
        kda.kda_attn_fwd(x[..., ::2], k, v, 0.1)


@pytest.mark.parametrize("dtype,engine,d", [("bf16", "auto", 128), ("bf16", "auto", 64),
                                            ("bf16", "simt", 128), ("f32", "auto", 64)])
def test_rows_outside_every_sequence_stay(dtype, engine, d):
    """Rows before the first and behind the last sequence are not written, and
    what they hold (NaN here) does not reach the sequences."""
    lens, start, T = [100, 29], 7, 200
    q, k, v = _qkv(11, T, 4, 2, d, dtype)
    for x in (q, k, v):
        x[:start] = float("nan")
        x[start + sum(lens):] = float("inf")
    out = torch.full((T, 4, d), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, 4), 7.0, device="cuda")
    kda.kda_attn_fwd(q, k, v, 0.1, _cu(lens, start), out, lse, engine=engine)
    end = start + sum(lens)
    assert (out[:start] == 7).all() and (out[end:] == 7).all()
    assert (lse[:start] == 7).all() and (lse[end:] == 7).all()
    _check_packed(q, k, v, 0.1, lens, out, lse, _tensor(dtype, d, engine), start)


@pytest.mark.parametrize("dtype,engine,d", [("bf16", "auto", 128), ("bf16", "auto", 64),
                                            ("bf16", "simt", 128), ("f32", "auto", 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_masked_places_do_not_reach_a_row(dtype, engine, d, value):
    """Non-finite keys and values at a later token leave every earlier row as
    it is; the neighbouring sequences too.  From the token on, a non-finite
    value shows in its channel."""
    lens, HQ, HKV = [60, 300, 60], 4, 2
    q, k, v = _qkv(13, sum(lens), HQ, HKV, d, dtype)
    bad = 60 + 170
    v[bad, 1, 3] = value
    k2 = k.clone()
    k2[bad, 0, 5] = value
    out, _ = kda.kda_attn_fwd(q, k, v, 0.1, _cu(lens), engine=engine)
    out2, _ = kda.kda_attn_fwd(q, k2, v, 0.1, _cu(lens), engine=engine)
    wb = _tensor(dtype, d, engine)
    for o, kk in ((out, k), (out2, k2)):
        ref = reference(q[60:bad], kk[60:bad], v[60:bad], 0.1, 0)
        check(o[60:bad], None, ref, bad - 60, d, wb)
        for a, n in ((0, 60), (360, 60)):
            check(o[a:a + n], None, reference(q[a:a + n], kk[a:a + n], v[a:a + n], 0.1, 0), n, d, wb)
    # heads 2, 3 read kv head 1, whose channel 3 carries the value from `bad` on
    seen = out[bad:360, 2:, 3].float()
    assert (torch.isnan(seen) if value != value else seen == value).all()
    assert torch.isfinite(out[bad:360, :2]).all()
    rest = torch.cat((out[bad:360, 2:, :3], out[bad:360, 2:, 4:]), dim=-1)
    assert torch.isfinite(rest).all()


@pytest.mark.parametrize("d", [64, 128])
def test_scores_far_apart(d):
    """Scores of +-hundreds: the running maximum moves by more than fp32's
    exponent range within a row."""
    q, k, v = _qkv(17, 400, 2, 1, d, "bf16")
    k = (k * torch.linspace(0.1, 6, 400, device="cuda")[torch.randperm(400, generator=torch.Generator().manual_seed(1))][:, None, None]).bfloat16()
    out, _ = kda.kda_attn_fwd(q, k, v, 2.0)
    _check_packed(q, k, v, 2.0, [400], out, None, True)
    out, _ = kda.kda_attn_fwd(q, k, v, 2.0, engine="simt")
    _check_packed(q, k, v, 2.0, [400], out, None, False)


@pytest.mark.parametrize("d", [64, 128])
def test_equal_scores_and_tiny_scale(d):
    """scale so small that every weight is equal: the mean of the values."""
    q, k, v = _qkv(18, 300, 2, 2, d, "bf16")
    out, _ = kda.kda_attn_fwd(q, k, v, 1e-30)
    _check_packed(q, k, v, 1e-30, [300], out, None, True)


def test_more_sequences_than_a_warp_and_garbage_offsets():
    lens = [3, 0, 11, 1] * 40
    q, k, v = _qkv(19, sum(lens), 2, 1, 64, "bf16")
    out, _ = kda.kda_attn_fwd(q, k, v, 0.1, _cu(lens))
    _check_packed(q, k, v, 0.1, lens, out, None, True)
    # offsets outside [0, T] are clamped: whatever is computed stays in bounds
    bad = torch.tensor([-5, 1 << 30, 20, -7, 1 << 30], dtype=torch.int32, device="cuda")
    guard = torch.full((sum(lens) + 8, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    for engine in ("auto", "simt"):
        kda.kda_attn_fwd(q, k, v, 0.1, bad, guard[4:-4], engine=engine)
        torch.cuda.synchronize()
        assert (guard[:4] == 3).all() and (guard[-4:] == 3).all()


@pytest.mark.parametrize("engine", ["auto", "simt"])
def test_thousands_of_sequences(engine):
    """More sequences than one search step covers, empty ones among them: every
    row is some sequence's, and none is missed."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 6, (3000,), generator=g).tolist()
    T = sum(lens)
    q, k, v = _qkv(31, T, 2, 1, 64, "bf16")
    out = torch.full((T, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    kda.kda_attn_fwd(q, k, v, 0.1, _cu(lens), out, engine=engine)
    _check_packed(q, k, v, 0.1, lens, out, None, engine != "simt")


@pytest.mark.parametrize("engine,d", [("auto", 128), ("auto", 64), ("simt", 64)])
def test_a_rows_own_nan_stays_its_own(engine, d):
    """A NaN query makes its row NaN and no other."""
    q, k, v = _qkv(37, 300, 6, 2, d, "bf16")
    q[100, 1, 3] = float("nan")
    out, _ = kda.kda_attn_fwd(q, k, v, 0.1, engine=engine)
    assert torch.isnan(out[100, 1]).all()
    out[100, 1], q[100, 1, 3] = 0, 0
    ref = reference(q, k, v, 0.1, 0)
    keep = torch.ones(300, 6, dtype=torch.bool)
    keep[100, 1] = False
    flat = [x[keep][:, None] for x in ref]
    check(out.cpu()[keep][:, None], None, flat, 300, d, engine != "simt")


def test_nothing_to_do():
    q, k, v = _qkv(1, 0, 4, 2, 64, "bf16")
    out, _ = kda.kda_attn_fwd(q, k, v, 0.1, _cu([0, 0]))
    assert out.shape == q.shape
    q, k, v = _qkv(1, 5, 4, 2, 64, "bf16")
    out = torch.full_like(q, 3.0)
    for engine in ("auto", "simt"):
        kda.kda_attn_fwd(q, k, v, 0.1, _cu([0, 0]), out, engine=engine)
        assert (out == 3).all()


def test_offsets_past_32_bits():
    """More than 2^31 elements of q and out: the last sequences are right."""
    T, HQ, HKV, d = 140000, 128, 8, 128
    q = torch.empty(T, HQ, d, dtype=torch.bfloat16, device="cuda").normal_()
    k = torch.empty(T, HKV, d, dtype=torch.bfloat16, device="cuda").normal_()
    v = torch.empty_like(k).normal_()
    lens = [T - 30 - 100] + [30, 100]
    cu = torch.tensor([0] + list(range(100, T - 130, 100)) + [T - 130, T - 100, T],
                      dtype=torch.int32, device="cuda")
    out, _ = kda.kda_attn_fwd(q, k, v, 0.1, cu)
    for a, b in ((0, 100), (T - 130, T - 100), (T - 100, T)):
        check(out[a:b], None, reference(q[a:b], k[a:b], v[a:b], 0.1, 0), b - a, d, True)


def test_streams_and_graph_replay():
    """Two calls at once on two streams, and a captured call replayed on new
    inputs, give what calls one after another give."""
    lens, HQ, HKV, d = [200, 333, 5], 8, 2, 128
    a = _qkv(23, sum(lens), HQ, HKV, d, "bf16")
    b = _qkv(24, sum(lens), HQ, HKV, d, "bf16")
    cu = _cu(lens)
    want = [kda.kda_attn_fwd(*x, 0.1, cu)[0] for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [kda.kda_attn_fwd(*x, 0.1, cu, stream=s)[0] for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert torch.equal(w, o)
    static = [x.clone() for x in a]
    out = torch.empty_like(static[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_attn_fwd(*static, 0.1, cu, out)
    for src, w in ((b, want[1]), (a, want[0])):
        for x, y in zip(static, src):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_beside_a_kda_layer_on_another_stream():
    """A mixed stack's two kinds of layer at once: the prompt attention and the
    KDA prefill on two streams give the bits they give one after another."""
    T, H, d = 1500, 16, 128
    q, k, v = _qkv(41, T, H, 4, d, "bf16")
    x = [t / t.float().norm(dim=-1, keepdim=True) for t in _qkv(42, T, H, H, d, "bf16")[:2]]
    x = [t.bfloat16() for t in x] + [_qkv(43, T, H, H, d, "bf16")[2]]
    g = torch.Generator().manual_seed(44)
    la = (-torch.rand(T, H, d, generator=g) * 0.1).cuda()
    beta = torch.rand(T, H, generator=g).cuda()
    cu = _cu([700, 800])
    attn = lambda s=None: kda.kda_attn_fwd(q, k, v, 0.1, cu, stream=s)[0]
    mixer = lambda s=None: kda.kda_chunk_fwd(*x, la, beta, 0.1, None, cu, stream=s)[0]
    want = attn(), mixer()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        got = attn(s1), mixer(s2)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_tensor_engine_refuses_what_it_lacks():
    q, k, v = _qkv(1, 8, 2, 1, 32, "bf16")
    with pytest.raises(kda.KdaError) as e:
        kda.kda_attn_fwd(q, k, v, 0.1, engine="tensor")
    assert e.value.status == kda.KDA_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        kda.kda_attn_fwd(q.half(), k.half(), v.half(), 0.1)
    with pytest.raises(ValueError):
        kda.kda_attn_fwd(q, k[:, :0], v[:, :0], 0.1)


@pytest.mark.parametrize("HQ,HKV,d", [(8, 2, 128), (4, 2, 128), (4, 2, 64), (3, 3, 64)])
@pytest.mark.parametrize("mean", [64, 128, 512])
@pytest.mark.parametrize("over", [0, 1])
def test_both_key_tiles(HQ, HKV, d, mean, over):
    """Tiles of 64 and of 128 keys, on both sides of the lengths at which one
    gives way to the other, with a prompt much longer than the mean; and
    with infinite values in the later tokens' odd channels."""
    for lens in ([mean + over], [mean * 5 - 70 + 5 * over, 0, 0, 70, 0]):
        T = sum(lens)
        q, k, v = _qkv(mean + over, T, HQ, HKV, d, "bf16")
        lse = torch.empty(T, HQ, device="cuda")
        out, _ = kda.kda_attn_fwd(q, k, v, d ** -0.5, _cu(lens), None, lse)
        _check_packed(q, k, v, d ** -0.5, lens, out, lse, True)
        bad = v.clone()
        bad[T // 2:, :, 1::2] = float("inf")
        again, _ = kda.kda_attn_fwd(q, k, bad, d ** -0.5, _cu(lens))
        assert torch.equal(again[:T // 2], out[:T // 2])
        assert torch.equal(again[..., ::2], out[..., ::2])


@pytest.mark.parametrize("lens,HQ,HKV", [([430, 1, 390], 12, 4), ([50, 64, 1] * 70, 2, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_core_engine_with_tiles_for_every_sm(lens, HQ, HKV, dtype, d):
    """The CUDA-core engine's larger tiles: long and one-tile sequences, and
    infinite values in the later tokens' odd channels."""
    T = sum(lens)
    q, k, v = _qkv(d, T, HQ, HKV, d, dtype)
    lse = torch.empty(T, HQ, device="cuda")
    out, _ = kda.kda_attn_fwd(q, k, v, d ** -0.5, _cu(lens), None, lse, engine="simt")
    _check_packed(q, k, v, d ** -0.5, lens, out, lse, False)
    v[T // 2:, :, 1::2] = float("inf")
    again, _ = kda.kda_attn_fwd(q, k, v, d ** -0.5, _cu(lens), engine="simt")
    assert torch.equal(again[:T // 2], out[:T // 2])
    assert torch.equal(again[..., ::2], out[..., ::2])


@pytest.mark.parametrize("HQ,HKV,d", [(8, 8, 128), (8, 8, 64), (16, 4, 64)])
@pytest.mark.parametrize("longest", [300, 1400])
def test_items_of_one_and_two_row_tiles_in_turn(HQ, HKV, d, longest):
    """Ragged sequences, many items to a CTA: items with one row tile and with
    two follow one another in every order."""
    g = torch.Generator().manual_seed(longest + d)
    lens = torch.randint(1, longest, (60000 // longest,), generator=g).tolist()
    q, k, v = _qkv(longest, sum(lens), HQ, HKV, d, "bf16")
    lse = torch.empty(sum(lens), HQ, device="cuda")
    out, _ = kda.kda_attn_fwd(q, k, v, d ** -0.5, _cu(lens), None, lse)
    for _ in range(5):
        assert torch.equal(kda.kda_attn_fwd(q, k, v, d ** -0.5, _cu(lens))[0], out)
    assert kda.kda_device_status() == 0
    _check_packed(q, k, v, d ** -0.5, lens, out, lse, True)
