"""kda_attn_step_q8 keeps 2^-15 of every weight times its row's scale, however far
apart the rows' scales and weights are (against the definition in 64 bits)."""
import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from attn_testutil import reference
from cache_testutil import FP32, TWO_PARTS, check, i32, mma, put, widen

pytestmark = pytest.mark.gpu
EXACT_SUMS = -6   # (check's d: its d + 9 roundings of a score)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()


def _one_sequence(k, v, kf, vf, page=16):
    """(cache on the GPU, table, k rows, v rows in 64 bits) of codes k, v [n, 1, d]
    and scales kf, vf [n, 1]; scales of NaN behind them."""
    n, _, d = k.shape
    need = -(-n // page)
    t = torch.arange(need, dtype=torch.int32).flip(0)[None].contiguous()
    codes = [put(torch.zeros(need, 1, page, d, dtype=torch.int8), x, t, [0], [n]) for x in (k, v)]
    scales = [put(torch.full((need, 1, page), float("nan")), x, t, [0], [n]) for x in (kf, vf)]
    rows = [c.double() * f.double()[..., None] for c, f in ((k, kf), (v, vf))]
    return [x.cuda() for x in (*codes, *scales)], t, *rows


def _check(q, cache, t, k, v, dtype):
    """Short tables and wide ones take different kernels.  The queries are ones, so
    that the sums of codes are exact, and a score has three roundings at most."""
    n, d = k.shape[0], k.shape[2]
    ref = reference(q, k, v, 1.0, n - 1)
    for table in (t, widen(t)):
        lse = torch.empty(1, q.shape[1], device="cuda")
        out, _ = kda.kda_attn_step_q8(q.cuda(), *cache, table.cuda(), i32([n]), 1.0, None, lse,
                                      out_f32=True)
        check(out, lse, ref, n, EXACT_SUMS, TWO_PARTS if mma(dtype, d) else FP32)


@pytest.mark.parametrize("dtype,d,HQ", [("bf16", 128, 3), ("bf16", 64, 4), ("bf16", 128, 8),
                                        ("f32", 64, 2)])
@pytest.mark.parametrize("ratio", [40, 100])
@pytest.mark.parametrize("weight", ["none", "as much in all", "the largest"])
def test_a_row_with_a_scale_far_above_the_others(dtype, d, HQ, ratio, weight):
    """One value row's scale is 2^ratio times the others'.  Its weight leaves nothing
    of it, or as much as of one of the others, or it is everything in the even
    channels and, its codes being 0 there, nothing in the odd ones.  The result is
    the mean of what has weight: an error of 2^-15 of each product, no more.

    Scores: q of ones, keys of one code in all channels (their sum is exact) times
    the scale that makes the score; weights of e^0 for the others, e^-gap here."""
    n = 300
    g = torch.Generator().manual_seed(d + ratio)
    gap = {"none": 120.0, "as much in all": ratio * 0.6931471805599453, "the largest": 0.0}[weight]
    q = torch.ones(1, HQ, d, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    for at in (0, 100, 299):
        k = torch.zeros(n, 1, d, dtype=torch.int8)
        kf = torch.full((n, 1), 0.01)
        k[at], kf[at] = -100, gap / (100 * d)
        v = torch.randint(30, 128, (n, 1, d), generator=g, dtype=torch.int8)
        v[at, :, 1::2] = 0
        vf = (0.5 + torch.rand(n, 1, generator=g)) / 127
        vf[at] *= 2.0 ** ratio
        _check(q, *_one_sequence(k, v, kf, vf), dtype)


@pytest.mark.parametrize("dtype,d,HQ", [("bf16", 128, 2), ("bf16", 64, 4), ("bf16", 64, 8),
                                        ("f32", 64, 2)])
@pytest.mark.parametrize("below", [8.0, 26.0, 45.0, 70.0])
@pytest.mark.parametrize("zero", ["scale", "codes"])
def test_weights_far_below_the_largest(dtype, d, HQ, below, zero):
    """One key takes nearly all the weight and has a value of zero, by its scale or
    (in the odd channels) by its codes; the others' weights, e^-below of it, keep
    2^-15 of their own."""
    n = 300
    g = torch.Generator().manual_seed(d)
    q = torch.ones(1, HQ, d, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    k = torch.randint(-3, 4, (n, 1, d), generator=g, dtype=torch.int8)
    k[7] = 100
    kf = torch.full((n, 1), 0.01 * below / (100 * d))
    kf[7] *= 100
    v = torch.randint(1, 128, (n, 1, d), generator=g, dtype=torch.int8)
    vf = 0.01 * (1 + torch.rand(n, 1, generator=g))
    if zero == "scale":
        vf[7] = 0.0
    else:
        v[7, :, 1::2] = 0
    _check(q, *_one_sequence(k, v, kf, vf), dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("HQ", [1, 3, 8])
def test_scores_and_scales_that_grow_and_fall_in_turn(d, HQ):
    """Scores that rise by tens from key to key while the scales fall, fall while
    they rise, and jump both ways: references of both move all the time."""
    n = 700
    g = torch.Generator().manual_seed(HQ)
    q = torch.ones(1, HQ, d, dtype=torch.bfloat16)
    z = torch.linspace(-300, 300, n)
    z = torch.cat((z[:250], z[250:500].flip(0), z[500:][torch.randperm(n - 500, generator=g)]))
    k = torch.full((n, 1, d), 50, dtype=torch.int8)
    kf = (z / (50 * d))[:, None]
    v = torch.randint(1, 128, (n, 1, d), generator=g, dtype=torch.int8)
    # (scales that undo a part of the weights, from 2^-60 to 2^60)
    vf = torch.exp2((-0.2 * z + 5 * torch.randn(n, generator=g)).clamp(-60, 60))[:, None]
    for r in range(0, n, 90):
        v[r, :, r % d::3] = 0
    _check(q, *_one_sequence(k, v, kf.float(), vf.float()), "bf16")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("HQ", [2, 8])
def test_scales_at_the_ends_of_the_numbers(d, HQ):
    """Rows of the largest scales an append writes (2^121) among others of 1e-30 and
    of 0, with weights of 0: a mean of rows of 1e-30 all the same."""
    n = 100
    g = torch.Generator().manual_seed(d)
    q = torch.ones(1, HQ, d, dtype=torch.bfloat16)
    k = torch.zeros(n, 1, d, dtype=torch.int8)
    kf = torch.full((n, 1), 0.01)
    v = torch.randint(30, 128, (n, 1, d), generator=g, dtype=torch.int8)
    vf = torch.full((n, 1), 2.0 ** -100)
    for r, f in ((0, 2.0 ** 121), (40, 2.0 ** 121), (41, 0.0), (99, 2.0 ** 119)):
        k[r], kf[r], vf[r] = -127, 500.0 / (127 * d), f
    cache, t, kr, vr = _one_sequence(k, v, kf, vf)
    ref = reference(q, kr, vr * 2.0 ** 100, 1.0, n - 1)
    for table in (t, widen(t)):
        out, _ = kda.kda_attn_step_q8(q.cuda(), *cache, table.cuda(), i32([n]), 1.0, out_f32=True)
        check(out.double() * 2.0 ** 100, None, ref, n, EXACT_SUMS, TWO_PARTS + 2.0 ** -23)
