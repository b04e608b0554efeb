"""kda_attn_step_shared keeps kda_attn_step's 2^-15 of every weight, whichever kernels
a call takes: few rows or many behind the shared tokens, short tables or wide ones,
sequences that hold the shared tokens or fewer (against the definition in 64 bits)."""
import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from attn_testutil import reference
from cache_testutil import DT, FP32, TWO_PARTS, check, i32, mma, paged_shared, randn, widen

pytestmark = pytest.mark.gpu
EXACT_SUMS = -6   # (check's d: its d + 9 roundings of a score)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()


def _peaked(seed, common, lens, HQ, HKV, d, page, dtype):
    """Queries of one channel alone, so that the scores' sums are exact, and keys
    whose scores leave a few of them most of the weight.  (q, k and v rows, caches,
    table)."""
    ks, vs, kc, vc, table = paged_shared(seed, common, lens, HKV, d, page, dtype, 0.0)
    size = torch.tensor(6.0, dtype=DT[dtype])
    q = torch.zeros(len(lens), HQ, d, dtype=DT[dtype])
    q[..., 0] = 1 + randn(seed, len(lens), HQ).abs().to(DT[dtype])
    fall = lambda x: -(x.abs() * size.to(x.device))
    kc[..., 0] = fall(kc[..., 0])
    ks = [k.clone() for k in ks]
    for k in ks:
        k[..., 0] = fall(k[..., 0])
    return q, ks, vs, kc, vc, table


def _rows(q, ks, vs, out, lse, weights):
    for s in range(q.shape[0]):
        n = ks[s].shape[0]
        if n:
            check(out[s:s + 1], lse[s:s + 1], reference(q[s:s + 1], ks[s], vs[s], 1.0, n - 1), n,
                  EXACT_SUMS, weights)
        else:
            assert (out[s] == 0).all() and (lse[s] == -float("inf")).all()


CASES = [
    # shared pages, lens, HQ, HKV, d, page
    (4, [300, 256, 280], 4, 2, 128, 64),                           # 6 rows to a key-value head
    (4, [300, 256, 280, 270, 400], 4, 2, 128, 64),                 # 10: one row tile
    (9, [147 + i for i in range(20)], 32, 8, 128, 16),             # 80
    (8, [512 + 3 * i for i in range(50)] + [500, 3, 0], 8, 2, 64, 64),     # two row tiles
    (3, [200 + i % 7 for i in range(40)], 32, 4, 128, 64),         # several blocks of them
    (2, [260 + i for i in range(9)], 16, 1, 64, 128),              # 16 query heads to one
    (5, [90 + i for i in range(4)], 40, 1, 128, 16),
    (24, [1536 + 9 * i for i in range(30)], 12, 2, 128, 64),
]


@pytest.mark.parametrize("common,lens,HQ,HKV,d,page", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_weights(common, lens, HQ, HKV, d, page, dtype):
    q, ks, vs, kc, vc, table = _peaked(HQ + d, common, lens, HQ, HKV, d, page, dtype)
    for t in (table, widen(table)):
        lse = torch.empty(len(lens), HQ, device="cuda")
        out, _ = kda.kda_attn_step_shared(q.cuda(), kc, vc, t, i32(lens), i32([common]), 1.0, None,
                                          lse, out_f32=True)
        _rows(q, ks, vs, out, lse, TWO_PARTS if mma(dtype, d) else FP32)


@pytest.mark.parametrize("d,HQ", [(128, 8), (64, 4), (128, 12)])
def test_a_sequence_alone_and_among_others(d, HQ):
    """What a sequence's row comes to is the same to 2^-15 of each weight whether it
    is one of 2, 20 or 100 that share their pages, and as kda_attn_step has it."""
    common, page, HKV = 16, 64, 2
    lens = [common * page + 5 * i % 90 for i in range(100)]
    q, ks, vs, kc, vc, table = _peaked(d, common, lens, HQ, HKV, d, page, "bf16")
    for n in (2, 20, 100):
        args = (q[:n].cuda().contiguous(), kc, vc, widen(table[:n]), i32(lens[:n]))
        lse = torch.empty(n, HQ, device="cuda")
        out, _ = kda.kda_attn_step_shared(*args, i32([common]), 1.0, None, lse, out_f32=True)
        plain, _ = kda.kda_attn_step(*args, 1.0, out_f32=True)
        for o in (out, plain):
            _rows(q[:2], ks, vs, o, lse, TWO_PARTS)


@pytest.mark.parametrize("dtype,HQ,HKV,d", [("f32", 4, 1, 64), ("f32", 16, 2, 16), ("bf16", 8, 2, 32)])
def test_calls_that_the_plain_step_does(dtype, HQ, HKV, d):
    """Row blocks that sharing would not save: kda_attn_step's kernels, and its bits,
    with the shared form's own checks of pages and of their number."""
    common, page = 8, 32
    lens = [common * page + 11 * i % 97 for i in range(20)] + [100, 0, 3]
    q, ks, vs, kc, vc, table = _peaked(d, common, lens, HQ, HKV, d, page, dtype)
    wide, n, q = widen(table), i32(lens), q.cuda()
    lse = torch.empty(len(lens), HQ, device="cuda")
    out, _ = kda.kda_attn_step_shared(q, kc, vc, wide, n, i32([common]), 1.0, None, lse, out_f32=True)
    _rows(q.cpu(), ks, vs, out, lse, FP32)
    assert torch.equal(out, kda.kda_attn_step(q, kc, vc, wide, n, 1.0, out_f32=True)[0])
    assert kda.kda_device_status() == kda.KDA_SUCCESS
    for bad in (-1, wide.shape[1] + 1):
        got, _ = kda.kda_attn_step_shared(q, kc, vc, wide, n, i32([bad]), 1.0, out_f32=True)
        assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
        assert torch.equal(got, out)
    wide[:20, 2] = kc.shape[0]
    kda.kda_attn_step_shared(q, kc, vc, wide, n, i32([common]), 1.0)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
