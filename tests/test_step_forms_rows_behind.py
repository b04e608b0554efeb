"""Rows behind a sequence's length in pages that it holds: what they hold, and what
another stream writes to them while a step runs, changes no result."""
import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from cache_testutil import i32, paged_q8, paged_shared, randn, widen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()


def _behind(cache, table, lens):
    """Index of every row of `cache` [P, HKV, page, ...] behind a length."""
    page = cache.shape[2]
    free = torch.ones(cache.shape[0], page, dtype=torch.bool)
    for s, n in enumerate(lens):
        for j in range(-(-n // page)):
            free[int(table[s, j]), :min(page, n - j * page)] = False
    p, r = free.nonzero(as_tuple=True)
    return p.cuda(), r.cuda()


def _while_written(call, tensors, at):
    """The bits of `call` with the rows `at` holding one thing, then changing all the time."""
    p, r = at
    other = torch.cuda.Stream()
    want = call()
    torch.cuda.synchronize()
    fills = {torch.int8: (-128, 127, 3)}
    for i in range(40):
        with torch.cuda.stream(other):
            for t in tensors:
                for x in fills.get(t.dtype, (float("nan"), float("inf"), -float("inf"), 1e30)):
                    t[p, :, r] = x
        got = [call() for _ in range(4)]
        torch.cuda.synchronize()
        for g in got:
            assert torch.equal(g, want)


@pytest.mark.parametrize("dtype,d,HQ", [("bf16", 128, 4), ("bf16", 64, 8), ("bf16", 128, 16),
                                        ("f32", 64, 4)])
@pytest.mark.parametrize("page", [16, 64])
def test_q8_rows_behind_a_length(dtype, d, HQ, page):
    lens = [1, 15, 17, 31, 33, 900, 0, 63, 3001]
    _, _, cache, table = paged_q8(d, lens, 1, d, page)
    q, n, wide = randn(1, len(lens), HQ, d, dtype=dtype).cuda(), i32(lens), widen(table)
    _while_written(lambda: kda.kda_attn_step_q8(q, *cache, wide, n, 0.1)[0], cache,
                   _behind(cache[0], table.cpu(), lens))


@pytest.mark.parametrize("dtype,d,HQ", [("bf16", 128, 4), ("bf16", 64, 8), ("f32", 64, 3)])
def test_shared_rows_behind_a_length(dtype, d, HQ):
    lens = [640 + x for x in (1, 15, 17, 31, 33, 900, 0, 63, 3001)] + [300]
    _, _, kc, vc, table = paged_shared(d, 10, lens, 1, d, 64, dtype)
    q, n, wide = randn(1, len(lens), HQ, d, dtype=dtype).cuda(), i32(lens), widen(table)
    _while_written(lambda: kda.kda_attn_step_shared(q, kc, vc, wide, n, i32([10]), 0.1)[0], (kc, vc),
                   _behind(kc, table.cpu(), lens))
