"""The step's wide tables: every way in which an item (a sequence's tiles under one
block of query heads) can be shared by several CTAs and joined by the second
kernel, against the definition in 64 bits."""
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


def _plan(lens, HQ, HKV, d, dtype, capacity):
    """The step's plan: (items, CTAs, CTAs that work on each item)."""
    G = HQ // HKV
    mma = dtype == "bf16" and d >= 64
    rows = 4 if not mma or G <= 4 else 8 if G <= 8 else 16
    blocks = -(-G // rows)
    items = len(lens) * HKV * blocks
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    grid = min(sms * (3 if rows <= 8 else 2), items * (capacity // 64 + 1))
    tiles = [-(-n // 64) for n in lens for _ in range(HKV * blocks)]
    units = sum(tiles)
    work = min(grid, units)
    starts = [units * c // work for c in range(work)]
    shared, at = [], 0
    for t in tiles:
        first = max(c for c in range(work) if starts[c] <= at) if t else 0
        last = max(c for c in range(work) if starts[c] < at + t) if t else -1
        shared.append(last - first + 1)
        at += t
    return items, grid, shared


def _spread(seed, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(seed)).tolist()


# lens, HQ, HKV, d, type, whether the join goes by item, CTAs on some item at least
CASES = {
    # more items than CTAs: a join CTA to every border between two of the step's
    "bf16 more items than CTAs": (_spread(1, 130, 0, 700), 8, 4, 128, "bf16", False, 2),
    "bf16 d = 64 more items than CTAs": (_spread(2, 64, 100, 3000), 16, 8, 64, "bf16", False, 2),
    "bf16 G = 8 more items than CTAs": (_spread(3, 240, 0, 500), 16, 2, 64, "bf16", False, 2),
    "bf16 G = 12 more items than CTAs": (_spread(4, 160, 0, 400), 24, 2, 128, "bf16", False, 2),
    "f32 more items than CTAs": (_spread(5, 130, 0, 700), 8, 4, 64, "f32", False, 2),
    "f32 G = 6, two blocks of heads": (_spread(6, 120, 0, 400), 12, 2, 128, "f32", False, 2),
    # fewer: a join CTA to every item, all of its query heads in it
    "bf16 G = 4 by item": (_spread(7, 20, 300, 900), 8, 2, 128, "bf16", True, 3),
    "bf16 G = 8 by item": (_spread(8, 20, 300, 900), 16, 2, 128, "bf16", True, 3),
    "bf16 G = 12 by item": (_spread(9, 20, 300, 900), 24, 2, 128, "bf16", True, 2),
    "bf16 G = 16 by item": (_spread(10, 40, 0, 900), 32, 2, 64, "bf16", True, 2),
    "bf16 G = 40 by item": (_spread(11, 16, 0, 900), 40, 1, 128, "bf16", True, 2),
    "f32 by item": (_spread(12, 20, 300, 900), 8, 2, 128, "f32", True, 3),
    # few items, each over very many CTAs: a join CTA to a query head
    "bf16 G = 16 few": ([9000, 0, 300], 16, 1, 128, "bf16", True, 50),
    "f32 few": ([9000, 300], 6, 1, 64, "f32", True, 50),
}


@pytest.mark.parametrize("case", list(CASES))
def test_shared_items(case):
    lens, HQ, HKV, d, dtype, by_item, most = CASES[case]
    N, page, width = len(lens), 64, 16384
    items, grid, shared = _plan(lens, HQ, HKV, d, dtype, width * page)
    assert (items < grid) == by_item and max(shared) >= most
    pages = [-(-n // page) for n in lens]
    order = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1)).int()
    kc, vc = (torch.full((sum(pages), HKV, page, d), float("nan"), dtype=DT[dtype]) for _ in range(2))
    table = torch.full((N, width), -1, dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    ks, vs, at = [], [], 0
    for s, n in enumerate(lens):
        table[s, :pages[s]] = order[at:at + pages[s]]
        at += pages[s]
        for c, rows in ((kc, ks), (vc, vs)):
            x = torch.randn(n, HKV, d, generator=g).to(DT[dtype])
            rows.append(x)
            for j in range(pages[s]):
                m = min(page, n - j * page)
                c[int(table[s, j]), :, :m] = x[j * page:j * page + m].transpose(0, 1)
    q = torch.randn(N, HQ, d, generator=g).to(DT[dtype])
    lse = torch.full((N, HQ), float("nan"), device="cuda")
    args = (q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), d ** -0.5)
    out, _ = kda.kda_attn_step(*args, None, lse)
    assert torch.equal(kda.kda_attn_step(*args)[0], out)
    for s, n in enumerate(lens):
        if n == 0:
            assert (out[s] == 0).all() and (lse[s] == -float("inf")).all()
        else:
            check(out[s:s + 1], lse[s:s + 1],
                  reference(q[s:s + 1], ks[s], vs[s], d ** -0.5, n - 1), n, d, dtype == "bf16")
