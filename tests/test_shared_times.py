"""kda_attn_step_shared leaves no SMs to work that there is not, and does not share
where nothing is gained: times against the same call's with nothing shared and
against kda_attn_step's, medians of replayed graphs in turn."""
import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()


def _captured(call, reps=10):
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(reps):
            call()
    return g


def _medians(graphs, times=9):
    """Median time of every graph, replayed in turn."""
    found = [[] for _ in graphs]
    for _ in range(times):
        for g, f in zip(graphs, found):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            f.append(a.elapsed_time(b))
    return [sorted(f)[times // 2] for f in found]


@pytest.mark.parametrize("n,common", [(16, 1024), (32, 512)])
def test_shared_pages_that_no_sequence_holds(n, common):
    """A document's pages are still said to be shared when the sequences that held
    them have ended: the others' step takes as long as with none shared (the time
    was twice that when most SMs were kept for the shared pages)."""
    HQ, HKV, d, page = 32, 8, 128, 64
    g = torch.Generator(device="cuda").manual_seed(n)
    lens = torch.randint(500, 2000, (n,), generator=g, device="cuda", dtype=torch.int32)
    kc, vc = (torch.randn(32 * n, HKV, page, d, generator=g, device="cuda").bfloat16()
              for _ in range(2))
    table = torch.full((n, common), -1, dtype=torch.int32, device="cuda")
    table[:, :32] = torch.arange(32 * n, dtype=torch.int32, device="cuda").view(n, 32)
    q = torch.randn(n, HQ, d, generator=g, device="cuda").bfloat16()
    pages = [torch.tensor([p], dtype=torch.int32, device="cuda") for p in (0, common)]
    none, unheld = _medians([
        _captured(lambda: kda.kda_attn_step_shared(q, kc, vc, table, lens, p, 0.1)) for p in pages])
    assert unheld < 1.4 * none, f"{unheld * 100:.1f} us, with none shared {none * 100:.1f}"


@pytest.mark.parametrize("HQ,HKV,d,dtype", [(32, 8, 16, torch.float32), (16, 2, 16, torch.float32),
                                            (16, 2, 32, torch.bfloat16)])
def test_sharing_that_saves_no_reads(HQ, HKV, d, dtype):
    """With 4 or 8 query heads to a key-value head the CUDA-core blocks behind shared
    pages are as many as kda_attn_step's: the call takes no longer than that."""
    n, common, page = 57, 36, 64
    g = torch.Generator(device="cuda").manual_seed(d)
    lens = common * page + torch.randint(1, 200, (n,), generator=g, device="cuda", dtype=torch.int32)
    kc, vc = (torch.randn(common + 4 * n, HKV, page, d, generator=g, device="cuda").to(dtype)
              for _ in range(2))
    table = torch.arange(common, dtype=torch.int32, device="cuda").repeat(n, 1)
    table = torch.cat((table, common + torch.arange(4 * n, dtype=torch.int32, device="cuda").view(n, 4)),
                      dim=1)
    q = torch.randn(n, HQ, d, generator=g, device="cuda").to(dtype)
    pages = torch.tensor([common], dtype=torch.int32, device="cuda")
    shared, plain = _medians([
        _captured(lambda: kda.kda_attn_step_shared(q, kc, vc, table, lens, pages, 0.1)),
        _captured(lambda: kda.kda_attn_step(q, kc, vc, table, lens, 0.1))])
    assert shared < 1.1 * plain, f"{shared * 100:.1f} us, kda_attn_step {plain * 100:.1f}"
