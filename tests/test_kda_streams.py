"""The KDA calls on a stream other than the current one: results and scratch come
from the pool of the stream that writes them, as the full-attention calls' do
(a block of the current stream's pool may still be read by work queued there)."""
import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from test_attn_streams import _dev, _stream, gpu, notes  # noqa: F401

F32 = torch.float32


def _calls(stream):
    T, H, d, C, W = 8, 2, 128, 16, 4
    q, la, b = _dev(T, H, d), _dev(T, H, d, dtype=F32), _dev(T, H, dtype=F32)
    state, pool = _dev(T, H, d, d, dtype=F32), _dev(3, H, d, d, dtype=F32)
    x, weight, cache = _dev(T, C), _dev(C, W, dtype=F32), _dev(T, C, W)
    args = (q, q, q, la, b, 0.1)
    kw = dict(stream=stream)
    return {
        "chunk_fwd": lambda: kda.kda_chunk_fwd(*args, **kw)[:1],
        "chunk_fwd f32": lambda: kda.kda_chunk_fwd(*args, out_f32=True, **kw)[:1],
        "chunk_fwd_static": lambda: kda.kda_chunk_fwd_static(*args, **kw)[:1],
        "recurrent_step": lambda: (kda.kda_recurrent_step(*args, state, **kw),),
        "recurrent_fwd": lambda: (kda.kda_recurrent_fwd(*args, pool, **kw),),
        "short_conv_fwd": lambda: (kda.kda_short_conv_fwd(x, weight, **kw),),
        "short_conv_step": lambda: (kda.kda_short_conv_step(x, weight, cache, **kw),),
        "recurrent_bwd": lambda: kda.kda_recurrent_bwd(*args, d_out=q, **kw),
        "chunk_bwd": lambda: kda.kda_chunk_bwd(*args, d_out=q, **kw),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("call", list(_calls(None)))
def test_another_streams_call_makes_its_tensors_there(notes, call, raw):
    returned = _calls(22 if raw else _stream(22))[call]()
    assert notes.made and [s for _, s in notes.launched] == [22]
    assert all(s.cuda_stream == 22 for _, s in notes.made)
    for t, _ in notes.made:
        mine = any(t is r for r in returned)
        assert getattr(t, "recorded", []) == ([notes.here] if mine else [])
    assert notes.now is notes.here


@pytest.mark.parametrize("call", list(_calls(None)))
def test_the_current_streams_call_needs_no_marks(notes, call):
    for stream in (None, 11):
        _calls(stream)[call]()
    assert [s for _, s in notes.launched] == [11, 11]
    assert all(s is notes.here and not hasattr(t, "recorded") for t, s in notes.made)


@pytest.mark.gpu
def test_results_leave_the_current_streams_pending_reads_alone(gpu):
    """A temporary of the output's size, freed while work queued on the current
    stream still reads it, keeps its contents beside a call on another."""
    T, H, d = 2000, 4, 128
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(T, H, d, generator=g).bfloat16().cuda() for _ in range(3))
    q, k = (x / x.float().norm(dim=-1, keepdim=True).bfloat16() for x in (q, k))
    la = -torch.rand(T, H, d, generator=g).cuda() * 0.1
    beta = torch.rand(T, H, generator=g).cuda()
    side = torch.cuda.Stream()
    want, _ = kda.kda_chunk_fwd(q, k, v, la, beta, 0.1)
    kept = torch.empty_like(want)
    torch.cuda.synchronize()
    for i in range(10):
        temporary = torch.full_like(want, float(i + 1))
        torch.cuda._sleep(2000000)   # a millisecond
        kept.copy_(temporary)
        del temporary
        got, _ = kda.kda_chunk_fwd(q, k, v, la, beta, 0.1, stream=side)
        torch.cuda.synchronize()
        assert (kept == i + 1).all() and torch.equal(got, want)
        del got
