"""The step's other forms on a stream other than the current one: what a call makes
comes from the pool of the stream that writes it (on the host; how the calls share
the GPU is in test_parity_q8.py and test_parity_shared.py)."""
from types import SimpleNamespace

import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from test_attn_streams import _dev, _stream, notes  # noqa: F401 (a fixture)

I8, I32, F32 = torch.int8, torch.int32, torch.float32


def _calls(stream):
    N, HQ, HKV, d = 5, 8, 2, 64
    q, k, v = _dev(N, HQ, d), _dev(N, HKV, d), _dev(N, HKV, d)
    codes, scales = ([_dev(4, HKV, 16, *x, dtype=t) for _ in range(2)] for x, t in (((d,), I8), ((), F32)))
    kc, vc = _dev(4, HKV, 16, d), _dev(4, HKV, 16, d)
    table, lens, shared = _dev(N, 2, dtype=I32), _dev(N, dtype=I32), _dev(1, dtype=I32)
    strided, given = _dev(N, HQ + 1, d)[:, 1:], _dev(N, HQ, d)
    q8 = (*codes, *scales, table, lens)
    return [
        lambda: kda.kda_cache_append_q8(k, v, *q8, q=q, stream=stream)[:1],
        lambda: kda.kda_attn_step_q8(q, *q8, 0.1, stream=stream)[:1],
        lambda: kda.kda_attn_step_q8(strided, *q8, 0.1, given, stream=stream)[:1],
        lambda: kda.kda_attn_step_shared(q, kc, vc, table, lens, shared, 0.1, stream=stream)[:1],
        lambda: kda.kda_attn_step_shared(strided, kc, vc, table, lens, shared, 0.1, given,
                                         stream=stream)[:1],
    ]


@pytest.mark.parametrize("stream", [_stream(22), 22, SimpleNamespace(cuda_stream=22)])
def test_another_streams_call_makes_its_tensors_there(notes, stream):
    for call in _calls(stream):
        notes.made.clear()
        notes.launched.clear()
        returned = call()
        assert notes.made and [s for _, s in notes.launched] == [22]
        assert all(s.cuda_stream == 22 for _, s in notes.made)
        # the caller's tensors are in use on the caller's stream; scratch is not
        for t, _ in notes.made:
            mine = any(t is r for r in returned)
            assert getattr(t, "recorded", []) == ([notes.here] if mine else [])
        assert notes.now is notes.here


@pytest.mark.parametrize("stream", [None, 11, _stream(11)])
def test_the_current_streams_call_needs_no_marks(notes, stream):
    for call in _calls(stream):
        notes.made.clear()
        notes.launched.clear()
        call()
        assert [s for _, s in notes.launched] == [11]
        for t, s in notes.made:
            assert s is notes.here and not hasattr(t, "recorded")


def test_a_stream_of_another_device_is_refused(notes):
    for call in _calls(SimpleNamespace(cuda_stream=33, device_index=1)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    assert not notes.made and not notes.launched
