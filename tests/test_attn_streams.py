"""The full-attention layer's calls on a stream other than the current one: what
a call makes comes from the pool of the stream that writes it.  A block of the
current stream's pool may still be read by work queued there, which only that
stream's later work may overwrite."""
import contextlib
import functools
from types import SimpleNamespace

import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from kimi_delta_attention_chunkwise_gb300 import binding

BF16, I32 = torch.bfloat16, torch.int32


# ---------------------------------------------------------------------------
# on the host: a device that only takes notes
# ---------------------------------------------------------------------------
class _OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0 and notes record_stream()."""
    is_cuda = True

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream]


def _dev(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


def _stream(handle):
    return SimpleNamespace(cuda_stream=handle, device_index=0)


class _Notes:
    """Stands in for torch in the binding: made holds (tensor, the stream that
    was current when it was made), launched the calls' (name, stream)."""

    def __init__(self):
        self.here = _stream(11)
        self.now, self.made, self.launched = self.here, [], []
        current = lambda dev=None: self.now
        self.cuda = SimpleNamespace(stream=self._as_current, current_stream=current,
                                    device=lambda dev: contextlib.nullcontext(),
                                    current_device=lambda: 0,
                                    ExternalStream=lambda h, device=None: _stream(h))
        self._C = SimpleNamespace(_cuda_getCurrentRawStream=lambda dev: self.now.cuda_stream,
                                  _cuda_getDevice=lambda: 0)

    def __getattr__(self, name):
        if name.startswith("kda_"):
            return self._size if name.endswith("_size") else functools.partial(self._launch, name)
        return getattr(torch, name)

    @contextlib.contextmanager
    def _as_current(self, stream):
        before, self.now = self.now, stream
        yield
        self.now = before

    def _note(self, t):
        self.made.append((t, self.now))
        return t

    def empty(self, shape, dtype, device):
        return self._note(_dev(*((shape,) if isinstance(shape, int) else shape), dtype=dtype))

    def empty_like(self, t):
        return self._note(_dev(*t.shape, dtype=t.dtype))

    # libkda
    def _size(self, *args):
        args[-1]._obj.value = 4096
        return 0

    def _launch(self, name, *args):
        self.launched.append((name, args[-1]))
        return 0


@pytest.fixture
def notes(monkeypatch):
    n = _Notes()
    monkeypatch.setattr(binding, "_torch", lambda: n)
    monkeypatch.setattr(binding, "load", lambda: n)
    monkeypatch.setattr(binding, "_step_bytes", {})
    monkeypatch.setattr(binding, "_ws_cache", {})
    return n


def _calls(stream):
    N, HQ, HKV, d = 5, 8, 2, 64
    q, k, v = _dev(N, HQ, d), _dev(N, HKV, d), _dev(N, HKV, d)
    kc, vc, table, lens = _dev(4, HKV, 16, d), _dev(4, HKV, 16, d), _dev(N, 2, dtype=I32), \
        _dev(N, dtype=I32)
    strided, given = _dev(N, HQ + 1, d)[:, 1:], _dev(N, HQ, d)
    return [
        lambda: kda.kda_attn_fwd(q, k, v, 0.1, stream=stream)[:1],
        lambda: kda.kda_attn_fwd(q, k, v, 0.1, stream=stream, out_f32=True)[:1],
        lambda: kda.kda_attn_fwd(strided, k, v, 0.1, stream=stream)[:1],
        lambda: kda.kda_cache_append(k, v, kc, vc, table, lens, q=q, stream=stream)[:1],
        lambda: kda.kda_attn_step(q, kc, vc, table, lens, 0.1, stream=stream)[:1],
        lambda: kda.kda_attn_step(strided, kc, vc, table, lens, 0.1, given, stream=stream)[:1],
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


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------
@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()
    torch.cuda.synchronize()


def _randn(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _cache(N, width, HKV, d, page, dtype):
    """Random pages, and a table of `width` entries that uses the first ones."""
    pages = 40
    kc, vc = (_randn(i, pages, HKV, page, d, dtype=dtype) for i in (1, 2))
    table = torch.full((N, width), -1, dtype=I32)
    table[:, :8] = torch.randint(0, pages, (N, 8), generator=torch.Generator().manual_seed(3))
    return kc, vc, table.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_steps_on_two_streams_at_once(gpu, dtype):
    """A wide table's step on the current stream and one on another right
    after it, many times: the bits of steps that run alone."""
    N, HQ, HKV, d, page = 8, 8, 2, 128, 64
    kc, vc, table = _cache(N, 16384, HKV, d, page, dtype)
    lens = torch.tensor([512, 500, 3, 64, 0, 333, 512, 100], dtype=I32, device="cuda")
    q = [_randn(i, N, HQ, d, dtype=dtype) for i in (5, 6)]
    want = [kda.kda_attn_step(x, kc, vc, table, lens, 0.1)[0] for x in q]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(200):
        a, _ = kda.kda_attn_step(q[0], kc, vc, table, lens, 0.1)
        b, _ = kda.kda_attn_step(q[1], kc, vc, table, lens, 0.1, stream=side)
        c, _ = kda.kda_attn_step(q[0], kc, vc, table, lens, 0.1)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_results_leave_the_current_streams_pending_reads_alone(gpu, raw):
    """A temporary of an output's size, freed while work queued on the current
    stream still reads it, keeps its contents beside a call on another."""
    T, HQ, HKV, d, page = 4096, 8, 2, 64, 64
    q, k, v = _randn(1, T, HQ, d), _randn(2, T, HKV, d), _randn(3, T, HKV, d)
    kc, vc = torch.zeros(80, HKV, page, d, dtype=BF16, device="cuda"), \
        torch.zeros(80, HKV, page, d, dtype=BF16, device="cuda")
    table = torch.arange(80, dtype=I32, device="cuda")[None]
    held = torch.zeros(1, dtype=I32, device="cuda")
    side = torch.cuda.Stream()
    on = side.cuda_stream if raw else side
    calls = [lambda s: kda.kda_attn_fwd(q, k, v, 0.1, stream=s)[0],
             lambda s: kda.kda_cache_append(k, v, kc, vc, table, held, q=q, stream=s)[0]]
    for call in calls:
        want = call(None)
        kept = torch.empty_like(want)
        torch.cuda.synchronize()
        for i in range(10):
            temporary = torch.full_like(want, float(i + 1))
            torch.cuda._sleep(2000000)   # a millisecond
            kept.copy_(temporary)
            del temporary
            got = call(on)
            torch.cuda.synchronize()
            assert (kept == i + 1).all() and torch.equal(got, want)
            del got


@pytest.mark.gpu
def test_a_captured_call_on_a_forked_stream(gpu):
    """A call on a stream that a capture has forked: its tensors live in the
    graph's memory, and replays on other queries give their results."""
    N, HQ, HKV, d, page = 8, 8, 2, 128, 64
    kc, vc, table = _cache(N, 16384, HKV, d, page, BF16)
    lens = torch.tensor([512, 500, 3, 64, 0, 333, 512, 100], dtype=I32, device="cuda")
    q = [_randn(i, N, HQ, d) for i in (5, 6)]
    want = [kda.kda_attn_step(x, kc, vc, table, lens, 0.1)[0] for x in q]
    static, side = q[0].clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        out, _ = kda.kda_attn_step(static, kc, vc, table, lens, 0.1, stream=side)
        here, _ = kda.kda_attn_step(static, kc, vc, table, lens, 0.1)
        torch.cuda.current_stream().wait_stream(side)
        both = torch.cat((out, here))
    for x, w in ((q[1], want[1]), (q[0], want[0]), (q[1], want[1])):
        static.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(both, torch.cat((w, w)))
