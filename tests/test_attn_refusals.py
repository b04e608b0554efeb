"""The full-attention layer's entry points refuse what they do not support, on
the host, before any CUDA call (no kernel runs here)."""
import ctypes

import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from kimi_delta_attention_chunkwise_gb300 import binding, build

FAKE, OTHER = 0x10000, 0x20000  # never dereferenced
OK, INVALID, UNSUPPORTED = (kda.KDA_SUCCESS, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _shape(**kw):
    b = dict(N=1, T=64, HQ=8, HKV=2, d=64, dtype_code=kda.KDA_DTYPE_BF16)
    b.update(kw)
    return kda.make_attn_shape(**b)


def _cache(**kw):
    b = dict(k=FAKE, v=FAKE, block_table=FAKE, num_pages=4, page_size=16, max_pages=2)
    b.update(kw)
    return kda.kdaPagedCache_t(**b)


def _fwd(lib, shape, scale=0.125, cu=None, **kw):
    p = dict(q=FAKE, k=FAKE, v=FAKE, out=OTHER, lse=None)
    p.update(kw)
    return lib.kda_attn_fwd(p["q"], p["k"], p["v"], ctypes.c_float(scale), cu, p["out"], p["lse"],
                            ctypes.byref(shape) if shape is not None else None, None)


def _append(lib, shape, cache=None, cu=None, rope=None, **kw):
    p = dict(q=FAKE, k=FAKE, v=FAKE, lens=FAKE, q_out=FAKE, k_out=None)
    p.update(kw)
    cache = _cache() if cache is None else cache
    return lib.kda_cache_append(p["q"], p["k"], p["v"], cu, p["lens"],
                                ctypes.byref(rope) if rope is not None else None, p["q_out"],
                                p["k_out"], ctypes.byref(cache), ctypes.byref(shape), None)


def _step(lib, shape, cache=None, scale=0.125, ws=FAKE, nbytes=1 << 40, **kw):
    p = dict(q=FAKE, lens=FAKE, out=OTHER, lse=None)
    p.update(kw)
    cache = _cache() if cache is None else cache
    return lib.kda_attn_step_ws(p["q"], ctypes.byref(cache), p["lens"], ctypes.c_float(scale),
                                p["out"], p["lse"], ctypes.byref(shape), ws, nbytes, None)


SHAPES_INVALID = [dict(N=0), dict(T=-1), dict(HQ=0), dict(HKV=0), dict(HQ=8, HKV=3), dict(d=0),
                  dict(dtype_code=5), dict(out_f32=2), dict(q_stride=8 * 64 - 8),
                  dict(q_stride=8 * 64 + 4), dict(k_stride=64), dict(v_stride=-512)]
SHAPES_UNSUPPORTED = [dict(d=96), dict(d=256), dict(HQ=129, HKV=1), dict(HQ=65536, HKV=65536),
                      dict(T=1 << 30, HQ=8)]


@pytest.mark.parametrize("kw", SHAPES_INVALID)
def test_shape_invalid(lib, kw):
    s = _shape(**kw)
    assert _fwd(lib, s, cu=FAKE) == INVALID
    assert _append(lib, s, cu=FAKE) == INVALID
    n = ctypes.c_size_t(0)
    assert lib.kda_attn_step_workspace_size(ctypes.byref(_cache()), ctypes.byref(s),
                                            ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("kw", SHAPES_UNSUPPORTED)
def test_shape_unsupported(lib, kw):
    s = _shape(**kw)
    assert _fwd(lib, s) == UNSUPPORTED
    assert _append(lib, s) == UNSUPPORTED


def test_fwd_arguments(lib):
    assert _fwd(lib, None) == INVALID
    assert _fwd(lib, _shape(N=2)) == INVALID                     # N > 1 needs cu_seqlens
    for bad in (float("nan"), float("inf"), 0.0, -0.5, 3e38):    # 3e38 log2(e) overflows
        assert _fwd(lib, _shape(), scale=bad) == INVALID
    for name in ("q", "k", "v", "out"):
        assert _fwd(lib, _shape(), **{name: None}) == INVALID
        assert _fwd(lib, _shape(), **{name: FAKE + 8}) == INVALID
    assert _fwd(lib, _shape(), out=FAKE) == INVALID              # in place
    assert _fwd(lib, _shape(), lse=FAKE + 2) == INVALID
    assert _fwd(lib, _shape(), cu=FAKE + 2) == INVALID
    assert _fwd(lib, _shape(engine=7)) == INVALID
    # the tensor engine: bf16 with d = 64 or 128
    tensor = kda.KDA_ENGINE_TENSOR
    assert _fwd(lib, _shape(engine=tensor, dtype_code=kda.KDA_DTYPE_F32)) == UNSUPPORTED
    assert _fwd(lib, _shape(engine=tensor, d=32)) == UNSUPPORTED
    # nothing to do: accepted without a launch
    assert _fwd(lib, _shape(T=0), q=None, k=None, v=None, out=None) == OK


def test_append_arguments(lib):
    s = _shape()
    assert _append(lib, _shape(N=2)) == INVALID                  # 64 tokens of 2 sequences
    assert _append(lib, s, lens=None) == INVALID
    assert _append(lib, s, k=None) == INVALID
    assert _append(lib, s, v=FAKE + 8) == INVALID
    assert _append(lib, s, q=None) == INVALID                    # q_out without q
    assert _append(lib, s, q_out=None) == INVALID                # q without q_out
    assert _append(lib, s, k_out=FAKE + 4) == INVALID
    # in place only where a row is its own output
    assert _append(lib, _shape(q_stride=1024)) == INVALID
    assert _append(lib, _shape(k_stride=1024), q_out=FAKE + 64, k_out=FAKE) == INVALID
    R = lambda **kw: kda.kdaRope_t(**{**dict(table=FAKE, num_positions=8, rot_dim=64,
                                             interleaved=0), **kw})
    assert _append(lib, s, rope=R(table=None)) == INVALID
    assert _append(lib, s, rope=R(table=FAKE + 4)) == INVALID
    assert _append(lib, s, rope=R(num_positions=-1)) == INVALID
    assert _append(lib, s, rope=R(interleaved=2)) == INVALID
    assert _append(lib, s, rope=R(rot_dim=0)) == INVALID
    assert _append(lib, s, rope=R(rot_dim=24)) == UNSUPPORTED
    assert _append(lib, s, rope=R(rot_dim=128)) == UNSUPPORTED   # wider than a head
    assert _append(lib, _shape(T=0), k=None, v=None, q=None, q_out=None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=0), INVALID), (dict(page_size=-16), INVALID), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
    (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(k=None), INVALID),
    (dict(v=FAKE + 8), INVALID), (dict(block_table=None), INVALID),
    (dict(block_table=FAKE + 2), INVALID), (dict(max_pages=1 << 28), UNSUPPORTED)])
def test_cache_arguments(lib, kw, code):
    c = _cache(**kw)
    assert _append(lib, _shape(), cache=c) == code
    assert _step(lib, _shape(N=64), cache=c) == code


def test_step_arguments(lib):
    s = _shape(N=64)
    assert _step(lib, _shape(N=63)) == INVALID                   # one token per sequence
    assert _step(lib, s, scale=0.0) == INVALID
    for name in ("q", "out", "lens"):
        assert _step(lib, s, **{name: None}) == INVALID
    assert _step(lib, s, q=FAKE + 8) == INVALID
    assert _step(lib, s, out=FAKE) == INVALID                    # in place
    assert _step(lib, s, lse=FAKE + 1) == INVALID
    assert _step(lib, s, ws=FAKE + 16) == INVALID                # 256-byte alignment
    n = ctypes.c_size_t(0)
    size = lib.kda_attn_step_workspace_size
    assert size(None, ctypes.byref(s), ctypes.byref(n)) == INVALID
    assert size(ctypes.byref(_cache()), ctypes.byref(s), None) == INVALID
    assert size(ctypes.byref(_cache()), ctypes.byref(_shape(N=2)), ctypes.byref(n)) == INVALID


def test_binding_refuses_host_and_misfit_tensors():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_attn_fwd(z(4, 8, 64), z(4, 2, 64), z(4, 2, 64), 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_cache_append(z(4, 2, 64), z(4, 2, 64), z(3, 2, 16, 64), z(3, 2, 16, 64),
                             z(1, 2, dt=torch.int32), z(1, dt=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_attn_step(z(4, 8, 64), z(3, 2, 16, 64), z(3, 2, 16, 64),
                          z(4, 2, dt=torch.int32), z(4, dt=torch.int32), 0.1)
    with pytest.raises(TypeError):
        kda.kda_attn_fwd([1.0], None, None, 0.1)
