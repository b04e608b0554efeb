"""The step's other forms (a cache of 8-bit codes, shared pages) refuse what they do
not support on the host, before any CUDA call (no kernel runs here)."""
import ctypes
import os
import shutil
import subprocess

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


def _cache8(**kw):
    b = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, num_pages=4,
             page_size=16, max_pages=2)
    b.update(kw)
    return kda.kdaPagedCacheQ8_t(**b)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _append(lib, shape, cache=None, cu=None, rope=None, **kw):
    p = dict(q=FAKE, k=FAKE, v=FAKE, lens=FAKE, q_out=FAKE, k_out=None, ks=None, vs=None)
    p.update(kw)
    cache = _cache8() if cache is None else cache
    return lib.kda_cache_append_q8(p["q"], p["k"], p["v"], cu, p["lens"], _ref(rope), p["q_out"],
                                   p["k_out"], p["ks"], p["vs"], _ref(cache), _ref(shape), None)


def _step8(lib, shape, cache=None, scale=0.125, ws=FAKE, nbytes=1 << 40, **kw):
    p = dict(q=FAKE, lens=FAKE, out=OTHER, lse=None)
    p.update(kw)
    cache = _cache8() if cache is None else cache
    return lib.kda_attn_step_q8_ws(p["q"], _ref(cache), p["lens"], ctypes.c_float(scale),
                                   p["out"], p["lse"], _ref(shape), ws, nbytes, None)


def _shared(lib, shape, cache=None, scale=0.125, ws=FAKE, nbytes=1 << 40, **kw):
    p = dict(q=FAKE, lens=FAKE, n=FAKE, out=OTHER, lse=None)
    p.update(kw)
    cache = _cache() if cache is None else cache
    return lib.kda_attn_step_shared_ws(p["q"], _ref(cache), p["lens"], p["n"],
                                       ctypes.c_float(scale), p["out"], p["lse"], _ref(shape), ws,
                                       nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), INVALID), (dict(T=-1), INVALID), (dict(HQ=0), INVALID), (dict(HKV=0), INVALID),
    (dict(HQ=8, HKV=3), INVALID), (dict(d=0), INVALID), (dict(dtype_code=5), INVALID),
    (dict(out_f32=2), INVALID), (dict(q_stride=8 * 64 - 8), INVALID),
    (dict(q_stride=8 * 64 + 4), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(HQ=129, HKV=1), UNSUPPORTED), (dict(HQ=65536, HKV=65536), UNSUPPORTED),
    (dict(N=64, T=1 << 30, HQ=8), UNSUPPORTED), (dict(N=(1 << 30) + 1, HQ=1, HKV=1), UNSUPPORTED)])
def test_shapes(lib, kw, code):
    s = _shape(**{"N": 64, **kw})
    n = ctypes.c_size_t(0)
    assert _append(lib, s, cu=FAKE) == code
    assert lib.kda_attn_step_q8_workspace_size(_ref(_cache8()), _ref(s), ctypes.byref(n)) == code
    assert lib.kda_attn_step_shared_workspace_size(_ref(_cache()), _ref(s), ctypes.byref(n)) == code
    assert _step8(lib, s) == code and _shared(lib, s) == code


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=0), INVALID), (dict(page_size=-16), INVALID), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
    (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(k=None), INVALID),
    (dict(v=FAKE + 8), INVALID), (dict(block_table=None), INVALID),
    (dict(block_table=FAKE + 2), INVALID), (dict(max_pages=1 << 28), UNSUPPORTED)])
def test_caches(lib, kw, code):
    s = _shape(N=64)
    assert _append(lib, s, cache=_cache8(**kw)) == code
    assert _step8(lib, s, cache=_cache8(**kw)) == code
    assert _shared(lib, s, cache=_cache(**kw)) == code


@pytest.mark.parametrize("kw", [dict(k_scale=None), dict(v_scale=None), dict(k_scale=FAKE + 2),
                                dict(v_scale=FAKE + 1)])
def test_scales(lib, kw):
    s, n = _shape(N=64), ctypes.c_size_t(0)
    c = _cache8(**kw)
    assert _append(lib, s, cache=c) == INVALID and _step8(lib, s, cache=c) == INVALID
    assert lib.kda_attn_step_q8_workspace_size(_ref(c), _ref(s), ctypes.byref(n)) == INVALID


def test_append_arguments(lib):
    s = _shape()
    assert lib.kda_cache_append_q8(FAKE, FAKE, FAKE, None, FAKE, None, FAKE, None, None, None, None,
                                   _ref(s), None) == INVALID                       # no cache
    assert _append(lib, None) == INVALID
    assert _append(lib, _shape(N=2)) == INVALID                  # 64 tokens of 2 sequences
    assert _append(lib, s, lens=None) == INVALID
    assert _append(lib, s, k=None) == INVALID
    assert _append(lib, s, v=FAKE + 8) == INVALID
    assert _append(lib, s, q=None) == INVALID                    # q_out without q
    assert _append(lib, s, q_out=None) == INVALID                # q without q_out
    for name in ("k_out", "ks", "vs"):
        assert _append(lib, s, **{name: OTHER + 4}) == INVALID
    # what the codes stand for lies in tensors of its own
    for kw in (dict(ks=FAKE), dict(vs=FAKE), dict(ks=OTHER, vs=OTHER), dict(ks=OTHER, k_out=OTHER),
               dict(vs=OTHER, k_out=OTHER), dict(vs=OTHER, q=OTHER, q_out=FAKE + 64)):
        assert _append(lib, s, **kw) == INVALID
    # in place only where a row is its own output
    assert _append(lib, _shape(q_stride=1024)) == INVALID
    assert _append(lib, _shape(k_stride=1024), q_out=FAKE + 64, k_out=FAKE) == INVALID
    R = lambda **kw: kda.kdaRope_t(**{**dict(table=FAKE, num_positions=8, rot_dim=64,
                                             interleaved=0), **kw})
    for kw, code in ((dict(table=None), INVALID), (dict(table=FAKE + 4), INVALID),
                     (dict(num_positions=-1), INVALID), (dict(interleaved=2), INVALID),
                     (dict(rot_dim=0), INVALID), (dict(rot_dim=24), UNSUPPORTED),
                     (dict(rot_dim=128), UNSUPPORTED)):
        assert _append(lib, s, rope=R(**kw)) == code
    assert _append(lib, _shape(T=0), k=None, v=None, q=None, q_out=None) == OK


@pytest.mark.parametrize("step", [_step8, _shared])
def test_step_arguments(lib, step):
    s = _shape(N=64)
    assert step(lib, None) == INVALID
    assert step(lib, _shape(N=63)) == INVALID                    # one token per sequence
    for bad in (float("nan"), float("inf"), 0.0, -0.5, 3e38):
        assert step(lib, s, scale=bad) == INVALID
    for name in ("q", "out", "lens"):
        assert step(lib, s, **{name: None}) == INVALID
    assert step(lib, s, q=FAKE + 8) == INVALID
    assert step(lib, s, out=FAKE) == INVALID                     # in place
    assert step(lib, s, lse=FAKE + 1) == INVALID
    assert step(lib, s, ws=FAKE + 16) == INVALID                 # 256-byte alignment


def test_shared_pages_argument(lib):
    s = _shape(N=64)
    assert _shared(lib, s, n=None) == INVALID and _shared(lib, s, n=FAKE + 2) == INVALID


def test_sizes_want_somewhere_to_go(lib):
    s, n = _shape(N=64), ctypes.c_size_t(0)
    for size, cache in ((lib.kda_attn_step_q8_workspace_size, _cache8()),
                        (lib.kda_attn_step_shared_workspace_size, _cache())):
        assert size(None, _ref(s), ctypes.byref(n)) == INVALID
        assert size(_ref(cache), _ref(s), None) == INVALID
        assert size(_ref(cache), None, ctypes.byref(n)) == INVALID
        assert size(_ref(cache), _ref(_shape(N=2)), ctypes.byref(n)) == INVALID


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


def _dev(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt).as_subclass(_OnDevice)


I32, I8, F32 = torch.int32, torch.int8, torch.float32


def _args8(**kw):
    a = dict(k_cache=_dev(3, 2, 16, 64, dt=I8), v_cache=_dev(3, 2, 16, 64, dt=I8),
             k_scale=_dev(3, 2, 16, dt=F32), v_scale=_dev(3, 2, 16, dt=F32),
             block_table=_dev(4, 2, dt=I32))
    a.update(kw)
    return a


WRONG8 = [
    (dict(k_cache=_dev(3, 2, 16, 64)), TypeError), (dict(v_cache=_dev(3, 2, 16, 64)), TypeError),
    (dict(k_cache=_dev(3, 2, 16, 32, dt=I8)), ValueError),
    (dict(v_cache=_dev(2, 2, 16, 64, dt=I8)), ValueError),
    (dict(k_scale=_dev(3, 2, 16)), TypeError), (dict(v_scale=_dev(3, 2, 8, dt=F32)), ValueError),
    (dict(k_scale=_dev(3, 16, 2, dt=F32).transpose(1, 2)), ValueError),
    (dict(k_scale=None), TypeError), (dict(v_scale=torch.zeros(3, 2, 16)), ValueError),
    (dict(block_table=_dev(3, 2, dt=I32)), ValueError),
    (dict(block_table=_dev(4, 2, dt=torch.int64)), TypeError)]


@pytest.mark.parametrize("kw,error", WRONG8)
def test_binding_refuses_caches_of_codes(kw, error):
    with pytest.raises(error):
        kda.kda_attn_step_q8(_dev(4, 8, 64), **_args8(**kw), seq_lens=_dev(4, dt=I32), scale=0.1)
    with pytest.raises(error):
        kda.kda_cache_append_q8(_dev(4, 2, 64), _dev(4, 2, 64), **_args8(**kw),
                                cache_lens=_dev(4, dt=I32))


def test_binding_refuses_other_arguments():
    k, lens = _dev(4, 2, 64), _dev(4, dt=I32)
    for kw, error in ((dict(k_stored=_dev(4, 2, 32)), ValueError),
                      (dict(v_stored=_dev(4, 2, 64, dt=F32)), TypeError),
                      (dict(k_out=_dev(4, 64, 2).transpose(1, 2)), ValueError),
                      (dict(q=_dev(4, 3, 64)), ValueError), (dict(q_out=_dev(4, 2, 64)), ValueError),
                      (dict(rope=_dev(64, dt=F32)), ValueError),
                      (dict(rope=_dev(8, 64)), TypeError),
                      (dict(cu_seqlens=_dev(4, dt=I32)), ValueError),
                      (dict(cache_lens=None), ValueError), (dict(cache_lens=_dev(3, dt=I32)), ValueError)):
        with pytest.raises(error):
            kda.kda_cache_append_q8(k, k, **_args8(), **{"cache_lens": lens, **kw})
    with pytest.raises(ValueError, match="heads"):
        kda.kda_cache_append_q8(_dev(4, 1, 64), _dev(4, 1, 64), **_args8(), cache_lens=lens)
    q, c, t = _dev(4, 8, 64), _dev(3, 2, 16, 64), _dev(4, 2, dt=I32)
    n = _dev(1, dt=I32)
    shared = lambda q=q, c=c, t=t, l=lens, n=n, **kw: kda.kda_attn_step_shared(q, c, c, t, l, n, 0.1, **kw)
    for kw, error in ((dict(n=3), TypeError), (dict(n=torch.zeros(1, dtype=I32)), ValueError),
                      (dict(n=_dev(2, dt=I32)), ValueError), (dict(n=_dev(1, dt=torch.int64)), TypeError),
                      (dict(n=None), TypeError), (dict(l=_dev(3, dt=I32)), ValueError),
                      (dict(c=_dev(3, 3, 16, 64)), ValueError), (dict(q=_dev(4, 8, 32)), ValueError),
                      (dict(c=_dev(3, 2, 16, 64, dt=I8)), TypeError),
                      (dict(lse=_dev(4, 7, dt=F32)), ValueError), (dict(out=_dev(4, 8, 64, dt=I32)), TypeError)):
        with pytest.raises(error):
            shared(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        shared(q=torch.zeros(4, 8, 64, dtype=torch.bfloat16))


def test_struct_layout_matches_the_header(tmp_path):
    """kdaPagedCacheQ8_t as the C compiler lays it out."""
    gcc, cuda_inc = shutil.which("gcc"), "/usr/local/cuda/include"
    if not gcc or not os.path.exists(os.path.join(cuda_inc, "cuda_runtime_api.h")):
        pytest.skip("gcc or the CUDA headers are missing")
    cls = binding.kdaPagedCacheQ8_t
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "kda.h"', "int main(void) {",
             '  printf("%zu\\n", sizeof(kdaPagedCacheQ8_t));']
    lines += [f'  printf("%zu\\n", offsetof(kdaPagedCacheQ8_t, {f}));' for f, _ in cls._fields_]
    (tmp_path / "layout.c").write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = str(tmp_path / "layout")
    subprocess.run([gcc, "-std=c99", "-I", build.INCLUDE, "-I", cuda_inc, str(tmp_path / "layout.c"),
                    "-o", exe], check=True, capture_output=True)
    seen = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in seen] == [ctypes.sizeof(cls)] + \
        [getattr(cls, f).offset for f, _ in cls._fields_]
