"""Waits of the step's other forms that run out, without a GPU fault: one copy is made
and never taken as landed (a barrier with one arrival more than it gets), with a limit
of about two milliseconds.  The kernel gives up by itself, says so in the device status
word and leaves the context usable; the next call is right."""
import ctypes
import time

import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda
from cache_testutil import i32, paged_q8, paged_shared, randn, widen
from kimi_delta_attention_chunkwise_gb300 import binding, build

SHORT_WAIT = 4_000_000  # SM clocks, ~2 ms at 2 GHz
NONE, STEP, SHARED = 0, 1, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _q8(lens, HQ, HKV, d, dtype="bf16", wide=True):
    """(the plain call, the diagnostic one) over the same inputs."""
    _, _, cache, table = paged_q8(3, lens, HKV, d, 32)
    table = widen(table) if wide else table
    q, n = randn(1, len(lens), HQ, d, dtype=dtype).cuda(), i32(lens)
    code = kda.KDA_DTYPE_BF16 if dtype == "bf16" else kda.KDA_DTYPE_F32
    shape = kda.make_attn_shape(len(lens), len(lens), HQ, HKV, d, code)
    c = kda.kdaPagedCacheQ8_t(*(x.data_ptr() for x in (*cache, table)), cache[0].shape[0], 32,
                              table.shape[1])
    need = kda.kda_attn_step_q8_workspace_size(c, shape)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")

    def diag(withhold, wait=SHORT_WAIT):
        out = torch.full_like(q, float("nan"))
        st = binding.load().kda_attn_step_q8_ws_diag(
            q.data_ptr(), ctypes.byref(c), n.data_ptr(), 0.1, out.data_ptr(), None,
            ctypes.byref(shape), (ws.data_ptr() + 255) // 256 * 256, need, withhold, wait,
            torch.cuda.current_stream().cuda_stream)
        return st, out

    return lambda: kda.kda_attn_step_q8(q, *cache, table, n, 0.1)[0], diag


def _shared(common, lens, HQ, HKV, d, dtype="bf16", wide=True):
    _, _, kc, vc, table = paged_shared(3, common, lens, HKV, d, 32, dtype)
    table = widen(table) if wide else table
    q, n, num = randn(1, len(lens), HQ, d, dtype=dtype).cuda(), i32(lens), i32([common])
    code = kda.KDA_DTYPE_BF16 if dtype == "bf16" else kda.KDA_DTYPE_F32
    shape = kda.make_attn_shape(len(lens), len(lens), HQ, HKV, d, code)
    c = kda.kdaPagedCache_t(kc.data_ptr(), vc.data_ptr(), table.data_ptr(), kc.shape[0], 32,
                            table.shape[1])
    need = kda.kda_attn_step_shared_workspace_size(c, shape)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")

    def diag(withhold, wait=SHORT_WAIT):
        out = torch.full_like(q, float("nan"))
        st = binding.load().kda_attn_step_shared_ws_diag(
            q.data_ptr(), ctypes.byref(c), n.data_ptr(), num.data_ptr(), 0.1, out.data_ptr(), None,
            ctypes.byref(shape), (ws.data_ptr() + 255) // 256 * 256, need, withhold, wait,
            torch.cuda.current_stream().cuda_stream)
        return st, out

    return lambda: kda.kda_attn_step_shared(q, kc, vc, table, n, num, 0.1)[0], diag


CALLS = [
    (_q8, ([3000, 17, 0, 64], 8, 2, 128), [STEP]),
    (_q8, ([700] * 12, 16, 1, 64), [STEP]),
    (_shared, (20, [700, 640, 3000, 5, 0], 8, 2, 128), [STEP, SHARED]),
    (_shared, (40, [1300 + i for i in range(90)], 16, 4, 64), [STEP, SHARED]),
    (_shared, (20, [700, 3000], 4, 2, 128), [STEP]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("make,args,withheld", CALLS)
def test_a_copy_that_never_counts_is_reported(make, args, withheld):
    plain, diag = make(*args)
    want = plain()
    assert kda.kda_device_status() == kda.KDA_SUCCESS
    for what in withheld:
        t0 = time.perf_counter()
        st, _ = diag(what)
        assert st == kda.KDA_SUCCESS
        assert kda.kda_device_status() == kda.KDA_ERR_TIMEOUT
        assert time.perf_counter() - t0 < 5.0
        # read and cleared; the next calls are right
        assert kda.kda_device_status() == kda.KDA_SUCCESS
        assert torch.equal(plain(), want)
        st, out = diag(NONE, 200 * SHORT_WAIT)
        assert st == kda.KDA_SUCCESS and torch.equal(out, want)
        assert kda.kda_device_status() == kda.KDA_SUCCESS


@pytest.mark.gpu
@pytest.mark.parametrize("make,args,withheld", [
    (_q8, ([300], 2, 1, 64, "f32"), [STEP, SHARED]), (_q8, ([300], 2, 1, 64, "bf16", False), [STEP]),
    (_q8, ([300], 2, 1, 64), [SHARED]), (_shared, (2, [100], 2, 1, 64), [SHARED]),
    (_shared, (2, [100, 70], 8, 1, 64, "f32"), [STEP, SHARED]),
    (_shared, (2, [100, 70], 8, 1, 64, "bf16", False), [STEP, SHARED])])
def test_calls_without_such_a_wait_say_so(make, args, withheld):
    plain, diag = make(*args)
    for what in withheld:
        st, out = diag(what)
        assert st == kda.KDA_ERR_UNSUPPORTED and out.isnan().all()
    st, out = diag(NONE)
    assert st == kda.KDA_SUCCESS and torch.equal(out, plain())


def test_other_numbers_are_refused():
    """(before any CUDA call; nothing is dereferenced)"""
    fake, lib = 0x10000, binding.load()
    shape = kda.make_attn_shape(1, 1, 8, 2, 64, kda.KDA_DTYPE_BF16)
    c8 = kda.kdaPagedCacheQ8_t(*[fake] * 5, 4, 16, 2)
    c = kda.kdaPagedCache_t(*[fake] * 3, 4, 16, 2)
    for what in (-1, 3):
        assert lib.kda_attn_step_q8_ws_diag(
            fake, ctypes.byref(c8), fake, 0.1, 2 * fake, None, ctypes.byref(shape), fake, 1 << 40,
            what, 0, None) == kda.KDA_ERR_INVALID_ARG
        assert lib.kda_attn_step_shared_ws_diag(
            fake, ctypes.byref(c), fake, fake, 0.1, 2 * fake, None, ctypes.byref(shape), fake,
            1 << 40, what, 0, None) == kda.KDA_ERR_INVALID_ARG
