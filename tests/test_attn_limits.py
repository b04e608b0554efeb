"""The full-attention layer at the ends of the sizes it accepts."""
import ctypes

import pytest
import torch

import kimi_delta_attention_chunkwise_gb300 as kda

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOP = 1 << 31


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kimi_delta_attention_chunkwise_gb300 import build
    build.build()
    torch.cuda.empty_cache()


def test_more_than_2_30_sequences_are_refused():
    """The kernels find a token's sequence, and the sequences' tiles, with sums
    of two sequence indices in 32 bits."""
    from kimi_delta_attention_chunkwise_gb300 import binding, build
    build.build()
    lib, fake, other = binding.load(), 0x10000, 0x20000   # never dereferenced
    cache = kda.kdaPagedCache_t(fake, fake, fake, 4, 16, 2)
    n = ctypes.c_size_t(0)
    for N, T, code in (((1 << 30) + 1, 9, kda.KDA_ERR_UNSUPPORTED),
                       (TOP - 1, 9, kda.KDA_ERR_UNSUPPORTED), (1 << 30, 0, kda.KDA_SUCCESS)):
        s = ctypes.byref(kda.make_attn_shape(N, T, 1, 1, 64, kda.KDA_DTYPE_BF16))
        assert lib.kda_attn_fwd(fake, fake, fake, 0.1, fake, other, None, s, None) == code
        assert lib.kda_cache_append(None, fake, fake, fake, fake, None, None, None,
                                    ctypes.byref(cache), s, None) == code
    s = ctypes.byref(kda.make_attn_shape((1 << 30) + 1, (1 << 30) + 1, 1, 1, 64, kda.KDA_DTYPE_BF16))
    assert lib.kda_attn_step_workspace_size(ctypes.byref(cache), s, ctypes.byref(n)) == \
        kda.KDA_ERR_UNSUPPORTED


def test_sizes_past_32_bits_are_refused_not_cut_off():
    """2^32 + 5 of anything would arrive as 5."""
    from kimi_delta_attention_chunkwise_gb300 import binding
    many = (1 << 32) + 5
    for i in range(5):
        sizes = [1, 1, 1, 1, 64]
        sizes[i] = many
        with pytest.raises(ValueError, match="2\\^31"):
            kda.make_attn_shape(*sizes, kda.KDA_DTYPE_BF16)
        with pytest.raises(ValueError, match="2\\^31"):
            binding._shape_ref(*sizes, kda.KDA_DTYPE_BF16, 0, 0, 0, 0, 0)
    meta = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="meta")   # device -1
    for pages, width in ((4, many), (many, 4)):
        cache = meta(pages, 1, 16, 16)
        with pytest.raises(ValueError, match="2\\^31"):
            binding._paged_cache(cache, cache, meta(1, width, dt=torch.int32), -1, torch.bfloat16,
                                 torch.int32, 1, 16)


def _randn(seed, *shape, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 16)])
@pytest.mark.parametrize("length", [TOP - 65, TOP - 63, TOP - 32])
def test_step_lengths_up_to_2_31(gpu, dtype, d, length):
    """A table of 2^31 - 32 tokens whose entries name one page of 32 over and
    over, beside a sequence of 70 tokens.  A row's weight is its number of
    occurrences times its exponential.

    Bound: the accumulators of the sums and of the outputs take at most two
    additions per tile of 64 tokens, with a whole step of fp32 (2^-23) each, and
    a CTA has its share of the tiles (plus the joins', far fewer than a tenth).
    Weights of bf16 values are rounded by 2^-8 at most, and so is the output."""
    page, width = 32, TOP // 32 - 1
    k, v = (_randn(i, 1, 1, page, d, dtype=dtype) for i in (1, 2))
    v += 1   # (means that are not near zero)
    q = _randn(3, 2, 1, d, dtype=dtype)
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    lens = [length, 70]
    lse = torch.full((2, 1), float("nan"), device="cuda")
    out = torch.full((2, 1, d), float("nan"), dtype=DT[dtype], device="cuda")
    scale = d ** -0.5
    kda.kda_attn_step(q.cuda(), k.cuda(), v.cuda(), table,
                      torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, out, lse)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    additions = 2.2 * (length / 64 / sms + 1)
    for s, n in enumerate(lens):
        count = n // page + (torch.arange(page) < n % page)
        z = scale * (k[0, 0].double() @ q[s, 0].double())
        w = count * torch.exp(z - z.max())
        want = (w @ v[0, 0].double()) / w.sum()
        size = (w @ v[0, 0].double().abs()) / w.sum()
        rel = additions * 2.0 ** -23 + 1e-4
        assert abs(lse[s, 0].item() - (z.max() + w.sum().log()).item()) <= rel + 1e-5
        assert ((out[s, 0].cpu().double() - want).abs() <= (2 * rel + 2.0 ** -7) * size).all()
    # the last row of the table, too, takes a new token
    if length == TOP - 32:
        kc, vc = torch.zeros(1, 1, page, d, dtype=DT[dtype], device="cuda"), v.cuda()
        new = _randn(4, 2, 1, d, dtype=dtype).cuda()
        kda.kda_cache_append(new, new, kc, vc, table,
                             torch.tensor([length - 1, 3], dtype=torch.int32, device="cuda"))
        assert torch.equal(kc[0, 0, 31], new[0, 0]) and torch.equal(kc[0, 0, 3], new[1, 0])


@pytest.mark.gpu
def test_append_of_2_31_less_one_tokens(gpu):
    """The largest token count: all but the first and the last few rows lie
    outside every sequence.  (64 GB of keys, which are the values too.)"""
    T, d, page = TOP - 1, 16, 16
    if torch.cuda.mem_get_info()[0] < 3 * T * d:
        pytest.skip("not enough free memory")
    x = torch.empty(T, 1, d, dtype=torch.bfloat16, device="cuda")
    rows = _randn(1, 6, 1, d, dtype="bf16").cuda()
    x[:3], x[T - 3:] = rows[:3], rows[3:]
    kc = torch.zeros(2, 1, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    for cu, page_of in (((0, 3, 3), 0), ((T - 3, T - 3, T), 1)):
        want = torch.zeros_like(kc)
        want[page_of, 0, 5:8] = rows[:3, 0] if page_of == 0 else rows[3:, 0]
        kc.zero_(), vc.zero_()
        kda.kda_cache_append(x, x, kc, vc, table, i32(5, 5), i32(*cu))
        assert torch.equal(kc, want) and torch.equal(vc, want)
    del x
    torch.cuda.empty_cache()
