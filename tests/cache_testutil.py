"""Caches for the tests of the step's other forms, and the bounds their results keep.

Bounds: those of attn_testutil, with
  * the products' rounding one step larger where a score is multiplied by a
    row's scale, (d + 9) u Z1, and one step more on the weights' sums;
  * the weights' own rounding as a number: 2^-15 where they go to the tensor core
    as two bf16 parts, 2^-8 as one (half a step of bf16), 0 in fp32.
"""
import torch

from attn_testutil import U, reference, tables

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TWO_PARTS, ONE_PART, FP32 = 2.0 ** -15, 2.0 ** -8, 0.0
SMALLEST = 2.0 ** -100


def randn(seed, *shape, dtype="f32"):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lens, start=0):
    c = [start]
    for n in lens:
        c.append(c[-1] + n)
    return i32(c)


def mma(dtype, d):
    return dtype == "bf16" and d in (64, 128)


def check(out, lse, ref, keys, d, weights):
    """attn_testutil.check with the bounds above; ref = (out, A, lse, Z1)."""
    o, A, z, z1 = ref
    dz = (d + 9) * U * z1
    ex = 4 * U * (2 * z1 + 2)
    rel = 2 * (dz + ex) + 2 * (keys + 17) * U + weights
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    got = out.detach().cpu().double()
    assert not torch.isnan(got).any()
    tol = rel[..., None] * A + half * o.abs() * (1 + rel[..., None]) + 1e-37
    over = (got - o).abs() - tol
    assert over.max().item() <= 0, \
        f"out off by {(got - o).abs().max().item():.3g}, {over.max().item():.3g} past the bound"
    if lse is not None:
        g = lse.detach().cpu().double()
        tl = dz + ex + (keys + 16) * U + U * (z.abs() + 1)
        assert ((g - z).abs() <= tl).all(), f"lse off by {(g - z).abs().max().item():.3g}"


def check_rows(q, ks, vs, scale, out, lse, weights):
    """Row s of q attends to ks[s], vs[s] [L, HKV, d] (any type; L = 0: out 0, lse -inf)."""
    for s in range(q.shape[0]):
        n = ks[s].shape[0]
        if n == 0:
            assert (out[s] == 0).all()
            assert lse is None or (lse[s] == -float("inf")).all()
            continue
        check(out[s:s + 1], None if lse is None else lse[s:s + 1],
              reference(q[s:s + 1], ks[s], vs[s], scale, n - 1), n, q.shape[2], weights)


# ---------------------------------------------------------------------------
# 8-bit codes
# ---------------------------------------------------------------------------
def encode(x):
    """Codes (float32 whole numbers) and scales of rows x [..., d], operation by
    operation in fp32 on the CPU."""
    x = x.float()
    top = x.abs().amax(dim=-1)
    bad = ~torch.isfinite(x).all(dim=-1)
    most = torch.full_like(top, 127.0)
    scale, turn = torch.div(top, most), torch.div(most, top)
    small = top < SMALLEST
    scale[small] = turn[small] = 0.0
    codes = torch.round(x * turn[..., None])
    codes[small] = 0.0
    scale[bad] = float("nan")
    codes[bad] = 0.0
    return codes, scale


def put(cache, rows, table, held, lens):
    """cache [P, HKV, page, ...] with rows [sum(lens), HKV, ...] put in place."""
    page, t = cache.shape[2], 0
    for s, n in enumerate(lens):
        for i in range(n):
            p = held[s] + i
            b = int(table[s, p // page])
            if b >= 0:
                cache[b, :, p % page] = rows[t]
            t += 1
    return cache


def paged_q8(seed, lens, HKV, d, page):
    """A cache of random codes and scales for the lengths; behind them codes of
    -128 (which no call writes) and scales of NaN.  (dequantised k and v rows
    per sequence in float64, (k, v, k_scale, v_scale) on the GPU, table)."""
    need = [(n + page - 1) // page for n in lens]
    table, pages = tables(need, max(max(need), 1) + 1, seed=seed)
    g = torch.Generator().manual_seed(seed)
    codes = [torch.full((pages, HKV, page, d), -128, dtype=torch.int8) for _ in range(2)]
    scales = [torch.full((pages, HKV, page), float("nan")) for _ in range(2)]
    rows = [[], []]
    for s, n in enumerate(lens):
        for i in range(2):
            c = torch.randint(-127, 128, (n, HKV, d), generator=g, dtype=torch.int8)
            f = (0.5 + 3 * torch.rand(n, HKV, generator=g)) / 127
            rows[i].append(c.double() * f.double()[..., None])
            for j in range(need[s]):
                m = min(page, n - j * page)
                at = slice(j * page, j * page + m)
                codes[i][int(table[s, j]), :, :m] = c[at].transpose(0, 1)
                scales[i][int(table[s, j]), :, :m] = f[at].transpose(0, 1)
    return rows[0], rows[1], tuple(x.cuda() for x in (*codes, *scales)), table.cuda()


def widen(table, width=16384):
    wide = torch.full((table.shape[0], width), -1, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    return wide


# ---------------------------------------------------------------------------
# caches whose first pages are shared
# ---------------------------------------------------------------------------
def paged_shared(seed, common, lens, HKV, d, page, dtype, garbage=float("nan")):
    """Sequences of lens[s] tokens whose first `common` pages are the same ones
    for those that hold them whole (the others have pages of their own from the
    first token on, and what they leave of their row of the table names no page).
    `garbage` lies behind every length.  (k, v rows per sequence, k cache, v cache,
    table)."""
    need = [(n + page - 1) // page for n in lens]
    holds = [n >= common * page for n in lens]
    own = [m - common if h else m for m, h in zip(need, holds)]
    g = torch.Generator().manual_seed(seed)
    pages = common + sum(own) + 2
    order = torch.randperm(pages, generator=g).to(torch.int32)
    width = max(max(need), common, 1) + 1
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    caches = [torch.full((pages, HKV, page, d), garbage, dtype=DT[dtype]) for _ in range(2)]
    first = [torch.randn(common * page, HKV, d, generator=g).to(DT[dtype]) for _ in range(2)]
    for c, f in zip(caches, first):
        for j in range(common):
            c[int(order[j])] = f[j * page:(j + 1) * page].transpose(0, 1)
    rows, at = [[], []], common
    for s, n in enumerate(lens):
        start = common if holds[s] else 0
        table[s, :start] = order[:start]
        table[s, start:need[s]] = order[at:at + own[s]]
        at += own[s]
        m = n - start * page
        for c, f, r in zip(caches, first, rows):
            x = torch.randn(m, HKV, d, generator=g).to(DT[dtype])
            r.append(torch.cat((f[:start * page], x)))
            for j in range(own[s]):
                e = min(page, m - j * page)
                c[int(table[s, start + j]), :, :e] = x[j * page:j * page + e].transpose(0, 1)
    return rows[0], rows[1], caches[0].cuda(), caches[1].cuda(), table.cuda()
