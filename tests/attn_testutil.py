"""The full-attention layer in 64 bits, element by element, and the error
bounds its tests use.

Bounds.  With z = scale <q, k>, p = softmax(z) and A = sum_j p_j |v_j| (per
output element), a computed output differs from the exact one by at most

  * the dot product's rounding: |dz| <= (d + 8) u Z1, with
    Z1 = scale * max_j sum_c |q_c k_jc| and u = 2^-23 (an fp32 sum, the tensor
    core's among them, may truncate: a whole step per addition);
  * the exponent's argument and the exponential: 4 u (Z2 + 2) relative, with
    Z2 = max_j |z_j - max z| <= 2 Z1, and both enter numerator and
    denominator: 2 (|dz| + 4 u (2 Z1 + 2)) A;
  * the two sums over the keys, u per addition: 2 (L + 16) u A;
  * where the weights are rounded to bf16 for their product with v: 2^-8 A;
  * the final rounding, half a step of the output type: 2^-8 |o| for bf16,
    2^-24 |o| for fp32.

lse carries |dz| + 4 u (2 Z1 + 2), the sum's L u and its own rounding
u (|lse| + 1).
"""
import torch

U = 2.0 ** -23


def reference(q, k, v, scale, first):
    """q [R, HQ, d] (row r sees keys 0 .. first + r), k, v [L, HKV, d] ->
    out, A [R, HQ, d], lse, Z1 [R, HQ], all float64 on the CPU.  A key that a
    row does not see is left out of its sums altogether."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    R, HQ, d = q.shape
    L, HKV, _ = k.shape
    G = HQ // HKV
    out = torch.zeros(R, HQ, d, dtype=torch.float64)
    A, lse, z1 = torch.zeros_like(out), torch.full((R, HQ), -float("inf"), dtype=torch.float64), \
        torch.zeros(R, HQ, dtype=torch.float64)
    finite = bool(torch.isfinite(k).all() and torch.isfinite(v).all())
    step = R if finite else 1
    for h in range(HQ):
        kh, vh = k[:, h // G], v[:, h // G]
        for r in range(0, R, step):
            e = min(R, r + step)
            n = min(first + e, L)
            if n <= 0:
                continue
            z = scale * (q[r:e, h] @ kh[:n].T)
            keep = torch.arange(n)[None, :] <= (torch.arange(r, e) + first)[:, None]
            z = torch.where(keep, z, torch.full_like(z, -float("inf")))
            m = z.max(dim=1, keepdim=True).values
            p = torch.exp(z - m)
            s = p.sum(dim=1, keepdim=True)
            lse[r:e, h] = (m + torch.log(s))[:, 0]
            out[r:e, h] = (p / s) @ vh[:n]
            A[r:e, h] = (p / s) @ vh[:n].abs()
            z1[r:e, h] = scale * (q[r:e, h].abs() @ kh[:n].abs().T).max(dim=1).values
    return out, A, lse, z1


def check(out, lse, ref, keys, d, weights_bf16):
    """Asserts the bounds above for [R, HQ, d] outputs; keys: the longest row."""
    o, A, z, z1 = ref
    dz = (d + 8) * U * z1
    ex = 4 * U * (2 * z1 + 2)
    rel = 2 * (dz + ex) + 2 * (keys + 16) * U + (2.0 ** -8 if weights_bf16 else 0.0)
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    got = out.detach().cpu().double()
    tol = rel[..., None] * A + half * o.abs() * (1 + rel[..., None]) + 1e-37
    over = (got - o).abs() - tol
    assert not torch.isnan(got).any()
    assert over.max().item() <= 0, \
        f"out off by {(got - o).abs().max().item():.3g}, {over.max().item():.3g} past the bound"
    if lse is not None:
        g = lse.detach().cpu().double()
        none = torch.isinf(z)
        assert torch.equal(g[none], z[none])
        tl = dz + ex + (keys + 16) * U + U * (z.abs() + 1)
        assert ((g - z).abs()[~none] <= tl[~none]).all(), \
            f"lse off by {(g - z).abs()[~none].max().item():.3g}"


def rope_table(positions, rot, base=10000.0):
    half = rot // 2
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * \
        base ** (-torch.arange(half, dtype=torch.float64) / half)[None, :]
    return torch.cat((ang.cos(), ang.sin()), dim=1).float()


def rotate(x, pos, table, interleaved):
    """x [T, H, d] rotated by the rows `pos` of the table, each product and
    sum rounded to fp32, then once to x's type (CPU)."""
    rot = table.shape[1]
    cos, sin = table[pos, :rot // 2][:, None], table[pos, rot // 2:][:, None]
    y = x.float().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    xa, xb = x[..., a].float(), x[..., b].float()
    y[..., a] = xa * cos - xb * sin
    y[..., b] = xb * cos + xa * sin
    return y.to(x.dtype)


def tables(need, width, spare=2, seed=0):
    """Block tables with `need[s]` pages for sequence s in shuffled order, -1
    behind them; returns (table [N, width] int32, number of pages)."""
    g = torch.Generator().manual_seed(seed)
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    t = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for s, m in enumerate(need):
        t[s, :m] = order[at:at + m]
        at += m
    return t, pages
