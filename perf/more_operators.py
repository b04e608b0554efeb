"""Decoding operators of the full-attention layer that spare its cache's bytes.

* ``append_q8``: rotation of the new queries and keys by their positions, and
  the new keys and values written to a paged cache of 8-bit codes, with one
  scale per token and key-value head;
* ``step_q8``: one new token of every sequence attends to such a cache;
* ``step_shared``: one new token of every sequence of a batch whose sequences
  have their first pages in common, which are read once for all of them.

``run`` computes each in its plain form (``own`` false) or through the
package's entry points (``own`` true).  Caches are
[pages, kv heads, rows of a page, channels], scales [pages, kv heads, rows];
block tables hold, per sequence, the pages of its tokens in order.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SMALLEST = 2.0 ** -100  # rows below this in magnitude are stored as zeros


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the new tokens of a packed prefill batch: q and k rotated, cache filled
        dict(name="append_q8_prompt", op="append_q8", dtype="bf16", lens="8192 1913 512 5767",
             heads=32, kv_heads=8, dim=128, page=64, rot=128, interleaved=False, held=2048),
        # one new token for each of 256 decoding sequences
        dict(name="append_q8_step", op="append_q8", dtype="bf16", lens="1 " * 255 + "1", heads=32,
             kv_heads=8, dim=128, page=16, rot=128, interleaved=False, held=1000),
        # a few single-precision tokens, half of each head rotated in neighbouring pairs
        dict(name="append_q8_f32", op="append_q8", dtype="f32", lens="130 1 403", heads=6,
             kv_heads=2, dim=64, page=32, rot=32, interleaved=True, held=500),
        # a handful of short sequences: call latency
        dict(name="step_q8_tiny", op="step_q8", dtype="bf16", lens="1 17 300 77", heads=8,
             kv_heads=2, dim=64, page=16),
        # a decode batch whose sequences lie between 512 and 8192 tokens
        dict(name="step_q8_batch", op="step_q8", dtype="bf16", lens=_spread(64, 512, 8192),
             heads=32, kv_heads=8, dim=128, page=64),
        # two long conversations: few rows, a long axis
        dict(name="step_q8_long", op="step_q8", dtype="bf16", lens="131072 40007", heads=32,
             kv_heads=8, dim=128, page=64),
        # single-precision queries over the 8-bit cache of a small model
        dict(name="step_q8_f32", op="step_q8", dtype="f32", lens=_spread(16, 200, 2000), heads=8,
             kv_heads=4, dim=64, page=32),
        # three short sequences after a short common instruction: call latency
        dict(name="shared_tiny", op="step_shared", dtype="bf16", shared=192, lens="1 50 23",
             heads=8, kv_heads=2, dim=64, page=16),
        # a service's system prompt, 64 conversations at different lengths behind it
        dict(name="shared_system", op="step_shared", dtype="bf16", shared=4096,
             lens=_spread(64, 100, 1500), heads=32, kv_heads=8, dim=128, page=64),
        # one long document, 24 questions about it under way
        dict(name="shared_document", op="step_shared", dtype="bf16", shared=65536,
             lens=_spread(24, 1, 700), heads=32, kv_heads=8, dim=128, page=64),
        # many answers sampled for one prompt: more rows than the cache's bytes can hide
        dict(name="shared_samples", op="step_shared", dtype="bf16", shared=16384,
             lens=_spread(256, 1, 600), heads=32, kv_heads=8, dim=128, page=64),
        # single-precision decoding of a small model, some examples in front
        dict(name="shared_f32", op="step_shared", dtype="f32", shared=1024,
             lens=_spread(12, 1, 200), heads=6, kv_heads=2, dim=64, page=32),
    ]


def _spread(n, lo, hi):
    """n lengths spread over [lo, hi] in no order (a fixed multiplicative walk)."""
    out, x = [], 12345
    for _ in range(n):
        x = (x * 48271) % 2147483647
        out.append(lo + x % (hi - lo + 1))
    return " ".join(map(str, out))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append_q8", "step_q8", "step_shared", "step_shared"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    kv = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
    while kv * group > 40:
        group = rng.choice((1, 2, 3, 4, 5, 7, 8))
    dim = rng.choice((64, 128, 64, 128, 32, 16)) if dtype == "f32" else rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128))
    case = dict(op=op, dtype=dtype, heads=kv * group, kv_heads=kv, dim=dim, page=page)
    if op == "append_q8":
        n = _log(rng, 1, 256)
        most = max(1, _log(rng, 1, 16000) // n)
        case["lens"] = " ".join(str(rng.randint(1, most)) for _ in range(n))
        case["rot"] = rng.choice((dim, dim, max(16, dim // 2)))
        case["interleaved"] = rng.random() < 0.4
        case["held"] = _log(rng, 1, min(8000, 250000 // n))
    elif op == "step_q8":
        n = _log(rng, 1, 128)
        most = max(1, _log(rng, 16, (60000 if dtype == "f32" else 250000)) // n)
        # a batch may hold rows without a sequence
        case["lens"] = " ".join(str(rng.randint(0 if i % 9 == 4 else 1, 2 * most))
                                for i in range(n))
    else:
        n = _log(rng, 1, 64 if dtype == "f32" else 256)
        most = max(1, _log(rng, 4, 60000) // n)
        longest = 4000 if dtype == "f32" else min(65536, 3200000 // n)
        case["shared"] = page * _log(rng, 1, longest // page)
        case["lens"] = " ".join(str(rng.randint(0 if i % 9 == 4 else 1, 2 * most))
                                for i in range(n))
    return case


def _lens(case):
    return [int(x) for x in case["lens"].split()]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    lens = _lens(case)
    t, hq, hkv, d = sum(lens), case["heads"], case["kv_heads"], case["dim"]
    n = len(lens)
    if case["op"] == "append_q8":
        # q in and out; k and v in, as codes and scales to the cache, and out as
        # the values that those stand for
        return {"bytes": es * t * d * (2 * hq + 4 * hkv) + t * hkv * (2 * d + 8)
                + 4 * t * case["rot"],
                "flops": 3 * t * case["rot"] * (hq + hkv) + 6 * t * hkv * d}
    if case["op"] == "step_q8":
        return {"bytes": t * hkv * (2 * d + 8) + es * 2 * n * hq * d + 4 * n * hq,
                "flops": 4 * d * hq * t}
    s = case["shared"]
    return {"bytes": es * d * (2 * (s + t) * hkv + 2 * n * hq) + 4 * n * hq,
            "flops": 4 * d * hq * (n * s + t)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 29)
    dt = _DTYPES[case["dtype"]]
    lens = _lens(case)
    n, hq, hkv, d, page = len(lens), case["heads"], case["kv_heads"], case["dim"], case["page"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    st = dict(case=case, scale=d ** -0.5)
    if case["op"] == "append_q8":
        # tokens that each sequence holds already: up to `held`
        held = [int(x) for x in _spread(n, 0, case["held"]).split()]
    elif case["op"] == "step_q8":
        held = lens
    else:
        # every sequence's tokens behind the shared ones
        held = [case["shared"] + x for x in lens]
    after = [h + x for h, x in zip(held, lens)] if case["op"] == "append_q8" else held
    need = [(x + page - 1) // page for x in after]
    common = case["shared"] // page if case["op"] == "step_shared" else 0
    pages = sum(need) - (n - 1) * common + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, max(max(need), 1)), -1, dtype=torch.int32, device=dev)
    table[:, :common] = order[:common]
    at = common
    for s, m in enumerate(need):
        table[s, common:m] = order[at:at + m - common]
        at += m - common
    st["held"] = torch.tensor(held, dtype=torch.int32, device=dev)
    st["table"] = table
    if case["op"] == "step_shared":
        st["q"] = randn(n, hq, d)
        st["k_cache"], st["v_cache"] = randn(pages, hkv, page, d), randn(pages, hkv, page, d)
        st["shared_pages"] = torch.tensor([common], dtype=torch.int32, device=dev)
        st["lse"] = torch.empty((n, hq), device=dev)
        return st
    # what the cache holds: codes of rows whose largest is 127
    shape = (pages, hkv, page, d)
    for x in ("k", "v"):
        codes = torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8)
        st[x + "_cache"] = codes
        st[x + "_scale"] = (2.5 + torch.rand(shape[:3], generator=g, device=dev)) / 127
    if case["op"] == "step_q8":
        st["q"] = randn(n, hq, d)
        st["lse"] = torch.empty((n, hq), device=dev)
        return st
    t = sum(lens)
    # a few channels of the keys are larger than the others
    st["q"], st["v"] = randn(t, hq, d), randn(t, hkv, d)
    wide = torch.randn(hkv, d, generator=g, device=dev).mul(0.5).exp()
    st["k"] = (randn(t, hkv, d) * wide).to(dt)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st["cu"] = None if t == n else torch.tensor(cu, dtype=torch.int32, device=dev)
    # each token's sequence and position
    st["seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor(lens)).to(dev)
    first = torch.tensor([h - c for h, c in zip(held, cu)]).to(dev)
    st["pos"] = first[st["seq"]] + torch.arange(t, device=dev)
    half = case["rot"] // 2
    p = torch.arange(case["held"] + max(lens) + 1, dtype=torch.float64, device=dev)
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    ang = p[:, None] * freq[None, :]
    st["rope"] = torch.cat((ang.cos(), ang.sin()), dim=1).float()
    st["q_out"] = torch.empty_like(st["q"])
    st["k_stored"], st["v_stored"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        return {"append_q8": _own_append, "step_q8": _own_step, "step_shared": _own_shared}[op](st)
    return {"append_q8": _plain_append, "step_q8": _plain_step, "step_shared": _plain_shared}[op](st)


def _own_append(st):
    import kimi_delta_attention_chunkwise_gb300 as kda
    kda.kda_cache_append_q8(st["k"], st["v"], st["k_cache"], st["v_cache"], st["k_scale"],
                            st["v_scale"], st["table"], st["held"], st["cu"], q=st["q"],
                            q_out=st["q_out"], k_stored=st["k_stored"], v_stored=st["v_stored"],
                            rope=st["rope"], rope_interleaved=st["case"]["interleaved"])
    return _append_outputs(st)


def _own_step(st):
    import kimi_delta_attention_chunkwise_gb300 as kda
    return kda.kda_attn_step_q8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"],
                                st["v_scale"], st["table"], st["held"], st["scale"], None,
                                st["lse"])


def _own_shared(st):
    import kimi_delta_attention_chunkwise_gb300 as kda
    return kda.kda_attn_step_shared(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                    st["held"], st["shared_pages"], st["scale"], None, st["lse"])


def _append_outputs(st):
    # the new rows' values, and the whole updated cache as it lies
    return [st["q_out"], st["k_stored"], st["v_stored"], st["k_scale"], st["v_scale"],
            st["k_cache"], st["v_cache"]]


def _plain_append(st):
    case = st["case"]
    page, rot, pos = case["page"], case["rot"], st["pos"]
    cos, sin = st["rope"][pos].split(rot // 2, dim=1)
    cos, sin = cos[:, None], sin[:, None]

    def rotate(x):
        y = x.float().clone()
        if case["interleaved"]:
            a, b = slice(0, rot, 2), slice(1, rot, 2)
        else:
            a, b = slice(0, rot // 2), slice(rot // 2, rot)
        xa, xb = x[..., a].float(), x[..., b].float()
        y[..., a] = xa * cos - xb * sin
        y[..., b] = xb * cos + xa * sin
        return y

    def quantise(x):
        top = x.abs().amax(dim=-1)
        most = torch.full_like(top, 127.0)
        small = top < _SMALLEST
        scale = torch.where(small, torch.zeros_like(top), torch.div(top, most))
        turn = torch.where(small, torch.zeros_like(top), torch.div(most, top))
        return torch.round(x * turn[..., None]), scale

    st["q_out"].copy_(rotate(st["q"]).to(st["q"].dtype))
    where = st["table"][st["seq"], pos // page].long()
    row = pos % page
    kc, ks = quantise(rotate(st["k"]))
    vc, vs = quantise(st["v"].float())
    st["k_cache"][where, :, row] = kc.to(torch.int8)
    st["v_cache"][where, :, row] = vc.to(torch.int8)
    st["k_scale"][where, :, row] = ks
    st["v_scale"][where, :, row] = vs
    st["k_stored"].copy_((kc * ks[..., None]).to(st["k"].dtype))
    st["v_stored"].copy_((vc * vs[..., None]).to(st["v"].dtype))
    return _append_outputs(st)


def _rows(cache, table, first, count, scale=None):
    """Tokens [first, first + count) of every row of `table`: [N, HKV, count, d], in float32."""
    page = cache.shape[2]
    at = first + torch.arange(count, device=cache.device)
    block = table[:, at // page].long().clamp(min=0)
    row = at % page
    x = cache[block, :, row].float()              # [N, count, HKV, d]
    if scale is not None:
        x = x * scale[block, :, row][..., None]
    return x.transpose(1, 2)


def _softmax(z, lens, first):
    """Weights (not divided by their sum), sums and log of the sums of scores z
    [N, HKV, G, L] of the keys from `first` on, of which a row sees those before lens."""
    j = first + torch.arange(z.shape[-1], device=z.device)
    z = z.masked_fill(j >= lens[:, None, None, None], float("-inf"))
    m = z.amax(dim=-1, keepdim=True) if z.shape[-1] else z.new_full(z.shape[:3] + (1,), -math.inf)
    p = torch.exp(z - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return p, m


def _finish(st, o, l, m):
    """out = o / l (0 for a row without keys), lse."""
    n, hq = st["q"].shape[:2]
    out = torch.where(l > 0, o / l, torch.zeros_like(o)).reshape(st["q"].shape)
    st["lse"].copy_((m + torch.log(l)).reshape(n, hq))
    return out.to(st["q"].dtype), st["lse"]


def _queries(st):
    n, hq, d = st["q"].shape
    hkv = st["case"]["kv_heads"]
    return st["q"].float().view(n, hkv, hq // hkv, d)


def _plain_step(st):
    q = _queries(st)
    # the longest length that the table has room for
    most = st["table"].shape[1] * st["case"]["page"]
    k = _rows(st["k_cache"], st["table"], 0, most, st["k_scale"])
    z = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    del k
    p, m = _softmax(z, st["held"], 0)
    v = _rows(st["v_cache"], st["table"], 0, most, st["v_scale"])
    return _finish(st, torch.matmul(p, v), p.sum(dim=-1, keepdim=True), m)


def _plain_shared(st):
    q, table, s = _queries(st), st["table"], st["case"]["shared"]
    n, hkv, g, d = q.shape
    most = table.shape[1] * st["case"]["page"] - s
    # the shared keys against all rows of a kv head at once, each row's own keys by themselves
    kp, vp = (_rows(st[x], table[:1], 0, s)[0] for x in ("k_cache", "v_cache"))
    ko, vo = (_rows(st[x], table, s, most) for x in ("k_cache", "v_cache"))
    rows = q.transpose(0, 1).reshape(hkv, n * g, d)
    z = torch.matmul(rows, kp.transpose(1, 2)).view(hkv, n, g, s).transpose(0, 1) * st["scale"]
    p, m = _softmax(z, st["held"], 0)
    po, mo = _softmax(torch.matmul(q, ko.transpose(2, 3)) * st["scale"], st["held"], s)
    top = torch.maximum(m, mo)
    f, fo = torch.exp(m - top), torch.exp(mo - top)
    o = torch.matmul(p.transpose(0, 1).reshape(hkv, n * g, s), vp)
    o = o.view(hkv, n, g, d).transpose(0, 1) * f + torch.matmul(po, vo) * fo
    l = p.sum(dim=-1, keepdim=True) * f + po.sum(dim=-1, keepdim=True) * fo
    return _finish(st, o, l, top)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append_q8":
        return _exact_append(st)
    # 4 d flops of 64-bit products per (row, key, head): too long past this
    if work(case)["flops"] > 6e12:
        return None
    hq, page = case["heads"], case["page"]
    group = hq // case["kv_heads"]
    q = st["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for s, n in enumerate(st["held"].tolist()):
        if n == 0:
            continue
        token = torch.arange(n, device=q.device)
        block, row = st["table"][s].long()[token // page], token % page
        for c in range(case["kv_heads"]):
            heads = slice(c * group, (c + 1) * group)
            k, v = (st[x][block, c, row].double() for x in ("k_cache", "v_cache"))
            if case["op"] == "step_q8":
                k *= st["k_scale"][block, c, row].double()[:, None]
                v *= st["v_scale"][block, c, row].double()[:, None]
            z = st["scale"] * (q[s, heads] @ k.T)
            lse[s, heads] = torch.logsumexp(z, dim=1)
            out[s, heads] = (z - lse[s, heads, None]).exp() @ v
    return out, lse


def _exact_append(st):
    case = st["case"]
    page, rot = case["page"], case["rot"]
    half = rot // 2
    q, k, v = (st[x].double() for x in ("q", "k", "v"))
    # a rotation of a pair is a product of complex numbers
    turn = torch.complex(st["rope"][:, :half].double(), st["rope"][:, half:].double())
    w = turn[st["pos"]][:, None]
    for x in (q, k):
        part = x[..., :rot]
        if case["interleaved"]:
            y = torch.view_as_complex(part.reshape(*part.shape[:2], half, 2).contiguous()) * w
            x[..., :rot] = torch.view_as_real(y).reshape(part.shape)
        else:
            y = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * w
            x[..., :rot] = torch.cat((y.real, y.imag), dim=-1)
    flat = st["table"][st["seq"], st["pos"] // page].long() * page + st["pos"] % page
    scales, stored = [], []
    for x, before in ((k, st["k_scale"]), (v, st["v_scale"])):
        step = x.abs().amax(dim=-1) / 127.0
        by_row = before.double().transpose(1, 2).reshape(-1, before.shape[1])
        by_row[flat] = step
        scales.append(by_row.view(before.shape[0], page, -1).transpose(1, 2))
        # (a value on the border between two codes may go either way in 32 bits: within what a
        # 16-bit result may be off by, not a 32-bit one)
        stored.append(torch.round(x / step[..., None]) * step[..., None]
                      if case["dtype"] == "bf16" else None)
    return [q, *stored, *scales, None, None]
