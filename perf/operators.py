"""The full-attention layer's operators, as a serving program calls them.

Three operators that run together in the softmax-attention layers of a stack
whose other layers are KDA:

* ``prompt``: causal attention over whole packed prompts with grouped heads;
* ``append``: rotation of the new queries and keys by their positions, and
  the new keys and values written to a paged cache;
* ``step``: one new token of every sequence attends to its paged cache.

``run`` computes each in its plain form (``own`` false) or through the
package's entry points (``own`` true).  Caches are
[pages, kv heads, rows of a page, channels]; block tables hold, per sequence,
the pages of its tokens in order.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # three very short prompts of an interactive service: call latency
        dict(name="prompt_tiny", op="prompt", dtype="bf16", lens="5 1 33", heads=8, kv_heads=2,
             dim=64),
        # one 4096-token prompt, 16 heads that share nothing
        dict(name="prompt_4096x16", op="prompt", dtype="bf16", lens="4096", heads=16, kv_heads=16,
             dim=128),
        # a packed prefill batch of ragged prompts between 512 and 8192 tokens
        dict(name="prompt_packed", op="prompt", dtype="bf16",
             lens="1913 8192 512 5127 700 6400 2751 3001", heads=32, kv_heads=8, dim=128),
        # one long document
        dict(name="prompt_long", op="prompt", dtype="bf16", lens="16384", heads=32, kv_heads=8,
             dim=128),
        # single-precision checks of a small model
        dict(name="prompt_f32", op="prompt", dtype="f32", lens="300 701 24", heads=6, kv_heads=2,
             dim=64),
        # the new tokens of a packed prefill batch: q and k rotated, cache filled
        dict(name="append_prompt", op="append", dtype="bf16", lens="8192 1913 512 5767", heads=32,
             kv_heads=8, dim=128, page=64, rot=128, interleaved=False, held=2048, keep_k=True),
        # one new token for each of 256 decoding sequences
        dict(name="append_step", op="append", dtype="bf16", lens="1 " * 255 + "1", heads=32,
             kv_heads=8, dim=128, page=16, rot=128, interleaved=False, held=1000, keep_k=False),
        # a few single-precision tokens, half of each head rotated in neighbouring pairs
        dict(name="append_f32", op="append", dtype="f32", lens="130 1 403", heads=6, kv_heads=2,
             dim=64, page=32, rot=32, interleaved=True, held=500, keep_k=True),
        # a handful of short sequences: call latency
        dict(name="step_tiny", op="step", dtype="bf16", lens="1 17 300 77", heads=8, kv_heads=2,
             dim=64, page=16),
        # a decode batch whose sequences lie between 512 and 8192 tokens
        dict(name="step_batch", op="step", dtype="bf16", lens=_spread(64, 512, 8192), heads=32,
             kv_heads=8, dim=128, page=64),
        # two long conversations: few rows, a long axis
        dict(name="step_long", op="step", dtype="bf16", lens="131072 40007", heads=32, kv_heads=8,
             dim=128, page=64),
        # single-precision decoding
        dict(name="step_f32", op="step", dtype="f32", lens=_spread(16, 200, 2000), heads=8,
             kv_heads=4, dim=64, page=32),
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
    op = rng.choice(("prompt", "append", "step"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    kv = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
    while kv * group > 40:
        group = rng.choice((1, 2, 3, 4, 5, 7, 8))
    dim = rng.choice((64, 128, 64, 128, 32, 16)) if dtype == "f32" else rng.choice((64, 128))
    case = dict(op=op, dtype=dtype, heads=kv * group, kv_heads=kv, dim=dim)
    if op == "prompt":
        total = _log(rng, 8, 2000 if dtype == "f32" else 16000)
        n = min(total, _log(rng, 1, 24))
        cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        case["lens"] = " ".join(str(x) for x in lens if x > 0)
    elif op == "append":
        n = _log(rng, 1, 256)
        most = max(1, _log(rng, 1, 16000) // n)
        case["lens"] = " ".join(str(rng.randint(1, most)) for _ in range(n))
        case["page"] = rng.choice((16, 32, 64, 128))
        case["rot"] = rng.choice((dim, dim, dim // 2))
        case["interleaved"] = rng.random() < 0.4
        case["held"] = _log(rng, 1, min(8000, 250000 // n))
        case["keep_k"] = rng.random() < 0.5
    else:
        n = _log(rng, 1, 128)
        most = max(1, _log(rng, 16, (60000 if dtype == "f32" else 250000)) // n)
        case["lens"] = " ".join(str(rng.randint(1, 2 * most)) for _ in range(n))
        case["page"] = rng.choice((16, 32, 64, 128))
    return case


def _lens(case):
    return [int(x) for x in case["lens"].split()]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    lens = _lens(case)
    t, hq, hkv, d = sum(lens), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        return {"bytes": es * t * d * (2 * hq + 2 * hkv) + 4 * t * hq,
                "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    if case["op"] == "append":
        # q in and out; k and v in and to the cache; k once more where it is kept
        rows = 2 * hq + 4 * hkv + (hkv if case["keep_k"] else 0)
        return {"bytes": es * t * d * rows + 4 * t * case["rot"],
                "flops": 3 * t * case["rot"] * (hq + hkv)}
    n = len(lens)
    return {"bytes": es * d * (2 * t * hkv + 2 * n * hq) + 4 * n * hq,
            "flops": 4 * d * hq * t}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 17)
    dt = _DTYPES[case["dtype"]]
    lens = _lens(case)
    n, hq, hkv, d = len(lens), case["heads"], case["kv_heads"], case["dim"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    st = dict(case=case, lens=lens, scale=d ** -0.5)
    if case["op"] != "step":
        t = sum(lens)
        st["q"], st["k"], st["v"] = randn(t, hq, d), randn(t, hkv, d), randn(t, hkv, d)
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        st["cu_host"] = cu
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["op"] == "prompt":
        st["lse"] = torch.empty((t, hq), device=dev)
        return st
    page = case["page"]
    if case["op"] == "append":
        # tokens that each sequence holds already: up to `held`
        held = [int(x) for x in _spread(n, 0, case["held"]).split()]
        need = [(h + x + page - 1) // page for h, x in zip(held, lens)]
    else:
        st["q"] = randn(n, hq, d)
        held = lens
        need = [(x + page - 1) // page for x in lens]
    pages = sum(need) + 3
    width = max(need)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    st["held_host"] = held
    st["held"] = torch.tensor(held, dtype=torch.int32, device=dev)
    st["table"] = table
    if case["op"] == "append":
        # the pages hold what was there before; only the new rows change
        st["k_cache"], st["v_cache"] = randn(pages, hkv, page, d), randn(pages, hkv, page, d)
        half = case["rot"] // 2
        pos = torch.arange(case["held"] + max(lens) + 1, dtype=torch.float64, device=dev)
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        ang = pos[:, None] * freq[None, :]
        st["rope"] = torch.cat((ang.cos(), ang.sin()), dim=1).float()
        st["q_out"] = torch.empty_like(st["q"])
        st["k_out"] = torch.empty_like(st["k"]) if case["keep_k"] else None
    else:
        st["k_cache"], st["v_cache"] = randn(pages, hkv, page, d), randn(pages, hkv, page, d)
        st["lse"] = torch.empty((n, hq), device=dev)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "append": _own_append, "step": _own_step}[op](st)
    return {"prompt": _plain_prompt, "append": _plain_append, "step": _plain_step}[op](st)


def _own_prompt(st):
    import kimi_delta_attention_chunkwise_gb300 as kda
    return kda.kda_attn_fwd(st["q"], st["k"], st["v"], st["scale"], st["cu"], None, st["lse"])


def _own_append(st):
    import kimi_delta_attention_chunkwise_gb300 as kda
    # one token of each sequence needs no offsets
    cu = None if len(st["lens"]) == st["q"].shape[0] else st["cu"]
    kda.kda_cache_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["held"],
                         cu, q=st["q"], q_out=st["q_out"], k_out=st["k_out"],
                         rope=st["rope"], rope_interleaved=st["case"]["interleaved"])
    return _append_outputs(st)


def _own_step(st):
    import kimi_delta_attention_chunkwise_gb300 as kda
    return kda.kda_attn_step(st["q"], st["k_cache"], st["v_cache"], st["table"], st["held"],
                             st["scale"], None, st["lse"])


def _append_outputs(st):
    out = [st["q_out"], st["k_cache"], st["v_cache"]]
    if st["k_out"] is not None:
        out.append(st["k_out"])
    return out


def _plain_attend(q, k, v, scale, first):
    """Rows of q [R, HQ, d] (row r sees keys 0 .. first + r) against k, v
    [L, HKV, d], all float32 -> out [R, HQ, d], lse [R, HQ]."""
    rows, hq, d = q.shape
    keys, hkv, _ = k.shape
    qg = q.view(rows, hkv, hq // hkv, d).permute(1, 2, 0, 3)      # [HKV, G, R, d]
    s = torch.matmul(qg, k.permute(1, 2, 0)[:, None]) * scale     # [HKV, G, R, L]
    if first + 1 < keys:
        i = torch.arange(rows, device=q.device)[:, None] + first
        j = torch.arange(keys, device=q.device)[None, :]
        s = s.masked_fill(j > i, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v.permute(1, 0, 2)[:, None]) / l
    lse = (m + torch.log(l))[..., 0]
    return o.permute(2, 0, 1, 3).reshape(rows, hq, d), lse.permute(2, 0, 1).reshape(rows, hq)


def _plain_prompt(st):
    q, k, v, cu = st["q"].float(), st["k"].float(), st["v"].float(), st["cu_host"]
    out = torch.empty_like(st["q"])
    lse = st["lse"]
    for a, b in zip(cu, cu[1:]):
        # blocks of queries that keep the scores of all heads within 2 GB
        step = max(64, (1 << 29) // (q.shape[1] * (b - a)))
        for r in range(a, b, step):
            e = min(b, r + step)
            o, z = _plain_attend(q[r:e], k[a:e], v[a:e], st["scale"], r - a)
            out[r:e] = o.to(out.dtype)
            lse[r:e] = z
    return out, lse


def _plain_append(st):
    case, dev = st["case"], st["q"].device
    page, rot = case["page"], case["rot"]
    pos = torch.cat([torch.arange(h, h + n) for h, n in zip(st["held_host"], st["lens"])])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(st["lens"])])
    pos, seq = pos.to(dev), seq.to(dev)
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
        return y.to(x.dtype)

    k = rotate(st["k"])
    st["q_out"].copy_(rotate(st["q"]))
    where = st["table"][seq, pos // page].long()
    st["k_cache"][where, :, pos % page] = k
    st["v_cache"][where, :, pos % page] = st["v"]
    if st["k_out"] is not None:
        st["k_out"].copy_(k)
    return _append_outputs(st)


def _plain_step(st):
    q, page = st["q"].float(), st["case"]["page"]
    out, lse = torch.empty_like(st["q"]), st["lse"]
    hkv, d = st["k_cache"].shape[1], st["k_cache"].shape[3]
    for s, n in enumerate(st["lens"]):
        used = st["table"][s, :(n + page - 1) // page].long()
        k = st["k_cache"][used].float().transpose(1, 2).reshape(-1, hkv, d)[:n]
        v = st["v_cache"][used].float().transpose(1, 2).reshape(-1, hkv, d)[:n]
        o, z = _plain_attend(q[s:s + 1], k, v, st["scale"], n - 1)
        out[s:s + 1] = o.to(out.dtype)
        lse[s:s + 1] = z
    return out, lse


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    hq, d = case["heads"], case["dim"]
    group = hq // case["kv_heads"]
    q = st["q"].double()
    if case["op"] == "prompt":
        # 4 d flops of 64-bit products per (row, key, head): too long past this
        if 4 * d * hq * sum(n * n for n in st["lens"]) > 6e12:
            return None
        out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
        for a, b in zip(st["cu_host"], st["cu_host"][1:]):
            for h in range(hq):
                kh = st["k"][a:b, h // group].double()
                vh = st["v"][a:b, h // group].double()
                for r in range(a, b, 8192):
                    e = min(b, r + 8192)
                    z = st["scale"] * (q[r:e, h] @ kh[:e - a].T)
                    z += torch.full_like(z, float("-inf")).triu(r - a + 1)
                    lse[r:e, h] = torch.logsumexp(z, dim=1)
                    out[r:e, h] = (z - lse[r:e, h, None]).exp_() @ vh[:e - a]
        return out, lse
    page = case["page"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for s, n in enumerate(st["lens"]):
        token = torch.arange(n, device=q.device)
        block, row = st["table"][s].long()[token // page], token % page
        for c in range(case["kv_heads"]):
            heads = slice(c * group, (c + 1) * group)
            z = st["scale"] * (q[s, heads] @ st["k_cache"][block, c, row].double().T)
            lse[s, heads] = torch.logsumexp(z, dim=1)
            out[s, heads] = (z - lse[s, heads, None]).exp() @ st["v_cache"][block, c, row].double()
    return out, lse


def _exact_append(st):
    case = st["case"]
    page, rot = case["page"], case["rot"]
    half = rot // 2
    q, k = st["q"].double(), st["k"].double()
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    # a rotation of a pair is a product of complex numbers
    turn = torch.complex(st["rope"][:, :half].double(), st["rope"][:, half:].double())
    for s, (a, n) in enumerate(zip(st["cu_host"], st["lens"])):
        first = st["held_host"][s]
        w = turn[first:first + n, None, :]
        for x in (q, k):
            part = x[a:a + n, :, :rot]
            if case["interleaved"]:
                y = torch.view_as_complex(part.reshape(n, -1, half, 2).contiguous()) * w
                x[a:a + n, :, :rot] = torch.view_as_real(y).reshape(n, -1, rot)
            else:
                y = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * w
                x[a:a + n, :, :rot] = torch.cat((y.real, y.imag), dim=-1)
        # the new rows, page by page
        i = 0
        while i < n:
            p = first + i
            m = min(page - p % page, n - i)
            b = int(st["table"][s, p // page])
            kc[b, :, p % page:p % page + m] = k[a + i:a + i + m].transpose(0, 1)
            vc[b, :, p % page:p % page + m] = st["v"][a + i:a + i + m].double().transpose(0, 1)
            i += m
    out = [q, kc, vc]
    if case["keep_k"]:
        out.append(k)
    return out
