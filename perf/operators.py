"""What the serving and training operators around the attention are measured on: the page plan of a
step, the norm + rotation of queries and keys (with the cache append and the gradient), and the
attention of packed queries over a paged cache.

A case is a dict of plain values; ``prepare`` makes its inputs from a seed, ``run`` makes one pass
(the plain torch form, or the library's calls where ``own`` is true), ``exact`` the same in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # the plan of a decode step: 32 requests, one token each (latency is all that counts)
        dict(name="plan-decode-32", op="plan", B=32, cached_max=4096, chunk=1, chunk_share=0.0, page=64),
        # a large batch with prefill chunks among the decodes, small pages
        dict(name="plan-mixed-2048", op="plan", B=2048, cached_max=16384, chunk=513, chunk_share=0.25, page=16),
        # append of a decode step: 16 tokens, K and V into the cache
        dict(name="append-decode-16", op="append", T=16, h_q=32, h_kv=8, d=128, rot=128, pairs="half", type="bf16", page=64, far=32768),
        # append of a prefill chunk, wide heads, a quarter of each head rotated, adjacent pairs
        dict(name="append-chunk-8192", op="append", T=8192, h_q=16, h_kv=2, d=256, rot=64, pairs="adjacent", type="f16", page=16, far=131072),
        # training forward and gradient: two sequences of 8192
        dict(name="norm-train", op="norm", T=16384, s=8192, h_q=32, h_kv=8, d=128, rot=128, pairs="half", type="bf16"),
        dict(name="norm-grad", op="grad", T=16384, s=8192, h_q=32, h_kv=8, d=128, rot=128, pairs="half", type="bf16"),
        # a small gradient, narrow heads without sharing, an odd token count
        dict(name="norm-grad-small", op="grad", T=777, s=259, h_q=12, h_kv=12, d=64, rot=32, pairs="adjacent", type="f16"),
        # four short requests decoding: the smallest attention call
        dict(name="decode-4-short", op="attend", B=4, ctx_min=17, ctx_max=900, chunk=1, chunk_share=1.0, h_q=32, h_kv=8, d=128, page=16, window=-1, sinks=False, type="bf16"),
        # 64 requests decoding over caches of 2k to 32k keys: a stream over the cache
        dict(name="decode-64-long", op="attend", B=64, ctx_min=2048, ctx_max=32768, chunk=1, chunk_share=1.0, h_q=32, h_kv=8, d=128, page=64, window=-1, sinks=False, type="bf16"),
        # verification of five drafted tokens per request, wide heads with sinks
        dict(name="verify-32x5", op="attend", B=32, ctx_min=500, ctx_max=8192, chunk=5, chunk_share=1.0, h_q=16, h_kv=2, d=256, page=128, window=-1, sinks=True, type="bf16"),
        # decodes with a few chunks of prefill among them, narrow heads in groups of five, a sliding window
        dict(name="mixed-window", op="attend", B=24, ctx_min=64, ctx_max=4096, chunk=387, chunk_share=0.15, h_q=40, h_kv=8, d=64, page=16, window=1023, sinks=False, type="f16"),
        # chunked prefill: eight chunks of 1024 tokens over caches of up to 16k keys
        dict(name="chunk-8x1024", op="attend", B=8, ctx_min=1024, ctx_max=16384, chunk=1024, chunk_share=1.0, h_q=32, h_kv=8, d=128, page=64, window=-1, sinks=False, type="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "norm", "grad", "attend", "attend"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "plan":
        return dict(op=op, B=_spread(rng, 1, 2048), cached_max=_spread(rng, 16, 16384), chunk=_spread(rng, 1, 500),
                    chunk_share=rng.choice([0.0, 0.1, 0.25]), page=page)
    d = rng.choice([64, 128, 192, 256])
    h_kv = rng.choice([1, 2, 3, 4, 8])
    h_q = h_kv * rng.choice([1, 2, 4, 5, 8] if h_kv < 8 else [1, 2, 4])
    kind = rng.choice(["bf16", "f16"])
    if op in ("append", "norm", "grad"):
        # at most the largest listed case's 16384 tokens of 40 heads of 128
        T = _spread(rng, 1, min(16384, 16384 * 40 * 128 // ((h_q + 2 * h_kv) * d)))
        rot = rng.choice([r for r in (16, 32, 64, 128, 192, 256) if r <= d])
        c = dict(op=op, T=T, h_q=h_q, h_kv=h_kv, d=d, rot=rot, pairs=rng.choice(["half", "adjacent"]), type=kind)
        return dict(c, page=page, far=_spread(rng, 1024, 131072)) if op == "append" else dict(c, s=rng.randint(1, T))
    ctx_max = _spread(rng, 40, 16384)
    chunk = rng.choice([1, 1, rng.randint(2, 9), _spread(rng, 16, 512)])
    share = 1.0 if chunk < 10 else rng.choice([0.2, 1.0])
    # rows x keys within the largest listed case's
    B = _spread(rng, 1, max(1, min(48, int(2.5e9 / (ctx_max * max(chunk, 16) * h_q)))))
    return dict(op=op, B=B, ctx_min=rng.randint(1, ctx_max), ctx_max=ctx_max, chunk=chunk, chunk_share=share, h_q=h_q,
                h_kv=h_kv, d=d, page=page, window=rng.choice([-1, -1, 100, 1023]), sinks=rng.choice([False, True]), type=kind)


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _lengths(case, seed):
    """Cached and new tokens of each request, as lists: a case's own lengths, in an order of the seed's."""
    rng = random.Random(str([case[n] for n in ("B", "chunk", "chunk_share", "page")]))
    chunks = int(round(case["B"] * case["chunk_share"]))
    new = [case["chunk"]] * chunks + [1] * (case["B"] - chunks)
    if case["op"] == "plan":
        new[:chunks] = [rng.randint(1, case["chunk"]) for _ in range(chunks)]
        cached = [rng.randint(0, case["cached_max"]) for _ in new]
    else:
        cached = [max(0, _spread(rng, case["ctx_min"], case["ctx_max"]) - n) for n in new]
        if len(cached) > 1 or case["chunk"] == 1024:
            cached[-1] = max(0, case["ctx_max"] - new[-1])  # one request as long as the range allows
    order = list(range(len(new)))
    random.Random(seed).shuffle(order)
    return [cached[i] for i in order], [new[i] for i in order]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, kind):
    return torch.randn(shape, generator=g, device="cuda", dtype=TYPES[kind])


def _angles(n, rot):
    """cos and sin [n, rot / 2] of position x base^(-2 j / rot), in 64 bits and rounded once."""
    f = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return a.cos().float(), a.sin().float()


def _pages(case, lengths, g, spare):
    """A random table [B, blocks] for caches of these lengths, and the pages it leaves over."""
    P = case["page"]
    blocks = [-(-n // P) for n in lengths]
    width, total = max(blocks + [1]), sum(blocks)
    pool = total + spare
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    b = _i32(blocks)
    first = torch.cumsum(b, 0) - b
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j).clamp(max=pool - 1)
    table = torch.where(j < b[:, None], order[at.long()], torch.full_like(order[:1], -1)).to(torch.int32)
    return table.contiguous(), order[total:].contiguous(), pool


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "plan":
        cached, new = _lengths(case, seed)
        P = case["page"]
        table, free, pool = _pages(case, cached, g, sum(-(-(c + n) // P) - -(-c // P) for c, n in zip(cached, new)) + 7)
        wide = max(-(-(c + n) // P) for c, n in zip(cached, new))
        full = torch.full((len(new), wide), -1, dtype=torch.int32, device="cuda")
        full[:, : min(wide, table.shape[1])] = table[:, :wide]
        return dict(op=op, cached=_i32(cached), new=_i32(new), table=full, free=free, head=_i32([2]), page=P,
                    pool=pool, tokens=sum(new) + 5)
    if op == "attend":
        cached, new = _lengths(case, seed)
        used = [c + n for c, n in zip(cached, new)]
        table, _, pool = _pages(case, used, g, 3)
        table = table.clamp(min=0)
        shape = (pool, case["page"], case["h_kv"], case["d"])
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        return dict(op=op, q=_normal((cu[-1], case["h_q"], case["d"]), g, case["type"]), k=_normal(shape, g, case["type"]),
                    v=_normal(shape, g, case["type"]), cu=_i32(cu), used=_i32(used), table=table, s_kv=max(used),
                    longest=max(new), window=case["window"], scale=case["d"] ** -0.5,
                    sinks=torch.randn(case["h_q"], generator=g, device="cuda") if case["sinks"] else None)
    T, h_q, h_kv, d, kind = case["T"], case["h_q"], case["h_kv"], case["d"], case["type"]
    x = _normal((T, h_q + 2 * h_kv, d), g, kind) * 1.7  # the fused projection's rows
    s = dict(op=op, q=x[:, :h_q], k=x[:, h_q:h_q + h_kv], v=x[:, h_q + h_kv:], eps=1e-6, adjacent=case["pairs"] == "adjacent",
             wq=(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TYPES[kind]),
             wk=(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TYPES[kind]))
    if op == "append":
        n = -(-T // case["page"]) + 4
        s["cos"], s["sin"] = _angles(case["far"], case["rot"])
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["slots"] = torch.randperm(n * case["page"], generator=g, device="cuda")[:T].to(torch.int32)
        s["k_cache"] = _normal((n, case["page"], h_kv, d), g, kind)
        s["v_cache"] = _normal((n, case["page"], h_kv, d), g, kind)
        return s
    s["cos"], s["sin"] = _angles(case["s"], case["rot"])
    s["positions"] = torch.arange(T, device="cuda", dtype=torch.int32) % case["s"]
    if op == "grad":
        s["dq"], s["dk"] = _normal((T, h_q, d), g, kind), _normal((T, h_kv, d), g, kind)
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _plain_plan(s):
    P, cached, new, table = s["page"], s["cached"].long(), s["new"].long(), s["table"]
    used = cached + new
    cu = torch.cat([torch.zeros_like(used[:1]), torch.cumsum(new, 0)])
    old, tot = (cached + P - 1) // P, (used + P - 1) // P
    first = torch.cumsum(tot - old, 0) - (tot - old) + s["head"]
    j = torch.arange(table.shape[1], device="cuda")
    at = (first[:, None] + j - old[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where((j >= old[:, None]) & (j < tot[:, None]), s["free"][at], table))
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=new.numel() - 1)
    pos = cached[b] + t - cu[b]
    real = t < cu[-1]
    pos = torch.where(real, pos, torch.zeros_like(pos))
    slot = table[b, pos // P].long() * P + pos % P
    none = torch.full_like(pos, -1)
    i32 = torch.int32
    return dict(cu=cu.to(i32), used=used.to(i32), positions=torch.where(real, pos, none).to(i32),
                slots=torch.where(real, slot, none).to(i32), table=table, head=(s["head"] + (tot - old).sum()).to(i32))


def _turn(a, cos, sin, adjacent, back=False):
    """The rotation of the leading dims of a [T, h, d] by each token's angles (back: the inverse)."""
    rot = 2 * cos.shape[1]
    c, n = cos[:, None], (-sin if back else sin)[:, None]
    if adjacent:
        x, y = a[..., 0:rot:2], a[..., 1:rot:2]
        turned = torch.stack([x * c - y * n, y * c + x * n], -1).flatten(-2)
    else:
        x, y = a[..., :rot // 2], a[..., rot // 2:rot]
        turned = torch.cat([x * c - y * n, y * c + x * n], -1)
    return torch.cat([turned, a[..., rot:]], -1)


def _plain_norm(s):
    p = s["positions"].long()
    cos, sin = s["cos"][p], s["sin"][p]

    def one(x, w):
        f = x.float()
        f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        return _turn(f, cos, sin, s["adjacent"]).to(x.dtype)

    return dict(q=one(s["q"], s["wq"]), k=one(s["k"], s["wk"]))


def _plain_append(s):
    y = _plain_norm(s)
    at, shape = s["slots"].long(), s["k"].shape[1:]
    s["k_cache"].view(-1, *shape)[at] = y["k"]
    s["v_cache"].view(-1, *shape)[at] = s["v"]
    return dict(q=y["q"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_grad(s):
    p = s["positions"].long()
    cos, sin = s["cos"][p], s["sin"][p]

    def one(x, w, dy):
        f = x.float()
        r = torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"])
        xh = f * r
        g = _turn(dy.float(), cos, sin, s["adjacent"], back=True)
        gw = g * w.float()
        return (r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(x.dtype), (g.double() * xh).sum((0, 1)).float()

    dq, dwq = one(s["q"], s["wq"], s["dq"])
    dk, dwk = one(s["k"], s["wk"], s["dk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _plain_attend(s):
    q, table, cu, used = s["q"], s["table"], s["cu"].long(), s["used"].long()
    (T, h_q, d), (B, _), h_kv, n = q.shape, table.shape, s["k"].shape[2], s["longest"]
    G = h_q // h_kv
    i = torch.arange(n, device="cuda")
    count = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=T - 1)
    qp = q[at].float().view(B, n, h_kv, G, d).permute(0, 2, 3, 1, 4).reshape(B, h_kv, G * n, d)
    k = s["k"][table.long()].view(B, -1, h_kv, d).permute(0, 2, 3, 1).float()
    score = torch.matmul(qp, k).view(B, h_kv, G, n, -1) * s["scale"]
    del k
    j = torch.arange(score.shape[-1], device="cuda")
    last = (used - count)[:, None] + i  # the key at the query's own place
    keep = (j <= last[..., None]) & (j < used[:, None, None])
    if s["window"] >= 0:
        keep &= j >= last[..., None] - s["window"]
    score.masked_fill_(~keep[:, None, None], float("-inf"))
    m = score.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, h_kv, G, 1, 1)
        m = torch.maximum(m, sink)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = score.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(sink - m)
    v = s["v"][table.long()].view(B, -1, h_kv, d).permute(0, 2, 1, 3).float()
    o = torch.matmul(e.view(B, h_kv, G * n, -1), v).view(B, h_kv, G, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(-1)
    real = i < count[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, h_q, d)[real].to(q.dtype)
    return dict(o=o, lse=lse.permute(0, 3, 1, 2).reshape(B, n, h_q)[real].t().contiguous())


def _own_plan(s):
    from exact_attention_bwd_gb300 import binding as fa
    cu, used, positions, slots, head = fa.page_plan(s["cached"], s["new"], s["table"], s["free"], page_size=s["page"],
                                                    num_pages=s["pool"], tokens=s["tokens"], free_head=s["head"])
    return dict(cu=cu, used=used, positions=positions, slots=slots, table=s["table"], head=head)


def _own_norm(s):
    from exact_attention_bwd_gb300 import binding as fa
    q, k = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], positions=s["positions"], eps=s["eps"],
                           interleaved=s["adjacent"])
    return dict(q=q, k=k)


def _own_append(s):
    from exact_attention_bwd_gb300 import binding as fa
    q, _ = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], positions=s["positions"], eps=s["eps"],
                           interleaved=s["adjacent"], v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"])
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_grad(s):
    from exact_attention_bwd_gb300 import binding as fa
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], s["cos"], s["sin"],
                                                positions=s["positions"], eps=s["eps"], interleaved=s["adjacent"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _own_attend(s):
    from exact_attention_bwd_gb300 import binding as fa
    o, lse, _ = fa.forward(s["q"], s["k"], s["v"], causal=True, window=(s["window"], -1), softmax_scale=s["scale"],
                           sinks=s["sinks"], cu_q=s["cu"], seqused_k=s["used"], block_table=s["table"], s_kv=s["s_kv"],
                           max_seqlen_q=s["longest"])
    return dict(o=o, lse=lse)


_plain = dict(plan=_plain_plan, norm=_plain_norm, append=_plain_append, grad=_plain_grad, attend=_plain_attend)
_own = dict(plan=_own_plan, norm=_own_norm, append=_own_append, grad=_own_grad, attend=_own_attend)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _lengths(case, 0)
        P = case["page"]
        pages = sum(-(-(c + n) // P) - -(-c // P) for c, n in zip(cached, new))
        return dict(bytes=4 * (2 * len(new) + 2 * pages + 2 * len(new) + 1 + 2 * sum(new)), flops=0)
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    if op == "attend":
        cached, new = _lengths(case, 0)
        keys = pairs = 0
        for c, n in zip(cached, new):
            w = case["window"] if case["window"] >= 0 else c + n
            keys += min(c + n, n + w)
            pairs += sum(min(c + i + 1, w + 1) for i in range(n))
        return dict(bytes=2 * d * (2 * h_kv * keys + 2 * h_q * sum(new)) + 4 * h_q * sum(new), flops=4 * h_q * d * pairs)
    T, row = case["T"], 2 * d
    table = 4 * case["rot"] * (min(T, case["far"]) if op == "append" else min(T, case["s"])) + 4 * T
    if op == "append":
        return dict(bytes=2 * T * (h_q + 2 * h_kv) * row + table + 4 * T, flops=8 * T * (h_q + h_kv) * d)
    if op == "norm":
        return dict(bytes=2 * T * (h_q + h_kv) * row + table, flops=8 * T * (h_q + h_kv) * d)
    return dict(bytes=3 * T * (h_q + h_kv) * row + table + 8 * d, flops=16 * T * (h_q + h_kv) * d)


# ------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "plan":
        return None  # whole numbers: the plain form is their definition
    return _exact_attend(s) if s["op"] == "attend" else _exact_norm(s, case)


def _exact_attend(s):
    q, B = s["q"].double(), s["table"].shape[0]
    T, h_q, d = q.shape
    h_kv = s["k"].shape[2]
    o = torch.zeros_like(q)
    lse = torch.full((h_q, T), float("-inf"), dtype=torch.float64, device="cuda")
    cu, used = s["cu"].tolist(), s["used"].tolist()
    for b in range(B):
        n, keys = cu[b + 1] - cu[b], used[b]
        if n == 0 or keys == 0:
            continue
        blocks = -(-keys // s["k"].shape[1])
        pages = s["table"][b, :blocks].long()
        k = s["k"][pages].reshape(-1, h_kv, d)[:keys].double()
        v = s["v"][pages].reshape(-1, h_kv, d)[:keys].double()
        at = torch.arange(keys - n, keys, device="cuda")[:, None]
        j = torch.arange(keys, device="cuda")[None]
        out = (j > at) | ((j < at - s["window"]) if s["window"] >= 0 else torch.zeros_like(j > at))
        for h in range(h_q):
            a = q[cu[b]:cu[b + 1], h] @ k[:, h * h_kv // h_q].t() * s["scale"]
            a[out] = float("-inf")
            if s["sinks"] is not None:
                a = torch.cat([a, s["sinks"][h].double().expand(n, 1)], 1)
            z = torch.logsumexp(a, 1)
            w = torch.exp(a - z[:, None])[:, :keys]
            w[torch.isinf(z)] = 0
            o[cu[b]:cu[b + 1], h] = w @ v[:, h * h_kv // h_q]
            lse[h, cu[b]:cu[b + 1]] = z
    return dict(o=o, lse=lse)


def _exact_norm(s, case):
    rot, adjacent, p = case["rot"], s["adjacent"], s["positions"].long()
    first = torch.arange(0, rot, 2, device="cuda") if adjacent else torch.arange(rot // 2, device="cuda")
    second = first + (1 if adjacent else rot // 2)
    turn = torch.complex(s["cos"][p].double(), s["sin"][p].double())[:, None]

    def rotate(y, z):
        y = y.clone()
        w = torch.complex(y[..., first], y[..., second]) * z
        y[..., first], y[..., second] = w.real, w.imag
        return y

    def forward(x, w):
        x = x.double()
        return rotate(x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double(), turn)

    def gradient(x, w, dy):
        x, w, dy = x.double(), w.double(), rotate(dy.double(), turn.conj())
        d, ms = x.shape[-1], (x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]
        gw = dy * w
        return gw / ms.sqrt() - x * (gw * x).sum(-1, keepdim=True) / (d * ms ** 1.5), (dy * x / ms.sqrt()).sum((0, 1))

    if s["op"] == "norm":
        return dict(q=forward(s["q"], s["wq"]), k=forward(s["k"], s["wk"]))
    if s["op"] == "grad":
        (dq, dwq), (dk, dwk) = gradient(s["q"], s["wq"], s["dq"]), gradient(s["k"], s["wk"], s["dk"])
        return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    for cache, rows in ((k_cache, forward(s["k"], s["wk"])), (v_cache, s["v"].double())):
        cache.view(-1, *rows.shape[1:]).index_copy_(0, s["slots"].long(), rows)
    return dict(q=forward(s["q"], s["wq"]), k_cache=k_cache, v_cache=v_cache)
