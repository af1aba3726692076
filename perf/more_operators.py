"""What the operators of a serving step over an 8-bit cache, and the rotation with several position axes, are
measured on: the rotation of queries and keys by positions with axes (time, height, width), with or without the
norm, and its gradient; the append of rotated keys and of values to an e4m3 paged cache with a scale for each block of
tokens and head; the attention of packed queries over that cache.

A case is a dict of plain values; ``prepare`` makes its inputs from a seed, ``run`` makes one pass
(the plain torch form, or the library's calls where ``own`` is true), ``exact`` the same in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # a decode step's rotation: 16 tokens with three axes, no norm (latency is all that counts)
        dict(name="turn-decode-16", op="turn", T=16, h_q=32, h_kv=8, d=128, rot=128, axes=3, order="split", norm=False, pairs="half", type="bf16", far=32768),
        # training forward over packed text and images, norm and rotation by time, height and width in turn
        dict(name="turn-train", op="turn", T=16384, h_q=32, h_kv=8, d=128, rot=128, axes=3, order="cycle", norm=True, pairs="half", type="bf16", far=8192),
        # its gradient for a model without the norm: a stream from dy to dx
        dict(name="turn-grad", op="grad", T=16384, h_q=32, h_kv=8, d=128, rot=128, axes=3, order="split", norm=False, pairs="half", type="bf16", far=8192),
        # an image encoder's gradient: height and width, narrow heads without sharing, an odd token count
        dict(name="turn-grad-odd", op="grad", T=1555, h_q=12, h_kv=12, d=64, rot=64, axes=2, order="split", norm=True, pairs="adjacent", type="f16", far=64),
        # append of a decode step: 32 requests, one token each
        dict(name="append8-decode-32", op="append", B=32, ctx_min=64, ctx_max=4096, chunk=1, chunk_share=1.0, h_q=32, h_kv=8, d=128, rot=128, axes=3, order="split", norm=True, pairs="half", type="bf16", page=64, block=64),
        # prefill chunks of 512 tokens, wide heads, a quarter of each head rotated, a scale for each small page
        dict(name="append8-chunk-8192", op="append", B=16, ctx_min=512, ctx_max=8192, chunk=512, chunk_share=1.0, h_q=16, h_kv=2, d=256, rot=64, axes=1, order="split", norm=False, pairs="adjacent", type="f16", page=16, block=16),
        # four short requests decoding: the smallest attention call
        dict(name="attend8-4-short", op="attend", B=4, ctx_min=17, ctx_max=900, chunk=1, chunk_share=1.0, h_q=32, h_kv=8, d=128, page=16, block=16, window=-1, sinks=False, type="bf16"),
        # 64 requests decoding over caches of 2k to 32k keys: a stream over the cache
        dict(name="attend8-64-long", op="attend", B=64, ctx_min=2048, ctx_max=32768, chunk=1, chunk_share=1.0, h_q=32, h_kv=8, d=128, page=64, block=64, window=-1, sinks=False, type="bf16"),
        # verification of five drafted tokens per request, wide heads with sinks
        dict(name="attend8-verify-32x5", op="attend", B=32, ctx_min=500, ctx_max=8192, chunk=5, chunk_share=1.0, h_q=16, h_kv=2, d=256, page=128, block=32, window=-1, sinks=True, type="bf16"),
        # decodes with a few chunks of prefill among them, narrow heads in groups of five, a sliding window
        dict(name="attend8-mixed-window", op="attend", B=24, ctx_min=64, ctx_max=4096, chunk=387, chunk_share=0.15, h_q=40, h_kv=8, d=64, page=48, block=16, window=1023, sinks=False, type="f16"),
        # chunked prefill: eight chunks of 1024 tokens over caches of up to 16k keys
        dict(name="attend8-chunk-8x1024", op="attend", B=8, ctx_min=1024, ctx_max=16384, chunk=1024, chunk_share=1.0, h_q=32, h_kv=8, d=128, page=64, block=64, window=-1, sinks=False, type="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["turn", "grad", "append", "append", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 192, 256])
    h_kv = rng.choice([1, 2, 3, 4, 8])
    h_q = h_kv * rng.choice([1, 2, 4, 5, 8] if h_kv < 8 else [1, 2, 4])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    block = rng.choice([n for n in (16, 32, 48, 64, 128, 256) if page % n == 0])
    c = dict(op=op, h_q=h_q, h_kv=h_kv, d=d, type=rng.choice(["bf16", "f16"]))
    turn = dict(rot=rng.choice([r for r in (16, 32, 64, 128, 192, 256) if r <= d]), axes=rng.choice([1, 2, 3, 3, 4]),
                order=rng.choice(["split", "cycle"]), norm=rng.choice([False, True]), pairs=rng.choice(["half", "adjacent"]))
    most = min(16384, 16384 * 40 * 128 // ((h_q + 2 * h_kv) * d))  # tokens: the largest listed case's
    if op in ("turn", "grad"):
        return dict(c, **turn, T=_spread(rng, 1, most), far=_spread(rng, 64, 32768))
    ctx_max = _spread(rng, 40, 16384)
    chunk = min(ctx_max, rng.choice([1, 1, rng.randint(2, 9), _spread(rng, 16, 512)]))
    share = 1.0 if chunk < 10 else rng.choice([0.2, 1.0])
    c.update(ctx_min=rng.randint(1, ctx_max), ctx_max=ctx_max, chunk=chunk, chunk_share=share, page=page, block=block)
    if op == "append":
        return dict(c, **turn, B=_spread(rng, 1, max(1, min(256, most // chunk, 500000 // ctx_max))))
    # rows x keys within the largest listed case's
    return dict(c, B=_spread(rng, 1, max(1, min(48, int(2.5e9 / (ctx_max * max(chunk, 16) * h_q))))),
                window=rng.choice([-1, -1, 100, 1023]), sinks=rng.choice([False, True]))


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _lengths(case, seed):
    """Cached and new tokens of each request, as lists: a case's own lengths, in an order of the seed's."""
    rng = random.Random(str([case[n] for n in ("B", "chunk", "chunk_share", "page")]))
    chunks = int(round(case["B"] * case["chunk_share"]))
    new = [case["chunk"]] * chunks + [1] * (case["B"] - chunks)
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


def _pair_axis(case):
    """The axis of each pair: the pairs split between the axes (the first gets a quarter of three), or in turn."""
    half, axes = case["rot"] // 2, case["axes"]
    if case["order"] == "cycle":
        return [j % axes for j in range(half)]
    first = half // 4 if axes == 3 else half // axes
    rest = max(1, -(-(half - first) // max(1, axes - 1)))
    return [0 if j < first else min(axes - 1, 1 + (j - first) // rest) for j in range(half)] if axes > 1 else [0] * half


def _grid_positions(T, axes, far, g):
    """Positions of text and images in turn: spans of text with one position for all axes, images of 24 columns."""
    t = torch.arange(T, device="cuda")
    start = torch.randint(0, max(1, far - 48), (1,), generator=g, device="cuda")
    span, at = t // 720, t % 720
    text = (span % 2 == 0)[None].expand(axes, T)
    step = torch.stack([torch.zeros_like(at), at // 24, at % 24, at // 360][:axes])
    p = torch.where(text, (at % 97)[None].expand(axes, T), step) + start + span
    return (p % far).to(torch.int32).contiguous()


def _pages(case, lengths, g, spare):
    """A random table [B, blocks] for caches of these lengths, and the pool's pages."""
    P = case["page"]
    blocks = [-(-n // P) for n in lengths]
    width, total = max(blocks + [1]), sum(blocks)
    pool = total + spare
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    b = _i32(blocks)
    first = torch.cumsum(b, 0) - b
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j).clamp(max=pool - 1)
    table = torch.where(j < b[:, None], order[at.long()], torch.zeros_like(order[:1])).to(torch.int32)
    return table.contiguous(), pool


def _power(amax):
    """The smallest power of two s with amax <= 448 s (2^-126 at least), as the cache's scales are made."""
    m, e = torch.frexp(amax.clamp(min=2.0 ** -118))
    return torch.ldexp(torch.ones_like(amax), torch.where(m > 0.875, e - 8, e - 9))


def _cache(case, pool, g):
    """A filled cache: rows as a projection gives them (some channels larger, blocks of unlike size), quantised."""
    P, N, h, d = case["page"], case["block"], case["h_kv"], case["d"]
    x = _normal((pool, P // N, N, h, d), g, case["type"])
    x *= torch.exp(0.5 * torch.randn((pool, P // N, 1, h, 1), generator=g, device="cuda")).to(x.dtype)
    x[..., 3::16] *= 4
    scale = _power(x.abs().amax((2, 4)).float())
    x.div_(scale[:, :, None, :, None].to(x.dtype))
    return x.view(pool, P, h, d).to(E4M3).view(torch.uint8), scale.contiguous()


def prepare(case, seed):
    g, op, kind = _gen(seed), case["op"], case["type"]
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    s = dict(op=op)
    if op in ("append", "attend"):
        cached, new = _lengths(case, seed)
        used = [c + n for c, n in zip(cached, new)]
        s["table"], pool = _pages(case, used, g, 3)
        (s["k8"], s["k_scale"]), (s["v8"], s["v_scale"]) = _cache(case, pool, g), _cache(case, pool, g)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s.update(cu=_i32(cu), used=_i32(used), block=case["block"])
        T = cu[-1]
    else:
        T = case["T"]
    if op == "attend":
        s.update(q=_normal((T, h_q, d), g, kind), s_kv=max(used), longest=max(new), window=case["window"], scale=d ** -0.5,
                 sinks=torch.randn(h_q, generator=g, device="cuda") if case["sinks"] else None)
        return s
    x = _normal((T, h_q + 2 * h_kv, d), g, kind) * 1.7  # the fused projection's rows
    s.update(q=x[:, :h_q], k=x[:, h_q:h_q + h_kv], v=x[:, h_q + h_kv:], eps=1e-6, adjacent=case["pairs"] == "adjacent",
             norm=case["norm"], axis_list=tuple(_pair_axis(case)), axis=torch.tensor(_pair_axis(case), device="cuda"), wq=None, wk=None)
    if case["norm"]:
        s["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TYPES[kind])
        s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TYPES[kind])
    if op == "append":
        far = case["ctx_max"] + 64
        place = torch.cat([torch.arange(c, c + n) for c, n in zip(cached, new)])
        shift = torch.randint(0, 64, (case["axes"], 1), generator=g, device="cuda")
        s["positions"] = (place.cuda()[None] + shift).to(torch.int32).contiguous()  # later than the cache's place: an image was earlier
    else:
        far = case["far"]
        s["positions"] = _grid_positions(T, case["axes"], far, g)
    s["cos"], s["sin"] = _angles(far, case["rot"])
    if op == "grad":
        s["dq"], s["dk"] = _normal((T, h_q, d), g, kind), _normal((T, h_kv, d), g, kind)
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _token_angles(s):
    """cos and sin [T, rot / 2] of each token: pair j at the position of its axis."""
    p = s["positions"].long()[s["axis"]].t()
    j = torch.arange(p.shape[1], device=p.device)
    return s["cos"][p, j], s["sin"][p, j]


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


def _rows(s, x, w):
    """x [T, h, d] with norm and rotation, in 32 bits."""
    f = x.float()
    if s["norm"]:
        f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
    return _turn(f, *_token_angles(s), s["adjacent"])


def _plain_turn(s):
    return dict(q=_rows(s, s["q"], s["wq"]).to(s["q"].dtype), k=_rows(s, s["k"], s["wk"]).to(s["k"].dtype))


def _plain_grad(s):
    cos, sin = _token_angles(s)

    def one(x, w, dy):
        g = _turn(dy.float(), cos, sin, s["adjacent"], back=True)
        if not s["norm"]:
            return g.to(x.dtype), None
        f = x.float()
        r = torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"])
        xh = f * r
        gw = g * w.float()
        return (r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(x.dtype), (g.double() * xh).sum((0, 1)).float()

    dq, dwq = one(s["q"], s["wq"], s["dq"])
    dk, dwk = one(s["k"], s["wk"], s["dk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _quantise(pool, scale, rows, s):
    """Stores rows [T, h, d] (32 bits) at the new tokens' places of one pool of the cache."""
    N, P, T, h = s["block"], pool.shape[1], rows.shape[0], pool.shape[2]
    cu, used, table = s["cu"].long(), s["used"].long(), s["table"].long()
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    place = used[b] - cu[b + 1] + t
    at = table[b, place // P] * P + place % P          # the token's row of the pool
    block = at // N
    flat = scale.view(-1, h)
    amax = torch.zeros_like(flat).index_reduce_(0, block, rows.abs().amax(-1), "amax")
    fresh = torch.zeros(flat.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, block[at % N == 0], True)
    touched = torch.zeros_like(fresh).index_fill_(0, block, True)[:, None]
    new = torch.where(touched, torch.maximum(torch.where(fresh[:, None], 0.0, flat), _power(amax)), flat)
    # rows of a sequence's first block ahead of its new ones
    start = (used - cu[1:] + cu[:-1]).clamp(max=table.shape[1] * P - 1)
    i = torch.arange(N, device="cuda")
    first = (table.gather(1, (start // P)[:, None])[:, 0] * P + start % P) // N
    old = (i < (start % P % N)[:, None]) & (cu[1:] > cu[:-1])[:, None]
    line, keep = (first[:, None] * N + i)[old], first[:, None].expand(-1, N)[old]
    v8 = pool.view(E4M3).view(-1, h, pool.shape[3])
    u8 = pool.view(-1, h, pool.shape[3])
    before = u8[line].view(E4M3).float() * (flat[keep] / new[keep])[..., None]
    u8[line] = before.to(E4M3).view(torch.uint8)
    u8[at] = (rows / new[block][..., None]).to(E4M3).view(torch.uint8)
    flat.copy_(new)
    return v8.view(pool.shape)


def _plain_append(s):
    q = _rows(s, s["q"], s["wq"]).to(s["q"].dtype)
    k = _quantise(s["k8"], s["k_scale"], _rows(s, s["k"], s["wk"]), s)
    v = _quantise(s["v8"], s["v_scale"], s["v"].float(), s)
    return dict(q=q, k=k, v=v, k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_attend(s):
    q, table, cu, used = s["q"], s["table"].long(), s["cu"].long(), s["used"].long()
    (T, h_q, d), (B, _), h_kv, n = q.shape, table.shape, s["k8"].shape[2], s["longest"]
    G = h_q // h_kv

    def rows(pool, scale):  # [B, keys, h_kv, d] in 32 bits
        x = pool[table].view(E4M3).float().view(B, -1, s["block"], h_kv, d)
        return x.mul_(scale[table].view(B, -1, 1, h_kv, 1)).view(B, -1, h_kv, d)

    i = torch.arange(n, device="cuda")
    count = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=T - 1)
    qp = q[at].float().view(B, n, h_kv, G, d).permute(0, 2, 3, 1, 4).reshape(B, h_kv, G * n, d)
    score = torch.matmul(qp, rows(s["k8"], s["k_scale"]).permute(0, 2, 3, 1)).view(B, h_kv, G, n, -1) * s["scale"]
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
    o = torch.matmul(e.view(B, h_kv, G * n, -1), rows(s["v8"], s["v_scale"]).permute(0, 2, 1, 3)).view(B, h_kv, G, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(-1)
    real = i < count[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, h_q, d)[real].to(q.dtype)
    return dict(o=o, lse=lse.permute(0, 3, 1, 2).reshape(B, n, h_q)[real].t().contiguous())


def _own_turn(s):
    from exact_attention_bwd_gb300 import binding as fa
    q, k = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], positions=s["positions"], eps=s["eps"],
                           interleaved=s["adjacent"], pair_axis=s["axis_list"], norm=s["norm"])
    return dict(q=q, k=k)


def _own_grad(s):
    from exact_attention_bwd_gb300 import binding as fa
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], s["cos"], s["sin"],
                                                positions=s["positions"], eps=s["eps"], interleaved=s["adjacent"],
                                                pair_axis=s["axis_list"], norm=s["norm"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _own_append(s):
    from exact_attention_bwd_gb300 import binding as fa
    q = fa.qk_norm_rope_append8(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], k_cache=s["k8"], v_cache=s["v8"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"], cu_q=s["cu"], seqused_k=s["used"],
                                block_table=s["table"], positions=s["positions"], eps=s["eps"], interleaved=s["adjacent"],
                                pair_axis=s["axis_list"], norm=s["norm"])
    # the bytes as the e4m3 values that they are, in units of the blocks' scales, which come beside them
    return dict(q=q, k=s["k8"].view(E4M3), v=s["v8"].view(E4M3), k_scale=s["k_scale"], v_scale=s["v_scale"])


def _own_attend(s):
    from exact_attention_bwd_gb300 import binding as fa
    o, lse, _ = fa.forward(s["q"], s["k8"], s["v8"], causal=True, window=(s["window"], -1), softmax_scale=s["scale"],
                           sinks=s["sinks"], cu_q=s["cu"], seqused_k=s["used"], block_table=s["table"], s_kv=s["s_kv"],
                           max_seqlen_q=s["longest"], cache_scale=(s["k_scale"], s["v_scale"]))
    return dict(o=o, lse=lse)


_plain = dict(turn=_plain_turn, grad=_plain_grad, append=_plain_append, attend=_plain_attend)
_own = dict(turn=_own_turn, grad=_own_grad, append=_own_append, attend=_own_attend)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------

def work(case):
    op, h_q, h_kv, d = case["op"], case["h_q"], case["h_kv"], case["d"]
    if op in ("append", "attend"):
        cached, new = _lengths(case, 0)
        T = sum(new)
    else:
        T = case["T"]
    if op == "attend":
        keys = blocks = pairs = 0
        for c, n in zip(cached, new):
            w = case["window"] if case["window"] >= 0 else c + n
            seen = min(c + n, n + w)
            keys += seen
            blocks += -(-seen // case["block"])
            pairs += sum(min(c + i + 1, w + 1) for i in range(n))
        return dict(bytes=2 * h_kv * (d * keys + 4 * blocks) + 4 * d * h_q * T + 4 * h_q * T, flops=4 * h_q * d * pairs)
    far = case["ctx_max"] if op == "append" else case["far"]
    table = 4 * case["rot"] * min(T, far) + 4 * case["axes"] * T
    rows = 2 * T * (h_q + h_kv) * d
    flops = (8 if case["norm"] else 4) * T * (h_q + h_kv) * d
    if op == "turn":
        return dict(bytes=2 * rows + table, flops=flops)
    if op == "grad":
        return dict(bytes=(3 if case["norm"] else 2) * rows + table, flops=2 * flops)
    blocks = sum(-(-n // case["block"]) for n in new)
    return dict(bytes=4 * T * h_q * d + 6 * T * h_kv * d + 8 * h_kv * blocks + table, flops=flops)


# ------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return dict(turn=_exact_turn, grad=_exact_grad, append=_exact_append, attend=_exact_attend)[case["op"]](s, case)


def _exact_turner(s, case):
    """The rotation as a product of complex numbers, and its inverse."""
    rot = case["rot"]
    first = torch.arange(0, rot, 2, device="cuda") if s["adjacent"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if s["adjacent"] else rot // 2)
    columns = []
    for j, axis in enumerate(s["axis_list"]):
        p = s["positions"][axis].long()
        columns.append(torch.complex(s["cos"][p, j].double(), s["sin"][p, j].double()))
    unit = torch.stack(columns, 1)[:, None]

    def rotate(y, back=False):
        y = y.clone()
        w = torch.complex(y[..., first], y[..., second]) * (unit.conj() if back else unit)
        y[..., first], y[..., second] = w.real, w.imag
        return y

    return rotate


def _exact_rows(s, case, x, w):
    x = x.double()
    if s["norm"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
    return _exact_turner(s, case)(x)


def _exact_turn(s, case):
    return dict(q=_exact_rows(s, case, s["q"], s["wq"]), k=_exact_rows(s, case, s["k"], s["wk"]))


def _exact_grad(s, case):
    rotate = _exact_turner(s, case)

    def gradient(x, w, dy):
        x, dy = x.double(), rotate(dy.double(), back=True)
        if not s["norm"]:
            return dy, None
        w = w.double()
        d, ms = x.shape[-1], (x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]
        gw = dy * w
        return gw / ms.sqrt() - x * (gw * x).sum(-1, keepdim=True) / (d * ms ** 1.5), (dy * x / ms.sqrt()).sum((0, 1))

    (dq, dwq), (dk, dwk) = gradient(s["q"], s["wq"], s["dq"]), gradient(s["k"], s["wk"], s["dk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _exact_append(s, case):
    cu, used, N, P = s["cu"].tolist(), s["used"].tolist(), case["block"], case["page"]

    def store(pool, scale, rows):
        values, out = pool.view(E4M3).double(), scale.double()
        for b in range(len(used)):
            start = used[b] - (cu[b + 1] - cu[b])
            for at in range(start - start % N, used[b], N):
                page, first = int(s["table"][b, at // P]), at % P
                lo, hi = max(at, start), min(at + N, used[b])
                x = rows[cu[b] + lo - start:cu[b] + hi - start]
                most = x.abs().amax((0, 2))
                need = 2.0 ** torch.ceil(torch.log2(most / 448))  # (a logarithm next to a whole number may be off)
                need = torch.where(448 * need / 2 >= most, need / 2, torch.where(448 * need < most, 2 * need, need))
                before = out[page, first // N].clone()
                now = need if lo == at else torch.maximum(before, need)
                if lo > at:
                    values[page, first:first + lo - at] *= (before / now)[:, None]
                values[page, first + lo - at:first + hi - at] = x / now[:, None]
                out[page, first // N] = now
        return values, out

    k, k_scale = store(s["k8"], s["k_scale"], _exact_rows(s, case, s["k"], s["wk"]))
    v, v_scale = store(s["v8"], s["v_scale"], s["v"].double())
    return dict(q=_exact_rows(s, case, s["q"], s["wq"]), k=k, v=v, k_scale=k_scale, v_scale=v_scale)


def _exact_attend(s, case):
    q, N = s["q"].double(), case["block"]
    T, h_q, d = q.shape
    h_kv = s["k8"].shape[2]
    o = torch.zeros_like(q)
    lse = torch.full((h_q, T), float("-inf"), dtype=torch.float64, device="cuda")
    cu, used = s["cu"].tolist(), s["used"].tolist()
    for b in range(len(used)):
        n, keys = cu[b + 1] - cu[b], used[b]
        if n == 0 or keys == 0:
            continue
        pages = s["table"][b, :-(-keys // case["page"])].long()

        def true(pool, scale):
            return (pool[pages].view(E4M3).double().view(-1, N, h_kv, d) * scale[pages].double().view(-1, 1, h_kv, 1)).view(-1, h_kv, d)[:keys]

        k, v = true(s["k8"], s["k_scale"]), true(s["v8"], s["v_scale"])
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
