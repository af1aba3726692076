"""Norm + rotation of queries and keys, the append to a paged cache and the gradient, on the GPU
against the 64-bit formulas.

Bounds.  An output is rounded once: half a step, eps / 2 of the value (plus the smallest
subnormal's half, fp16).  Ahead of it stand fp32 operations: the mean of d squares and its
inverse root (their relative error at most (d / 8 + 8) 2^-24 for sums of d / lanes products
and a few shuffles; 2^-18 covers d = 256), two products and a rotation (two products and a sum,
relative to |a| + |b|).  So |error| <= eps / 2 |y| + 2^-17 (|a| + |b|), with |a| + |b| the
rotation's operands.  The gradient subtracts two terms of that accuracy, so its fp32 part is
relative to r (|g w| + |xh| mean|g w xh|).  A weight's gradient is a sum of T h terms, each with
relative error 2^-17, added in chains of fewer than 64 terms per lane and trees above:
2^-16 of the sum of the terms' sizes.
"""
import numpy as np
import pytest

import step_helpers as ref
from exact_attention_bwd_gb300 import inputs
from gpu_helpers import Guarded, from_dev

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def torch_type(kind):
    import torch
    return torch.bfloat16 if kind == "bf16" else torch.float16


def dev(x, kind):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(torch_type(kind))


def case(T, h_q, h_kv, d, rot, adjacent, kind, seed, positions="random", max_pos=5000, f32_weights=False):
    import torch
    rng = np.random.default_rng(seed)
    x = dev(rng.standard_normal((T, h_q + 2 * h_kv, d)) * rng.choice([0.05, 1.0, 6.0], (T, 1, 1)), kind)
    wt = torch.float32 if f32_weights else torch_type(kind)
    c = dict(T=T, h_q=h_q, h_kv=h_kv, d=d, rot=rot, adjacent=adjacent, kind=kind, x=x,
             q=x[:, :h_q], k=x[:, h_q:h_q + h_kv], v=x[:, h_q + h_kv:],
             wq=torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).cuda().to(wt),
             wk=torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).cuda().to(wt),
             pos=rng.integers(0, max_pos, T).astype(np.int32))
    c["cos"], c["sin"] = ref.angles(max_pos, rot) if rot else (None, None)
    c["angles"] = tuple(None if a is None else torch.from_numpy(a).cuda() for a in (c["cos"], c["sin"]))
    return c


def tables(c, pos):
    if not c["rot"]:
        return np.ones((len(pos), 0)), np.zeros((len(pos), 0))
    return c["cos"][pos], c["sin"][pos]


def check_rows(name, got, x, w, cos, sin, adjacent, kind):
    want = ref.norm_rope(x, w, cos, sin, EPS, adjacent)
    y = np.abs(x / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS) * w)
    size = ref.rotate(y, np.abs(cos), np.abs(sin), adjacent, back=False)
    size = np.maximum(np.abs(size), y) + np.abs(ref.rotate(y, np.abs(cos), np.abs(sin), adjacent, back=True))
    bound = TYPES[kind] * np.abs(want) + 2.0 ** -17 * size + 2.0 ** -25
    err = np.abs(got - want)
    assert np.all(err <= bound), (name, float((err - bound).max()))


SHAPES = [
    (1, 1, 1, 64, 64, False, "bf16"), (1, 32, 8, 128, 128, False, "bf16"), (37, 12, 12, 64, 32, True, "f16"),
    (130, 5, 1, 128, 64, False, "f16"), (7, 16, 2, 256, 256, True, "bf16"), (19, 6, 3, 192, 192, False, "bf16"),
    (33, 9, 3, 192, 16, True, "f16"), (4, 2, 2, 256, 0, False, "bf16"), (257, 8, 8, 64, 16, False, "bf16"),
    (3, 40, 8, 256, 48, False, "f16"), (65, 3, 3, 192, 96, False, "f16"),
]


@pytest.mark.parametrize("T,h_q,h_kv,d,rot,adjacent,kind", SHAPES)
def test_forward(T, h_q, h_kv, d, rot, adjacent, kind):
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case(T, h_q, h_kv, d, rot, adjacent, kind, seed=T + d, f32_weights=T % 2 == 1)
    out = Guarded((T, h_q, d), torch_type(kind)), Guarded((T, h_kv, d), torch_type(kind))
    fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], positions=torch.from_numpy(c["pos"]).cuda(), eps=EPS,
                    interleaved=adjacent, out=(out[0].t, out[1].t))
    for name, g, x, w in (("q", out[0], c["q"], c["wq"]), ("k", out[1], c["k"], c["wk"])):
        g.check(name)
        check_rows(name, from_dev(g.t), from_dev(x), from_dev(w), *tables(c, c["pos"]), adjacent, kind)


def test_forward_dense_default_positions_in_place_and_no_weights():
    from exact_attention_bwd_gb300 import binding as fa
    c = case(2 * 45, 4, 2, 128, 128, False, "bf16", seed=3, max_pos=45)
    q, k = c["q"].reshape(2, 45, 4, 128).contiguous(), c["k"].reshape(2, 45, 2, 128).contiguous()
    x, y = from_dev(q).reshape(90, 4, 128), from_dev(k).reshape(90, 2, 128)
    q2, k2 = fa.qk_norm_rope(q, k, None, None, *c["angles"], eps=EPS, out=(q, k))
    assert q2 is q and k2 is k
    pos = np.arange(90) % 45
    check_rows("q", from_dev(q).reshape(90, 4, 128), x, np.ones(128), *tables(c, pos), False, "bf16")
    check_rows("k", from_dev(k).reshape(90, 2, 128), y, np.ones(128), *tables(c, pos), False, "bf16")


def test_zero_rows_and_large_rows():
    """A row of zeros stays zero (eps keeps the root finite); one of the largest values that the type
    squares to in fp32 is normalised like any other."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case(4, 2, 2, 128, 128, False, "bf16", seed=4)
    c["q"][1] = 0
    c["q"][2] = c["q"][2].sign() * 2.0 ** 59
    q, _ = fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], positions=torch.from_numpy(c["pos"]).cuda(), eps=EPS)
    assert torch.all(q[1] == 0)
    check_rows("q", from_dev(q), from_dev(c["q"]), from_dev(c["wq"]), *tables(c, c["pos"]), False, "bf16")


@pytest.mark.parametrize("T,h_q,h_kv,d,rot,adjacent,kind,page", [
    (1, 32, 8, 128, 128, False, "bf16", 64), (77, 6, 2, 64, 64, True, "f16", 16), (40, 16, 2, 256, 64, False, "bf16", 48),
    (29, 5, 5, 192, 192, False, "f16", 32),
])
def test_append(T, h_q, h_kv, d, rot, adjacent, kind, page):
    """Keys and values land in their slots; padding tokens, slot -1 and every other row of the
    pools stay as they were; a bad position or slot is skipped and reported."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case(T, h_q, h_kv, d, rot, adjacent, kind, seed=T)
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    pos = c["pos"].copy()
    skip = np.zeros(T, bool)       # no output at all
    unstored = np.zeros(T, bool)   # no cache row
    if T > 20:
        pos[3], slots[5] = -1, -1
        pos[7], pos[8], slots[9], slots[10] = -2, 5000, pages * page, -9
        skip[[3, 7, 8]] = True
        unstored[[5, 9, 10]] = True
    caches = [Guarded((pages, page, h_kv, d), torch_type(kind)) for _ in range(2)]
    before = [dev(rng.standard_normal((pages, page, h_kv, d)), kind) for _ in range(2)]
    for g, b in zip(caches, before):
        g.t.copy_(b)
    q_out = torch.full((T, h_q, d), 9.0, dtype=torch_type(kind), device="cuda")
    k_out = torch.full((T, h_kv, d), 9.0, dtype=torch_type(kind), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], positions=torch.from_numpy(pos).cuda(), eps=EPS,
                    interleaved=adjacent, v=c["v"], k_cache=caches[0].t, v_cache=caches[1].t, slots=torch.from_numpy(slots).cuda(),
                    out=(q_out, k_out), status=status)
    for g in caches:
        g.check("cache")
    assert status.item() == (fa.FA_ERR_DEVICE_CHECK if T > 20 else 0)
    live = ~skip
    check_rows("q", from_dev(q_out)[live], from_dev(c["q"])[live], from_dev(c["wq"]), *tables(c, pos[live]), adjacent, kind)
    check_rows("k", from_dev(k_out)[live], from_dev(c["k"])[live], from_dev(c["wk"]), *tables(c, pos[live]), adjacent, kind)
    assert torch.all(q_out[torch.from_numpy(skip).cuda()] == 9) and torch.all(k_out[torch.from_numpy(skip).cuda()] == 9)
    stored = live & ~unstored
    want_k, want_v = (b.clone().view(-1, h_kv, d) for b in before)
    at = torch.from_numpy(slots[stored]).cuda().long()
    rows = torch.from_numpy(stored).cuda()
    want_k[at], want_v[at] = k_out[rows], c["v"][rows]
    assert torch.equal(caches[0].t.view(-1, h_kv, d), want_k) and torch.equal(caches[1].t.view(-1, h_kv, d), want_v)


@pytest.mark.parametrize("T,h_q,h_kv,d,rot,adjacent,kind", SHAPES)
def test_gradient(T, h_q, h_kv, d, rot, adjacent, kind):
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case(T, h_q, h_kv, d, rot, adjacent, kind, seed=T + d + 1, f32_weights=T % 2 == 0)
    rng = np.random.default_rng(T + 2)
    dq_out, dk_out = (dev(rng.standard_normal((T, h, d)), kind) for h in (h_q, h_kv))
    pos = c["pos"].copy()
    if T > 20:
        pos[2] = -1  # a padding token has no part in the sums, and its gradient is not written
    fused = Guarded((T, h_q + 2 * h_kv, d), torch_type(kind))  # the fused projection's gradient
    fused.t.fill_(3.0)
    dw = Guarded((d,), torch.float32), Guarded((d,), torch.float32)
    grads = (fused.t[:, :h_q], fused.t[:, h_q:h_q + h_kv], dw[0].t, dw[1].t)
    args = (c["q"], c["k"], dq_out, dk_out, c["wq"], c["wk"], *c["angles"])
    kw = dict(positions=torch.from_numpy(pos).cuda(), eps=EPS, interleaved=adjacent)
    fa.qk_norm_rope_backward(*args, **kw, grads=grads)
    for g in (fused, *dw):
        g.check("gradient")
    live = pos >= 0
    assert torch.all(fused.t[:, h_q + h_kv:] == 3) and torch.all(fused.t[torch.from_numpy(~live).cuda()] == 3)
    cos, sin = tables(c, pos[live])
    for name, x, w, dy, dx, dwt in (("q", c["q"], c["wq"], dq_out, grads[0], dw[0].t), ("k", c["k"], c["wk"], dk_out, grads[1], dw[1].t)):
        x, w, dy = from_dev(x)[live], from_dev(w), from_dev(dy)[live]
        want, want_w, size_w = ref.norm_rope_bwd(x, w, cos, sin, EPS, adjacent, dy)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
        g = np.abs(ref.rotate(np.abs(dy), np.abs(cos), -np.abs(sin), adjacent, back=True)) + np.abs(
            ref.rotate(np.abs(dy), np.abs(cos), np.abs(sin), adjacent, back=True))
        gw, xh = g * np.abs(w), np.abs(x) * r
        size = r * (gw + xh * np.mean(gw * xh, -1, keepdims=True))
        bound = TYPES[kind] * np.abs(want) + 2.0 ** -17 * size + 2.0 ** -25
        err = np.abs(from_dev(dx)[live] - want)
        assert np.all(err <= bound), ("d" + name, float((err - bound).max()))
        size_w = (g * xh).sum((0, 1))
        err = np.abs(dwt.cpu().numpy().astype(np.float64) - want_w)
        assert np.all(err <= 2.0 ** -16 * size_w + 1e-30), ("dw" + name, float(err.max()))
    again = fa.qk_norm_rope_backward(*args, **kw)
    assert torch.equal(again[2], dw[0].t) and torch.equal(again[3], dw[1].t), "the weights' gradients are the same bits"


def test_gradient_of_no_tokens_is_zero():
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case(0, 4, 2, 64, 64, False, "bf16", seed=9)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(c["q"], c["k"], torch.empty_like(c["q"]), torch.empty_like(c["k"]), c["wq"], c["wk"],
                                                *c["angles"], positions=torch.from_numpy(c["pos"]).cuda())
    assert dq.numel() == 0 and torch.all(dwq == 0) and torch.all(dwk == 0)
    q, k = fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], positions=torch.from_numpy(c["pos"]).cuda())
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
