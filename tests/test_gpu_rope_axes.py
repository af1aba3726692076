"""Rotation by positions with several axes, with and without the norm, and its gradient, on the GPU
against the 64-bit formulas.  Bounds as in test_gpu_norm_rope.py (an output is rounded once, eps / 2 of the
value; fp32 ahead of it, 2^-17 of the operands' sizes)."""
import numpy as np
import pytest

import step_helpers as ref
from gpu_helpers import Guarded, from_dev
from test_gpu_norm_rope import EPS, TYPES, case, torch_type

pytestmark = pytest.mark.gpu

PATTERNS = {
    "split": lambda half, axes: sorted(j * axes // half for j in range(half)),
    "cycle": lambda half, axes: [j % axes for j in range(half)],
    "last": lambda half, axes: [axes - 1] * half,
}


def axes_case(T, h_q, h_kv, d, rot, adjacent, kind, axes, pattern, norm, seed):
    import torch
    c = case(T, h_q, h_kv, d, rot, adjacent, kind, seed, f32_weights=T % 2 == 1)
    rng = np.random.default_rng(seed + 1)
    c["pos"] = rng.integers(0, 5000, (axes, T)).astype(np.int32)
    c["pair_axis"] = PATTERNS[pattern](rot // 2, axes)
    c["norm"] = norm
    if not norm:
        c["wq"] = c["wk"] = None
    c["kw"] = dict(positions=torch.from_numpy(c["pos"]).cuda(), pair_axis=c["pair_axis"], norm=norm, eps=EPS, interleaved=adjacent)
    return c


def tables(c, pos=None):
    pos = c["pos"] if pos is None else pos
    if not c["rot"]:
        return np.ones((c["T"], 0)), np.zeros((c["T"], 0))
    at, j = np.asarray(pos)[c["pair_axis"]].T, np.arange(c["rot"] // 2)
    return c["cos"][at, j], c["sin"][at, j]


def rows(c, x, w, cos, sin):
    """(rows in 64 bits, the sizes that their fp32 errors go by)."""
    y = x if not c["norm"] else x / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS) * (1 if w is None else from_dev(w))
    a = np.abs(y)
    size = a + np.abs(ref.rotate(a, np.abs(cos), np.abs(sin), c["adjacent"])) + np.abs(ref.rotate(a, np.abs(cos), np.abs(sin), c["adjacent"], back=True))
    return ref.rotate(y, cos, sin, c["adjacent"]), size


def check(name, got, want, size, kind):
    err, bound = np.abs(got - want), TYPES[kind] * np.abs(want) + 2.0 ** -17 * size + 2.0 ** -25
    assert np.all(err <= bound), (name, float((err - bound).max()))


SHAPES = [
    (1, 32, 8, 128, 128, False, "bf16", 3, "split", False), (37, 12, 12, 64, 64, True, "f16", 2, "split", True),
    (130, 5, 1, 128, 64, False, "f16", 4, "cycle", False), (7, 16, 2, 256, 256, True, "bf16", 3, "cycle", True),
    (19, 6, 3, 192, 192, False, "bf16", 3, "last", True), (33, 9, 3, 192, 16, True, "f16", 2, "cycle", False),
    (4, 2, 2, 256, 0, False, "bf16", 3, "split", False), (3, 40, 8, 256, 48, False, "f16", 1, "split", False),
    (1555, 3, 3, 64, 32, False, "bf16", 3, "split", True), (65, 3, 3, 256, 256, False, "f16", 4, "last", False),
]


@pytest.mark.parametrize("T,h_q,h_kv,d,rot,adjacent,kind,axes,pattern,norm", SHAPES)
def test_forward(T, h_q, h_kv, d, rot, adjacent, kind, axes, pattern, norm):
    from exact_attention_bwd_gb300 import binding as fa
    c = axes_case(T, h_q, h_kv, d, rot, adjacent, kind, axes, pattern, norm, seed=T + d)
    out = Guarded((T, h_q, d), torch_type(kind)), Guarded((T, h_kv, d), torch_type(kind))
    fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], out=(out[0].t, out[1].t), **c["kw"])
    for name, g, x, w in (("q", out[0], c["q"], c["wq"]), ("k", out[1], c["k"], c["wk"])):
        g.check(name)
        check(name, from_dev(g.t), *rows(c, from_dev(x), w, *tables(c)), kind)


@pytest.mark.parametrize("T,h_q,h_kv,d,rot,adjacent,kind,axes,pattern,norm", SHAPES)
def test_gradient(T, h_q, h_kv, d, rot, adjacent, kind, axes, pattern, norm):
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = axes_case(T, h_q, h_kv, d, rot, adjacent, kind, axes, pattern, norm, seed=T + d)
    rng = np.random.default_rng(9)
    gq, gk = (torch.from_numpy(rng.standard_normal((T, h, d))).cuda().to(torch_type(kind)) for h in (h_q, h_kv))
    g = [Guarded((T, h_q, d), torch_type(kind)), Guarded((T, h_kv, d), torch_type(kind))]
    w = [Guarded((d,), torch.float32), Guarded((d,), torch.float32)] if norm else []
    fa.qk_norm_rope_backward(c["q"] if norm else None, c["k"] if norm else None, gq, gk, c["wq"], c["wk"], *c["angles"],
                             grads=(g[0].t, g[1].t, *([x.t for x in w] or [None, None])), **c["kw"])
    cos, sin = tables(c)
    for i, (x, wt, dy) in enumerate(((c["q"], c["wq"], gq), (c["k"], c["wk"], gk))):
        g[i].check("dx")
        x, dy = from_dev(x), from_dev(dy)
        a = np.abs(dy)
        size = a + np.abs(ref.rotate(a, np.abs(cos), np.abs(sin), adjacent)) + np.abs(ref.rotate(a, np.abs(cos), np.abs(sin), adjacent, back=True))
        if not norm:
            check("dx", from_dev(g[i].t), ref.rotate(dy, cos, sin, adjacent, back=True), size, kind)
            continue
        w[i].check("dw")
        wt = from_dev(wt)
        dx, dw, terms = ref.norm_rope_bwd(x, wt, cos, sin, EPS, adjacent, dy)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
        xh = np.abs(x) * r
        check("dx", from_dev(g[i].t), dx, r * (size * np.abs(wt) + xh * np.mean(size * np.abs(wt) * xh, -1, keepdims=True)), kind)
        size_w = (size * xh).sum((0, 1))
        assert np.all(np.abs(from_dev(w[i].t) - dw) <= 2.0 ** -16 * np.maximum(terms, size_w) + 1e-12)


@pytest.mark.parametrize("norm", [False, True])
def test_equal_axes_are_one_axis(norm):
    """The same position on every axis is what one axis gives: the angles are the same numbers."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = axes_case(50, 8, 2, 128, 128, False, "bf16", 3, "split", norm, seed=4)
    one = torch.from_numpy(c["pos"][0]).cuda()
    kw = dict(c["kw"], positions=one[None].expand(3, -1).contiguous())
    several = fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], **kw)
    single = fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], **dict(c["kw"], positions=one, pair_axis=None))
    assert all(torch.equal(a, b) for a, b in zip(several, single))


@pytest.mark.parametrize("norm", [False, True])
def test_padding_and_bad_positions(norm):
    """-1 on any axis is padding; another position outside the tables sets the status; both are skipped."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = axes_case(40, 4, 2, 64, 64, False, "f16", 3, "cycle", norm, seed=6)
    pos = c["pos"].copy()
    pos[2, 3] = pos[:, 7] = pos[0, 39] = -1
    skipped = [3, 7, 39]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(c["kw"], positions=torch.from_numpy(pos).cuda(), status=status)
    good = np.setdiff1d(np.arange(40), skipped)
    full = fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], **c["kw"])
    for bad in (False, True):
        if bad:
            pos[1, 11], pos[2, 12] = 5000, -2
            skipped += [11, 12]
            good = np.setdiff1d(good, skipped)
            kw["positions"] = torch.from_numpy(pos).cuda()
        q, k = fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], **kw)
        assert status.item() == (fa.FA_ERR_DEVICE_CHECK if bad else 0)
        for got, want in ((q, full[0]), (k, full[1])):
            assert torch.equal(got[good], want[good]) and not got[skipped].any()
        kept = [torch.full_like(x, 7.0) for x in (q, k)]
        fa.qk_norm_rope(c["q"], c["k"], c["wq"], c["wk"], *c["angles"], out=tuple(kept), **kw)
        assert all((x[skipped] == 7).all() for x in kept)
        dq, dk, *_ = fa.qk_norm_rope_backward(c["q"], c["k"], q, k, c["wq"], c["wk"], *c["angles"], **kw)
        assert not dq[skipped].any() and not dk[skipped].any() and dq[good].any()


def test_append_with_axes_and_without_the_norm():
    """The 16-bit append takes both: the cache's keys are the rows that k_out would hold."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = axes_case(33, 8, 2, 128, 64, True, "bf16", 2, "split", False, seed=8)
    pools = [torch.zeros(6, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.randperm(96, device="cuda")[:33].to(torch.int32)
    q, _ = fa.qk_norm_rope(c["q"], c["k"], None, None, *c["angles"], v=c["v"], k_cache=pools[0], v_cache=pools[1], slots=slots, **c["kw"])
    want = fa.qk_norm_rope(c["q"], c["k"], None, None, *c["angles"], **c["kw"])
    assert torch.equal(q, want[0])
    assert torch.equal(pools[0].view(96, 2, 128)[slots.long()], want[1]) and torch.equal(pools[1].view(96, 2, 128)[slots.long()], c["v"])


def test_gradient_in_place_and_in_a_graph():
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = axes_case(70, 8, 2, 128, 128, False, "bf16", 3, "cycle", False, seed=11)
    g = [torch.randn(70, h, 128, device="cuda", dtype=torch.bfloat16) for h in (8, 2)]
    first = [x.clone() for x in g]
    want = fa.qk_norm_rope_backward(None, None, *g, None, None, *c["angles"], **c["kw"])[:2]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    run = lambda: fa.qk_norm_rope_backward(None, None, *g, None, None, *c["angles"], grads=(*g, None, None), workspace=ws, **c["kw"])  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        for x, y in zip(g, first):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("adjacent", [False, True])
def test_infinities_behind_the_rotated_part_stay_where_they_are(adjacent):
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = axes_case(9, 2, 2, 128, 32, adjacent, "bf16", 2, "split", False, seed=3)
    c["q"][4, 1, 90], c["k"][5, 0, 40], c["q"][2, 0, 41] = float("inf"), float("-inf"), float("nan")
    q, k = fa.qk_norm_rope(c["q"], c["k"], None, None, *c["angles"], **c["kw"])
    assert torch.equal(q[..., 32:].nan_to_num(7), c["q"][..., 32:].nan_to_num(7)) and torch.equal(k[..., 32:], c["k"][..., 32:])
    assert q[..., :32].isfinite().all() and k[..., :32].isfinite().all()
    dq, dk, *_ = fa.qk_norm_rope_backward(None, None, c["q"].contiguous(), c["k"].contiguous(), None, None, *c["angles"], **c["kw"])
    assert torch.equal(dq[..., 32:].nan_to_num(7), c["q"][..., 32:].nan_to_num(7)) and torch.equal(dk[..., 32:], c["k"][..., 32:])
