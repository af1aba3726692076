"""Norm + rotation with append to an 8-bit cache, on the GPU against the 64-bit definition.

Bounds.  A new row is rounded once, to e4m3: half a step is 2^-4 of the value, or 2^-10 scales below the
normal range.  Keys carry the rotation's fp32 error ahead of that (2^-17 of the operands' sizes, as in
test_gpu_norm_rope.py); values none.  A block's scale is the one of the definition for some
maximum within that error.  Rows ahead of the new ones are rounded once more where the scale grew."""
import numpy as np
import pytest

import cache8_helpers as c8
import step_helpers as ref
from gpu_helpers import Guarded, from_dev
from test_gpu_norm_rope import EPS, TYPES, torch_type
from test_gpu_rope_axes import PATTERNS, check, rows, tables

pytestmark = pytest.mark.gpu


def append_case(cached, new, h_q, h_kv, d, rot, P, N, kind="bf16", adjacent=False, axes=1, pattern="split", norm=True, spare=0,
                seed=0, size=1.0, max_pos=3000):
    import torch
    rng = np.random.default_rng(seed)
    cached, new = np.asarray(cached), np.asarray(new)
    used = (cached + new).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1]) + spare
    width = max(1, int(-(-used.max() // P)))
    pages = int((-(-used // P)).sum()) + 2
    order, table, at = rng.permutation(pages), np.full((len(new), width), -1, np.int32), 0
    for b, n in enumerate(-(-used // P)):
        table[b, :n] = order[at:at + n]
        at += n
    x = torch.from_numpy(rng.standard_normal((T, h_q + 2 * h_kv, d)) * size * rng.choice([0.05, 1.0, 6.0], (T, 1, 1))).cuda().to(torch_type(kind))
    c = dict(T=T, h_q=h_q, h_kv=h_kv, d=d, rot=rot, adjacent=adjacent, kind=kind, norm=norm, P=P, N=N, cu=cu, used=used, table=table,
             q=x[:, :h_q], k=x[:, h_q:h_q + h_kv], v=x[:, h_q + h_kv:], wq=None, wk=None)
    if norm:
        c["wq"], c["wk"] = (torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).cuda().to(torch_type(kind)) for _ in range(2))
    c["pos"] = rng.integers(0, max_pos, (axes, T)).astype(np.int32)
    c["pos"][:, cu[-1]:] = -1
    c["pair_axis"] = PATTERNS[pattern](rot // 2, axes)
    c["cos"], c["sin"] = ref.angles(max_pos, rot) if rot else (None, None)
    c["angles"] = tuple(None if a is None else torch.from_numpy(a).cuda() for a in (c["cos"], c["sin"]))
    c["cache"] = [c8.random_cache(rng, pages, P, N, h_kv, d) for _ in range(2)]
    for _, scale in c["cache"]:  # what a block's scale was before its first row is written does not count
        scale[rng.random(scale.shape) < 0.1] *= np.float32(2.0 ** 10)
    return c


def run(c, **kw):
    """Runs the append on guarded copies of the cache; returns (q_out, [(bytes, scales) of K, of V])."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    g = []
    for pool, scale in c["cache"]:
        g += [Guarded(pool.shape, torch.uint8), Guarded(scale.shape, torch.float32)]
        g[-2].t.copy_(torch.from_numpy(pool))
        g[-1].t.copy_(torch.from_numpy(scale))
    out = Guarded((c["T"], c["h_q"], c["d"]), torch_type(c["kind"]))
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    args = dict(k_cache=g[0].t, v_cache=g[2].t, k_scale=g[1].t, v_scale=g[3].t, cu_q=i32(c["cu"]), seqused_k=i32(c["used"]),
                block_table=i32(c["table"]), positions=i32(c["pos"]), pair_axis=c["pair_axis"], norm=c["norm"], eps=EPS,
                interleaved=c["adjacent"], out=out.t)
    fa.qk_norm_rope_append8(c["q"], c["k"], c["v"], c["wq"], c["wk"], *c["angles"], **{**args, **kw})
    for x in g + [out]:
        x.check("append8")
    a = [x.t.cpu().numpy() for x in g]
    return out.t, [(a[0], a[1]), (a[2], a[3])]


def verify(c, q, after, stored=None):
    stored = np.ones(c["T"], bool) if stored is None else stored
    cos, sin = tables(c, np.where((c["pos"] < 0) | (c["pos"] >= 3000), 0, c["pos"]))
    live = (c["pos"] >= 0).all(0) & (c["pos"] < 3000).all(0)
    want, size = rows(c, from_dev(c["q"]), c["wq"], cos, sin)
    check("q", from_dev(q)[live], want[live], size[live], c["kind"])
    k, size = rows(c, from_dev(c["k"]), c["wk"], cos, sin)
    args = (stored & live, c["cu"], c["used"], c["table"])
    c8.check_append("k", c["cache"][0], after[0], k, 2.0 ** -17 * size, *args)
    c8.check_append("v", c["cache"][1], after[1], from_dev(c["v"]), np.zeros(1), *args)


CASES = [
    dict(cached=[0], new=[1], h_q=1, h_kv=1, d=64, rot=64, P=16, N=16),
    dict(cached=[63, 64, 200, 15], new=[1, 1, 1, 1], h_q=32, h_kv=8, d=128, rot=128, P=64, N=64, axes=3),
    dict(cached=[5, 0, 17], new=[40, 33, 0], h_q=6, h_kv=3, d=192, rot=96, P=48, N=16, kind="f16", pattern="cycle", axes=2),
    dict(cached=[100, 3, 30], new=[29, 300, 2], h_q=8, h_kv=2, d=256, rot=64, P=256, N=128, adjacent=True, norm=False),
    dict(cached=[7], new=[513], h_q=5, h_kv=1, d=64, rot=16, P=128, N=32, adjacent=True, kind="f16", axes=4, pattern="cycle"),
    dict(cached=[0, 31, 16], new=[3, 1, 16], h_q=4, h_kv=4, d=128, rot=0, P=32, N=32, norm=False, spare=5),
    dict(cached=[1000] * 40, new=[1, 2, 5, 0] * 10, h_q=2, h_kv=2, d=64, rot=32, P=16, N=16, axes=3, spare=3),
]


@pytest.mark.parametrize("kw", CASES)
def test_append(kw):
    c = append_case(seed=len(kw["new"]) + kw["d"], **kw)
    verify(c, *run(c))


@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 2.0 ** 9])
def test_scales_grow_and_rows_are_rescaled(size):
    """Rows behind a block's older ones: with small values its scale stays, with large ones it grows."""
    c = append_case([37, 70, 129], [9, 20, 1], 8, 2, 128, 128, 64, 64, norm=False, size=size, seed=5)
    q, after = run(c)
    verify(c, q, after)
    grown = [(after[i][1] > c["cache"][i][1]).any() for i in range(2)]
    assert all(grown) == (size > 1) or size == 1.0


def test_blocks_without_a_scale_start_anew():
    """An old scale that is no positive finite number counts as 0: the rows ahead become 0."""
    c = append_case([5, 5, 5, 5], [2, 2, 2, 2], 4, 1, 64, 64, 16, 16, seed=9)
    for i, bad in enumerate((np.nan, np.inf, 0.0, -1.0)):
        c["cache"][0][1][c["table"][i, 0]] = bad
        c["cache"][1][1][c["table"][i, 0]] = bad
    q, after = run(c)
    for i in range(2):
        for b in range(4):
            assert not (after[i][0][c["table"][b, 0], :5] & 127).any()
            assert (after[i][1][c["table"][b, 0]] > 0).all()
    verify(c, q, after)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_infinities_nan_zeros_and_the_ends_of_the_range(kind):
    c = append_case([0, 16, 3, 0, 0], [16, 16, 4, 16, 16], 2, 2, 64, 0, 16, 16, norm=False, kind=kind, seed=2)
    t = c["cu"]
    for x in (c["k"], c["v"]):
        x[t[0], 0, 3] = float("inf")
        x[t[0] + 5, 0, 4] = float("-inf")
        x[t[1] + 2, 1, 60] = float("nan")
        x[t[2]:t[3]] = 0
        x[t[3]:t[4]] = 0 if kind == "f16" else 2.0 ** -130  # (below 448 x the smallest scale)
        x[t[4]:t[5]] = 448.0  # a power of two times 448: the scale is 1 exactly
    q, after = run(c)
    verify(c, q, after)
    first = c["table"][4, 0]
    assert (after[0][1][first] == 1).all() and (after[1][1][first] == 1).all()


def test_skipped_tokens_and_bad_places():
    """Tokens at position -1 are not stored and count for no scale; places outside the sequence or the table and pages
    outside the pool set the status and store nothing; the other tokens are as ever."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = append_case([20, 3, 60, 0, 10], [8, 8, 8, 8, 8], 4, 2, 128, 64, 16, 16, axes=2, spare=4, seed=3)
    c["pos"][1, 2] = c["pos"][0, 30] = -1
    c["pos"][:, 8:16] = -1  # a sequence of padding alone
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, after = run(c, status=status)
    assert status.item() == 0
    verify(c, q, after)
    stored = np.ones(c["T"], bool)
    c["used"][2] = c["table"].shape[1] * 16 + 3   # three places behind the table
    c["table"][2, 4] = c["table"][2, 3]           # (a page of its own all the same)
    c["used"][3] = 5                              # three tokens ahead of the sequence's start
    stored[24:27] = False
    c["table"][4, 0], c["table"][4, 1] = 999, -1
    c["pos"][0, 1] = 3000
    q, after = run(c, status=status)
    assert status.item() == fa.FA_ERR_DEVICE_CHECK
    verify(c, q, after, stored)


def test_several_appends_are_a_decode():
    """Tokens one by one: each row keeps within a step of its block's last scale, however often the scale grew."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((40, 6, 64)) * 1.3 ** np.arange(40)[:, None, None]).cuda().bfloat16()
    pools = [torch.zeros(3, 16, 2, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((3, 1, 2), float("nan"), device="cuda") for _ in range(2)]
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    used, pos = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(40):
        used += 1
        fa.qk_norm_rope_append8(x[t:t + 1, :2], x[t:t + 1, 2:4], x[t:t + 1, 4:], None, None, None, None, k_cache=pools[0], v_cache=pools[1],
                                k_scale=scales[0], v_scale=scales[1], cu_q=cu, seqused_k=used, block_table=table, positions=pos, norm=False)
    for i, first in ((0, 2), (1, 4)):
        got = c8.true_values(pools[i].cpu().numpy(), scales[i].cpu().numpy())[[2, 0, 1]].reshape(48, 2, 64)[:40]
        s = np.repeat(scales[i].cpu().numpy()[[2, 0, 1], 0], 16, 0)[:40]
        want = from_dev(x[:, first:first + 2])
        # a block's scale doubles at most 8 times over 16 rows (1.3^15 < 2^6): each rounding is half a step
        bound = np.maximum(2.0 ** -4 * np.abs(want), s[..., None] * 2.0 ** -10) * 1.07 * 8
        assert np.all(np.abs(got - want) <= bound)
        small = np.abs(want) < s[..., None] * 2.0 ** -6  # (only these are rounded more than once)
        assert np.all((np.abs(got - want) <= 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -20)) | small)


def test_in_a_graph_on_another_stream():
    import torch
    c = append_case([20, 47, 3], [5, 1, 30], 4, 2, 128, 128, 16, 16, axes=3, seed=12)
    want = run(c)
    from exact_attention_bwd_gb300 import binding as fa
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    cache = [(torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()) for a, b in c["cache"]]
    first = [(a.clone(), b.clone()) for a, b in cache]
    args = dict(cu_q=i32(c["cu"]), seqused_k=i32(c["used"]), block_table=i32(c["table"]), positions=i32(c["pos"]),
                pair_axis=c["pair_axis"], eps=EPS, k_cache=cache[0][0], k_scale=cache[0][1], v_cache=cache[1][0], v_scale=cache[1][1])
    q = torch.zeros(c["T"], 4, 128, device="cuda", dtype=torch.bfloat16)
    step = lambda: fa.qk_norm_rope_append8(c["q"], c["k"], c["v"], c["wq"], c["wk"], *c["angles"], out=q, **args)  # noqa: E731
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step()
    with torch.cuda.stream(stream):
        for _ in range(2):
            for (a, b), (x, y) in zip(cache, first):
                a.copy_(x)
                b.copy_(y)
            q.zero_()
            graph.replay()
            got = q.clone(), [(a.clone(), b.clone()) for a, b in cache]
            stream.synchronize()
            assert torch.equal(got[0], want[0])
            for (a, b), (x, y) in zip(got[1], want[1]):
                assert np.array_equal(a.cpu().numpy(), x) and np.array_equal(b.cpu().numpy(), y)
