"""Calls of the serving-step operators that their documentation allows and a plain use does not
make: used query lengths, other streams, two calls at once, the workspace-free entry, pools past
32-bit offsets, one page in several tables, more row tiles than the schedule looks at in one go.

Bounds where the oracle is compared: those of test_gpu_paged (probabilities and outputs rounded
once each); where two ways to the same result are compared, the bits are the same.
"""
import ctypes

import numpy as np
import pytest

import step_helpers as ref
from gpu_helpers import from_dev
from test_gpu_paged import HALF, case, compare, gpu, up

pytestmark = pytest.mark.gpu


def i32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def arguments(c, hint=0):
    return [up(c[n], c["kind"]) for n in ("qb", "kb", "vb")], dict(
        causal=True, cu_q=i32(c["cu"]), seqused_k=i32(c["used"]), block_table=i32(c["table"]), s_kv=c["s_kv"], max_seqlen_q=hint)


@pytest.mark.parametrize("d", [64, 256])
def test_used_query_lengths(d):
    """Only the first seqused_q[b] tokens of a slot are queries, aligned to the end of the keys; the
    other rows are left as they were.  Negative and too large values are clamped."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case([9, 300, 1, 20, 5], [50, 700, 90, 20, 64], h_q=6, h_kv=2, d=d, page=16)
    given = [4, 250, 0, 33, -2]
    n = np.clip(given, 0, c["new"])
    (q, k, v), kw = arguments(c)
    out, lse = torch.full_like(q, 7.0), torch.full((6, c["T"]), 7.0, device="cuda")
    _, _, ws = fa.forward(q, k, v, **kw, seqused_q=i32(given), out=out, lse=lse)
    assert fa.device_status(ws) == 0
    rows = np.concatenate([c["cu"][b] + np.arange(n[b]) for b in range(5)])
    want, want_lse, spread = ref.attention(c["q"][rows], c["k"], c["v"], np.concatenate([[0], np.cumsum(n)]), c["used"], c["table"],
                                           causal=True, scale=d ** -0.5)
    got, h = from_dev(out), HALF["bf16"]
    assert np.all(np.abs(got[rows] - want) <= h * np.abs(want) + (h + 2.0 ** -13) * spread + 2.0 ** -24)
    assert np.abs(lse.cpu().numpy()[:, rows] - want_lse).max() <= 3e-4
    rest = np.setdiff1d(np.arange(c["T"]), rows)
    assert np.all(got[rest] == 7) and np.all(lse.cpu().numpy()[:, rest] == 7)


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, and neither on the default one."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    cases = [case([1] * 12 + [200], [300 * (i + 1) for i in range(13)], h_q=8, h_kv=2, d=128, page=64, seed=1),
             case([1, 5, 1, 400], [4000, 900, 70, 2000], h_q=16, h_kv=2, d=256, page=32, seed=2)]
    calls = [arguments(c) for c in cases]
    want = [fa.forward(*a, **kw)[:2] for a, kw in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(10):
        for i, (a, kw) in enumerate(calls):
            with torch.cuda.stream(streams[i]):
                got[i].append(fa.forward(*a, **kw))
    torch.cuda.synchronize()
    for i in range(2):
        for o, z, ws in got[i]:
            assert fa.device_status(ws) == 0
            assert torch.equal(o.view(torch.int16), want[i][0].view(torch.int16)) and torch.equal(z, want[i][1])


@pytest.mark.parametrize("d", [128, 256])
def test_without_a_workspace(d):
    """fa_fwd_noalloc takes the form and gives the same bits."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case([1, 300, 7], [2000, 700, 40], h_q=8, h_kv=2, d=d, page=64)
    (q, k, v), kw = arguments(c)
    want, want_lse, _ = fa.forward(q, k, v, **kw)
    p = fa.make_params(q, k, dtype=fa._type_code(q.dtype), **kw)
    assert fa.fa_fwd_workspace_size(p) <= 64 << 20
    o, z = torch.full_like(q, 7.0), torch.full_like(want_lse, 7.0)
    at = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert fa.fa_fwd_noalloc(p, at(q), at(k), at(v), at(o), at(z), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == fa.FA_OK
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(z, want_lse)


def test_pools_past_32_bit_offsets():
    """Append and attention at the far end of a pool of more than 2^31 values, against a small one."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    T, h_q, h_kv, d, page, far = 200, 8, 8, 128, 64, 33000
    assert far * page * h_kv * d > 2 ** 31
    torch.manual_seed(1)
    qkv = torch.randn(T, h_q + 2 * h_kv, d, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    angles = [torch.from_numpy(x).cuda() for x in ref.angles(T, d)]
    results = []
    for first in (0, far):
        k, v = (torch.empty(first + 4, page, h_kv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        positions = torch.arange(T, device="cuda", dtype=torch.int32)
        q, _ = fa.qk_norm_rope(qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], w, w, *angles, positions=positions, v=qkv[:, h_q + h_kv:],
                               k_cache=k, v_cache=v, slots=positions + first * page)
        for last in (1, T):  # one token, and all of them
            o, z, ws = fa.forward(q[T - last:].contiguous(), k, v, causal=True, cu_q=i32([0, last]), seqused_k=i32([T]),
                                  block_table=i32([[first, first + 1, first + 2, first + 3]]), s_kv=4 * page)
            assert fa.device_status(ws) == 0
            results.append((o, z))
        del k, v
    for (a, x), (b, y) in zip(results[:2], results[2:]):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b) and torch.equal(x, y)


def test_pages_shared_by_sequences():
    """Sequences with a common prefix in the same pages, one of them with the same page twice."""
    c = case([1, 3, 40, 1], [200, 200, 260, 96], h_q=8, h_kv=2, d=128, page=32)
    c["table"][1, :5] = c["table"][2, :5] = c["table"][0, :5]
    c["table"][3, :3] = c["table"][0, 0]
    compare(c)


def test_more_row_tiles_than_one_look():
    """50 row tiles to a head, under a window: the schedule finds an item's place 32 tiles at a time."""
    compare(case([2500, 1, 700], [2600, 40, 700], h_q=5, h_kv=1, d=64, page=48), window=(100, -1))


def test_norm_rope_and_plan_on_a_stream_of_their_own():
    """The whole step on a side stream, captured there, and replayed on another stream."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    T, h_q, h_kv, d, page = 6, 8, 2, 128, 16
    torch.manual_seed(2)
    qkv = torch.randn(T, h_q + 2 * h_kv, d, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    angles = [torch.from_numpy(x).cuda() for x in ref.angles(300, d)]
    k, v = (torch.randn(60, page, h_kv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = i32(np.arange(45).reshape(3, 15))
    cached, fresh, free = i32([20, 0, 200]), i32([1, 4, 1]), i32(np.arange(45, 60))

    def step(table, k, v):
        cu, used, positions, slots, _ = fa.page_plan(cached, fresh, table, free, page_size=page, num_pages=60, tokens=T)
        q, _ = fa.qk_norm_rope(qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], w, w, *angles, positions=positions, v=qkv[:, h_q + h_kv:],
                               k_cache=k, v_cache=v, slots=slots)
        return fa.forward(q, k, v, causal=True, cu_q=cu, seqused_k=used, block_table=table, s_kv=240)

    want = step(table.clone(), k.clone(), v.clone())[0]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = step(table.clone(), k.clone(), v.clone())[0]
        own = [table.clone(), k.clone(), v.clone()]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            replayed = step(*own)[0]
    with torch.cuda.stream(t):
        for _ in range(3):
            replayed.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(side, want) and torch.equal(replayed, want)


@pytest.mark.parametrize("d,h_q,h_kv,new,used,hint", [
    (64, 8, 1, [1], [60000], 1), (64, 16, 1, [4], [60000], 4), (128, 16, 1, [3], [60000], 3), (192, 8, 1, [1], [40000], 1),
    (256, 16, 1, [4], [40000], 4), (128, 8, 2, [300, 1], [20000, 9000], 0), (256, 8, 2, [300, 1], [9000, 20000], 0),
])
def test_wait_limit_in_every_kernel(d, h_q, h_kv, new, used, hint):
    """Each variant's waits are bounded: a limit of 1 ns ends the call with a timeout status (or, where
    nothing had to wait, a right result), and the same call with the default limit is right."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case(new, used, h_q=h_q, h_kv=h_kv, d=d, page=64)
    args, kw = arguments(c, hint)
    want, want_lse, ws = fa.forward(*args, **kw)
    assert fa.device_status(ws) == 0
    _, _, ws = fa.forward(*args, **kw, wait_limit_ns=1)
    assert fa.device_status(ws) in (fa.FA_ERR_TIMEOUT, 0)
    o, z, ws = fa.forward(*args, **kw)
    assert fa.device_status(ws) == 0
    assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(z, want_lse)


@pytest.mark.parametrize("d,h_q,new", [(64, 8, 1), (64, 8, 4), (64, 16, 4), (128, 8, 1), (128, 8, 4), (128, 16, 4), (192, 8, 1), (192, 16, 4),
                                       (256, 8, 1), (256, 8, 4), (256, 16, 4)])
def test_long_streams(d, h_q, new):
    """Some twenty tiles and several items to a CTA, so that its rings go round many times in every
    variant of the few-row kernel; against the plain form in 64 bits, call after call the same bits."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    torch.manual_seed(d + h_q + new)
    rng, page = np.random.default_rng(d + new), 64
    used = rng.integers(6000, 14000, 40)
    blocks = -(-used // page)
    k, v = (torch.randn(int(blocks.sum()), page, 1, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(40 * new, h_q, d, device="cuda", dtype=torch.bfloat16)
    order, table, at = rng.permutation(int(blocks.sum())), np.zeros((40, blocks.max()), np.int32), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    kw = dict(causal=True, cu_q=i32(np.arange(41) * new), seqused_k=i32(used), block_table=i32(table), s_kv=int(used.max()), max_seqlen_q=new)
    results = [fa.forward(q, k, v, **kw) for _ in range(3)]
    o, z, ws = results[0]
    assert fa.device_status(ws) == 0
    for x in results[1:]:
        assert torch.equal(o.view(torch.int16), x[0].view(torch.int16)) and torch.equal(z, x[1])
    h = HALF["bf16"]
    for b, n in enumerate(used):
        rows = slice(b * new, (b + 1) * new)
        kb, vb = (t[torch.from_numpy(table[b, :blocks[b]]).cuda().long()].view(-1, d)[:n].double() for t in (k, v))
        s = torch.einsum("ihd,jd->ihj", q[rows].double(), kb) * d ** -0.5
        i, j = torch.arange(new, device="cuda")[:, None, None], torch.arange(n, device="cuda")
        s = s.masked_fill(j > i + int(n) - new, -float("inf"))
        w = torch.softmax(s, -1)
        want, spread = w @ vb, w @ vb.abs()
        assert torch.all((o[rows].double() - want).abs() <= h * want.abs() + (h + 2.0 ** -13) * spread + 2.0 ** -24)
        assert (z[:, rows].double() - torch.logsumexp(s, -1).T).abs().max() <= 3e-4
