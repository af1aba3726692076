"""Serving-step and training-step operators at the edges of what their documentation allows: copies that
land out of order, roots of nothing, the largest windows and pages, one slot twice, waits that run out.

Bounds are those of test_gpu_paged and test_gpu_norm_rope, where they are derived.
"""
import numpy as np
import pytest

import step_helpers as ref
from gpu_helpers import from_dev
from test_gpu_norm_rope import TYPES, dev
from test_gpu_page_plan import compare as plan_compare
from test_gpu_paged import HALF, case
from test_gpu_step_calls import arguments, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,h_q,new", [(256, 8, 4), (256, 8, 5), (256, 16, 4), (256, 8, 1), (192, 16, 4), (128, 16, 4), (64, 16, 4)])
def test_values_behind_their_keys(d, h_q, new):
    """Keys that lie in the L2 cache and values that do not: the keys of a sequence's last tile arrive
    ahead of the values of the tile before it.  The last tile's unused value rows hold NaN, which has to be
    cleared in the tile that they belong to, and there alone; call after call the same bits."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    torch.manual_seed(d + h_q + new)
    rng, page, B = np.random.default_rng(d + new), 64, 160
    used = rng.integers(130, 1400, B)
    blocks = -(-used // page)
    pool = int(blocks.sum())
    k, v = (torch.randn(pool, page, 1, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(B * new, h_q, d, device="cuda", dtype=torch.bfloat16)
    order, table, at = rng.permutation(pool), np.zeros((B, blocks.max()), np.int32), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
        if used[b] % page:
            k[int(table[b, n - 1]), used[b] % page:] = float("nan")
            v[int(table[b, n - 1]), used[b] % page:] = float("nan")
    kw = dict(causal=True, cu_q=i32(np.arange(B + 1) * new), seqused_k=i32(used), block_table=i32(table), s_kv=int(used.max()), max_seqlen_q=new)
    flush = torch.empty(64 << 20, device="cuda")  # 256 MB, twice the L2
    results = []
    for _ in range(6):
        flush.fill_(1.0)
        k.view(torch.int16).sum()
        results.append(fa.forward(q, k, v, **kw))
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


@pytest.mark.parametrize("T,h_q,h_kv,d,kind", [(5, 3, 2, 64, "bf16"), (7, 5, 2, 128, "f16"), (6, 3, 1, 192, "bf16"), (9, 5, 3, 256, "f16")])
def test_gradient_without_eps(T, h_q, h_kv, d, kind):
    """eps = 0, and heads that do not fill a warp's batch of rows: lanes without a row leave the
    weights' gradients alone."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    rng = np.random.default_rng(d)
    rot = d // 2
    x = [dev(rng.standard_normal((T, h, d)), kind) for h in (h_q, h_kv)]
    dy = [dev(rng.standard_normal((T, h, d)), kind) for h in (h_q, h_kv)]
    w = [dev(1 + 0.3 * rng.standard_normal(d), kind) for _ in range(2)]
    cos, sin = ref.angles(T, rot)
    got = fa.qk_norm_rope_backward(*x, *dy, *w, *(torch.from_numpy(a).cuda() for a in (cos, sin)), eps=0.0)
    for n in range(2):
        X, DY, W = (from_dev(t[n]) for t in (x, dy, w))
        want, want_w, _ = ref.norm_rope_bwd(X, W, cos, sin, 0.0, False, DY)
        r = 1 / np.sqrt(np.mean(X * X, -1, keepdims=True))
        c, s = np.abs(cos), np.abs(sin)
        g = np.abs(ref.rotate(np.abs(DY), c, -s, False, back=True)) + np.abs(ref.rotate(np.abs(DY), c, s, False, back=True))
        gw, xh = g * np.abs(W), np.abs(X) * r
        size = r * (gw + xh * np.mean(gw * xh, -1, keepdims=True))
        assert np.all(np.abs(from_dev(got[n]) - want) <= TYPES[kind] * np.abs(want) + 2.0 ** -17 * size + 2.0 ** -25)
        err = np.abs(got[2 + n].cpu().numpy().astype(np.float64) - want_w)
        assert np.all(err <= 2.0 ** -16 * (g * xh).sum((0, 1)) + 1e-30)


def test_results_have_their_shapes():
    """A result's tensor of the right size and another shape is refused, as in the other forms of the
    forward: an LSE [T, h_q] would be filled as [h_q, T]."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case([3, 4], [40, 50], h_q=4, h_kv=2, d=64, page=16)
    args, kw = arguments(c)
    q = args[0]
    for bad in (dict(lse=torch.empty(7, 4, device="cuda")), dict(lse=torch.empty(28, device="cuda")),
                dict(out=torch.empty(4, 7, 64, device="cuda", dtype=q.dtype)), dict(out=torch.empty(7, 256, device="cuda", dtype=q.dtype))):
        with pytest.raises(ValueError, match="shape"):
            fa.forward(*args, **kw, **bad)
    k = torch.randn(7, 2, 64, device="cuda", dtype=q.dtype)
    cos, sin = (torch.from_numpy(a).cuda() for a in ref.angles(8, 32))
    rope = dict(positions=i32(np.arange(7)))
    new = lambda *s: torch.empty(*s, device="cuda", dtype=q.dtype)  # noqa: E731
    for out in ((new(4, 7, 64), new(7, 2, 64)), (new(7, 4, 64), new(2, 7, 64)), (new(7, 256), None)):
        with pytest.raises(ValueError, match="shape"):
            fa.qk_norm_rope(q, k, None, None, cos, sin, **rope, out=out)
    with pytest.raises(ValueError, match="shape"):
        fa.qk_norm_rope(q, k, None, None, cos, sin.view(16, 8), **rope)
    with pytest.raises(ValueError, match="shape"):
        fa.qk_norm_rope_backward(q, k, q, k, None, None, cos, sin.view(16, 8), **rope)
    lengths, table = i32([3, 4]), i32(np.zeros((2, 4)))
    n = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    for i, shape in ((0, (1, 3)), (1, (2, 1)), (2, (2, 4)), (3, (4, 2))):
        out = [n(3), n(2), n(8), n(8), n(1)]
        out[i] = n(*shape)
        with pytest.raises(ValueError, match="shape"):
            fa.page_plan(lengths, lengths, table, i32(np.arange(9)), page_size=16, num_pages=9, tokens=8, out=out)


@pytest.mark.parametrize("P,width,cached,fresh", [
    (3 << 29, 1, [(3 << 29) - 1, 0], [1, 0]), (3 << 28, 2, [(3 << 28) + 7, 5, 2 * (3 << 28) - 2], [3, 2, 2]), (2 ** 31 - 1, 1, [2 ** 31 - 5, 1], [4, 3]),
])
def test_page_plan_of_the_largest_pages(P, width, cached, fresh):
    """Page sizes and lengths whose sum passes 31 bits."""
    pages = (2 ** 31 - 1) // P
    plan_compare(dict(cached=np.asarray(cached, np.int32), fresh=np.asarray(fresh, np.int32),
                      table=np.tile(np.arange(width, dtype=np.int32) % pages, (len(cached), 1)), free=np.zeros(0, np.int32), head=0, P=P,
                      num_pages=pages, T=sum(fresh) + 2))


@pytest.mark.parametrize("new,used,d", [([1, 2], [300, 77], 64), ([1, 200], [300, 500], 128), ([300, 3], [300, 9], 256)])
def test_the_largest_windows(new, used, d):
    """A window of 2^31 - 1 keys to either side is no window: the same bits."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    args, kw = arguments(case(new, used, h_q=4, h_kv=2, d=d, page=16))
    kw.pop("causal")
    for causal in (True, False):
        want = fa.forward(*args, **kw, causal=causal)
        for window in ((2 ** 31 - 1, -1), (-1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 2, 2 ** 30)):
            got = fa.forward(*args, **kw, causal=causal, window=window)
            assert fa.device_status(got[2]) == 0
            assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("s_q,s_kv,h_q,h_kv,d", [(130, 300, 4, 2, 64), (300, 300, 16, 1, 128), (70, 260, 4, 4, 256), (1, 500, 8, 2, 128)])
def test_the_largest_windows_of_dense_calls(s_q, s_kv, h_q, h_kv, d):
    """The same in the forward and backward of dense batches, against a window that just hides nothing."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    torch.manual_seed(d)
    new = lambda s, h: torch.randn(2, s, h, d, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, dout, k, v = new(s_q, h_q), new(s_q, h_q), new(s_kv, h_kv), new(s_kv, h_kv)
    big = 2 ** 31 - 1
    for plain, largest in (((5000, -1), (big, -1)), ((-1, 5000), (-1, big)), ((5000, 5000), (big, big))):
        out = []
        for window in (plain, largest):
            o, z, ws = fa.forward(q, k, v, window=window)
            assert fa.device_status(ws) == 0
            grads = fa.backward(q, k, v, o, z, dout, window=window, flags=fa.FA_FLAG_DETERMINISTIC)
            assert fa.device_status(grads[-1]) == 0
            out.append((o, z, *grads[:3]))
        for x, y in zip(*out):
            assert torch.isfinite(x.float()).all() and torch.equal(x, y)


@pytest.mark.parametrize("dense", [False, True])
def test_padding_tokens(dense):
    """Without tensors to write the binding makes the results, and the rows of tokens that take no part are zero
    in them rather than whatever the memory held; in given ones, and in the cache, they stay as they were."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    T, h_q, h_kv, d = 66, 9, 5, 128
    shape = lambda h: (2, T // 2, h, d) if dense else (T, h, d)  # noqa: E731
    torch.manual_seed(5)
    new = lambda h: torch.randn(shape(h), device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, dq_out, k, dk_out, v = new(h_q), new(h_q), new(h_kv), new(h_kv), new(h_kv)
    cos, sin = (torch.from_numpy(a).cuda() for a in ref.angles(50, 64))
    pos = np.arange(T) % 40
    pos[[0, 13, 14, 40, 65]] = -1
    pos[20] = 50  # (outside the table)
    skip = torch.from_numpy((pos < 0) | (pos >= 50)).cuda()
    tables, kw = (None, None, cos, sin), dict(positions=i32(pos))

    def poison():  # (what the allocator hands out next)
        dirty = [torch.full((T * h, d), float("nan"), device="cuda", dtype=torch.bfloat16) for h in (h_q, h_kv) for _ in range(4)]
        del dirty

    pools = [torch.full((5, 16, h_kv, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    append = dict(v=v, k_cache=pools[0], v_cache=pools[1], slots=i32(np.arange(T)))
    for run, given in (
            (lambda **o: fa.qk_norm_rope(q, k, *tables, **kw, **o), lambda x: dict(out=x)),
            (lambda **o: fa.qk_norm_rope(q, k, *tables, **kw, **append, **o), lambda x: dict(out=x)),
            (lambda **o: fa.qk_norm_rope_backward(q, k, dq_out, dk_out, *tables, **kw, **o), lambda x: dict(grads=x))):
        poison()
        got = run()
        own = tuple(None if x is None else torch.full_like(x, 7.0) for x in got)
        run(**given(own))
        for x, y in zip(got[:2], own[:2]):
            if x is not None:
                x, y = x.reshape(T, -1), y.reshape(T, -1)
                assert torch.all(x[skip] == 0) and torch.all(y[skip] == 7) and torch.equal(x[~skip], y[~skip])
        for x, y in zip(got[2:], own[2:]):
            assert torch.equal(x, y)
    for pool in pools:
        assert torch.all(pool.view(80, -1)[:T][skip] == 7) and not torch.any(pool.view(80, -1)[:T][~skip] == 7)
    poison()
    k_new = fa.qk_norm_rope(q, k, *tables, **kw, out=(torch.empty_like(q), None))[1]
    assert torch.all(k_new.reshape(T, -1)[skip] == 0)


def test_one_slot_twice():
    """Two tokens with one slot leave values of either there, eight at a time, and every other row alone."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    T, h_q, h_kv, d, page = 300, 4, 2, 128, 16
    torch.manual_seed(6)
    q, k, v = (torch.randn(T, h, d, device="cuda", dtype=torch.bfloat16) for h in (h_q, h_kv, h_kv))
    slots = np.arange(T) // 2 * 3
    pools = [torch.full((-(-int(slots.max() + 1) // page), page, h_kv, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    _, k_out = fa.qk_norm_rope(q, k, None, None, None, None)
    fa.qk_norm_rope(q, k, None, None, None, None, v=v, k_cache=pools[0], v_cache=pools[1], slots=i32(slots))
    for pool, rows in zip(pools, (k_out, v)):
        pool, rows = pool.view(-1, h_kv * d // 8, 8), rows.reshape(T, -1, 8)
        first, second = ((pool[slots[::2]] == rows[n::2]).all(-1) for n in range(2))
        assert torch.all(first | second)
        others = np.setdiff1d(np.arange(len(pool)), slots)
        assert torch.all(pool[others] == 7)


def test_gradients_over_their_inputs():
    """dq and dk over q and k inside one fused projection, over the incoming gradients, and in rows that lie
    between q's: what does not overlap row by row is taken, with the same bits."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    T, h_q, h_kv, d = 77, 6, 2, 64
    torch.manual_seed(8)
    fused = torch.randn(T, 2 * (h_q + 2 * h_kv), d, device="cuda", dtype=torch.bfloat16)
    dq_out, dk_out = (torch.randn(T, h, d, device="cuda", dtype=torch.bfloat16) for h in (h_q, h_kv))
    cos, sin = (torch.from_numpy(a).cuda() for a in ref.angles(T, 64))
    n = h_q + h_kv
    want = fa.qk_norm_rope_backward(fused[:, :h_q], fused[:, h_q:n], dq_out, dk_out, None, None, cos, sin)
    dw = lambda: [torch.empty(d, device="cuda") for _ in range(2)]  # noqa: E731
    for place in ("inputs", "gradients", "between"):
        x, gq, gk = fused.clone(), dq_out.clone(), dk_out.clone()
        q, k = x[:, :h_q], x[:, h_q:n]
        dq, dk = {"inputs": (q, k), "gradients": (gq, gk), "between": (x[:, n + 4:n + 4 + h_q], x[:, n:n + h_kv])}[place]
        got = fa.qk_norm_rope_backward(q, k, gq, gk, None, None, cos, sin, grads=(dq, dk, *dw()))
        for a, b in zip(got, want):
            assert torch.equal(a, b), place
    with pytest.raises(fa.FaError):
        fa.qk_norm_rope_backward(q, k, gq, gk, None, None, cos, sin, grads=(x[:, 1:1 + h_q], dk, *dw()))


@pytest.mark.parametrize("d,h_q,h_kv,kind", [(64, 16, 4, "f16"), (128, 32, 8, "bf16"), (192, 6, 2, "bf16"), (256, 16, 2, "bf16")])
@pytest.mark.parametrize("form", ["forward", "append", "gradient"])
@pytest.mark.parametrize("rows", ["in the L2", "in memory", "in memory, positions by place"])
def test_norm_rope_wait_limit(form, d, h_q, h_kv, kind, rows):
    """A limit of 1 ns on the waits ends the call with a timeout status, or, where every copy had landed by the
    time that it was looked for, with a right result.  Copies lag for certain where rows come from memory and
    neither positions nor slots are read ahead of them (a read takes as long as a copy).  The same call with
    a long limit, next, has the bits that it had before."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    torch.manual_seed(d)
    T, page = 8192 if rows == "in the L2" else 2 ** 27 // (h_q * d) // 64 * 64, 64
    new = lambda h: torch.randn(T, h, d, device="cuda").to(torch.bfloat16 if kind == "bf16" else torch.float16)  # noqa: E731
    q, k, v, dq_out, dk_out = new(h_q), new(h_kv), new(h_kv), new(h_q), new(h_kv)
    cos, sin = (torch.from_numpy(a).cuda() for a in ref.angles(8192, d))
    places = dict(seq_len=8192) if rows.endswith("place") else dict(positions=i32(np.arange(T) % 8192))
    lags = rows.endswith("place") and form != "append"
    pools = [torch.zeros(T // page, page, h_kv, d, device="cuda", dtype=q.dtype) for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(**kw):
        status.zero_()
        kw.update(**places, status=status)
        if form == "gradient":
            return fa.qk_norm_rope_backward(q, k, dq_out, dk_out, None, None, cos, sin, **kw)
        if form == "forward":
            return fa.qk_norm_rope(q, k, None, None, cos, sin, **kw)
        q_out, _ = fa.qk_norm_rope(q, k, None, None, cos, sin, v=v, k_cache=pools[0], v_cache=pools[1], slots=i32(np.arange(T)), **kw)
        return q_out, pools[0].clone(), pools[1].clone()

    want = run()
    assert status.item() == 0
    for _ in range(3):
        for limit in (1, 10 ** 9):
            got = run(wait_limit_ns=limit)
            code = status.item()
            assert code == 0 or (limit == 1 and code == fa.FA_ERR_TIMEOUT)
            assert limit > 1 or code == fa.FA_ERR_TIMEOUT or not lags
            if code == 0:
                for x, y in zip(got, want):
                    assert torch.equal(x, y)


@pytest.mark.parametrize("d,h_q,h_kv,new,used,hint", [
    *((d, h, 1, [n], [used], n) for d, used in ((64, 60000), (128, 60000), (192, 40000), (256, 40000)) for h, n in ((8, 1), (16, 2), (16, 4))),
    (64, 8, 2, [300], [20000], 0), (128, 8, 2, [300], [20000], 0), (128, 8, 2, [300, 1], [20000, 9000], 0), (192, 8, 2, [300], [9000], 0),
    (256, 8, 2, [300], [9000], 0),
])
def test_paged_wait_limit_of_every_kernel(d, h_q, h_kv, new, used, hint):
    """A limit of 1 ns ends the call with a timeout status in each variant of either kernel (16, 32 and 64 rows;
    chunks): every CTA waits for dozens of tiles from memory.  The next call, without the limit, is right."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    args, kw = arguments(case(new, used, h_q=h_q, h_kv=h_kv, d=d, page=64), hint)
    want, want_lse, ws = fa.forward(*args, **kw)
    assert fa.device_status(ws) == 0
    flush = torch.empty(64 << 20, device="cuda")  # 256 MB, twice the L2
    for _ in range(3):
        flush.fill_(1.0)
        _, _, ws = fa.forward(*args, **kw, wait_limit_ns=1)
        assert fa.device_status(ws) == fa.FA_ERR_TIMEOUT
        o, z, ws = fa.forward(*args, **kw)
        assert fa.device_status(ws) == 0
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(z, want_lse)
