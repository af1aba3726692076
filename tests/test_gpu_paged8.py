"""Attention of packed queries over a cache in 8 bits, on the GPU against the 64-bit oracle on the
values that the bytes stand for.

Bound of O, element by element: the output is rounded once (half a step h of its type), each probability
times its value's scale is rounded once to 16 bits before the second product (to fp16, 2^-11, or for
sequences of many rows to the queries' type, as keys and values times their scales are there: a power of two
times an e4m3 value is a value of that type), and a score of d products has an error of at most
d 2^-24 of the sum of their sizes, which changes its probability by as much (and their sum as well).  The LSE has
the scores' error.  Below fp16's normal range a rounding is half of its smallest step, 2^-25, where a row's largest
product of probability and scale is 1 and more: in all at most 2^-25 max_j(p_j vs_j) sum_j |byte_j| <= 2^-25
sum_j(p_j vs_j) sum_j |byte_j|."""
import numpy as np
import pytest

import cache8_helpers as c8
import step_helpers as ref
from gpu_helpers import Guarded, from_dev
from test_gpu_paged import HALF, draw, up

pytestmark = pytest.mark.gpu


def case(new, used, *, h_q, h_kv, d, page, block=None, kind="bf16", seed=0, spare=3, extra_rows=0, sinks=False, v_spread=1.0):
    """Sequences of new[b] query tokens over caches of used[b] keys, pages in random order."""
    rng = np.random.default_rng(seed + 1000 * d + page)
    blocks = [-(-n // page) for n in used]
    width, pool = max(blocks + [1]), sum(blocks) + spare
    order = rng.permutation(pool)
    table = rng.integers(-5, pool + 50, (len(used), width))  # entries that are not needed: anything
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    c = dict(used=np.asarray(used, np.int32), cu=cu, table=table.astype(np.int32), kind=kind, T=int(cu[-1]) + extra_rows,
             s_kv=max(list(used) + [1]), d=d, h_q=h_q, h_kv=h_kv)
    c["qb"], c["q"] = draw(rng, (c["T"], h_q, d), kind)
    block = block or page
    c["k"] = c8.random_cache(rng, pool, page, block, h_kv, d, 0.5)
    c["v"] = c8.random_cache(rng, pool, page, block, h_kv, d, v_spread)
    c["sinks"] = rng.standard_normal(h_q).astype(np.float32) if sinks else None
    return c


def gpu(c, *, causal=True, window=(-1, -1), hint=0, flags=0, scale=None):
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q = up(c["qb"], c["kind"])
    out, lse = Guarded(q.shape, q.dtype), Guarded((c["h_q"], c["T"]), torch.float32)
    k, v = i32(c["k"][0]), i32(c["v"][0])
    kw = dict(causal=causal, window=window, softmax_scale=scale, sinks=None if c["sinks"] is None else i32(c["sinks"]), cu_q=i32(c["cu"]),
              seqused_k=i32(c["used"]), block_table=i32(c["table"]), s_kv=c["s_kv"], flags=flags, max_seqlen_q=hint)
    p = fa.make_params(q, k, **kw, dtype=fa._type_code(q.dtype))
    scales = i32(c["k"][1]), i32(c["v"][1])
    p.cache_dtype, p.scale_block = fa.FA_DTYPE_E4M3, k.shape[1] // scales[0].shape[1]
    p.k_scale, p.v_scale = scales[0].data_ptr(), scales[1].data_ptr()
    ws = Guarded((fa.fa_fwd_workspace_size(p),), torch.uint8)
    o, z, w = fa.forward(q, k, v, **kw, cache_scale=scales, out=out.t, lse=lse.t, workspace=ws.t)
    torch.cuda.synchronize()
    status = fa.device_status(w)
    for name, g in (("O", out), ("LSE", lse), ("workspace", ws)):
        g.check(name)
    return o, z, status


def compare(c, *, causal=True, window=(-1, -1), scale=None, rounding=None, **kw):
    import torch
    o, z, status = gpu(c, causal=causal, window=window, scale=scale, **kw)
    assert status == 0
    n, d = int(c["cu"][-1]), c["d"]
    scale = scale or d ** -0.5
    k, v = c8.true_values(*c["k"]), c8.true_values(*c["v"])
    want, lse, spread = ref.attention(c["q"][:n], k, v, c["cu"], c["used"], c["table"], causal=causal, window=window, scale=scale,
                                      sinks=None if c["sinks"] is None else c["sinks"].astype(np.float64))
    most = max((np.abs(ref.gather(k, c["table"], c["used"])).sum(-1).max() if c["used"].sum() else 0) * np.abs(c["q"]).max(), 1)
    score = min(most * scale * d * 2.0 ** -24, 2.0 ** -9) + 2.0 ** -18
    h = HALF[c["kind"]]
    unit = c8.true_values(np.full_like(c["v"][0], 0x38), c["v"][1])  # the scales (0x38 is 1)
    units, _, _ = ref.attention(c["q"][:n], k, unit, c["cu"], c["used"], c["table"], causal=causal, window=window, scale=scale,
                                sinks=None if c["sinks"] is None else c["sinks"].astype(np.float64))
    sizes = np.zeros_like(want)  # sum of the bytes' sizes over a sequence's keys
    for b in range(len(c["used"])):
        x = np.abs(c8.E4M3[ref.gather(c["v"][0], c["table"][b:b + 1], c["used"][b:b + 1])]).sum(0)
        sizes[c["cu"][b]:c["cu"][b + 1]] = np.repeat(x, c["h_q"] // c["h_kv"], 0)
    small = 2.0 ** -25 * units * sizes
    err, bound = np.abs(from_dev(o)[:n] - want), h * np.abs(want) + (max(rounding or h, 2.0 ** -11) + 2 * score) * spread + small + 2.0 ** -24 * (c["kind"] == "f16")
    assert np.all(err <= bound), (float(err.max()), float((err - bound).max()), np.argwhere(~(err <= bound))[:4])
    got = z.cpu().numpy()[:, :n].astype(np.float64)
    fin = np.isfinite(lse)
    assert np.array_equal(np.isneginf(got), np.isneginf(lse))
    off = np.abs(got[fin] - lse[fin])
    assert np.all(off <= score + 2.0 ** -22 * np.abs(lse[fin])), float(off.max())
    # rows behind the last sequence keep their bytes
    assert torch.all(o[n:].contiguous().view(torch.uint8) == 0xFF) and torch.all(z[:, n:].contiguous().view(torch.uint8) == 0xFF)
    return o, z


HEADS = [(64, 5, 1), (128, 8, 2), (192, 3, 3), (256, 16, 2)]


@pytest.mark.parametrize("d,h_q,h_kv", HEADS)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_decode(d, h_q, h_kv, kind):
    """One token a sequence: caches of one key, around a warp's, a tile's and a page's end, long ones."""
    used = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 700, 3001]
    compare(case([1] * len(used), used, h_q=h_q, h_kv=h_kv, d=d, page=16, kind=kind), hint=1, rounding=2.0 ** -11)


@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (48, 48), (48, 16), (64, 32), (80, 80), (96, 48), (128, 64), (256, 256), (384, 128)])
def test_pages_and_blocks(page, block):
    used = [page - 1, page, page + 1, 5 * page + 3, 1000]
    compare(case([1, 3, 1, 7, 2], used, h_q=8, h_kv=2, d=128, page=page, block=block), hint=7)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 24, 32, 33, 40, 64, 65, 128])
def test_rows_of_a_tile(d, rows):
    """From one row to a head to several tiles of them: rows tokens of one head, a token of rows heads."""
    used = [300, 129, 40]
    compare(case([rows, 1, min(rows, 5)], used, h_q=2, h_kv=2, d=d, page=32, kind="f16"), hint=rows)
    compare(case([1, 1, 1], used, h_q=rows, h_kv=1, d=d, page=64, block=16), hint=1)


@pytest.mark.parametrize("d,h_q,h_kv", HEADS)
@pytest.mark.parametrize("hint", [0, 300])
def test_ragged_chunks(d, h_q, h_kv, hint):
    """Decodes, drafts, chunks, a whole prompt, a sequence without queries and one without keys."""
    new = [1, 0, 5, 130, 64, 1, 17, 300, 2]
    used = [400, 90, 5, 130, 1000, 1, 33, 301, 0]
    compare(case(new, used, h_q=h_q, h_kv=h_kv, d=d, page=32, kind="bf16" if hint else "f16", extra_rows=9), hint=hint)


@pytest.mark.parametrize("window,causal", [((100, -1), True), ((0, -1), True), ((200, 30), False), ((-1, 0), False), ((-1, -1), False),
                                           ((5, 300), False)])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_masks(window, causal, d):
    """Windows and no mask; rows that see nothing (fewer keys than queries) give 0 and -inf, or the sink."""
    c = case([1, 40, 200, 3, 20], [500, 40, 777, 130, 6], h_q=4, h_kv=2, d=d, page=48, block=16)
    o, z = compare(c, window=window, causal=causal)
    if causal:
        assert np.all(np.isneginf(z[:, c["cu"][4]].cpu().numpy())) and np.all(from_dev(o)[c["cu"][4]] == 0)
    compare(dict(c, sinks=np.linspace(-2, 3, 4).astype(np.float32)), window=window, causal=causal)


@pytest.mark.parametrize("chunk", [1, 5, 200])
def test_scales_of_all_sizes(chunk):
    """Value scales over 2^-60 .. 2^60 from block to block, some 0 and some the smallest: a row's error goes by its own terms."""
    c = case([chunk, chunk], [900, 250], h_q=8, h_kv=2, d=128, page=64, block=16, v_spread=20.0, kind="bf16")
    rng = np.random.default_rng(1)
    scale = c["v"][1]
    np.clip(scale, 2.0 ** -60, 2.0 ** 60, out=scale)
    scale[rng.random(scale.shape) < 0.2] = 0.0
    scale[rng.random(scale.shape) < 0.2] = 2.0 ** -126
    c["k"][1][rng.random(scale.shape) < 0.2] = 0.0
    compare(c, hint=chunk)


@pytest.mark.parametrize("chunk", [1, 5, 200])
def test_scales_that_are_no_powers_of_two(chunk):
    c = case([chunk, chunk], [900, 250], h_q=8, h_kv=2, d=128, page=32, block=32)
    rng = np.random.default_rng(1)
    for pool in (c["k"], c["v"]):
        pool[1][:] *= (1 + rng.random(pool[1].shape)).astype(np.float32)
    # (a chunk's kernel rounds key * scale to the queries' type, half a step h: d products with errors of h of their sizes)
    compare_loose = chunk > 64
    if compare_loose:
        o, z, status = gpu(c, hint=chunk)
        n, d = int(c["cu"][-1]), 128
        k, v = c8.true_values(*c["k"]), c8.true_values(*c["v"])
        want, lse, spread = ref.attention(c["q"], k, v, c["cu"], c["used"], c["table"], causal=True, scale=d ** -0.5)
        sizes = max(np.abs(c["q"][i]).max() for i in range(n)) * np.abs(ref.gather(k, c["table"], c["used"])).sum(-1).max() * d ** -0.5
        assert status == 0 and np.all(np.abs(from_dev(o) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * (1 + sizes) * spread)
        assert np.abs(z.cpu().numpy() - lse).max() <= 2.0 ** -8 * sizes
    else:
        compare(c, hint=chunk)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("chunk", [1, 9, 150])
def test_what_lies_behind_the_used_keys(d, chunk):
    """NaN bytes and NaN scales in pages and rows that no query sees change no bit."""
    used = [250, 70, 513]
    c = case([chunk, 3, chunk], used, h_q=4, h_kv=2, d=d, page=48, block=16)
    first = gpu(c, hint=chunk)
    seen = np.zeros(c["k"][0].shape[:2], bool)
    for b, n in enumerate(used):
        seen[c["table"][b, np.arange(n) // 48], np.arange(n) % 48] = True
    dark = ~seen.reshape(len(seen), 3, 16).any(-1)
    for pool, scale in (c["k"], c["v"]):
        pool[~seen] = 0x7F
        scale[dark] = np.nan
    again = gpu(c, hint=chunk)
    assert first[2] == again[2] == 0
    assert np.array_equal(from_dev(first[0]), from_dev(again[0])) and np.array_equal(first[1].cpu().numpy(), again[1].cpu().numpy())


@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_chunks_of_fp16_beyond_its_largest_value(d):
    """A byte times its scale that fp16 rounds to infinity becomes fp16's largest value in the 16-bit tiles of a chunk (a scale that is a
    power of two lies up to twice above what its block needs), and NaN stays NaN.  Each query sees one key, so P is 1
    but for the rounding of its exponent, 65504 (1 + 2^-20) rounds to 65504, and what is NaN is known."""
    n, sign = 200, np.where(np.arange(d) % 3 == 0, -1.0, 1.0)
    c = case([n], [n], h_q=4, h_kv=2, d=d, page=32, kind="f16")
    page, row = c["table"][0, np.arange(n) // 32], np.arange(n) % 32
    pool, scale = c["v"]
    pool[...] = np.where(sign < 0, 0xF8, 0x78)  # 256
    scale[...] = 256.0
    c["k"][0][page[130], row[130], 0, 5] = 0x7F
    pool[page[70], row[70], 1, 7] = 0xFF
    o, z, status = gpu(c, window=(0, 0))
    out = from_dev(o)
    assert status == 0
    assert np.isnan(out[130, :2]).all() and np.isnan(out[70, 2:, 7]).all()
    out[130, :2] = out[70, 2:, 7] = np.nan
    near = np.isnan(out)  # (a value's NaN may reach the same sequence's other queries, at its head and column)
    near[130, :2] = near[:, 2:, 7] = False
    assert not near.any()
    want = np.broadcast_to(65504.0 * sign, out.shape)
    assert np.array_equal(np.where(np.isnan(out), want, out), want)


def test_large_and_small_queries():
    """Rows of queries from 2^-40 to 2^60 (bf16), zeros among them: they are brought into fp16's range by their own power."""
    from exact_attention_bwd_gb300 import inputs
    c = case([9, 40], [200, 90], h_q=8, h_kv=2, d=128, page=32)
    rng = np.random.default_rng(2)
    q = (c["q"] * 2.0 ** rng.integers(-40, 60, c["q"].shape[:2])[..., None]).astype(np.float32)
    q[3, 2] = q[30] = 0
    q[5, 1, 1:] = 0
    c["qb"] = inputs.bf16_bits(q)
    c["q"] = inputs.bf16_to_f64(c["qb"])
    o, z, status = gpu(c, hint=9)
    want, lse, spread = ref.attention(c["q"], c8.true_values(*c["k"]), c8.true_values(*c["v"]), c["cu"], c["used"], c["table"], causal=True, scale=128 ** -0.5)
    assert status == 0 and np.isfinite(from_dev(o)).all()
    # scores of a row are off by at most 128 x 2^-24 of the sum of their products' sizes; where that is small, so is O's error
    size = np.abs(c["q"]).max(-1) * np.abs(c8.true_values(*c["k"])).sum(-1).max() * 128 ** -0.5
    fine = size * 128 * 2.0 ** -24 < 2.0 ** -10
    err = np.abs(from_dev(o) - want)
    assert fine.any() and np.all(err[fine] <= (2.0 ** -8 * np.abs(want) + 2.0 ** -7 * spread)[fine])
    assert np.all(np.abs(z.cpu().numpy().T - lse.T) <= size * 128 * 2.0 ** -24 + 2.0 ** -18 + 2.0 ** -22 * np.abs(lse.T))


def test_bad_table_entries_and_validation():
    from exact_attention_bwd_gb300 import binding as fa
    for chunk in (1, 200):
        c = case([chunk, 1], [300, 40], h_q=4, h_kv=2, d=128, page=16)
        c["table"][0, 5] = c["k"][0].shape[0]
        assert gpu(c, hint=chunk)[2] == fa.FA_ERR_DEVICE_CHECK
        c["table"][0, 5] = -1
        assert gpu(c, hint=chunk)[2] == fa.FA_ERR_DEVICE_CHECK
        c = case([chunk, 1], [300, 40], h_q=4, h_kv=2, d=128, page=16)
        c["used"][1] = 1000
        o, z, status = gpu(c, hint=chunk, flags=fa.FA_FLAG_VALIDATE_CU)
        assert status == fa.FA_ERR_DEVICE_CHECK and np.isnan(from_dev(o)).all()  # nothing was written


@pytest.mark.parametrize("chunk", [1, 300])
def test_same_bits_and_no_split(chunk):
    from exact_attention_bwd_gb300 import binding as fa
    c = case([chunk, 1, chunk], [4000, 90, 2500], h_q=8, h_kv=2, d=64, page=64, block=32, sinks=True)
    a, b = gpu(c), gpu(c)
    assert np.array_equal(from_dev(a[0]), from_dev(b[0])) and np.array_equal(a[1].cpu().numpy(), b[1].cpu().numpy())
    compare(c, flags=fa.FA_FLAG_NO_SPLIT)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes, its last pages in use."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    small = case([1, 3, 150], [200, 77, 400], h_q=8, h_kv=8, d=128, page=64)
    pages = (1 << 32) // (64 * 8 * 128) + small["k"][0].shape[0] + 5
    shift = pages - small["k"][0].shape[0]
    want = gpu(small)
    big = []
    for pool, scale in (small["k"], small["v"]):
        x = torch.empty(pages, 64, 8, 128, dtype=torch.uint8, device="cuda")
        y = torch.empty(pages, 1, 8, dtype=torch.float32, device="cuda")
        x[shift:], y[shift:] = torch.from_numpy(pool).cuda(), torch.from_numpy(scale).cuda()
        big += [x, y]
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    table = small["table"].copy()
    table[(table >= 0) & (table < pages - shift)] += shift
    o, z, ws = fa.forward(up(small["qb"], "bf16"), big[0], big[2], causal=True, cu_q=i32(small["cu"]), seqused_k=i32(small["used"]),
                          block_table=i32(table), s_kv=400, cache_scale=(big[1], big[3]))
    assert fa.device_status(ws) == 0
    assert torch.equal(o, want[0]) and torch.equal(z, want[1])


@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_a_wait_limit_ends_chunks_with_a_timeout(d):
    """The chunks' kernels give up after 1 ns; the same call without the limit is right next (nothing was left behind).
    The few-row kernel waits for its own copies only and has no limit to pass."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case([300, 200], [3000, 700], h_q=8, h_kv=2, d=d, page=16)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    kw = dict(causal=True, cu_q=i32(c["cu"]), seqused_k=i32(c["used"]), block_table=i32(c["table"]), s_kv=3000,
              cache_scale=(i32(c["k"][1]), i32(c["v"][1])))
    q, k, v = up(c["qb"], "bf16"), i32(c["k"][0]), i32(c["v"][0])
    want, lse, ws = fa.forward(q, k, v, **kw)
    assert fa.device_status(ws) == 0
    for _ in range(2):
        _, _, ws = fa.forward(q, k, v, **kw, wait_limit_ns=1)
        assert fa.device_status(ws) == fa.FA_ERR_TIMEOUT
        o, z, ws = fa.forward(q, k, v, **kw)
        assert fa.device_status(ws) == 0 and torch.equal(o, want) and torch.equal(z, lse)
