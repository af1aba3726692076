"""Calls of the operators over an 8-bit cache at the edges of what the header allows, on the GPU against the 64-bit
definition.  Bounds are those of test_gpu_append8.py and test_gpu_paged8.py."""
import numpy as np
import pytest

import cache8_helpers as c8
import step_helpers as ref
import test_gpu_append8 as ap
import test_gpu_paged8 as at
from gpu_helpers import from_dev

pytestmark = pytest.mark.gpu


def behind(c, rows):
    """The case with `rows` tokens of no sequence ahead of the first one (the case has as many to spare)."""
    c["cu"] = (c["cu"] + rows).astype(np.int32)
    assert c["cu"][-1] == c["T"]
    c["pos"] = np.random.default_rng(rows).integers(0, 3000, c["pos"].shape).astype(np.int32)
    return c


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 48, 100, 700])
@pytest.mark.parametrize("kw", [
    dict(cached=[39, 9, 199], new=[1, 1, 1], h_q=2, h_kv=1, d=64, rot=64, P=16, N=16),          # decodes behind a prompt's rows
    dict(cached=[0], new=[32], h_q=2, h_kv=2, d=128, rot=64, P=16, N=16, axes=2),
    dict(cached=[500, 0, 3], new=[40, 5, 0], h_q=4, h_kv=2, d=192, rot=96, P=96, N=48, kind="f16"),
])
def test_append_with_rows_ahead_of_the_first_sequence(rows, kw):
    """Offsets that begin behind 0, with caches shorter and longer than that many rows: rows ahead of them are stored nowhere."""
    import torch
    c = behind(ap.append_case(seed=rows, spare=rows, **kw), rows)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ap.verify(c, *ap.run(c, status=status))
    assert status.item() == 0


def test_append_with_offsets_that_decrease():
    """The status is set, and nothing outside the blocks of the sequences' new places is written."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = ap.append_case([64] * 40, [3] * 40, 2, 2, 64, 64, 16, 16, seed=4)
    c["cu"][10:20] = c["cu"][10:20][::-1].copy()
    c["cu"][30] = -7
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, after = ap.run(c, status=status)
    assert status.item() == fa.FA_ERR_DEVICE_CHECK
    mine = np.zeros(c["cache"][0][0].shape[0], bool)
    for b in range(40):
        mine[c["table"][b][c["table"][b] >= 0]] = True
    for (pool, scale), (pool2, scale2) in zip(c["cache"], after):
        assert np.array_equal(pool[~mine], pool2[~mine]) and np.array_equal(scale[~mine], scale2[~mine])


def groups_case(new, groups, d, seed=0):
    """One sequence over 528 keys in pages of 16.  Its queries are ones and groups[g] = (e, b, s): the keys of group g
    have the byte b and the scale 2^e, which is a score of 2^e E4M3[b] at softmax scale 1 / d, their values random bytes and the
    scale s (groups that are not named: score 0, value scale 0).  Groups 0, 8, 16, ... lie in one warp's stream."""
    from exact_attention_bwd_gb300 import inputs
    c = at.case([new], [528], h_q=4, h_kv=2, d=d, page=16, seed=seed)
    q = np.ones(c["q"].shape, np.float32)
    c["qb"], c["q"] = inputs.bf16_bits(q), q.astype(np.float64)
    c["k"][0][...], c["k"][1][...], c["v"][1][...] = 0, 1.0, 0.0
    for g, (e, b, s) in groups.items():
        page = c["table"][0, g]
        c["k"][0][page], c["k"][1][page], c["v"][1][page] = b, 2.0 ** e, s
    return c


def far_scores(c, d, new):
    """Bounds of test_gpu_paged8.py for scores of up to 2^8 units, which are off by 2^-13 at most (five roundings of 2^-24), and the
    probabilities below fp32's normal range, which are 0 on the GPU: 2^-126 sum_j vs_j |byte_j| at most."""
    o, z, status = at.gpu(c, causal=False, scale=1.0 / d, hint=new)
    assert status == 0
    v = c8.true_values(*c["v"])
    args = (c["cu"], c["used"], c["table"])
    want, lse, spread = ref.attention(c["q"], c8.true_values(*c["k"]), v, *args, causal=False, scale=1.0 / d)
    unit = c8.true_values(np.full_like(c["v"][0], 0x38), c["v"][1])
    units, _, _ = ref.attention(c["q"], c8.true_values(*c["k"]), unit, *args, causal=False, scale=1.0 / d)
    sizes = np.repeat(np.abs(c8.E4M3[ref.gather(c["v"][0], c["table"], c["used"])]).sum(0), 2, 0)  # (two query heads to a group)
    gone = 2.0 ** -126 * np.repeat(np.abs(ref.gather(v, c["table"], c["used"])).sum(0), 2, 0)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12) * spread + 2.0 ** -25 * units * sizes + gone
    err = np.abs(from_dev(o) - want)
    assert np.all(err <= bound), (float(err.max()), float((err - bound).max()), np.argwhere(~(err <= bound))[:4])
    assert np.abs(z.cpu().numpy() - lse).max() <= 2.0 ** -13


HIGHEST = [(6, 0x3D)]  # a score of 104: 150 in powers of two


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("new", [1, 5, 200])
@pytest.mark.parametrize("first,last", [(8.0, 0.0), (8.0, 2.0 ** -126), (2.0 ** 40, 0.0), (2.0 ** 100, 2.0 ** -126), (1.0, 2.0 ** -60)])
def test_scores_that_leave_all_before_them_behind(d, new, first, last):
    """Keys whose scores pass those before them by 2^150 and whose values are 0, or nearly: the output is theirs, not NaN."""
    far_scores(groups_case(new, {0: (0, 0, first), 8: (0, 0, first), 16: (*HIGHEST[0], last), 32: (*HIGHEST[0], last)}, d), d, new)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("new", [1, 5, 200])
@pytest.mark.parametrize("first,last", [(2.0 ** -50, 2.0 ** 60), (2.0 ** -50, 2.0 ** 65), (2.0 ** -57, 2.0 ** 52), (2.0 ** -100, 2.0 ** 16)])
def test_large_values_of_small_probabilities(d, new, first, last):
    """Keys far below the highest score whose values are as much larger: both count (2^-115 last is about first)."""
    far_scores(groups_case(new, {0: (6, 0x3A, first), 16: (0, 0, last), 32: (0, 0, last)}, d), d, new)


@pytest.mark.parametrize("d,G,new", [(64, 4, 1), (64, 4, 4), (64, 4, 8), (128, 4, 1), (128, 4, 4), (128, 4, 8), (192, 4, 2), (192, 4, 4),
                                     (256, 4, 2), (256, 4, 4)])
@pytest.mark.parametrize("long", [False, True])
def test_a_wait_limit_ends_the_few_row_kernel_with_a_timeout(d, G, new, long):
    """Each tile of the few-row kernel: a limit of 1 ns ends it with a timeout, and the same call without the limit is right next (no
    copy landed late, nothing was left behind).  Whether anything is waited for is a matter of speed where the arithmetic is the longer
    part, and where a CTA has one tile (short caches): those calls may end either way, and are right where they end well."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    g = torch.Generator(device="cuda").manual_seed(d)
    B, page = (25, 32) if long else (100, 128)
    used, i32 = (40000 - 777 * np.arange(B) if long else 128 - np.arange(B)), lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
    blocks = -(-used // page)
    table = np.zeros((B, blocks.max()), np.int32)
    for b in range(B):
        table[b, :blocks[b]] = blocks[:b].sum() + np.arange(blocks[b])
    k, v = (torch.randint(0, 0x70, (int(blocks.sum()), page, 1, d), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    scales = tuple(torch.full((k.shape[0], 1, 1), 2.0 ** -6, device="cuda") for _ in range(2))
    q = torch.randn(B * new, G, d, generator=g, device="cuda", dtype=torch.bfloat16)
    kw = dict(causal=True, cu_q=i32(new * np.arange(B + 1)), seqused_k=i32(used), block_table=i32(table), s_kv=int(used.max()),
              max_seqlen_q=new, cache_scale=scales)
    want, lse, ws = fa.forward(q, k, v, **kw)
    assert fa.device_status(ws) == 0 and torch.isfinite(lse).all()
    flush, ended = torch.empty(64 << 20, device="cuda"), 0  # 256 MB, twice the L2
    for _ in range(6):
        flush.fill_(1.0)
        q.mul_(1.0)
        o, z, ws = fa.forward(q, k, v, **kw, wait_limit_ns=1)
        status = fa.device_status(ws)
        assert status in (0, fa.FA_ERR_TIMEOUT)
        ended += status != 0
        if status != 0:
            o, z, ws = fa.forward(q, k, v, **kw)
            assert fa.device_status(ws) == 0
        assert torch.equal(o, want) and torch.equal(z, lse)
    assert ended or not (long and (d, new) in ((128, 1), (256, 2), (256, 4)))


@pytest.mark.parametrize("d,h_q,h_kv", at.HEADS)
@pytest.mark.parametrize("new", [1, 5, 200])
def test_fp16_outputs_stay_finite(d, h_q, h_kv, new):
    """Values of 65504, fp16's largest, are appended as 65536 (e4m3 has no nearer one): the output of every kernel, of items
    that are cut as well, is 65504 again.  (All values of a head's column are alike, so its exact output is 65536.)"""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    T = 3000
    sign = torch.where(torch.arange(d, device="cuda") % 3 == 0, -1.0, 1.0).half()
    x = torch.randn(T, h_q, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).half()
    k, v = torch.randn(T, h_kv, d, device="cuda").half(), (65504.0 * sign).expand(T, h_kv, d).contiguous()
    i32 = lambda *y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    pools = [torch.zeros(-(-T // 64), 64, h_kv, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(-(-T // 64), 2, h_kv, device="cuda") for _ in range(2)]
    table = torch.arange(-(-T // 64), dtype=torch.int32, device="cuda")[None].contiguous()
    fa.qk_norm_rope_append8(x, k, v, None, None, None, None, k_cache=pools[0], v_cache=pools[1], k_scale=scales[0], v_scale=scales[1],
                            cu_q=i32(0, T), seqused_k=i32(T), block_table=table, positions=torch.zeros(T, dtype=torch.int32, device="cuda"), norm=False)
    assert (scales[1] == 256).all()
    for used in (T, 40 + new):
        o, _, ws = fa.forward(x[:new], pools[0], pools[1], causal=True, cu_q=i32(0, new), seqused_k=i32(used), block_table=table, s_kv=T,
                              cache_scale=tuple(scales), max_seqlen_q=new)
        assert fa.device_status(ws) == 0 and torch.equal(o, (65504.0 * sign).expand_as(o))


def f16_queries(c, factor):
    """The case with queries times a power of two."""
    from exact_attention_bwd_gb300 import inputs
    c["qb"] = inputs.f16_bits((c["q"] * factor).astype(np.float32))
    c["q"] = inputs.f16_to_f64(c["qb"])
    return c


@pytest.mark.parametrize("d,h_q,h_kv", at.HEADS)
@pytest.mark.parametrize("new", [1, 4, 200])
@pytest.mark.parametrize("power", [12, 3, -20, -26])
def test_keys_outside_the_range_of_fp16(d, h_q, h_kv, new, power):
    """fp16 queries: keys beyond 65504 (up to 448 x 2^14), and keys below fp16's smallest step, count as what they are in
    every kernel.  (Queries are as much smaller or larger.)"""
    c = f16_queries(at.case([new, new], [900, 250], h_q=h_q, h_kv=h_kv, d=d, page=64, block=16, kind="f16"), 2.0 ** -min(power + 4, 14) if power > 0 else 2.0 ** 10)
    c["k"][1][...] = 2.0 ** power * 2.0 ** np.random.default_rng(d).integers(-2, 3, c["k"][1].shape)
    at.compare(c, hint=new)
    at.compare(c, hint=new, window=(70, -1))


def compare_f16(c, *, causal=True, window=(-1, -1), hint=0):
    """The bound of test_gpu_paged8.py for fp16, element by element, but that a probability that is rounded below fp16's normal
    range is off by 2^-25 at most, where the row's largest is 1 and more before their sum divides them (a chunk's kernel moves its
    reference when a score passes it, and does not bring values into the probabilities, as the few-row kernel does):
    2^-25 sum_j |v_j| in all.  What lies outside fp16's range is limited to it on both sides."""
    o, z, status = at.gpu(c, causal=causal, window=window, hint=hint)
    assert status == 0
    k, v = c8.true_values(*c["k"]), c8.true_values(*c["v"])
    scale, args = c["d"] ** -0.5, (c["cu"], c["used"], c["table"])
    want, lse, spread = ref.attention(c["q"], k, v, *args, causal=causal, window=window, scale=scale,
                                      sinks=None if c["sinks"] is None else c["sinks"].astype(np.float64))
    most = np.abs(ref.gather(k, c["table"], c["used"])).sum(-1).max() * np.abs(c["q"]).max()
    score = min(most * scale * c["d"] * 2.0 ** -24, 2.0 ** -9) + 2.0 ** -18
    sizes = np.zeros_like(want)
    for b in range(len(c["used"])):
        x = np.abs(ref.gather(v, c["table"][b:b + 1], c["used"][b:b + 1])).sum(0)
        sizes[c["cu"][b]:c["cu"][b + 1]] = np.repeat(x, c["h_q"] // c["h_kv"], 0)
    want = np.clip(want, -65504, 65504)
    err = np.abs(from_dev(o) - want)
    bound = 2.0 ** -11 * np.abs(want) + (2.0 ** -11 + 2 * score) * spread + 2.0 ** -25 * sizes + 2.0 ** -24
    assert np.all(err <= bound), (float(err.max()), float((err - bound).max()), np.argwhere(~(err <= bound))[:4])
    assert np.abs(z.cpu().numpy() - lse).max() <= score + 2.0 ** -22 * np.abs(lse).max()


@pytest.mark.parametrize("d,h_q,h_kv", at.HEADS)
@pytest.mark.parametrize("new", [1, 4, 200])
@pytest.mark.parametrize("power", [9, -16, -30])
def test_values_outside_the_range_of_fp16(d, h_q, h_kv, new, power):
    """fp16 outputs from values beyond 65504 (up to 448 x 2^11, of both signs, whose means may pass it as well), and from values
    of fp16's smallest steps and less."""
    c = at.case([new, new], [900, 250], h_q=h_q, h_kv=h_kv, d=d, page=64, block=16, kind="f16")
    c["v"][1][...] = 2.0 ** power * 2.0 ** np.random.default_rng(d).integers(-2, 3, c["v"][1].shape)
    compare_f16(c, hint=new)
    compare_f16(dict(c, sinks=np.linspace(-1, 2, h_q).astype(np.float32)), hint=0, causal=False)


@pytest.mark.parametrize("d,h_q,h_kv", at.HEADS)
def test_blocks_of_unlike_size_in_one_item(d, h_q, h_kv):
    """fp16: scales of keys and of values over 2^-16 .. 2^3 within an item's reach, some 0, entries of pages behind a window anything."""
    c = at.case([300, 1, 150], [1900, 77, 400], h_q=h_q, h_kv=h_kv, d=d, page=32, block=16, kind="f16")
    rng = np.random.default_rng(d)
    for pool in (c["k"], c["v"]):
        pool[1][...] = 2.0 ** rng.integers(-16, 4, pool[1].shape) * (rng.random(pool[1].shape) < 0.9)
    f16_queries(c, 2.0 ** -8)
    compare_f16(c)
    table = c["table"].copy()
    table[0, :(1900 - 300 - 500) // 32] = -1
    compare_f16(c, window=(500, -1))
    want = at.gpu(c, window=(500, -1))
    got = at.gpu(dict(c, table=table), window=(500, -1))
    assert got[2] == 0 and np.array_equal(from_dev(got[0]), from_dev(want[0]))


@pytest.mark.parametrize("reset", [False, True])
def test_a_block_whose_first_tokens_were_skipped(reset):
    """A call leaves alone a block of which it stores nothing; the next tokens take the scale that is there for old, or
    none where the caller has set it to 0."""
    c = ap.append_case([0], [5], 4, 2, 64, 64, 16, 16, seed=7)
    page = c["table"][0, 0]
    for _, scale in c["cache"]:
        scale[page] = 2.0 ** 20  # of an earlier owner of the page
    c["pos"][:] = -1
    _, after = ap.run(c)
    for (a, b), (x, y) in zip(c["cache"], after):
        assert np.array_equal(a, x) and np.array_equal(b, y)
    c = dict(ap.append_case([5], [6], 4, 2, 64, 64, 16, 16, seed=8), table=c["table"], cache=after)
    if reset:
        for _, scale in c["cache"]:
            scale[page] = 0
    q, after = ap.run(c)
    ap.verify(c, q, after)
    assert all(((y[page] < 1) == reset).all() for _, y in after)
