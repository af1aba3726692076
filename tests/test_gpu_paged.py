"""Packed queries over a paged cache, on the GPU against the 64-bit oracle.

Bound of O, element by element: the output is rounded once (half a step h: 2^-8 of the value
in bf16, 2^-11 in fp16), each probability is rounded once before the second product (h
sum_j p_j |v_j| in all) and the fp32 part (scores, exponentials, sums) stays below 2^-13
sum_j p_j |v_j|: a score is a sum of d products with an error of at most d 2^-24 of the sum
of their sizes, about 2^-13 at d = 256 and unit normal inputs times the scale.  The LSE has the
scores' error: 3e-4.
"""
import numpy as np
import pytest

import step_helpers as ref
from exact_attention_bwd_gb300 import inputs
from gpu_helpers import Guarded, check_lse, from_dev

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def draw(rng, shape, kind):
    x = rng.standard_normal(shape).astype(np.float32)
    bits = inputs.bf16_bits(x) if kind == "bf16" else inputs.f16_bits(x)
    return bits, (inputs.bf16_to_f64 if kind == "bf16" else inputs.f16_to_f64)(bits)


def up(bits, kind):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()
    return t.view(torch.bfloat16 if kind == "bf16" else torch.float16)


def case(new, used, *, h_q, h_kv, d, page, kind="bf16", seed=0, spare=3, extra_rows=0, sinks=False):
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
    c = dict(new=new, used=np.asarray(used, np.int32), cu=cu, table=table.astype(np.int32), kind=kind, page=page, pool=pool,
             T=int(cu[-1]) + extra_rows, s_kv=max(list(used) + [1]), d=d, h_q=h_q, h_kv=h_kv)
    c["qb"], c["q"] = draw(rng, (c["T"], h_q, d), kind)
    c["kb"], c["k"] = draw(rng, (pool, page, h_kv, d), kind)
    c["vb"], c["v"] = draw(rng, (pool, page, h_kv, d), kind)
    c["sinks"] = rng.standard_normal(h_q).astype(np.float32) if sinks else None
    return c


def gpu(c, *, causal=True, window=(-1, -1), hint=0, flags=0, kb=None, vb=None, scale=None):
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q = up(c["qb"], c["kind"])
    out, lse = Guarded(q.shape, q.dtype), Guarded((c["h_q"], c["T"]), torch.float32)
    kw = dict(causal=causal, window=window, softmax_scale=scale, sinks=None if c["sinks"] is None else i32(c["sinks"]), cu_q=i32(c["cu"]),
              seqused_k=i32(c["used"]), block_table=i32(c["table"]), s_kv=c["s_kv"], flags=flags, max_seqlen_q=hint)
    k, v = up(c["kb"] if kb is None else kb, c["kind"]), up(c["vb"] if vb is None else vb, c["kind"])
    p = fa.make_params(q, k, **{n: x for n, x in kw.items()}, dtype=fa._type_code(q.dtype))
    ws = Guarded((fa.fa_fwd_workspace_size(p),), torch.uint8)
    o, z, w = fa.forward(q, k, v, **kw, out=out.t, lse=lse.t, workspace=ws.t)
    torch.cuda.synchronize()
    status = fa.device_status(w)
    for name, g in (("O", out), ("LSE", lse), ("workspace", ws)):
        g.check(name)
    return o, z, status


def compare(c, *, causal=True, window=(-1, -1), hint=0, flags=0, scale=None, **kw):
    o, z, status = gpu(c, causal=causal, window=window, hint=hint, flags=flags, scale=scale, **kw)
    assert status == 0
    n = int(c["cu"][-1])
    # the oracle reads the same table through the pages that are needed
    want, lse, spread = ref.attention(c["q"][:n], c["k"], c["v"], c["cu"], c["used"], c["table"], causal=causal, window=window,
                                      scale=scale if scale else c["d"] ** -0.5,
                                      sinks=None if c["sinks"] is None else c["sinks"].astype(np.float64))
    got = from_dev(o)
    h = HALF[c["kind"]]
    bound = h * np.abs(want) + (h + 2.0 ** -13) * spread + 2.0 ** -24
    err = np.abs(got[:n] - want)
    assert np.all(err <= bound), (float(err.max()), float((err - bound).max()), np.argwhere(err > bound)[:4])
    check_lse("LSE", z.cpu().numpy()[:, :n], lse, tol=3e-4)
    # rows behind the last sequence keep their bytes
    import torch
    assert torch.all(o[n:].contiguous().view(torch.uint8) == 0xFF) and torch.all(z[:, n:].contiguous().view(torch.uint8) == 0xFF)
    return o, z


HEADS = [(64, 5, 1), (128, 8, 2), (192, 3, 3), (256, 16, 2)]


@pytest.mark.parametrize("d,h_q,h_kv", HEADS)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_decode(d, h_q, h_kv, kind):
    """One token a sequence: caches of one key, around a tile's and a page's end, long ones."""
    used = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 700, 3001]
    compare(case([1] * len(used), used, h_q=h_q, h_kv=h_kv, d=d, page=16, kind=kind), hint=1)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 96, 128, 144, 192, 256, 384])
def test_page_sizes(page):
    used = [page - 1, page, page + 1, 5 * page + 3, 1000]
    compare(case([1, 3, 1, 7, 2], used, h_q=8, h_kv=2, d=128, page=page), hint=7)


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
    """Windows and no mask; rows that see nothing (fewer keys than queries) give 0 and -inf."""
    c = case([1, 40, 200, 3, 20], [500, 40, 777, 130, 6], h_q=4, h_kv=2, d=d, page=48)
    o, z = compare(c, window=window, causal=causal)
    if causal:
        assert np.all(np.isneginf(z[:, c["cu"][4]].cpu().numpy())) and np.all(from_dev(o)[c["cu"][4]] == 0)


@pytest.mark.parametrize("hint", [1, 9, 40])
def test_sinks(hint):  # hint 40: the tensor-core kernel
    c = case([1, hint, 1], [900, 70, 0], h_q=8, h_kv=2, d=128, page=16, sinks=True)
    compare(c, hint=hint)


@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (16, 1), (24, 1), (64, 1), (128, 1), (7, 7)])
def test_head_groups(h_q, h_kv):
    compare(case([1, 2, 30], [200, 513, 64], h_q=h_q, h_kv=h_kv, d=64, page=64))


def test_few_units_and_many_pieces():
    """One sequence cut over many CTAs (the combine merges up to all of them), and fewer units than CTAs."""
    compare(case([1], [40000], h_q=4, h_kv=1, d=128, page=64), hint=1)
    compare(case([3], [9000], h_q=2, h_kv=1, d=256, page=128, sinks=True), hint=3)
    compare(case([1, 1], [60, 300], h_q=2, h_kv=2, d=64, page=16), hint=1)
    # long chunks of one sequence: items of the tensor-core kernels cut many times
    compare(case([100], [12000], h_q=4, h_kv=1, d=128, page=64, sinks=True))
    compare(case([100], [7000], h_q=4, h_kv=1, d=256, page=256, sinks=True))
    compare(case([130, 1], [5000, 900], h_q=3, h_kv=1, d=192, page=16, kind="f16"))


def test_many_sequences():
    rng = np.random.default_rng(5)
    used = rng.integers(0, 300, 1100)
    new = np.minimum(rng.integers(0, 3, 1100), used)
    compare(case(list(new), list(used), h_q=2, h_kv=1, d=64, page=16), hint=2)


def test_no_split_and_validation_flags_agree():
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case([1, 9, 1], [3000, 2000, 1], h_q=8, h_kv=2, d=128, page=16)
    compare(c, flags=fa.FA_FLAG_NO_SPLIT)
    o, z = compare(c, flags=fa.FA_FLAG_VALIDATE_CU)
    o2, z2 = compare(c)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(z, z2), "the same call, the same bits"


def test_a_small_hint_costs_no_correctness():
    compare(case([1, 60, 1], [300, 600, 70], h_q=8, h_kv=2, d=128, page=16), hint=1)


@pytest.mark.parametrize("d", [128, 256])
def test_what_lies_behind_the_used_keys_has_no_effect(d):
    """NaN and infinities in unused rows of a page, in unused pages and at keys before every row's
    window leave O and LSE as they are, bit for bit."""
    import torch
    c = case([1, 30, 2], [77, 333, 150], h_q=8, h_kv=2, d=d, page=32)
    for window in ((-1, -1), (40, -1)):
        o, z = compare(c, window=window)
        seen = np.zeros((c["pool"], c["page"]), bool)
        for b, n in enumerate(c["used"]):
            first = 0 if window[0] < 0 else max(0, n - c["new"][b] - window[0])
            j = np.arange(first, n)
            seen[c["table"][b, j // 32], j % 32] = True
        kb, vb = c["kb"].copy(), c["vb"].copy()
        kb[~seen], vb[~seen] = 0x7FC0, 0x7FC0  # NaN
        vb[~seen, :, ::2] = 0xFF80             # -inf
        o2, z2, status = gpu(c, window=window, kb=kb, vb=vb)
        assert status == 0
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(z, z2)


def test_large_scores_move_the_reference():
    """Scores that grow along the keys by far more than the lazy reference allows, tile after tile."""
    c = case([1, 4], [1000, 700], h_q=4, h_kv=2, d=128, page=16)
    grow = np.repeat(np.arange(1, c["pool"] + 1), 1)[:, None, None, None] * 0.25
    for b in range(2):  # pages in the order of the keys
        n = -(-int(c["used"][b]) // 16)
        c["table"][b, :n] = np.arange(n) + (63 if b else 0)
    kb = inputs.bf16_bits((inputs.bf16_to_f32(c["kb"]) * grow).astype(np.float32))
    c["kb"], c["k"] = kb, inputs.bf16_to_f64(kb)
    q, k = c["q"], c["k"]
    # the scores' fp32 error grows with them: d 2^-24 of the sum of the products' sizes
    size = float(np.abs(q).max() * np.abs(k).max())
    scale = 128 ** -0.5
    o, z, status = gpu(c, scale=scale)
    assert status == 0
    want, lse, spread = ref.attention(q, k, c["v"], c["cu"], c["used"], c["table"], causal=True, scale=scale)
    slack = 128 * 2.0 ** -24 * 128 * size * scale
    err = np.abs(from_dev(o) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * slack) * spread + 2.0 ** -24)
    assert np.all(np.abs(z.cpu().numpy() - lse) <= slack + 2.0 ** -22 * np.abs(lse))


def test_bad_entries_and_offsets_are_reported():
    """A needed page outside the pool reads as zeros and is reported; offsets and lengths that break
    the rules are reported under the validation flag and stay in bounds without it."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case([1, 2, 1], [100, 200, 300], h_q=4, h_kv=2, d=64, page=16)
    for entry in (-1, c["pool"], 2 ** 31 - 1):
        bad = dict(c, table=c["table"].copy())
        bad["table"][1, 3] = entry
        assert gpu(bad)[2] == fa.FA_ERR_DEVICE_CHECK
    for cu in ([0, 3, 2, 4], [1, 2, 3, 4], [0, 1, 3, 9]):
        bad = dict(c, cu=np.asarray(cu, np.int32))
        assert gpu(bad, flags=fa.FA_FLAG_VALIDATE_CU)[2] == fa.FA_ERR_DEVICE_CHECK
        gpu(bad)
    for used in ([100, -3, 300], [100, 301, 300]):
        bad = dict(c, used=np.asarray(used, np.int32))
        assert gpu(bad, flags=fa.FA_FLAG_VALIDATE_CU)[2] == fa.FA_ERR_DEVICE_CHECK
        assert gpu(bad)[2] in (0, fa.FA_ERR_DEVICE_CHECK)


def test_wait_limit_gives_up_cleanly():
    """The bounded waits: a limit of 1 ns ends the call with a timeout status, and the next call on
    the device is right."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    c = case([1], [60000], h_q=8, h_kv=1, d=128, page=64)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    args = [up(c[n], "bf16") for n in ("qb", "kb", "vb")]
    _, _, ws = fa.forward(*args, causal=True, cu_q=i32(c["cu"]), seqused_k=i32(c["used"]), block_table=i32(c["table"]),
                          s_kv=c["s_kv"], wait_limit_ns=1)
    assert fa.device_status(ws) == fa.FA_ERR_TIMEOUT
    compare(c, hint=1)


def test_graph_replay_with_new_lengths():
    """A captured call replayed after its lengths, table and queries changed in place: what it computes
    follows the device arrays, not the capture; two graphs share one workspace in turn."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    a = case([1, 1, 1], [40, 500, 77], h_q=8, h_kv=2, d=128, page=16, seed=1)
    b = case([1, 1, 1], [900, 3, 260], h_q=8, h_kv=2, d=128, page=16, seed=2)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    width, pool = max(a["table"].shape[1], b["table"].shape[1]), max(a["pool"], b["pool"])
    q = torch.zeros_like(up(a["qb"], "bf16"))
    k, v = (torch.zeros(pool, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
    cu, used = i32(a["cu"]), i32(a["used"])
    out, lse = torch.empty_like(q), torch.empty(8, 3, device="cuda")
    kw = dict(causal=True, cu_q=cu, seqused_k=used, block_table=table, s_kv=900, max_seqlen_q=1, out=out, lse=lse)

    def load(c):
        q.copy_(up(c["qb"], "bf16"))
        for t, n in ((k, "kb"), (v, "vb")):
            t[:c["pool"]].copy_(up(c[n], "bf16"))
        table[:, :c["table"].shape[1]].copy_(i32(c["table"]))
        used.copy_(i32(c["used"]))

    load(a)
    _, _, ws = fa.forward(q, k, v, **kw)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.forward(q, k, v, **kw, workspace=ws)
        graphs.append(g)
    for c, g in ((a, graphs[0]), (b, graphs[1]), (a, graphs[1]), (b, graphs[0])):
        load(c)
        out.fill_(float("nan"))
        g.replay()
        assert fa.device_status(ws) == 0
        want, _, spread = ref.attention(c["q"], c["k"], c["v"], c["cu"], c["used"], c["table"], causal=True, scale=128 ** -0.5)
        assert np.all(np.abs(from_dev(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -13) * spread + 2.0 ** -24)
