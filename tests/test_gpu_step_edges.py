"""Serving-step and training-step operators at the edges of what their documentation allows: copies that
land out of order, roots of nothing, the largest windows and pages, one slot twice, waits that run out.

Bounds are those of test_gpu_paged and test_gpu_norm_rope, where they are derived.
"""
import numpy as np
import pytest

import step_helpers as ref
from gpu_helpers import from_dev
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
