"""Pages that were freed behind a sliding window: table entries that no query needs may lie outside the pool, in either
cache and in every kernel of the packed queries over pages; those that some query needs set the status."""
import numpy as np
import pytest

import test_gpu_paged as p16
import test_gpu_paged8 as p8
from gpu_helpers import from_dev

pytestmark = pytest.mark.gpu

NEW, USED = [1, 150, 7, 300, 2, 40], [901, 1000, 530, 1777, 64, 700]


def freed(c, left, page):
    """The table without the entries whose keys are all more than `left` behind a sequence's first query, and the
    last of those that are needed at its front, for each sequence that has one behind it."""
    table, rng, front = c["table"].copy(), np.random.default_rng(0), {}
    for b, (n, m) in enumerate(zip(NEW, USED)):
        first = max(0, m - n - left) // page
        table[b, :first] = rng.choice([-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1], first)
        if first:
            front[b] = first
    return table, front


@pytest.mark.parametrize("cache", [p16, p8], ids=["16", "8"])
@pytest.mark.parametrize("d,h_q,h_kv", [(64, 5, 1), (64, 16, 8), (128, 8, 2), (192, 3, 3), (256, 16, 2)])
@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("left", [0, 100, 383])
def test_entries_that_no_query_needs(cache, d, h_q, h_kv, page, left):
    from exact_attention_bwd_gb300 import binding as fa
    c = cache.case(NEW, USED, h_q=h_q, h_kv=h_kv, d=d, page=page)
    for hint in (0, 300):
        want = cache.gpu(c, window=(left, -1), hint=hint)
        table, front = freed(c, left, page)
        got = cache.gpu(dict(c, table=table), window=(left, -1), hint=hint)
        assert want[2] == got[2] == 0
        assert np.array_equal(from_dev(got[0]), from_dev(want[0])) and np.array_equal(got[1].cpu().numpy(), want[1].cpu().numpy())
        for b, first in front.items():  # one that is needed
            bad = table.copy()
            bad[b, first] = -1
            assert cache.gpu(dict(c, table=bad), window=(left, -1), hint=hint)[2] == fa.FA_ERR_DEVICE_CHECK


@pytest.mark.parametrize("cache", [p16, p8], ids=["16", "8"])
@pytest.mark.parametrize("d,G", [(64, 4), (64, 16), (128, 2), (128, 8), (192, 4), (256, 2)])
def test_entries_that_no_decoded_token_needs(cache, d, G):
    """The few-row kernel alone, in tiles of 2 to 64 rows."""
    c = cache.case([2] * 6, USED, h_q=2 * G, h_kv=2, d=d, page=32)
    table = c["table"].copy()
    for b, m in enumerate(USED):
        table[b, :max(0, m - 2 - 150) // 32] = -1
    for hint in (2, 4):
        want, got = cache.gpu(c, window=(150, -1), hint=hint), cache.gpu(dict(c, table=table), window=(150, -1), hint=hint)
        assert want[2] == got[2] == 0
        assert np.array_equal(from_dev(got[0]), from_dev(want[0])) and np.array_equal(got[1].cpu().numpy(), want[1].cpu().numpy())
