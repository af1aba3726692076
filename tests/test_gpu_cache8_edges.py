"""Calls of the operators over an 8-bit cache at the edges of what the header allows, on the GPU against the 64-bit
definition.  Bounds are those of test_gpu_append8.py and test_gpu_paged8.py."""
import numpy as np
import pytest

import test_gpu_append8 as ap

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
