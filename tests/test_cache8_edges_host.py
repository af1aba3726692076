"""Calls of the operators over an 8-bit cache and of the rotation with several axes at the edges of what the binding
and the header allow, on a host without a GPU."""
import array
import ctypes

import numpy as np
import pytest

from exact_attention_bwd_gb300 import binding as fa
from test_cache8_host import append, call, over_cache8
from test_step_host import A, B, C, D, E, paged, rope


@pytest.mark.parametrize("half", [8, 64, 128])
def test_axes_of_the_pairs_as_any_sequence(half):
    """Lists, tuples, bytes, arrays of any whole type and tensors hold the same entries; nothing is written behind the field."""
    import torch
    want = [j % 3 for j in range(half)]
    positions = torch.zeros(3, 5, dtype=torch.int32)
    for x in (want, tuple(want), bytes(want), bytearray(want), array.array("i", want), array.array("q", want), np.array(want, np.uint8),
              np.array(want, np.int32), np.array(want, np.int64), torch.tensor(want), torch.tensor(want, dtype=torch.uint8)):
        room = (ctypes.c_ubyte * (ctypes.sizeof(fa.FaRopeParams) + 1024))(*[0xAA] * (ctypes.sizeof(fa.FaRopeParams) + 1024))
        p = fa.FaRopeParams.from_buffer(room)
        p.rot_dim = 2 * half
        fa._set_axes(p, positions, x, True)
        assert p.axes == 3 and list(p.pair_axis)[:half] == want
        behind = fa.FaRopeParams.pair_axis.offset + half
        assert all(b == 0xAA for b in bytes(room)[behind:])


@pytest.mark.parametrize("bad", [
    [0.0] * 8, np.zeros(8), np.zeros((8, 1), np.int32), [0] * 7 + [3], [0] * 7 + [-1], [0] * 7 + [256], np.array([0] * 7 + [259], np.int32),
    ["0"] * 8, "00000000", [None] * 8,
])
def test_axes_that_are_refused(bad):
    import torch
    p = fa.FaRopeParams()
    p.rot_dim = 16
    with pytest.raises(ValueError, match="pair_axis must hold axes"):
        fa._set_axes(p, torch.zeros(3, 5, dtype=torch.int32), bad, True)


@pytest.mark.parametrize("form", [paged, over_cache8])
@pytest.mark.parametrize("s_kv,right,taken", [
    (2 ** 31 - 1, 0, False), (2 ** 31 - 256, 0, False), (2 ** 31 - 257, 0, True), (2 ** 31 - 257, -1, True),
    (2 ** 31 - 5000, 4000, True), (2 ** 31 - 5000, 5000, False), (2 ** 31 - 2 ** 22, 2 ** 31 - 1, False), (2 ** 30, 2 ** 31 - 1, True),
])
def test_keys_are_counted_in_32_bits(form, s_kv, right, taken):
    """The last key tile of a longest cache, and the last key of a right window, would pass 2^31 and be taken for negative."""
    p = form(s_kv=s_kv, page_size=1024, max_blocks_per_seq=1 << 21, window_right=right, causal=0)
    assert (fa.fa_fwd_workspace_size(p) > 0) == taken
    if not taken:
        assert fa.fa_fwd(p, A, B, C, D, None, E, 1 << 40, None) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("off", [1, 2, 3])
def test_scales_that_are_not_aligned_are_refused(off):
    """They are copied four bytes at a time."""
    for name in ("k_scale", "v_scale"):
        p = over_cache8(**{name: 0x6000 + off})
        assert fa.fa_fwd_workspace_size(p) == 0 and fa.fa_fwd(p, A, B, C, D, None, E, 1 << 40, None) == fa.FA_ERR_INVALID_ARG
    for name in ("ks", "vs"):
        assert call(rope(positions=0x3000), append(), **{name: ctypes.c_void_p((11 << 32) + off)}) == fa.FA_ERR_INVALID_ARG
