"""The operators over an 8-bit cache and the rotation with several axes on a host without a GPU: their
refusals (every call here is refused, or empty, before anything is launched), and the plain forms."""
import ctypes

import numpy as np
import pytest

import cache8_helpers as c8
import step_helpers as ref
from exact_attention_bwd_gb300 import binding as fa
from test_step_host import A, B, C, D, E, F, G, H, MISAL, rope

I = ctypes.c_void_p(10 << 32)


def test_structure_matches_the_header(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "fa.h"', "int main(void) {", 'printf("%zu\\n", sizeof(fa_cache8_params));']
    lines += [f'printf("%zu\\n", offsetof(fa_cache8_params, {f}));' for f, _ in fa.FaCache8Params._fields_] + ["return 0; }"]
    (tmp_path / "a.c").write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(fa.FaCache8Params)] + [getattr(fa.FaCache8Params, f).offset for f, _ in fa.FaCache8Params._fields_]


def pairs(*x):
    return (ctypes.c_ubyte * fa.FA_ROPE_MAX_PAIRS)(*x)


@pytest.mark.parametrize("kw", [
    dict(axes=-1), dict(axes=5, positions=0x3000), dict(axes=3),                                 # several axes without positions
    dict(axes=2, positions=0x3000, pair_axis=pairs(*[0] * 31, 2)), dict(axes=3, positions=0x3000, pair_axis=pairs(255)),
    dict(no_norm=1, q_weight=0x1000), dict(no_norm=1, k_weight=0x1000),
])
def test_rotation_refuses(kw):
    base = dict(q_weight=None, k_weight=None)
    p = rope(**{**base, **kw})
    assert fa.fa_qk_norm_rope(p, A, B, None, C, D, None, None, None) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_qk_norm_rope_bwd_workspace_size(p) == 0
    assert fa.fa_qk_norm_rope_bwd(p, A, B, C, D, E, F, G, H, A, 1 << 30, None) == fa.FA_ERR_INVALID_ARG


def test_gradient_without_the_norm():
    p = rope(no_norm=1, q_weight=None, k_weight=None)
    n = fa.fa_qk_norm_rope_bwd_workspace_size(p)
    bad = fa.FA_ERR_INVALID_ARG
    bwd = lambda *a: fa.fa_qk_norm_rope_bwd(p, *a, I, n, None)  # noqa: E731
    assert bwd(None, None, C, D, E, F, G, None) == bad and bwd(None, None, C, D, E, F, None, H) == bad  # no weights' gradients
    for i in range(4):
        x = [C, D, E, F]
        x[i] = None
        assert bwd(None, None, *x, None, None) == bad
    assert bwd(None, None, C, D, D, F, None, None) == bad  # dq over dk_out
    p.T = 0
    with_norm = rope(T=0)
    assert fa.fa_qk_norm_rope_bwd(with_norm, A, B, C, D, E, F, None, None, I, 1 << 30, None) == bad


def append(**kw):
    c = fa.FaCache8Params()
    base = dict(B=3, page_size=64, max_blocks_per_seq=10, num_pages=30, scale_block=32, cu_seqlens_q=1 << 20, seqused_k=2 << 20, block_table=3 << 20)
    base.update(kw)
    for k, v in base.items():
        setattr(c, k, v)
    return c


def call(p, c, q=A, k=B, v=C, q_out=D, kc=E, vc=F, ks=G, vs=H):
    return fa.fa_qk_norm_rope_append8(p, c, q, k, v, q_out, kc, vc, ks, vs, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), fa.FA_ERR_INVALID_ARG), (dict(page_size=0), fa.FA_ERR_INVALID_ARG), (dict(page_size=24, scale_block=8), fa.FA_ERR_INVALID_ARG),
    (dict(scale_block=0), fa.FA_ERR_INVALID_ARG), (dict(scale_block=24, page_size=48), fa.FA_ERR_INVALID_ARG),
    (dict(scale_block=48), fa.FA_ERR_INVALID_ARG), (dict(scale_block=128), fa.FA_ERR_INVALID_ARG), (dict(scale_block=-16), fa.FA_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=0), fa.FA_ERR_INVALID_ARG), (dict(num_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=1 << 26), fa.FA_ERR_UNSUPPORTED), (dict(B=1 << 30), fa.FA_ERR_UNSUPPORTED),
    (dict(cu_seqlens_q=None), fa.FA_ERR_INVALID_ARG), (dict(seqused_k=None), fa.FA_ERR_INVALID_ARG), (dict(block_table=None), fa.FA_ERR_INVALID_ARG),
])
def test_append_refuses(kw, code):
    assert call(rope(positions=0x3000), append(**kw)) == code


def test_append_pointers():
    bad, c, p = fa.FA_ERR_INVALID_ARG, append(), rope(positions=0x3000)
    for name in ("q", "k", "v", "q_out", "kc", "vc", "ks", "vs"):
        assert call(p, c, **{name: None}) == bad
    for name in ("q", "k", "v", "q_out", "kc", "vc"):
        assert call(p, c, **{name: MISAL}) == bad
    assert call(rope(), c) == bad                                          # no positions
    assert call(rope(positions=0x3000, slots=0x9000), c) == bad            # the table says where a token goes
    assert call(rope(positions=0x3000, v_stride=100), c) == bad
    assert call(rope(positions=0x3000, q_stride=1024), c, q_out=A) == bad  # in place only in the same layout
    for kw in (dict(q_out=B), dict(q_out=C), dict(kc=A), dict(vc=E), dict(ks=E), dict(vs=G), dict(kc=B), dict(vc=C), dict(q_out=F),
               dict(ks=ctypes.c_void_p(2 << 20)), dict(vs=ctypes.c_void_p(3 << 20)), dict(ks=ctypes.c_void_p(0x3000))):
        assert call(p, c, **kw) == bad
    assert call(rope(T=0, positions=0x3000), c, *[None] * 8) == fa.FA_OK


# ------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------

def test_e4m3_values_and_scales():
    import torch
    want = torch.arange(256).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c8.E4M3, want, equal_nan=True)
    for x in (1e-30, 0.3, 447.9, 448.0, 448.1, 896.0, 3e38, 2.0 ** -118 * 1.75):
        s = c8.need(x)
        assert x <= 448 * s and (s == 2.0 ** -126 or x > 448 * s / 2) and np.frexp(s)[0] == 0.5
    assert c8.need(0.0) == c8.need(2.0 ** -140) == 2.0 ** -126


def test_blocks_of_new_tokens():
    cu, used = np.array([0, 3, 3, 40]), np.array([18, 5, 50])
    table = np.arange(12).reshape(3, 4)
    got = c8.blocks_of(cu, used, table, 32, 16, 12)
    assert got == [(0, 0, 15, 16, 0), (0, 16, 0, 2, 1), (8, 0, 13, 16, 3), (8, 16, 0, 16, 6), (9, 0, 0, 16, 22), (9, 16, 0, 2, 38)]
    assert sum(hi - lo for _, _, lo, hi, _ in got) == 40


def test_rotation_gradient_by_differences():
    """The rotation's transpose is the turn back: <g, turn(x + h e) - turn(x - h e)> / 2h = turn back(g)."""
    rng = np.random.default_rng(0)
    x, g = rng.standard_normal((2, 1, 2, 16))
    a = rng.standard_normal((1, 8))
    turn = lambda y, back=False: ref.rotate(y, np.cos(a), np.sin(a), True, back=back)  # noqa: E731
    back = turn(g, True)
    for i in range(2):
        for j in range(16):
            e = np.zeros_like(x)
            e[0, i, j] = 1e-3
            assert abs(((turn(x + e) - turn(x - e)) * g).sum() / 2e-3 - back[0, i, j]) < 1e-10


# ------------------------------------------------------------------------------------------
# attention over the cache
# ------------------------------------------------------------------------------------------

def over_cache8(**kw):
    from test_step_host import paged
    return paged(**{**dict(cache_dtype=fa.FA_DTYPE_E4M3, page_size=64, max_blocks_per_seq=8, scale_block=32, k_scale=0x6000, v_scale=0x7000), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(cache_dtype=2), fa.FA_ERR_INVALID_ARG), (dict(cache_dtype=-1), fa.FA_ERR_INVALID_ARG),
    (dict(scale_block=0), fa.FA_ERR_INVALID_ARG), (dict(scale_block=8), fa.FA_ERR_INVALID_ARG), (dict(scale_block=48), fa.FA_ERR_INVALID_ARG),
    (dict(scale_block=128), fa.FA_ERR_INVALID_ARG), (dict(scale_block=-64), fa.FA_ERR_INVALID_ARG), (dict(page_size=0), fa.FA_ERR_INVALID_ARG),
    (dict(k_scale=None), fa.FA_ERR_INVALID_ARG), (dict(v_scale=None), fa.FA_ERR_INVALID_ARG),
    (dict(dtype=fa.FA_DTYPE_E4M3), fa.FA_ERR_UNSUPPORTED), (dict(cu_seqlens_k=0x5000), fa.FA_ERR_UNSUPPORTED),
    (dict(cu_seqlens_q=None), fa.FA_ERR_UNSUPPORTED), (dict(block_table=None, cu_seqlens_k=0x5000), fa.FA_ERR_UNSUPPORTED),
    (dict(cu_seqlens_q=None, block_table=None), fa.FA_ERR_UNSUPPORTED), (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(seqused_k=None), fa.FA_ERR_INVALID_ARG),
])
def test_forward_refuses(kw, code):
    p = over_cache8(**kw)
    assert fa.fa_fwd(p, A, B, C, D, None, E, 1 << 40, None) == code
    assert fa.fa_fwd_workspace_size(p) == 0


def test_forward_pointers_and_workspace():
    p = over_cache8()
    n = fa.fa_fwd_workspace_size(p)
    assert n > 256 and fa.fa_fwd_workspace_size(over_cache8(max_seqlen_q=1)) < n
    assert fa.fa_fwd(p, A, B, C, D, None, E, n - 1, None) == fa.FA_ERR_WORKSPACE
    for bad in ((None, B, C, D, E), (A, None, C, D, E), (A, B, None, D, E), (A, B, C, None, E), (A, B, C, D, None), (MISAL, B, C, D, E),
                (A, MISAL, C, D, E), (A, B, MISAL, D, E), (A, B, C, MISAL, E), (A, B, C, D, MISAL)):
        assert fa.fa_fwd(p, *bad[:4], None, bad[4], n, None) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_bwd(p, *([A] * 9), None, E, 1 << 40, None) == fa.FA_ERR_UNSUPPORTED
