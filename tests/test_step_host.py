"""The operators around the attention on a host without a GPU: their arguments' checks (every call
here is refused, or empty, before anything is launched), the parameter structures' layout, and
the plain forms that the GPU tests compare with."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import step_helpers as ref
from exact_attention_bwd_gb300 import binding as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E, F, G, H = (ctypes.c_void_p(x << 32) for x in range(1, 9))  # 16-byte aligned, never dereferenced
MISAL = ctypes.c_void_p((9 << 32) + 8)


def test_structures_match_the_header(tmp_path):
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "fa.h"', "int main(void) {"]
    for name, st in (("fa_rope_params", fa.FaRopeParams), ("fa_page_plan_params", fa.FaPagePlanParams)):
        src.append(f'printf("%zu\\n", sizeof({name}));')
        src += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in st._fields_]
    src.append("return 0; }")
    (tmp_path / "a.c").write_text("\n".join(src))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for st in (fa.FaRopeParams, fa.FaPagePlanParams):
        want.append(ctypes.sizeof(st))
        want += [getattr(st, f).offset for f, _ in st._fields_]
    assert got == want


# ------------------------------------------------------------------------------------------
# packed queries over a paged cache
# ------------------------------------------------------------------------------------------

def paged(**kw):
    p = fa.FaParams()
    base = dict(B=3, s_q=40, s_kv=500, h_q=8, h_kv=2, d=128, window_left=-1, window_right=-1, cu_seqlens_q=0x2000, seqused_k=0x3000,
                block_table=0x4000, page_size=16, max_blocks_per_seq=32, num_pages=90)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(seqused_k=None), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=24), fa.FA_ERR_INVALID_ARG), (dict(page_size=8), fa.FA_ERR_INVALID_ARG), (dict(page_size=0), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=-16), fa.FA_ERR_INVALID_ARG), (dict(num_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=31), fa.FA_ERR_INVALID_ARG),        # 31 x 16 < 500
    (dict(cu_seqlens_k=0x5000), fa.FA_ERR_UNSUPPORTED), (dict(dtype=fa.FA_DTYPE_E4M3), fa.FA_ERR_UNSUPPORTED),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(h_q=7), fa.FA_ERR_INVALID_ARG), (dict(h_q=512), fa.FA_ERR_UNSUPPORTED),
    (dict(window_left=-2), fa.FA_ERR_INVALID_ARG), (dict(s_q=2 ** 29, h_q=32), fa.FA_ERR_UNSUPPORTED),
])
def test_paged_forward_refuses(kw, code):
    p = paged(**kw)
    assert fa.fa_fwd(p, A, B, C, D, None, E, 1 << 40, None) == code
    assert fa.fa_fwd_workspace_size(p) == 0


def test_paged_forward_pointers_and_workspace():
    p = paged()
    n = fa.fa_fwd_workspace_size(p)
    assert n > 256
    # the workspace goes by the rows of a tile and the device, not by the lengths
    assert fa.fa_fwd_workspace_size(paged(s_kv=100000, max_blocks_per_seq=6250)) == n
    assert fa.fa_fwd_workspace_size(paged(max_seqlen_q=1)) < n
    assert fa.fa_fwd(p, A, B, C, D, None, E, n - 1, None) == fa.FA_ERR_WORKSPACE
    for bad in ((None, B, C, D, E), (A, None, C, D, E), (A, B, None, D, E), (A, B, C, None, E), (A, B, C, D, None), (MISAL, B, C, D, E),
                (A, MISAL, C, D, E), (A, B, MISAL, D, E), (A, B, C, MISAL, E), (A, B, C, D, MISAL)):
        assert fa.fa_fwd(p, *bad[:4], None, bad[4], n, None) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_bwd(p, *([A] * 9), None, E, 1 << 40, None) == fa.FA_ERR_UNSUPPORTED
    assert fa.fa_bwd_workspace_size(p) == 0
    assert fa.fa_fwd_workspace_size(paged(B=0)) == 256 and fa.fa_fwd_workspace_size(paged(s_q=0)) == 256


# ------------------------------------------------------------------------------------------
# norm + rotation
# ------------------------------------------------------------------------------------------

def rope(**kw):
    p = fa.FaRopeParams()
    base = dict(T=10, h_q=4, h_kv=2, d=128, rot_dim=128, seq_len=10, max_pos=64, eps=1e-6, dtype=fa.FA_DTYPE_BF16, q_stride=512,
                k_stride=256, v_stride=256, dq_stride=512, dk_stride=256, cos=0x1000, sin=0x2000)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), fa.FA_ERR_INVALID_ARG), (dict(h_q=0), fa.FA_ERR_INVALID_ARG), (dict(h_kv=-1), fa.FA_ERR_INVALID_ARG),
    (dict(rot_dim=256), fa.FA_ERR_INVALID_ARG), (dict(rot_dim=-16), fa.FA_ERR_INVALID_ARG), (dict(rot_dim=24), fa.FA_ERR_UNSUPPORTED),
    (dict(d=96, rot_dim=96, q_stride=384, k_stride=192), fa.FA_ERR_UNSUPPORTED), (dict(dtype=fa.FA_DTYPE_E4M3), fa.FA_ERR_UNSUPPORTED),
    (dict(dtype=9), fa.FA_ERR_INVALID_ARG), (dict(eps=-1.0), fa.FA_ERR_INVALID_ARG), (dict(eps=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(q_stride=511), fa.FA_ERR_INVALID_ARG), (dict(q_stride=516), fa.FA_ERR_INVALID_ARG), (dict(k_stride=248), fa.FA_ERR_INVALID_ARG),
    (dict(cos=None), fa.FA_ERR_INVALID_ARG), (dict(sin=None), fa.FA_ERR_INVALID_ARG), (dict(cos=0x1004), fa.FA_ERR_INVALID_ARG),
    (dict(max_pos=0), fa.FA_ERR_INVALID_ARG), (dict(max_pos=9), fa.FA_ERR_INVALID_ARG),  # 10 positions, 9 rows
    (dict(seq_len=0), fa.FA_ERR_INVALID_ARG), (dict(q_weight=0x1008), fa.FA_ERR_INVALID_ARG), (dict(k_weight=0x1001), fa.FA_ERR_INVALID_ARG),
])
def test_norm_rope_refuses(kw, code):
    p = rope(**kw)
    assert fa.fa_qk_norm_rope(p, A, B, None, C, D, None, None, None) == code
    assert fa.fa_qk_norm_rope_bwd_workspace_size(p) == 0
    assert fa.fa_qk_norm_rope_bwd(p, A, B, C, D, E, F, G, H, A, 1 << 30, None) == code


def test_norm_rope_pointers():
    fwd = lambda p, *a: fa.fa_qk_norm_rope(p, *a, None)  # noqa: E731
    bad = fa.FA_ERR_INVALID_ARG
    p = rope()
    for args in ((None, B, None, C, D, None, None), (A, None, None, C, D, None, None), (A, B, None, None, D, None, None),
                 (A, B, None, C, None, None, None), (MISAL, B, None, C, D, None, None), (A, B, None, C, MISAL, None, None),
                 (A, B, E, C, D, None, None),                       # a value without a cache
                 (A, B, None, B, D, None, None), (A, B, None, C, A, None, None), (A, B, None, C, C, None, None)):  # overlaps
        assert fwd(p, *args) == bad
    # q_out over q is in place only in the same layout
    assert fwd(rope(q_stride=1024), A, B, None, A, D, None, None) == bad
    p = rope(slots=0x3000, num_slots=64)
    for args in ((A, B, E, C, None, F, None), (A, B, E, C, None, None, G), (A, B, None, C, None, F, G), (A, B, E, C, None, F, F),
                 (A, B, E, C, None, A, G), (A, B, E, C, None, F, E), (A, B, E, C, F, F, G), (A, B, E, C, None, MISAL, G)):
        assert fwd(p, *args) == bad
    assert fwd(rope(num_slots=64), A, B, E, C, None, F, G) == bad   # no slots
    assert fwd(rope(slots=0x3000), A, B, E, C, None, F, G) == bad   # no rows in the pool
    assert fwd(rope(slots=0x3000, num_slots=64, v_stride=100), A, B, E, C, None, F, G) == bad
    assert fwd(rope(T=0), None, None, None, None, None, None, None) == fa.FA_OK


def test_norm_rope_gradient_pointers():
    n = fa.fa_qk_norm_rope_bwd_workspace_size(rope())
    assert n >= 2 * 128 * 4
    bwd = lambda p, *a, ws=H, size=n: fa.fa_qk_norm_rope_bwd(p, *a, ws, size, None)  # noqa: E731
    bad = fa.FA_ERR_INVALID_ARG
    full = [A, B, C, D, E, F, G, ctypes.c_void_p(0x77000)]
    for i in range(8):
        assert bwd(rope(), *(full[:i] + [None] + full[i + 1:])) == bad
    for i in range(6):
        assert bwd(rope(), *(full[:i] + [MISAL] + full[i + 1:])) == bad
    assert bwd(rope(), *full, ws=None) == bad and bwd(rope(), *full, ws=MISAL) == bad
    assert bwd(rope(), *full, size=n - 1) == fa.FA_ERR_WORKSPACE
    assert bwd(rope(dq_stride=504), *full) == bad and bwd(rope(dk_stride=260), *full) == bad
    for dq, dk in ((E, E), (D, F), (E, C), (A, F)):  # one for both; over the other gradient; over q at another stride
        assert bwd(rope(q_stride=1024), A, B, C, D, dq, dk, G, full[7]) == bad


# ------------------------------------------------------------------------------------------
# page plan
# ------------------------------------------------------------------------------------------

def plan(p, cached=A, fresh=B, free=C, head=D, table=E, cu=F, used=G, pos=H, slots=ctypes.c_void_p(9 << 32), out=ctypes.c_void_p(10 << 32)):
    return fa.fa_page_plan(p, cached, fresh, free, head, table, cu, used, pos, slots, out, None, None)


@pytest.mark.parametrize("args,code", [
    ((-1, 8, 16, 4, 9, 3), fa.FA_ERR_INVALID_ARG), ((2, -8, 16, 4, 9, 3), fa.FA_ERR_INVALID_ARG), ((2, 8, 0, 4, 9, 3), fa.FA_ERR_INVALID_ARG),
    ((2, 8, 16, 0, 9, 3), fa.FA_ERR_INVALID_ARG), ((2, 8, 16, 4, 0, 3), fa.FA_ERR_INVALID_ARG), ((2, 8, 16, 4, 9, -3), fa.FA_ERR_INVALID_ARG),
    ((2, 8, 1 << 16, 1 << 16, 9, 3), fa.FA_ERR_UNSUPPORTED), ((2, 8, 1 << 16, 4, 1 << 16, 3), fa.FA_ERR_UNSUPPORTED),
])
def test_page_plan_refuses_sizes(args, code):
    assert plan(fa.FaPagePlanParams(*args)) == code


def test_page_plan_pointers():
    p = fa.FaPagePlanParams(2, 8, 16, 4, 9, 3)
    bad = fa.FA_ERR_INVALID_ARG
    for name in ("cached", "fresh", "free", "table", "cu", "used", "pos", "slots", "out"):
        assert plan(p, **{name: None}) == bad
    # an output over an input or another output: lengths are read by every CTA while others write
    for name, other in (("used", A), ("used", B), ("out", D), ("cu", C), ("table", A), ("pos", ctypes.c_void_p((9 << 32) + 28)), ("used", F)):
        assert plan(p, **{name: other}) == bad


def test_plain_page_plan_by_hand():
    """Two requests on pages of 4: 3 cached + 2 new reach into a second page, 0 + 5 take two."""
    table = np.array([[7, -1, -1], [-1, -1, -1]], np.int32)
    cu, used, positions, slots, head, table, bad = ref.page_plan([3, 0], [2, 5], table, [9, 5, 2, 8], 1, 4, 10, 9)
    assert cu.tolist() == [0, 2, 7] and used.tolist() == [5, 5] and head == 4 and not bad
    assert table.tolist() == [[7, 5, -1], [2, 8, -1]]
    assert positions.tolist() == [3, 4, 0, 1, 2, 3, 4, -1, -1]
    assert slots.tolist() == [7 * 4 + 3, 5 * 4, 8, 9, 10, 11, 32, -1, -1]


@pytest.mark.parametrize("adjacent", [False, True])
def test_plain_gradient_against_differences(adjacent):
    """The gradient's formula against central differences of the forward's, in 64 bits: the
    truncation h^2 / 6 times a third derivative of order 1 and the rounding 2^-53 |L| / h are both
    below 1e-8 at h = 1e-5."""
    rng = np.random.default_rng(3)
    T, heads, d, rot, eps, h = 3, 2, 16, 8, 1e-3, 1e-5
    x, w, dy = rng.standard_normal((T, heads, d)), 1 + 0.3 * rng.standard_normal(d), rng.standard_normal((T, heads, d))
    a = rng.standard_normal((T, rot // 2))
    cos, sin = np.cos(a), np.sin(a)
    loss = lambda x, w: float((ref.norm_rope(x, w, cos, sin, eps, adjacent) * dy).sum())  # noqa: E731
    dx, dw, _ = ref.norm_rope_bwd(x, w, cos, sin, eps, adjacent, dy)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        assert abs((loss(up, w) - loss(down, w)) / (2 * h) - dx[i]) < 1e-8
    for i in range(d):
        up, down = w.copy(), w.copy()
        up[i] += h
        down[i] -= h
        assert abs((loss(x, up) - loss(x, down)) / (2 * h) - dw[i]) < 1e-8


def test_binding_refuses_before_it_calls():
    """Host tensors and wrong shapes are refused by the binding in words."""
    import torch
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope(q, k, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope_backward(q, k, q, k, None, None, None, None)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.page_plan(i, i, i.view(1, 2), i, page_size=16, num_pages=2, tokens=2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.forward(q, k, k, cu_q=i, seqused_k=i, block_table=i.view(1, 2), s_kv=16)
    with pytest.raises(TypeError):
        fa.page_plan([1], i, i, i, page_size=16, num_pages=2, tokens=2)
