"""Refusals of the serving-step and training-step operators on a host without a GPU, at the edges of what
their documentation allows (every call here is refused before anything is launched)."""
import ctypes

import pytest

from exact_attention_bwd_gb300 import binding as fa
from test_step_host import A, B, C, D, E, F, G, H, rope

BAD = fa.FA_ERR_INVALID_ARG
W = ctypes.c_void_p(0x77000)


def at(p, n):
    return ctypes.c_void_p(p.value + n)


def gradient(p, q=A, k=B, dq_out=C, dk_out=D, dq=E, dk=F, dwq=G, dwk=W, ws=H):
    return fa.fa_qk_norm_rope_bwd(p, q, k, dq_out, dk_out, dq, dk, dwq, dwk, ws, 1 << 30, None)


# 10 tokens, 4 + 2 heads of 128: rows of 1024 and 512 bytes, contiguous unless said otherwise
@pytest.mark.parametrize("p,kw", [
    (rope(h_kv=4, k_stride=512, dk_stride=512), dict(dq=B)),       # dq over k, of the same shape
    (rope(h_kv=4, k_stride=512, dk_stride=512), dict(dk=A)),       # dk over q
    (rope(), dict(dq=B)), (rope(), dict(dk=A)),
    (rope(), dict(dq=at(A, 1024))),                                # dq a token behind q
    (rope(), dict(dq=at(A, -16))), (rope(), dict(dq=at(A, 10 * 1024 - 16))),
    (rope(), dict(dq=at(C, 16))), (rope(), dict(dk=at(D, 5 * 512))), (rope(), dict(dk=at(B, -512))),
    (rope(), dict(dk=at(E, 1024))),                                # dk inside dq
    (rope(q_stride=1024), dict(dq=A)),                             # in place at another stride
    # fused rows of 2048 bytes: q at 0, k at 1024; dq a row later and 16 bytes into k
    (rope(q_stride=1024, k_stride=1024, dq_stride=1024), dict(k=at(A, 1024), dq=at(A, 2048 + 528))),
    (rope(q_stride=1024, k_stride=1024, dk_stride=1024), dict(k=at(A, 1024), dk=at(A, 5 * 2048 + 1008))),
    # the weights' gradients and the workspace over anything else
    (rope(), dict(dwq=W)), (rope(), dict(dwq=at(W, 256))), (rope(), dict(dwq=A)), (rope(), dict(dwk=at(B, 4096))),
    (rope(), dict(dwq=C)), (rope(), dict(dwk=D)), (rope(), dict(dwq=at(E, 9 * 1024))), (rope(), dict(dwk=F)), (rope(), dict(dwq=H)),
    (rope(), dict(dwk=at(H, 16))), (rope(), dict(ws=A)), (rope(), dict(ws=E)), (rope(), dict(ws=F)), (rope(), dict(ws=D)),
    (rope(), dict(dwq=ctypes.c_void_p(0x1000))), (rope(), dict(ws=ctypes.c_void_p(0x2000))),     # cos, sin
    (rope(), dict(dq=ctypes.c_void_p(0x1000))), (rope(), dict(dk=ctypes.c_void_p(0x3000))), (rope(positions=E.value + 1024), {}),
    (rope(q_weight=W.value), {}), (rope(positions=G.value), {}), (rope(k_weight=H.value), {}),
])
def test_gradient_refuses_overlaps(p, kw):
    assert gradient(p, **kw) == BAD
