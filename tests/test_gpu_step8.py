"""The operators of a serving step over an 8-bit cache run together: page plan, norm + rotation by three axes with
append, and attention over the cache, step after step, and replayed from two captured graphs that share a
workspace; a training step with the rotation's gradient; and the binding's refusals."""
import numpy as np
import pytest

import cache8_helpers as c8
import oracle
import step_helpers as ref
from exact_attention_bwd_gb300 import inputs
from gpu_helpers import from_dev
from test_gpu_step import STEPS

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, PAGE, BLOCK, BLOCKS, POOL, MAX_POS = 6, 2, 64, 32, 16, 12, 60, 400
HALF = 2.0 ** -8
AXES = [0] * 8 + [1] * 12 + [2] * 12


class Engine:
    """Static buffers of a small serving engine over an 8-bit cache."""

    def __init__(self, requests, rows, seed):
        import torch
        from exact_attention_bwd_gb300 import binding as fa
        self.fa, self.torch, self.rows, self.rng = fa, torch, rows, np.random.default_rng(seed)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.cached, self.fresh, self.head, self.status = i32(requests), i32(requests), i32(1), i32(1)
        self.table = i32(requests, BLOCKS)
        self.table.fill_(-1)
        self.free = torch.from_numpy(self.rng.permutation(POOL).astype(np.int32)).cuda()
        self.plan = [i32(requests + 1), i32(requests), i32(rows), i32(rows), i32(1)]
        self.shift = torch.tensor([[0], [3], [7]], dtype=torch.int32, device="cuda")
        # the pools hold NaN bytes and scales wherever nothing has been written
        self.pools = [torch.full((POOL, PAGE, H_KV, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.full((POOL, PAGE // BLOCK, H_KV), float("nan"), device="cuda") for _ in range(2)]
        self.qkv, self.q, self.out = b16(rows, H_Q + 2 * H_KV, D), b16(rows, H_Q, D), b16(rows, H_Q, D)
        self.lse = torch.zeros(H_Q, rows, device="cuda")
        cos, sin = ref.angles(MAX_POS, D)
        self.angles = cos, sin
        self.tables = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
        self.wq, self.wk = (torch.from_numpy(1 + 0.2 * self.rng.standard_normal(D)).cuda().to(torch.bfloat16) for _ in range(2))
        self.ws = None

    def call(self):
        q, k, v = self.qkv[:, :H_Q], self.qkv[:, H_Q:H_Q + H_KV], self.qkv[:, H_Q + H_KV:]
        cu, used, positions, _, _ = self.fa.page_plan(self.cached, self.fresh, self.table, self.free, page_size=PAGE, num_pages=POOL,
                                                      tokens=self.rows, free_head=self.head, out=self.plan, status=self.status)
        axes = self.torch.where(positions < 0, positions, positions + self.shift).contiguous()
        self.fa.qk_norm_rope_append8(q, k, v, self.wq, self.wk, *self.tables, k_cache=self.pools[0], v_cache=self.pools[1],
                                     k_scale=self.scales[0], v_scale=self.scales[1], cu_q=cu, seqused_k=used, block_table=self.table,
                                     positions=axes, pair_axis=AXES, out=self.q, status=self.status)
        _, _, ws = self.fa.forward(self.q, *self.pools, causal=True, cu_q=cu, seqused_k=used, block_table=self.table,
                                   s_kv=BLOCKS * PAGE, out=self.out, lse=self.lse, workspace=self.ws, cache_scale=self.scales)
        return ws

    def state(self):
        return [(p.cpu().numpy(), s.cpu().numpy()) for p, s in zip(self.pools, self.scales)]

    def step(self, fresh, run):
        """One step with these new tokens a request: fills the buffers, runs, checks."""
        torch, n = self.torch, int(sum(fresh))
        assert n <= self.rows
        bits = inputs.bf16_bits(self.rng.standard_normal((self.rows, H_Q + 2 * H_KV, D)).astype(np.float32))
        self.qkv.copy_(torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16))
        self.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        self.out.fill_(7.0)
        self.q.fill_(5.0)
        before = self.state()
        run()
        assert self.fa.device_status(self.ws) == 0 and self.status.item() == 0
        after = self.state()
        cu, used, table = (x.cpu().numpy() for x in (self.plan[0], self.plan[1], self.table))
        assert torch.all(self.q[n:] == 5) and torch.all(self.out[n:] == 7)
        if n:
            place = self.plan[2][:n].cpu().numpy()
            at = (place + np.array([[0], [3], [7]]))[AXES].T
            cos, sin = (x[at, np.arange(D // 2)] for x in self.angles)
            x = from_dev(self.qkv[:n])
            size = lambda y: np.abs(y) + 2 * np.abs(ref.rotate(np.abs(y), np.abs(cos), np.abs(sin), False)) + 2 * np.abs(ref.rotate(np.abs(y), np.abs(cos), np.abs(sin), False, back=True))  # noqa: E731
            rows = {}
            for name, y, w in (("q", x[:, :H_Q], self.wq), ("k", x[:, H_Q:H_Q + H_KV], self.wk)):
                rows[name] = ref.norm_rope(y, from_dev(w), cos, sin, 1e-6, False)
            qr = from_dev(self.q[:n])
            assert np.all(np.abs(qr - rows["q"]) <= HALF * np.abs(rows["q"]) + 2.0 ** -17 * size(rows["q"]))
            stored = np.ones(n, bool)
            c8.check_append("k", before[0], after[0], rows["k"], 2.0 ** -17 * size(rows["k"]), stored, cu, used, table)
            c8.check_append("v", before[1], after[1], x[:, H_Q + H_KV:], np.zeros(1), stored, cu, used, table)
            k, v = (c8.true_values(*y) for y in after)
            kw = dict(causal=True, scale=D ** -0.5)
            want, lse, spread = ref.attention(qr, k, v, cu, used, table, **kw)
            err = np.abs(from_dev(self.out[:n]) - want)
            assert np.all(err <= HALF * np.abs(want) + (HALF + 2.0 ** -13) * spread + 2.0 ** -24)
            assert np.abs(self.lse[:, :n].cpu().numpy() - lse).max() <= 3e-4
        # the engine's state moves on
        self.cached.copy_(self.plan[1])
        self.head.copy_(self.plan[4])


def test_serving_steps():
    e = Engine(5, 128, 1)
    for fresh in STEPS:
        def run():
            e.ws = e.call()
        e.step(fresh, run)


def test_serving_steps_from_two_graphs():
    """The whole step captured twice on one workspace and replayed in turn on a stream of its own."""
    import torch
    e = Engine(5, 128, 2)
    side = torch.cuda.Stream()
    e.ws = e.call()  # (no new tokens: sizes the workspace)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            e.call()
        graphs.append(g)
    for i, fresh in enumerate(STEPS):
        def run():
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graphs[i % 2].replay()
            torch.cuda.current_stream().wait_stream(side)
        e.step(fresh, run)


@pytest.mark.parametrize("norm", [False, True])
def test_training_step(norm):
    """Rotation by three axes, causal attention over it and both gradients, against the chain in 64 bits."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    rng = np.random.default_rng(4)
    S = 150
    bits = [inputs.bf16_bits(rng.standard_normal((S, h, D)).astype(np.float32)) for h in (H_Q, H_KV, H_KV, H_Q)]
    q, k, v, do = (torch.from_numpy(b.view(np.int16)).cuda().view(torch.bfloat16) for b in bits)
    pos = rng.integers(0, MAX_POS, (3, S)).astype(np.int32)
    cos, sin = ref.angles(MAX_POS, D)
    w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).cuda().bfloat16() if norm else None for _ in range(2)]
    tables = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    kw = dict(positions=torch.from_numpy(pos).cuda(), pair_axis=AXES, norm=norm)
    qr, kr = fa.qk_norm_rope(q, k, *w, *tables, **kw)
    batch = lambda x: x[None]  # noqa: E731
    o, lse, _ = fa.forward(batch(qr), batch(kr), batch(v), causal=True)
    dqr, dkr, dv, _, _ = fa.backward(batch(qr), batch(kr), batch(v), o, lse, batch(do), causal=True)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q, k, dqr[0], dkr[0], *w, *tables, **kw)
    c, s = (x[pos[AXES].T, np.arange(D // 2)] for x in (cos, sin))
    xq, xk, xv, xdo = (inputs.bf16_to_f64(b) for b in bits)
    ones = np.ones(D)
    wq, wk = (from_dev(x) if norm else ones for x in w)
    turn = lambda x, wt: ref.norm_rope(x, wt, c, s, 1e-6, False) if norm else ref.rotate(x, c, s, False)  # noqa: E731
    gq, gk, gv, _ = oracle.bwd(batch(turn(xq, wq)), batch(turn(xk, wk)), batch(xv), batch(xdo), scale=D ** -0.5, causal=True)
    for got, x, wt, g, dw in ((dq, xq, wq, gq[0], dwq), (dk, xk, wk, gk[0], dwk)):
        if norm:
            want, want_w, _ = ref.norm_rope_bwd(x, wt, c, s, 1e-6, False, g)
            assert np.linalg.norm(from_dev(dw) - want_w) <= 0.02 * np.linalg.norm(want_w)
        else:
            want = ref.rotate(g, c, s, False, back=True)
            assert dw is None
        # (q, k, P, dS and the gradient between the two are rounded to bf16, 2^-8 each: five of them, added in the worst case)
        assert np.linalg.norm(from_dev(got) - want) <= 5 * HALF * np.linalg.norm(want)
    assert np.linalg.norm(from_dev(dv[0]) - gv[0]) <= 5 * HALF * np.linalg.norm(gv[0])


def test_refusals_of_the_binding():
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    e = Engine(2, 8, 3)
    q, k, v = e.qkv[:, :H_Q], e.qkv[:, H_Q:H_Q + H_KV], e.qkv[:, H_Q + H_KV:]
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    used, pos = torch.ones(2, dtype=torch.int32, device="cuda"), torch.zeros(3, 8, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, BLOCKS, dtype=torch.int32, device="cuda")
    base = dict(k_cache=e.pools[0], v_cache=e.pools[1], k_scale=e.scales[0], v_scale=e.scales[1], cu_q=cu, seqused_k=used, block_table=table,
                positions=pos, pair_axis=AXES)

    def append(error, match, *args, **kw):
        with pytest.raises(error, match=match):
            fa.qk_norm_rope_append8(*(args or (q, k, v)), e.wq, e.wk, *e.tables, **{**base, **kw})

    append(ValueError, "positions", positions=None)
    append(ValueError, "pair_axis", positions=pos[0].contiguous())
    append(ValueError, "entries", pair_axis=AXES[:-1])
    append(ValueError, "pair_axis", pair_axis=AXES[:-1] + [3])
    append(ValueError, "pair_axis", pair_axis=AXES[:-1] + [-1])
    append(ValueError, "axes", positions=torch.zeros(5, 8, dtype=torch.int32, device="cuda"))
    append(ValueError, "elements", positions=pos[:, :7].contiguous())
    append(ValueError, "weights", norm=False)
    append(TypeError, "k_cache", k_cache=e.pools[0].view(torch.float8_e4m3fn))
    append(ValueError, "v_cache", v_cache=e.pools[1][:, :, :1].contiguous())
    append(ValueError, "blocks", k_scale=torch.zeros(POOL, 3, H_KV, device="cuda"), v_scale=torch.zeros(POOL, 3, H_KV, device="cuda"))
    append(ValueError, "v_scale", v_scale=torch.zeros(POOL, 1, H_KV, device="cuda"))
    append(TypeError, "k_scale", k_scale=e.scales[0].half())
    append(ValueError, "device", k_scale=e.scales[0].cpu())
    append(ValueError, "cu_q", cu_q=cu[:2].contiguous())
    append(ValueError, "block_table", block_table=table[0])
    append(ValueError, "shape", q, k, v[:, :1])
    append(TypeError, "type", q, k, v.half())
    append(ValueError, "out", out=torch.zeros(8, H_Q, D + 1, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(fa.FaError):  # a scale for 8 rows
        fa.qk_norm_rope_append8(q, k, v, e.wq, e.wk, *e.tables, **{**base, "k_scale": torch.zeros(POOL, 4, H_KV, device="cuda"),
                                                                "v_scale": torch.zeros(POOL, 4, H_KV, device="cuda")})

    kw = dict(causal=True, cu_q=cu, seqused_k=used, block_table=table, s_kv=64)

    def forward(error, match, *args, **more):
        with pytest.raises(error, match=match):
            fa.forward(*args, **{**kw, **more})

    scale = tuple(e.scales)
    forward(TypeError, "uint8|k must", e.q, e.pools[0].view(torch.int8), e.pools[1], cache_scale=scale)
    forward(TypeError, "k must be", e.q, *e.pools)                                   # bytes without their scales
    forward(TypeError, "8 bits", torch.zeros(8, H_Q, D, dtype=torch.uint8, device="cuda"), *e.pools, cache_scale=scale)
    forward(ValueError, "cache_scale", e.q, *e.pools, cache_scale=scale, block_table=None, cu_k=cu)
    forward(ValueError, "v_scale", e.q, *e.pools, cache_scale=(scale[0], scale[1][:, :1].contiguous()))
    forward(ValueError, "v_cache|one shape", e.q, e.pools[0], e.pools[1][:50], cache_scale=scale)
    forward(ValueError, "contiguous", e.q, *e.pools, cache_scale=(scale[0].transpose(1, 2).contiguous().transpose(1, 2), scale[1]))
    with pytest.raises(ValueError, match="weights' gradients"):
        fa.qk_norm_rope_backward(None, None, e.q, e.q[:, :2].contiguous(), None, None, *e.tables, norm=False, positions=pos, pair_axis=AXES,
                                 grads=(torch.empty_like(e.q), torch.empty_like(e.q[:, :2]), torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")))
    # the same calls with valid arguments run
    fa.qk_norm_rope_append8(q, k, v, e.wq, e.wk, *e.tables, **base)
    _, _, ws = fa.forward(e.q, *e.pools, cache_scale=scale, **kw)
    assert fa.device_status(ws) == 0


def test_a_wait_limit_on_the_rotation():
    """1 ns ends the extended rotation with a timeout status or with a right result; the next call is right."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    x = torch.randn(4096, 10, 128, device="cuda", dtype=torch.bfloat16)
    cos, sin = (torch.from_numpy(a).cuda() for a in ref.angles(MAX_POS, 128))
    pos = torch.randint(0, MAX_POS, (3, 4096), device="cuda", dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(positions=pos, pair_axis=[j % 3 for j in range(64)], norm=False, status=status)
    want = fa.qk_norm_rope(x[:, :8], x[:, 8:], None, None, cos, sin, **kw)
    for _ in range(3):
        fa.qk_norm_rope(x[:, :8], x[:, 8:], None, None, cos, sin, **kw, wait_limit_ns=1)
        assert status.item() in (0, fa.FA_ERR_TIMEOUT)
        status.zero_()
        got = fa.qk_norm_rope(x[:, :8], x[:, 8:], None, None, cos, sin, **kw)
        assert status.item() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
