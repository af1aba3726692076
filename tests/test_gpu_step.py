"""The operators around the attention run together, as a serving engine and a training step use
them: page plan, norm + rotation with the cache append, and attention over the paged cache, step
after step and replayed from one captured graph; and norm + rotation, attention and both gradients
in a row."""
import numpy as np
import pytest

import oracle
import step_helpers as ref
from exact_attention_bwd_gb300 import inputs
from gpu_helpers import from_dev

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, PAGE, BLOCKS, POOL, MAX_POS = 6, 2, 64, 16, 24, 90, 400
HALF = 2.0 ** -8


class Engine:
    """Static buffers of a small serving engine: what a captured step reads and writes."""

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
        # the pools hold NaN wherever nothing has been written
        self.k_cache, self.v_cache = (torch.full((POOL, PAGE, H_KV, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.qkv, self.q, self.out = b16(rows, H_Q + 2 * H_KV, D), b16(rows, H_Q, D), b16(rows, H_Q, D)
        self.lse = torch.zeros(H_Q, rows, device="cuda")
        cos, sin = ref.angles(MAX_POS, D)
        self.tables = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
        self.wq, self.wk = (torch.from_numpy(1 + 0.2 * self.rng.standard_normal(D)).cuda().to(torch.bfloat16) for _ in range(2))
        self.ws = None
        self.keys = [[] for _ in range(requests)]  # what the caches should hold
        self.values = [[] for _ in range(requests)]

    def call(self):
        q, k, v = self.qkv[:, :H_Q], self.qkv[:, H_Q:H_Q + H_KV], self.qkv[:, H_Q + H_KV:]
        cu, used, positions, slots, _ = self.fa.page_plan(self.cached, self.fresh, self.table, self.free, page_size=PAGE, num_pages=POOL,
                                                          tokens=self.rows, free_head=self.head, out=self.plan, status=self.status)
        self.fa.qk_norm_rope(q, k, self.wq, self.wk, *self.tables, positions=positions, v=v, k_cache=self.k_cache, v_cache=self.v_cache,
                             slots=slots, out=(self.q, None), status=self.status)
        _, _, ws = self.fa.forward(self.q, self.k_cache, self.v_cache, causal=True, cu_q=cu, seqused_k=used, block_table=self.table,
                                   s_kv=BLOCKS * PAGE, out=self.out, lse=self.lse, workspace=self.ws)
        return ws

    def step(self, fresh, run):
        """One step with these new tokens a request: fills the buffers, runs, checks."""
        torch = self.torch
        n = int(sum(fresh))
        assert n <= self.rows
        bits = inputs.bf16_bits(self.rng.standard_normal((self.rows, H_Q + 2 * H_KV, D)).astype(np.float32))
        self.qkv.copy_(torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16))
        self.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        self.out.fill_(7.0)
        run()
        assert self.fa.device_status(self.ws) == 0 and self.status.item() == 0
        lengths = [len(k) for k in self.keys]
        positions = np.concatenate([np.arange(c, c + f) for c, f in zip(lengths, fresh)]).astype(np.int32)
        np.testing.assert_array_equal(self.plan[2][:n].cpu().numpy(), positions)
        # the rows that should be cached: the same operator without a cache
        if n:
            qr, kr = self.fa.qk_norm_rope(self.qkv[:n, :H_Q], self.qkv[:n, H_Q:H_Q + H_KV], self.wq, self.wk, *self.tables,
                                          positions=torch.from_numpy(positions).cuda())
            assert torch.equal(qr, self.q[:n])
            kr, vr, at = from_dev(kr), from_dev(self.qkv[:n, H_Q + H_KV:]), 0
            for b, f in enumerate(fresh):
                self.keys[b] += list(kr[at:at + f])
                self.values[b] += list(vr[at:at + f])
                at += f
            used = [len(k) for k in self.keys]
            cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (fresh, used))
            k, v = (np.concatenate([np.stack(x) for x in y if x]) for y in (self.keys, self.values))
            kw = dict(causal=True, cu_q=cu_q, cu_k=cu_k, scale=D ** -0.5)
            want, lse, _ = oracle.fwd(from_dev(qr), k, v, **kw)
            spread, _, _ = oracle.fwd(from_dev(qr), k, np.abs(v), **kw)
            err = np.abs(from_dev(self.out[:n]) - want)
            assert np.all(err <= HALF * np.abs(want) + (HALF + 2.0 ** -13) * spread + 2.0 ** -24)
            assert np.abs(self.lse[:, :n].cpu().numpy() - lse).max() <= 3e-4
        assert torch.all(self.out[n:] == 7)
        # the engine's state moves on
        self.cached.copy_(self.plan[1])
        self.head.copy_(self.plan[4])


STEPS = [[40, 17, 0, 3, 0], [1, 1, 0, 1, 0], [60, 1, 33, 1, 0], [1, 1, 1, 1, 1], [5, 0, 5, 0, 5], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0], [1, 90, 1, 1, 1]]


def test_serving_steps():
    e = Engine(5, 128, 1)
    for fresh in STEPS:
        def run():
            e.ws = e.call()
        e.step(fresh, run)


def test_serving_steps_from_two_graphs():
    """The whole step captured twice on one workspace and replayed in turn, the lengths and inputs
    changing in place; on a stream of its own."""
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


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_training_step(kind):
    """x -> norm + rotation -> attention -> loss and back, against 64-bit automatic differentiation.
    Each stage rounds its result once (half a step h relative to it), the attention's two products
    of either direction round P and dS besides: eight roundings in a row, and the products and
    sums between them keep relative errors (2-norm) to within a small factor: 16 h in all."""
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    h = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    B, S, h_q, h_kv, d, rot = 2, 150, 4, 2, 64, 32
    g = torch.Generator().manual_seed(5)
    x = torch.randn(B, S, h_q + 2 * h_kv, d, generator=g, dtype=torch.float64).to(dt)
    w = [(1 + 0.2 * torch.randn(d, generator=g, dtype=torch.float64)).to(dt) for _ in range(2)]
    dout = torch.randn(B, S, h_q, d, generator=g, dtype=torch.float64).to(dt)
    cos, sin = (torch.from_numpy(t) for t in ref.angles(S, rot))

    leaves = [t.double().requires_grad_() for t in (x, *w)]
    xx, wq, wk = leaves

    def turn(y):
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        c, s = cos.double()[:, None], sin.double()[:, None]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), y[..., rot:]], -1)

    def norm(y, w):
        return turn(y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w)

    q, k, v = norm(xx[:, :, :h_q], wq), norm(xx[:, :, h_q:h_q + h_kv], wk), xx[:, :, h_q + h_kv:]
    k, v = (t.repeat_interleave(h_q // h_kv, 2) for t in (k, v))
    p = torch.einsum("bihd,bjhd->bhij", q, k) * d ** -0.5
    p = p.masked_fill(torch.ones(S, S).triu(1).bool(), float("-inf")).softmax(-1)
    (torch.einsum("bhij,bjhd->bihd", p, v) * dout.double()).sum().backward()

    xd, (wqd, wkd), dod, tables = x.cuda(), [t.cuda() for t in w], dout.cuda(), (cos.cuda(), sin.cuda())
    rq, rk, rv = xd[:, :, :h_q], xd[:, :, h_q:h_q + h_kv], xd[:, :, h_q + h_kv:].contiguous()
    q, k = fa.qk_norm_rope(rq, rk, wqd, wkd, *tables, interleaved=True)
    o, lse, _ = fa.forward(q, k, rv, causal=True)
    dq, dk, dv, _, _ = fa.backward(q, k, rv, o, lse, dod, causal=True)
    dx = torch.empty_like(xd)
    dwq, dwk = (torch.empty(d, device="cuda") for _ in range(2))
    fa.qk_norm_rope_backward(rq, rk, dq, dk, wqd, wkd, *tables, interleaved=True, grads=(dx[:, :, :h_q], dx[:, :, h_q:h_q + h_kv], dwq, dwk))
    dx[:, :, h_q + h_kv:] = dv
    for name, got, want in (("dx", dx, xx.grad), ("dwq", dwq, wq.grad), ("dwk", dwk, wk.grad)):
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= 16 * h, (name, err)
