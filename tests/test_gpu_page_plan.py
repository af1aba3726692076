"""The page plan on the GPU against a token-by-token plain form: every output equal."""
import numpy as np
import pytest

import step_helpers as ref
from gpu_helpers import Guarded

pytestmark = pytest.mark.gpu


def make(B, P, cached_max, fresh_max, seed, width=None, spare=5, head=3):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, cached_max + 1, B).astype(np.int32)
    fresh = rng.integers(0, fresh_max + 1, B).astype(np.int32)
    blocks = -(-(cached + fresh) // P)
    width = width or max(1, int(blocks.max(initial=1)) + 1)
    old = -(-cached // P)
    need = int((blocks - old).sum())
    num_pages = int(old.sum()) + need + spare + head
    order = rng.permutation(num_pages).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :old[b]] = order[at:at + old[b]]
        at += old[b]
    return dict(cached=cached, fresh=fresh, table=table, free=order[at:], head=head, P=P, num_pages=num_pages,
                T=int(fresh.sum()) + 4)


def run(c, with_head=True):
    import torch
    from exact_attention_bwd_gb300 import binding as fa
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    B, T = len(c["cached"]), c["T"]
    outs = [Guarded((n,), torch.int32) for n in (B + 1, B, T, T, 1)]
    table = Guarded(c["table"].shape, torch.int32)
    table.t.copy_(up(c["table"]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    head = torch.tensor([c["head"]], dtype=torch.int32, device="cuda") if with_head else None
    got = fa.page_plan(up(c["cached"]), up(c["fresh"]), table.t, up(c["free"]), page_size=c["P"], num_pages=c["num_pages"],
                       tokens=T, free_head=head, out=[g.t for g in outs], status=status)
    for g in outs + [table]:
        g.check("page plan")
    return [x.cpu().numpy() for x in got] + [table.t.cpu().numpy(), int(status.item())]


def compare(c, with_head=True, bad=False):
    cu, used, positions, slots, head, table, want_bad = ref.page_plan(
        c["cached"], c["fresh"], c["table"], c["free"], c["head"] if with_head else 0, c["P"], c["num_pages"], c["T"])
    assert want_bad == bad
    got = run(c, with_head)
    for name, x, y in zip(("cu", "used", "positions", "slots", "head", "table"), got, (cu, used, positions, slots, [head], table)):
        np.testing.assert_array_equal(x, y, err_msg=name)
    assert got[-1] == (6 if bad else 0)


@pytest.mark.parametrize("B,P,cached_max,fresh_max", [
    (1, 16, 0, 1), (1, 64, 100, 1), (3, 16, 40, 1), (5, 48, 500, 0), (7, 128, 300, 9), (33, 16, 200, 40),
    (513, 16, 90, 3), (1025, 32, 50, 20), (40, 1, 20, 7), (4, 16, 50, 5000), (1, 16, 17, 40000),
])
def test_page_plan(B, P, cached_max, fresh_max):
    compare(make(B, P, cached_max, fresh_max, seed=B + P))


def test_page_plan_without_head_and_empty():
    compare(make(6, 16, 60, 5, seed=1, head=0), with_head=False)
    c = make(2, 16, 60, 5, seed=2)
    c["fresh"][:] = 0
    c["T"] = 0
    compare(c)
    empty = dict(cached=np.zeros(0, np.int32), fresh=np.zeros(0, np.int32), table=np.zeros((0, 3), np.int32),
                 free=np.arange(4, dtype=np.int32), head=2, P=16, num_pages=4, T=3)
    compare(empty)


def test_page_plan_bad_inputs_are_reported():
    """Each rule broken in turn; every output still has the stated value and nothing is written
    out of place."""
    c = make(6, 16, 60, 30, seed=3)
    c["free"] = c["free"][:c["head"] + 2]                 # pages run out
    compare(c, bad=True)
    c = make(6, 16, 60, 30, seed=4)
    c["free"][c["head"] + 1] = c["num_pages"]             # a page outside the pool
    compare(c, bad=True)
    c = make(3, 16, 60, 30, seed=5)
    c["cached"][1], c["fresh"][1] = 17, 3
    c["table"][1, :2] = -1                                # the part-filled page is missing
    c["free"] = np.arange(20, dtype=np.int32)
    c["num_pages"] = 40
    c["T"] = int(c["fresh"].sum())
    compare(c, bad=True)
    c = make(4, 16, 60, 30, seed=6)
    c["cached"][2], c["fresh"][3] = -5, -1                # negative lengths
    c["free"] = np.arange(60, dtype=np.int32) % 40
    c["num_pages"] = 60
    compare(c, bad=True)
    c = make(4, 16, 60, 30, seed=7, width=4)              # a request beyond its row of the table
    c["cached"][0], c["fresh"][0] = 60, 30
    c["free"] = np.arange(40, dtype=np.int32)
    c["num_pages"] = 200
    c["T"] = int(c["fresh"].sum())
    compare(c, bad=True)
    c = make(9, 16, 60, 30, seed=8)
    c["T"] = int(c["fresh"].sum()) - 3                    # more tokens than rows
    compare(c, bad=True)
