"""GPU: spec_block_tables against a stack of page numbers popped and pushed by hand: growth and return in one
call, a shared prefix, a stack that runs out, requests in error, padding rows, many requests; two calls that undo
each other; the slots as spec_compact takes them."""
import random

import pytest
import torch

from speculative_decoding_verification_43_gb300 import api

pytestmark = pytest.mark.gpu


def blocks(x, page):
    return (x + page - 1) // page


class Pool:
    """Requests holding pages out of a shuffled pool; `spare` pages on the stack."""

    def __init__(self, held, page, spare, shared=0, width=None, seed=0):
        r = random.Random(seed)
        self.page, self.n_shared = page, shared
        own = [max(h - shared, 0) for h in held]
        self.n_pages = shared + sum(own) + spare
        ids = list(range(self.n_pages))
        r.shuffle(ids)
        self.shared = ids[:shared]
        self.width = width or max([1, *held]) + 40
        at = shared
        self.table = []
        for h, k in zip(held, own):
            row = self.shared[:min(h, shared)] + [-1] * max(shared - h, 0) + ids[at:at + k]
            self.table.append(row + [-1] * (self.width - len(row)))
            at += k
        self.held, self.stack = list(held), ids[at:]

    def device(self, dev="cuda"):
        i32 = dict(dtype=torch.int32, device=dev)
        self.d = dict(n_blocks=torch.tensor(self.held, **i32), block_table=torch.tensor(self.table, **i32),
                      free_pages=torch.tensor(self.stack + [-1] * (self.n_pages - len(self.stack)), **i32),
                      n_free=torch.tensor([len(self.stack)], **i32))
        self.dev_shared = torch.tensor(self.shared, **i32) if self.n_shared else None
        return self

    def step(self, kv):
        """The definition; returns the requests' status."""
        page, sh = self.page, self.n_shared
        status = [0] * len(kv)
        need = list(self.held)
        for i, x in enumerate(kv):
            if x < 0 or not 0 <= self.held[i] <= self.width:
                status[i] = 4
            elif blocks(x, page) > self.width:
                status[i] = 16
            else:
                need[i] = blocks(x, page)
        for i in reversed(range(len(kv))):
            for b in reversed(range(max(need[i], sh), self.held[i])):
                self.stack.append(self.table[i][b])
        out = False
        for i in range(len(kv)):
            take = max(need[i] - max(self.held[i], sh), 0)
            if take and (out or take > len(self.stack)):
                out = True
                status[i] = 16
                continue
            for b in range(self.held[i], need[i]):
                self.table[i][b] = self.shared[b] if b < sh else self.stack.pop()
            self.held[i] = need[i]
        return status

    def same(self):
        d = {n: t.cpu().tolist() for n, t in self.d.items()}
        assert d["n_blocks"] == self.held
        assert d["n_free"] == [len(self.stack)]
        assert d["free_pages"][:len(self.stack)] == self.stack
        for i, h in enumerate(self.held):
            assert d["block_table"][i][:h] == self.table[i][:h], i

    def rows(self, n, kv, status):
        """slot_map and positions of n[i] rows each."""
        slots, pos = [], []
        for i, c in enumerate(n):
            for j in range(c):
                p = kv[i] - c + j
                ok = p >= 0 and status[i] == 0
                slots.append(self.table[i][p // self.page] * self.page + p % self.page if ok else -1)
                pos.append(p if p >= 0 and kv[i] >= 0 else -1)
        return slots, pos


def call(pool, kv, n=None):
    i32 = dict(dtype=torch.int32, device="cuda")
    off = None
    if n is not None:
        off = [0]
        for c in n:
            off.append(off[-1] + c)
    o = api.block_tables(torch.tensor(kv, **i32), *pool.d.values(), pool.page,
                         row_off=torch.tensor(off, **i32) if n is not None else None, total_rows=off[-1] if n else 0,
                         shared_table=pool.dev_shared)
    torch.cuda.synchronize()
    return o


def check_step(pool, kv, n=None):
    o = call(pool, kv, n)
    status = pool.step(kv)
    assert o.req_status.cpu().tolist() == status
    pool.same()
    if n is not None:
        slots, pos = pool.rows(n, kv, status)
        assert o.slot_map.cpu().tolist() == slots
        assert o.positions.cpu().tolist() == pos
    return status


@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("B", [1, 5, 64, 1024, 1500])
@pytest.mark.parametrize("shared", [0, 3])
def test_random_steps(page, B, shared):
    r = random.Random(B * 31 + page + shared)
    kv = [r.randrange(0, 200) + shared * page for _ in range(B)]
    pool = Pool([blocks(x, page) for x in kv], page, B * 30, shared, width=blocks(400, page) + shared, seed=B).device()
    for step in range(4):
        n = [r.choice([0, 1, 4, r.randrange(0, 9)]) for _ in range(B)]
        kv = [max(c, x + r.choice([0, 1, c, -5, r.randrange(-60, 60)])) if r.random() < 0.9 else 0 for x, c in zip(kv, n)]
        check_step(pool, kv, n if step != 2 else None)


def test_prompts_in_two_kernels():
    r = random.Random(3)
    n = [r.randrange(1, 900) for _ in range(40)]
    pool = Pool([0] * 40, 16, 2500, 5, width=80).device()
    kv = [c + 80 for c in n]
    check_step(pool, kv, n)
    check_step(pool, [0] * 40)
    check_step(pool, kv[::-1], n[::-1])


def test_back_undoes_forth():
    r = random.Random(9)
    kv = [r.randrange(1, 300) for _ in range(50)]
    pool = Pool([blocks(x, 16) for x in kv], 16, 300, seed=4).device()
    before = {n: t.clone() for n, t in pool.d.items()}
    call(pool, [x + r.randrange(0, 60) for x in kv])
    call(pool, kv)
    for name in ("n_blocks", "free_pages", "n_free"):
        assert torch.equal(pool.d[name], before[name]), name
    for i, x in enumerate(kv):
        h = blocks(x, 16)
        assert torch.equal(pool.d["block_table"][i, :h], before["block_table"][i, :h])


def test_stack_runs_out():
    """From the first request that does not fit on, those that need pages get none; others go on."""
    pool = Pool([1, 1, 3, 1, 1, 2], 8, 2, width=20).device()
    status = check_step(pool, [16, 8, 8, 60, 16, 16], [2, 1, 1, 3, 2, 1])
    assert status == [0, 0, 0, 16, 16, 0]
    status = check_step(pool, [0, 8, 8, 40, 16, 16], [0, 1, 1, 3, 2, 1])
    assert 16 in status or status == [0] * 6


def test_requests_in_error():
    pool = Pool([2, 3, 1, 2, 2], 4, 10, width=6).device()
    status = check_step(pool, [12, -1, 25, 8, 3], [2, 1, 3, 0, 4])
    assert status == [0, 4, 16, 0, 0]


@pytest.mark.parametrize("held", [-1, 7, 1 << 30])
def test_counts_out_of_range(held):
    pool = Pool([2, 3, 1], 4, 10, width=6).device()
    pool.held[1] = held
    pool.d["n_blocks"][1] = held
    status = pool.step([12, 28, 8])
    o = call(pool, [12, 28, 8], [1, 2, 1])
    assert o.req_status.cpu().tolist() == status == [0, 4, 0]
    assert pool.d["n_blocks"].cpu().tolist() == pool.held
    assert o.slot_map.cpu().tolist()[1:3] == [-1, -1]


@pytest.mark.parametrize("n_free", [-1, 1000, 15])
def test_stack_that_cannot_be_right(n_free):
    """n_free out of range: nobody takes or gives. In range, but with what comes back more than there are pages:
    nobody gives."""
    pool = Pool([2, 3, 1, 2], 4, 8, width=6).device()   # 16 pages
    pool.d["n_free"][0] = n_free
    before = {n: t.clone() for n, t in pool.d.items()}
    o = call(pool, [8, 4, 12, 8])                       # request 1 gives two, request 2 takes two
    status = o.req_status.cpu().tolist()
    assert status == [0, 16, 16 if n_free != 15 else 0, 0]
    if n_free != 15:
        for n, t in pool.d.items():
            assert torch.equal(t, before[n]), n
    else:
        assert pool.d["n_free"].item() == 13 and pool.d["n_blocks"].cpu().tolist() == [2, 3, 3, 2]


def test_offsets_in_doubt_cost_the_rows_alone():
    pool = Pool([1, 1, 1, 1], 8, 20, width=10).device()
    i32 = dict(dtype=torch.int32, device="cuda")
    t = api.BlockTables(4, 8, 8, pool.n_pages).bind(torch.tensor([20, 21, 22, 23], **i32), *pool.d.values(),
                                                    row_off=torch.tensor([1, 3, 99, 5, 7], **i32))
    t.out.slot_map.fill_(-7)
    o = t.run()
    torch.cuda.synchronize()
    assert o.req_status.cpu().tolist() == [0, 4, 4, 0]
    pool.step([20, 21, 22, 23])
    pool.same()
    want = [-7] * 8
    for i, rows in ((0, (1, 2)), (3, (5, 6))):
        for j, row in enumerate(rows):
            p = [20, 21, 22, 23][i] - 2 + j
            want[row] = pool.table[i][p // 8] * 8 + p % 8
    assert o.slot_map.cpu().tolist() == want


def test_pages_outside_the_pool_have_no_slot():
    pool = Pool([2], 4, 5, width=6).device()
    pool.d["block_table"][0, 1] = 10 ** 6
    o = call(pool, [8], [6])
    assert o.slot_map.cpu().tolist()[2:] == [-1] * 4 and min(o.slot_map.cpu().tolist()[:2]) >= 0


def test_without_outputs():
    """slot_map, positions and status are optional."""
    pool = Pool([1, 2], 4, 10, width=6).device()
    i32 = dict(dtype=torch.int32, device="cuda")
    t = api.BlockTables(2, 3, 4, pool.n_pages).bind(torch.tensor([9, 12], **i32), *pool.d.values(),
                                                    row_off=torch.tensor([0, 1, 3], **i32))
    t.args.slot_map = t.args.positions = t.args.req_status = None
    t.run()
    torch.cuda.synchronize()
    pool.step([9, 12])
    pool.same()


@pytest.mark.parametrize("more", [0, 600], ids=["one block", "two kernels"])
def test_rows_whose_offsets_are_contradicted_have_no_slot(more):
    """Requests 1 and 3 have offsets that contradict one another's: their rows get -1, which a reader of slot_map can
    tell from a slot. Rows of no request keep what was there. `more` requests of a row each behind them."""
    off = [1, 3, 6, 4, 8, *range(9, 9 + more)]
    kv = [20, 21, 22, 23] + [5 + i % 30 for i in range(more)]
    pool = Pool([1, 1, 1, 1] + [0] * more, 8, 20 + 5 * more, width=10).device()
    T = off[-1] + 2
    i32 = dict(dtype=torch.int32, device="cuda")
    t = api.BlockTables(4 + more, T, 8, pool.n_pages).bind(torch.tensor(kv, **i32), *pool.d.values(),
                                                           row_off=torch.tensor(off, **i32))
    t.out.slot_map.fill_(-7)
    t.out.positions.fill_(-7)
    o = t.run()
    torch.cuda.synchronize()
    assert o.req_status.cpu().tolist() == [0, 4, 4, 4] + [0] * more
    pool.step(kv)
    pool.same()
    slots, pos = [-7, 0, 0, -1, -1, -1, -1, -1] + [-7] * (T - 8), [-7, 18, 19, -1, -1, -1, -1, -1] + [-7] * (T - 8)
    for r in (1, 2):
        slots[r] = pool.table[0][pos[r] // 8] * 8 + pos[r] % 8
    for i in range(more):
        p = pos[8 + i] = kv[4 + i] - 1
        slots[8 + i] = pool.table[4 + i][p // 8] * 8 + p % 8
    assert o.slot_map.cpu().tolist() == slots
    assert o.positions.cpu().tolist() == pos


def test_rows_of_no_request_have_no_slot():
    pool = Pool([2, 1], 8, 4, width=6).device()
    i32 = dict(dtype=torch.int32, device="cuda")
    o = api.block_tables(torch.tensor([9, 8], **i32), *pool.d.values(), 8, row_off=torch.tensor([2, 4, 5], **i32), total_rows=8)
    torch.cuda.synchronize()
    assert o.slot_map.cpu().tolist()[:2] == [-1, -1] and o.slot_map.cpu().tolist()[5:] == [-1] * 3
    assert o.positions.cpu().tolist() == [-1, -1, 7, 8, 7, -1, -1, -1]
