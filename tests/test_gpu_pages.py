"""mk_assign_pages against a plain restatement that walks the requests one by one: every output is a whole number and has to be
equal."""
import gc
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import persistent_megakernel_decode_sm_gb300 as mk  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def nothing_left_behind():
    """Tracebacks of refused calls hold tensors in cycles: they go before the next module's tests look at the memory."""
    yield
    gc.collect()


class Pool:
    """A paged cache's books in Python: a list of free blocks (front first) and a row of blocks per request."""

    def __init__(self, batch, block, columns, n_blocks, prefix=0, front=0, seed=0):
        r = random.Random(seed)
        ids = list(range(n_blocks))
        r.shuffle(ids)
        self.block, self.columns, self.n_blocks, self.prefix, self.front = block, columns, n_blocks, prefix, front
        self.whole = prefix // block
        self.shared, self.free = ids[:self.whole], ids[self.whole:]
        self.rows = [list(self.shared) for _ in range(batch)]
        self.lens = [0] * batch

    def device(self):
        """(ring, ends, table, lens) of this state; places that hold nothing are -7."""
        ring = [-7] * self.n_blocks
        for i, b in enumerate(self.free):
            ring[(self.front + i) % self.n_blocks] = b
        table = [row + [-7] * (self.columns - len(row)) for row in self.rows]
        return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ring, [self.front, len(self.free), 0], table, self.lens)]

    def step(self, new, max_tokens):
        """The books after the step, and (slots, positions, sequences, first)."""
        need = [max(self.whole, -(-n // self.block)) for n in new]
        for b, n in enumerate(need):
            self.free += self.rows[b][n:]
            del self.rows[b][n:]
        for b, n in enumerate(need):
            while len(self.rows[b]) < n:
                self.rows[b].append(self.free.pop(0))
                self.front = (self.front + 1) % self.n_blocks
        slots, pos, seq, first = [], [], [], [0]
        for b, (old, n) in enumerate(zip(self.lens, new)):
            for p in range(old, n):
                slots.append(self.rows[b][p // self.block] * self.block + p % self.block)
                pos.append(p)
                seq.append(b)
            first.append(len(slots))
        pad = max_tokens - len(slots)
        self.lens = list(new)
        return slots + [-1] * pad, pos + [0] * pad, seq + [-1] * pad, first


def same(got, want):
    assert got.tolist() == list(want)


def run_step(pool, state, new, max_tokens, in_place):
    ring, ends, table, lens = state
    target = torch.tensor(new, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ends_out = None if in_place else torch.full_like(ends, 9)
    out = mk.assign_pages(ring, ends, table, lens, target, pool.block, max_tokens, shared_prefix=pool.prefix, ends_out=ends_out, status=status)
    want = pool.step(new, max_tokens)
    assert status.item() == 0
    for g, w in zip(out, want):
        same(g, w)
    ends_now = ends if in_place else ends_out
    same(ends_now, [pool.front, len(pool.free), 0])
    same(ring.roll(-pool.front)[:len(pool.free)], pool.free)
    for row, blocks in zip(table.tolist(), pool.rows):
        assert row[:len(blocks)] == blocks
    return [ring, ends_now, table, target]


@pytest.mark.parametrize("batch,block,prefix", [(1, 16, 0), (8, 128, 0), (5, 1, 0), (33, 8, 100), (200, 48, 96), (256, 16, 0), (257, 7, 20), (1024, 8, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_requests_that_grow_shrink_and_end(batch, block, prefix, in_place):
    r = random.Random(batch)
    columns = -(-(prefix + 900) // block)
    pool = Pool(batch, block, columns, prefix // block + batch * (-(-300 // block) + 1), prefix, front=3, seed=batch)
    state = pool.device()
    state[0] = state[0].clone()
    for step in range(6):
        new, left = [], len(pool.free)
        for b, old in enumerate(pool.lens):
            how = r.random()
            n = 0 if how < 0.15 else max(0, old - r.randint(0, 50)) if how < 0.25 else old if how < 0.4 else old + r.choice([1, 1, 1, r.randint(1, 200)])
            n = max(n, prefix) if n else 0
            if old == 0 and n:
                n = prefix + r.randint(1, 60)
            more = max(pool.whole, -(-n // block)) - len(pool.rows[b])
            if n > prefix + 900 or more > left:
                n = old
                more = 0
            left -= max(more, 0)
            new.append(n)
        tokens = sum(max(a - b, 0) for a, b in zip(new, pool.lens))
        state = run_step(pool, state, new, tokens + (0, 1, 7, 1000)[step % 4], in_place)


def test_a_million_tokens():
    pool = Pool(256, 128, 64, 256 * 64 + 5, front=100)
    new = [random.Random(b).randint(1, 8192) for b in range(256)]
    for in_place in (False, True):
        p = Pool(256, 128, 64, 256 * 64 + 5, front=100)
        run_step(p, p.device(), new, sum(new) + 3, in_place)
    assert pool.lens == [0] * 256


def test_blocks_that_this_call_returns_are_taken_again():
    pool = Pool(3, 4, 6, 8, front=6)
    state = run_step(pool, pool.device(), [20, 12, 0], 32, False)          # every block is taken
    assert pool.free == []
    state = run_step(pool, state, [2, 12, 15], 32, True)                   # four come back, four are wanted
    assert pool.free == []
    run_step(pool, state, [0, 0, 20], 40, False)


def test_the_same_call_twice_from_one_state():
    pool = Pool(20, 8, 40, 900, front=880)
    state = pool.device()
    new = [random.Random(b).randint(0, 300) for b in range(20)]
    target, ends_out = torch.tensor(new, dtype=torch.int32, device="cuda"), torch.zeros_like(state[1])
    a = [t.clone() for t in mk.assign_pages(*state, target, 8, sum(new), ends_out=ends_out)]
    ring, table = state[0].clone(), state[2].clone()
    b = mk.assign_pages(*state, target, 8, sum(new), ends_out=ends_out)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(ring, state[0]) and torch.equal(table, state[2])


@pytest.mark.parametrize("why", ["blocks", "tokens", "negative", "long", "front", "free", "many", "negative_old", "long_old"])
@pytest.mark.parametrize("big", [False, True])
def test_what_cannot_be_served_changes_nothing(why, big):
    pool = Pool(4, 8, 1000, 700)
    ring, ends, table, lens = run_step(pool, pool.device(), [30, 8, 100, 0], 200, True)
    new, room, want = [40, 9, 0, 20], 100000 if big else 100, mk.MK_ERR_BOUNDS
    if why == "blocks":
        new, room, want = [40, 9, 7000, 20], 100000, mk.MK_ERR_CAPACITY
    elif why == "tokens":
        room, want = 30, mk.MK_ERR_CAPACITY
    elif why == "negative":
        new[1] = -1
    elif why == "long":
        new[1] = 8001
    elif why == "front":
        ends[0] = 700
    elif why == "free":
        ends[1] = -1
    elif why == "many":
        ends[1] = 690                       # with 13 returned more than there are
    elif why == "negative_old":
        lens[2] = -5
    elif why == "long_old":
        lens[2] = 2 ** 31 - 1
    target = torch.tensor(new, dtype=torch.int32, device="cuda")
    before = [t.clone() for t in (ring, ends, table)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots, pos, seq, first = mk.assign_pages(ring, ends, table, lens, target, 8, room, status=status)
    assert status.item() == want
    assert all(torch.equal(a, b) for a, b in zip(before, (ring, ends, table)))
    assert (slots == -1).all() and (seq == -1).all() and not pos.any() and not first.any()


def test_block_ids_outside_the_pool_give_no_slot():
    pool = Pool(2, 4, 10, 12)
    ring, ends, table, lens = run_step(pool, pool.device(), [6, 3], 20, True)
    table[0, 1], status = 12, torch.zeros(1, dtype=torch.int32, device="cuda")
    ring[int(ends[0])] = -3
    target = torch.tensor([9, 5], dtype=torch.int32, device="cuda")
    slots, pos, seq, first = mk.assign_pages(ring, ends, table, lens, target, 4, 10, status=status)
    assert status.item() == mk.MK_ERR_BOUNDS
    assert slots.tolist()[:3] == [-1, -1, -1]            # two in the entry of 12, one in the ring's -3
    assert slots.tolist()[3] == table[1, 0].item() * 4 + 3 and slots.tolist()[4] == table[1, 1].item() * 4
    assert pos.tolist() == [6, 7, 8, 3, 4, 0, 0, 0, 0, 0] and first.tolist() == [0, 3, 5]


def test_no_tokens_given_buffers_and_odd_addresses():
    pool = Pool(3, 8, 4, 20)
    state = run_step(pool, pool.device(), [9, 1, 0], 10, True)
    state = run_step(pool, state, [9, 1, 0], 0, False)
    ring, ends, table, lens = state
    wide = torch.full((100,), 55, dtype=torch.int32, device="cuda")
    out = [wide[1:22], wide[31:52], wide[55:76], wide[80:84]]                # not 16-byte aligned
    target = torch.tensor([17, 30, 2], dtype=torch.int32, device="cuda")
    mk.assign_pages(ring, ends, table, lens, target, 8, 21, out=out)
    assert pool.step([17, 30, 2], 40)[0][:21] != out[0].tolist()             # (39 tokens: more than 21, nothing is assigned)
    assert (out[0] == -1).all() and wide[0] == 55 and (wide[22:31] == 55).all() and (wide[52:55] == 55).all() and (wide[84:] == 55).all()


def test_captured_and_replayed_in_place():
    pool = Pool(6, 4, 50, 400)
    ring, ends, table, lens = pool.device()
    target = lens.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = mk.assign_pages(ring, ends, table, lens, target, 4, 3000)
        lens.copy_(target)
    r = random.Random(1)
    for _ in range(6):
        new = [r.choice([0, n + 1, n + 17]) for n in pool.lens]
        target.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        for got, want in zip(out, pool.step(new, 3000)):
            same(got, want)
        same(ends, [pool.front, len(pool.free), 0])


def test_slots_and_lengths_up_to_2_to_the_31():
    block, columns, n_blocks = 1 << 20, 2047, 2047
    ring = torch.full((n_blocks,), -7, dtype=torch.int32, device="cuda")
    ring[2046], ring[0] = 2046, 5
    table = torch.full((2, columns), -7, dtype=torch.int32, device="cuda")
    table[0, 2045], table[1, 0] = 2045, 3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    most = columns * block
    lens, new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([most - block - 3, 7], [most - block + 2, block + 1]))
    ends = torch.tensor([2046, 2, 0], dtype=torch.int32, device="cuda")
    total = 5 + block + 1 - 7
    slots, pos, seq, first = mk.assign_pages(ring, ends, table, lens, new, block, total + 1, status=status)
    assert status.item() == 0 and ends.tolist() == [1, 0, 0] and table[0, 2046].item() == 2046 and table[1, 1].item() == 5
    a = torch.arange(most - block - 3, most - block + 2, device="cuda")
    b = torch.arange(7, block + 1, device="cuda")
    assert torch.equal(slots[:5].long(), a.where(a < most - block, 2046 * block + (a - (most - block)))) and torch.equal(pos[:5].long(), a)
    assert torch.equal(slots[5:-1].long(), torch.where(b < block, 3 * block + b, 5 * block + (b - block))) and torch.equal(pos[5:-1].long(), b)
    assert slots[-1] == -1 and first.tolist() == [0, 5, total] and seq[:5].sum() == 0 and (seq[5:-1] == 1).all()


def test_the_c_call_without_what_may_be_null():
    import ctypes
    pool = Pool(4, 8, 9, 40, front=35)
    ring, ends, table, lens = pool.device()
    new = [20, 0, 61, 8]
    target, slots = torch.tensor(new, dtype=torch.int32, device="cuda"), torch.full((100,), 9, dtype=torch.int32, device="cuda")
    args = mk.mk_pages_args(4, 8, 9, 40, 0, 100, ring.data_ptr(), ends.data_ptr(), ends.data_ptr(), table.data_ptr(), lens.data_ptr(),
                            target.data_ptr(), slots.data_ptr(), None, None, None, None)
    assert mk.lib.mk_assign_pages(ctypes.addressof(args), torch.cuda.current_stream().cuda_stream) == 0
    same(slots, pool.step(new, 100)[0])
    lens.copy_(target)
    target.zero_()
    args.max_tokens, args.slots = 0, None            # only takes blocks and gives them back
    assert mk.lib.mk_assign_pages(ctypes.addressof(args), torch.cuda.current_stream().cuda_stream) == 0
    pool.step([0] * 4, 0)
    same(ends, [pool.front, len(pool.free), 0])
    same(ring.roll(-pool.front)[:len(pool.free)], pool.free)


def test_two_pools_on_two_streams_at_once():
    pools = [Pool(64, 16, 400, 24000, front=i, seed=i) for i in range(2)]
    states = [p.device() for p in pools]
    streams = [torch.cuda.Stream() for _ in pools]
    r = random.Random(2)
    torch.cuda.synchronize()
    got, want = [], []
    for _ in range(12):
        new = [[min(n + r.choice([1, 40, 700]), 6400) if r.random() < 0.8 else 0 for n in p.lens] for p in pools]
        targets = [torch.tensor(n, dtype=torch.int32, device="cuda") for n in new]
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(mk.assign_pages(*states[i], targets[i], 16, 50000))
                states[i][3] = targets[i]
        want += [p.step(n, 50000) for p, n in zip(pools, new)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            same(a, b)


def test_refusals():
    pool = Pool(3, 8, 4, 20)
    ring, ends, table, lens = pool.device()
    for call in (lambda: mk.assign_pages(ring.long(), ends, table, lens, lens.clone(), 8, 4), lambda: mk.assign_pages(ring, ends[:2], table, lens, lens.clone(), 8, 4),
                 lambda: mk.assign_pages(ring, ends, table[:2], lens, lens.clone(), 8, 4), lambda: mk.assign_pages(ring, ends, table, lens, lens[:2], 8, 4),
                 lambda: mk.assign_pages(ring, ends, table.T, lens, lens.clone(), 8, 4), lambda: mk.assign_pages(ring.cpu(), ends, table, lens, lens.clone(), 8, 4),
                 lambda: mk.assign_pages(ring, ends, table, lens, lens.clone(), 8, 4, out=[torch.empty(3, dtype=torch.int32, device="cuda")] * 4)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mk.assign_pages(ring, ends, table, lens, lens.clone(), 0, 4), lambda: mk.assign_pages(ring, ends, table, lens, lens.clone(), 1 << 29, 4),
                 lambda: mk.assign_pages(ring, ends, table, lens, lens.clone(), 8, 4, shared_prefix=-1), lambda: mk.assign_pages(ring, ends, table, lens, lens.clone(), 8, 4, shared_prefix=40),
                 lambda: mk.assign_pages(ring, ends, table, ring[:3], lens, 8, 4), lambda: mk.assign_pages(ring, ends, table, lens, lens.clone(), 8, 4, ends_out=ring[:3])):
        with pytest.raises(mk.MkError) as e:
            call()
        assert e.value.status == mk.MK_ERR_ARG
