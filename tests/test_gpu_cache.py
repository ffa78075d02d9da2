"""kv_slots and kv_write against plain host models: whole numbers and copies, so equal."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def w12():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lossless_bit_weights_gb300 as m
    m.lib()
    return m


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def i64(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int64))).cuda()


class Pool:
    """Host model: a free list in order, tables as lists."""

    def __init__(self, rng, lens, block, free, width, head=0):
        self.block, self.width = block, width
        need = [-(-n // block) for n in lens]
        self.blocks = sum(need) + free
        ids = rng.permutation(self.blocks).tolist()
        self.lens = list(lens)
        self.tables, at = [], 0
        for n in need:
            self.tables.append(ids[at:at + n])
            at += n
        self.free, self.head, self.tail = ids[at:], head, head + free

    def device(self):
        table = np.full((len(self.lens), self.width), -7, np.int32)
        for r, t in enumerate(self.tables):
            table[r, :len(t)] = t
        pool = np.full(self.blocks, -9, np.int32)
        pool[(self.head + np.arange(len(self.free))) % self.blocks] = self.free
        return i32(table), i32(pool), i64([self.head, self.tail])

    def step(self, add, extra=0, path=None, off=None):
        slot, src, back = [], [], []
        for r, a in enumerate(x + extra for x in add):
            if a == -1:
                back += self.tables[r]
                self.tables[r], self.lens[r] = [], 0
                continue
            for j in range(a):
                p = self.lens[r] + j
                if p // self.block == len(self.tables[r]):
                    self.tables[r].append(self.free.pop(0))
                    self.head += 1
                src.append(len(slot) if path is None else off[r] + path[off[r] + j])
                slot.append(self.tables[r][p // self.block] * self.block + p % self.block)
            self.lens[r] += a
        self.free += back
        self.tail += len(back)
        return slot, src

    def check(self, out, table, pool, slot, src, capacity):
        assert int(out.status) == 0
        assert int(out.total) == len(slot)
        assert out.slot.tolist() == slot + [-1] * (capacity - len(slot))
        assert out.src.tolist() == src + [-1] * (capacity - len(slot))
        assert out.new_len.tolist() == self.lens
        assert out.pool_pos.tolist() == [self.head, self.tail]
        t, p = table.cpu().numpy(), pool.cpu().numpy()
        for r, want in enumerate(self.tables):
            assert t[r, :len(want)].tolist() == want
        assert p[np.arange(self.head, self.tail) % self.blocks].tolist() == self.free


@pytest.mark.parametrize("block", [1, 7, 16, 128])
@pytest.mark.parametrize("n_req", [1, 2, 31, 256, 257, 1000, 4096])
def test_prompts_and_releases(w12, n_req, block):
    rng = np.random.default_rng(n_req * 1000 + block)
    lens = rng.integers(0, 40, n_req).tolist()
    width = -(-(40 + 60) // block)
    pool = Pool(rng, lens, block, n_req * (width + 1), width, head=int(rng.integers(0, 10 ** 6)))
    table, ring, pos = pool.device()
    length = i32(lens)
    for step in range(3):                                # each step on the last one's results
        add = rng.integers(-1, 21, n_req)
        add[rng.random(n_req) < 0.3] = 0
        total = int(np.maximum(add, 0).sum())
        capacity = max(1, total + step)
        slot, src = pool.step(add.tolist())
        out = w12.kv_slots(length, i32(add), table, ring, pos, block, capacity)
        pool.check(out, table, ring, slot, src, capacity)
        length, pos = out.new_len, out.pool_pos


@pytest.mark.parametrize("n_req,block", [(1, 16), (24, 16), (24, 3), (300, 64)])
def test_commits(w12, n_req, block):
    rng = np.random.default_rng(n_req + block)
    lens = rng.integers(0, 100, n_req).tolist()
    counts = rng.integers(1, 12, n_req)
    off = np.concatenate([[0], np.cumsum(counts)])
    path_len = np.array([rng.integers(-1, n) for n in counts])
    path = np.concatenate([rng.permutation(n) for n in counts])
    width = -(-120 // block)
    pool = Pool(rng, lens, block, n_req * 13, width)
    table, ring, pos = pool.device()
    slot, src = pool.step(path_len.tolist(), 1, path.tolist(), off.tolist())
    capacity = int(off[-1])
    out = w12.kv_slots(i32(lens), i32(path_len), table, ring, pos, block, capacity, extra=1, path_nodes=i32(path),
                       req_offsets=i32(off))
    pool.check(out, table, ring, slot, src, capacity)


def test_one_long_prompt(w12):
    rng = np.random.default_rng(3)
    pool = Pool(rng, [5, 0], 16, 20000, 10000)
    table, ring, pos = pool.device()
    slot, src = pool.step([131072, 0])
    out = w12.kv_slots(i32([5, 0]), i32([131072, 0]), table, ring, pos, 16, 131072)
    pool.check(out, table, ring, slot, src, 131072)


@pytest.mark.parametrize("case", ["pool", "capacity", "width", "length", "append", "ring", "ring over", "path", "offsets"])
def test_all_or_nothing(w12, case):
    rng = np.random.default_rng(4)
    lens, add, extra, capacity, path, off = [20, 33, 16], [5, 3, 40], 0, 100, None, None
    free, width, want = 9, 6, 1
    if case == "pool":
        free, want = 2, 2
    if case == "capacity":
        capacity, want = 47, 4
    if case == "width":
        add = [5, 3, 16 * 6 - 15]
    if case == "append":
        add = [5, -2, 3]
    pool = Pool(rng, lens, 16, free, width)
    table, ring, pos = pool.device()
    length = i32(lens)
    if case == "length":
        length[1] = -3
    if case == "ring":
        pos, want = i64([7, 5]), 2
    if case == "ring over":                              # more blocks returned than the ring can hold
        add, pos, want = [-1, -1, -1], i64([0, pool.blocks - 1]), 2
    if case == "path":
        path, off, add, extra = list(range(12)), [0, 4, 8, 12], [2, 4, 1], 1
    if case == "offsets":
        path, off, add, extra = list(range(12)), [0, 4, 8, 13], [2, 2, 1], 1
    before = table.clone(), ring.clone()
    out = w12.kv_slots(length, i32(add), table, ring, pos, 16, capacity, extra=extra,
                       path_nodes=None if path is None else i32(path), req_offsets=None if off is None else i32(off))
    assert int(out.status) == want
    assert int(out.total) == 0 and (out.slot == -1).all() and (out.src == -1).all()
    assert torch.equal(out.new_len, length) and torch.equal(out.pool_pos, pos)
    assert torch.equal(table, before[0]) and torch.equal(ring, before[1])


def test_a_path_node_outside_its_request(w12):
    pool = Pool(np.random.default_rng(5), [4, 4], 16, 4, 3)
    table, ring, pos = pool.device()
    out = w12.kv_slots(i32([4, 4]), i32([1, 1]), table, ring, pos, 16, 4, extra=1, path_nodes=i32([0, 3, 1, 0, 1, 9]),
                       req_offsets=i32([0, 3, 6]))
    assert int(out.status) == 8
    assert out.src.tolist() == [0, -1, 3, 4]
    assert int(out.total) == 4


@pytest.mark.parametrize("where", ["table", "pool"])
def test_a_negative_entry_does_not_pass_for_padding(w12, where):
    """-1 times the block size plus the last place of a block is -1, kv_slots' own padding."""
    table, ring, pos = i32([[0, 1, 2]]), i32([3, 4, 5, 6]), i64([0, 3])
    if where == "table":
        table[0, 1] = -1  # positions 4 to 7
    else:
        ring[0] = -1      # positions 8 to 11 (two blocks are held)
    out = w12.kv_slots(i32([5]), i32([7]), table, ring, pos, 4, 9)
    want = [-2] * 3 + [12, 13, 14, 15] if where == "table" else [5, 6, 7] + [-2] * 4
    assert out.slot.tolist() == want + [-1] * 2
    assert int(out.status) == 8 and int(out.total) == 7


def test_slot_refusals(w12):
    table, ring, pos = Pool(np.random.default_rng(6), [4, 4], 16, 4, 3).device()
    lens, add = i32([4, 4]), i32([1, 1])
    with pytest.raises(ValueError):
        w12.kv_slots(lens[:1], add, table, ring, pos, 16, 4)
    with pytest.raises(ValueError):
        w12.kv_slots(lens, add, table.long(), ring, pos, 16, 4)
    with pytest.raises(ValueError):
        w12.kv_slots(lens, add, table, ring, pos.int(), 16, 4)
    with pytest.raises(ValueError):
        w12.kv_slots(lens, add, table, ring, pos, 16, 4, path_nodes=i32([0, 0]), req_offsets=i32([0, 1]))
    with pytest.raises(w12.W12Error) as e:
        w12.kv_slots(lens, add, table[:1].expand(2, 3), ring, pos, 16, 4)
    assert e.value.status == 2
    for block, capacity in ((0, 4), (16, 0)):
        with pytest.raises(w12.W12Error) as e:
            w12.kv_slots(lens, add, table, ring, pos, block, capacity)
        assert e.value.status == 2


# ---------------------------------------------------------------- rows into slots

@pytest.mark.parametrize("layers,hkv,d,block,layout", [(1, 1, 8, 16, "nhd"), (1, 8, 128, 16, "nhd"), (3, 2, 64, 8, "hnd"),
                                                       (16, 4, 256, 64, "nhd"), (2, 3, 1024, 1, "hnd"), (2, 5, 40, 24, "nhd")])
def test_rows_land_in_their_slots(w12, layers, hkv, d, block, layout):
    g = torch.Generator(device="cuda").manual_seed(d)
    rng = np.random.default_rng(d)
    blocks, n_rows, n = 9, 50, 40
    n = min(n, blocks * block)
    shape = (layers + 1, blocks, block, hkv, d) if layout == "nhd" else (layers + 1, blocks, hkv, block, d)
    kc, vc = (torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda", dtype=torch.int16) for _ in range(2))
    if layout == "hnd":
        kc, vc = kc.transpose(2, 3), vc.transpose(2, 3)
    rows = torch.randint(-2 ** 15, 2 ** 15, (layers, n_rows, 2 * hkv, d), generator=g, device="cuda", dtype=torch.int16)
    k, v = rows[:, :, :hkv], rows[:, :, hkv:]
    slot = rng.permutation(blocks * block)[:n]
    src = rng.integers(0, n_rows, n)
    slot[::7] = -1
    want = []
    for c, x in ((kc, k), (vc, v)):
        w = c.cpu().clone()
        for t in range(n):
            if slot[t] >= 0:
                w[1:, slot[t] // block, slot[t] % block] = x[:, src[t]].cpu()
        want.append(w)
    st = w12.kv_write(w12.KVCache(kc, vc), k, v, i64(slot), src=i32(src), layer=1)
    assert int(st) == 0
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


def test_rows_in_order_without_a_source(w12):
    kc, vc = (torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.randn((5, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    w12.kv_write(w12.KVCache(kc, vc), k, v, i64([3, 60, 17, -1, 0]))
    flat = kc.view(64, 2, 64), vc.view(64, 2, 64)
    for c, x in zip(flat, (k, v)):
        for t, s in enumerate((3, 60, 17, -1, 0)):
            if s >= 0:
                assert torch.equal(c[s], x[t])
        assert int((c != 0).any(2).any(1).sum()) == 4


def test_slots_and_rows_out_of_range_are_skipped_and_reported(w12):
    kc, vc = (torch.zeros((4, 16, 1, 64), dtype=torch.int16, device="cuda") for _ in range(2))
    k = torch.ones((3, 1, 64), dtype=torch.int16, device="cuda")
    cache = w12.KVCache(kc, vc)
    for slot, src in (([64], [0]), ([-2], [0]), ([2 ** 40], [0]), ([5], [3]), ([5], [-1])):
        st = w12.kv_write(cache, k, k, i64(slot), src=i32(src))
        assert int(st) == 1 and not kc.any() and not vc.any()
    st = w12.kv_write(cache, k, k, i64([-1, 7, 99]))
    assert int(st) == 1 and int(kc.any(2).any(2).sum()) == 1 and kc[0, 7].all()


def test_a_cache_past_32_bits(w12):
    block, hkv, d = 64, 2, 128
    blocks = (1 << 31) // (block * hkv * d) + 3
    kc, vc = (torch.empty((blocks, block, hkv, d), dtype=torch.int16, device="cuda") for _ in range(2))
    k, v = (torch.randint(-9, 9, (2, hkv, d), device="cuda", dtype=torch.int16) for _ in range(2))
    last = blocks * block - 1
    st = w12.kv_write(w12.KVCache(kc, vc), k, v, i64([last, 0]))
    assert int(st) == 0
    assert torch.equal(kc[-1, -1], k[0]) and torch.equal(vc[-1, -1], v[0]) and torch.equal(kc[0, 0], k[1])


def test_write_refusals(w12):
    kc, vc = (torch.zeros((4, 16, 2, 64), dtype=torch.int16, device="cuda") for _ in range(2))
    cache = w12.KVCache(kc, vc)
    k = torch.ones((3, 2, 64), dtype=torch.int16, device="cuda")
    with pytest.raises(ValueError):
        w12.kv_write(cache, k[:, :1], k[:, :1], i64([0]))
    with pytest.raises(ValueError):
        w12.kv_write(cache, k, k, i32([0]))
    with pytest.raises(ValueError):
        w12.kv_write(cache, k, k, i64([0, 1, 2, 3]))
    with pytest.raises(ValueError):
        w12.kv_write(cache, k, k, i64([0, 1]), src=i32([0]))
    with pytest.raises(w12.W12Error) as e:
        w12.kv_write(cache, k, k, i64([0]), layer=1)
    assert e.value.status == 2
    flat = torch.ones(3 * 2 * 64 + 4, dtype=torch.int16, device="cuda")
    with pytest.raises(w12.W12Error) as e:               # rows at 8 bytes
        w12.kv_write(cache, flat[4:].view(3, 2, 64), k, i64([0]))
    assert e.value.status == 1


# ---------------------------------------------------------------- slots again

_MANY = """
import sys, torch
import lossless_bit_weights_gb300 as w12
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
n = int(sys.argv[1])
table, pool = torch.zeros((n, 1), dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
pos = torch.tensor([0, n], dtype=torch.int64, device="cuda")
out = w12.kv_slots(i32([0] * n), i32([1] * n), table, pool, pos, 4, n)
assert int(out.status) == 0 and out.slot.tolist() == [4 * i for i in range(n)] and out.new_len.tolist() == [1] * n
"""


@pytest.mark.parametrize("n_req", [4079, 4080, 4095, 4096])
def test_any_number_of_requests_as_a_process_s_first_call(w12, n_req):
    """Shared memory beside the prefix sums counts too; a call of more requests before must not matter."""
    r = subprocess.run([sys.executable, "-c", _MANY, str(n_req)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("entry", [-1, -7, -2 ** 31])
def test_a_released_negative_entry_is_reported(w12, entry):
    table, ring, pos = i32([[0, 1], [2, entry]]), i32([3, 9, 9, 9]), i64([0, 1])
    out = w12.kv_slots(i32([8, 8]), i32([0, -1]), table, ring, pos, 4, 2)
    assert int(out.status) == 8
    assert int(out.total) == 0 and out.new_len.tolist() == [8, 0] and out.pool_pos.tolist() == [0, 3]
    assert ring.tolist() == [3, 2, entry, 9]
    # the request that takes it is told too, and its tokens have no place
    out = w12.kv_slots(out.new_len, i32([0, 9]), i32([[0, 1, 9], [9, 9, 9]]), ring, out.pool_pos, 4, 9)
    assert int(out.status) == 8 and out.slot.tolist() == [12, 13, 14, 15, 8, 9, 10, 11, -2]
