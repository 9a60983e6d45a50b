"""Pages and slots from lengths, on the GPU, against the definition in plain Python (whole numbers: all are equal)."""
import random

import pytest
import torch

import nucleus_token_sampler_gb300 as tps

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda:0"


class Plain:
    def __init__(self, table, length, free, count, page):
        self.table, self.length, self.free, self.page = [list(r) for r in table], list(length), list(free), page
        self.count = min(max(count, 0), len(self.free))

    def pages(self, n):
        return -(-n // self.page)

    def extend(self, new, tokens):
        width = len(self.table[0]) if self.table else 0
        slots, positions, cu, status = [-1] * tokens, [0] * tokens, [], []
        rows = asked = taken = 0
        count = self.count
        for b, n in enumerate(new):
            s = self.length[b]
            cu.append(min(rows, tokens))
            valid = s >= 0 and n >= 0 and s + n <= width * self.page
            need = self.pages(s + n) - self.pages(s) if valid else 0
            at, rows, asked = rows, rows + max(n, 0), asked + need
            if not valid or (n and rows > tokens):
                status.append(3)
            elif need and asked > count:
                status.append(5)
            else:
                status.append(0)
                for i in range(need):
                    self.table[b][self.pages(s) + i] = self.free[count - 1 - taken - i]
                taken += need
                for i in range(n):
                    slots[at + i] = self.table[b][(s + i) // self.page] * self.page + (s + i) % self.page
                    positions[at + i] = s + i
                self.length[b] = s + n
        cu.append(min(rows, tokens))
        self.count = count - taken
        return slots, positions, cu, status

    def trim(self, keep):
        width = len(self.table[0]) if self.table else 0
        back, status, asked = [], [], 0
        for b, k in enumerate(keep):
            s = self.length[b]
            valid = 0 <= k <= s <= width * self.page
            n = self.pages(s) - self.pages(k) if valid else 0
            asked += n
            if not valid:
                status.append(3)
            elif n and self.count + asked > len(self.free):
                status.append(5)
            else:
                status.append(0)
                back += self.table[b][self.pages(k):self.pages(s)]
                self.length[b] = k
        for p in reversed(back):
            self.free[self.count] = p
            self.count += 1
        return status


def _device(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _state(rng, B, width, page, most, spare, entries=None):
    """A consistent state: tables whose used entries are pages of their own, and a shuffled list of free ones."""
    length = [rng.randint(0, most) for _ in range(B)]
    need = sum(-(-n // page) for n in length)
    ids = list(range(need + spare))
    rng.shuffle(ids)
    table = [[-7] * width for _ in range(B)]
    for b in range(B):
        for i in range(-(-length[b] // page)):
            table[b][i] = ids.pop()
    free = ids + [-9] * (entries - len(ids) if entries else rng.randint(0, 20))
    return table, length, free, len(ids)


def _run(table, length, free, count, page, steps):
    """Extensions and trims on both sides: ("extend", lengths, rows) and ("trim", lengths)."""
    plain = Plain(table, length, free, count, page)
    B = len(length)
    t, s, f, c = _device(table).view(B, len(table[0]) if table else 0), _device(length), _device(free), _device([count])
    for kind, change, *rows in steps:
        st = torch.full((B,), 77, dtype=torch.int32, device=DEV)
        if kind == "extend":
            slots, positions, cu = tps.kv_extend(t, s, _device(change), f, c, page, rows[0], status=st)
            ws, wp, wc, wst = plain.extend(change, rows[0])
            assert slots.tolist() == ws and positions.tolist() == wp and cu.tolist() == wc
        else:
            tps.kv_trim(t, s, _device(change), f, c, page, status=st)
            wst = plain.trim(change)
        assert st.tolist() == wst
        assert s.tolist() == plain.length and c.tolist() == [plain.count] and f.tolist() == plain.free and t.tolist() == plain.table
    return plain


@pytest.mark.parametrize("B,most,grow,page", [(1, 0, 1, 16), (1, 5000, 3000, 64), (8, 100, 1, 16), (33, 500, 17, 32), (300, 40, 200, 256), (1024, 60, 5, 16),
                                              (1025, 30, 3, 16), (2500, 20, 40, 32)])
def test_grow_and_shrink(B, most, grow, page):
    rng = random.Random(B * page)
    width = -(-(most + 2 * grow) // page) + 1
    table, length, free, count = _state(rng, B, width, page, most, B * (2 * grow // page + 2))
    new = [[rng.randint(0, grow) for _ in range(B)] for _ in range(2)]
    after = [a + b for a, b in zip(length, new[0])]
    keep = [rng.randint(0, n) for n in after]
    _run(table, length, free, count, page, [("extend", new[0], sum(new[0])), ("trim", keep), ("extend", new[1], sum(new[1]) + rng.randint(0, 50)),
                                            ("trim", [0] * B)])


def test_a_trim_undoes_an_extension_entry_for_entry():
    rng = random.Random(4)
    table, length, free, count = _state(rng, 1500, 20, 16, 200, 9000)
    new = [rng.randint(0, 90) for _ in length]
    plain = _run(table, length, free, count, 16, [("extend", new, sum(new)), ("trim", length)])
    assert plain.free == free and plain.count == count and plain.length == length


@pytest.mark.parametrize("B", [7, 1030])
def test_too_few_pages_and_no_room_in_the_list(B):
    rng = random.Random(B)
    for spare in (0, 1, B // 2, 2 * B):
        table, length, free, count = _state(rng, B, 12, 16, 60, spare, entries=spare + 3)
        new = [rng.choice([0, 1, 16, 40, 100]) for _ in range(B)]
        small = [rng.randint(0, 3) for _ in range(B)]
        _run(table, length, free, count, 16, [("extend", new, sum(new)), ("extend", small, sum(small)), ("trim", [0] * B), ("extend", new, sum(new))])


@pytest.mark.parametrize("rows", [0, 1, 50, 20000])
def test_rows_that_do_not_suffice_and_rows_behind_the_last(rows):
    rng = random.Random(rows)
    table, length, free, count = _state(rng, 40, 30, 16, 100, 2000)
    new = [rng.choice([0, 3, 20]) for _ in length]
    _run(table, length, free, count, 16, [("extend", new, rows)])


@pytest.mark.parametrize("rows", [400, 40000])
def test_impossible_numbers(rows):
    big = 2 ** 31 - 1
    table = [[3 * b, 3 * b + 1, 3 * b + 2] for b in range(8)]
    length, free = [5, -1, 16, 48, 10, 49, 0, big], list(range(100, 140))
    new = [3, 2, -5, 1, big, 0, 48, 1]
    _run(table, length, free, 40, 16, [("extend", new, rows), ("trim", [9, 0, 4, 48, 11, 3, -2, 5])])
    for count in (-4, 1000):
        _run(table, length, free, count, 16, [("extend", [20, 0, 1, 0, 3, 0, 9, 0], rows), ("trim", [0] * 8)])


def test_no_sequences_no_tables_and_no_list():
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    c = _device([0])
    slots, positions, cu = tps.kv_extend(none.view(0, 4), none, none, none, c, 16, 5)
    assert slots.tolist() == [-1] * 5 and positions.tolist() == [0] * 5 and cu.tolist() == [0]
    tps.kv_trim(none.view(0, 4), none, none, none, c, 16)
    _run([[], []], [0, 0], [], 0, 16, [("extend", [0, 1], 3), ("trim", [0, 0])])


@pytest.mark.parametrize("B,width,page,most", [(1024, 32, 16, 300), (700, 50, 32, 900), (64, 600, 16, 5000), (1, 40000, 16, 600000), (300, 128, 64, 6000),
                                               (1024, 40, 16, 640)])
def test_trims_of_wide_tables(B, width, page, most):
    """Up to 1,024 sequences whose tables have 32,768 places or more share a cluster: no CTA may overwrite what another still reads."""
    assert B <= 1024 and B * width >= 32768 and most <= width * page
    rng = random.Random(B + width)
    table, length, free, count = _state(rng, B, width, page, most, 60, entries=B * (most // page + 1) + 60)
    keep = [rng.choice([0, n, n, rng.randint(0, n), max(0, n - 1)]) for n in length]
    _run(table, length, free, count, page, [("trim", keep), ("trim", [rng.randint(0, k) for k in keep]), ("trim", [0] * B), ("trim", [0] * B)])


@pytest.mark.parametrize("B,width", [(1024, 32), (40, 900)])
def test_trims_of_wide_tables_refused(B, width):
    """Impossible numbers, a list without room and one with room for some, in rows that are cut out of a wider table."""
    rng = random.Random(B)
    table, length, _, _ = _state(rng, B, width, 16, width * 16, 0)
    pages = sum(-(-n // 16) for n in length)
    keep = [rng.choice([0, 0, n, n // 2, n + 1, -1, -2 ** 31, 2 ** 31 - 1]) for n in length]
    for b in rng.sample(range(B), 9):
        length[b] = rng.choice([-1, width * 16 + 1, 2 ** 31 - 1, -2 ** 31])
    for room in (0, 1, pages // 7, pages // 2, pages + 5):
        for count in (0, 3, room + 9):
            plain = Plain(table, length, [-9] * (room + 3), count, 16)
            wide = torch.full((B, width + 6), -1, dtype=torch.int32, device=DEV)
            t = wide[:, 5:5 + width]
            t.copy_(_device(table))
            s, f, c, st = _device(length), _device([-9] * (room + 3)), _device([count]), torch.full((B,), 77, dtype=torch.int32, device=DEV)
            before = wide.clone()
            tps.kv_trim(t, s, _device(keep), f, c, 16, status=st)
            assert st.tolist() == plain.trim(keep)
            assert s.tolist() == plain.length and c.tolist() == [plain.count] and f.tolist() == plain.free and torch.equal(wide, before)


def test_trims_of_wide_tables_undo_extensions_in_graphs():
    """A captured extension and its trim, many times over: the list stays entry for entry."""
    rng = random.Random(5)
    table, length, free, count = _state(rng, 512, 80, 16, 900, 9000)
    t, s, f, c, new, keep = _device(table), _device(length), _device(free), _device([count]), _device([rng.randint(0, 90) for _ in length]), _device(length)
    want = [x.clone() for x in (s, f, c)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tps.kv_extend(t, s, new, f, c, 16, int(512 * 90))
        tps.kv_trim(t, s, keep, f, c, 16)
    for _ in range(200):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((s, f, c), want))
    held = torch.arange(80, device=DEV) < ((s + 15) // 16)[:, None]
    assert torch.equal(t[held], _device(table)[held])


def test_strided_tables_and_given_outputs():
    wide = torch.full((3, 10), -1, dtype=torch.int32, device=DEV)
    t, s, f, c = wide[:, 2:6], _device([0, 15, 20]), _device([9, 8, 7, 6]), _device([4])
    t[1, 0], t[2, 0], t[2, 1] = 3, 4, 5
    raw = torch.full((2 * 41 + 1,), 5, dtype=torch.int32, device=DEV)
    out = (torch.full((41,), 5, dtype=torch.int64, device=DEV), raw[1:42], torch.full((4,), 5, dtype=torch.int32, device=DEV))
    got = tps.kv_extend(t, s, _device([17, 2, 12]), f, c, 16, 41, out=out)
    assert got is out
    assert wide.tolist() == [[-1, -1, 6, 7, -1, -1, -1, -1, -1, -1], [-1, -1, 3, 8, -1, -1, -1, -1, -1, -1], [-1, -1, 4, 5, -1, -1, -1, -1, -1, -1]]
    assert out[0].tolist() == list(range(96, 112)) + [112] + [63, 128] + list(range(84, 96)) + [-1] * 10
    assert c.tolist() == [1] and s.tolist() == [17, 17, 32] and out[2].tolist() == [0, 17, 19, 31] and (raw[42:] == 5).all() and raw[0] == 5


def test_captured_steps_on_a_stream_of_their_own():
    rng = random.Random(11)
    for rows in (300, 30000):
        table, length, free, count = _state(rng, 60, 40, 16, 200, 3000)
        t, s, f, c, new = _device(table), _device(length), _device(free), _device([count]), _device([5] * 60)
        plain = Plain(table, length, free, count, 16)
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g):
            slots, positions, cu = tps.kv_extend(t, s, new, f, c, 16, rows)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(4):
                g.replay()
        side.synchronize()
        for _ in range(4):
            want = plain.extend([5] * 60, rows)
        assert slots.tolist() == want[0] and positions.tolist() == want[1] and cu.tolist() == want[2]
        assert s.tolist() == plain.length and c.tolist() == [plain.count] and t.tolist() == plain.table
        tps.kv_trim(t, s, _device([0] * 60), f, c, 16, stream=side)
        side.synchronize()
        plain.trim([0] * 60)
        assert f.tolist() == plain.free and c.tolist() == [plain.count]


def test_refusals():
    t, s, f, c = (torch.zeros(x, dtype=torch.int32, device=DEV) for x in ((2, 3), (2,), (4,), (1,)))
    for args in ((t.long(), s, s, f, c, 16, 5), (t.cpu(), s, s, f, c, 16, 5), (t.T, s, s, f, c, 16, 5), (t, s[:1], s, f, c, 16, 5), (t, s, s.long(), f, c, 16, 5),
                 (t, s, s, f.long(), c, 16, 5), (t, s, s, f, s, 16, 5), (t, s, s, f, c, 24, 5), (t, s, s, f, c, 16, -1), (t, s, s, f, c, 16, 2 ** 31),
                 (t[:1].expand(2, 3), s, s, f, c, 16, 5), (None, s, s, f, c, 16, 5)):
        with pytest.raises(ValueError):
            tps.kv_extend(*args)
        if args[-1] == 5:
            with pytest.raises(ValueError):
                tps.kv_trim(*args[:-1])
    with pytest.raises(ValueError):
        tps.kv_extend(t, s, s, f, c, 16, 5, out=(s, s, s))
    with pytest.raises(ValueError):
        tps.kv_extend(t, s, s, f, c, 16, 5, status=c)
