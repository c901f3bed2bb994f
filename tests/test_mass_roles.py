"""The barriers of the attention mass kernel (csrc/mass.cu), as a model on the
CPU: every warp or thread with a role of its own is a coroutine, and roles, copies
and tensor-core work proceed at random speeds. No barrier gets more arrivals than
it counts, what a role reads is what it means to read, and all roles end.

As in the kernel a wait names a parity only: it cannot tell a phase from the last
but one. A role that lets a phase go by unseen may read too early, and a ring
whose places are free before all have seen them may leave a role behind. The model
finds both: the last test plants them.
"""

import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_decoding_gb300", "csrc", "mass.cu")
GROUPS, AHEAD, INFO, Q_STAGES = 4, 8, 3, 2
STEPS = 400_000


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = self.tx = 0

    def arrive(self, n=1, tx=0):
        assert self.pending >= n, "more arrivals than counted"
        self.pending -= n
        self.land(-tx)

    def land(self, n):
        self.tx -= n
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def wait(self, parity):
        while (self.phase & 1) == parity:
            yield


class Ring:
    def __init__(self, at=0, round=0):
        self.at, self.round = at, round

    def next(self, n):
        self.at += 1
        if self.at == n:
            self.at, self.round = 0, self.round ^ 1

    def copy(self):
        return Ring(self.at, self.round)


class Item:
    def __init__(self, tiles, first, chunks, part):
        self.tiles, self.first, self.chunks, self.part = tiles, first, chunks, part
        self.again = self.keep = False


class Kernel:
    """form: "codes" (e4m3 rows go to the tensor cores as they are, two keys a thread),
    "convert" (e4m3, converted by the groups), "rows" (bf16)."""

    def __init__(self, items, form, stages, rng, see_all=True, hold=True):
        self.items, self.form, self.stages, self.rng = items, form, stages, rng
        self.see_all, self.hold = see_all, hold      # convert: groups see every stage; a stage is theirs until they have
        codes = form == "codes"
        self.tiles, self.slots = (8, 2) if codes else (4, 4)
        self.bf16_rows = not codes                   # query rows by TMA
        bars = lambda n, count: [Bar(count) for _ in range(n)]   # noqa: E731
        self.k_full = bars(stages, 1)
        self.k_empty = bars(stages, 2 + (4 * GROUPS if form == "convert" and see_all and hold else 0))
        self.q_full, self.q_empty = bars(Q_STAGES, 5 if self.bf16_rows else 4), bars(Q_STAGES, 2)
        self.n_full, self.n_empty = bars(INFO, 4), bars(INFO, 4 * GROUPS)
        self.slot_full, self.slot_empty = bars(self.slots, 33), bars(self.slots, 4 * GROUPS)
        self.c_full, self.c_read = bars(GROUPS, 4), bars(GROUPS, 4)
        self.s_full, self.s_empty = bars(self.tiles, 1), bars(self.tiles, 4)
        self.piece_full, self.piece_empty = bars(AHEAD, 1), bars(AHEAD, 1 + 2 + 4 + 4 * GROUPS)
        # what the shared memory holds: stages by tile and 32 rows, the others whole
        self.pieces, self.slot = [None] * AHEAD, [None] * self.slots
        self.k = [[[None] * 4, [None] * 4] for _ in range(stages)]
        self.q, self.numbers, self.scores = [None] * Q_STAGES, [None] * INFO, [None] * self.tiles
        self.flying, self.pipe, self.sums = [], [], 0

    # ---- work that lands some time
    def copies(self):
        while True:
            if self.flying:
                self.flying.pop(self.rng.randrange(len(self.flying)))()
            yield

    def tensor_cores(self):
        while True:
            if self.pipe:
                self.pipe.pop(0)()
            yield

    # ---- roles
    def piece(self, seg):
        yield from self.piece_full[seg % AHEAD].wait(seg // AHEAD & 1)
        return self.pieces[seg % AHEAD]

    def walker(self):
        for seg in range(len(self.items) + 1):
            if seg >= AHEAD:
                yield from self.piece_empty[seg % AHEAD].wait((seg // AHEAD - 1) & 1)
            self.pieces[seg % AHEAD] = (seg, self.items[seg]) if seg < len(self.items) else None
            self.piece_full[seg % AHEAD].arrive()
            yield

    def loader(self):
        k, sl = Ring(), Ring()

        def slots_land(at, seg, n):
            def land():
                self.slot[at] = seg
                self.slot_full[at].arrive(n)
            return land

        def tile_lands(at, half, what):
            def land():
                self.k[at][half] = [what + ("loaded",)] * 4
                self.k_full[at].land(1)
            return land

        p = yield from self.piece(0)
        while p:
            seg, item = p
            after = yield from self.piece(seg + 1)
            yield from self.slot_empty[sl.at].wait(sl.round ^ 1)
            self.flying += [slots_land(sl.at, seg, 8) for _ in range(4)]
            self.slot_full[sl.at].arrive()
            sl.next(self.slots)
            yield
            for j in range(0, item.tiles if item.first < item.chunks else 0, 2):
                yield from self.k_empty[k.at].wait(k.round ^ 1)
                self.k_full[k.at].arrive(tx=2)
                self.flying += [tile_lands(k.at, half, (seg, j + half)) for half in range(2)]
                k.next(self.stages)
                yield
            self.piece_empty[seg % AHEAD].arrive()
            p = after

    def mma(self, j):
        t, q, info = Ring(), Ring(), Ring()
        units, converted = [0] * (self.tiles // 2), [0] * (self.tiles // 2)
        seg = 0

        def multiply(tile, at, what, q_at, info_at, unit):
            def done():
                state = "rows" if self.form == "convert" else "loaded"
                assert self.k[at][j] == [what + (state,)] * 4, "tile of another item"
                assert self.q[q_at] == self.numbers[info_at], "rows of another chunk"
                self.scores[tile] = (what, self.q[q_at], unit)
            return done

        while True:
            p = yield from self.piece(seg)
            if not p:
                return
            _, item = p
            stage = t.copy()
            for c in range(item.first, item.chunks):
                if not item.again:
                    yield from self.q_full[q.at].wait(q.round)
                stage = t.copy()
                for s in range(self.tiles // 2):
                    if 2 * s >= item.tiles:
                        break
                    tile = 2 * s + j
                    if c == item.first:
                        yield from self.k_full[stage.at].wait(stage.round)
                    if tile < item.tiles:
                        if self.form == "convert" and c == item.first:
                            yield from self.c_full[tile].wait(converted[s] & 1)
                            converted[s] += 1
                        yield from self.s_empty[tile].wait(units[s] & 1 ^ 1)
                        units[s] += 1
                        self.pipe += [multiply(tile, stage.at, (seg, tile), q.at, info.at, c), self.s_full[tile].arrive]
                        yield
                    if c + 1 == item.chunks:
                        self.pipe.append(self.k_empty[stage.at].arrive)
                    stage.next(self.stages)
                if not item.keep:
                    self.pipe.append(self.q_empty[q.at].arrive)
                    q.next(Q_STAGES)
                    info.next(INFO)
                yield
            t = stage
            self.piece_empty[seg % AHEAD].arrive()
            seg += 1
            yield

    def rows(self, warp):
        q, info, seg = Ring(), Ring(), 0

        def rows_land(at, what):
            def land():
                self.q[at] = what
                self.q_full[at].land(1)
            return land

        while True:
            p = yield from self.piece(seg)
            if not p:
                return
            _, item = p
            for c in range(item.chunks if item.again else item.first, item.chunks):
                yield from self.q_empty[q.at].wait(q.round ^ 1)
                if self.bf16_rows and warp == 0:
                    self.q_full[q.at].arrive(tx=1)
                    self.flying.append(rows_land(q.at, (seg, c)))
                    yield
                yield from self.n_empty[info.at].wait(info.round ^ 1)
                self.numbers[info.at] = (seg, c)
                if not self.bf16_rows:
                    self.q[q.at] = (seg, c)
                yield
                self.n_full[info.at].arrive()
                self.q_full[q.at].arrive()
                q.next(Q_STAGES)
                info.next(INFO)
                yield
            self.piece_empty[seg % AHEAD].arrive()
            seg += 1
            yield

    def convert(self, g, quarter, seg, at, count):
        tile = self.k[at][g & 1]
        assert tile[quarter] == (seg, g, "loaded"), "codes of another item"
        yield
        self.c_read[g].arrive()
        yield from self.c_read[g].wait(count & 1)
        assert self.k[at][g & 1] is tile, "a load into rows that are converted"
        tile[quarter] = (seg, g, "rows")
        yield
        self.c_full[g].arrive()

    def group(self, g, quarter):
        info, sl, t = Ring(), Ring(), Ring()
        seg = converted = whose = 0
        units = [0] * self.tiles
        while True:
            p = yield from self.piece(seg)
            if not p:
                return
            _, item = p
            yield from self.slot_full[sl.at].wait(sl.round)
            assert self.slot[sl.at] == seg, "slots of another item"
            if self.form == "convert" and item.first < item.chunks:
                for s in range((item.tiles + 1) // 2):
                    own = s == g // 2 and g < item.tiles
                    if own or self.see_all:
                        yield from self.k_full[t.at].wait(t.round)
                    if self.see_all and self.hold:
                        self.k_empty[t.at].arrive()
                    if own:
                        yield from self.convert(g, quarter, seg, t.at, converted)
                        converted += 1
                    t.next(self.stages)
            if not item.again:
                whose = seg
            for c in range(item.first, item.chunks):
                mine = [x for x in range(g, self.tiles, GROUPS) if x < item.tiles]
                if not mine:
                    if not item.again:
                        yield from self.n_full[info.at].wait(info.round)
                else:
                    for x in mine:
                        yield from self.s_full[x].wait(units[x] & 1)
                        units[x] += 1
                    assert self.numbers[info.at] == (whose, c), "numbers of another chunk"
                    assert all(self.scores[x] == ((seg, x), (whose, c), c) for x in mine), "scores of another unit"
                    self.sums += 1
                    yield
                    for x in mine:
                        self.s_empty[x].arrive()
                if not item.keep:
                    self.n_empty[info.at].arrive()
                    info.next(INFO)
                yield
            assert self.slot[sl.at] == seg, "slots of another item"
            self.slot_empty[sl.at].arrive()
            sl.next(self.slots)
            self.piece_empty[seg % AHEAD].arrive()
            seg += 1
            yield

    def run(self):
        rng = self.rng
        work = [self.copies(), self.tensor_cores()]
        roles = [self.walker(), self.loader(), self.mma(0), self.mma(1)] + [self.rows(w) for w in range(4)] + \
                [self.group(g, w) for g in range(GROUPS) for w in range(4)]
        speed = [rng.random() ** 3 + 0.02 for _ in roles]
        lag = rng.choice([0.5, 0.15, 0.04])          # how soon copies land
        for _ in range(STEPS):
            if not roles:
                break
            if rng.random() < lag:
                next(work[0])
            if rng.random() < 0.5:
                next(work[1])
            k = rng.choices(range(len(roles)), speed)[0]
            try:
                next(roles[k])
            except StopIteration:
                del roles[k], speed[k]
        assert not roles, "roles that never end"
        while self.pipe:
            next(work[1])
        assert not self.flying
        return self.sums


def items(rng, form, count=20):
    """The items of a CTA: heads and requests of some items each, the last one of them not full."""
    full, out = 8 if form == "codes" else 4, []
    while len(out) < count:
        chunks = 1 if form == "codes" else rng.choice([1, 1, 1, 2, 3])
        run = rng.choice([1, 1, 2, 4])
        for part in range(run):
            last = part + 1 == run
            first = rng.randint(0, chunks) if last and rng.random() < 0.3 else 0
            out.append(Item(rng.choice([1, 2, 3, rng.randint(1, full)]) if last else full, first, chunks, part))
    for a, b in zip(out, out[1:]):
        a.keep = b.again = a.chunks == 1 and a.first == 0 and b.part == a.part + 1 and b.first == 0
    return out


@pytest.mark.parametrize("form,stages", [("codes", 4), ("codes", 6), ("convert", 2), ("convert", 5), ("rows", 2), ("rows", 5)])
def test_roles_read_what_they_mean_and_end(form, stages):
    rng = random.Random(f"{form}{stages}")
    for _ in range(25):
        work = items(rng, form)
        want = sum(4 * min(GROUPS, x.tiles) * (x.chunks - x.first) for x in work)
        assert Kernel(work, form, stages, rng).run() == want


@pytest.mark.parametrize("form", ["codes", "convert", "rows"])
def test_the_kernel_counts_as_the_model_does(form):
    inits = dict(re.findall(r"mbar_init\(&(\w+)\[s\], ([^;]+)\);", open(SOURCE).read()))
    model = Kernel([], form, 2, random.Random(0))
    assert len(inits) == 14
    for name, count in inits.items():
        count = re.sub(r"(\w+) \? (.+) : (.+)", r"(\2) if \1 else (\3)", count)
        assert eval(count, {"kGroups": GROUPS, "kCodes": form == "codes", "kConvert": form == "convert"}) == getattr(model, name)[0].count, name


@pytest.mark.parametrize("kw,what", [(dict(see_all=False), "codes of another item"), (dict(hold=False), "never end|another item|more arrivals")])
def test_the_model_finds_stages_that_go_by_unseen(kw, what):
    rng = random.Random(3)
    with pytest.raises(AssertionError, match=what):
        for _ in range(60):
            Kernel(items(rng, "convert"), "convert", 2, rng, **kw).run()
