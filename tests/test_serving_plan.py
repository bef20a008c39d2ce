"""CPU models of the shared-prefix kernels' index arithmetic and barriers."""
import random

import numpy as np

UNIT, TR, TK, UNIT_COST = 256, 128, 128, 16


def _groups(g, spans, lens):
    out = []
    for (a, b), L in zip(spans, lens):
        tiles, K = -(-(b - a) * g // TR), -(-L // TK)
        units = (tiles + 1) // 2
        out.append((a, b - a, tiles, K, units, tiles * K + units * UNIT_COST if tiles * K else 0))
    return out


def _prefix_plan(groups, slots):
    """What the kernel's walk gives each slot: (slot, unit) -> (group, unit in
    group, tiles, k0, k1); and the cut."""
    W = sum(x[5] for x in groups) - UNIT_COST
    used = max(0, min(W, slots))
    q = W // used if used else 0
    rem = W - q * used if used else 0

    def start(s):
        return UNIT_COST + s * q + min(s, rem)

    def slot_of(x):
        x -= UNIT_COST
        y = x - rem * (q + 1)
        return min(used - 1, x // (q + 1) if y < 0 else rem + y // q)

    segs = {}
    for s in range(used):
        pos, end = start(s), start(s + 1)
        gi = gstart = ubase = 0
        while pos < end and gi < len(groups):
            a, nb, tiles, K, units, cost = groups[gi]
            if pos >= gstart + cost:
                gstart, ubase, gi = gstart + cost, ubase + units, gi + 1
                continue
            u = (pos - gstart) // (2 * K + UNIT_COST)
            first = gstart + u * (2 * K + UNIT_COST) + UNIT_COST
            nq = min(2, tiles - 2 * u)
            stop = min(end, first + nq * K)
            if stop <= first:
                break
            pos = max(pos, first)
            k0, k1 = -(-(pos - first) // nq), -(-(stop - first) // nq)
            assert (s + ubase + u) not in segs
            segs[s + ubase + u] = (s, gi, u, nq, k0, k1)
            pos = stop
    return segs, slot_of


def test_prefix_plan_covers_every_tile_once_and_the_merge_finds_it():
    rng = random.Random(1)
    for _ in range(3000):
        g, G = rng.randint(1, 8), rng.randint(1, 5)
        cuts = sorted(rng.randint(0, 200) for _ in range(G + 1))
        spans = list(zip(cuts, cuts[1:]))
        lens = [rng.choice([0, rng.randint(1, 6000)]) for _ in range(G)]
        groups, slots = _groups(g, spans, lens), rng.randint(1, 152)
        if not sum(x[5] for x in groups):
            continue
        segs, slot_of = _prefix_plan(groups, slots)
        max_units = 200 * g // UNIT + G
        gstart = ubase = 0
        for gi, (a, nb, tiles, K, units, cost) in enumerate(groups):
            for u in range(units if cost else 0):
                nq = min(2, tiles - 2 * u)
                c0 = gstart + u * (2 * K + UNIT_COST) + UNIT_COST
                s0, s1 = slot_of(c0), slot_of(c0 + nq * K - 1)
                tiles_seen = []
                for s in range(s0, s1 + 1):  # every segment that the merge reads is written, and by this unit
                    assert segs[s + ubase + u][:4] == (s, gi, u, nq)
                    tiles_seen += range(*segs[s + ubase + u][4:])
                assert tiles_seen == list(range(K))
                assert ubase + u < max_units
            gstart, ubase = gstart + cost, ubase + units


def _w(x):
    """x as a 32-bit integer wraps."""
    return (x + 2**31) % 2**32 - 2**31


def _div(a, b):
    """C's division (toward zero); a division by zero gives some value."""
    return (abs(a) // abs(b)) * (1 if (a < 0) == (b < 0) else -1) if b else -1


def test_a_wrapped_plan_stays_in_bounds():
    """Overlapping groups (reported as faulty) can push the summed cost past 32
    bits; no segment and no merge entry may then leave its arrays."""
    rng = random.Random(3)
    for _ in range(20000):
        max_units, slots = rng.randint(1, 4000), rng.randint(1, 152)
        tiles, K = rng.randint(1, 4000), rng.randint(1, 1 << 20)
        nb_rows = rng.randint((tiles - 1) * TR + 1, tiles * TR)
        W = rng.choice([_w(rng.getrandbits(32)), rng.randint(-40, 40), 2**31 - 1 - rng.randint(0, 40)])
        gstart, ubase = _w(rng.getrandbits(32)), rng.choice([rng.randint(0, 4000), _w(rng.getrandbits(32))])
        w = _w(W - UNIT_COST)
        used = max(0, min(w, slots))
        q = w // used if used else 0
        rem = w - q * used if used else 0

        def slot_of(x):
            x = _w(x - UNIT_COST)
            y = _w(x - _w(rem * _w(q + 1)))
            return max(0, min(used - 1, _div(x, _w(q + 1)) if y < 0 else _w(rem + _div(y, q))))

        units = (tiles + 1) // 2
        # the merge table's entry of a row of the group
        un = rng.randint(0, nb_rows - 1) // UNIT
        if 0 <= _w(ubase + un) < max_units:
            c0 = _w(gstart + _w(un * (2 * K + UNIT_COST)) + UNIT_COST)
            s0 = slot_of(c0)
            ns = max(1, slot_of(_w(c0 + min(2, tiles - 2 * un) * K - 1)) - s0 + 1)
            assert 0 <= s0 and s0 + ns <= slots and 0 <= _w(ubase + un) + s0 + ns - 1 < slots + max_units
        # a step of a slot's walk
        slot = rng.randint(0, slots - 1)
        if slot >= used:
            continue
        pos = _w(UNIT_COST + _w(slot * q) + min(slot, rem))
        end = _w(UNIT_COST + _w((slot + 1) * q) + min(slot + 1, rem))
        cost = _w(tiles * K + units * UNIT_COST)
        if pos >= end or pos >= _w(gstart + cost):
            continue
        u = 0
        if _w(pos - gstart) >= 2 * K + UNIT_COST:
            u = _w((_w(pos - gstart) % 2**32) // (2 * K + UNIT_COST))
        first = _w(gstart + _w(u * (2 * K + UNIT_COST)) + UNIT_COST)
        nq = min(2, _w(tiles - _w(2 * u)))
        stop = min(end, _w(first + _w(nq * K)))
        if stop <= first or u < 0 or u >= units:
            continue
        pos = max(pos, first)
        k0, k1 = ((_w(_w(x - first) + 1) >> 1) if nq == 2 else _w(x - first) for x in (pos, stop))
        unit = _w(ubase + u)
        if not (k0 >= 0 and k1 >= k0 and k1 <= K and 0 <= unit < max_units):
            continue
        assert nq in (1, 2) and 0 <= k0 <= k1 <= K and 0 <= slot + unit < slots + max_units
        assert 0 < min(UNIT, nb_rows - u * UNIT)  # its rows are the group's


def test_wide_plan_covers_every_page_once():
    """The own tokens' plan: slots of the batch's pages laid end to end."""
    rng = random.Random(2)
    for _ in range(3000):
        B, hi = rng.randint(1, 256), rng.choice([1, 16, 50, 2000])
        pages = np.array([rng.choice([0, -(-rng.randint(0, hi) // 16)]) for _ in range(B)])
        T, slots = int(pages.sum()), rng.randint(1, 152)
        if not T:
            continue
        N = min(slots, max(-(-T // 4), min(B, T)))
        starts = np.concatenate([[0], np.cumsum(pages)])
        per = -(-B // 32)
        lanes = np.add.reduceat(np.concatenate([pages, np.zeros(32 * per - B, int)]), np.arange(0, 32 * per, per))
        incl = np.cumsum(lanes)
        written, cover = {}, np.zeros(T, int)
        for slot in range(N):
            pos, end = slot * T // N, (slot + 1) * T // N
            at = int((incl <= pos).sum())
            b, start = at * per, int(incl[at] - lanes[at])
            x = np.cumsum(pages[b:b + per])
            skip = int((start + x <= pos).sum())
            start, b = start + (int(x[skip - 1]) if skip else 0), b + skip
            assert start == starts[b]
            while pos < end:
                if start + pages[b] <= pos:
                    start, b = start + pages[b], b + 1
                    continue
                stop = min(end, start + pages[b])
                cover[pos:stop] += 1
                assert slot + b not in written
                written[slot + b] = b
                pos = stop
        assert (cover == 1).all()
        for b in range(B):
            if pages[b]:
                s0, s1 = (-(-(x + 1) * N // T) - 1 for x in (int(starts[b]), int(starts[b + 1]) - 1))
                assert all(written[s + b] == b for s in range(s0, s1 + 1))
                assert sum(v == b for v in written.values()) == s1 - s0 + 1


class _Bar:
    """An mbarrier: `count` arrivals complete a phase; a parity wait passes when
    the phase of that parity is the last complete one."""

    def __init__(self, count):
        self.count, self.n, self.phase = count, 0, 0

    def arrive(self):
        self.n += 1
        if self.n == self.count:
            self.n, self.phase = 0, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != (parity & 1)


def _run_pipeline(segs, stages, seed):
    """The prefix kernel's roles as coroutines under a random schedule: every
    stream consumes its own tiles in order, from stages that still hold them,
    and nothing waits forever."""
    rng = random.Random(seed)
    kf, vf = ([_Bar(1) for _ in range(stages)] for _ in range(2))
    ke, ve = [_Bar(2) for _ in range(stages)], [_Bar(1) for _ in range(stages)]
    hf, he = [_Bar(1), _Bar(1)], [_Bar(2), _Bar(2)]
    qf, sf, of, turn = ([_Bar(1), _Bar(1)] for _ in range(4))
    pf = [[_Bar(1), _Bar(1)] for _ in range(2)]
    kd, vd, hd = [None] * stages, [None] * stages, [None, None]
    total, done = sum(n for n, _ in segs), {0: [], 1: []}

    def producer(full, empty, data):
        for it in range(total):
            st = it % stages
            while not empty[st].passed(it // stages + 1):
                yield
            data[st] = it
            yield
            full[st].arrive()

    def converter():
        for it in range(total):
            st = it % stages
            while not vf[st].passed(it // stages) or not he[it & 1].passed((it >> 1) + 1):
                yield
            assert vd[st] == it
            hd[it & 1] = it
            yield
            ve[st].arrive()
            hf[it & 1].arrive()

    def issuer(x):
        tile0 = seen = kn = vn = rnd = queries = 0
        for n, pair in segs:
            cnt = n if pair else (n + 1 - x) // 2

            def tile(j):
                return tile0 + (j if pair else 2 * j + x)

            def pass_k(upto):
                nonlocal kn
                while kn < upto:
                    while not kf[kn % stages].passed(kn // stages):
                        yield
                    ke[kn % stages].arrive()
                    kn += 1

            def pass_v(upto):
                nonlocal vn
                while vn < upto:
                    while not hf[vn & 1].passed(vn >> 1):
                        yield
                    he[vn & 1].arrive()
                    vn += 1

            def scores(j):
                nonlocal kn
                t = tile(j)
                yield from pass_k(t)
                while not kf[t % stages].passed(t // stages):
                    yield
                kn += 1
                for _ in range(rng.randint(0, 5)):
                    yield
                assert kd[t % stages] == t
                sf[x].arrive()
                ke[t % stages].arrive()

            if cnt:
                while not qf[x].passed(queries):
                    yield
                queries += 1
                yield from scores(0)
            for j in range(n if pair else (n + 1) // 2):
                if x == 1:
                    while not turn[rnd & 1].passed(rnd >> 1):
                        yield
                if j < cnt:
                    t = tile(j)
                    yield from pass_v(t)
                    while not hf[t & 1].passed(t >> 1):
                        yield
                    vn += 1
                    for h in range(2):
                        while not pf[x][h].passed(seen):
                            yield
                    seen += 1
                    for _ in range(rng.randint(0, 5)):
                        yield
                    assert hd[t & 1] == t
                    done[x].append(t)
                    he[t & 1].arrive()
                    if j == cnt - 1:
                        of[x].arrive()
                    if j + 1 < cnt:
                        yield from scores(j + 1)
                if x == 0:
                    turn[rnd & 1].arrive()
                rnd += 1
            yield from pass_k(tile0 + n)
            yield from pass_v(tile0 + n)
            tile0 += n

    def softmax(x):
        tiles = sums = 0
        for n, pair in segs:
            cnt = n if pair else (n + 1 - x) // 2
            if not cnt:
                continue
            qf[x].arrive()
            yield
            for _ in range(cnt):
                while not sf[x].passed(tiles):
                    yield
                tiles += 1
                for h in range(2):
                    for _ in range(rng.randint(0, 6)):
                        yield
                    pf[x][h].arrive()
            while not of[x].passed(sums):
                yield
            sums += 1

    roles = [producer(kf, ke, kd), producer(vf, ve, vd), converter(), issuer(0), issuer(1), softmax(0), softmax(1)]
    pace = [rng.random() ** 2 + 0.01 for _ in roles]
    live, steps = list(range(len(roles))), 0
    while live:
        i = rng.choices(live, [pace[j] for j in live])[0]
        try:
            next(roles[i])
        except StopIteration:
            live.remove(i)
        steps += 1
        assert steps < 500_000, "a wait that nothing ends"
    for x in (0, 1):
        at, want = 0, []
        for n, pair in segs:
            want += [at + i for i in range(n) if pair or i % 2 == x]
            at += n
        assert done[x] == want


def test_prefix_pipeline_barriers():
    for seed in range(250):
        rng = random.Random(seed)
        _run_pipeline([(rng.randint(0, 8), rng.random() < 0.5) for _ in range(rng.randint(1, 5))], rng.choice([3, 6]), seed)
