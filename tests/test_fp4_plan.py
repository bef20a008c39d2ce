"""The 4-bit decode's plan, restated from its kernel's arithmetic: every page
is covered once, a piece's row of partials is its own, and the combine finds
the rows that were written."""
import random

import pytest

MIN_PART = 4


def spans(lens, window, cap):
    """Attended pages (first, count) of each sequence."""
    out = []
    for n in lens:
        n = min(max(n, 0), cap * 16)
        lo = n - window if window > 0 and n > window else 0
        out.append((lo // 16, (n + 15) // 16 - lo // 16))
    return out


def pieces(sp, heads, parts):
    """(part, sequence, head, first page, count) as the CTAs walk them."""
    total = sum(n for _, n in sp)
    chunk = max(MIN_PART, (total * heads + parts - 1) // parts)
    prefix = [0]
    for _, n in sp:
        prefix.append(prefix[-1] + n)
    for part in range(parts):
        pos, end = part * chunk, min(total * heads, (part + 1) * chunk)
        b = next((i for i in range(len(sp)) if pos < prefix[i + 1] * heads), None)
        while pos < end:
            if sp[b][1] == 0:
                b += 1
                continue
            within = pos - prefix[b] * heads
            h, pg = divmod(within, sp[b][1])
            n = min(end - pos, sp[b][1] - pg)
            yield part, b, h, pg, n
            pos += n
            if within + n == sp[b][1] * heads:
                b += 1


@pytest.mark.parametrize("seed", range(300))
def test_plan(seed):
    rng = random.Random(seed)
    B, heads, sms = rng.choice([1, 2, 7, 60]), rng.choice([1, 2, 8]), rng.choice([1, 3, 152])
    cap = rng.choice([1, 5, 100])
    lens = [rng.choice([0, 1, 16, 17, rng.randint(0, cap * 16)]) for _ in range(B)]
    window = rng.choice([-1, -1, 1, 40, 500])
    parts = min(4 * sms, (B * heads * cap + MIN_PART - 1) // MIN_PART)
    rows = parts + B * heads
    sp = spans(lens, window, cap)
    covered, ids, direct = set(), {}, set()
    for part, b, h, pg, n in pieces(sp, heads, parts):
        for x in range(pg, pg + n):
            assert (b, h, x) not in covered
            covered.add((b, h, x))
        if n == sp[b][1]:
            direct.add((b, h))
            continue
        at = part + b * heads + h
        assert at not in ids and 0 <= at < rows
        ids[at] = (b, h)
    assert len(covered) == heads * sum(n for _, n in sp)
    # the combine
    total = sum(n for _, n in sp)
    chunk = max(MIN_PART, (total * heads + parts - 1) // parts)
    before = 0
    for b, (_, n) in enumerate(sp):
        for h in range(heads if n else 0):
            x = before * heads + h * n
            first, last = x // chunk, (x + n - 1) // chunk
            if first == last:
                assert (b, h) in direct
                continue
            assert last < parts
            for part in range(first, last + 1):
                assert ids.pop(part + b * heads + h) == (b, h)
        before += n
    assert not ids
