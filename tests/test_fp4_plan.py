"""The 4-bit decode's plan, restated from its kernel's arithmetic: every page
is covered once, a piece's row of partials is its own, and the combine finds
the rows that were written."""
import random

import pytest

MIN_PART = 2


def spans(lens, window, cap):
    """Attended pages (first, count) of each sequence."""
    out = []
    for n in lens:
        n = min(max(n, 0), cap * 16)
        lo = n - window if window > 0 and n > window else 0
        out.append((lo // 16, (n + 15) // 16 - lo // 16))
    return out


def pieces(sp, heads, parts):
    """(part, sequence, head, first page, count) as the warps walk them."""
    total = sum(n for _, n in sp)
    chunk = max(MIN_PART, ((total * heads + parts - 1) // parts + 1) // 2 * 2)
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
    cap = rng.choice([1, 5, 100, 1000])
    lens = [rng.choice([0, 1, 16, 17, rng.randint(0, cap * 16)]) for _ in range(B)]
    window = rng.choice([-1, -1, 1, 40, 500])
    parts = min(12 * sms, (B * heads * cap + MIN_PART - 1) // MIN_PART)
    rows = parts + B * heads
    sp = spans(lens, window, cap)
    total = heads * sum(n for _, n in sp)
    chunk = max(MIN_PART, ((total + parts - 1) // parts + 1) // 2 * 2)
    starts, x = {}, 0
    for b, (_, n) in enumerate(sp):
        for h in range(heads):
            starts[b, h] = x
            x += n

    def joined(part, b, h):
        """A warp's view, from the piece that its part begins with."""
        c0 = part // 4 * 4 * chunk
        c1 = min(total, c0 + 4 * chunk)
        return c1 - c0 > chunk and starts[b, h] <= c0 and c1 <= starts[b, h] + sp[b][1]

    covered, ids, direct, verdict = set(), {}, set(), {}
    for part, b, h, pg, n in pieces(sp, heads, parts):
        for x in range(pg, pg + n):
            assert (b, h, x) not in covered
            covered.add((b, h, x))
        if part not in [k[1] for k in verdict if k[0] == part // 4]:
            verdict[part // 4, part] = joined(part, b, h)
        if verdict[part // 4, part]:
            at = part // 4 * 4 + b * heads + h  # written once, by all of the CTA's warps
            assert ids.get(at, (b, h)) == (b, h)
            ids[at] = (b, h)
        elif n == sp[b][1]:
            direct.add((b, h))
        else:
            at = part + b * heads + h
            assert at not in ids and 0 <= at < rows
            ids[at] = (b, h)
    assert len(covered) == total
    for cta in {c for c, _ in verdict}:  # the warps of a CTA agree, and those without a part are not waited for
        views = [v for (c, _), v in verdict.items() if c == cta]
        assert len(set(views)) == 1
        if views[0]:
            assert len(views) == -(-(min(total, (cta + 1) * 4 * chunk) - cta * 4 * chunk) // chunk)
    # the combine
    for (b, h), x in starts.items():
        n = sp[b][1]
        if n == 0:
            continue
        first, last = x // chunk, (x + n - 1) // chunk
        if first == last:
            assert (b, h) in direct
            continue
        assert last < parts
        cta = 4 * chunk
        c0, c1 = -(-x // cta), (x + n) // cta
        if x + n == total and total % cta > chunk:
            c1 = total // cta + 1
        if c1 > c0:
            found = [*range(first, 4 * c0), *range(4 * c0, 4 * c1, 4), *range(4 * c1, last + 1)]
        else:
            found = list(range(first, last + 1))
        for part in found:
            assert ids.pop(part + b * heads + h) == (b, h)
    assert not ids
