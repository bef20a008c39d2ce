"""How the cache's writes and reads give tokens to tiles that follow the pages
(find_tokens), restated: each token to one tile, a page in order to one."""
import random

import pytest

P = 16


def tiles(slots):
    """The tokens of each aligned tile, as a warp finds them: its lanes look at 32
    tokens from 16 (tile - 1) on."""
    T = len(slots)
    out = []
    for tile in range((T - 1) // P + 2):
        mine = []
        for lane in range(32):
            t = P * (tile - 1) + lane
            if 0 <= t < T and slots[t] >= 0 and 0 <= lane - slots[t] % P < P:
                mine.append(t)
        out.append(mine)
    return out


@pytest.mark.parametrize("seed", range(200))
def test_every_token_once(seed):
    rng = random.Random(seed)
    T = rng.choice([1, 2, 15, 16, 17, 31, 33, 100, 257])
    kind = rng.choice(["any", "run", "sequences"])
    if kind == "any":
        slots = [rng.randrange(-2, 5000) for _ in range(T)]
    elif kind == "run":
        s = rng.randrange(0, 64)
        slots = list(range(s, s + T))
    else:
        slots = []
        while len(slots) < T:
            s = rng.randrange(0, 4000)
            slots += range(s, s + rng.randint(1, 50))
        slots = slots[:T]
    found = tiles(slots)
    assert sorted(t for tile in found for t in tile) == [t for t in range(T) if slots[t] >= 0]
    assert all(len(tile) <= 31 for tile in found)
    if kind == "run":  # every whole page is a tile of its own
        for t in range(T - P + 1):
            if slots[t] % P == 0:
                assert list(range(t, t + P)) in found
