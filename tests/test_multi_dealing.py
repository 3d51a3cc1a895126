"""The dealing rule of the multi-token attention (tests/multi_dealing.py) over
random batches: every tile in one segment, every join entry in its list and
every state that a join reads written."""
import random

import pytest

from multi_dealing import Dealing


@pytest.mark.parametrize("seed", range(20))
def test_dealing_covers_every_tile_and_entry(seed):
    r = random.Random(seed)
    for _ in range(10):
        B = r.choice([1, 2, 5, 40, 70])
        n = [r.choice([0, 1, 5, 60, 100, 300]) for _ in range(B)]
        n[r.randrange(B)] = 33
        T = [x + r.choice([0, 10, 2000, 9000]) for x in n]
        if r.random() < 0.2:
            T[0] = max(1, n[0] - 20)  # fewer rows than new tokens
        Dealing(n, T, r.choice([1, 2, 8]), r.choice([1, 4, 16]), r.random() < 0.5, ctas=r.choice([148, 7])).check()
