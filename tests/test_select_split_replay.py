"""A CPU replay of the group selection launch's work decomposition (groups.cu): index arithmetic only.

  * the groups of one CTA are the fewest multiple of what its threads hold in flight that leaves no
    more CTAs than the device holds at once (or all of the longest unit), found in a few steps;
  * every group of every unit that has more than n_select is scored by one CTA, and a unit's
    ticket counts the CTAs that have some;
  * scores, error scales and exact keys stay inside the unit's words of the scratch."""
import random

import pytest


def groups_per_cta(lengths, units, n_select, step, room):
    """The launch's choice, and how often it counted the CTAs."""
    most = max([n for n in lengths if n > n_select], default=0)
    counted = 0

    def ctas(per):
        nonlocal counted
        counted += 1
        return sum(units * ((n + per - 1) // per) for n in lengths if n > n_select)
    least, enough = 1, max(1, (most + step - 1) // step)
    while least < enough:
        m = least + (enough - least) // 2
        if ctas(step * m) <= room:
            enough = m
        else:
            least = m + 1
    return step * enough, most, counted


def plain_choice(lengths, units, n_select, step, room):
    most = max([n for n in lengths if n > n_select], default=0)
    per = step
    while per < most and sum(units * ((n + per - 1) // per) for n in lengths if n > n_select) > room:
        per += step
    return per


def check(lengths, units, n_select, step, n_sm):
    room = 2 * n_sm
    per, most, counted = groups_per_cta(lengths, units, n_select, step, room)
    assert per == plain_choice(lengths, units, n_select, step, room)
    assert counted <= max(1, most // step).bit_length() + 1
    blocks = max(1, (most + per - 1) // per)
    for n in lengths:
        if n <= n_select:
            continue                       # block 0 writes every index
        nblk = (n + per - 1) // per
        assert 1 <= nblk <= blocks
        scored = []
        for blk in range(blocks):
            if blk >= nblk:
                continue                   # leaves without a ticket
            first, end = blk * per, min(n, (blk + 1) * per)
            assert first < end
            scored.append((first, end))
        assert scored[0][0] == 0 and scored[-1][1] == n
        assert all(a[1] == b[0] for a, b in zip(scored, scored[1:]))
        # n 64-bit words per unit: n fp32 scores, then a scale per CTA; or n exact keys
        assert 4 * (n + nblk) <= 8 * n


@pytest.mark.parametrize("seed", range(4))
def test_random_launches(seed):
    rng = random.Random(seed)
    for _ in range(300):
        layers = rng.choice([1, 1, 2, 5, 64])
        lengths = [rng.choice([0, 1, 2, 17, rng.randint(1, 6000)]) for _ in range(layers)]
        check(lengths, rng.choice([1, 2, 8, 40, 160, 500]), rng.choice([1, 7, 64, 5000]),
              rng.choice([64, 128]), rng.choice([1, 7, 148, 152]))


def test_the_cases():
    assert groups_per_cta([1024], 160, 64, 64, 304)[0] == 1024     # one CTA a unit
    assert groups_per_cta([4094], 8, 64, 64, 304)[0] == 128        # two steps of its threads
    assert groups_per_cta([15], 4, 4, 128, 304)[0] == 128
    assert groups_per_cta([], 8, 4, 64, 304)[:2] == (64, 0)
    # many units of long caches in many layers: counted a few times, not once for every step
    assert groups_per_cta([32768] * 64, 512, 64, 64, 304)[2] <= 10
