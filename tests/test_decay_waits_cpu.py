"""A model of the barrier that the eight W V warps of linear attention with a
decay meet at ahead of the chunk with tokens behind the end."""

import pytest


def arrivals(N, ragged, leaves, late):
    """How often each of eight warps arrives at the barrier when warp w's wait gives up at chunk leaves[w] (N: never)."""
    count = []
    for w in range(8):
        ok, meets, n, c = True, ragged >= 0, 0, 0
        while c < N and ok:
            ok = c != leaves[w]
            if c == ragged:
                meets, n = False, n + 1
                ok = ok and all(x > c for x in leaves)
            c += 1
        if late and meets:
            n += 1
        count.append(n)
    return count


@pytest.mark.parametrize("N", [1, 2, 4])
def test_all_meet(N):
    """The barrier ends whoever leaves when; without the late arrival it would not."""
    for ragged in range(-1, N):
        for w in (0, 5):
            for c in range(N + 1):
                leaves = [N] * 8
                leaves[w] = c
                assert len(set(arrivals(N, ragged, leaves, True))) == 1
                one_sided = len(set(arrivals(N, ragged, leaves, False))) > 1
                assert one_sided == (c < ragged)
