"""What a draft token sees of an evicted shard, counted on the CPU: the batched
multi-query form is right for one shard, and over several each (request, query)
needs a length of its own.
"""
import numpy as np
import pytest


def _drafts(lens, kept, N, s, Q):
    """Positions of the rows a shard holds (the kept ones below the length, then the step's tokens that it owns)."""
    return [np.concatenate([kept[b], [t for t in range(L, L + Q) if t % N == s]]) for b, L in enumerate(lens)]


@pytest.mark.parametrize("Q", [1, 2, 3, 5])
@pytest.mark.parametrize("N", [1, 2, 3, 4])
def test_lengths_of_drafts_over_evicted_shards(N, Q):
    g = np.random.default_rng(N * 10 + Q)
    lens = [40, 41, 97, 130]
    wrong = 0
    for s in range(N):
        kept = [g.permutation(np.arange(s, L, N))[:12] for L in lens]      # any rows, in any order
        for b, pos in enumerate(_drafts(lens, kept, N, s, Q)):
            L, held = lens[b], len(kept[b])
            for i in range(Q):
                seen = np.nonzero(pos <= L + i)[0]
                own = sum(t % N == s for t in range(L, L + i + 1))
                assert np.array_equal(seen, np.arange(held + own))          # a length says it
                batched = max(0, len(pos) - (Q - 1 - i))
                wrong += batched != len(seen)
                assert N > 1 or batched == len(seen)
    assert (wrong > 0) == (N > 1 and Q > 1)
