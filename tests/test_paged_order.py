"""The order of events inside the chunk kernel for quantised caches, on the host: which slots of
the ring of tile scales may be rewritten while a softmax warpgroup has still to read them."""
import os
import re

import numpy as np
import pytest

import io_aware_exact_07_gb300 as fa

CSRC = os.path.join(os.path.dirname(os.path.abspath(fa.__file__)), "csrc")


def unread_distances(pieces, k_stages, queries=False):
    """For every key tile n of a CTA's pieces (lists of tile counts), how far back the oldest
    tile lies that no wait orders before the write of tile n's scales; or, for every piece, how
    far back the oldest one whose query exponents (which a warpgroup reads with its first tile)
    may be unread when the piece's are written, after the S products of the piece before. Events,
    as the sets of tiles whose scales have been read (bits) when they happen:
      S(n), issued in order, after the softmax warpgroup that it is for (the tile's place in its
        piece, mod 2) has read its last tile;
      read(n), by that warpgroup, after S(n) and what it did before;
      a piece's end, for either warpgroup, after both have read all of theirs in it;
      the write of tile n's scales, after S(n - k_stages) has completed."""
    s, group, last_read = [], [0, 0], [None, None]
    worst, n, first = 0, 0, []
    for i, tiles in enumerate(pieces):
        if queries and s:
            unread = [k for k, ts in enumerate(first) if any(not s[-1] >> t & 1 for t in ts)]
            worst = max([worst] + [i - k for k in unread])
        first.append([n + p for p in range(min(tiles, 2))])
        for p in range(tiles):
            g = p & 1
            before = s[-1] if s else 0
            if last_read[g] is not None:
                before |= last_read[g]
            s.append(before)
            group[g] |= before | (1 << n)
            last_read[g] = group[g]
            done = s[n - k_stages] if n >= k_stages else 0
            unread = [t for t in range(n) if not done >> t & 1]
            if unread and not queries:
                worst = max(worst, n - unread[0])
            n += 1
        group = [group[0] | group[1]] * 2  # the exchange at the piece's end
    return worst


def constant(name):
    """The value that fa_paged_chunk.cu gives a ring's depth for a quantised cache."""
    text = open(os.path.join(CSRC, "fa_paged_chunk.cu")).read()
    expr = re.search(rf"constexpr int {name} = ([^;]*);", text).group(1)
    return int(re.fullmatch(r"E4M3 \? (\d+) : 0|D == 64 && !E4M3 \? 4 : (\d+)", expr)[
        1 if expr.startswith("E4M3") else 2])


def test_a_tiles_scales_are_not_rewritten_before_they_are_read():
    rng = np.random.RandomState(0)
    batches = [[3, 1], [2, 3, 2], [1] * 20, [2] + [1] * 9, [5, 4, 3, 2, 1] * 3]
    batches += [list(rng.randint(1, 8, 12)) for _ in range(200)]
    stages = constant("kKStages")
    worst = max(unread_distances(b, stages) for b in batches)
    # four slots would not do: the latest tile of one warpgroup may be unread when the other has
    # ended one piece and begun the next
    assert worst == stages + 2 == 4
    assert constant("kScaleSlots") > worst
    assert constant("kQExpSlots") > max(unread_distances(b, stages, True) for b in batches) == 2


@pytest.mark.parametrize("pieces,distance", [([8], 3), ([3, 3], 4), ([4, 4], 3), ([1, 1, 1, 1], 2)])
def test_where_a_piece_of_an_odd_number_of_tiles_ends(pieces, distance):
    assert unread_distances(pieces, 2) == distance
