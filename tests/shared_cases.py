"""Calls of the paged cache's attention whose sequences share their first pages, one for
each way that they can be run; a CPU test checks that they cover every way, GPU tests run them."""
import collections

import numpy as np

# groups: (shared pages, sequences) each; own: most tokens of a sequence's own; new: rows of a sequence
# on average; wide: columns of the block table beyond what is needed
Case = collections.namedtuple("Case", "d page n_kv n_q groups own new wide")


def lengths(c):
    """Tokens of their own and rows of the call, for each sequence."""
    rng = np.random.default_rng(c.own * 1000 + c.new + sum(n for _, n in c.groups))
    B = sum(n for _, n in c.groups)
    new = rng.multinomial(c.new * B, np.full(B, 1 / B)) if c.new > 1 else np.ones(B, int)
    own = rng.integers(0, c.own + 1, B)
    own[0] = c.own
    return np.maximum(own, new).tolist(), [int(n) for n in new]


def sizes(c):
    """(tokens, batch, table_cols, groups, max_pages) of the call."""
    own, new = lengths(c)
    most = max(1, *(p for p, _ in c.groups))
    cols = max(p + -(-o // c.page) for p, o in zip([p for p, n in c.groups for _ in range(n)], own)) + 1 + c.wide
    return sum(new), len(new), cols, len(c.groups), most


CASES = [
    Case(128, 64, 8, 8, ((3, 70),), 60, 1, 0),                        # <128, false, 2>, 1 cuts, 1 waves
    Case(128, 64, 8, 8, ((3, 70),), 60, 1, 8),                        # <128, false, 2>, 1 cuts, 2 waves
    Case(128, 64, 1, 8, ((3, 5),), 60, 1, 0),                         # <128, false, 2>, 1 cuts, 4 waves
    Case(128, 64, 8, 8, ((6, 260),), 60, 3, 0),                       # <128, true, 2>, 1 cuts, 1 waves
    Case(128, 64, 8, 16, ((12, 180),), 60, 1, 8),                     # <128, true, 2>, 1 cuts, 2 waves
    Case(128, 64, 1, 32, ((20, 180),), 60, 1, 8),                     # <128, true, 2>, 3 cuts, 4 waves
    Case(256, 64, 2, 8, ((3, 100),), 60, 1, 0),                       # <256, false, 1>, 1 cuts, 1 waves
    Case(256, 64, 2, 8, ((3, 100),), 60, 1, 8),                       # <256, false, 1>, 1 cuts, 2 waves
    Case(256, 64, 1, 8, ((3, 5),), 60, 1, 0),                         # <256, false, 1>, 1 cuts, 4 waves
    Case(64, 64, 8, 8, ((3, 100),), 60, 1, 0),                        # <64, false, 2>, 1 cuts, 1 waves
    Case(64, 64, 8, 8, ((3, 100),), 60, 1, 8),                        # <64, false, 2>, 1 cuts, 2 waves
    Case(64, 64, 1, 8, ((3, 5),), 60, 1, 0),                          # <64, false, 2>, 1 cuts, 4 waves
    Case(64, 64, 2, 16, ((6, 400),), 60, 3, 0),                       # <64, true, 2>, 1 cuts, 1 waves
    Case(64, 64, 4, 64, ((6, 260),), 60, 1, 8),                       # <64, true, 2>, 1 cuts, 2 waves
    Case(64, 64, 2, 32, ((12, 130),), 60, 3, 8),                      # <64, true, 2>, 1 cuts, 4 waves
    Case(96, 64, 8, 8, ((3, 70),), 60, 1, 0),                         # <96, false, 2>, 1 cuts, 1 waves
    Case(96, 64, 8, 8, ((3, 70),), 60, 1, 8),                         # <96, false, 2>, 1 cuts, 2 waves
    Case(96, 64, 1, 8, ((3, 5),), 60, 1, 0),                          # <96, false, 2>, 1 cuts, 4 waves
    Case(96, 64, 8, 8, ((6, 400),), 60, 3, 0),                        # <96, true, 2>, 1 cuts, 1 waves
    Case(96, 64, 2, 16, ((6, 180),), 60, 3, 8),                       # <96, true, 2>, 1 cuts, 2 waves
    Case(96, 64, 1, 32, ((6, 260),), 60, 1, 8),                       # <96, true, 2>, 1 cuts, 4 waves
    Case(256, 64, 4, 64, ((3, 260),), 60, 1, 0),                      # rows_kernel<256, 8, 1>, 1 cuts, 1 waves
    Case(256, 64, 4, 64, ((3, 260),), 60, 1, 8),                      # rows_kernel<256, 8, 1>, 1 cuts, 2 waves
    Case(256, 64, 2, 8, ((60, 70),), 60, 3, 0),                       # rows_kernel<256, 8, 1>, 8 cuts, 4 waves
    # tables much wider than the sequences, and sequences as long as theirs: chunks of own tokens
    Case(128, 128, 2, 8, ((3, 5),), 200, 1, 40),
    Case(64, 64, 1, 8, ((7, 20), (2, 3), (1, 1)), 2500, 1, 0),
    Case(256, 64, 2, 2, ((5, 4),), 3000, 3, 10),
    # several rows a sequence, pages of 256, one sequence, single rows, many groups
    Case(96, 64, 2, 8, ((4, 6), (5, 9)), 90, 5, 0),
    Case(128, 256, 1, 40, ((2, 9),), 300, 1, 3),
    Case(64, 64, 2, 2, ((1, 1),), 3, 1, 0),
    Case(128, 64, 2, 4, tuple((i % 4, 1 + i % 3) for i in range(1, 80)), 70, 1, 0),
    # more rows than that: as without shared pages
    Case(128, 128, 2, 16, ((4, 3),), 400, 60, 0),
]
