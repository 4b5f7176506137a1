"""Calls of the paged cache's attention, one for each way that it can be run.  A CPU test
checks that they cover every way the sizes of a call can choose, a GPU test runs them."""
import collections

import numpy as np

Case = collections.namedtuple("Case", "d page n_kv n_q batch held new limit window")

FRONT, BACK = 1, 2                       # rows of no sequence before and behind the call's


def table_cols(c):
    return c.limit // c.page + 2


def lengths(c):
    """Tokens that the sequences hold and, as the last of them, the call's: ragged, `held`
    at most, `new` on average (some sequences without any)."""
    rng = np.random.default_rng(c.held * 1000 + c.new)
    n = rng.multinomial(c.new * c.batch, np.full(c.batch, 1 / c.batch)) if c.batch > 1 else np.array([c.new])
    if c.batch > 2:
        n[1], n[2] = n[1] + n[2], 0
    held = rng.integers(c.held // 3, c.held + 1, c.batch)
    held[0] = c.held
    return np.maximum(held, n).tolist(), n.tolist()


def tokens(c):
    return sum(lengths(c)[1]) + FRONT + BACK


CASES = [
    Case(128, 64, 1, 8, 2, 200, 70, 256, 0),                   # rows<128, 4, 2>
    Case(128, 128, 2, 4, 2, 700, 70, 1024, 0),                 # rows<128, 4, 2>, join_rows<128>
    Case(128, 128, 1, 64, 8, 200, 70, 256, 0),                 # rows<128, 8, 2>
    Case(128, 128, 2, 4, 8, 700, 70, 8192, 0),                 # rows<128, 8, 2>, join_rows<128>
    Case(256, 64, 2, 16, 2, 200, 70, 256, 0),                  # rows<256, 8, 1>
    Case(256, 64, 2, 4, 2, 700, 70, 1024, 0),                  # rows<256, 8, 1>, join_rows<256>
    Case(64, 64, 2, 16, 2, 200, 70, 256, 0),                   # rows<64, 4, 2>
    Case(64, 64, 2, 4, 2, 700, 70, 1024, 0),                   # rows<64, 4, 2>, join_rows<64>
    Case(64, 64, 1, 64, 8, 200, 70, 256, 0),                   # rows<64, 8, 2>
    Case(64, 64, 2, 4, 8, 700, 70, 8192, 0),                   # rows<64, 8, 2>, join_rows<64>
    Case(96, 64, 2, 4, 5, 200, 70, 256, 0),                    # rows<96, 4, 2>
    Case(96, 64, 2, 4, 2, 700, 70, 1024, 0),                   # rows<96, 4, 2>, join_rows<96>
    Case(96, 64, 1, 64, 8, 200, 70, 256, 0),                   # rows<96, 8, 2>
    Case(96, 64, 2, 4, 8, 700, 70, 8192, 0),                   # rows<96, 8, 2>, join_rows<96>
    Case(128, 128, 8, 8, 5, 700, 1, 1024, 0),                  # split<128, 1, 2>, join<128, 1, 1>
    Case(128, 128, 2, 4, 2, 700, 1, 1024, 0),                  # split<128, 1, 2>, join<128, 1, 4>
    Case(128, 64, 2, 4, 2, 330, 1, 512, 0),                    # split<128, 1, 2>, whole row blocks
    Case(128, 128, 3, 21, 8, 700, 2, 1024, 0),                 # split<128, 2, 1>, join<128, 2, 1>
    Case(128, 128, 1, 8, 2, 700, 1, 1024, 0),                  # split<128, 2, 1>, join<128, 2, 4>
    Case(128, 128, 1, 8, 2, 200, 1, 256, 0),                   # split<128, 2, 1>, whole row blocks
    Case(128, 128, 3, 21, 8, 700, 5, 1024, 0),                 # split<128, 3, 1>, join<128, 3, 1>
    Case(128, 128, 1, 8, 2, 700, 3, 1024, 0),                  # split<128, 3, 1>, join<128, 3, 4>
    Case(128, 128, 1, 8, 2, 200, 3, 256, 0),                   # split<128, 3, 1>, whole row blocks
    Case(256, 64, 8, 8, 3, 700, 1, 1024, 0),                   # split<256, 1, 1>, join<256, 1, 1>
    Case(256, 64, 2, 4, 2, 700, 1, 1024, 0),                   # split<256, 1, 1>, join<256, 1, 4>
    Case(256, 64, 2, 4, 2, 200, 1, 256, 0),                    # split<256, 1, 1>, whole row blocks
    Case(64, 64, 8, 8, 5, 700, 1, 1024, 0),                    # split<64, 1, 2>, join<64, 1, 1>
    Case(64, 64, 2, 4, 2, 700, 1, 1024, 0),                    # split<64, 1, 2>, join<64, 1, 4>
    Case(64, 64, 1, 8, 3, 330, 1, 512, 0),                     # split<64, 1, 2>, whole row blocks
    Case(64, 64, 1, 8, 40, 700, 2, 1024, 0),                   # split<64, 2, 2>, join<64, 2, 1>
    Case(64, 64, 1, 8, 2, 700, 1, 1024, 0),                    # split<64, 2, 2>, join<64, 2, 4>
    Case(64, 64, 1, 8, 2, 330, 1, 512, 0),                     # split<64, 2, 2>, whole row blocks
    Case(64, 64, 3, 21, 8, 700, 5, 1024, 0),                   # split<64, 3, 1>, join<64, 3, 1>
    Case(64, 64, 1, 8, 2, 700, 3, 1024, 0),                    # split<64, 3, 1>, join<64, 3, 4>
    Case(64, 64, 16, 80, 8, 330, 6, 512, 0),                   # split<64, 3, 1>, whole row blocks
    Case(96, 64, 8, 8, 5, 700, 1, 1024, 0),                    # split<96, 1, 2>, join<96, 1, 1>
    Case(96, 64, 2, 4, 2, 700, 1, 1024, 0),                    # split<96, 1, 2>, join<96, 1, 4>
    Case(96, 64, 2, 4, 2, 330, 1, 512, 0),                     # split<96, 1, 2>, whole row blocks
    Case(96, 64, 3, 21, 8, 700, 2, 1024, 0),                   # split<96, 2, 1>, join<96, 2, 1>
    Case(96, 64, 1, 8, 2, 700, 1, 1024, 0),                    # split<96, 2, 1>, join<96, 2, 4>
    Case(96, 64, 3, 21, 40, 330, 2, 512, 0),                   # split<96, 2, 1>, whole row blocks
    Case(96, 64, 3, 21, 8, 700, 5, 1024, 0),                   # split<96, 3, 1>, join<96, 3, 1>
    Case(96, 64, 1, 8, 2, 700, 3, 1024, 0),                    # split<96, 3, 1>, join<96, 3, 4>
    Case(96, 64, 1, 8, 2, 200, 3, 256, 0),                     # split<96, 3, 1>, whole row blocks
    Case(128, 128, 8, 8, 140, 200, 1, 256, 0),                 # wave<128, 1, 2>
    Case(128, 64, 16, 80, 40, 200, 3, 256, 0),                 # wave<128, 2, 1>
    Case(128, 64, 16, 80, 40, 200, 6, 256, 0),                 # wave<128, 3, 1>
    Case(256, 64, 8, 8, 70, 200, 1, 256, 150),                 # wave<256, 1, 1>
    Case(64, 64, 8, 8, 140, 200, 1, 256, 0),                   # wave<64, 1, 2>
    Case(64, 64, 16, 80, 70, 200, 3, 256, 0),                  # wave<64, 2, 2>
    Case(64, 64, 16, 80, 40, 200, 6, 256, 0),                  # wave<64, 3, 1>
    Case(96, 64, 8, 8, 140, 200, 1, 256, 0),                   # wave<96, 1, 2>
    Case(96, 64, 16, 80, 40, 200, 3, 256, 0),                  # wave<96, 2, 1>
    Case(96, 64, 16, 80, 40, 200, 6, 256, 0),                  # wave<96, 3, 1>
    # five drafted tokens of 64 heads on 8, behind a table of 4096 tokens
    Case(128, 128, 8, 64, 4, 2300, 5, 4096, 0),
]
