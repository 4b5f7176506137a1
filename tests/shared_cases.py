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
    most = max(p for p, _ in c.groups)
    cols = max(p + -(-o // c.page) for p, o in zip([p for p, n in c.groups for _ in range(n)], own)) + 1 + c.wide
    return sum(new), len(new), cols, len(c.groups), most
