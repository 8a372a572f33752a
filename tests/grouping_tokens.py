"""Tokens that fill single buckets of the grouping, over tables whose rows take one, two and three
digits to tell apart (not a test module)."""
import numpy as np

# 262144 is the largest table of one digit, 2^28 the largest of two
ROWS = [5000, 262144, 262145, 300000, 1 << 20, (1 << 28) + 1003]
KINDS = ["words", "crowd", "apart", "one", "edges"]


def tokens_of(kind, n, rows, seed):
    """words: as words are, the ids in order of frequency, a tenth padding; crowd: the first rows, alike;
    apart: rows whose low digits are alike, by turns; one: most of one row, others beside it; edges: about the
    borders of buckets and digits, and outside the table."""
    rng = np.random.default_rng([seed, rows])
    if kind == "words":
        t = np.minimum(np.exp(rng.random(n) * np.log(rows + 1.0)).astype(np.int64) - 1, rows - 1)
        return np.where(rng.random(n) < 0.1, -1, t)
    if kind == "crowd":
        return rng.integers(0, min(rows, 2000), n)
    if kind == "apart":
        some = np.array([0, 1, 1024, 1025, 2048, 2049, 1 << 20, (1 << 20) + 1, (1 << 20) + 1024])
        some = some[some < rows]
        return some[np.arange(n) % len(some)]
    if kind == "one":
        return np.where(rng.random(n) < 0.7, 3, rng.integers(0, min(rows, 4000), n))
    bits = max(0, int(rows - 1).bit_length() - 8)
    some = np.array([0, 1, (1 << bits) - 1, 1 << bits, (1 << bits) + 1, 1023, 1024, 1025, (1 << 20) - 1, 1 << 20, rows - 2,
                     rows - 1, rows, -1])
    return some[rng.integers(0, len(some), n)]
