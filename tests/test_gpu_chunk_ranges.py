"""Chunk attention over numbers at the ends of their ranges, against 64-bit references (GPU)."""
import numpy as np
import pytest

from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [4, 8, 16])
@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC0])
@pytest.mark.parametrize("where", ["key", "value"])
def test_non_finite_new_token_beside_cached_ones(fmt, bad, where):
    """One infinity or NaN in a new token that shares its 16-token piece with the cache's last tokens (70 = 4 * 16 + 6):
    rows before the token and the other head's rows are those of the reference, rows that see it are not finite."""
    case = Case(fmt, [70, 33], [40, 9], R=0, seed=200 + fmt).fill()
    for token in (5, 45):                        # positions 75 and 38: in pieces that start with cached tokens
        rows = case.kn if where == "key" else case.vn
        keep = rows[token, 1, 17]
        rows[token, 1, 17] = bad
        out = case.attend()
        rows[token, 1, 17] = keep
        last = 40 if token < 40 else 49          # rows [token, last) see it
        seen = out[token:last, 4:].copy()
        if where == "value" or bad == 0x7FC0:
            assert not np.any(np.isfinite(seen).all(-1))
        else:                                    # a score of -inf leaves the token out, one of +inf is not a number
            q = case.q[token:last, 4:, 17]
            up = ((q >> 15) == (bad >> 15)) & ((q & 0x7FFF) != 0)
            assert not np.any(np.isfinite(seen[up]))
        out[token:last, 4:] = case.attend()[token:last, 4:]
        case.check(out)
    assert case.cache.error() == 0
