"""Chunk attention over numbers at the ends of their ranges, against 64-bit references (GPU)."""
import numpy as np
import pytest
import torch

from chunk_ref import bf16
from test_gpu_chunk import FORMATS, Case, bits_of

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


def large(rng, shape):
    """Numbers whose sets have scales and zeros that are halves, and dequantized numbers that are not (up to 120000)."""
    return bits_of(rng.uniform(-20000.0, 120000.0, shape))


@pytest.mark.parametrize("fmt,G,R,paged", FORMATS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 130)])
@pytest.mark.parametrize("what", ["keys", "values", "both"])
def test_cached_numbers_past_halves(fmt, G, R, paged, window, sinks, what):
    """Packed tokens of every format beyond fp16's largest number, in clear tiles, at a window's edge and beside new ones."""
    case = Case(fmt, [700, 70, 0], [40, 3, 20], G=G, R=R, paged=paged, seed=220 + fmt)
    rng = np.random.default_rng(fmt + G)
    if what != "values":
        case.k = large(rng, case.k.shape)
        case.q = bits_of(bf16(case.q) * 2.0 ** -16)          # scores of ordinary size
    if what != "keys":
        case.v = large(rng, case.v.shape)
    if fmt == 8:
        amax = np.stack([np.abs(bf16(a)).max((0, 2)) for a in (case.k, case.v)]).astype(np.float32)
        case.cache.region("fp8_scale").view(torch.float32).copy_(torch.from_numpy((amax / np.float32(448)).ravel()))
    case.fill()
    case.check(case.attend(window=window, sinks=sinks), window, sinks)
    assert case.cache.error() == 0


@pytest.mark.parametrize("fmt,G", [(2, 32), (4, 32), (6, 32), (16, 32)])
@pytest.mark.parametrize("far", ["key", "value"])
def test_one_far_token_among_ordinary_ones(fmt, G, far):
    """A run of ordinary pieces broken by one whose numbers do not fit: each piece keeps its own scaling."""
    case = Case(fmt, [900], [9], G=G, R=0, seed=230 + fmt)
    rows = case.k if far == "key" else case.v
    rows[[40, 333, 513, 850], 1, 17] = bits_of(np.array([90000.0, 90000.0, 120000.0, 90000.0]))
    if far == "key":
        case.q[:, :, 17] = 0                                  # (the far channel must not decide every weight)
    case.fill()
    case.check(case.attend())
    case.check(case.attend(splits=3, window=700, sinks=20), 700, 20)
