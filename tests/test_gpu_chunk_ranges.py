"""Chunk attention over numbers at the ends of their ranges, against 64-bit references (GPU)."""
import numpy as np
import pytest
import torch

from bit_kv_cache_16_b200 import kvq
from chunk_ref import attend, bf16, cached_rows
from gpu_harness import to_dev
from layout import GpuState
from test_gpu_chunk import FORMATS, SCALE, Case, bits_of, cu_of

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


@pytest.mark.parametrize("fmt", [4, 8, 16])
@pytest.mark.parametrize("sink_at", [0, 20000])
@pytest.mark.parametrize("splits", [1, 3])
def test_many_small_weights_beside_a_sink(fmt, sink_at, splits):
    """One token's logit about 17.7 above 40000 others whose weights, 2^-25.5 of the sink's each, are the whole output (the
    sink's value is zero)."""
    n, m = 40000, 3
    rng = np.random.default_rng(fmt)
    k = np.full((n, 2, 128), 0.609375)
    k[sink_at] = 1.0
    v = rng.uniform(0.5, 1.5, (n, 2, 128))
    v[sink_at] = 0.0
    c = kvq.Cache(fmt, 1, 8, 2, 40064, 32, 0)
    if fmt == 8:
        c.region("fp8_scale").view(torch.float32).copy_(torch.tensor([1.0 / 64, 1.0 / 64, 1.5 / 448, 1.5 / 448]))
    c.append_chunk(to_dev(bits_of(k)), to_dev(bits_of(v)), cu_of([n]), n)
    q = bits_of(np.full((m, 8, 128), 4.0))
    kn, vn = bits_of(np.full((m, 2, 128), 0.609375)), bits_of(rng.uniform(0.5, 1.5, (m, 2, 128)))
    out = torch.zeros(m, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(c.chunk_workspace_bytes(splits, m, m, n), 16), dtype=torch.uint8, device="cuda")
    c.chunk_attention(to_dev(q), to_dev(kn), to_dev(vn), cu_of([m]), m, out, SCALE, ws, splits, n)
    for h in range(8):
        kk, vv = cached_rows(GpuState(c), 0, h // 4)
        kk, vv = np.concatenate([kk, bf16(kn[:, h // 4])]), np.concatenate([vv, bf16(vn[:, h // 4])])
        ref, _, tol = attend(bf16(q[:, h]), kk, vv, np.arange(n, n + m), SCALE)
        # attend allows each weight an error of 2^-25 of the largest.  Here that holds for a key range's first three tiles
        # of 128 tokens; then weights are held at 2^6 times that and more, so that half a step of fp16's smallest numbers is
        # 2^-31.  (Most of what is left of attend's tolerance is e^(2d) - 1 with d = 45.3 2^-11: keys rounded to halves.)
        tol -= (2.0 ** -25 * (kk.shape[0] - 384) - 2.0 ** -31 * kk.shape[0]) * np.abs(vv).max()
        # together 5.3 %, 2.0 % and 3.3 % of the output, where all the small weights were lost with the largest at 1
        assert np.all(ref > 5e-4) and np.all(tol < 0.2 * ref)
        assert np.all(np.abs(out[:, h].float().cpu().numpy() - ref) <= tol), h
    assert c.error() == 0


@pytest.mark.parametrize("fmt", [4, 16])
@pytest.mark.parametrize("top", [0, 14, 30, -20])
@pytest.mark.parametrize("far", [12, 18, 22, 30])
def test_tiny_new_token_beside_ordinary_ones(fmt, top, far):
    """Sixteen new tokens share a piece; the first one's values lie 2^far below the others'.  Row 0 sees it alone: its output
    is off by half a step of the smallest half in the piece's scale, and by the output's own rounding."""
    case = Case(fmt, [0], [16], R=0, seed=250 + far)
    rng = np.random.default_rng(far)
    v = rng.uniform(0.5, 1.0, case.vn.shape) * 2.0 ** top
    v[0] *= 2.0 ** -far
    case.vn = bits_of(v)
    out = case.attend()
    case.check(out)
    tiny = bf16(case.vn[0]).repeat(4, 0)                      # (8 query heads, 2 kv heads)
    # nothing is taken out of a piece whose largest magnitude is in [2^-8, 2^15); otherwise that comes to [2^-2, 2^-1) or
    # [2^8, 2^9)
    largest = np.abs(bf16(case.vn)).max((0, 2)).repeat(4)
    e = np.floor(np.log2(largest))
    e = np.where((largest >= 2.0 ** -8) & (largest < 2.0 ** 15), 0.0, np.where(largest < 1, e + 2, e - 8))
    step = 2.0 ** (e - 25)[:, None]
    assert np.all(np.abs(out[0] - tiny) <= step + 2.0 ** -8 * tiny)
    # numbers down to 2^-17 in that scale are halves as they are
    whole = tiny >= 2.0 ** (e - 17)[:, None]
    assert np.all(out[0][whole] == tiny[whole])


@pytest.mark.parametrize("qexp,scale_exp", [(-60, -30), (-110, -60), (-120, -90)])
def test_scores_too_small_for_floats(qexp, scale_exp):
    """Queries and FP8 key scales whose product is below every float: each visible token weighs the same."""
    case = Case(8, [70, 300], [40, 9], seed=270)
    s = case.cache.region("fp8_scale").view(torch.float32)
    s[:2] = 2.0 ** scale_exp
    case.k = bits_of(bf16(case.k) * 2.0 ** (scale_exp + 4))
    case.kn = bits_of(bf16(case.kn) * 2.0 ** (scale_exp + 4))
    case.q = bits_of(bf16(case.q) * 2.0 ** qexp)
    case.fill()
    case.check(case.attend())
    case.check(case.attend(window=50, sinks=4), 50, 4)
    assert case.cache.error() == 0



@pytest.mark.parametrize("fmt,G,R,paged", FORMATS)
@pytest.mark.parametrize("vexp", [-6, -8, -10, -13, -16, -20, -30, -60])
def test_small_values(fmt, G, R, paged, vexp):
    """All values about 2^vexp: packed, window and new tokens in one key range, their weights held alike."""
    case = Case(fmt, [200, 37, 70, 0], [40, 20, 9, 3], G=G, R=R, paged=paged, seed=260 + G)
    case.v, case.vn = bits_of(bf16(case.v) * 2.0 ** vexp), bits_of(bf16(case.vn) * 2.0 ** vexp)
    if fmt == 8:
        s = case.cache.region("fp8_scale").view(torch.float32)
        s[2:4] = s[2:4] * 2.0 ** vexp
    case.fill()
    check_small(case, case.attend(splits=1))
    check_small(case, case.attend(splits=1, window=90, sinks=20), 90, 20)
    assert case.cache.error() == 0


def check_small(case, out, window=0, sinks=0):
    """Case.check, with the tolerance for weights: halves of 2^-25 in units of the largest product of a weight and its piece's
    power.  A value stands for 2^-e of itself, so the output is off by N 2^-25 |v| 2^d if the pieces' powers are within 2^d of
    another: 2^4 (their largest values, a packed piece's taken as scale * top + zero), and 2^6 more about 2^-8, where none is
    taken out any more.  Raw values are held to 2^-25 in that scale: 2^-17 of their piece's largest."""
    st, at = GpuState(case.cache), 0
    for b, (n, m) in enumerate(zip(case.lens, case.new)):
        for h in range(8):
            k, v = cached_rows(st, b, h // 4)
            k = np.concatenate([k, bf16(case.kn[at:at + m, h // 4])])
            v = np.concatenate([v, bf16(case.vn[at:at + m, h // 4])])
            ref, _, tol = attend(bf16(case.q[at:at + m, h]), k, v, np.arange(n, n + m), SCALE, window, sinks)
            largest = np.abs(v).max()
            d = 10 if 2.0 ** -10 < largest < 2.0 ** -4 else 4
            tol += largest * (k.shape[0] * (2.0 ** (d - 25) - 2.0 ** -25) + 2.0 ** -17) - 1e-30
            err = np.abs(out[at:at + m, h] - ref)
            assert np.all(err <= tol), (b, h, float(np.max(err / tol)))
        at += m


@pytest.mark.parametrize("fmt", [2, 4, 6, 8, 16])
@pytest.mark.parametrize("zero", ["cached", "some cached", "new"])
def test_zero_values_beside_small_ones(fmt, zero):
    """Pieces whose values are all zero have weights but do not push those of small values out of the halves' range."""
    case = Case(fmt, [200, 33], [40, 9], R=0, seed=265)
    rng = np.random.default_rng(fmt)
    small = lambda a: bits_of(rng.uniform(0.5, 1.0, a.shape) * 2.0 ** -15)
    case.v, case.vn = small(case.v), small(case.vn)
    if zero == "cached":
        case.v[:] = 0
    elif zero == "some cached":
        case.v[:64] = 0
    else:
        case.vn[:] = 0
    if fmt == 8:
        case.cache.region("fp8_scale").view(torch.float32)[2:4] = 2.0 ** -15 / 448
    case.fill()
    check_small(case, case.attend(splits=1))
    assert case.cache.error() == 0


@pytest.mark.parametrize("n", [70, 300])
@pytest.mark.parametrize("cached,new", [(-95, -95), (-110, -110), (-110, -97), (-80, -110)])
def test_values_too_small_for_a_scale(n, cached, new):
    """FP8 value scales and new values near the smallest floats: right to what halves keep in a scale of 2^-90."""
    case = Case(8, [n], [40], seed=280)
    case.v, case.vn = bits_of(bf16(case.v) * 2.0 ** cached), bits_of(bf16(case.vn) * 2.0 ** new)
    s = case.cache.region("fp8_scale").view(torch.float32)
    s[2:4] = 2.0 ** (cached - 6)
    case.fill()
    for window, sinks in ((0, 0), (50, 4)):
        out = case.attend(window=window, sinks=sinks)
        # no power below 2^-90 is taken out, where half a step of the smallest halves is 2^-115
        st = GpuState(case.cache)
        for h in range(8):
            k, v = cached_rows(st, 0, h // 4)
            k, v = np.concatenate([k, bf16(case.kn[:, h // 4])]), np.concatenate([v, bf16(case.vn[:, h // 4])])
            ref, _, tol = attend(bf16(case.q[:, h]), k, v, n + np.arange(40), SCALE, window, sinks)
            tol += 2.0 ** -115 + k.shape[0] * 2.0 ** (4 - 25) * np.abs(v).max() - 1e-30      # (weights: check_small's)
            assert np.all(np.abs(out[:, h] - ref) <= tol), (h, float(np.max(np.abs(out[:, h] - ref) / tol)))
    assert case.cache.error() == 0
