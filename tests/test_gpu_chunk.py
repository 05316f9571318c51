"""Chunk append, read-back and chunk attention on the GPU against 64-bit references."""
import numpy as np
import pytest
import torch

from bit_kv_cache_16_b200 import kvq, synth

from chunk_ref import HALF_BF16, HALF_FP16, attend, bf16, cached_rows, rotate
from gpu_harness import (assert_fp8_state, assert_int8_state, assert_unit_state, make_gpu_cache, oracle_cache, round_up,
                         to_dev)
from layout import GpuState

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(128.0)


def bits_of(x: np.ndarray) -> np.ndarray:
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


class Case:
    """A cache filled by one append_chunk of w's tokens, and a ragged chunk behind it."""

    def __init__(self, fmt, lens, new, hq=8, hkv=2, G=32, R=32, paged=False, rope=0.0, sparse=False, seed=0, extra=0,
                 k_outlier=4.0):
        self.fmt, self.lens, self.new = fmt, list(lens), list(new)
        total = [n + m + extra for n, m in zip(self.lens, self.new)]
        self.w = w = synth.make_workload("chunk", 9000 + seed, total, hq, hkv, fmt, G, R, page_size=16 if paged else 0,
                                         k_outlier=k_outlier, q_outlier=1.0)
        self.cache = make_gpu_cache(w, capacity=0 if paged else max(round_up(max(total), max(G, 16)), max(G, 16)),
                                    rope_theta=rope, sparse=sparse)
        self.classes = synth.token_classes(9000 + seed, total)
        rows = [slice(w.cu_seqlens[b], w.cu_seqlens[b] + n) for b, n in enumerate(self.lens)]
        fresh = [slice(r.stop, r.stop + m) for r, m in zip(rows, self.new)]
        pick = lambda a, part: np.ascontiguousarray(np.concatenate([a[p] for p in part]))
        self.k, self.v, self.cls = (pick(a, rows) for a in (w.k, w.v, self.classes))
        self.kn, self.vn, self.clsn = (pick(a, fresh) for a in (w.k, w.v, self.classes))
        rng = np.random.default_rng(seed)
        self.q = bits_of(rng.standard_normal((sum(self.new), hq, 128)))
        self.cu, self.cu_new = cu_of(self.lens), cu_of(self.new)
        if fmt == 8:
            amax = np.stack([np.abs(bf16(a)).max((0, 2)) for a in (w.k, w.v)]).astype(np.float32)
            self.cache.region("fp8_scale").view(torch.float32).copy_(torch.from_numpy((amax / np.float32(448)).ravel()))

    def append(self, k, v, cls, lens):
        self.cache.append_chunk(to_dev(k), to_dev(v), cu_of(lens), max(lens),
                                token_class=to_dev(cls) if self.fmt == 6 else None)

    def fill(self):
        self.append(self.k, self.v, self.cls, self.lens)
        return self

    def attend(self, splits=0, window=0, sinks=0, max_len=None, out=None, stream=None):
        c, w = self.cache, self.w
        rows = sum(self.new)
        if out is None:
            out = torch.full((rows, w.num_q_heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        max_len = max(self.lens) if max_len is None else max_len
        n = c.chunk_workspace_bytes(splits, rows, max(self.new), max_len, window, sinks)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        c.chunk_attention(to_dev(self.q), to_dev(self.kn), to_dev(self.vn), self.cu_new, max(self.new), out, SCALE, ws,
                          splits, max_len, window=window, sinks=sinks, stream=stream)
        torch.cuda.synchronize()
        return out.float().cpu().numpy().astype(np.float64)

    def check(self, out, window=0, sinks=0, rope=0.0, skip_pages=()):
        st = GpuState(self.cache)
        gq = self.w.num_q_heads // self.w.num_kv_heads
        at = 0
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            for h in range(self.w.num_kv_heads):
                if not m:
                    continue
                k, v = cached_rows(st, b, h, rope > 0, rope)
                kn, vn = bf16(self.kn[at:at + m, h]), bf16(self.vn[at:at + m, h])
                if rope > 0:
                    kn = rotate(kn, np.arange(n, n + m, dtype=np.float64), rope)
                k, v = np.concatenate([k, kn]), np.concatenate([v, vn])
                present = np.ones(n + m, bool)
                for bb, page in skip_pages:
                    if bb == b:
                        present[16 * page:16 * page + 16] = False
                for g in range(gq):
                    ref, _, tol = attend(bf16(self.q[at:at + m, h * gq + g]), k, v, np.arange(n, n + m), SCALE, window,
                                         sinks, present)
                    got = out[at:at + m, h * gq + g]
                    err = np.abs(got - ref)
                    assert np.all(err <= tol), (b, h, g, float(np.nanmax(err / tol)), int(np.isnan(got).sum()))
            at += m


FORMATS = [(2, 32, 128, False), (4, 32, 32, False), (4, 16, 16, True), (2, 16, 0, True), (4, 64, 0, False),
           (2, 128, 100, False), (6, 32, 32, False), (6, 64, 16, False), (8, 32, 0, False), (16, 32, 0, False)]


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------

def assert_state(case, oc):
    torch.cuda.synchronize()
    st = GpuState(case.cache)
    units = [(b, h) for b in range(case.w.batch) for h in range(case.w.num_kv_heads)]
    if case.fmt == 8:
        assert_fp8_state(st, oc, units)
    elif case.fmt == 16:
        assert_int8_state(st, oc, units)
    else:
        for b, h in units:
            assert_unit_state(st, oc, b, h)


def oracle_of(case, lens):
    """The oracle after a prefill of the first lens[b] tokens of every sequence."""
    import dataclasses
    w = case.w
    part = [slice(w.cu_seqlens[b], w.cu_seqlens[b] + n) for b, n in enumerate(lens)]
    pick = lambda a: np.ascontiguousarray(np.concatenate([a[p] for p in part]))
    v = dataclasses.replace(w, lengths=np.asarray(lens), k=pick(w.k), v=pick(w.v),
                            cu_seqlens=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    return oracle_cache(v, case.cache.shape.capacity, classes=pick(case.classes),
                        sparse=bool(case.cache.shape.sparse))


@pytest.mark.parametrize("fmt,G,R,paged", [f for f in FORMATS if f[0] != 8])
def test_append_chunk_state(fmt, G, R, paged):
    """Pieces of every size, into empty and filled caches, leave the state of a prefill of all the tokens."""
    lens = [0, 1, 15, 16, R + G - 1, R + G, 3 * G + R + 5, 500]
    new = [1, 0, 17, G, 1, 2 * G + 3, R + G + 1, 401]
    case = Case(fmt, lens, new, G=G, R=R, paged=paged, seed=fmt + G).fill()
    assert_state(case, oracle_of(case, lens))
    case.append(case.kn, case.vn, case.clsn, new)
    assert_state(case, oracle_of(case, [n + m for n, m in zip(lens, new)]))
    assert case.cache.error() == 0


def test_append_chunk_fp8_scales():
    """FP8: codes with the stored scales; the batch's own amax gives the prefill's codes."""
    lens, new = [0, 1, 15, 16, 300], [1, 30, 17, 0, 77]
    case = Case(8, lens, new, seed=3).fill()
    case.append(case.kn, case.vn, case.clsn, new)
    assert_state(case, oracle_of(case, [n + m for n, m in zip(lens, new)]))


@pytest.mark.parametrize("sparse,G", [(True, 16), (True, 32), (False, 32)])
def test_append_chunk_sparse_and_many_heads(sparse, G):
    lens, new = [0, 77, 200], [100, 1, 90]
    case = Case(4, lens, new, hq=20, hkv=10, G=G, R=32, sparse=sparse, seed=5).fill()
    case.append(case.kn, case.vn, case.clsn, new)
    assert_state(case, oracle_of(case, [n + m for n, m in zip(lens, new)]))


@pytest.mark.parametrize("fmt,G,R", [(4, 32, 32), (2, 16, 100), (6, 32, 0), (16, 32, 0)])
def test_append_chunk_in_pieces_equals_tokens(fmt, G, R):
    """Many small pieces of changing size, then single tokens, step by step against append + flush."""
    steps = [1, 2, 3, 5, 8, 13, 21, 34, 55, 1, 1, 89, 7]
    case = Case(fmt, [0, 40], [sum(steps)] * 2, G=G, R=R, seed=8, extra=4).fill()
    w, at = case.w, 0
    for m in steps:
        part = [slice(w.cu_seqlens[b] + n + at, w.cu_seqlens[b] + n + at + m) for b, n in enumerate(case.lens)]
        pick = lambda a: np.ascontiguousarray(np.concatenate([a[p] for p in part]))
        case.append(pick(w.k), pick(w.v), pick(case.classes), [m, m])
        at += m
        assert_state(case, oracle_of(case, [n + at for n in case.lens]))
    rows = [w.cu_seqlens[b] + n + at for b, n in enumerate(case.lens)]
    kn, vn, cls = (np.ascontiguousarray(a[rows]) for a in (w.k, w.v, case.classes))
    if fmt == 6:
        case.cache.append_flush_mixed(to_dev(kn), to_dev(vn), to_dev(cls))
    else:
        case.cache.append_flush(to_dev(kn), to_dev(vn))
    assert_state(case, oracle_of(case, [n + at + 1 for n in case.lens]))


def test_append_chunk_flushes_a_full_window():
    """A window left full by append_token (no flush) is flushed by an empty chunk, as kvq_flush_group would."""
    G, R = 32, 32
    case = Case(4, [R + G - 1, 10], [1, 1], G=G, R=R, seed=11, extra=2).fill()
    case.cache.append_token(to_dev(case.kn), to_dev(case.vn))
    assert GpuState(case.cache).n_quant[:2].tolist() == [0, 0]
    case.append(case.kn[:0], case.vn[:0], case.clsn[:0], [0, 0])
    assert_state(case, oracle_of(case, [R + G, 11]))


def test_append_chunk_dropped():
    """A chunk past the capacity or longer than max_new, and a bad page, drop that sequence's chunk only."""
    case = Case(4, [50, 60, 30], [14, 4, 40], G=32, R=0, seed=12)
    cap = case.cache.shape.capacity                      # 96
    case.fill()
    before = GpuState(case.cache)
    case.append(case.kn, case.vn, case.clsn, [14, 4, 40])
    assert case.cache.error() == 0 and GpuState(case.cache).seq_len[:3].tolist() == [64, 64, 70]
    rng = np.random.default_rng(1)
    k = bits_of(rng.standard_normal((cap - 64 + 1 + 3 + 9, 2, 128)))
    lens = [cap - 64 + 1, 3, 9]                          # the first does not fit
    case.append(k, k, None, lens)
    assert case.cache.error() == kvq.KVQ_DEVERR_APPEND_FULL
    st = GpuState(case.cache)
    assert st.seq_len[:3].tolist() == [64, 67, 79] and st.n_quant[:3].tolist() == [64, 64, 64]
    case.cache.clear_error()
    case.cache.append_chunk(to_dev(k[:13]), to_dev(k[:13]), cu_of([1, 3, 9]), 3)
    assert case.cache.error() == kvq.KVQ_DEVERR_PREFILL_LEN
    assert GpuState(case.cache).seq_len[:3].tolist() == [65, 70, 79]
    assert before.cap == cap


def test_rows_outside_the_arrays():
    """Offsets that leave the given rows drop that sequence: nothing is read or written outside."""
    case = Case(4, [50, 60], [10, 4], seed=15).fill()
    k = torch.zeros(10, 2, 128, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 7, 12], dtype=torch.int32, device="cuda")          # rows 10 and 11 do not exist
    case.cache.append_chunk(k, k, cu, 10)
    assert case.cache.error() == kvq.KVQ_DEVERR_PREFILL_LEN
    assert GpuState(case.cache).seq_len[:2].tolist() == [57, 60]
    case.cache.clear_error()
    case.cache.append_chunk(k, k, torch.tensor([-3, 2, 4], dtype=torch.int32, device="cuda"), 10)
    assert case.cache.error() == kvq.KVQ_DEVERR_PREFILL_LEN
    assert GpuState(case.cache).seq_len[:2].tolist() == [57, 62]
    case.cache.clear_error()
    out = [torch.full((14, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    case.cache.read_tokens(None, cu, 10, out[0][:10], out[1][:10])
    assert case.cache.error() == kvq.KVQ_DEVERR_PREFILL_LEN
    assert not torch.any(out[0][:7] == 7.0) and torch.all(out[0][7:] == 7.0) and torch.all(out[1][7:] == 7.0)


def test_append_chunk_bad_page():
    case = Case(4, [40, 40], [40, 40], G=16, R=16, paged=True, seed=13).fill()
    table = case.cache.region("page_table").view(torch.int32).view(2, -1)
    keep = table.clone()
    table[1, 3] = case.cache.shape.num_pages             # a page that the second chunk needs
    case.append(case.kn, case.vn, None, [40, 40])
    assert case.cache.error() == kvq.KVQ_DEVERR_PAGE_RANGE
    st = GpuState(case.cache)
    assert st.seq_len[:2].tolist() == [80, 40] and st.n_quant[:2].tolist() == [64, 16]
    case.cache.clear_error()
    table.copy_(keep)
    case.append(case.kn[40:], case.vn[40:], None, [0, 40])
    assert_state(case, oracle_of(case, [80, 80]))


def test_append_chunk_leaves_other_bytes():
    """8-bit tiles: the codes of tokens already held in a partly filled tile stay, and bytes of other units too."""
    for fmt in (8, 16):
        case = Case(fmt, [5, 37], [6, 3], seed=14).fill()
        a = GpuState(case.cache)
        case.append(case.kn, case.vn, None, [6, 3])
        b = GpuState(case.cache)
        for s, n in enumerate([5, 37]):
            ua, ub = a.unit(s, 1, round_up(n, 16)), b.unit(s, 1, round_up(n, 16))
            for name in ua:
                assert np.array_equal(ua[name][:n], ub[name][:n]), (fmt, name)


# ---------------------------------------------------------------------------
# Read back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,G,R,paged", FORMATS)
def test_read_tokens(fmt, G, R, paged):
    lens = [0, 1, 15, 16, 17, R + G, 3 * G + R + 5, 700]
    case = Case(fmt, lens, [0] * 8, G=G, R=R, paged=paged, seed=20 + fmt).fill()
    st = GpuState(case.cache)
    start = [0, 0, 3, 0, 16, 5, 2 * G + 7, 133]
    take = [max(0, min(n - s, t)) for n, s, t in zip(lens, start, [0, 1, 100, 16, 1, R + G - 9, 3 * G, 555])]
    for begin, length in ((None, lens), (torch.tensor(start, dtype=torch.int32, device="cuda"), take)):
        rows = sum(length)
        out = [torch.full((rows + 3, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        case.cache.read_tokens(begin, cu_of(length), max(length), *out)
        torch.cuda.synchronize()
        got = [o.float().cpu().numpy().astype(np.float64) for o in out]
        at = 0
        for b, n in enumerate(length):
            s0 = 0 if begin is None else start[b]
            for h in range(2):
                for x, ref in zip(got, cached_rows(st, b, h)):
                    r = ref[s0:s0 + n]
                    # one rounding to fp32 and one to bf16
                    assert np.all(np.abs(x[at:at + n, h] - r) <= np.abs(r) * (HALF_BF16 + 2.0 ** -20) + 1e-38), (b, h)
            at += n
        assert all(np.all(x[rows:] == 7.0) for x in got)     # rows behind the last range
    only = torch.zeros(sum(lens), 2, 128, dtype=torch.bfloat16, device="cuda")
    case.cache.read_tokens(None, cu_of(lens), max(lens), None, only)
    full = torch.zeros_like(only)
    case.cache.read_tokens(None, cu_of(lens), max(lens), torch.zeros_like(only), full)
    assert torch.equal(only, full) and case.cache.error() == 0


@pytest.mark.parametrize("fmt,G", [(4, 32), (2, 16)])
def test_read_tokens_sparse_and_rope(fmt, G):
    case = Case(fmt, [130, 64], [0, 0], G=G, R=16, sparse=True, seed=30).fill()
    rope = Case(fmt, [130, 64], [0, 0], G=32, R=16, rope=10000.0, seed=30).fill()
    for c in (case, rope):
        out = [torch.empty(194, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        c.cache.read_tokens(None, c.cu, 130, *out)
        torch.cuda.synchronize()
        st = GpuState(c.cache)
        for b, part in enumerate((slice(0, 130), slice(130, 194))):
            for h in range(2):
                for o, ref in zip(out, cached_rows(st, b, h)):
                    x = o[part, h].float().cpu().numpy()
                    assert np.all(np.abs(x - ref) <= np.abs(ref) * (HALF_BF16 + 2.0 ** -20) + 1e-38)


@pytest.mark.parametrize("fmt,G,R,paged", FORMATS)
def test_rows_at_odd_sixteenths(fmt, G, R, paged):
    """Arrays that start 16 bytes past a 32-byte boundary: the same numbers."""
    case = Case(fmt, [130, 33], [40, 1], G=G, R=R, paged=paged, seed=33).fill()

    def shifted(like):
        t = torch.zeros(like.numel() + 8, dtype=like.dtype, device="cuda")[8:].view(like.shape)
        assert t.data_ptr() % 32 == 16
        return t.copy_(like)

    rows = [torch.zeros(163, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    odd = [shifted(r) for r in rows]
    case.cache.read_tokens(None, case.cu, 130, *rows)
    case.cache.read_tokens(None, case.cu, 130, *odd)
    assert torch.equal(rows[0], odd[0]) and torch.equal(rows[1], odd[1]) and rows[1].abs().sum() > 0
    q, kn, vn = (to_dev(x) for x in (case.q, case.kn, case.vn))
    out = [torch.zeros(41, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out[1] = shifted(out[0])
    case.cache.chunk_attention(q, kn, vn, case.cu_new, 40, out[0], SCALE, None, 1, 130)
    case.cache.chunk_attention(shifted(q), shifted(kn), shifted(vn), case.cu_new, 40, out[1], SCALE, None, 1, 130)
    assert torch.equal(*out) and out[0].abs().sum() > 0
    other = Case(fmt, [130, 33], [40, 1], G=G, R=R, paged=paged, seed=33).fill()
    cls = to_dev(case.clsn) if fmt == 6 else None
    case.cache.append_chunk(kn, vn, case.cu_new, 40, token_class=cls)
    other.cache.append_chunk(shifted(kn), shifted(vn), case.cu_new, 40, token_class=cls)
    for name in ("k_codes", "v_codes", "k_meta", "v_meta", "k_res", "v_res", "seq_len"):
        x, y = case.cache.buffers[name], other.cache.buffers[name]
        assert x is None or torch.equal(x, y), name
    assert case.cache.error() == 0 and other.cache.error() == 0


def test_read_tokens_refused_ranges():
    case = Case(4, [50, 60, 70], [0, 0, 0], G=16, R=16, paged=True, seed=31).fill()
    out = [torch.full((100, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    start = torch.tensor([40, 0, 69], dtype=torch.int32, device="cuda")
    case.cache.read_tokens(start, cu_of([11, 20, 1]), 20, *out)      # sequence 0 reads past its end
    assert case.cache.error() == kvq.KVQ_DEVERR_PREFILL_LEN
    assert torch.all(out[0][:11] == 7.0) and not torch.any(out[0][11:32] == 7.0) and torch.all(out[0][32:] == 7.0)
    case.cache.clear_error()
    table = case.cache.region("page_table").view(torch.int32).view(3, -1)
    table[1, 1] = -1
    out[1].fill_(7.0)
    case.cache.read_tokens(None, cu_of([0, 40, 0]), 40, None, out[1])
    assert case.cache.error() == kvq.KVQ_DEVERR_PAGE_RANGE
    assert not torch.any(out[1][:16] == 7.0) and torch.all(out[1][16:32] == 7.0) and not torch.any(out[1][32:40] == 7.0)


# ---------------------------------------------------------------------------
# Chunk attention
# ---------------------------------------------------------------------------

LENS = [0, 1, 15, 33, 64, 130, 700]
NEW = [5, 1, 0, 40, 129, 3, 70]


@pytest.mark.parametrize("fmt,G,R,paged", FORMATS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4), (1, 0), (129, 70)])
def test_chunk_attention(fmt, G, R, paged, window, sinks):
    case = Case(fmt, LENS, NEW, G=G, R=R, paged=paged, seed=40 + fmt + G).fill()
    case.check(case.attend(window=window, sinks=sinks), window, sinks)
    assert case.cache.error() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (7, 1), (16, 2), (12, 6)])
def test_chunk_attention_heads(hq, hkv):
    case = Case(4, [200, 0, 47], [37, 61, 2], hq=hq, hkv=hkv, seed=50 + hq).fill()
    case.check(case.attend())


@pytest.mark.parametrize("fmt", [2, 4, 6, 8, 16])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40])
def test_chunk_attention_splits(fmt, splits):
    case = Case(fmt, [1300, 5, 400], [3, 1, 9], seed=60 + fmt).fill()
    case.check(case.attend(splits=splits))
    case.check(case.attend(splits=splits, window=300, sinks=7), 300, 7)


@pytest.mark.parametrize("n,m", [(1, 1), (127, 1), (128, 1), (129, 255), (2049, 300), (0, 513)])
def test_chunk_attention_edges(n, m):
    for fmt, R in ((4, 0), (4, 128), (16, 0)):
        case = Case(fmt, [n], [m], hq=4, hkv=1, R=R, seed=70).fill()
        case.check(case.attend())
        case.check(case.attend(window=64, sinks=130), 64, 130)


@pytest.mark.parametrize("fmt,G", [(4, 32), (2, 16)])
def test_chunk_attention_sparse(fmt, G):
    case = Case(fmt, [130, 0, 64], [33, 5, 1], G=G, R=16, sparse=True, seed=80, k_outlier=20.0).fill()
    case.check(case.attend())
    case.check(case.attend(window=40, sinks=3), 40, 3)


@pytest.mark.parametrize("fmt", [2, 4])
def test_chunk_attention_rope(fmt):
    case = Case(fmt, [130, 0, 700], [33, 5, 1], R=16, rope=10000.0, seed=81).fill()
    case.check(case.attend(), rope=10000.0)
    case.check(case.attend(window=40, sinks=3), 40, 3, rope=10000.0)


@pytest.mark.parametrize("splits", [0, 1, 3])
def test_chunk_attention_bound_of_zero(splits):
    """max_new = 0: empty chunks are fine, any other is refused on the device and its rows stay."""
    case = Case(4, [70, 9], [3, 2], seed=35).fill()
    out = torch.full((5, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(case.cache.chunk_workspace_bytes(splits, 5, 0, 70), 16), dtype=torch.uint8, device="cuda")
    q, kn, vn = (to_dev(x) for x in (case.q, case.kn, case.vn))
    for cu, error in ((cu_of([0, 0]), 0), (case.cu_new, kvq.KVQ_DEVERR_PREFILL_LEN)):
        case.cache.chunk_attention(q, kn, vn, cu, 0, out, SCALE, ws, splits, 70)
        assert case.cache.error() == error and torch.all(out == 7.0)


def test_chunk_attention_bad_page():
    case = Case(4, [200, 90], [20, 7], G=16, R=16, paged=True, seed=82).fill()
    st = GpuState(case.cache)
    table = case.cache.region("page_table").view(torch.int32).view(2, -1)
    keep = table.clone()
    table[0, 3] = -1
    table[1, 0] = case.cache.shape.num_pages
    out = case.attend()
    assert case.cache.error() == kvq.KVQ_DEVERR_PAGE_RANGE
    table.copy_(keep)
    case.check(out, skip_pages=[(0, 3), (1, 0)])
    assert st.seq_len[:2].tolist() == [200, 90]


def test_chunk_attention_skips_and_leaves_rows():
    """A chunk longer than max_new and rows behind the last chunk stay as they were."""
    case = Case(4, [100, 50], [9, 4], seed=83).fill()
    out = torch.full((16, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(16, 8, 128, dtype=torch.bfloat16, device="cuda")
    q[:13] = to_dev(case.q).view(torch.bfloat16)
    k, v = (torch.full((16, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[:13], v[:13] = to_dev(case.kn).view(torch.bfloat16), to_dev(case.vn).view(torch.bfloat16)
    n = case.cache.chunk_workspace_bytes(0, 16, 9, 100)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    case.cache.chunk_attention(q, k, v, case.cu_new, 9, out, SCALE, ws, 0, 100)
    torch.cuda.synchronize()
    assert torch.all(out[13:] == 7.0)
    case.check(out[:13].float().cpu().numpy().astype(np.float64))
    out.fill_(7.0)
    case.cache.chunk_attention(q, k, v, case.cu_new, 8, out, SCALE, ws, 0, 100)      # the first chunk has 9
    assert case.cache.error() == kvq.KVQ_DEVERR_PREFILL_LEN
    assert torch.all(out[:9] == 7.0) and not torch.any(out[9:13] == 7.0)


def test_prompt_in_pieces_then_decode():
    """The operators as a server uses them: pieces of a prompt attend and are appended, then a decode step; the cache ends
    up as one prefill of the whole prompt leaves it, and the last piece's output is that of the reference."""
    pieces = [[100, 3], [64, 0], [33, 50]]
    case = Case(4, [0, 0], [197, 53], seed=90)
    w = case.w
    at = [0, 0]
    for piece in pieces:
        part = [slice(w.cu_seqlens[b] + at[b], w.cu_seqlens[b] + at[b] + m) for b, m in enumerate(piece)]
        pick = lambda a: np.ascontiguousarray(np.concatenate([a[p] for p in part]))
        step = Case.__new__(Case)
        step.__dict__.update(case.__dict__)
        step.lens, step.new, step.kn, step.vn = list(at), piece, pick(w.k), pick(w.v)
        step.q = case.q[:sum(piece)]
        step.cu_new = cu_of(piece)
        step.check(step.attend())
        case.append(step.kn, step.vn, None, piece)
        at = [a + m for a, m in zip(at, piece)]
    assert_state(case, oracle_of(case, at))
    out = torch.empty(2, 8, 128, device="cuda")
    ws = torch.empty(case.cache.workspace_bytes(0, max(at)), dtype=torch.uint8, device="cuda")
    case.cache.decode_attention(to_dev(w.q), out, SCALE, ws, 0, max(at))
    st = GpuState(case.cache)
    for b in range(2):
        for h in range(8):
            k, v = cached_rows(st, b, h // 4)
            ref, _, tol = attend(bf16(w.q[b, h])[None], k, v, [at[b] - 1], SCALE)
            assert np.all(np.abs(out[b, h].cpu().numpy() - ref[0]) <= tol[0])


def test_chunk_captured_and_replayed():
    """Append, read and chunk attention in a CUDA graph on a side stream, replayed on new inputs."""
    case = Case(4, [300, 7], [20, 4], seed=91, extra=60).fill()
    c, w = case.cache, case.w
    q, k, v = (to_dev(a).view(torch.bfloat16).clone() for a in (case.q, case.kn, case.vn))
    out = torch.empty_like(q)
    n = c.chunk_workspace_bytes(0, 24, 20, 360)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step():
        c.chunk_attention(q, k, v, case.cu_new, 20, out, SCALE, ws, 0, 360)
        c.append_chunk(k, v, case.cu_new, 20)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                      # warm-up: the first piece
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    lens = [320, 11]
    for i in range(2):                              # the same piece again and again, behind itself
        graph.replay()
        torch.cuda.synchronize()
        lens = [n + m for n, m in zip(lens, case.new)]
        assert GpuState(c).seq_len[:2].tolist() == lens
        eager = torch.empty_like(out)
        # what the replay saw: the state before its append
        c.seq_len()[:2].copy_(torch.tensor([n - m for n, m in zip(lens, case.new)], dtype=torch.int32))
        st = GpuState(c)
        if all(st.n_quant <= st.seq_len):
            c.chunk_attention(q, k, v, case.cu_new, 20, eager, SCALE, ws, 0, 360)
        c.seq_len()[:2].copy_(torch.tensor(lens, dtype=torch.int32))
    assert c.error() == 0


@pytest.mark.parametrize("bad", ["inf", "nan"])
def test_later_tokens_do_not_reach_earlier_rows(bad):
    """An infinity or NaN in a new token is hidden from the rows before it."""
    case = Case(4, [70], [40], seed=92).fill()
    clean = case.attend()
    kn, vn = case.kn.copy(), case.vn.copy()
    kn[25], vn[25] = (0x7F80, 0x7F80) if bad == "inf" else (0x7FC0, 0x7FC0)
    case.kn, case.vn = kn, vn
    out = case.attend()
    assert np.array_equal(out[:25], clean[:25])
    assert not np.any(np.isfinite(out[25:]))


# ---------------------------------------------------------------------------
# Windowed decode
# ---------------------------------------------------------------------------

def decode_window(case, window, sinks, splits=0, max_len=None):
    c, w = case.cache, case.w
    out = torch.full((w.batch, w.num_q_heads, 128), float("nan"), device="cuda")
    lse = torch.full((w.batch, w.num_q_heads), float("nan"), device="cuda")
    max_len = max(case.lens) if max_len is None else max_len
    n = c.window_workspace_bytes(splits, max_len, window, sinks)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    c.decode_attention_window(to_dev(w.q), out, SCALE, window, sinks, ws, splits, max_len, lse=lse)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def check_decode(case, got, window, sinks, rope=0.0, skip_pages=()):
    out, lse = got
    st = GpuState(case.cache)
    gq = case.w.num_q_heads // case.w.num_kv_heads
    for b, n in enumerate(case.lens):
        present = np.ones(n, bool)
        for bb, page in skip_pages:
            if bb == b:
                present[16 * page:16 * page + 16] = False
        for h in range(case.w.num_q_heads):
            if n == 0:
                assert np.all(out[b, h] == 0) and lse[b, h] == -np.inf
                continue
            k, v = cached_rows(st, b, h // gq, rope > 0, rope)
            q = bf16(case.w.q[b, h])[None]
            # products of exact codes with operands split into two halves (22 bits), sums in 32 bits
            ref, ref_lse, tol = attend(q, k, v, [n - 1], SCALE, window, sinks, present, rounded=False)
            err = np.abs(out[b, h] - ref[0])
            assert np.all(err <= tol[0]), (b, h, float(np.nanmax(err / tol[0])), int(np.isnan(out[b, h]).sum()))
            # a score is off by at most d (attend's comment), and so is the log of their exponentials' sum
            d = SCALE * (np.abs(q) @ np.abs(k).T).max() * 2.0 ** -18 + 2.0 ** -18 + abs(ref_lse[0]) * 2.0 ** -22
            assert abs(lse[b, h] - ref_lse[0]) <= d, (b, h, lse[b, h], ref_lse[0])


@pytest.mark.parametrize("fmt,G,R,paged", FORMATS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 4), (129, 70), (10000, 3)])
def test_window_decode(fmt, G, R, paged, window, sinks):
    case = Case(fmt, [0, 1, 15, 33, 64, 130, 1100], [0] * 7, G=G, R=R, paged=paged, seed=100 + fmt + G).fill()
    for splits in (0, 1, 3):
        check_decode(case, decode_window(case, window, sinks, splits), window, sinks)
    assert case.cache.error() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (8, 1), (12, 6)])
def test_window_decode_heads(hq, hkv):
    case = Case(2, [300, 0, 47], [0] * 3, hq=hq, hkv=hkv, seed=110).fill()
    check_decode(case, decode_window(case, 100, 5), 100, 5)


def test_window_decode_sparse_and_rope():
    for kw in (dict(sparse=True, G=16, k_outlier=20.0), dict(rope=10000.0)):
        case = Case(4, [300, 1, 47], [0] * 3, R=16, seed=111, **kw).fill()
        check_decode(case, decode_window(case, 100, 5), 100, 5, rope=kw.get("rope", 0.0))


def test_window_decode_bad_page_and_state():
    case = Case(4, [200, 90, 40], [0] * 3, G=16, R=16, paged=True, seed=112).fill()
    table = case.cache.region("page_table").view(torch.int32).view(3, -1)
    keep = table.clone()
    table[0, 3], table[1, 0] = -1, case.cache.shape.num_pages
    got = decode_window(case, 170, 20)
    assert case.cache.error() == kvq.KVQ_DEVERR_PAGE_RANGE
    table.copy_(keep)
    check_decode(case, got, 170, 20, skip_pages=[(0, 3), (1, 0)])
    case.cache.clear_error()
    case.cache.n_quant()[1] = 7
    out, _ = decode_window(case, 0, 0)
    assert case.cache.error() == kvq.KVQ_DEVERR_STATE
    assert np.all(out[1] == 0) and np.all(np.isfinite(out)) and np.any(out[0] != 0) and np.any(out[2] != 0)


@pytest.mark.parametrize("fmt", [2, 4, 6, 8, 16])
def test_window_decode_equals_full_decode(fmt):
    """A window over everything gives what the unwindowed decode gives, within the roundings of both."""
    case = Case(fmt, [700, 90, 0], [0] * 3, seed=113).fill()
    c, w = case.cache, case.w
    out = torch.empty(3, 8, 128, device="cuda")
    ws = torch.empty(c.workspace_bytes(0, 700), dtype=torch.uint8, device="cuda")
    c.decode_attention(to_dev(w.q), out, SCALE, ws, 0, 700)
    got, _ = decode_window(case, 700, 0)
    st = GpuState(c)
    for b, n in enumerate(case.lens):
        for h in range(8):
            k, v = cached_rows(st, b, h // 4)
            if n:
                tol = attend(bf16(w.q[b, h])[None], k, v, [n - 1], SCALE)[2][0]
                assert np.all(np.abs(got[b, h] - out[b, h].cpu().numpy()) <= 2 * tol)


def test_hidden_values_do_not_reach_the_row():
    """NaN and infinities in tokens outside the window (quantized ones and window ones) change nothing."""
    for fmt, R in ((4, 64), (16, 0)):
        case = Case(fmt, [200], [0], R=R, seed=114).fill()
        clean = decode_window(case, 20, 3)
        kq, vq = case.k.copy(), case.v.copy()
        for t, x in ((45, 0x7FC0), (70, 0x7F80), (150, 0x7FC0), (178, 0x7F80)):
            kq[t], vq[t] = x, x
        vq[10] = 0x7FC0                             # in the sinks' value tile (keys share their group's scale)
        case.cache.reset()
        case.append(kq, vq, None, [200])
        got = decode_window(case, 20, 3)
        for a, b in zip(clean, got):
            assert np.array_equal(a, b), fmt


# ---------------------------------------------------------------------------
# Ranges, scales and use
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-6, 3.0])
def test_softmax_scales(scale):
    """Any finite softmax scale: 0 (the plain mean), negative, tiny, and one that leaves little but the largest score."""
    case = Case(4, [200, 0], [40, 3], seed=120).fill()
    c = case.cache
    out = torch.empty(43, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(c.chunk_workspace_bytes(2, 43, 40, 200), 16), dtype=torch.uint8, device="cuda")
    c.chunk_attention(to_dev(case.q), to_dev(case.kn), to_dev(case.vn), case.cu_new, 40, out, scale, ws, 2, 200)
    o2 = torch.empty(2, 8, 128, device="cuda")
    ws = torch.empty(c.window_workspace_bytes(0, 200, 90, 2), dtype=torch.uint8, device="cuda")
    c.decode_attention_window(to_dev(case.w.q), o2, scale, 90, 2, ws, 0, 200)
    torch.cuda.synchronize()
    st, at = GpuState(c), 0
    for b, (n, m) in enumerate(zip(case.lens, case.new)):
        for h in range(8):
            k, v = cached_rows(st, b, h // 4)
            if n:
                ref, _, tol = attend(bf16(case.w.q[b, h])[None], k, v, [n - 1], scale, 90, 2, rounded=False)
                assert np.all(np.abs(o2[b, h].cpu().numpy() - ref[0]) <= tol[0])
            k = np.concatenate([k, bf16(case.kn[at:at + m, h // 4])])
            v = np.concatenate([v, bf16(case.vn[at:at + m, h // 4])])
            ref, _, tol = attend(bf16(case.q[at:at + m, h]), k, v, np.arange(n, n + m), scale)
            assert np.all(np.abs(out[at:at + m, h].float().cpu().numpy() - ref) <= tol), (b, h)
        at += m


@pytest.mark.parametrize("n,kexp,vexp,qexp", [(70, 17, 0, -17), (0, -20, 20, 20), (70, 0, -30, 0), (70, 0, 60, 0),
                                              (70, 30, -60, -30), (0, -60, -60, 60)])
def test_chunk_of_any_magnitude(n, kexp, vexp, qexp):
    """New tokens (and queries) far outside fp16's range beside cached ones of ordinary size: the powers of two taken out
    of their rows come back in the scores and the output."""
    case = Case(4, [n], [40], R=64, seed=121).fill()
    up = lambda a, e: bits_of(bf16(a) * 2.0 ** e)
    case.kn, case.vn, case.q = up(case.kn, kexp), up(case.vn, vexp), up(case.q, qexp)
    case.check(case.attend())
    assert case.cache.error() == 0
    # the same tokens from the window ring
    case.append(case.kn, case.vn, None, [40])
    case.lens, case.kn, case.vn, case.q = [n + 40], case.kn[:5], case.vn[:5], case.q[:5]
    case.new, case.cu_new = [5], cu_of([5])
    assert GpuState(case.cache).n_quant[0] <= n               # none of the new tokens is quantized
    case.check(case.attend())


@pytest.mark.parametrize("fmt", [4, 8, 16, 2])
def test_chunk_hidden_cached_values(fmt):
    """NaN and infinities in cached tokens that the window hides from every row change nothing."""
    case = Case(fmt, [330], [20], R=0, seed=122).fill()
    clean = case.attend(window=60, sinks=3)
    kq, vq = case.k.copy(), case.v.copy()
    for t, x in ((100, 0x7FC0), (150, 0x7F80), (200, 0x7FC0)):
        kq[t], vq[t] = x, x
    vq[[10, 262, 268]] = np.array([0x7FC0, 0x7F80, 0x7FC0])[:, None, None]      # beside visible ones (values: by token)
    case.cache.reset()
    case.append(kq, vq, None, [330])
    got = case.attend(window=60, sinks=3)
    # (the first visible token of row 0 is 330 - 59 = 271.)  The weights are the same bit for bit; where a tile is looked
    # at closely, their sum is taken in another order: 64 steps of 2^-24, which can only turn the last rounding to bf16
    # over, by one step of at most 2^-7 of the value
    assert np.all(np.abs(got - clean) <= 2.0 ** -7 * np.abs(clean))


def test_chunk_visible_nan_makes_its_rows_nan():
    case = Case(16, [100], [30], seed=123).fill()
    vq = case.v.copy()
    vq[60, 1] = 0x7FC0
    case.cache.reset()
    case.append(case.k, vq, None, [100])
    out = case.attend(window=60, sinks=0)
    # row i sees tokens > 100 + i - 60: token 60 for i < 20
    assert not np.any(np.isfinite(out[:20, 4:])) and np.all(np.isfinite(out[20:])) and np.all(np.isfinite(out[:, :4]))


def test_calls_on_two_streams():
    """Two caches attended and appended on two streams at once give what they give one after the other."""
    cases = [Case(f, [900, 33], [70, 5], seed=124 + f).fill() for f in (4, 16)]
    want = [c.attend(splits=2) for c in cases]
    args = []
    for c in cases:
        n = c.cache.chunk_workspace_bytes(2, 75, 70, 900)
        args.append([to_dev(c.q), to_dev(c.kn), to_dev(c.vn), torch.empty(75, 8, 128, dtype=torch.bfloat16, device="cuda"),
                     torch.empty(n, dtype=torch.uint8, device="cuda")])
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, (q, k, v, out, ws) in zip(cases, streams, args):
            c.cache.chunk_attention(q, k, v, c.cu_new, 70, out, SCALE, ws, 2, 900, stream=s)
    torch.cuda.synchronize()
    for c, w, a in zip(cases, want, args):
        assert np.array_equal(a[3].float().cpu().numpy().astype(np.float64), w)


def test_window_decode_captured():
    """Append, windowed decode and read back in a graph, replayed while the sequences grow."""
    case = Case(2, [300, 7], [1, 1], G=16, R=16, seed=126, extra=8).fill()
    c = case.cache
    k, v = to_dev(case.kn), to_dev(case.vn)
    q, out, lse = to_dev(case.w.q), torch.empty(2, 8, 128, device="cuda"), torch.empty(2, 8, device="cuda")
    ws = torch.empty(c.window_workspace_bytes(0, 320, 100, 4), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step():
        c.append_chunk(k, v, case.cu_new, 1)
        c.decode_attention_window(q, out, SCALE, 100, 4, ws, 0, 320, lse=lse)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        case.lens = [300 + 2 + i, 7 + 2 + i]
        check_decode(case, (out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)), 100, 4)
    assert c.error() == 0


def test_long_offsets():
    """A unit whose packed rows pass 2^31 bytes: reads, chunk attention and windowed decode at its far end."""
    cap = 17 * 2 ** 20                                       # x 128 bytes per row = 2.1 GiB of keys for one head
    c = kvq.Cache(16, 1, 2, 1, cap)
    n = cap - 300
    c.seq_len()[0] = c.n_quant()[0] = n
    rng = np.random.default_rng(7)
    k, v = (to_dev(bits_of(rng.standard_normal((200, 1, 128)))) for _ in range(2))
    cu = cu_of([200])
    c.append_chunk(k, v, cu, 200)
    out = [torch.empty(200, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c.read_tokens(torch.tensor([n], dtype=torch.int32, device="cuda"), cu, 200, *out)
    q, kn, vn = (to_dev(bits_of(rng.standard_normal((7, h, 128)))) for h in (2, 1, 1))
    o = torch.empty(7, 2, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(c.chunk_workspace_bytes(3, 7, 7, cap, 150), 16), dtype=torch.uint8, device="cuda")
    c.chunk_attention(q, kn, vn, cu_of([7]), 7, o, SCALE, ws, 3, cap, window=150)
    o1 = torch.empty(1, 2, 128, device="cuda")
    ws = torch.empty(c.window_workspace_bytes(0, cap, 150), dtype=torch.uint8, device="cuda")
    c.decode_attention_window(q[:1], o1, SCALE, 150, 0, ws, 0, cap)
    torch.cuda.synchronize()
    assert c.error() == 0 and c.seq_len()[0] == n + 200
    rows = [x.float().cpu().numpy().astype(np.float64)[:, 0] for x in out]
    for x, given in zip(rows, (k, v)):
        g = bf16(given.cpu().numpy().view(np.uint16))[:, 0]
        step = (g.max(1) - g.min(1))[:, None] / 255           # half a code's step and the roundings of scale, zero, bf16
        assert np.all(np.abs(x - g) <= 0.5 * step * (1 + 2.0 ** -9) + 255 * step * 2.0 ** -11 + np.abs(g) * 2.0 ** -7)
    # attention over what the cache holds: rows as read back are rounded to bf16, hence the wider tolerance
    kk, vv = (np.concatenate([a, bf16(b.cpu().numpy().view(np.uint16))[:, 0]]) for a, b in zip(rows, (kn, vn)))
    qq = bf16(q.cpu().numpy().view(np.uint16))
    for h in range(2):
        ref, _, tol = attend(qq[:, h], kk, vv, np.arange(200, 207), SCALE, 150)
        d = SCALE * (np.abs(qq[:, h]) @ np.abs(kk).T).max(1)[:, None] * HALF_BF16
        wide = tol + np.expm1(2 * d) * np.abs(vv).max() + HALF_BF16 * np.abs(vv).max()
        assert np.all(np.abs(o[:, h].float().cpu().numpy() - ref) <= wide)
        ref, _, _ = attend(qq[:1, h], kk[:200], vv[:200], [199], SCALE, 150)
        assert np.all(np.abs(o1[0, h].cpu().numpy() - ref[0]) <= wide[0])
