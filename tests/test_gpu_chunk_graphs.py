"""Chunk calls captured in CUDA graphs, replayed on new inputs and compared with the same calls made one by one (GPU)."""
import numpy as np
import pytest
import torch

from gpu_harness import to_dev
from test_gpu_chunk import SCALE, Case, bits_of

pytestmark = pytest.mark.gpu


def held(cache):
    return {name: t.clone() for name, t in cache.buffers.items() if t is not None}


def put_back(cache, state):
    for name, t in state.items():
        cache.buffers[name].copy_(t)


@pytest.mark.parametrize("fmt", [2, 4, 6, 8, 16])
@pytest.mark.parametrize("splits", [1, 3])
def test_replays_equal_calls(fmt, splits):
    """Attend, append and read back in one graph: each replay, on new inputs behind the tokens of the last, gives what the
    calls give from the same state, in the outputs and in every buffer of the cache."""
    new = [20, 4]
    case = Case(fmt, [300, 7], new, R=32, seed=300 + fmt, extra=90).fill()
    c = case.cache
    rng = np.random.default_rng(fmt)
    q, k, v = (to_dev(a).view(torch.bfloat16).clone() for a in (case.q, case.kn, case.vn))
    cls = to_dev(case.clsn).clone() if fmt == 6 else None
    out, out_k, out_v = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(c.chunk_workspace_bytes(splits, 24, 20, 390, 200, 4), 16), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step(out, out_k, out_v):
        c.chunk_attention(q, k, v, case.cu_new, 20, out, SCALE, ws, splits, 390, window=200, sinks=4)
        c.append_chunk(k, v, case.cu_new, 20, token_class=cls)
        c.read_tokens(start, case.cu_new, 20, out_k, out_v)

    first = held(c)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out, out_k, out_v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(out, out_k, out_v)
    put_back(c, first)
    lens = [300, 7]
    for _ in range(3):
        q.copy_(to_dev(bits_of(rng.standard_normal(q.shape))).view(torch.bfloat16))
        k.copy_(to_dev(bits_of(rng.standard_normal(k.shape))).view(torch.bfloat16))
        v.copy_(to_dev(bits_of(rng.standard_normal(v.shape))).view(torch.bfloat16))
        start.copy_(torch.tensor(lens, dtype=torch.int32))
        before = held(c)
        for t in (out, out_k, out_v):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        after = held(c)
        put_back(c, before)
        one = [torch.zeros_like(t) for t in (out, out_k, out_v)]
        step(*one)
        torch.cuda.synchronize()
        for a, b in zip((out, out_k, out_v), one):
            assert torch.equal(a, b) and not torch.any(a == 7.0)
        for name, t in after.items():
            assert torch.equal(t, c.buffers[name]), name
        lens = [n + m for n, m in zip(lens, new)]
        assert c.seq_len()[:2].tolist() == lens
        # and the attention is that of the reference
        case.lens, case.kn, case.vn, case.q = ([n - m for n, m in zip(lens, new)],
                                               *(t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (k, v, q)))
        put_back(c, before)
        case.check(one[0].float().cpu().numpy().astype(np.float64), 200, 4)
        put_back(c, after)
    assert c.error() == 0


@pytest.mark.parametrize("kind", ["stream", "handle", "default"])
def test_reset_on_a_stream(kind):
    """reset() given a stream takes its turn there: behind an append that waits, before the next one."""
    case = Case(4, [50, 9], [20, 4], seed=320)
    side = torch.cuda.default_stream() if kind == "default" else torch.cuda.Stream()
    other = torch.cuda.Stream()
    stream = side if kind == "stream" else side.cuda_stream
    k, v, kn, vn = (to_dev(a) for a in (case.k, case.v, case.kn, case.vn))
    torch.cuda.synchronize()
    with torch.cuda.stream(other):                            # the current stream is not the one that is given
        for _ in range(3):
            with torch.cuda.stream(side):
                torch.cuda._sleep(20000000)                   # about 10 ms: a clear that did not wait would be long past
            case.cache.append_chunk(k, v, case.cu, 50, stream=stream)
            case.cache.reset(stream=stream)
            case.cache.append_chunk(kn, vn, case.cu_new, 20, stream=stream)
            torch.cuda.synchronize()
            assert case.cache.seq_len()[:2].tolist() == [20, 4]
            case.cache.reset(stream=stream)
    torch.cuda.synchronize()
    assert case.cache.seq_len()[:2].tolist() == [0, 0] and case.cache.error() == 0
