"""Calls on the 8-bit cache one after the other, on several streams and in captured graphs: each gives
what it gives alone."""
import pytest
import torch

from tests.cache_util import make, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("Hq,Hkv,D,block,Sq", [(8, 2, 128, 16, 1), (16, 16, 64, 64, 1), (4, 1, 128, 32, 5), (32, 4, 64, 128, 9)])
def test_attention_between_writes_that_raise_the_scales(Hq, Hkv, D, block, Sq):
    """Attention, write, attention, read ... without a wait in between: every call sees the scales, codes and
    table of the write before it.  The expected results are the same calls with a wait after each."""
    B, n, steps = 5, 1100, 24
    cache, table = make(B, Hkv, D, block, n, seed=31)
    lens = [n, n - 7, 300, block + 3, 9]
    fill_k, fill_v = rows((B, Hkv, n, D), 1), rows((B, Hkv, n, D), 2, 0.5)
    # the last tokens once more, each time larger, so that their block's scale grows and its other codes move
    grow = [2.0 ** (s % 12) for s in range(steps)]
    k = [(rows((B, Hkv, 3, D), 10 + s).float() * grow[s]).bfloat16().cuda() for s in range(steps)]
    q = rows((B, Hq, Sq, D), 5).cuda()

    def run(wait):
        cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        cache.write(fill_k.cuda(), fill_v.cuda(), new_lens=cache.seq_lens.clone())
        got = []
        for s in range(steps):
            got.append(cache.attention(q))
            wait()
            cache.write(k[s], k[s])
            wait()
            got.append(cache.attention(q))
            wait()
            got.append(cache.read(20, first=max(0, lens[3] - 20)))
            wait()
        torch.cuda.synchronize()
        return got

    want = run(torch.cuda.synchronize)
    for _ in range(4):
        for i, (a, b) in enumerate(zip(run(lambda: None), want)):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), i


def test_handles_of_the_default_stream():
    """0 and 1 are the default stream's handles: calls on it run behind what it holds already."""
    cache, _ = make(2, 2, 64, 32, 2000, seed=33)
    k, q = rows((2, 2, 2000, 64), 1).cuda(), rows((2, 4, 1, 64), 2).cuda()
    cache.seq_lens.fill_(2000)
    cache.write(k, k)
    want = cache.attention(q)
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    for handle in (0, 1):
        with cache._on(handle) as st:
            assert st == default.cuda_stream and torch.cuda.current_stream() == default
        late = torch.zeros_like(q)
        torch.cuda.synchronize()
        with torch.cuda.stream(default):
            torch.cuda._sleep(20_000_000)  # some milliseconds
            late.copy_(q)
        with torch.cuda.stream(torch.cuda.Stream()):
            got = cache.attention(late, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_calls_replayed_at_once():
    """Graphs of attention calls of different shapes, split over all blocks and joined, replayed on streams of their
    own without a wait in between: each has its own workspace."""
    made = []
    for i, (lens, Hq, Hkv, Sq) in enumerate((([20000, 300], 8, 2, 1), ([9000, 8000], 4, 2, 9), ([16000, 5], 32, 2, 1),
                                             ([5000, 4000], 16, 2, 16))):
        cache, _ = make(2, Hkv, 128, 64, max(lens), seed=41 + i)
        k = rows((2, Hkv, max(lens), 128), 50 + i).cuda()
        cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        cache.write(k, k, new_lens=cache.seq_lens.clone())
        q = rows((2, Hq, Sq, 128), 60 + i).cuda()
        want = cache.attention(q, check_status=True)
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            got = cache.attention(q)
        made.append((graph, stream, got, want, cache, q, k))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, _, got, *_ in made:
            got[0].fill_(3), got[1].fill_(3)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, stream, *_ in made:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for i, (_, _, got, want, *_) in enumerate(made):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
