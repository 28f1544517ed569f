"""ff_attention_noalloc recorded into a stream capture.

A capture is one of the places the entry point exists for.  The recorded call
has to give the bits of the direct one, at every replay and for what its input
buffers hold then, with and without key-range splits.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


@pytest.mark.parametrize("nq,nk,heads,d", [(1, 1, 1, 64), (100, 130, 3, 64), (256, 8192, 2, 128), (1000, 1560, 12, 128)])
def test_captured_call_matches_the_direct_one(ff, nq, nk, heads, d):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(nq + nk)
    draw = lambda n: torch.randn(n, heads, d, device=dev, generator=gen, dtype=torch.float32).to(torch.bfloat16)
    q, k, v = draw(nq), draw(nk), draw(nk)
    want, got = torch.empty_like(q), torch.empty_like(q)
    ff.attention_noalloc(q, k, v, want)  # sets the device up, before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ff.attention_noalloc(q, k, v, got, stream=torch.cuda.current_stream())
    for turn in range(3):
        if turn:
            for x, n in ((q, nq), (k, nk), (v, nk)):
                x.copy_(draw(n))
            ff.attention_noalloc(q, k, v, want)
        got.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want.view(torch.int16), got.view(torch.int16))
