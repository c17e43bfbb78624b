"""Graphs of captured calls keep working when later calls need more scratch than there was at the capture."""
import ctypes

import numpy as np
import pytest

import inputs

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_matmul_gb300 import build
    build.build()
    import q8_quantized_matmul_gb300 as m
    torch.cuda.set_device(0)
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def long_decode(q8, lens, heads, kv, dim):
    """A decode call whose sequences are split over many CTAs, so that pieces and counters are used."""
    page, n_pages = 64, sum(-(-n // 64) for n in lens)
    cache = q8.KVCache.empty(q8.Q8_TYPE_BF16, 1, n_pages, page, kv, dim)
    for pool in (cache.k, cache.v):
        pool.view(torch.bfloat16).normal_()
    table, at = np.full((len(lens), max(-(-n // page) for n in lens)), -1, np.int32), 0
    for i, n in enumerate(lens):
        table[i, :-(-n // page)] = np.arange(at, at + -(-n // page))
        at += -(-n // page)
    q = torch.randn(len(lens), heads, dim, device=DEV).bfloat16()
    t, n = torch.from_numpy(table).to(DEV), i32(lens)
    return lambda: q8.attn_decode(q, cache, 0, t, n)


def grow(q8):
    """Calls that need more of every buffer than the captured ones, and new owners for whatever was given back."""
    before = q8.q8_scratch_bytes()
    n, kv = 40_000, 16
    cache = q8.KVCache.empty(q8.Q8_TYPE_BF16, 1, 2, 16, kv, 64)
    q = torch.zeros(n, kv, 64, device=DEV, dtype=torch.bfloat16)
    q8.attn_decode(q, cache, 0, torch.zeros(n, 1, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV))
    W = torch.from_numpy(inputs.weights(512, 8192, seed=1)).to(DEV)
    q8.matmul(W, torch.randn(8192, 8192, device=DEV), 512)
    torch.cuda.synchronize()
    assert q8.q8_scratch_bytes() > before + (64 << 20)
    return [torch.full((1 << 20,), 0x55555555, dtype=torch.int32, device=DEV) for _ in range(256)]


@pytest.mark.parametrize("mode", ["global", "relaxed"])
def test_graphs_outlive_growing_buffers(q8, mode):
    torch.cuda.synchronize()
    q8.q8_release()
    W = torch.from_numpy(inputs.weights(1024, 2048, seed=2)).to(DEV)
    x = torch.randn(64, 2048, device=DEV)
    start = i32([0, *np.cumsum([70] * 40)])
    pq, pk = (torch.randn(2800, h, 64, device=DEV).bfloat16() for h in (8, 2))
    calls = {"mma.sync decode": long_decode(q8, [20000, 700], 8, 2, 128), "tcgen05 decode": long_decode(q8, [6000, 90], 24, 1, 512),
             "prompt": lambda: q8.attn_prompt(pq, pk, pk, start), "matmul": lambda: q8.matmul(W, x, 1024)}
    refs = {name: f().clone() for name, f in calls.items()}          # sizes the buffers
    held = q8.q8_scratch_bytes()
    graphs = {}
    for name, f in calls.items():
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode=mode):
            out = f()
        graphs[name] = (g, out)
    assert q8.q8_scratch_bytes() == held
    others = grow(q8)
    for _ in range(3):
        for name, (g, out) in graphs.items():
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, refs[name]), name
        for name, f in calls.items():                                 # and calls beside them
            assert torch.equal(f(), refs[name]), name
    assert all(bool((o == 0x55555555).all()) for o in others) and q8.q8_last_error() == 0
    del graphs, g
    torch.cuda.synchronize()
    q8.q8_release()
    assert q8.q8_scratch_bytes() == 0


def test_counters_made_within_a_capture(q8):
    """A relaxed capture may allocate; what it makes serves the calls before the graph's first replay too."""
    decode = long_decode(q8, [20000, 700], 8, 2, 128)
    ref = decode().clone()
    torch.cuda.synchronize()
    q8.q8_release()
    torch.cuda.empty_cache()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        out = decode()
    # no clearing in the graph: the calls before its replay would do without
    cu, n, kind = ctypes.CDLL("libcuda.so.1"), ctypes.c_size_t(), ctypes.c_int()
    graph = ctypes.c_void_p(g.raw_cuda_graph())
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        assert kind.value == 0, "a node that is not a kernel"
    g.instantiate()
    for _ in range(3):
        assert torch.equal(decode(), ref)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    assert q8.q8_last_error() == 0
    del g
    torch.cuda.synchronize()
    q8.q8_release()
