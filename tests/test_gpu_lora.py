"""GPU tests of q8_lora against its definition in 64 bits."""
import time

import numpy as np
import pytest

import oracle
from tests import layer_plain

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def typed(rng, shape, name, size=1.0):
    return torch.from_numpy((size * rng.standard_normal(shape)).astype(np.float32)).to(DT[name])


class Case:
    def __init__(self, seed, n, n_in, n_out, rank, adapters, kind, x="f32", ragged=True, base=True, ids=None):
        rng = np.random.default_rng(seed)
        self.a, self.b = typed(rng, (adapters, rank, n_in), kind, n_in ** -0.5), typed(rng, (adapters, n_out, rank), kind, 0.05)
        self.ranks = rng.integers(0, rank + 1, adapters) if ragged else np.full(adapters, rank)
        self.ranks[-1] = rank
        self.scales = rng.uniform(-2, 2, adapters).astype(np.float32)
        self.ids = rng.integers(-1, adapters, n) if ids is None else np.asarray(ids)
        xv = rng.standard_normal((n, n_in)).astype(np.float32) * (1 + 19 * (rng.uniform(size=(n, n_in)) < 0.01)).astype(np.float32)
        if x == "q8":
            blocks = oracle.get().quantize(xv)
            self.x = torch.from_numpy(blocks)
            raw = blocks.reshape(n, -1, 34)
            d = np.ascontiguousarray(raw[:, :, :2]).view(np.float16).astype(np.float64)
            self.xv = (np.ascontiguousarray(raw[:, :, 2:]).view(np.int8) * d).reshape(n, n_in)
        else:
            self.x = torch.from_numpy(xv).to(DT[x])
            self.xv = self.x.double().numpy()
        self.base = rng.standard_normal((n, n_out)).astype(np.float32) if base else None
        # what lies behind an adapter's rank is never used
        for k, r in enumerate(self.ranks):
            self.a[k, r:] = float("nan")
            self.b[k, :, r:] = float("inf")
        self.plain = layer_plain.lora(self.xv, np.nan_to_num(self.a.double().numpy(), posinf=0.0), np.nan_to_num(self.b.double().numpy(), posinf=0.0),
                                      self.ids, self.ranks, self.scales, self.base)

    def call(self, q8, **kw):
        args = dict(ranks=i32(self.ranks), scales=torch.from_numpy(self.scales).to(DEV),
                    base=None if self.base is None else torch.from_numpy(self.base).to(DEV))
        args.update(kw)
        return q8.lora(self.x.to(DEV), self.a.to(DEV), self.b.to(DEV), i32(self.ids), **args)

    def check(self, got):
        want, bound = self.plain
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= bound).all(), f"error {err.max()} at {np.unravel_index((err / bound).argmax(), err.shape)}, {(err / bound).max()} of the bound"


SIZES = [
    # tokens, in, out, rank, adapters
    (1, 32, 1, 8, 1), (1, 4096, 4096, 16, 3), (2, 1024, 300, 8, 2), (5, 96, 7, 24, 4), (9, 2080, 1025, 64, 3),
    (16, 1024, 4100, 32, 40), (33, 512, 64, 128, 5), (64, 256, 2048, 16, 64), (100, 992, 515, 40, 7), (129, 512, 384, 16, 2), (193, 512, 384, 16, 2),
    (257, 1024, 130, 64, 3), (300, 96, 2050, 8, 300), (700, 2048, 257, 128, 9), (1025, 320, 640, 48, 1), (300, 512, 388, 128, 3),
    (200, 4096, 1000, 72, 2), (450, 256, 4108, 16, 2), (513, 64, 20, 64, 1)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("kind,x", [("bf16", "f32"), ("f16", "f32"), ("bf16", "q8"), ("f16", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
def test_against_64_bits(q8, size, kind, x):
    n, n_in, n_out, rank, adapters = size
    c = Case(sum(size), n, n_in, n_out, rank, adapters, kind, x)
    c.check(c.call(q8))
    assert q8.q8_last_error() == 0


@pytest.mark.parametrize("n", [1, 3, 40, 200])
@pytest.mark.parametrize("ids", ["none", "one", "sorted", "turns"])
def test_who_has_which_adapter(q8, n, ids):
    pick = {"none": np.full(n, -1), "one": np.full(n, 2), "sorted": np.arange(n) * 4 // n, "turns": np.arange(n) % 4}[ids]
    c = Case(n, n, 256, 200, 16, 4, "bf16", ids=pick)
    got = c.call(q8)
    c.check(got)
    if ids == "none":
        assert torch.equal(got.cpu(), torch.from_numpy(c.base))
        assert not c.call(q8, base=None).any()


def test_tiles_and_groups_of_many_tokens(q8):
    """More tokens than one round of the ordering, adapters with many, few and single tokens: so many tiles that small shares go
    in groups; and a full list of adapters."""
    rng = np.random.default_rng(7)
    n = 5300
    ids = np.concatenate([rng.integers(0, 3, 4000), 3 + np.arange(600) // 15, 43 + np.arange(300) // 20, 58 + np.arange(200), np.full(200, -1)])
    c = Case(7, n, 64, 136, 16, 258, "bf16", ids=rng.permutation(ids))
    c.check(c.call(q8))
    c = Case(8, 400, 32, 12, 8, 16384, "f16", "bf16")
    c.check(c.call(q8))
    assert q8.q8_last_error() == 0


@pytest.mark.parametrize("n", [50, 130])
def test_rows_far_apart(q8, n):
    """Rows whose offsets pass 32 bits."""
    stride = 1 << (25 if n < 100 else 24)
    c = Case(n, n, 128, 256, 40, 3, "bf16")
    x = torch.empty(n * stride, device=DEV).view(n, stride)[:, :128]
    out = torch.empty(n * stride, device=DEV).view(n, stride)[:, 64:320]
    x.copy_(c.x), out.copy_(torch.from_numpy(c.base))
    c.check(c.call(q8, base=out, out=out) if n < 100 else
            q8.lora(x, c.a.to(DEV), c.b.to(DEV), i32(c.ids), i32(c.ranks), torch.from_numpy(c.scales).to(DEV), out, out))


def test_graphs_outlive_a_larger_call(q8):
    """Two captured calls and a later one that needs more scratch: the replays still give their results."""
    graphs = []
    for n in (200, 333):
        c = Case(n, n, 256, 200, 16, 3, "bf16")
        x, a, b, ids, ranks = c.x.to(DEV), c.a.to(DEV), c.b.to(DEV), i32(c.ids), i32(c.ranks)
        scales, base = torch.from_numpy(c.scales).to(DEV), torch.from_numpy(c.base).to(DEV)
        q8.lora(x, a, b, ids, ranks, scales, base)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = q8.lora(x, a, b, ids, ranks, scales, base)
        graphs.append((c, graph, out, (x, a, b, ids, ranks, scales, base)))
    big = Case(1, 6000, 32, 64, 128, 2, "f16")
    big.check(big.call(q8))
    for c, graph, out, _ in graphs + graphs[::-1]:
        out.zero_()
        graph.replay()
        c.check(out)


@pytest.mark.parametrize("n", [2, 250])
def test_without_base_scales_ranks(q8, n):
    c = Case(n, n, 512, 260, 16, 3, "f16", ragged=False, base=False)
    c.check(c.call(q8))
    c.scales = np.ones(3, np.float32)
    c.plain = layer_plain.lora(c.xv, c.a.double().numpy(), c.b.double().numpy(), c.ids, c.ranks, c.scales, None)
    c.check(c.call(q8, scales=None, ranks=None))


@pytest.mark.parametrize("n", [3, 140, 240])
def test_strides_and_in_place(q8, n):
    """Adapters of two projections in one pool each, x and out slices of wider tensors, out on base."""
    c = Case(n, n, 256, 192, 16, 3, "bf16")
    a, b = torch.full((3, 2, 16, 256), float("nan"), dtype=torch.bfloat16, device=DEV), torch.full((3, 2, 192, 16), float("nan"), dtype=torch.bfloat16, device=DEV)
    a[:, 1], b[:, 1] = c.a.to(DEV), c.b.to(DEV)
    x = torch.full((n, 1024), float("nan"), device=DEV)
    x[:, 512:768] = c.x.to(DEV)
    out = torch.full((n, 1000), 7.0, device=DEV)
    out[:, 400:592] = torch.from_numpy(c.base).to(DEV)
    part = out[:, 400:592]
    q8.lora(x[:, 512:768], a[:, 1], b[:, 1], i32(c.ids), ranks=i32(c.ranks), scales=torch.from_numpy(c.scales).to(DEV), base=part, out=part)
    c.check(part)
    assert (out[:, :400] == 7).all() and (out[:, 592:] == 7).all()
    wide = torch.full((n, 195), 7.0, device=DEV)                       # rows that are not 16-byte aligned
    q8.lora(x[:, 512:768], a[:, 1], b[:, 1], i32(c.ids), ranks=i32(c.ranks), scales=torch.from_numpy(c.scales).to(DEV),
            base=torch.from_numpy(c.base).to(DEV), out=wide[:, :192])
    c.check(wide[:, :192])
    assert (wide[:, 192:] == 7).all()


@pytest.mark.parametrize("n", [6, 250])
def test_bad_ids_and_ranks(q8, n):
    c = Case(n, n, 128, 96, 16, 4, "bf16", ragged=False)
    c.ids[1], c.ids[n - 2] = 4, 2 ** 31 - 1
    c.plain = layer_plain.lora(c.xv, c.a.double().numpy(), c.b.double().numpy(), c.ids, c.ranks, c.scales, c.base)
    c.check(c.call(q8))
    assert q8.q8_last_error() == q8.Q8_ERANGE
    c.ids = np.arange(n) % 4
    c.ranks = np.array([17, -3, 16, 5])
    c.plain = layer_plain.lora(c.xv, c.a.double().numpy(), c.b.double().numpy(), c.ids, c.ranks, c.scales, c.base)
    c.check(c.call(q8))
    assert q8.q8_last_error() == q8.Q8_ERANGE and q8.q8_last_error() == 0


@pytest.mark.parametrize("n", [8, 160, 260])
def test_values_that_are_not_finite_stay_in_their_row(q8, n):
    c = Case(n, n, 256, 130, 16, 2, "f16", ids=np.arange(n) % 3 - 1)
    clean = c.call(q8)
    c.x[0, 3] = float("nan")                       # no adapter: x does not count
    c.x[4, 5], c.x[n - 1, 0] = float("nan"), float("inf")
    got = c.call(q8)
    bad = [i for i in (4, n - 1) if c.ids[i] >= 0 and c.ranks[c.ids[i]] > 0]
    keep = [i for i in range(n) if i not in (4, n - 1)]
    assert torch.equal(got[keep], clean[keep])
    for i in bad:
        assert not torch.isfinite(got[i]).all()


@pytest.mark.parametrize("n", [7, 600])
def test_same_bits_every_time_and_captured(q8, n):
    c = Case(n, n, 1024, 520, 32, 5, "bf16")
    first = c.call(q8)
    x, a, b, ids, ranks = c.x.to(DEV), c.a.to(DEV), c.b.to(DEV), i32(c.ids), i32(c.ranks)
    scales, base = torch.from_numpy(c.scales).to(DEV), torch.from_numpy(c.base).to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = q8.lora(x, a, b, ids, ranks, scales, base)
    for _ in range(3):
        graph.replay()
        assert torch.equal(out, first)
    perm = torch.randperm(n, device=DEV)           # a token's result does not depend on its neighbours
    moved = q8.lora(x[perm], a, b, ids[perm], ranks, scales, base[perm])
    assert torch.equal(moved, first[perm])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = q8.lora(x, a, b, ids, ranks, scales, base)
    side.synchronize()
    assert torch.equal(other, first)


def test_beside_the_projection(q8):
    """In place on what q8_matmul_q gave, from the same blocks, for decoding and prompt sizes."""
    import inputs
    w = torch.from_numpy(inputs.weights(320, 512, seed=3)).to(DEV)
    for n in (4, 200):
        c = Case(n, n, 512, 320, 16, 3, "bf16", x="q8")
        out = q8.matmul_q(w, c.x.to(DEV), 512, 320)
        c.base = out.cpu().numpy()
        c.plain = layer_plain.lora(c.xv, np.nan_to_num(c.a.double().numpy()), np.nan_to_num(c.b.double().numpy(), posinf=0.0), c.ids, c.ranks, c.scales, c.base)
        got = q8.lora(c.x.to(DEV), c.a.to(DEV), c.b.to(DEV), i32(c.ids), ranks=i32(c.ranks), scales=torch.from_numpy(c.scales).to(DEV),
                      base=out, out=out)
        assert got.data_ptr() == out.data_ptr()
        c.check(out)


def test_helper_refusals(q8):
    x, a, b = torch.randn(3, 64, device=DEV), torch.zeros(2, 8, 64, device=DEV).half(), torch.zeros(2, 40, 8, device=DEV).half()
    ids = i32([0, 1, 0])
    for bad in (lambda: q8.lora(x, a, b.bfloat16(), ids), lambda: q8.lora(x, a.float(), b.float(), ids), lambda: q8.lora(x, a, b, ids[:2]),
                lambda: q8.lora(x, a, b, ids.long()), lambda: q8.lora(x[:, :32], a, b, ids), lambda: q8.lora(x, a, b[:1], ids),
                lambda: q8.lora(x, a, b, ids, base=x), lambda: q8.lora(x, a, b, ids, ranks=i32([1])), lambda: q8.lora(x.cpu(), a, b, ids),
                lambda: q8.lora(x, a[:, :, ::2], b, ids), lambda: q8.lora(x, a[:, :5], b[:, :, :5].contiguous(), ids),
                lambda: q8.lora(x, a, b, ids, out=torch.empty(3, 39, device=DEV))):
        with pytest.raises((TypeError, ValueError, q8.Q8Error)):
            bad()
    assert q8.lora(x[:0], a, b, ids[:0]).shape == (0, 40)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_adapters_expired_wait_and_recovery(q8, dtype):
    """The first tcgen05 kernel of q8_lora with its copies withheld: its clusters end with an error, and the next call is right."""
    x = torch.randn(700, 1024, device=DEV).to(dtype)
    a, b = (torch.randn(2, 16, 1024, device=DEV) / 32).bfloat16(), torch.randn(2, 256, 16, device=DEV).bfloat16()
    ids = (torch.arange(700, device=DEV) % 2).int()
    want = q8.lora(x, a, b, ids)
    assert q8.q8_last_error() == 0
    q8.q8_debug_expire_waits(1, 200_000)   # 0.2 ms instead of the normal 2 s
    try:
        t0 = time.perf_counter()
        q8.lora(x, a, b, ids)
        assert q8.q8_last_error() == q8.Q8_ETIMEOUT
        assert time.perf_counter() - t0 < 1.5, "an expired wait did not end its kernel promptly"
    finally:
        q8.q8_debug_expire_waits(0, 0)
    assert torch.equal(q8.lora(x, a, b, ids), want)
    assert q8.q8_last_error() == 0
