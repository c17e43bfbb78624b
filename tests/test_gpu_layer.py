"""A decoder layer's calls in a row, as a server makes them: norms on the residual path, projections with adapters, cache, its
reading back, attention.  Each new call is held to its plain form on the very inputs that it got."""
import numpy as np
import pytest

import inputs
import oracle
from tests import layer_plain

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"
DIM, HEADS, KV, HEAD, PAGE, EPS = 512, 4, 2, 64, 16, 1e-6
WIDE = (HEADS + 2 * KV) * HEAD


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


class Layer:
    def __init__(self, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
        self.wq, self.wo = (torch.from_numpy(inputs.weights(rows, cols, seed=seed + s, d_lo=3e-4, d_hi=5.5e-4)).to(DEV)
                            for rows, cols, s in ((WIDE, DIM, 1), (DIM, HEADS * HEAD, 2)))
        self.aq, self.bq = (rand(3, 16, DIM) * DIM ** -0.5).bfloat16(), (rand(3, WIDE, 16) * 0.05).bfloat16()
        self.ao, self.bo = (rand(3, 16, HEADS * HEAD) * 0.06).bfloat16(), (rand(3, DIM, 16) * 0.05).bfloat16()
        self.ranks, self.scales = i32([16, 5, 9]), rand(3)
        self.gp, self.gn, self.gate = 1 + 0.1 * rand(DIM), 1 + 0.1 * rand(DIM), rand(DIM)

    def __call__(self, q8, h, y, adapter_of, attend):
        """-> everything on the way."""
        xq, h1 = q8.residual_norm(h, y, self.gn, EPS, gamma_post=self.gp, post=True, gate=self.gate)
        bare = q8.matmul_q(self.wq, xq, DIM, WIDE)
        qkv = q8.lora(xq, self.aq, self.bq, adapter_of, self.ranks, self.scales, bare)
        o = attend(qkv.view(-1, HEADS + 2 * KV, HEAD))
        out = q8.matmul_q(self.wo, o, HEADS * HEAD, DIM)
        mixed = q8.lora(o, self.ao, self.bo, adapter_of, self.ranks, self.scales, out)
        xq2, h2 = q8.residual_norm(h1, mixed, self.gn, EPS, residual_scale=0.5)
        return dict(xq=xq, h1=h1, bare=bare, qkv=qkv, o=o, out=out, mixed=mixed, xq2=xq2, h2=h2)

    def check(self, r, h, y, adapter_of):
        num = lambda t: t.float().cpu().numpy()
        quantised = lambda x: oracle.get().quantize(np.ascontiguousarray(x))

        def values(blocks):
            raw = blocks.cpu().numpy().reshape(blocks.shape[0], -1, 34)
            d = np.ascontiguousarray(raw[:, :, :2]).view(np.float16).astype(np.float64)
            return (np.ascontiguousarray(raw[:, :, 2:]).view(np.int8) * d).reshape(blocks.shape[0], -1)
        n, h1 = layer_plain.residual_norm(num(h), num(y), num(self.gn), EPS, num(self.gp), True, num(self.gate))
        assert np.array_equal(num(r["h1"]), h1) and np.array_equal(r["xq"].cpu().numpy(), quantised(n))
        for x, a, b, base, got in ((r["xq"], self.aq, self.bq, r["bare"], r["qkv"]), (r["o"], self.ao, self.bo, r["out"], r["mixed"])):
            want, bound = layer_plain.lora(values(x), a.double().cpu().numpy(), b.double().cpu().numpy(), adapter_of.cpu().numpy(),
                                           self.ranks.cpu().numpy(), num(self.scales), num(base))
            assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
        n, h2 = layer_plain.residual_norm(num(r["h1"]), num(r["mixed"]), num(self.gn), EPS, scale=0.5)
        assert np.array_equal(num(r["h2"]), h2) and np.array_equal(r["xq2"].cpu().numpy(), quantised(n))


def test_prompts_in_parts(q8):
    """Two requests' prompts, the second part over what the cache gives back."""
    layer, g = Layer(), torch.Generator(device=DEV).manual_seed(3)
    lens, cut = [90, 37], [40, 20]
    cache = q8.KVCache.empty(q8.Q8_TYPE_BF16, 1, 12, PAGE, KV, HEAD)
    table = i32([[3, 1, 8, 0, 10, 2], [7, 5, 11, 9, 4, 6]])
    both = []
    for first, last in (([0, 0], cut), (cut, lens)):
        n = [b - a for a, b in zip(first, last)]
        h, y = (torch.randn(sum(n), DIM, generator=g, device=DEV) for _ in range(2))
        pos = i32(np.concatenate([np.arange(a, b) for a, b in zip(first, last)]))
        seq = i32(np.repeat([0, 1], n))
        start, k_start = i32(np.cumsum([0] + n)), i32(np.cumsum([0] + last))
        kept = {}

        def attend(qkv):
            q, k, v = q8.kv_append(cache, 0, qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:], pos, seq, table, want_kv=True)
            kept["k"], kept["v"] = k, v
            kr, vr = q8.kv_read(cache, 0, table, k_start, sum(last))
            for x, name in ((kr, "k"), (vr, "v")):
                at = np.concatenate([np.arange(s, s + b) for s, b in zip(np.cumsum([0] + last[:-1]), last)])
                new = np.concatenate([np.arange(s + a, s + b) for s, a, b in zip(np.cumsum([0] + last[:-1]), first, last)])
                assert len(at) == sum(last) and torch.equal(x[torch.from_numpy(new).to(DEV)], kept[name])
            return q8.attn_prompt(q, kr, vr, start, k_start, out_type=q8.Q8_TYPE_Q8_0).view(sum(n), -1)
        adapter_of = i32(np.repeat([2, -1], n))
        r = layer(q8, h, y, adapter_of, attend)
        assert q8.q8_last_error() == 0
        layer.check(r, h, y, adapter_of)
        both.append((kept["k"], kept["v"]))
    # all that was cached, in order
    k, v = q8.kv_read(cache, 0, table, i32([0, 90, 127]), 127)
    for x, i in ((k, 0), (v, 1)):
        a, b = both[0][i], both[1][i]
        assert torch.equal(x, torch.cat([a[:40], b[:50], a[40:], b[50:]]))


def test_a_decoding_step_captured(q8):
    """One new token each of 5 sequences, the whole layer in a graph: the replay has the bits of the eager calls."""
    layer, g = Layer(5), torch.Generator(device=DEV).manual_seed(4)
    cache = q8.KVCache.empty(q8.Q8_TYPE_Q8_0, 1, 20, PAGE, KV, HEAD)
    table, lens = i32(np.arange(20).reshape(5, 4)), i32([1, 17, 40, 64, 3])
    for pool in (cache.k, cache.v):
        pool[..., :].zero_()
    pos, seq, adapter_of = lens - 1, i32(np.arange(5)), i32([0, 2, 2, -1, 1])
    h, y = (torch.randn(5, DIM, generator=g, device=DEV) for _ in range(2))

    def attend(qkv):
        q = q8.kv_append(cache, 0, qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:], pos, seq, table)
        return q8.attn_decode(q, cache, 0, table, lens, out_type=q8.Q8_TYPE_Q8_0).view(5, -1)
    layer(q8, h, y, adapter_of, attend)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = layer(q8, h, y, adapter_of, attend)
    for _ in range(2):
        h.normal_(generator=g), y.normal_(generator=g)
        graph.replay()
        again = layer(q8, h, y, adapter_of, attend)
        layer.check(again, h, y, adapter_of)
        assert all(torch.equal(r[k], again[k]) for k in r)
    assert q8.q8_last_error() == 0
