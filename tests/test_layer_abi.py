"""Host-side validation of the calls around a layer's projections and of the cache's reading back (no GPU): bad
arguments are refused before any CUDA call, empty work is a no-op."""
import ctypes

import pytest

A, B, C = 0x10000, 0x20000, 0x30000     # 16-byte aligned fake addresses, never dereferenced


@pytest.fixture(scope="module")
def q8():
    from q8_quantized_matmul_gb300 import build
    build.build()
    import q8_quantized_matmul_gb300 as m
    return m


NAN, INF = float("nan"), float("inf")


def norm(q8, **kw):
    a = dict(n_out=A, n_type=8, h_out=B, h_out_stride=64, h=B, h_type=0, h_stride=64, y=C, y_type=0, y_stride=64, post=1,
             gamma_post=A, gate=A, gate_stride=0, scale=1.0, gamma_next=A, eps=1e-6, dim=64, n_tok=3)
    a.update(kw)
    return q8.lib.q8_residual_norm(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    ("EINVAL", dict(dim=0)), ("EINVAL", dict(dim=48)), ("EINVAL", dict(dim=32800, h_stride=32800, h_out_stride=32800, y_stride=32800)),
    ("EINVAL", dict(n_tok=1 << 31)), ("EINVAL", dict(h_type=8)), ("EINVAL", dict(y_type=3)), ("EINVAL", dict(n_type=4)),
    ("EINVAL", dict(eps=0.0)), ("EINVAL", dict(eps=-1.0)), ("EINVAL", dict(eps=NAN)), ("EINVAL", dict(eps=INF)),
    ("EINVAL", dict(scale=NAN)), ("EINVAL", dict(scale=INF)), ("EINVAL", dict(n_out=None, h_out=None)), ("EINVAL", dict(h=None)),
    ("EINVAL", dict(y=None)), ("EINVAL", dict(h_stride=56)), ("EINVAL", dict(y_stride=56)), ("EINVAL", dict(h_out_stride=56)),
    ("EINVAL", dict(h_out_stride=72)), ("EINVAL", dict(gate_stride=60)), ("EINVAL", dict(y_stride=1 << 33)),
    ("EALIGN", dict(n_out=A + 8)), ("EALIGN", dict(h=B + 4, h_out=C)), ("EALIGN", dict(y=C + 8)), ("EALIGN", dict(gate=A + 4)),
    ("EALIGN", dict(gamma_next=A + 4)), ("EALIGN", dict(y_stride=68)), ("EALIGN", dict(gate_stride=66)), ("OK", dict(n_tok=0))])
def test_residual_norm_refusals(q8, want, kw):
    assert norm(q8, **kw) == getattr(q8, "Q8_" + want)


def lora(q8, fields=None, **kw):
    ad = dict(a=A, b=B, a_stride=8 * 64, b_stride=8 * 40, ranks=A, scales=A, in_dim=64, out_dim=40, n_adapters=3, max_rank=8, type=2)
    ad.update(fields or {})
    s = q8.AdaptersStruct(*(ad[n] for n, _ in q8.AdaptersStruct._fields_))
    a = dict(out=A, out_stride=40, base=B, base_stride=40, x=C, x_type=0, x_stride=64, adapters=s, adapter_of=A, n_tok=5)
    a.update(kw)
    return q8.lib.q8_lora(*a.values(), None)


def test_struct_matches_the_header(q8):
    assert ctypes.sizeof(q8.AdaptersStruct) == 80


@pytest.mark.parametrize("want,ad,kw", [
    ("EINVAL", dict(a=None), {}), ("EINVAL", dict(b=None), {}), ("EINVAL", dict(a_stride=504), {}), ("EINVAL", dict(b_stride=312), {}),
    ("EALIGN", dict(a_stride=516), {}), ("EALIGN", dict(b_stride=324), {}), ("EINVAL", dict(in_dim=48), {}), ("EINVAL", dict(in_dim=0), {}),
    ("EINVAL", dict(n_adapters=0), {}), ("EINVAL", dict(n_adapters=16385), {}), ("EINVAL", dict(max_rank=0), {}),
    ("EINVAL", dict(max_rank=12), {}), ("EINVAL", dict(max_rank=136), {}), ("EINVAL", dict(type=0), {}), ("EINVAL", dict(type=8), {}),
    ("EALIGN", dict(a=A + 8), {}), ("EALIGN", dict(b=B + 2), {}), ("EALIGN", dict(ranks=A + 2), {}), ("EALIGN", dict(scales=A + 1), {}),
    ("EINVAL", {}, dict(adapters=None)), ("EINVAL", {}, dict(out=None)), ("EINVAL", {}, dict(x=None)), ("EINVAL", {}, dict(adapter_of=None)),
    ("EINVAL", {}, dict(out_stride=39)), ("EINVAL", {}, dict(base_stride=39)), ("EINVAL", {}, dict(out=B, out_stride=44)),
    ("EINVAL", {}, dict(x_type=3)), ("EINVAL", {}, dict(x_stride=56)), ("EINVAL", {}, dict(x_type=8, x_stride=96)),
    ("EALIGN", {}, dict(x_stride=68)), ("EALIGN", {}, dict(out=A + 4)), ("EALIGN", {}, dict(base=B + 8)), ("EALIGN", {}, dict(x=C + 8)),
    ("EALIGN", {}, dict(adapter_of=A + 2)), ("EINVAL", {}, dict(n_tok=1 << 31)), ("OK", {}, dict(n_tok=0)), ("OK", dict(out_dim=0), {}),
    ("EINVAL", dict(in_dim=1 << 30), dict(x_stride=1 << 30))])
def test_lora_refusals(q8, want, ad, kw):
    assert lora(q8, ad, **kw) == getattr(q8, "Q8_" + want)


def read(q8, cache=None, **kw):
    c = dict(k=A, v=B, layer_stride=1 << 20, page_stride=2 * 64 * 128 * 2, n_layers=2, n_pages=8, page_tokens=64, n_kv_heads=2, head_dim=128, type=1)
    c.update(cache or {})
    s = q8.KVCacheStruct(*(c[n] for n, _ in q8.KVCacheStruct._fields_))
    a = dict(k_out=A, k_stride=256, v_out=B, v_stride=256, out_type=1, c=s, layer=0, table=C, table_stride=4, max_pages=4, n_rows=3, seqs=None,
             first=None, k_start=A, n_seq=3, n_k=10)
    a.update(kw)
    return q8.lib.q8_kv_read(*a.values(), None)


@pytest.mark.parametrize("want,cache,kw", [
    ("EINVAL", dict(k=None), {}), ("EINVAL", dict(type=5), {}), ("EALIGN", dict(k=A + 8), {}), ("EINVAL", {}, dict(c=None)),
    ("EINVAL", {}, dict(layer=2)), ("EINVAL", {}, dict(table=None)), ("EINVAL", {}, dict(table_stride=3)), ("EINVAL", {}, dict(max_pages=0)),
    ("EINVAL", {}, dict(n_rows=0)), ("EINVAL", {}, dict(n_rows=2)), ("EINVAL", {}, dict(n_seq=(1 << 20) + 1)), ("EINVAL", {}, dict(n_k=(1 << 28) + 1)),
    ("EINVAL", {}, dict(out_type=8)), ("EINVAL", {}, dict(out_type=3)), ("EINVAL", {}, dict(k_out=None, v_out=None)), ("EINVAL", {}, dict(k_start=None)),
    ("EINVAL", {}, dict(k_stride=248)), ("EINVAL", {}, dict(v_stride=248)), ("EALIGN", {}, dict(k_stride=260)), ("EALIGN", {}, dict(v_out=B + 8)),
    ("EALIGN", {}, dict(k_start=A + 2)), ("EALIGN", {}, dict(first=A + 1)), ("EALIGN", {}, dict(seqs=A + 2)), ("OK", {}, dict(n_k=0)), ("OK", {}, dict(n_seq=0))])
def test_kv_read_refusals(q8, want, cache, kw):
    assert read(q8, cache, **kw) == getattr(q8, "Q8_" + want)
