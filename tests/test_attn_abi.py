"""Host-side validation of the cache and attention entry points (no GPU): bad arguments are refused before any
CUDA call, empty work is a no-op."""
import ctypes

import pytest

A, B = 0x10000, 0x20000     # 16-byte aligned fake addresses, never dereferenced


@pytest.fixture(scope="module")
def q8():
    from q8_quantized_matmul_gb300 import build
    build.build()
    import q8_quantized_matmul_gb300 as m
    return m


def no_gpu():
    import torch
    return not torch.cuda.is_available()


def cache(q8, **kw):
    a = dict(k=A, v=B, layer_stride=1 << 20, page_stride=2 * 64 * 128 * 2, n_layers=2, n_pages=8, page_tokens=64,
             n_kv_heads=2, head_dim=128, type=q8.Q8_TYPE_F16)
    a.update(kw)
    return q8.KVCacheStruct(*(a[n] for n, _ in q8.KVCacheStruct._fields_))


def test_struct_matches_the_header(q8):
    assert ctypes.sizeof(q8.KVCacheStruct) == 56


def test_page_bytes(q8):
    f = q8.q8_kv_page_bytes
    assert f(q8.Q8_TYPE_BF16, 64, 8, 128) == 64 * 8 * 128 * 2
    assert f(q8.Q8_TYPE_Q8_0, 32, 2, 64) == 2 * 32 * (64 + 4)
    for bad in ((0, 64, 8, 128), (3, 64, 8, 128), (1, 48, 8, 128), (1, 8, 8, 128), (1, 512, 8, 128), (1, 64, 0, 128),
                (1, 64, 8, 96), (1, 64, 8, 1024)):
        assert f(*bad) == 0


@pytest.mark.parametrize("field,value,want", [
    ("k", 0, "EINVAL"), ("v", 0, "EINVAL"), ("k", A + 8, "EALIGN"), ("page_stride", 2 * 64 * 128 * 2 - 16, "EINVAL"),
    ("page_stride", 2 * 64 * 128 * 2 + 8, "EALIGN"), ("layer_stride", 100, "EINVAL"), ("layer_stride", (1 << 20) + 4, "EALIGN"),
    ("n_layers", 0, "EINVAL"), ("n_pages", 0, "EINVAL"), ("n_pages", (1 << 24) + 1, "EINVAL"), ("page_tokens", 60, "EINVAL"),
    ("head_dim", 80, "EINVAL"), ("type", 0, "EINVAL"), ("type", 5, "EINVAL"), ("n_kv_heads", 0, "EINVAL")])
def test_bad_caches_are_refused(q8, field, value, want):
    want = getattr(q8, "Q8_" + want)
    c = cache(q8, **{field: value})
    L = q8.lib
    assert L.q8_kv_copy(c, A, B, 1, None) == want
    assert L.q8_kv_free(c, A, 4, 4, 2, A, A, A, 1, None) == want
    assert L.q8_attn_decode(A, 1, None, A, 2048, 1, c, 0, A, 4, 4, A, 1, 4, 1.0, 0, None, None) == want


def decode(q8, c=None, **kw):
    a = dict(out=A, out_type=1, lse=None, q=A, q_stride=512, q_type=1, layer=0, table=A, table_stride=4, max_pages=4,
             lens=A, n_seq=2, n_heads=4, scale=1.0, window=0, sinks=None)
    a.update(kw)
    return q8.lib.q8_attn_decode(a["out"], a["out_type"], a["lse"], a["q"], a["q_stride"], a["q_type"], c or cache(q8),
                                 a["layer"], a["table"], a["table_stride"], a["max_pages"], a["lens"], a["n_seq"],
                                 a["n_heads"], a["scale"], a["window"], a["sinks"], None)


def test_decode_arguments(q8):
    E, AL = q8.Q8_EINVAL, q8.Q8_EALIGN
    assert decode(q8, layer=2) == E
    assert decode(q8, n_heads=3) == E                      # not a multiple of the key-value heads
    assert decode(q8, n_heads=0) == E
    assert decode(q8, q_type=2, out_type=2) == E           # not the cache's type
    assert decode(q8, q_type=0) == E
    assert decode(q8, out_type=2) == E
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert decode(q8, scale=s) == E
    assert decode(q8, table=0) == E and decode(q8, max_pages=0) == E and decode(q8, table_stride=3) == E
    assert decode(q8, max_pages=1 << 25, table_stride=1 << 25) == E
    assert decode(q8, out=0) == E and decode(q8, q=0) == E and decode(q8, lens=0) == E
    assert decode(q8, q_stride=511) == E and decode(q8, q_stride=516) == AL
    assert decode(q8, q=A + 2) == AL and decode(q8, out=A + 4) == AL and decode(q8, table=A + 2) == AL
    assert decode(q8, lens=A + 1) == AL and decode(q8, sinks=A + 2) == AL and decode(q8, lse=A + 2) == AL
    assert decode(q8, n_seq=0) == q8.Q8_OK
    if no_gpu():
        assert decode(q8) == q8.Q8_ECUDA
        for t in (1, 2):                                   # Q8_0 caches take either query type
            assert decode(q8, cache(q8, type=8), q_type=t, out_type=t) == q8.Q8_ECUDA
        assert decode(q8, out_type=0) == q8.Q8_ECUDA and decode(q8, out_type=8) == q8.Q8_ECUDA


def prompt(q8, **kw):
    a = dict(out=A, out_type=2, lse=None, q=A, k=A, v=B, type=2, qs=512, ks=256, vs=256, q0=A, k0=None, n_seq=2, nq=9, nk=9,
             heads=4, kv=2, dim=128, scale=1.0, window=0, sinks=None)
    a.update(kw)
    return q8.lib.q8_attn_prompt(a["out"], a["out_type"], a["lse"], a["q"], a["k"], a["v"], a["type"], a["qs"], a["ks"], a["vs"],
                                 a["q0"], a["k0"], a["n_seq"], a["nq"], a["nk"], a["heads"], a["kv"], a["dim"], a["scale"],
                                 a["window"], a["sinks"], None)


def test_prompt_arguments(q8):
    E, AL = q8.Q8_EINVAL, q8.Q8_EALIGN
    for kw in (dict(dim=96), dict(kv=0), dict(heads=3), dict(heads=0), dict(type=8), dict(type=0), dict(out_type=1),
               dict(scale=0.0), dict(scale=float("nan")), dict(nq=1 << 29), dict(nk=1 << 29), dict(out=0), dict(q=0), dict(k=0),
               dict(v=0), dict(q0=0), dict(qs=504), dict(ks=248), dict(vs=8)):
        assert prompt(q8, **kw) == E, kw
    for kw in (dict(q=A + 8), dict(k=A + 2), dict(v=B + 4), dict(out=A + 8), dict(qs=516), dict(ks=257), dict(vs=260),
               dict(q0=A + 2), dict(k0=A + 1), dict(sinks=A + 3), dict(lse=A + 1)):
        assert prompt(q8, **kw) == AL, kw
    assert prompt(q8, n_seq=0) == q8.Q8_OK and prompt(q8, nq=0) == q8.Q8_OK
    if no_gpu():
        assert prompt(q8) == q8.Q8_ECUDA


def append(q8, c="c", **kw):
    a = dict(qo=A, ko=None, vo=None, ot=1, layer=0, q=A, qs=512, k=A, ks=256, v=B, vs=256, heads=4, kv=2, dim=128, pos=A,
             seq=A, table=A, ts=4, mp=4, rows=3, cs=A, npos=10, rot=64, rope=1, n=5)
    a.update(kw)
    c = cache(q8) if c == "c" else c
    return q8.lib.q8_kv_append(a["qo"], a["ko"], a["vo"], a["ot"], c, a["layer"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                               a["heads"], a["kv"], a["dim"], a["pos"], a["seq"], a["table"], a["ts"], a["mp"], a["rows"], a["cs"],
                               a["npos"], a["rot"], a["rope"], a["n"], None)


def test_append_arguments(q8):
    E, AL = q8.Q8_EINVAL, q8.Q8_EALIGN
    for kw in (dict(dim=64), dict(kv=4, ks=512, vs=512), dict(layer=2), dict(rows=0), dict(table=0), dict(ts=3), dict(ot=0),
               dict(ot=8), dict(rope=3), dict(rope=-1), dict(rot=0), dict(rot=24), dict(rot=144), dict(npos=0), dict(q=0),
               dict(k=0), dict(v=0), dict(pos=0), dict(seq=0), dict(cs=0), dict(qs=511), dict(ks=255), dict(vs=100),
               dict(heads=0), dict(n=1 << 31)):
        assert append(q8, **kw) == E, kw
    for kw in (dict(q=A + 4), dict(k=A + 4), dict(v=B + 8), dict(qo=A + 2), dict(ko=A + 2), dict(vo=A + 8), dict(cs=A + 4),
               dict(pos=A + 2), dict(seq=A + 1), dict(qs=514), dict(ks=258), dict(vs=257)):
        assert append(q8, **kw) == AL, kw
    assert append(q8, n=0) == q8.Q8_OK
    if no_gpu():
        assert append(q8) == q8.Q8_ECUDA
        assert append(q8, None, seq=0, table=0, ko=A, vo=A) == q8.Q8_ECUDA     # no cache: none of its arguments
        assert append(q8, qo=None, q=0, heads=0) == q8.Q8_ECUDA                 # no queries
        assert append(q8, rope=0, cs=0, rot=0, npos=0) == q8.Q8_ECUDA


def test_page_call_arguments(q8):
    L, c, E, AL = q8.lib, cache(q8), q8.Q8_EINVAL, q8.Q8_EALIGN
    for f, two in ((L.q8_kv_reserve, True), (L.q8_kv_fork, True), (L.q8_kv_free, False)):
        def call(table=A, ts=4, mp=4, rows=2, lens=A, refs=A, a=A, b=A, n=1):
            return f(c, table, ts, mp, rows, lens, refs, a, *((b,) if two else ()), n, None)
        assert call(table=0) == E and call(ts=3) == E and call(mp=0) == E and call(rows=0) == E
        assert call(lens=0) == E and call(refs=0) == E and call(a=0) == E and call(n=(1 << 20) + 1) == E
        assert call(lens=A + 2) == AL and call(refs=A + 1) == AL and call(a=A + 2) == AL and call(table=A + 2) == AL
        if two:
            assert call(b=0) == E and call(b=A + 2) == AL
        assert call(n=0) == q8.Q8_OK
        if no_gpu():
            assert call() == q8.Q8_ECUDA
    def compact(to=B, t=A, ro=B, r=A, u=A):
        return L.q8_kv_compact(c, to, t, 4, 4, 2, ro, r, u, None)
    assert compact(to=0) == E and compact(to=A) == E and compact(ro=A) == E and compact(r=0) == E and compact(u=0) == E
    assert compact(to=B + 2) == AL and compact(u=A + 2) == AL
    assert L.q8_kv_copy(c, 0, A, 1, None) == E and L.q8_kv_copy(c, A, B + 2, 1, None) == AL
    assert L.q8_kv_copy(c, A, B, 0, None) == q8.Q8_OK
    if no_gpu():
        assert compact() == q8.Q8_ECUDA and L.q8_kv_copy(c, A, B, 1, None) == q8.Q8_ECUDA


def test_wrong_tensors_are_refused(q8):
    """The tensor helpers refuse what does not fit before any call."""
    import torch
    k = torch.zeros(1, 4, 2 * 64 * 64 * 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        q8.KVCache(k, k[:, :, :-2], q8.Q8_TYPE_F16, 64, 2, 64)
    with pytest.raises(ValueError):
        q8.KVCache(k, k.clone(), q8.Q8_TYPE_Q8_0, 64, 2, 64)             # a page of another size
    with pytest.raises(q8.Q8Error):
        q8.KVCache(k, k.clone(), q8.Q8_TYPE_F16, 60, 2, 64)
    c = q8.KVCache(k, k.clone(), q8.Q8_TYPE_F16, 64, 2, 64)
    q = torch.zeros(1, 2, 64, dtype=torch.float16)
    with pytest.raises(TypeError):                                       # int32 on the GPU
        q8.attn_decode(q, c, 0, torch.zeros(1, 2, dtype=torch.int64), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        q8.attn_decode(q, c, 0, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        q8.attn_prompt(q, q, q[:, :1], torch.zeros(2, dtype=torch.int32))


def test_caches_on_the_host_are_refused(q8):
    """Every call refuses a cache whose pages lie in host memory, before anything else that is wrong with its tensors."""
    import torch
    c = q8.KVCache.empty(q8.Q8_TYPE_F16, 1, 4, 64, 2, 64, device="cpu")
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    x = torch.zeros(1, 2, 64)
    for call in (lambda: q8.attn_decode(x.half(), c, 0, i32(1, 2), i32(1)),
                 lambda: q8.kv_append(c, 0, x, x, x, i32(1), i32(1), i32(1, 2)),
                 lambda: q8.kv_reserve(c, i32(1, 2), i32(1), i32(4), i32(1), i32(1)),
                 lambda: q8.kv_fork(c, i32(1, 2), i32(1), i32(4), i32(1), i32(1)),
                 lambda: q8.kv_free(c, i32(1, 2), i32(1), i32(4), i32(1)),
                 lambda: q8.kv_compact(c, i32(1, 2), i32(1), i32(4)),
                 lambda: q8.kv_copy(c, i32(1), i32(1))):
        with pytest.raises(TypeError, match="cache: pages on the GPU"):
            call()


def test_pools_of_another_type_are_refused(q8):
    import torch
    for dt in (torch.float16, torch.bfloat16, torch.float32, torch.uint8, torch.int16):
        size = {torch.float32: 4, torch.uint8: 1}.get(dt, 2)
        for code, mine in ((q8.Q8_TYPE_F16, torch.float16), (q8.Q8_TYPE_BF16, torch.bfloat16), (q8.Q8_TYPE_Q8_0, None)):
            n = q8.q8_kv_page_bytes(code, 64, 2, 64) // size
            k = torch.zeros(1, 4, n, dtype=dt)
            if dt in (mine, torch.uint8, torch.int16):
                assert q8.KVCache(k, k.clone(), code, 64, 2, 64).n_pages == 4
            else:
                with pytest.raises(TypeError, match="cache's type"):
                    q8.KVCache(k, k.clone(), code, 64, 2, 64)
