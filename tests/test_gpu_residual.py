"""GPU tests of q8_residual_norm: bit for bit the fp32 steps of its definition, for every type and form."""
import numpy as np
import pytest

import oracle
from tests import layer_plain

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_matmul_gb300 import build
    build.build()
    import q8_quantized_matmul_gb300 as m
    torch.cuda.set_device(0)
    return m


DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def code(q8, name):
    return {"f32": q8.Q8_TYPE_F32, "f16": q8.Q8_TYPE_F16, "bf16": q8.Q8_TYPE_BF16, "q8": q8.Q8_TYPE_Q8_0}[name]


def up(x, name="f32"):
    return torch.from_numpy(x).to(DT[name]).to(DEV)


def typed(rng, shape, name, size=1.0):
    """Values that the type holds, as fp32."""
    x = torch.from_numpy((size * rng.standard_normal(shape)).astype(np.float32))
    return x.to(DT[name]).float().numpy()


def check(q8, n, out, want):
    if out == "q8":
        assert np.array_equal(n.cpu().numpy(), oracle.get().quantize(np.ascontiguousarray(want)))
    else:
        ref = torch.from_numpy(want).to(DT[out])
        assert n.dtype == DT[out] and torch.equal(n.cpu(), ref)


@pytest.mark.parametrize("dim", [32, 96, 256, 1024, 2080, 4096, 4128, 7168, 8192, 11232, 16384, 16416, 32768])
@pytest.mark.parametrize("h,y,out,post,gate", [
    ("f32", "f32", "q8", True, "row"), ("bf16", "bf16", "q8", False, "token"), ("f16", "f32", "f16", True, None),
    ("f32", "bf16", "f32", False, None), ("bf16", "f32", "bf16", True, "token"), ("f32", "f16", "q8", True, None)])
def test_bits(q8, dim, h, y, out, post, gate):
    rng = np.random.default_rng(dim + len(out))
    n = 7
    hv, yv = typed(rng, (n, dim), h, 3.0), typed(rng, (n, dim), y, 0.3)
    hv[3] = 0.0                                   # a row of nothing: n is zeros
    yv[3] = 0.0
    yv[4] *= 64.0
    gp, gn = (1 + 0.2 * rng.standard_normal((2, dim))).astype(np.float32)
    g = None if gate is None else rng.standard_normal((n, dim) if gate == "token" else dim).astype(np.float32)
    store = lambda v: torch.from_numpy(v).to(DT[h]).float().numpy()
    want_n, want_h = layer_plain.residual_norm(hv, yv, gn, EPS, gp, post, g, 0.7, store)
    got_n, got_h = q8.residual_norm(up(hv, h), up(yv, y), up(gn), EPS, gamma_post=up(gp), post=post,
                                    gate=None if g is None else up(g), residual_scale=0.7, out_type=code(q8, out))
    assert q8.q8_last_error() == 0
    assert got_h.dtype == DT[h] and np.array_equal(got_h.float().cpu().numpy(), want_h)
    check(q8, got_n, out, want_n)


@pytest.mark.parametrize("tokens", [1, 2, 151, 153, 700])
def test_many_rows_and_no_gammas(q8, tokens):
    rng = np.random.default_rng(tokens)
    hv, yv = typed(rng, (tokens, 640), "f32", 3.0), typed(rng, (tokens, 640), "f32")
    want_n, want_h = layer_plain.residual_norm(hv, yv, None, EPS, None, True)
    n, h = q8.residual_norm(up(hv), up(yv), None, EPS, post=True)
    assert np.array_equal(h.cpu().numpy(), want_h)
    check(q8, n, "q8", want_n)


@pytest.mark.parametrize("dim", [1024, 4128, 8192, 11232])
@pytest.mark.parametrize("h,y,out", [("f32", "f32", "q8"), ("bf16", "f16", "bf16")])
@pytest.mark.parametrize("shift", [0, 4])
def test_more_rows_than_two_an_sm(q8, dim, h, y, out, shift):
    """Every form for many rows; shift: rows that start between 32-byte boundaries (fp32)."""
    rng = np.random.default_rng(dim)
    n = 420
    hv, yv = typed(rng, (n, dim), h, 3.0), typed(rng, (n, dim), y)
    gp, gn = typed(rng, (dim,), "f32"), typed(rng, (dim + 4,), "f32")
    store = lambda v: torch.from_numpy(v).to(DT[h]).float().numpy()
    want_n, want_h = layer_plain.residual_norm(hv, yv, gn[shift:shift + dim], EPS, gp, True, store=store)
    wide = torch.zeros(n, dim + 8, device=DEV, dtype=DT[h])
    at = shift if h == "f32" else 2 * shift
    wide[:, at:at + dim] = up(hv, h)
    got_n, got_h = q8.residual_norm(wide[:, at:at + dim], up(yv, y), up(gn)[shift:shift + dim], EPS, gamma_post=up(gp), post=True,
                                    out_type=code(q8, out))
    assert np.array_equal(got_h.float().cpu().numpy(), want_h)
    check(q8, got_n, out, want_n)


def test_rows_far_apart(q8):
    """Rows whose offsets pass 32 bits."""
    rng = np.random.default_rng(2)
    n, dim, stride = 80, 256, 1 << 24
    hv, yv = typed(rng, (n, dim), "f32"), typed(rng, (n, dim), "bf16")
    want_n, want_h = layer_plain.residual_norm(hv, yv, None, EPS)
    h = torch.empty(n * stride, device=DEV).view(n, stride)[:, 8:8 + dim]
    y = torch.empty(n * stride, device=DEV, dtype=torch.bfloat16).view(n, stride)[:, :dim]
    h.copy_(up(hv)), y.copy_(up(yv, "bf16"))
    got, _ = q8.residual_norm(h, y, None, EPS, h_out=h)
    assert np.array_equal(h.cpu().numpy(), want_h)
    check(q8, got, "q8", want_n)


def test_strides_in_place_and_parts(q8):
    rng = np.random.default_rng(5)
    n, dim = 9, 128
    hv, yv, gv = typed(rng, (n, dim), "f32"), typed(rng, (n, dim), "f32"), typed(rng, (n, dim), "f32")
    gn = typed(rng, (dim,), "f32")
    want_n, want_h = layer_plain.residual_norm(hv, yv, gn, 1e-5, gate=gv)
    wide_h, wide_y, wide_g = (torch.full((n, 3 * dim), float("nan"), device=DEV) for _ in range(3))
    h, y, g = wide_h[:, dim:2 * dim], wide_y[:, 2 * dim:], wide_g[:, 64:64 + dim]
    h.copy_(up(hv)), y.copy_(up(yv)), g.copy_(up(gv))
    a, stored = q8.residual_norm(h, y, up(gn), 1e-5, gate=g, h_out=False)         # n alone
    assert stored is None and torch.equal(h.cpu(), torch.from_numpy(hv))
    b, none = q8.residual_norm(h, y, up(gn), 1e-5, gate=g, out_type=None)[::-1]   # h' alone
    assert none is None and np.array_equal(b.cpu().numpy(), want_h)
    c, same = q8.residual_norm(h, y, up(gn), 1e-5, gate=g, h_out=h)               # in place
    assert same is h or same.data_ptr() == h.data_ptr()
    assert np.array_equal(h.cpu().numpy(), want_h) and torch.isnan(wide_h[:, :dim]).all() and torch.isnan(wide_h[:, 2 * dim:]).all()
    for x in (a, c):
        check(q8, x, "q8", want_n)


def test_values_that_are_not_finite_stay_in_their_row(q8):
    rng = np.random.default_rng(6)
    hv, yv = typed(rng, (6, 256), "f32"), typed(rng, (6, 256), "f32")
    clean_n, clean_h = (x.float() for x in q8.residual_norm(up(hv), up(yv), None, EPS, post=True, out_type=q8.Q8_TYPE_F32))
    hv[1, 7], yv[2, 200], yv[4, 3] = np.inf, np.nan, -np.inf
    n, h = q8.residual_norm(up(hv), up(yv), None, EPS, post=True, out_type=q8.Q8_TYPE_F32)
    keep = [0, 3, 5]
    assert torch.equal(n[keep], clean_n[keep]) and torch.equal(h[keep], clean_h[keep])
    assert not torch.isfinite(n[[1, 2, 4]]).all(1).any()
    # squares beyond fp32: the sum is infinite, its inverse root 0
    big = np.full((1, 64), 1e25, np.float32)
    n, _ = q8.residual_norm(up(big), up(0 * big), None, EPS, out_type=q8.Q8_TYPE_F32)
    assert torch.equal(n, torch.zeros_like(n))


def test_captured(q8):
    h, y = torch.randn(33, 512, device=DEV), torch.randn(33, 512, device=DEV)
    g = torch.randn(512, device=DEV)
    q8.residual_norm(h, y, g, EPS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n, out = q8.residual_norm(h, y, g, EPS)
    for _ in range(2):
        h.normal_(), y.normal_()
        graph.replay()
        a, b = q8.residual_norm(h, y, g, EPS)
        assert torch.equal(n, a) and torch.equal(out, b)


def test_feeds_the_projection(q8):
    """The blocks are those of q8_quantize_act, so the projection's results are the same bits."""
    import inputs
    h, y = torch.randn(5, 512, device=DEV), torch.randn(5, 512, device=DEV)
    w = torch.from_numpy(inputs.weights(96, 512, seed=3)).to(DEV)
    xq, _ = q8.residual_norm(h, y, None, EPS)
    n, _ = q8.residual_norm(h, y, None, EPS, out_type=q8.Q8_TYPE_F32)
    assert torch.equal(xq, q8.quantize_act(n))
    assert torch.equal(q8.matmul_q(w, xq, 512, 96), q8.matmul_q(w, q8.quantize_act(n), 512, 96))


def test_helper_refusals(q8):
    h, y = torch.randn(3, 64, device=DEV), torch.randn(3, 64, device=DEV)
    for bad in (lambda: q8.residual_norm(h, y[:2], None, EPS), lambda: q8.residual_norm(h, y.cpu(), None, EPS),
                lambda: q8.residual_norm(h, y.T.contiguous().T, None, EPS), lambda: q8.residual_norm(h, y, None, EPS, gate=h[:2]),
                lambda: q8.residual_norm(h.double(), y, None, EPS), lambda: q8.residual_norm(h, y, h[0, :32], EPS),
                lambda: q8.residual_norm(h, y, None, EPS, h_out=h.half()), lambda: q8.residual_norm(h, y, None, EPS, out_type=7)):
        with pytest.raises((TypeError, ValueError, q8.Q8Error)):
            bad()
    with pytest.raises(q8.Q8Error):
        q8.residual_norm(h, y, None, 0.0)
    n, out = q8.residual_norm(h[:0], y[:0], None, EPS)
    assert n.shape == (0, 68) and out.shape == (0, 64)
