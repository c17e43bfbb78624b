"""GPU tests of the adapters of many tokens where tiles outnumber clusters: clusters of four CTAs with several steps each, more than
one tile a cluster, sums in runs, and the groups of adapters with few tokens."""
import numpy as np
import pytest

from tests.test_gpu_lora import Case, i32, q8   # noqa: F401  (the fixture)
from tests.test_gpu_lora_sums import LIMIT

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"


def check(c, got):
    """Each value within its bound, and the root mean square of the errors within that of fp32."""
    c.check(got)
    want = c.plain[0]
    part = want - (0 if c.base is None else c.base)
    err = got.double().cpu().numpy() - want
    # base + part is rounded to fp32 once more: half a step of the sum, 2^-24
    assert np.sqrt(np.mean(err ** 2)) <= LIMIT * np.sqrt(np.mean(part ** 2)) + 2.0 ** -24 * np.sqrt(np.mean(want ** 2))


# tokens of 3 adapters (or none): 16 to 36 tiles, more than 36 (a second tile of a cluster); inputs: even and odd numbers of steps for
# each CTA, one of them with half a step at the end
@pytest.mark.parametrize("n", [2500, 5000])
@pytest.mark.parametrize("n_in,rank", [(1024, 64), (1056, 80), (768, 48), (1312, 16), (1024, 128)])
@pytest.mark.parametrize("kind,x", [("bf16", "f32"), ("f16", "q8"), ("bf16", "f16"), ("f16", "bf16")])
def test_several_steps_and_tiles(q8, n, n_in, rank, kind, x):   # noqa: F811
    c = Case(n + n_in, n, n_in, 136, rank, 3, kind, x, ragged=False)
    check(c, c.call(q8))
    assert q8.q8_last_error() == 0


# in runs, with a second tile of a cluster: the sums of the runs before are the tile's own
@pytest.mark.parametrize("n_in,rank,kind,x", [(4160, 128, "f16", "f32"), (4096, 96, "bf16", "q8"), (4224, 64, "bf16", "f32"), (4128, 112, "bf16", "bf16")])
def test_runs_of_several_tiles(q8, n_in, rank, kind, x):   # noqa: F811
    c = Case(rank, 5000, n_in, 72, rank, 3, kind, x, ragged=False)
    check(c, c.call(q8))


def test_ragged_ranks_of_many_tiles(q8):   # noqa: F811
    c = Case(11, 5000, 2080, 136, 128, 6, "bf16")
    c.check(c.call(q8))


@pytest.mark.parametrize("n,adapters,n_in", [(600, 150, 512), (1000, 250, 256), (700, 500, 1024), (333, 60, 2048)])
def test_groups(q8, n, adapters, n_in):   # noqa: F811
    """Adapters of 1 to 15 tokens: which of them share a group, and which is alone, is left to chance, and does not show."""
    rng = np.random.default_rng(n)
    c = Case(n, n, n_in, 300, 32, adapters, "bf16", ids=rng.integers(-1, adapters, n))
    first = c.call(q8)
    c.check(first)
    x, a, b, ids, ranks = c.x.to(DEV), c.a.to(DEV), c.b.to(DEV), i32(c.ids), i32(c.ranks)
    scales, base = torch.from_numpy(c.scales).to(DEV), torch.from_numpy(c.base).to(DEV)
    for _ in range(5):
        assert torch.equal(q8.lora(x, a, b, ids, ranks, scales, base), first)
        perm = torch.randperm(n, device=DEV)
        assert torch.equal(q8.lora(x[perm], a, b, ids[perm], ranks, scales, base[perm]), first[perm])
    # values that are not finite stay in their token
    x[n // 2, 7], x[n - 1, 0] = float("nan"), float("inf")
    got, bad = q8.lora(x, a, b, ids, ranks, scales, base), torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[n // 2] = bad[n - 1] = True
    assert torch.equal(got[~bad], first[~bad])
    for t in (n // 2, n - 1):
        if c.ids[t] >= 0 and c.ranks[c.ids[t]] > 0:
            assert not torch.isfinite(got[t]).all()


def test_tiles_and_permutation_of_many_tiles(q8):   # noqa: F811
    c = Case(3, 5000, 1056, 200, 64, 3, "bf16")
    first = c.call(q8)
    x, a, b, ids, ranks = c.x.to(DEV), c.a.to(DEV), c.b.to(DEV), i32(c.ids), i32(c.ranks)
    scales, base = torch.from_numpy(c.scales).to(DEV), torch.from_numpy(c.base).to(DEV)
    for _ in range(3):
        perm = torch.randperm(5000, device=DEV)
        assert torch.equal(q8.lora(x[perm], a, b, ids[perm], ranks, scales, base[perm]), first[perm])
