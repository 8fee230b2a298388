"""Long batches through the residual-stream calls, on small integers: every
product and sum is exact in fp32 (all partial sums stay below 2^24), so that a
row, a share or a partial sum that is lost, read twice or read elsewhere shows
as a wrong integer, whatever the length of the sum."""

import numpy as np
import pytest

from test_gpu_residual import engine

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_embedding_02_b200 as eb
    return eb


def ffn_integers(n, d, f, seed):
    """x, Wgu, Wd of test_ffn_products_are_exact_on_small_integers, made on the device: g is 128 or 129 (act(g) = g and
    act'(g) = 1 in fp32), u and each column of Wd's one entry are 0 or 1"""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    x = torch.randint(0, 2, (n, d), generator=gen, device="cuda").float()
    x[:, 0] = 1
    Wg, Wu, Wd = np.zeros((f, d), np.float32), np.zeros((f, d), np.float32), np.zeros((d, f), np.float32)
    Wg[:, 0] = 128
    Wg[np.arange(f), 1 + rng.integers(0, d - 1, f)] = 1
    Wu[np.arange(f), rng.integers(0, d, f)] = 1
    Wd[rng.integers(0, d, f // 2), rng.choice(f, f // 2, replace=False)] = 1
    return x, torch.from_numpy(np.concatenate([Wg, Wu])).cuda(), torch.from_numpy(Wd).cuda()


@pytest.mark.parametrize("few", [True, False])
def test_ffn_gradients_beyond_32_bit_offsets(eb, few):
    """2.25e9 elements of g and u, and of dg and du: element 2^31 lies in row 104857.  `few`: d_y is zero but for some
    rows around it and elsewhere, so that the sums over the rows are small enough for bf16 to tell one apart."""
    n, d, f = 110007, 256, 10240
    eng = engine(eb, d)
    bf = torch.bfloat16
    x, Wgu, Wd = ffn_integers(n, d, f, 3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    d_y = torch.randint(0, 2, (n, d), generator=gen, device="cuda").float()
    if few:
        keep = torch.zeros(n, 1, device="cuda")
        keep[[0, 1, 31, 32, 255, 256, 52428, 52429, 104855, 104856, 104857, 104858, 104859, 104900, n - 40, n - 2, n - 1]] = 1
        d_y *= keep
    y, saved = eng.ffn(x.to(bf), Wgu.to(bf), Wd.to(bf), save=True)
    got = eng.ffn_grad(d_y.to(bf), x.to(bf), saved, Wgu.to(bf), Wd.to(bf))
    assert eng.status() == (eb.ENGRAM_OK, 0)
    d_Wgu, d_Wd = (torch.zeros(s, device="cuda", dtype=torch.float64) for s in ((2 * f, d), (d, f)))
    for lo in range(0, n, 8192):
        r = slice(lo, min(n, lo + 8192))
        gu = x[r] @ Wgu.t()
        g, u = gu[:, :f], gu[:, f:]
        a = g * u
        assert torch.equal(y[r], (a @ Wd.t()).to(bf)), lo
        da = d_y[r] @ Wd
        dgu = torch.cat([da * u, da * g], 1)
        assert torch.equal(got[0][r], (dgu @ Wgu).to(bf)), lo
        d_Wgu += (dgu.t() @ x[r]).double()
        d_Wd += (d_y[r].t() @ a).double()
    assert float(d_Wgu.max()) < 2 ** 24 and float(d_Wd.max()) < 2 ** 24
    assert torch.equal(got[1], d_Wgu.float().to(bf))
    assert torch.equal(got[2], d_Wd.float().to(bf))
