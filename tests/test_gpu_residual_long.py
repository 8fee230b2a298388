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


def runs(B, T, V, lengths, seed):
    """tokens of B x T positions: token 2 k + 1 occurs lengths[k] times, the rest of the batch is spread over the even
    tokens below V / 2 (the runs lie among them in the sorted list), all in random order"""
    rng = np.random.default_rng(seed)
    long = np.concatenate([np.full(m, 2 * k + 1) for k, m in enumerate(lengths)])
    rest = 2 * rng.integers(0, V // 4, B * T - long.size)
    t = np.concatenate([long, rest])
    return torch.from_numpy(rng.permutation(t).reshape(B, T).astype(np.int32)).cuda()


# Runs from one position to half of the batch, at lengths around the pieces (8 or 32 sorted entries) and around the
# counts where the join's groups (256 / lanes of them, lanes = the power of two from d / 4 up, 64 at most) take one part
# more each.
LENGTHS = [1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 100, 128, 250, 500, 1023, 1024, 1025, 3999, 4000, 4095, 4097, 4128]


def summation_depth(count, d, piece):
    """Additions in a row that a term of a run can pass through: in its piece, in its group of the join, over the
    groups, and the product with the scale.  embed_reduce_kernel adds at most `piece` terms; the run's m parts lie in
    ceil(count / piece) pieces or one more; each of the join's groups adds per = ceil(m / groups) of them, and the
    ceil(m / per) sums are added one after the other."""
    lanes = 1
    while lanes < 64 and lanes * 4 < d:
        lanes *= 2
    groups = 256 // lanes

    def join(m):
        per = (m + groups - 1) // groups
        return per + (m + per - 1) // per

    m = (count + piece - 1) // piece
    return count.clamp(max=piece) + torch.maximum(join(m), join(m + 1)) + 1


@pytest.mark.parametrize("B,T,V,d", [(1, 18000, 4000, 8), (3, 400001, 300000, 8), (2, 30011, 5000, 72), (1, 120007, 5000, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_embed_grad_of_long_runs(eb, B, T, V, d, dtype):
    eng = engine(eb, d, V, dtype)
    n = B * T
    lengths = [m for m in LENGTHS if m <= n // 10]
    if n > 10 ** 6:
        lengths.append(n // 2)                            # a token that takes half of the batch
    tok = runs(B, T, V, lengths, 5)
    idx = tok.view(-1).long()
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(6)

    def plain(t):
        return torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, idx, t.double())

    whole = torch.randint(-3, 4, (n, d), generator=gen, device="cuda").to(dt)
    assert torch.equal(eng.embed_grad(tok, whole), plain(whole).float())       # exact: below 2^24
    was = torch.randint(-9, 10, (V, d), generator=gen, device="cuda").float()
    got = eng.embed_grad(tok, whole, out=was.clone(), accumulate=True)
    assert torch.equal(got, (plain(whole) + was.double()).float())
    # positive terms: nothing cancels, so that the bound is a relative one
    t = (0.5 + torch.rand(n, d, generator=gen, device="cuda")).to(dt)
    want, count = plain(t), torch.bincount(idx, minlength=V)[:, None]
    piece = 32 if n >= 32 * 4 * torch.cuda.get_device_properties(0).multi_processor_count else 8
    bound = summation_depth(count.clamp(min=1), d, piece) * 2.0 ** -24 * want
    got = eng.embed_grad(tok, t)
    assert bool(((got.double() - want).abs() <= bound).all())
    assert torch.equal(got, eng.embed_grad(tok, t))


@pytest.mark.parametrize("T", [300, 2500, 9000, 40000])   # the sorts of one CTA, of several; pieces of 8 and of 32
def test_embed_grad_row_depends_on_its_own_positions(eb, T):
    """A token's sum has the same bits whatever the other tokens and rows are, as long as its positions and the number
    of smaller tokens in the batch (where its run lies among the cuts of the sorted list) stay."""
    V, v, d = 5000, 2500, 136
    eng = engine(eb, d, V)
    rng = np.random.default_rng(T)
    kind = rng.choice(3, 2 * T, p=[0.3, 0.4, 0.3])        # below v, v itself, above v
    d_h = torch.randn(2 * T, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    mine = torch.from_numpy(kind == 1).cuda()[:, None]
    want = None
    for seed in range(3):
        other = np.random.default_rng(seed)
        t = np.where(kind == 0, other.integers(0, v, 2 * T), np.where(kind == 1, v, other.integers(v + 1, V, 2 * T)))
        rows = torch.where(mine, d_h, torch.full_like(d_h, float("nan") if seed == 2 else seed))
        got = eng.embed_grad(torch.from_numpy(t.reshape(2, T).astype(np.int32)).cuda(), rows)[v]
        assert want is None or torch.equal(got, want), seed
        want = got
    assert bool(want.isfinite().all())
