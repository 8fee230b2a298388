"""Token embedding, residual norm and their backward passes on the GPU against
the plain fp64 reference (oracle.residual).

Tolerances, with u = 2^-24 (half an fp32 step) and m the half step of the
model dtype (torch.finfo(t).eps / 2):
  embed       the fp32 product and one rounding: (m + 2 u) |h|;
  embed grad  a sum of k terms in any order is within (k - 1) u sum|x| of the
              exact one (Higham, Accuracy and Stability of Numerical
              Algorithms, 2nd ed., section 4.2), the product with the scale and the
              addition to a given value add a rounding each: (k + 2) u sum|x|;
  norm        the sum of squares: a thread adds at most 64 products in a row,
              then ten levels of pairs, 2 * 74 u at most of a sum of positive
              terms, halved by the root; rsqrtf is within 2 ulp (4 u); the
              division by d, s itself, and the products with r and the gain
              add 5 u: 96 u |y|, and m |y| when stored;
  scale       96 u and the division: 97 u c;
  codes       half a step of E4M3 (2^-4 relative, 2^-10 below 2^-6) and the
              error of y / c before rounding, 194 u |y / c|;
  norm grad   the products and the mean, as above: 100 u of the magnitudes
              that enter, |d_sum| + r (|t| + |sh| mean|t sh|), and m |d_x|;
  gain grad   n terms: (n + 4) u sum|dy sh|.
"""

import numpy as np
import pytest

import synth
from oracle import residual as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def eb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_embedding_02_b200 as eb
    return eb


def engine(eb, d, V=50, dtype="bf16"):
    code = {"bf16": eb.ENGRAM_BF16, "f32": eb.ENGRAM_F32, "fp8": eb.ENGRAM_FP8}[dtype]
    return eb.Engram(eb.make_config(orders=(2,), heads=1, rows=[10007], mult=[[1, 3, 0, 0]], row_dim=128, hidden=d,
                                    conv_width=4, vocab=V, canon_vocab=V, dtype=code))


def half_step(t):
    return torch.finfo(t.dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(seed, *shape, sd=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * sd).to(dtype)


def tokens(seed, B, T, V, kind="zipf"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        t = np.full((B, T), V - 1)
    elif kind == "distinct":
        t = rng.permutation(B * T).reshape(B, T) % V
    elif kind == "half":                      # one token takes half of the batch
        t = np.where(rng.random((B, T)) < 0.5, 2, rng.integers(0, V, (B, T)))
    else:
        t = np.minimum(rng.zipf(1.3, (B, T)) - 1, V - 1)
    return torch.from_numpy(t.astype(np.int32)).cuda()


DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.bfloat16}


# ---------------------------------------------------------------- embedding

@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("B,T,t_begin,V,d", [(1, 1, 0, 50, 8), (3, 7, 2, 50, 2560), (256, 1, 0, 1000, 512),
                                             (2, 5001, 0, 4097, 136), (5, 9, 9, 50, 64), (4, 600, 599, 50, 5128)])
def test_embed(eb, B, T, t_begin, V, d, dtype):
    if dtype == "fp8":
        d = -(-d // 128) * 128
    eng = engine(eb, d, V, dtype)
    E, tok = randn(1, V, d, dtype=DT[dtype]), tokens(2, B, T, V)
    h = eng.embed(tok, E, t_begin=t_begin, scale=0.7)
    assert h.shape == (B * (T - t_begin), d) and h.dtype == DT[dtype]
    want = R.embed(tok.cpu().numpy()[:, t_begin:], f64(E), float(np.float32(0.7)))
    assert (np.abs(f64(h) - want) <= (half_step(h) + 2 * U) * np.abs(want)).all()
    assert eng.status() == (eb.ENGRAM_OK, 0)
    assert torch.equal(eng.embed(tok, E, t_begin=t_begin), E[tok[:, t_begin:].reshape(-1).long()])   # scale 1: the rows


def test_embed_reads_padded_token_rows_and_flags_bad_ids(eb):
    eng = engine(eb, 64)
    E = randn(1, 50, 64)
    wide = tokens(3, 4, 16, 50)
    wide[1, 2], wide[2, 0], wide[3, 10] = -1, 50, 99     # the last one lies in the padding
    tok = wide[:, :7]
    h = eng.embed(tok, E)
    st, flags = eng.status()
    assert st == eb.ENGRAM_E_DEVICE and flags == eb.ENGRAM_ERR_TOKEN
    want = R.embed(tok.cpu().numpy(), f64(E))
    assert np.array_equal(f64(h), want)
    d_h = randn(4, 28, 64)
    got = eng.embed_grad(tok, d_h)
    assert eng.status() == (eb.ENGRAM_E_DEVICE, eb.ENGRAM_ERR_TOKEN)
    check_embed_grad(got, tok, d_h, 50, 1.0)


def check_embed_grad(got, tok, d_h, V, scale, was=None):
    want, mag, cnt = R.embed_grad(tok.cpu().numpy(), f64(d_h), V, scale)
    base = np.zeros_like(want) if was is None else f64(was)
    bound = (cnt[:, None] + 2) * U * (mag + np.abs(base) * (cnt[:, None] > 0))
    err = np.abs(f64(got) - (want + base))
    assert (err <= bound).all(), (int((err > bound).sum()), float(err.max()))
    if was is not None:                                   # rows of other tokens are not touched
        rest = torch.from_numpy(cnt == 0)
        assert torch.equal(got.cpu()[rest], was.cpu()[rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["zipf", "one", "distinct", "half"])
@pytest.mark.parametrize("B,T,V,d", [(1, 1, 50, 8), (2, 33, 50, 136), (1, 2048, 513, 64), (1, 2049, 512, 64),
                                     (3, 7001, 300000, 24), (2, 12001, 70, 264)])
def test_embed_grad(eb, B, T, V, d, kind, dtype):
    eng = engine(eb, d, V, dtype)
    tok, d_h = tokens(5, B, T, V, kind), randn(6, B * T, d, sd=0.1, dtype=DT[dtype])
    scale = float(np.float32(1.7))
    out = torch.full((V, d), float("nan"), device="cuda")
    got = eng.embed_grad(tok, d_h, scale=scale, out=out)
    assert got is out
    check_embed_grad(got, tok, d_h, V, scale)
    assert eng.status() == (eb.ENGRAM_OK, 0)
    again = eng.embed_grad(tok, d_h, scale=scale)
    assert torch.equal(got, again)                        # the same bits on every run
    was = randn(7, V, d, dtype=torch.float32)
    acc = eng.embed_grad(tok, d_h, scale=scale, out=was.clone(), accumulate=True)
    check_embed_grad(acc, tok, d_h, V, scale, was)


def test_embed_grad_of_no_rows(eb):
    eng = engine(eb, 64)
    tok, d_h = tokens(1, 3, 4, 50), randn(1, 0, 64)
    was = randn(2, 50, 64, dtype=torch.float32)
    assert torch.equal(eng.embed_grad(tok, d_h, t_begin=4, out=was.clone(), accumulate=True), was)
    assert not eng.embed_grad(tok, d_h, t_begin=4, out=was.clone()).any()


def test_embed_grad_row_does_not_depend_on_the_other_tokens(eb):
    """a token's sum has the order of its own positions only up to the cuts of the sorted list: equal inputs, equal bits"""
    eng = engine(eb, 64, 5000)
    tok, d_h = tokens(8, 2, 9000, 5000), randn(9, 18000, 64)
    a = eng.embed_grad(tok, d_h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = eng.embed_grad(tok, d_h, stream=side)
    side.synchronize()
    assert torch.equal(a, b)


def test_embed_refuses(eb):
    eng = engine(eb, 64)
    E, tok, d_h = randn(1, 50, 64), tokens(1, 2, 8, 50), randn(2, 16, 64)
    g = torch.zeros(50, 64, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: eb.engram_embed(eng.ctx, tok, 2, 8, 7, 0, E, 1.0, d_h),                       # stride below T
        lambda: eb.engram_embed(eng.ctx, tok, 2, 8, 8, 9, E, 1.0, d_h),                       # t_begin beyond T
        lambda: eb.engram_embed(eng.ctx, None, 2, 8, 8, 0, E, 1.0, d_h),
        lambda: eb.engram_embed(eng.ctx, tok, 2, 8, 8, 0, E, float("nan"), d_h),
        lambda: eb.engram_embed(eng.ctx, tok, 2, 8, 8, 0, E.view(-1)[1:], 1.0, d_h),          # 2-byte aligned
        lambda: eb.engram_embed_grad(eng.ctx, tok, 2, 8, 8, 0, d_h, float("inf"), g, 0, ws, ws.numel()),
        lambda: eb.engram_embed_grad(eng.ctx, tok, 2, 8, 8, 0, d_h, 1.0, None, 0, ws, ws.numel()),
        lambda: eb.engram_embed_grad(eng.ctx, tok, 2, 8, 8, 0, d_h, 1.0, g, 0, ws[1:], ws.numel() - 1),
        lambda: eb.engram_embed_grad(eng.ctx, tok, 1 << 20, 32, 32, 0, d_h, 1.0, g, 0, ws, ws.numel()),
    ]
    for call in bad:
        with pytest.raises(eb.EngramError) as ei:
            call()
        assert ei.value.status == eb.ENGRAM_E_INVAL
    with pytest.raises(eb.EngramError) as ei:
        eb.engram_embed_grad(eng.ctx, tok, 2, 8, 8, 0, d_h, 1.0, g, 0, ws, 256)
    assert ei.value.status == eb.ENGRAM_E_NOMEM
    assert eb.engram_embed_grad_workspace_bytes(eng.ctx, (1 << 24) + 1) == 0


# ---------------------------------------------------------------- residual norm

WIDTHS = [8, 24, 256, 264, 520, 2560, 5128, 8200, 16384]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("with_res,with_gain", [(True, True), (False, False)])
def test_add_norm(eb, d, with_res, with_gain, dtype):
    eng = engine(eb, d, dtype=dtype)
    n = 37
    x = randn(1, n, d, sd=0.3, dtype=DT[dtype])
    x[3] = 0
    res = randn(2, n, d, sd=1.5, dtype=DT[dtype]) if with_res else None
    if with_res:
        res[3] = 0
    x[5] *= 1e-3
    gain = 1 + 0.1 * randn(3, d, dtype=torch.float32) if with_gain else None
    o = eng.add_norm(x, res, gain=gain, q=True, rstd=True)
    s, r, y = R.add_norm(f64(x), None if res is None else f64(res), None if gain is None else f64(gain),
                         float(np.float32(1e-6)))
    m = half_step(x)
    assert (np.abs(f64(o.sum) - s) <= (m + U) * np.abs(s)).all()
    assert (np.abs(f64(o.rstd) - r) <= 96 * U * r).all()
    assert (np.abs(f64(o.y) - y) <= (m + 96 * U) * np.abs(y)).all()
    c = np.abs(y).max(1) / R.E4M3_MAX
    assert (np.abs(f64(o.q_scale) - c) <= 97 * U * c).all()
    v = np.divide(y, c[:, None], out=np.zeros_like(y), where=c[:, None] > 0)
    assert (np.abs(f64(o.q.float()) - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 194 * U * np.abs(v)).all()
    assert f64(o.q_scale)[3] == 0 and not o.q[3].float().any() and not o.y[3].any()
    only = eng.add_norm(x, res, gain=gain, sum=False, y=False, q=True)
    assert only.sum is None and only.y is None and torch.equal(only.q.view(torch.uint8), o.q.view(torch.uint8))
    assert torch.equal(only.q_scale, o.q_scale)


def test_add_norm_in_place_and_special_values(eb):
    d = 264
    eng = engine(eb, d)
    x, res = randn(1, 6, d), randn(2, 6, d)
    x[1, 7], x[2, 0], x[4, 263] = float("nan"), float("inf"), float("-inf")
    o = eng.add_norm(x, res, q=True, rstd=True)
    s = x.float() + res.float()
    assert torch.equal(o.sum.isnan(), s.isnan()) and torch.equal(o.sum.isinf(), s.isinf())
    assert o.y[1].isnan().all()
    for row, col in ((2, 0), (4, 263)):                   # infinite rms: the infinity gives NaN, the others 0
        assert o.y[row, col].isnan() and o.y[row].isnan().sum() == 1 and not o.y[row].nan_to_num().any()
    assert o.q_scale.isnan().tolist() == [False, True, True, False, True, False]
    clean = [0, 3, 5]                                     # the other rows are what they are alone
    alone = eng.add_norm(x[clean], res[clean], q=True)
    assert torch.equal(alone.y, o.y[clean]) and torch.equal(alone.q.view(torch.uint8), o.q[clean].view(torch.uint8))
    xi, ri = x.clone(), res.clone()
    eb.engram_add_norm(eng.ctx, xi, ri, 6, None, ri, xi, None, None, None)
    assert torch.equal(ri.view(torch.int16), o.sum.view(torch.int16))
    assert torch.equal(xi.view(torch.int16), o.y.view(torch.int16))


def test_add_norm_tiny_rows_keep_their_scale(eb):
    """values far below eps: the normed row is s / sqrt(eps); a scale below 1e-37 is divided by, not inverted"""
    d = 64
    eng = engine(eb, d, dtype="f32")
    x = torch.full((3, d), 1e-12, device="cuda")
    x[1], x[2] = 1e-38, 1e-42
    x[:, ::2] *= -0.5
    o = eng.add_norm(x, q=True)
    back = o.q.float() * o.q_scale[:, None]
    assert torch.isfinite(back).all()
    for r in (0, 1):
        assert (back[r] - o.y[r]).abs().max() <= 2.0 ** -4 * o.y[r].abs().max() + 2e-45
    assert (o.q.float()[0].abs().max(), o.q.float()[1].abs().max()) == (448, 448)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(1, 8), (37, 24), (1000, 264), (5003, 520), (700, 2560), (9, 5128), (40, 16384)])
@pytest.mark.parametrize("with_sum,with_gain", [(True, True), (False, False)])
def test_add_norm_grad(eb, n, d, with_sum, with_gain, dtype):
    eng = engine(eb, d, dtype=dtype)
    x = randn(1, n, d, sd=1.5, dtype=DT[dtype])
    gain = 1 + 0.1 * randn(3, d, dtype=torch.float32) if with_gain else None
    o = eng.add_norm(x, gain=gain, rstd=True)
    d_y = randn(4, n, d, sd=0.1, dtype=DT[dtype])
    d_sum = randn(5, n, d, sd=0.1, dtype=DT[dtype]) if with_sum else None
    d_x, d_gain = eng.add_norm_grad(d_y, o.sum, o.rstd, gain=gain, d_sum=d_sum)
    s, r, dy, g = f64(o.sum), f64(o.rstd), f64(d_y), None if gain is None else f64(gain)
    ds = None if d_sum is None else f64(d_sum)
    want, want_g = R.add_norm_grad(dy, s, r, g, ds)
    sh = np.abs(s * r[:, None])
    t = np.abs(dy if g is None else dy * g)
    mag = r[:, None] * (t + sh * (t * sh).mean(1, keepdims=True)) + (0 if ds is None else np.abs(ds))
    assert (np.abs(f64(d_x) - want) <= half_step(d_x) * np.abs(want) + 100 * U * mag).all()
    assert (np.abs(f64(d_gain) - want_g) <= (n + 4) * U * (np.abs(dy) * sh).sum(0)).all()
    again = eng.add_norm_grad(d_y, o.sum, o.rstd, gain=gain, d_sum=d_sum)
    assert torch.equal(again[0], d_x) and torch.equal(again[1], d_gain)
    into = d_y.clone()                                    # d_x over d_y, no gain gradient
    eb.engram_add_norm_grad(eng.ctx, into, d_sum, o.sum, o.rstd, n, gain, into, None, None, 0)
    assert torch.equal(into, d_x)


def test_add_norm_of_no_rows_and_refusals(eb):
    eng = engine(eb, 64)
    o = eng.add_norm(randn(1, 0, 64), q=True, rstd=True)
    assert o.y.shape == (0, 64) and o.q_scale.shape == (0,)
    d_x, d_gain = eng.add_norm_grad(randn(1, 0, 64), randn(1, 0, 64), torch.zeros(0, device="cuda"))
    assert d_x.shape == (0, 64) and not d_gain.any()
    x, r = randn(1, 4, 64), torch.zeros(4, device="cuda")
    q, ws = torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: eb.engram_add_norm(eng.ctx, x, None, 4, None, None, None, None, None, None),     # no output
        lambda: eb.engram_add_norm(eng.ctx, x, None, 4, None, None, None, q, None, None),        # codes without a scale
        lambda: eb.engram_add_norm(eng.ctx, x, None, -1, None, x, None, None, None, None),
        lambda: eb.engram_add_norm(eng.ctx, None, None, 4, None, x, None, None, None, None),
        lambda: eb.engram_add_norm(eng.ctx, x.view(-1)[1:], None, 3, None, x, None, None, None, None),
        lambda: eb.engram_add_norm_grad(eng.ctx, x, None, x, None, 4, None, x, None, None, 0),
        lambda: eb.engram_add_norm_grad(eng.ctx, x, None, x, r, 4, None, x, r, None, 0),
    ]
    for call in bad:
        with pytest.raises(eb.EngramError) as ei:
            call()
        assert ei.value.status == eb.ENGRAM_E_INVAL
    with pytest.raises(eb.EngramError) as ei:
        eb.engram_add_norm_grad(eng.ctx, x, None, x, r, 4, None, x, torch.zeros(64, device="cuda"), ws, 256)
    assert ei.value.status == eb.ENGRAM_E_NOMEM
    big = engine(eb, 32776)
    with pytest.raises(eb.EngramError) as ei:
        big.add_norm(randn(1, 1, 32776))
    assert ei.value.status == eb.ENGRAM_E_UNSUPPORTED
