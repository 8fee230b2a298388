"""Gated feed-forward block on the GPU against the plain fp64 reference
(oracle.residual).

Tolerances, with m = 2^-8 (half a bf16 step, torch.finfo(bfloat16).eps / 2):
  a product of K terms accumulated in fp32 by the tensor cores is within
  K 2^-23 of the sum of magnitudes (2^-23 a term: the adder may truncate);
  the logistic function p through __expf and a fast division: the exponent k
  carries 2^-24 |k| and __expf 2 + 1.2 |k| ulp, so at |k| <= 40 (beyond, p is
  0 or 1 to fp32) p is within 2^-17 relative; act' within 2^-15 absolute
  (its terms are at most 2 in magnitude);
  each value stored in bf16 adds m of it, g and u saved with 24 bits (15 of
  the mantissa, cut off; the low byte is repeated below itself when read) one
  step, 2^-15 of theirs.  |act'| <= 1.13.
The bounds are carried through the products with magnitudes."""

import numpy as np
import pytest

from oracle import residual as R
from test_gpu_residual import engine, f64, randn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

M = 2.0 ** -8
A23 = 2.0 ** -23


@pytest.fixture(scope="module")
def eb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_embedding_02_b200 as eb
    return eb


def inputs(n, d, f, seed=1):
    x = randn(seed, n, d)
    Wgu, Wd = randn(seed + 1, 2 * f, d, sd=d ** -0.5), randn(seed + 2, d, f, sd=f ** -0.5)
    return x, Wgu, Wd


def planes(saved, n, f):
    """(g and u [n][2f] fp32, a [n][f] bf16) of what the forward saves: a (rows of whole 128-byte lines), then two
    planes of 8-column elements blocked [row / 32][column / 8][row % 32]"""
    rb, ld = (n + 31) // 32, (f + 63) // 64 * 64
    cut = n * ld * 2
    elems = rb * 32 * (f // 4)
    shape = (rb, f // 4, 32, 8)
    hi = saved[cut:cut + elems * 16].view(torch.int16).view(shape).to(torch.int32) << 16
    lo = saved[cut + elems * 16:].view(shape).to(torch.int32) * 0x101
    gu = (hi | lo).permute(0, 2, 1, 3).reshape(rb * 32, 2 * f)[:n].contiguous().view(torch.float32)
    return gu, saved[:cut].view(torch.bfloat16).view(n, ld)[:, :f]


def check_forward(y, saved, x, Wgu, Wd, kind, res=None):
    """x, Wgu, Wd, res in fp64"""
    f, d = Wd.shape[1], Wd.shape[0]
    want, guw = R.ffn(x, Wgu, Wd, kind, res)
    e_gu = d * A23 * (np.abs(x) @ np.abs(Wgu).T)
    if saved is not None:
        gu = planes(saved, x.shape[0], f)[0]
        assert (np.abs(f64(gu) - guw) <= 2.0 ** -15 * np.abs(guw) + (1 + M) * e_gu).all()
    h, u = R.act(guw[:, :f], kind)[0], guw[:, f:]
    a = np.abs(h * u)
    e_a = (M + 2.0 ** -17) * a + 1.13 * e_gu[:, :f] * np.abs(u) + np.abs(h) * e_gu[:, f:]
    if saved is not None:
        assert (np.abs(f64(planes(saved, x.shape[0], f)[1]) - h * u) <= (1 + M) * e_a).all()
    bound = M * np.abs(want) + (1 + M) * (e_a + f * A23 * a) @ np.abs(Wd).T + 1e-6
    err = np.abs(f64(y) - want)
    assert (err <= bound).all(), (int((err > bound).sum()), float(err.max()))


SHAPES = [(1, 64, 8), (1, 256, 72), (7, 136, 200), (128, 128, 128), (129, 264, 136), (200, 8, 24), (256, 512, 1000),
          (300, 2560, 264), (513, 72, 2056), (1000, 520, 392), (2, 520, 20000)]


@pytest.mark.parametrize("n,d,f", SHAPES)
@pytest.mark.parametrize("kind,with_res", [("silu", True), ("gelu", False)])
def test_ffn(eb, n, d, f, kind, with_res):
    eng = engine(eb, d)
    x, Wgu, Wd = inputs(n, d, f)
    res = randn(9, n, d) if with_res else None
    y, saved = eng.ffn(x, Wgu, Wd, act=kind, res=res, save=True)
    assert eng.status() == (eb.ENGRAM_OK, 0)
    check_forward(y, saved, f64(x), f64(Wgu), f64(Wd), kind, None if res is None else f64(res))
    assert torch.equal(eng.ffn(x, Wgu, Wd, act=kind, res=res), y)       # the same bits without saving


@pytest.mark.parametrize("n,d,f", [(1, 128, 8), (7, 128, 200), (129, 256, 136), (300, 2560, 264), (1000, 640, 392)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ffn_fp8(eb, n, d, f, kind):
    eng = engine(eb, d, dtype="fp8")
    x, Wgu, Wd = inputs(n, d, f)
    o = eng.add_norm(x, sum=False, y=False, q=True)
    scale = Wgu.float().abs().amax(1) / 448
    Wq = (Wgu.float() / scale[:, None]).to(torch.float8_e4m3fn)
    y = eng.ffn(o.q, Wq, Wd, act=kind, x_scale=o.q_scale, gu_scale=scale)
    assert eng.status() == (eb.ENGRAM_OK, 0)
    check_forward(y, None, f64(o.q.float()) * f64(o.q_scale)[:, None], f64(Wq.float()) * f64(scale)[:, None], f64(Wd), kind)


@pytest.mark.parametrize("n,d,f", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ffn_grad(eb, n, d, f, kind):
    eng = engine(eb, d)
    x, Wgu, Wd = inputs(n, d, f)
    _, saved = eng.ffn(x, Wgu, Wd, act=kind, save=True)
    d_y = randn(7, n, d, sd=0.5)
    got = eng.ffn_grad(d_y, x, saved, Wgu, Wd, act=kind)
    assert eng.status() == (eb.ENGRAM_OK, 0)
    X, W, D, G, dy = f64(x), f64(Wgu), f64(Wd), f64(planes(saved, n, f)[0]), f64(d_y)
    want = R.ffn_grad(dy, X, G, W, D, kind)
    h, dh = R.act(G[:, :f], kind)
    u = G[:, f:]
    da = dy @ D
    e_da = d * A23 * (np.abs(dy) @ np.abs(D))
    dg, du = da * u * dh, da * h
    e_dg = M * np.abs(dg) + (1 + M) * (e_da * np.abs(u * dh) + 2.0 ** -15 * np.abs(da * u))
    e_du = M * np.abs(du) + (1 + M) * (e_da * np.abs(h) + 2.0 ** -17 * np.abs(du))
    dgu, e = np.abs(np.concatenate([dg, du], 1)), np.concatenate([e_dg, e_du], 1)
    a = np.abs(h * u)
    bounds = ((e + 2 * f * A23 * dgu) @ np.abs(W), (e + n * A23 * dgu).T @ np.abs(X),
              np.abs(dy).T @ ((M + 2.0 ** -17 + n * A23) * a))
    for g, w, b, name in zip(got, want, bounds, ("d_x", "d_Wgu", "d_Wd")):
        err = np.abs(f64(g) - w)
        bound = M * np.abs(w) + (1 + M) * b + 1e-6
        assert (err <= bound).all(), (name, int((err > bound).sum()), float(err.max()))
    again = eng.ffn_grad(d_y, x, saved, Wgu, Wd, act=kind)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


# Tiles that do not fill a wave of SM pairs, each product's in turn: their contraction is shared among pairs, with
# and without whole waves before them.
@pytest.mark.parametrize("n,d,f", [(6389, 2504, 296), (6654, 264, 4936), (6275, 536, 1504), (399, 1400, 9648),
                                   (6240, 144, 6328)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ffn_shared_tiles(eb, n, d, f, kind):
    test_ffn(eb, n, d, f, kind, kind == "gelu")
    test_ffn_grad(eb, n, d, f, kind)


# Few rows: the CTAs that split a tile's contraction add their sums through each other's shared memory.
@pytest.mark.parametrize("n,d,f", [(1, 1152, 1456), (4, 1280, 1488), (37, 1784, 1960), (100, 1024, 4096), (128, 136, 5000)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ffn_few_rows(eb, n, d, f, kind):
    test_ffn(eb, n, d, f, kind, kind == "gelu")
    test_ffn_grad(eb, n, d, f, kind)


@pytest.mark.parametrize("n,d,f", [(1, 2560, 512), (3, 384, 1952), (20, 384, 7824), (128, 2432, 312)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ffn_few_rows_fp8(eb, n, d, f, kind):
    test_ffn_fp8(eb, n, d, f, kind)


# Between one and two waves of gate and up tiles: a pair takes two at once; the last pair of an odd number has one.
@pytest.mark.parametrize("n,d,f", [(200, 2560, 10240), (512, 2560, 5000), (700, 2048, 4096)])
@pytest.mark.parametrize("kind,with_res", [("silu", True), ("gelu", False)])
def test_ffn_two_tiles_at_once(eb, n, d, f, kind, with_res):
    test_ffn(eb, n, d, f, kind, with_res)


@pytest.mark.parametrize("n,d,f", [(6389, 2560, 296), (6240, 128, 6328), (300, 4096, 6000)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ffn_shared_tiles_fp8(eb, n, d, f, kind):
    test_ffn_fp8(eb, n, d, f, kind)


@pytest.mark.parametrize("n", [1, 5, 300])
def test_ffn_products_are_exact_on_small_integers(eb, n):
    """Gates far above zero (act(g) = g to fp32) and small integers make every product exact: a row, column or
    contraction index out of place shows as a wrong integer."""
    d, f = 72, 136
    eng = engine(eb, d)
    rng = np.random.default_rng(n)
    x = rng.integers(0, 2, (n, d)).astype(float)
    x[:, 0] = 1
    Wg, Wu = np.zeros((f, d)), np.zeros((f, d))
    Wg[:, 0] = 128                                        # g = 128 + (0 or 1), act(g) = g
    Wg[np.arange(f), 1 + rng.integers(0, d - 1, f)] = 1
    Wu[np.arange(f), rng.integers(0, d, f)] = 1           # u = 0 or 1
    Wd = np.zeros((d, f))
    Wd[rng.integers(0, d, f // 2), rng.choice(f, f // 2, replace=False)] = 1
    up = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()
    W = np.concatenate([Wg, Wu])
    g, u = x @ Wg.T, x @ Wu.T
    y, saved = eng.ffn(up(x), up(W), up(Wd), save=True)
    assert np.array_equal(f64(planes(saved, n, f)[0]), np.concatenate([g, u], 1))
    a = g * u
    assert np.array_equal(f64(y), f64(up(a @ Wd.T)))
    dy = rng.integers(0, 2, (n, d)).astype(float)
    d_x, d_Wgu, d_Wd = eng.ffn_grad(up(dy), up(x), saved, up(W), up(Wd))
    da = dy @ Wd
    dgu = f64(up(np.concatenate([da * u, da * g], 1)))    # act'(g) = 1; sums of two rounded to bf16 as stored
    assert np.array_equal(f64(d_x), f64(up(dgu @ W)))
    assert np.array_equal(f64(d_Wgu), f64(up(dgu.T @ x)))
    assert np.array_equal(f64(d_Wd), f64(up(dy.T @ a)))


def test_ffn_in_place_residual_and_no_rows(eb):
    eng = engine(eb, 264)
    x, Wgu, Wd = inputs(130, 264, 136)
    y = eng.ffn(x, Wgu, Wd, res=x)
    need = eb.engram_ffn_workspace_bytes(eng.ctx, 130, 136)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    into = x.clone()
    eb.engram_ffn(eng.ctx, into, None, 130, 136, 0, Wgu, None, Wd, into, into, None, ws, need)
    assert torch.equal(into, y)
    none = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    y0, saved0 = eng.ffn(none, Wgu, Wd, save=True)
    assert y0.shape == (0, 264) and saved0.shape == (0,)
    d_x, d_Wgu, d_Wd = eng.ffn_grad(y0, none, saved0, Wgu, Wd)
    assert d_x.shape == (0, 264) and not d_Wgu.any() and not d_Wd.any()


def test_ffn_rows_are_those_of_a_longer_call(eb):
    """rows behind the last one of the call are neither read nor written, and NaN in them reaches no other row"""
    eng = engine(eb, 136)
    x, Wgu, Wd = inputs(400, 136, 200)
    x[150:] = float("nan")
    ws_bytes = eb.engram_ffn_workspace_bytes(eng.ctx, 150, 200)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    y = torch.full((400, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    eb.engram_ffn(eng.ctx, x, None, 150, 200, 0, Wgu, None, Wd, None, y, None, ws, ws_bytes)
    check_forward(y[:150], None, f64(x[:150]), f64(Wgu), f64(Wd), "silu")
    assert (y[150:] == 7).all()


def test_ffn_refuses(eb):
    eng, f32, f8 = engine(eb, 128), engine(eb, 128, dtype="f32"), engine(eb, 128, dtype="fp8")
    x, Wgu, Wd = inputs(4, 128, 64)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    y, s = torch.empty_like(x), torch.ones(128, device="cuda")

    def call(e=eng, n=4, f=64, act=0, x=x, xs=None, gs=None, saved=None, ws=ws, size=ws.numel()):
        eb.engram_ffn(e.ctx, x, xs, n, f, act, Wgu, gs, Wd, None, y, saved, ws, size)

    for kw in (dict(n=-1), dict(f=0), dict(f=12), dict(act=2), dict(x=None), dict(xs=s), dict(ws=ws[1:], size=ws.numel() - 1),
               dict(ws=None), dict(x=x.view(-1)[1:]), dict(e=f8), dict(e=f8, xs=s, gs=s, saved=Wgu)):
        with pytest.raises(eb.EngramError) as ei:
            call(**kw)
        assert ei.value.status == eb.ENGRAM_E_INVAL, kw
    with pytest.raises(eb.EngramError) as ei:
        call(size=256)
    assert ei.value.status == eb.ENGRAM_E_NOMEM
    for e, fn in ((f32, call), (f8, None)):
        with pytest.raises(eb.EngramError) as ei:
            if fn:
                fn(e=e)
            else:
                eb.engram_ffn_grad(e.ctx, y, x, x, 4, 64, 0, Wgu, Wd, y, Wgu, Wd, ws, ws.numel())
        assert ei.value.status == eb.ENGRAM_E_UNSUPPORTED
    assert eb.engram_ffn_workspace_bytes(f32.ctx, 4, 64) == 0
    assert eb.engram_ffn_grad_workspace_bytes(f8.ctx, 4, 64) == 0
