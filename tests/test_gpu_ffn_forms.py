"""The feed-forward block's products in each form that their cut can take (whole
tiles, split contraction with partial sums, dealt tail, two tiles at once,
cluster), asserted through engram_debug_ffn_cut: a shape that no longer takes
the form it stands for fails.

The checks are those of test_gpu_ffn.  Its tolerances, derived for the
kernel's own arithmetic (u = 2^-24, m = 2^-8, p = 1 / (1 + 2^k') the logistic
function):
  k' = -log2(e) g for SiLU: the constant is within u / 4, the product within
  u; for GELU g (c1 g^2 + c0): the constants are products of two fp32 numbers,
  2.3 u each, g^2 u, the fma u, the product with g u: 5.3 u of |k'|;
  ex2.approx is within 2 ulp (4 u), the sum 1 + e within u, rcp.approx within
  1 ulp (2 u).  At |k'| <= 57.7 (beyond, p < 5e-18 or p = 1 to fp32) p is
  within 57.7 ln 2 * 5.3 u + 7 u = 219 u = 1.31e-5, and act(g) u, two products
  more, within 221 u = 1.32e-5 of itself (SiLU: 59 u = 3.6e-6 < 2^-17);
  stored in bf16 a value is off by m / (1 + m) of itself at most, so a value
  with a relative error D before it is within m / (1 + m) + (1 + m) D, which is
  at most m + 2^-17 as long as D <= (2^-17 + m^2 / (1 + m)) / (1 + m) = 2.27e-5."""

import time

import pytest

from test_gpu_ffn import inputs, test_ffn_fp8 as check_fp8, test_ffn_grad as check_grad
from test_gpu_residual import engine

torch = pytest.importorskip("torch")

PRODUCTS = {"gate_up": 0, "down": 1, "d_gate_up": 2, "d_Wd": 3, "d_x": 4, "d_Wgu": 5}


@pytest.fixture(scope="module")
def eb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_embedding_02_b200 as eb
    return eb


def cut(eb, eng, n, f, product):
    return eb.engram_debug_ffn_cut(eng.ctx, n, f, PRODUCTS[product])


def test_cut_of_a_null_context_is_refused():
    import hashed_gram_embedding_02_b200 as eb
    assert eb.engram_debug_ffn_cut(None, 4, 8, 0) is None


@pytest.mark.gpu
def test_cut_refuses_what_the_calls_refuse(eb):
    eng, f8, f32 = engine(eb, 128), engine(eb, 128, dtype="fp8"), engine(eb, 128, dtype="f32")
    ask = eb.engram_debug_ffn_cut
    for args in ((4, 64, -1), (4, 64, 6), (0, 64, 0), (-1, 64, 0), (4, 0, 0), (4, 12, 0)):
        assert ask(eng.ctx, *args) is None, args
    assert ask(f32.ctx, 4, 64, 0) is None and ask(f8.ctx, 4, 64, 2) is None
    assert ask(f8.ctx, 4, 64, 0) is not None and ask(eng.ctx, 4, 64, 5) is not None


# Narrow contexts with a batch of ordinary length: the weight gradients have at most 128 rows and a long contraction,
# so both operands are MN-major and the CTAs of a split are a cluster.
@pytest.mark.gpu
@pytest.mark.parametrize("n,d,f,in_cluster", [(1000, 128, 256, ["d_Wd"]), (4096, 128, 1024, ["d_Wd"]),
                                              (1500, 72, 136, ["d_Wd"]), (2284, 32, 64, ["d_Wd", "d_Wgu"]),
                                              (1777, 264, 56, ["d_Wgu"])])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_weight_gradients_in_a_cluster(eb, n, d, f, in_cluster, kind):
    eng = engine(eb, d)
    for name in in_cluster:
        assert cut(eb, eng, n, f, name) == ("cluster", False), name
    check_grad(eb, n, d, f, kind)


# E4M3 operands, tiles that do not fill a wave of SM pairs: the shares are raw sums, and the join applies the scales.
@pytest.mark.gpu
@pytest.mark.parametrize("n,d,f", [(1095, 3200, 3728), (552, 3200, 6392), (3777, 3584, 1280)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_dealt_tail_fp8(eb, n, d, f, kind):
    assert cut(eb, engine(eb, d, dtype="fp8"), n, f, "gate_up") == ("dealt", True)
    check_fp8(eb, n, d, f, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("n,d,f", [(6389, 2560, 296), (300, 4096, 6000)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_two_tiles_fp8(eb, n, d, f, kind):
    assert cut(eb, engine(eb, d, dtype="fp8"), n, f, "gate_up") == ("two tiles", True)
    check_fp8(eb, n, d, f, kind)


# A stage that is announced and never loaded, in each form of the gate/up product: the waits run out, CTAs that did not
# abort meet those that did at their barriers, the joins add sums that were never written, and the down product, which
# may have started early, gives up too.  All of it ends by itself, and the next call gives the right bits.
@pytest.mark.gpu
@pytest.mark.parametrize("n,d,f,form", [(1, 1152, 1456, ("cluster", False)), (512, 2560, 5000, ("two tiles", True)),
                                        (300, 2560, 264, ("split", True)), (6389, 2504, 296, ("dealt", True))])
@pytest.mark.parametrize("save", [False, True])
def test_stalled_forms_time_out_and_the_context_recovers(eb, n, d, f, form, save):
    eng = engine(eb, d)
    assert cut(eb, eng, n, f, "gate_up") == form
    x, Wgu, Wd = inputs(n, d, f)
    want = eng.ffn(x, Wgu, Wd, save=True)
    torch.cuda.synchronize()
    eb.engram_debug_stall_next(eng.ctx)
    t0 = time.time()
    eng.ffn(x, Wgu, Wd, save=save)
    st, flags = eng.status()
    assert st == eb.ENGRAM_E_TIMEOUT and flags & eb.ENGRAM_ERR_TIMEOUT, (st, flags)
    assert time.time() - t0 < 30.0
    again = eng.ffn(x, Wgu, Wd, save=True)
    assert torch.equal(again[0], want[0])
    a = n * ((f + 63) // 64 * 64) * 2                     # the saved a: its rows' padding is not written
    assert torch.equal(again[1][:a].view(n, -1)[:, :f * 2], want[1][:a].view(n, -1)[:, :f * 2])
    assert eng.status() == (eb.ENGRAM_OK, 0)
