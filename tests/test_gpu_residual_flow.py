"""The residual-stream calls together, as a layer uses them: token embedding,
the module, the residual sum with its norm, the feed-forward block, and the way
back; eager, on a side stream, captured and replayed; large offsets; and the
feed-forward block's bounded waits.  Stage tolerances are those of
test_gpu_residual and test_gpu_ffn."""

import time

import numpy as np
import pytest

import synth
from gpu_helpers import DeviceInputs, config_for
from oracle import residual as R
from test_gpu_ffn import check_forward, inputs
from test_gpu_residual import U, check_embed_grad, engine, f64, half_step, randn, tokens

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

WL = synth.WORKLOADS["c2"].replace(name="flow", B=3, T=111, V=4096, Vc=3154, M=10007, d=512, seed=81)
F = 1000
SCALE = float(np.float32(0.5))


@pytest.fixture(scope="module")
def eb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_embedding_02_b200 as eb
    return eb


class Layer:
    """one layer's inputs and a training step through it"""

    def __init__(self, eb, seed=1):
        self.inp = synth.Inputs(WL, gamma="random")
        self.di = DeviceInputs(self.inp)
        self.eng = eb.Engram(config_for(self.inp, eb), B=WL.B, L=WL.T)
        self.tok = self.di.tok.view(WL.B, -1)[:, :WL.T]
        self.E = randn(seed, WL.V, WL.d, sd=2.0)
        self.gain = 1 + 0.1 * randn(seed + 1, WL.d, dtype=torch.float32)
        _, self.Wgu, self.Wd = inputs(1, WL.d, F, seed + 2)
        self.d_out = randn(seed + 5, WL.n_tok, WL.d, sd=0.1)

    def forward(self, stream=None):
        o = {"h": self.eng.embed(self.tok, self.E, scale=SCALE, stream=stream)}
        o["y"] = torch.empty_like(o["h"])
        self.eng.forward(self.tok, self.di.P, self.di.tables, o["h"], self.di.Wk, self.di.Wv, self.di.conv_w, o["y"],
                         gq=self.di.gq, gk=self.di.gk, stream=stream)
        o["norm"] = self.eng.add_norm(o["y"], o["h"], gain=self.gain, q=True, rstd=True, stream=stream)
        o["out"], o["saved"] = self.eng.ffn(o["norm"].y, self.Wgu, self.Wd, res=o["norm"].sum, save=True, stream=stream)
        return o

    def backward(self, o, stream=None):
        """gradients of the block's weights, the gain and E (by the path past the module)"""
        e, nm = self.eng, o["norm"]
        g = {}
        g["n"], g["Wgu"], g["Wd"] = e.ffn_grad(self.d_out, nm.y, o["saved"], self.Wgu, self.Wd, stream=stream)
        g["s"], g["gain"] = e.add_norm_grad(g["n"], nm.sum, nm.rstd, gain=self.gain, d_sum=self.d_out, stream=stream)
        g["E"] = e.embed_grad(self.tok, g["s"], scale=SCALE, stream=stream)
        return g

    def step(self, stream=None):
        o = self.forward(stream)
        return o, self.backward(o, stream)


def flat(o, g):
    nm = o["norm"]
    return [o["h"], o["y"], nm.sum, nm.y, nm.q.view(torch.uint8), nm.q_scale, nm.rstd, o["out"]] + list(g.values())


def test_layer_step_matches_the_reference_stage_by_stage(eb):
    la = Layer(eb)
    o, g = la.step()
    torch.cuda.synchronize()
    assert la.eng.status() == (eb.ENGRAM_OK, 0)
    h = la.E.float()[la.tok.reshape(-1).long()] * SCALE
    assert torch.equal(o["h"], h.to(torch.bfloat16))
    y = torch.empty_like(o["y"])                          # the module on the same rows
    la.eng.forward(la.tok, la.di.P, la.di.tables, h.to(torch.bfloat16), la.di.Wk, la.di.Wv, la.di.conv_w, y,
                   gq=la.di.gq, gk=la.di.gk)
    assert torch.equal(o["y"], y)
    nm = o["norm"]
    s, r, ny = R.add_norm(f64(o["y"]), f64(o["h"]), f64(la.gain), float(np.float32(1e-6)))
    m = half_step(nm.y)
    assert (np.abs(f64(nm.sum) - s) <= (m + U) * np.abs(s)).all()
    assert (np.abs(f64(nm.y) - ny) <= (m + 96 * U) * np.abs(ny)).all()
    check_forward(o["out"], o["saved"], f64(nm.y), f64(la.Wgu), f64(la.Wd), "silu", f64(nm.sum))
    s, r, dn = f64(nm.sum), f64(nm.rstd), f64(g["n"])
    want, want_g = R.add_norm_grad(dn, s, r, f64(la.gain), f64(la.d_out))
    sh, t = np.abs(s * r[:, None]), np.abs(dn * f64(la.gain))
    mag = r[:, None] * (t + sh * (t * sh).mean(1, keepdims=True)) + np.abs(f64(la.d_out))
    assert (np.abs(f64(g["s"]) - want) <= m * np.abs(want) + 100 * U * mag).all()
    assert (np.abs(f64(g["gain"]) - want_g) <= (WL.n_tok + 4) * U * (np.abs(dn) * sh).sum(0)).all()
    check_embed_grad(g["E"], la.tok, g["s"], WL.V, SCALE)


def test_layer_step_on_a_side_stream_gives_the_same_bits(eb):
    la = Layer(eb)
    want = flat(*la.step())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(3):                                    # memory goes round in the side stream's order
        got = flat(*la.step(stream=side))
    raw = flat(*la.step(stream=side.cuda_stream))         # the raw handle
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(want, raw))


def test_two_layers_on_two_streams(eb):
    a, b = Layer(eb, 1), Layer(eb, 30)
    wa, wb = flat(*a.step()), flat(*b.step())
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        ga, gb = flat(*a.step(stream=sa)), flat(*b.step(stream=sb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(wa, ga))
    assert all(torch.equal(x, y) for x, y in zip(wb, gb))


def test_captured_steps_replay_the_eager_bits(eb):
    """two graphs of the same layer, replayed in turn with the inputs changed in between"""
    la = Layer(eb)
    la.step()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(flat(*la.step()))
        graphs.append(g)
    tok0, E0 = la.tok.clone(), la.E.clone()
    for k in range(4):
        la.tok.copy_(tokens(50 + k, WL.B, WL.T, WL.V, ["zipf", "one", "distinct", "half"][k]))
        la.E.copy_(randn(60 + k, WL.V, WL.d, sd=2.0))
        want = [t.clone() for t in flat(*la.step())]
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs[k % 2])), k
    la.tok.copy_(tok0)
    la.E.copy_(E0)
    want = [t.clone() for t in flat(*la.step())]
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    del graphs, outs


@pytest.mark.parametrize("T", [500, 3000, 20011])         # the sorts of one CTA, narrow and wide, and of several
def test_captured_embedding_gradient(eb, T):
    eng = engine(eb, 264, 70001)                          # 74 MB: the untouched rows are cleared apart
    small = engine(eb, 264, 5000)                         # cleared whole
    for e, V in ((eng, 70001), (small, 5000)):
        tok, d_h = tokens(1, 2, T, V), randn(2, 2 * T, 264)
        out = torch.full((V, 264), 3.0, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        e.embed_grad(tok, d_h, out=out, stream=side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            e.embed_grad(tok, d_h, out=out)
        for k, kind in enumerate(("half", "one", "distinct")):
            tok.copy_(tokens(k + 5, 2, T, V, kind))
            out.fill_(float("nan"))
            g.replay()
            assert torch.equal(out, e.embed_grad(tok, d_h)), kind


def test_embed_grad_into_rows_of_16_byte_alignment(eb):
    eng = engine(eb, 72, 500)
    tok, d_h = tokens(1, 3, 700, 500), randn(2, 2100, 72)
    want = eng.embed_grad(tok, d_h)
    flat = torch.full((500 * 72 + 8,), 9.0, device="cuda")
    out = flat[4:-4].view(500, 72)
    assert out.data_ptr() % 32 == 16
    assert torch.equal(eng.embed_grad(tok, d_h, out=out), want)
    assert (flat[:4] == 9).all() and (flat[-4:] == 9).all()


def test_norm_codes_feed_the_fp8_block(eb):
    """the 8-bit path: embed, norm with E4M3 output, feed-forward block on the codes, residual"""
    d, f, n = 256, 392, 77
    eng = engine(eb, d, dtype="fp8")
    h = eng.embed(tokens(1, 7, 11, 50), randn(2, 50, d))
    o = eng.add_norm(h, randn(3, n, d), y=False, q=True)
    _, Wgu, Wd = inputs(1, d, f)
    scale = Wgu.float().abs().amax(1) / 448
    Wq = (Wgu.float() / scale[:, None]).to(torch.float8_e4m3fn)
    y = eng.ffn(o.q, Wq, Wd, x_scale=o.q_scale, gu_scale=scale, res=o.sum)
    check_forward(y, None, f64(o.q.float()) * f64(o.q_scale)[:, None], f64(Wq.float()) * f64(scale)[:, None], f64(Wd),
                  "silu", f64(o.sum))
    with pytest.raises(ValueError, match="float8"):
        eng.ffn(h, Wgu, Wd, x_scale=o.q_scale, gu_scale=scale)
    with pytest.raises(ValueError, match="save"):
        eng.ffn(o.q, Wq, Wd, x_scale=o.q_scale, gu_scale=scale, save=True)


# ---------------------------------------------------------------- large offsets

def test_embed_beyond_32_bit_offsets(eb):
    V, d = 900001, 2560                                   # 2.3e9 elements
    eng = engine(eb, d, V)
    tok = torch.tensor([[V - 1, 0, 838861, V - 2, V - 1]], dtype=torch.int32, device="cuda")
    E = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    rows = tok.view(-1).long()
    E[rows] = randn(1, 5, d)
    assert torch.equal(eng.embed(tok, E), E[rows])
    del E
    d_h = randn(2, 5, d)
    g = eng.embed_grad(tok, d_h)
    want = torch.zeros(4, d, dtype=torch.float64, device="cuda")
    want[0] = d_h[1].double()
    want[1] = d_h[2].double()
    want[2] = d_h[3].double()
    want[3] = d_h[0].double() + d_h[4].double()
    at = torch.tensor([0, 838861, V - 2, V - 1], device="cuda")
    assert torch.equal(g[at], want.float())               # sums of two bf16 values are exact to fp32 here
    assert int(torch.count_nonzero(g)) == int(torch.count_nonzero(want))


def test_embed_grad_of_a_long_batch(eb):
    """1.2e6 positions: sort parts of several tiles, three digit passes"""
    B, T, V, d = 3, 400001, 300000, 8
    eng = engine(eb, d, V)
    tok = tokens(1, B, T, V, "half")
    d_h = randn(2, B * T, d)
    got = eng.embed_grad(tok, d_h)
    idx = tok.view(-1).long()
    want = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, idx, d_h.double())
    mag = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, idx, d_h.double().abs())
    cnt = torch.bincount(idx, minlength=V)[:, None]
    # a sum of k terms: pieces of at most 32, then at most k / 32 parts in two halves, so at most 32 + k / 64 + 2
    # additions in a row (plus the product with the scale)
    depth = 36 + cnt.double() / 64
    assert bool(((got.double() - want).abs() <= depth * U * mag).all())
    assert torch.equal(got, eng.embed_grad(tok, d_h))


def test_ffn_beyond_32_bit_offsets(eb):
    n, d, f = 110007, 256, 10240                          # 2.25e9 saved values of g and u
    eng = engine(eb, d)
    x, Wgu, Wd = inputs(n, d, f)
    y, saved = eng.ffn(x, Wgu, Wd, save=True)
    d_y = randn(5, n, d, sd=0.1)
    d_x, d_Wgu, d_Wd = eng.ffn_grad(d_y, x, saved, Wgu, Wd)
    assert eng.status() == (eb.ENGRAM_OK, 0)
    for lo in (0, 104857, n - 33):                        # row 104857: the element offset passes 2^31
        rows = slice(lo, lo + 33)
        check_forward(y[rows], None, f64(x[rows]), f64(Wgu), f64(Wd), "silu")
        # the rows alone: both calls are within the bound of test_gpu_ffn of the same value, whose terms of
        # d_x are: its rounding, and 2^-8 a value of dg and du (summed here with their magnitudes)
        y1, s1 = eng.ffn(x[rows].contiguous(), Wgu, Wd, save=True)
        one = eng.ffn_grad(d_y[rows].contiguous(), x[rows].contiguous(), s1, Wgu, Wd)[0]
        gu = f64(x[rows]) @ f64(Wgu).T
        a, da = R.act(gu[:, :f], "silu")
        d_a = f64(d_y[rows]) @ f64(Wd)
        dgu = np.abs(np.concatenate([d_a * gu[:, f:] * da, d_a * a], 1))
        bound = 2 * (2.0 ** -8 * np.abs(f64(one)) + 1.02 * 2.0 ** -8 * (dgu @ np.abs(f64(Wgu))))
        assert (np.abs(f64(d_x[rows]) - f64(one)) <= bound).all()


# ---------------------------------------------------------------- bounded waits

@pytest.mark.parametrize("n", [5, 700])                   # one CTA per tile, and CTA pairs
def test_stalled_ffn_times_out_and_the_context_recovers(eb, n):
    eng = engine(eb, 256)
    x, Wgu, Wd = inputs(n, 256, 520)
    want = eng.ffn(x, Wgu, Wd)
    torch.cuda.synchronize()
    eb.engram_debug_stall_next(eng.ctx)
    t0 = time.time()
    eng.ffn(x, Wgu, Wd)
    st, flags = eng.status()
    assert st == eb.ENGRAM_E_TIMEOUT and flags & eb.ENGRAM_ERR_TIMEOUT, (st, flags)
    assert time.time() - t0 < 30.0
    assert torch.equal(eng.ffn(x, Wgu, Wd), want)
    assert eng.status() == (eb.ENGRAM_OK, 0)
