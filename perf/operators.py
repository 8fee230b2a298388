"""The operators around the Engram module in the residual stream, as measured
work: the token embedding and its gradient, the residual sum with RMSNorm (and
an E4M3 output), and the gated feed-forward block with its backward.

`listed()` and `draw()` give cases (plain dicts), `prepare()` makes a case's
inputs on the GPU from a seed, `run()` makes one pass: in elementary torch
operations (`own` false) or through the package's entry points (`own` true).
`work()` counts the bytes and operations a pass cannot do without and
`exact()` evaluates the definitions in 64 bits.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token for each of 256 sequences: latency of a short gather
        {"name": "embed-decode", "op": "embed", "B": 256, "T": 1, "V": 128000, "d": 2560, "dtype": "bf16",
         "scale": 1.0, "zipf": 1.0},
        # a prefill or training batch of 8 x 4096 tokens, rows scaled by sqrt(d)
        {"name": "embed-prefill", "op": "embed", "B": 8, "T": 4096, "V": 128000, "d": 2560, "dtype": "bf16",
         "scale": math.sqrt(2560.0), "zipf": 1.1},
        # a micro-batch of the smallest configuration, fp32 (one sequence of 256 tokens)
        {"name": "embed-grad-small", "op": "embed_grad", "B": 1, "T": 256, "V": 4096, "d": 256, "dtype": "f32",
         "scale": 1.0, "zipf": 1.1},
        # the gradient of the 8 x 4096 batch: Zipf tokens, so a few rows take thousands of positions
        {"name": "embed-grad", "op": "embed_grad", "B": 8, "T": 4096, "V": 128000, "d": 2560, "dtype": "bf16",
         "scale": math.sqrt(2560.0), "zipf": 1.1},
        # decode step of 256 sequences: residual, norm and the 8-bit operand of the next projection
        {"name": "norm-decode-fp8", "op": "norm", "n": 256, "d": 2560, "dtype": "bf16", "y": False, "q": True},
        # prefill of 8 x 4096: both the bf16 and the 8-bit form of the normed rows (two consumers)
        {"name": "norm-prefill-both", "op": "norm", "n": 32768, "d": 2560, "dtype": "bf16", "y": True, "q": True},
        # training backward of a packed batch with an odd number of rows
        {"name": "norm-grad", "op": "norm_grad", "n": 16381, "d": 2560, "dtype": "bf16"},
        # one sequence, one token: the weights are read once for one row
        {"name": "ffn-token", "op": "ffn", "n": 1, "d": 2560, "f": 10240, "act": "silu", "fp8": False, "res": True},
        # decode step of 256 sequences
        {"name": "ffn-decode", "op": "ffn", "n": 256, "d": 2560, "f": 10240, "act": "silu", "fp8": False, "res": True},
        # prefill of 8 x 4096 tokens, 16-bit
        {"name": "ffn-prefill", "op": "ffn", "n": 32768, "d": 2560, "f": 10240, "act": "silu", "fp8": False,
         "res": True},
        # ragged prefill in 8 bits: x and the gate/up weights in E4M3
        {"name": "ffn-prefill-fp8", "op": "ffn", "n": 8 * 4091, "d": 2560, "f": 10240, "act": "silu", "fp8": True,
         "res": False},
        # a training step of the block: forward and backward, rows and inner width off the tile sizes
        {"name": "ffn-train", "op": "ffn_train", "n": 4 * 4093, "d": 2560, "f": 6824, "act": "gelu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "ffn", "ffn", "ffn_train"])
    if op in ("embed", "embed_grad"):
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, 32768 // B))
        return {"op": op, "B": B, "T": T, "V": _log(rng, 512, 128000), "d": 8 * _log(rng, 8, 320),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "scale": rng.choice([1.0, 16.0, 0.37]),
                "zipf": rng.choice([0.0, 1.0, 1.1, 1.5])}
    if op == "norm":
        y, q = rng.choice([(True, False), (False, True), (True, True)])
        return {"op": op, "n": _log(rng, 1, 32768), "d": 8 * _log(rng, 8, 320),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "y": y, "q": q}
    if op == "norm_grad":
        return {"op": op, "n": _log(rng, 1, 32768), "d": 8 * _log(rng, 8, 320),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    act = rng.choice(["silu", "gelu"])
    if op == "ffn":
        fp8 = rng.random() < 0.3
        d = 128 * _log(rng, 1, 20) if fp8 else 8 * _log(rng, 16, 320)
        f = 8 * _log(rng, 32, 1280)
        return {"op": op, "n": _log(rng, 1, 32768), "d": d, "f": f, "act": act, "fp8": fp8,
                "res": rng.random() < 0.5}
    return {"op": op, "n": _log(rng, 1, 16384), "d": 8 * _log(rng, 16, 320), "f": 8 * _log(rng, 32, 850), "act": act}


def _es(case):
    return 4 if case.get("dtype") == "f32" else 2


def _distinct(case):
    """Expected number of distinct tokens of the batch's Zipf law."""
    n, V, s = case["B"] * case["T"], case["V"], case["zipf"]
    w = torch.arange(1, V + 1, dtype=torch.float64).pow(-s)
    return float((1.0 - (1.0 - w / w.sum()).pow(n)).sum())


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        n, d, es = case["B"] * case["T"], case["d"], _es(case)
        if op == "embed":
            return {"bytes": n * 4 + _distinct(case) * d * es + n * d * es, "flops": n * d}
        return {"bytes": n * 4 + n * d * es + case["V"] * d * 4, "flops": n * d}
    n, d = case["n"], case["d"]
    if op == "norm":
        es = _es(case)
        per = 3 * es + (es if case["y"] else 0) + (1 if case["q"] else 0)
        return {"bytes": n * d * per + d * 4 + (n * 4 if case["q"] else 0), "flops": 6 * n * d}
    if op == "norm_grad":
        return {"bytes": 4 * n * d * _es(case) + n * 4 + 2 * d * 4, "flops": 10 * n * d}
    f = case["f"]
    if op == "ffn":
        xe = 1 if case["fp8"] else 2
        b = n * d * xe + 2 * f * d * xe + f * d * 2 + n * d * 2 + (n * d * 2 if case["res"] else 0)
        if case["fp8"]:
            b += n * 4 + 2 * f * 4
        return {"bytes": b, "flops": 6 * n * d * f}
    # x, dy, y, dx; the three weights read, their gradients written
    return {"bytes": 4 * n * d * 2 + 6 * d * f * 2, "flops": 18 * n * d * f}


# ---------------------------------------------------------------- inputs

class _State:
    def __init__(self, case):
        self.case = case
        self.eng = None


def _tokens(case, gen, dev):
    n, V = case["B"] * case["T"], case["V"]
    w = torch.arange(1, V + 1, device=dev, dtype=torch.float64).pow(-case["zipf"])
    c = torch.cumsum(w, 0)
    u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64) * c[-1]
    rank = torch.searchsorted(c, u).clamp_(max=V - 1)
    ids = torch.randperm(V, generator=gen, device=dev)
    return ids[rank].to(torch.int32).view(case["B"], case["T"])


def _codes(w):
    """E4M3 codes of the rows of w and their fp32 scales."""
    s = w.abs().amax(1) / E4M3_MAX
    return (w / s[:, None]).to(torch.float8_e4m3fn), s


def _tensors(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    t = {}
    op = case["op"]

    def randn(*shape, sd=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * sd).to(dtype)

    if op in ("embed", "embed_grad"):
        dt = DT[case["dtype"]]
        t["tok"] = _tokens(case, gen, dev)
        n = case["B"] * case["T"]
        if op == "embed":
            t["E"] = randn(case["V"], case["d"], sd=0.02, dtype=dt)
        else:
            t["d_h"] = randn(n, case["d"], sd=0.01, dtype=dt)
        return t
    n, d = case["n"], case["d"]
    if op == "norm":
        dt = DT[case["dtype"]]
        # a residual stream: a wide-spread h and the smaller update of a layer
        t["x"] = randn(n, d, sd=0.3, dtype=dt)
        t["res"] = randn(n, d, sd=1.5, dtype=dt)
        t["gain"] = 1.0 + 0.1 * torch.randn(d, generator=gen, device=dev)
        return t
    if op == "norm_grad":
        dt = DT[case["dtype"]]
        t["sum"] = randn(n, d, sd=1.5, dtype=dt)
        t["rstd"] = torch.rsqrt(t["sum"].float().pow(2).mean(1) + EPS)
        t["d_y"] = randn(n, d, sd=0.01, dtype=dt)
        t["d_sum"] = randn(n, d, sd=0.01, dtype=dt)
        t["gain"] = 1.0 + 0.1 * torch.randn(d, generator=gen, device=dev)
        return t
    f = case["f"]
    if case.get("fp8"):
        x = torch.randn(n, d, generator=gen, device=dev)
        t["x"], t["x_scale"] = _codes(x)
        w = torch.randn(2 * f, d, generator=gen, device=dev) / math.sqrt(d)
        t["Wgu"], t["gu_scale"] = _codes(w)
    else:
        t["x"] = randn(n, d)
        t["Wgu"] = randn(2 * f, d, sd=1.0 / math.sqrt(d))
    t["Wd"] = randn(d, f, sd=1.0 / math.sqrt(f))
    if case.get("res"):
        t["res"] = randn(n, d, sd=1.5)
    if op == "ffn_train":
        t["d_y"] = randn(n, d, sd=0.01)
    return t


def _engine(case):
    """The module's context: hidden width, vocabulary and dtype of the case."""
    import hashed_gram_embedding_02_b200 as eb
    dtype = eb.ENGRAM_FP8 if case.get("fp8") else eb.ENGRAM_F32 if case.get("dtype") == "f32" else eb.ENGRAM_BF16
    V = case.get("V", 1024)
    cfg = eb.make_config(orders=(2,), heads=1, rows=[10007], mult=[[1, 3, 0, 0]], row_dim=128, hidden=case["d"],
                         conv_width=4, vocab=V, canon_vocab=V, dtype=dtype, eps=EPS)
    return eb.Engram(cfg)


def prepare(case, seed):
    st = _State(case)
    st.__dict__.update(_tensors(case, seed))
    if own:
        st.eng = _engine(case)
    return st


# ---------------------------------------------------------------- one pass

def _act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, kind):
    if kind == "silu":
        s = torch.sigmoid(g)
        return s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _deq(q, s):
    return q.float() * s[:, None]


def _run_plain(st):
    c = st.case
    op = c["op"]
    if op == "embed":
        return {"h": (st.E[st.tok.reshape(-1).long()].float() * c["scale"]).to(st.E.dtype)}
    if op == "embed_grad":
        # 64-bit sums: a hot token has thousands of rows
        d_E = torch.zeros(c["V"], c["d"], device=st.tok.device, dtype=torch.float64)
        d_E.index_add_(0, st.tok.reshape(-1), st.d_h.double())
        return {"d_E": (d_E * c["scale"]).float()}
    if op == "norm":
        s = st.x.float() + st.res.float()
        r = torch.rsqrt(s.pow(2).mean(1, keepdim=True) + EPS)
        y = s * r * st.gain
        out = {"sum": s.to(st.x.dtype)}
        if c["y"]:
            out["y"] = y.to(st.x.dtype)
        if c["q"]:
            sc = y.abs().amax(1) / E4M3_MAX
            out["q"] = (y / sc[:, None]).to(torch.float8_e4m3fn)
            out["scale"] = sc
        return out
    if op == "norm_grad":
        xh = st.sum.float() * st.rstd[:, None]
        dy = st.d_y.float()
        t = dy * st.gain
        d_x = st.d_sum.float() + st.rstd[:, None] * (t - xh * (t * xh).mean(1, keepdim=True))
        return {"d_x": d_x.to(st.d_y.dtype), "d_gain": (dy * xh).sum(0)}
    f = c["f"]
    x = _deq(st.x, st.x_scale) if c.get("fp8") else st.x.float()
    W = _deq(st.Wgu, st.gu_scale) if c.get("fp8") else st.Wgu.float()
    Wd = st.Wd.float()
    g, u = x @ W[:f].t(), x @ W[f:].t()
    a = _act(g, c["act"]) * u
    y = a @ Wd.t()
    if op == "ffn":
        if c["res"]:
            y = y + st.res.float()
        return {"y": y.to(torch.bfloat16)}
    dy = st.d_y.float()
    d_Wd = dy.t() @ a
    da = dy @ Wd
    dgu = torch.cat([da * u * _act_grad(g, c["act"]), da * _act(g, c["act"])], 1)
    bf = torch.bfloat16
    return {"y": y.to(bf), "d_x": (dgu @ W).to(bf), "d_Wgu": (dgu.t() @ x).to(bf), "d_Wd": d_Wd.to(bf)}


def _run_own(st):
    c, eng = st.case, st.eng
    op = c["op"]
    if op == "embed":
        return {"h": eng.embed(st.tok, st.E, scale=c["scale"])}
    if op == "embed_grad":
        return {"d_E": eng.embed_grad(st.tok, st.d_h, scale=c["scale"])}
    if op == "norm":
        o = eng.add_norm(st.x, st.res, gain=st.gain, y=c["y"], q=c["q"])
        out = {"sum": o.sum}
        if c["y"]:
            out["y"] = o.y
        if c["q"]:
            out["q"] = o.q
            out["scale"] = o.q_scale
        return out
    if op == "norm_grad":
        d_x, d_gain = eng.add_norm_grad(st.d_y, st.sum, st.rstd, gain=st.gain, d_sum=st.d_sum)
        return {"d_x": d_x, "d_gain": d_gain}
    if op == "ffn":
        q = {"x_scale": st.x_scale, "gu_scale": st.gu_scale} if c["fp8"] else {}
        return {"y": eng.ffn(st.x, st.Wgu, st.Wd, act=c["act"], res=st.res if c["res"] else None, **q)}
    y, gu = eng.ffn(st.x, st.Wgu, st.Wd, act=c["act"], save=True)
    d_x, d_Wgu, d_Wd = eng.ffn_grad(st.d_y, st.x, gu, st.Wgu, st.Wd, act=c["act"])
    return {"y": y, "d_x": d_x, "d_Wgu": d_Wgu, "d_Wd": d_Wd}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_act(g, kind):
    """act(g) and its derivative, by the derivative of the product z * P(z)."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p + g * p * (1.0 - p)
    k = math.sqrt(8.0 / math.pi)       # tanh(z) = 2 sigma(2 z) - 1
    p = 1.0 / (1.0 + torch.exp(-k * (g + 0.044715 * g ** 3)))
    return g * p, p + g * p * (1.0 - p) * k * (1.0 + 0.134145 * g ** 2)


def exact(case, seed):
    t = _tensors(case, seed)
    D = {k: v.double() for k, v in t.items() if k != "tok" and k not in ("E", "d_h")}
    op = case["op"]
    if op == "embed":
        return {"h": torch.index_select(t["E"], 0, t["tok"].flatten()).double() * case["scale"]}
    if op == "embed_grad":
        # tokens in sorted order: each token's sum is a difference of running sums
        tok, order = torch.sort(t["tok"].flatten(), stable=True)
        rows, counts = torch.unique_consecutive(tok, return_counts=True)
        ends = torch.cumsum(counts, 0)
        d_E = torch.zeros(case["V"], case["d"], dtype=torch.float64, device="cuda")
        for lo in range(0, case["d"], 256):
            s = torch.cumsum(t["d_h"][:, lo:lo + 256][order].double(), 0)
            s = torch.cat((s.new_zeros(1, s.shape[1]), s))
            d_E[rows.long(), lo:lo + 256] = (s[ends] - s[ends - counts]) * case["scale"]
        return {"d_E": d_E}
    if op == "norm":
        s = D["x"] + D["res"]
        y = s / torch.sqrt((s * s).sum(1, keepdim=True) / case["d"] + EPS) * D["gain"]
        out = {"sum": s}
        if case["y"]:
            out["y"] = y
        if case["q"]:
            c = y.abs().max(1).values / E4M3_MAX
            out["q"] = (y / c.unsqueeze(1)).to(torch.float8_e4m3fn).double()
            out["scale"] = c
        return out
    if op == "norm_grad":
        r = D["rstd"].unsqueeze(1)
        t1 = D["d_y"] * D["gain"]
        dot = (t1 * D["sum"]).sum(1, keepdim=True) / case["d"]
        return {"d_x": D["d_sum"] + r * t1 - r ** 3 * D["sum"] * dot,
                "d_gain": torch.einsum("nd,nd,n->d", D["d_y"], D["sum"], D["rstd"])}
    n, d, f = case["n"], case["d"], case["f"]
    x, W, Wd = D["x"], D["Wgu"], D["Wd"]
    if case.get("fp8"):
        x = x * D["x_scale"].unsqueeze(1)
        W = W * D["gu_scale"].unsqueeze(1)
    train = op == "ffn_train"
    y = torch.empty(n, d, dtype=torch.float64, device="cuda")
    d_x = torch.empty_like(y) if train else None
    d_W = torch.zeros_like(W) if train else None
    d_Wd = torch.zeros_like(Wd) if train else None
    for lo in range(0, n, 4096):
        hi = min(n, lo + 4096)
        gu = torch.mm(x[lo:hi], W.t())
        g, u = gu.split(f, 1)
        p, dp = _exact_act(g, case["act"])
        torch.mm(p * u, Wd.t(), out=y[lo:hi])
        if train:
            dy = D["d_y"][lo:hi]
            d_Wd.addmm_(dy.t(), p * u)
            da = torch.mm(dy, Wd)
            dgu = torch.cat((da * u * dp, da * p), 1)
            d_W.addmm_(dgu.t(), x[lo:hi])
            torch.mm(dgu, W, out=d_x[lo:hi])
    if case.get("res"):
        y += D["res"]
    return {"y": y, "d_x": d_x, "d_Wgu": d_W, "d_Wd": d_Wd} if train else {"y": y}
