"""What the residual-stream methods refuse before anything is launched, on the
host (CPU only): tensors of another dtype, shape or device, or with gaps, and
at the C entry points a null context."""

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def eb():
    import hashed_gram_embedding_02_b200 as eb
    return eb


@pytest.fixture()
def eng(eb):
    """An engine with no context behind it: a call whose tensors pass the checks
    reaches the library, which refuses the null context."""
    e = object.__new__(eb.Engram)
    e.cfg = eb.make_config(orders=(2,), heads=1, rows=[10007], mult=[[1, 3, 0, 0]], row_dim=8, hidden=16,
                           conv_width=4, vocab=50, canon_vocab=50, dtype=eb.ENGRAM_BF16)
    e.ctx = None
    e.device = torch.device("cpu")
    return e


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


TOK = torch.zeros(2, 5, dtype=torch.int32)


@pytest.mark.parametrize("call,why", [
    (lambda e: e.embed(TOK.long(), bf(50, 16)), "torch.int32"),
    (lambda e: e.embed(TOK[0], bf(50, 16)), "dimensions"),
    (lambda e: e.embed(TOK, bf(49, 16)), "shape"),
    (lambda e: e.embed(TOK, torch.zeros(50, 16)), "torch.bfloat16"),
    (lambda e: e.embed(TOK, bf(50, 32)[:, ::2]), "contiguous"),
    (lambda e: e.embed(TOK, bf(50, 16), t_begin=6), "t_begin"),
    (lambda e: e.embed(TOK.t(), bf(50, 16)), "adjacent"),
    (lambda e: e.embed(TOK[:1].expand(2, 5), bf(50, 16)), "overlap"),
    (lambda e: e.embed(TOK, bf(50, 16), out=bf(9, 16)), "out"),
    (lambda e: e.embed(torch.zeros(2, 5, dtype=torch.int32, device="meta"), bf(50, 16)), "meta"),
    (lambda e: e.embed_grad(TOK, bf(9, 16)), "d_h"),
    (lambda e: e.embed_grad(TOK, bf(10, 16), accumulate=True), "accumulate"),
    (lambda e: e.embed_grad(TOK, bf(10, 16), out=bf(50, 16)), "torch.float32"),
    (lambda e: e.add_norm(bf(3, 8)), "shape"),
    (lambda e: e.add_norm(bf(3, 16), bf(4, 16)), "res"),
    (lambda e: e.add_norm(bf(3, 16), gain=bf(16)), "gain"),
    (lambda e: e.add_norm_grad(bf(3, 16), bf(3, 16), torch.zeros(4)), "rstd"),
    (lambda e: e.add_norm_grad(bf(3, 16), bf(3, 16).t().contiguous().t(), torch.zeros(3)), "contiguous"),
    (lambda e: e.add_norm_grad(bf(3, 16), bf(3, 16), torch.zeros(3), d_sum=torch.zeros(3, 16)), "d_sum"),
    (lambda e: e.ffn(bf(3, 16), bf(16, 16), bf(16, 8), act="relu"), "act"),
    (lambda e: e.ffn(bf(3, 16), bf(8, 16), bf(16, 8)), "Wgu"),
    (lambda e: e.ffn(bf(3, 16), bf(16, 16), bf(8, 16)), "Wgu"),
    (lambda e: e.ffn(bf(3, 16), bf(16, 16), bf(16, 8), res=bf(3, 8)), "res"),
    (lambda e: e.ffn(bf(3, 16), bf(16, 16), bf(16, 8), x_scale=torch.ones(3)), "FP8"),
    (lambda e: e.ffn_grad(bf(3, 16), bf(3, 16), bf(3, 8), bf(16, 16), bf(16, 8)), "saved"),
    (lambda e: e.ffn_grad(bf(2, 16), bf(3, 16), bf(3, 16), bf(16, 16), bf(16, 8)), "d_y"),
])
def test_methods_refuse_bad_tensors(eng, call, why):
    with pytest.raises(ValueError, match=why):
        call(eng)


def test_entry_points_refuse_a_null_context(eb):
    from hashed_gram_embedding_02_b200 import binding
    lib, inval = binding._lib, binding.ENGRAM_E_INVAL
    assert lib.engram_embed(None, None, 1, 1, 1, 0, None, 1.0, None, None) == inval
    assert lib.engram_embed_grad(None, None, 1, 1, 1, 0, None, 1.0, None, 0, None, 0, None) == inval
    assert lib.engram_add_norm(None, None, None, 1, None, None, None, None, None, None, None) == inval
    assert lib.engram_add_norm_grad(None, None, None, None, None, 1, None, None, None, None, 0, None) == inval
    assert lib.engram_ffn(None, None, None, 1, 8, 0, None, None, None, None, None, None, None, 0, None) == inval
    assert lib.engram_ffn_grad(None, None, None, None, 1, 8, 0, None, None, None, None, None, None, 0, None) == inval
    assert eb.engram_ffn_workspace_bytes(None, 4, 8) == 0
    assert eb.engram_ffn_saved_bytes(None, 4, 8) == 0
    assert eb.engram_embed_grad_workspace_bytes(None, 4) == 0
    assert eb.engram_add_norm_grad_workspace_bytes(None, 4) == 0
