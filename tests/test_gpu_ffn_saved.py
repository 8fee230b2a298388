"""What the feed-forward forward saves of g and u: 24 of their 32 bits, rounded.

A read value has the upper 16 bits of the fp32 value and 257 L below them, L the
saved byte: the nearest multiple of 257 to the lower 16 bits is off by 128 of
them at most, so a value is within 128 * 2^-23 = 2^-16 of itself (half a step).
The rows of x here hold one value each, so that g and u are products of two
bf16 numbers: 16 significant bits, exact in fp32 whatever the order of a sum."""

import numpy as np
import pytest

from test_gpu_ffn import planes
from test_gpu_residual import engine, f64, randn

torch = pytest.importorskip("torch")


def test_the_nearest_byte():
    """the rule the kernel rounds by, over all lower halves: off by 128 at most, in one byte; 0 stays 0 (zeros and
    infinities), 65535 stays so (the NaN that arithmetic gives); cutting off is off by up to 255"""
    low = np.arange(65536)
    L = (255 * low + 32895) >> 16
    assert L.min() == 0 and L.max() == 255 and L[0] == 0 and L[65535] == 255
    assert np.abs(257 * L - low).max() == 128
    assert np.abs(257 * (low >> 8) - low).max() == 255


@pytest.mark.gpu
@pytest.mark.parametrize("n,d,f", [(1, 1152, 1456), (5, 264, 136), (130, 136, 200), (300, 2560, 264), (700, 72, 520)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_saved_values_are_rounded(n, d, f, kind):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hashed_gram_embedding_02_b200 as eb
    eng = engine(eb, d)
    Wgu, Wd = randn(2, 2 * f, d), randn(3, d, f, sd=f ** -0.5)
    rng = np.random.default_rng(n)
    at = torch.from_numpy(rng.integers(0, d, n)).cuda()
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.arange(n, device="cuda")
    x[rows, at] = randn(4, n)
    if n >= 4:
        x[1] = 0
        x[2, at[2]], x[3, at[3]] = float("inf"), float("nan")
    _, saved = eng.ffn(x, Wgu, Wd, act=kind, save=True)
    assert eng.status() == (eb.ENGRAM_OK, 0)
    got = planes(saved, n, f)[0]
    want = f64(x[rows, at])[:, None] * f64(Wgu[:, at]).T
    got, finite = f64(got), np.isfinite(want)
    assert np.array_equal(got[~finite], want[~finite], equal_nan=True)
    err = np.abs(got[finite] - want[finite])
    bound = 2.0 ** -16 * np.abs(want[finite])
    assert (err <= bound).all(), (int((err > bound).sum()), float((err / np.maximum(bound, 1e-300)).max()))
