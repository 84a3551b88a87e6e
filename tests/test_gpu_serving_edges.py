"""Edges of the chunk attention over an fp8 cache, on the GPU, against the float64 definition: score
scales at the ends of what the call takes, small weights behind a large one, and each of its three
kernels (few rows, 128-row tiles, the CTA pair's) with the options that the bf16 tests cover."""

import pytest
import torch

import differential_attention_02_gb300 as da
import serving_reference as ref
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu
F8, BF = torch.float8_e4m3fn, torch.bfloat16

# New tokens and lengths of batches that go to the kernel for tiles of few rows, to it and the 128-row
# one in one call, to the 128-row one alone, and to the CTA pair's (d = 128).
KINDS = {"few": (64, [1, 5, 2], [65, 300, 700]), "both": (64, [1, 9, 2, 1], [65, 300, 700, 130]),
         "many": (64, [60, 1, 130], [60, 333, 500]), "wide": (128, [60, 1, 13], [60, 333, 500])}
kinds = pytest.mark.parametrize("kind", list(KINDS))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from differential_attention_02_gb300 import build
    build.build()
    da.load_library()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _case(kind, seed=0, group=2, **kw):
    d, n, lens = KINDS[kind]
    return Case(n, lens, 2 * group, group, d, True, seed=seed, **kw)


@pytest.mark.parametrize("k_scale", [1e-30, 1e-38, 1e-45])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -20, 1.0])
@kinds
def test_scores_that_vanish(kind, size, k_scale):
    """Rows of zeros, small rows and ordinary ones over K scales so small that every score is 0 to fp32:
    uniform weights over the visible keys (the masked ones stay out)."""
    c = _case(kind, seed=1)
    c.q = [(x.float() * size).to(BF) for x in c.q]
    c.scales = (k_scale, k_scale, ref.SCALES[2])
    c.check(c.run(), f"{kind} rows of {size}, K scale {k_scale}")


@kinds
def test_tiny_queries_and_a_large_scale(kind):
    """Query rows at the lower end of bf16's range against a K scale that brings their scores back to unit
    size: the rows' power of two has to cover the whole range."""
    c = _case(kind, seed=2)
    c.q = [(x.float() * 2.0 ** -122).to(BF) for x in c.q]
    g = torch.Generator().manual_seed(3)
    c.pools[:2] = [(torch.randn(p.shape, generator=g) * 16).to(F8) for p in c.pools[:2]]
    c.scales = (2.0 ** 118, 2.0 ** 118, ref.SCALES[2])
    c.check(c.run(), kind)
