"""Value scales of an 8-bit cache that lie many powers of two apart: what counts is probability times scale, whatever
the scales of keys that hardly count."""

import math

import numpy as np
import pytest
import torch

import long_context_tsa_b200 as T
from oracle import paged_oracle as PO

from .paged_util import Layer, host64

pytestmark = pytest.mark.gpu

M = {"int8": 127.0, "e4m3": 448.0}


def places(c, s, n):
    pos = np.arange(n)
    return torch.from_numpy(c.table[s, pos // c.page].numpy()).long(), torch.from_numpy(pos % c.page)


def prepare(kind, lens, G, D, logits, log2_scales, dtype="bf16", most=None):
    """Sequences whose logits (natural units, apart from small noise) and value scales at position j are given functions
    of j and the length: element 0 of every query is 1, of the key its logit, and the softmax scale is 1."""
    c = Layer(lens, Hkv=1, G=G, D=D, dtype=dtype, cache=kind, page=32, scale=1.0, seed=D + G)
    if most:
        c.desc.max_new = most
        c.ws = T.alloc_paged_workspace(c.desc)
    for s, (n, _) in enumerate(lens):
        page, slot = places(c, s, n)
        x = np.random.default_rng(s).standard_normal((n, D)) * 0.02
        x[:, 0] = logits(np.arange(n), n)
        codes, sc = PO.quantise(x.astype(np.float32), kind)
        c.k_pages.view(torch.uint8)[page, 0, slot] = torch.from_numpy(codes.view(np.uint8)).to(c.k_pages.device)
        c.k_scales[page, 0, slot] = torch.from_numpy(sc).to(c.k_pages.device)
        c.v_scales[page, 0, slot] = torch.from_numpy((2.0 ** log2_scales(np.arange(n), n) / M[kind]).astype(np.float32)).to(c.k_pages.device)
    q = c.packed(G)
    q *= 0.5
    q[..., 0] = 1.0
    return c, q


def check(c, q):
    """Against 64 bits with a bound of every element's own terms (those of Layer.check, but for the f16 one):
    2^-8 (|out| + A)     the result's rounding and the probabilities' (bf16; f16's is smaller)
    n 2^-32 W            f16 numbers of probability times scale that are subnormal: each is off by at most 2^-25 of the
                         unit, in which the row's largest such product so far is at least 2^7; W is that product of the
                         whole row times the largest code
    and fp32 sums."""
    out = c.packed(c.Hq, random=False)
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    assert T.tsa_check_status(c.ws) == 0
    bd = {}
    want = c.oracle(q, bd)
    A, B, W = bd["A"], bd["B"], np.abs(want)
    u = 2.0 ** -8 if c.dtype == "bf16" else 2.0 ** -24
    n = max(n for n, _ in c.lens)
    tol = u * (W + A) + (n + c.D + 64) * 2.0 ** -23 * (A + W) + (c.D + 8) * 2.0 ** -23 * B
    k, vs, q64 = c.values("k"), c.v_scales.cpu().numpy().astype(np.float64) * M[c.kind], host64(q)
    for s, (length, _) in enumerate(c.lens):
        page, slot = places(c, s, length)
        a, b = c.starts[s], c.starts[s + 1]
        sees = np.arange(length)[None] <= (length - (b - a) + np.arange(b - a))[:, None]
        for h in range(c.Hq):
            z = np.where(sees, q64[a:b, h] @ k[page, 0, slot].T, -np.inf)
            p = np.exp(z - z.max(1, keepdims=True))
            top = (p / p.sum(1, keepdims=True) * vs[page, 0, slot]).max(1, keepdims=True)
            tol[a:b, h] += n * 2.0 ** -32 * top
    err = np.abs(host64(out) - want)
    assert np.isfinite(host64(out)).all()
    assert (err <= tol).all(), f"worst error {(err / tol).max():.3g} of the bound"


SHAPES = [([(900, 1), (300, 1)], None), ([(900, 5), (2000, 3)], None), ([(900, 1), (400, 3)], 200), ([(700, 90)], None)]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,most", SHAPES)
@pytest.mark.parametrize("D,G", [(128, 4), (64, 2)])
@pytest.mark.parametrize("ratio", [10, 16, 24, 32, 40, 90])
@pytest.mark.parametrize("where", [3, 200])
def test_one_key_with_a_large_scale_and_a_small_probability(kind, lens, most, D, G, ratio, where):
    # It adds about 2^-12 of the result; all that the others hold has to be there.
    c, q = prepare(kind, lens, G, D, lambda j, n: np.where(j == where, -(ratio + 12) * math.log(2.0), 0.0),
                   lambda j, n: np.where(j == where, float(ratio), 0.0), most=most)
    check(c, q)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,most", SHAPES)
@pytest.mark.parametrize("D,G", [(128, 4), (64, 2)])
@pytest.mark.parametrize("span", [-110, -30, 30, 110])
def test_scales_that_fall_as_probabilities_grow(kind, lens, most, D, G, span):
    # Every key counts about the same: probability times scale is level over the sequence, each of them spans 2^|span|.
    c, q = prepare(kind, lens, G, D, lambda j, n: span * math.log(2.0) * j / n, lambda j, n: -span * j / n + min(span, 0), most=most)
    check(c, q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,most", SHAPES)
@pytest.mark.parametrize("base,spread", [(0, 20), (-90, 4), (-60, 40), (60, 20)])
def test_scales_of_any_size(dtype, kind, lens, most, base, spread):
    g = np.random.default_rng(1)
    c, q = prepare(kind, lens, 4, 64, lambda j, n: 10 * g.standard_normal(n), lambda j, n: base + spread * g.uniform(-1, 1, n), dtype, most)
    check(c, q)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [1, 5, 90])
def test_hidden_scales_and_zero_scales_do_not_matter(kind, n):
    # The new tokens' own scales, which the earlier of them must not notice, 2^80 above the rest; rows of scale 0 before.
    c, q = prepare(kind, [(400, n)], 4, 64, lambda j, L: 0.0 * j, lambda j, L: np.where(j < 100, -2000.0, 0.0))
    assert (c.v_scales == 0).any()
    check(c, q)
    page, slot = places(c, 0, 400)
    clean = c.packed(4, random=False)
    T.tsa_attend_paged(c.desc, c.cache, q, clean, c.ws)
    c.v_scales[page[-1], 0, slot[-1]] = 2.0 ** 80
    out = c.packed(4, random=False)
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    assert torch.equal(out[:n - 1], clean[:n - 1]) and not torch.equal(out[n - 1:], clean[n - 1:])
    check(c, q)
