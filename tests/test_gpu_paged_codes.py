"""Every byte that an 8-bit cache can hold, at every distance from the new tokens and through every kernel."""

import numpy as np
import pytest
import torch

import long_context_tsa_b200 as T
from oracle import paged_oracle as PO

from .paged_util import DEV, Layer, host64

pytestmark = pytest.mark.gpu


class Codes(Layer):
    """A layer whose pools hold any byte; e4m3's NaN codes stand for +-480 as include/tsa.h says."""

    def values(self, which):
        pages, scales = (self.k_pages, self.k_scales) if which == "k" else (self.v_pages, self.v_scales)
        codes = pages.view(torch.uint8).cpu().numpy()
        if self.kind == "int8":
            v = codes.view(np.int8).astype(np.float64)
        else:
            v = np.where((codes & 127) == 127, np.where(codes & 128, -480.0, 480.0), np.nan_to_num(PO.e4m3_value(codes)))
        return v * scales.cpu().numpy().astype(np.float64)[..., None]


def fill(c, pages, scales, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(0, 256, pages.shape, dtype=torch.uint8, generator=g)
    x.view(-1)[:512] = torch.arange(512).to(torch.uint8)  # every one of them, whatever the draw
    pages.view(torch.uint8).copy_(x)
    scales.copy_((0.5 + torch.rand(scales.shape, generator=g)) / 256)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("lens", [[(700, 1), (40, 1)], [(700, 7), (130, 3)], [(600, 200)], [(900, 120), (300, 2)], [(64, 64)]])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 1), (64, 16)])
def test_every_code_counts_as_its_value(dtype, kind, lens, D, G):
    c = Codes(lens, Hkv=2, G=G, D=D, dtype=dtype, cache=kind, page=16, seed=D + G)
    fill(c, c.k_pages, c.k_scales, 1)
    fill(c, c.v_pages, c.v_scales, 2)
    q = c.packed(c.Hq)
    out = c.packed(c.Hq, random=False)
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    assert T.tsa_check_status(c.ws) == 0
    c.check(out, q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("code,value", [(0x7F, 480.0), (0xFF, -480.0)])
@pytest.mark.parametrize("n,most", [(1, 1), (1, 200), (5, 5), (100, 100)])
def test_a_nan_code_of_e4m3_is_480_wherever_it_stands(dtype, code, value, n, most):
    # One value element is the code in every row: the average over the keys, whatever their weights, is the code's value.
    c = Layer([(900, n)], Hkv=1, G=4, D=128, dtype=dtype, cache="e4m3", page=64)
    c.desc.max_new = most
    c.ws = T.alloc_paged_workspace(c.desc)
    c.v_pages.view(torch.uint8)[..., 3] = code
    c.v_scales.fill_(0.5)
    q = c.packed(4)
    out = c.packed(4, random=False)
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    got = out[..., 3].float()
    # The probabilities are rounded for the product (bf16: at most 2^-8 each) and the result once more; f32: sums of 900.
    assert (got - value / 2).abs().max() <= 240 * (2.0 ** -7 if dtype == "bf16" else 1000 * 2.0 ** -23)
    back = [torch.empty(n, 1, 128, dtype=q.dtype, device=DEV) for _ in range(2)]
    T.tsa_cache_read(c.desc, c.cache, *back, c.ws)
    assert T.tsa_check_status(c.ws) == 0 and (back[1][..., 3] == value / 2).all()
    assert np.isfinite(host64(out)).all()
