"""tsa_cache_write and tsa_cache_read against the fp64 oracle: codes and scales bit for bit."""

import numpy as np
import pytest
import torch

import long_context_tsa_b200 as T
from long_context_tsa_b200 import _native as N
from oracle import paged_oracle as PO

from .paged_util import DEV, TORCH, Layer, host64

pytestmark = pytest.mark.gpu

LENS = [(70, 70), (33, 0), (129, 1), (16, 16), (40, 7), (1, 1)]


def hard_rows(rows, heads, D, dtype, seed):
    """Rows whose quotients lie on borders between codes and next to them, with extreme magnitudes and non-finite values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, heads, D, generator=g)
    for r in range(rows):
        k = r % 12
        if k == 0:    # int8 ties: a = 127, quotients k + 1/2
            x[r] = torch.randint(-126, 127, (heads, D), generator=g) + 0.5
            x[r, :, 0] = 127.0
        elif k == 1:  # the same at another magnitude
            x[r] = (torch.randint(-126, 127, (heads, D), generator=g) + 0.5) * 2.0 ** -100
            x[r, :, D - 1] = -127.0 * 2.0 ** -100
        elif k == 2:  # e4m3 ties: a = 448, odd multiples of half a step
            e = torch.randint(-8, 9, (heads, D), generator=g).float()
            x[r] = torch.exp2(e) * (1 + (2 * torch.randint(0, 8, (heads, D), generator=g) + 1) / 16)
            x[r, :, 3] = -448.0
            x[r].clamp_(-448, 448)
        elif k == 3:  # e4m3 subnormals
            x[r] = torch.randint(-40, 41, (heads, D), generator=g) * 2.0 ** -10
            x[r, :, 1] = 448.0
        elif k == 4:
            x[r] = 0.0
        elif k == 5:
            x[r] *= 1e38
            x[r].clamp_(-3e38, 3e38)
        elif k == 6:
            x[r] *= 1e-39
        elif k == 7:
            x[r, 0, 5], x[r, -1, 6] = float("nan"), float("inf")
        elif k == 8:
            x[r] = -0.0
            x[r, :, 7] = -float(np.float32(2.0 ** -149)) if dtype == "f32" else -2.0 ** -133
        elif k == 9:  # next to ties by one unit in the last place
            y = (torch.randint(-126, 127, (heads, D), generator=g) + 0.5)
            x[r] = torch.nextafter(y, torch.where(torch.rand(heads, D, generator=g) < 0.5, -1e9, 1e9))
            x[r, :, 0] = 127.0
        elif k == 10:  # an odd largest magnitude: x = border * a / M rounded, so quotients fall next to the border
            a = 1.0 + torch.rand(heads, 1, generator=g)
            x[r] = (torch.randint(-126, 127, (heads, D), generator=g) + 0.5) * a / 127
            x[r, :, 2] = a[:, 0]
    return x.to(TORCH[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["plain", "int8", "e4m3"])
@pytest.mark.parametrize("D,Hkv,page,layout", [(128, 2, 16, "tokens"), (64, 8, 64, "heads"), (128, 8, 32, "gaps"), (64, 1, 256, "tokens"),
                                               (128, 3, 1024, "heads")])
def test_write_then_read(dtype, kind, D, Hkv, page, layout):
    c = Layer(LENS, Hkv=Hkv, G=1, D=D, dtype=dtype, cache=None if kind == "plain" else kind, page=page, layout=layout, pad=3, first=2, seed=D + page)
    k, v = (c.packed(Hkv) for _ in range(2))
    k.copy_(hard_rows(c.rows, Hkv, D, dtype, 1))
    v.copy_(hard_rows(c.rows, Hkv, D, dtype, 2).flip(0))
    before = [t.clone() for t in (c.k_pages, c.v_pages)] + [t.clone() if c.quantised else None for t in (c.k_scales, c.v_scales)]
    T.tsa_cache_write(c.desc, c.cache, k, v, c.ws)
    assert T.tsa_check_status(c.ws) == 0
    raw = {2: torch.int16, 4: torch.int32, 1: torch.uint8}
    for x, pages, scales, pages0, scales0 in ((k, c.k_pages, c.k_scales, before[0], before[2]), (v, c.v_pages, c.v_scales, before[1], before[3])):
        want = pages0.view(raw[pages.element_size()]).cpu().numpy().copy()
        want_s = scales0.cpu().numpy().copy() if c.quantised else None
        if c.quantised:
            codes, sc = PO.quantise(host64(x), c.kind)
            codes = codes.view(np.uint8)
        else:
            codes = x.contiguous().view(raw[x.element_size()]).cpu().numpy()
        for t, _, _, pg, slot in PO.places(c.starts, [n for n, _ in LENS], c.table.numpy(), page):
            want[pg, :, slot] = codes[t]
            if c.quantised:
                want_s[pg, :, slot] = sc[t]
        got = pages.view(raw[pages.element_size()]).cpu().numpy()
        bad = np.argwhere(got != want)
        assert bad.size == 0, f"{len(bad)} codes differ, first at {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"
        if c.quantised:
            assert np.array_equal(scales.cpu().numpy(), want_s, equal_nan=True)
    # Read back: fp32 product, rounded to the type; rows of no sequence keep what they held.
    ko, vo = (c.packed(Hkv, random=False, fill=7.0) for _ in range(2))
    T.tsa_cache_read(c.desc, c.cache, ko, vo, c.ws)
    assert T.tsa_check_status(c.ws) == 0
    for x, got, name in ((k, ko, "k"), (v, vo, "v")):
        want = np.full((c.rows, Hkv, D), 7.0)
        val = c.values(name)
        for t, _, _, pg, slot in PO.places(c.starts, [n for n, _ in LENS], c.table.numpy(), page):
            want[t] = val[pg, :, slot]
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want.astype(np.float32)).to(TORCH[dtype]).float().numpy()
        assert np.array_equal(got.float().cpu().numpy(), want, equal_nan=True)
        if not c.quantised:
            assert torch.equal(got[2:c.starts[-1]].contiguous().view(raw[got.element_size()]), x[2:c.starts[-1]].contiguous().view(raw[x.element_size()]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_random_rows_of_many_magnitudes_code_exactly(dtype, kind):
    c = Layer([(4096, 4096)], Hkv=8, G=1, D=128, dtype=dtype, cache=kind, page=64)
    g = torch.Generator().manual_seed(5)
    x = [(torch.randn(4096, 8, 128, generator=g) * torch.exp(8 * torch.randn(4096, 8, 1, generator=g))).to(TORCH[dtype]) for _ in range(2)]
    T.tsa_cache_write(c.desc, c.cache, x[0].to(DEV), x[1].to(DEV), c.ws)
    for t, pages, scales in ((x[0], c.k_pages, c.k_scales), (x[1], c.v_pages, c.v_scales)):
        codes, sc = PO.quantise(host64(t), kind)
        order = c.table[0, :64].numpy()
        got = pages.view(torch.uint8).cpu().numpy()[order].transpose(0, 2, 1, 3).reshape(4096, 8, 128)
        assert np.array_equal(got, codes.view(np.uint8))
        assert np.array_equal(scales.cpu().numpy()[order].transpose(0, 2, 1).reshape(4096, 8), sc)


@pytest.mark.parametrize("what", ["page", "negative page", "length", "short length", "starts", "descending"])
def test_bad_tables_are_reported_and_touch_nothing(what):
    lens = [(40, 3), (50, 4), (20, 2)]
    c = Layer(lens, Hkv=2, G=1, D=64, dtype="bf16", cache="int8", page=16, pad=1)
    if what == "page":
        c.table_dev[1, 3] = c.n_pages
    elif what == "negative page":
        c.table_dev[1, 2:4] = -1
    elif what == "length":
        c.seq_len[1] = c.width * 16 + 4
    elif what == "short length":
        c.seq_len[1] = 0
    elif what == "starts":
        c.token_start[2] = c.rows + 5
    elif what == "descending":
        c.token_start[1:3] = torch.tensor([7, 3])
    bad = lambda: T.tsa_check_status(c.ws) == N.STATUS["TSA_ERR_DEVICE_BOUNDS"]
    k, v = c.packed(2), c.packed(2)
    before = [t.clone() for t in (c.k_pages, c.v_pages, c.k_scales, c.v_scales)]
    T.tsa_cache_write(c.desc, c.cache, k, v, c.ws)
    assert bad()
    ok_slots = torch.zeros(c.n_pages, 16, dtype=torch.bool)
    for _, s, _, pg, slot in PO.places(c.starts, [n for n, _ in lens], c.table.numpy(), 16):
        ok_slots[pg, slot] = True
    for t, t0 in zip((c.k_pages, c.v_pages, c.k_scales, c.v_scales), before):
        same = (t == t0) if t.dim() == 3 else (t == t0).all(-1)
        if what != "descending":  # there the tokens' places are not defined
            assert same.all(1).cpu()[~ok_slots].all()
    ko, vo = c.packed(2, random=False, fill=7.0), c.packed(2, random=False, fill=7.0)
    T.tsa_cache_read(c.desc, c.cache, ko, vo, c.ws)
    assert bad()
    q, out = c.packed(2), c.packed(2, random=False, fill=7.0)
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    assert bad()
    if what not in ("starts", "descending"):
        assert (out[9:] == 7.0).all() and (ko[9:] == 7.0).all()
    c.table_dev.copy_(c.table)
    c.seq_len.copy_(torch.tensor([n for n, _ in lens]))
    c.token_start.copy_(torch.tensor(c.starts))
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    assert T.tsa_check_status(c.ws) == 0
    c.check(out, q)
