"""Paged-cache calls without a GPU: the oracle's own pins, the binding's checks and the C entry points' refusals."""

import ctypes

import numpy as np
import pytest
import torch

import long_context_tsa_b200 as T
from long_context_tsa_b200 import _native as N
from oracle import paged_oracle as PO

FAKE = 0x100000  # never dereferenced: every call below fails validation first


def test_e4m3_values_are_torchs():
    b = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(PO.e4m3_value(b), want, equal_nan=True)


def test_quantise_pins():
    # a = 127: the quotient is x itself; ties go to the even code.
    c, s = PO.quantise(np.array([127.0, 0.5, 1.5, -2.5, -0.0, 126.5, -126.5]), "int8")
    assert c.tolist() == [127, 0, 2, -2, 0, 126, -126] and s == np.float32(1.0)
    # a = 448: 17 lies between 16 and 18, 19 between 18 and 20; subnormal step 2^-9.
    c, s = PO.quantise(np.array([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11]), "e4m3")
    assert PO.e4m3_value(c).tolist() == [448.0, 16.0, 20.0, -16.0, 0.0, 2.0 ** -8, 0.0] and s == np.float32(1.0)
    c, s = PO.quantise(np.array([[0.0, -0.0], [np.inf, 1.0], [np.nan, 1.0]]), "int8")
    assert not c.any() and s[0] == 0 and np.isnan(s[1:]).all()


def test_attend_oracle_is_softmax_attention():
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(4, 2, 16, 8, generator=g, dtype=torch.float64) for _ in range(2))
    table = np.array([[2, 0, 3]])
    q = torch.randn(3, 4, 8, generator=g, dtype=torch.float64)
    got = PO.attend(q.numpy(), k.numpy(), v.numpy(), table, [37], [0, 3], 0.3, np.zeros((3, 4, 8)))
    kk = k[[2, 0, 3]].transpose(0, 1).reshape(2, 48, 8)[:, :37].repeat_interleave(2, 0)
    vv = v[[2, 0, 3]].transpose(0, 1).reshape(2, 48, 8)[:, :37].repeat_interleave(2, 0)
    mask = torch.arange(37)[None] <= torch.arange(34, 37)[:, None]
    want = torch.softmax((q.transpose(0, 1) @ kk.transpose(1, 2) * 0.3).masked_fill(~mask, float("-inf")), -1) @ vv
    assert np.allclose(got, want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)


def desc(**kw):
    d = dict(n_tokens=8, n_seqs=4, Hq=32, Hkv=8, D=128, dtype=N.TSA_BF16, cache_dtype=N.TSA_I8, page_size=64, n_pages=100,
             max_pages=16, max_new=2, scale=0.0)
    d.update(kw)
    return N.TsaPagedDesc(*[d[f] for f, _ in N.TsaPagedDesc._fields_])


def cache(**kw):
    d = {f: FAKE for f, _ in N.TsaPagedCache._fields_}
    d.update(kw)
    return N.TsaPagedCache(*[d[f] for f, _ in N.TsaPagedCache._fields_])


def call(name="tsa_attend_paged", d=None, c=None, a=None, b=None, ws=FAKE, ws_bytes=1 << 40):
    d = desc() if d is None else d
    heads = d.Hq if name == "tsa_attend_paged" else d.Hkv
    a = N.TsaRows(FAKE, heads * d.D, d.D) if a is None else a
    b = N.TsaRows(FAKE, heads * d.D, d.D) if b is None else b
    return getattr(N.lib(), name)(ctypes.byref(d), ctypes.byref(c or cache()), ctypes.byref(a), ctypes.byref(b), ws, ws_bytes, None)


CALLS = ["tsa_cache_write", "tsa_cache_read", "tsa_attend_paged"]
INV, UNS, WSP = (N.STATUS[f"TSA_ERR_{x}"] for x in ("INVALID_ARG", "UNSUPPORTED", "WORKSPACE"))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=0), INV), (dict(n_seqs=0), INV), (dict(Hq=30), INV), (dict(dtype=N.TSA_I8), INV), (dict(dtype=-1), INV),
    (dict(cache_dtype=N.TSA_F32), INV), (dict(cache_dtype=9), INV), (dict(scale=float("nan")), INV), (dict(max_new=0), INV),
    (dict(max_pages=0), INV), (dict(n_pages=0), INV), (dict(D=96), UNS), (dict(Hq=256), UNS), (dict(Hq=24), UNS),
    (dict(page_size=8), UNS), (dict(page_size=48), UNS), (dict(page_size=2048), UNS), (dict(n_seqs=1025), UNS), (dict(Hq=1025, Hkv=1025), UNS),
    (dict(n_tokens=1 << 26), UNS), (dict(n_pages=1 << 22), UNS), (dict(max_pages=1 << 25), UNS), (dict(n_pages=0x7fffffff), UNS),
])
def test_bad_shapes(name, kw, code):
    d = desc(**kw)
    assert call(name, d) == code
    assert N.lib().tsa_paged_workspace_size(ctypes.byref(d)) == 0


@pytest.mark.parametrize("name", CALLS)
def test_bad_pointers_scales_and_workspace(name):
    for f in ("k_pages", "v_pages", "k_scales", "v_scales"):
        assert call(name, c=cache(**{f: None})) == INV
        assert call(name, c=cache(**{f: FAKE + 8})) == INV
    for f in ("page_table", "seq_len", "token_start"):
        assert call(name, c=cache(**{f: None})) == INV
        assert call(name, c=cache(**{f: FAKE + 2})) == INV
    plain = desc(cache_dtype=N.TSA_BF16)
    assert call(name, plain) == INV  # scales without 8-bit pages
    assert call(name, plain, cache(k_scales=None, v_scales=None), ws=None) == INV
    need = N.lib().tsa_paged_workspace_size(ctypes.byref(desc()))
    assert need > 256 and call(name, ws_bytes=need - 1) == WSP
    assert call(name, ws=FAKE + 8) == INV
    assert getattr(N.lib(), name)(None, None, None, None, FAKE, 1 << 40, None) == INV
    d = desc()
    assert getattr(N.lib(), name)(ctypes.byref(d), ctypes.byref(cache()), None, None, FAKE, 1 << 40, None) == INV


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("ptr,ts,hs", [(FAKE + 8, 4096, 128), (None, 4096, 128), (FAKE, 4100, 128), (FAKE, 4096, 129),
                                       (FAKE, -4096, 128), (FAKE, 4096, -128), (FAKE, 1 << 38, 128), (FAKE, 4096, 1 << 39)])
def test_bad_rows(name, ptr, ts, hs):
    bad = N.TsaRows(ptr, ts, hs)
    assert call(name, a=bad, ws_bytes=0) == INV
    assert call(name, b=bad, ws_bytes=0) == INV


def test_overlapping_output_rows_are_refused_and_broadcast_inputs_are_not():
    for ts, hs in [(0, 128), (4096, 0), (64, 4096), (128, 128), (128, 512), (1024, 128)]:
        bad = N.TsaRows(FAKE, ts, hs)
        assert call("tsa_attend_paged", b=bad, ws_bytes=0) == INV
        assert call("tsa_attend_paged", a=bad, ws_bytes=0) == WSP  # an input: checked further
    for ts, hs in [(4096, 128), (128, 1024), (8192, 144)]:
        assert call("tsa_attend_paged", b=N.TsaRows(FAKE, ts, hs), ws_bytes=0) == WSP
    one = desc(n_tokens=1)
    assert call("tsa_attend_paged", one, b=N.TsaRows(FAKE, 3, 128), ws_bytes=0) == WSP  # one row: its stride is not used


def tensors(dtype=torch.int8):
    pages = [torch.zeros(6, 2, 16, 64, dtype=dtype) for _ in range(2)]
    ints = [torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)]
    scales = [torch.zeros(6, 2, 16) for _ in range(2)] if dtype == torch.int8 else [None, None]
    return pages + ints + scales


def test_cache_object_checks():
    T.PagedCache(*tensors())
    T.PagedCache(*tensors(torch.bfloat16))
    for i, bad in [(0, torch.zeros(6, 2, 16, 32, dtype=torch.int8)), (0, torch.zeros(6, 2, 16, 64)), (1, torch.zeros(6, 2, 16, 64, dtype=torch.float16)),
                   (2, torch.zeros(3, 4, dtype=torch.int64)), (2, torch.zeros(4, 3, dtype=torch.int32).t()), (3, torch.zeros(2, dtype=torch.int32)),
                   (4, torch.zeros(3, dtype=torch.int32)), (5, None), (6, torch.zeros(6, 2, 8)), (5, torch.zeros(6, 2, 16, dtype=torch.float64))]:
        t = tensors()
        t[i] = bad
        if i == 2 and bad.dtype == torch.int32:
            t[3], t[4] = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
        with pytest.raises(ValueError):
            T.PagedCache(*t)
    with pytest.raises(ValueError):
        T.PagedCache(*(tensors(torch.bfloat16)[:5] + [torch.zeros(6, 2, 16)] * 2))


def test_binding_refuses_shapes_types_and_host_tensors():
    d = T.make_paged_desc(5, 3, 4, 2, 64, torch.bfloat16, torch.int8, 16, 6, 4, 2)
    c = T.PagedCache(*tensors())
    ws = torch.zeros(T.tsa_paged_workspace_size(d), dtype=torch.uint8)
    kv, q = torch.zeros(5, 2, 64, dtype=torch.bfloat16), torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        T.tsa_cache_write(d, c, kv, kv, ws)
    for bad in (kv[:4], kv.float(), q, torch.zeros(5, 2, 128, dtype=torch.bfloat16)[..., ::2]):
        with pytest.raises(ValueError, match="packed rows"):
            T.tsa_cache_read(d, c, bad, kv, ws)
    with pytest.raises(ValueError, match="shape"):
        T.tsa_attend_paged(T.make_paged_desc(5, 3, 4, 2, 64, torch.bfloat16, torch.int8, 32, 6, 4, 2), c, q, q, ws)
    with pytest.raises(ValueError, match="workspace"):
        T.tsa_attend_paged(d, c, q, q, ws.float())
    with pytest.raises(T.TsaError):
        T.alloc_paged_workspace(T.make_paged_desc(5, 3, 4, 2, 96, torch.bfloat16, torch.int8, 16, 6, 4, 2), device="cpu")
    assert T.make_paged_desc(5, 3, 4, 2, 64, torch.float16, torch.int8, 16, 6, 4, 2).dtype == -1
