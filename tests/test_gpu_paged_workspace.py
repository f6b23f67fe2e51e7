"""One workspace for the paged-cache calls and the sparse path's, in turn on one stream."""

import pytest
import torch

import long_context_tsa_b200 as T

from .paged_util import DEV, Layer

pytestmark = pytest.mark.gpu

LENS = {"decode": [(3000, 1), (77, 1), (1500, 1)], "runs": [(3000, 5), (900, 8)], "mixed": [(2000, 90), (700, 1), (64, 3)], "one": [(5000, 1)]}


def sparse_layer(dtype, L, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(1, 8, L, 128, generator=g).to(dtype).to(DEV)
    k, v = (torch.randn(1, 2, L, 128, generator=g).to(dtype).to(DEV) for _ in range(2))
    return q, k, v


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("bf16", "int8"), ("bf16", "e4m3"), ("f32", None), ("f32", "int8")])
@pytest.mark.parametrize("lens", sorted(LENS))
def test_paged_and_sparse_calls_share_a_workspace(dtype, cache, lens):
    c = Layer(LENS[lens], Hkv=2, G=4, D=128, dtype=dtype, cache=cache, page=32)
    paged_q = c.packed(8)
    want = c.packed(8, random=False)
    T.tsa_attend_paged(c.desc, c.cache, paged_q, want, c.ws)
    q, k, v = sparse_layer(c.k_pages.dtype if cache is None else paged_q.dtype, 1024, 3)
    desc = T.desc_for(q, k)
    alone = torch.empty_like(q)
    T.tsa_forward(desc, q, k, v, 32, [300, 511], alone, T.alloc_workspace(desc, 32))
    ws = torch.zeros(max(T.tsa_paged_workspace_size(c.desc), T.tsa_workspace_size(desc, 32)), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)  # scratch holds anything
    T.tsa_workspace_init(ws)
    for _ in range(3):
        sparse, out = torch.empty_like(q), c.packed(8, random=False, fill=7.0)
        T.tsa_forward(desc, q, k, v, 32, [300, 511], sparse, ws)
        T.tsa_attend_paged(c.desc, c.cache, paged_q, out, ws)
        assert T.tsa_check_status(ws) == 0
        assert torch.equal(sparse, alone) and torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_calls_of_several_shapes_share_a_workspace(dtype):
    cs = [Layer(LENS[n], Hkv=2, G=4, D=D, dtype=dtype, cache=cache, page=32, seed=i)
          for i, (n, D, cache) in enumerate([("decode", 128, "int8"), ("mixed", 64, None), ("one", 128, "e4m3"), ("runs", 64, None)])]
    qs = [c.packed(8) for c in cs]
    want = []
    for c, q in zip(cs, qs):
        want.append(c.packed(8, random=False))
        T.tsa_attend_paged(c.desc, c.cache, q, want[-1], c.ws)
    ws = torch.full((max(c.ws.numel() for c in cs),), 0xFF, dtype=torch.uint8, device=DEV)
    T.tsa_workspace_init(ws)
    for _ in range(3):
        for c, q, w in zip(cs, qs, want):
            out = c.packed(8, random=False, fill=7.0)
            T.tsa_attend_paged(c.desc, c.cache, q, out, ws)
            assert T.tsa_check_status(ws) == 0 and torch.equal(out, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_captured_graphs_and_the_sparse_path_share_a_workspace(dtype):
    cs = [Layer(LENS[n], Hkv=2, G=4, D=128, dtype=dtype, cache=cache, page=32, seed=i) for i, (n, cache) in enumerate([("decode", "e4m3"), ("mixed", None)])]
    qs, outs = [c.packed(8) for c in cs], [c.packed(8, random=False) for c in cs]
    q, k, v = sparse_layer(qs[0].dtype, 1024, 3)
    desc = T.desc_for(q, k)
    ws = torch.zeros(max([c.ws.numel() for c in cs] + [T.tsa_workspace_size(desc, 32)]), dtype=torch.uint8, device=DEV)
    graphs = []
    for c, x, o in zip(cs, qs, outs):
        T.tsa_attend_paged(c.desc, c.cache, x, o, ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            T.tsa_attend_paged(c.desc, c.cache, x, o, ws)
    want = [o.clone() for o in outs]
    sparse = torch.empty_like(q)
    for order in [(0, 1), (1, 0), (0, 0), (1, 1)]:
        for i in order:
            outs[i].fill_(7.0)
            T.tsa_forward(desc, q, k, v, 32, [300, 511], sparse, ws)
            graphs[i].replay()
            assert T.tsa_check_status(ws) == 0 and torch.equal(outs[i], want[i])
