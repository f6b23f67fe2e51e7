"""tsa_attend_paged against the fp64 oracle, within bounds from the arithmetic (paged_util.Layer.check)."""

import numpy as np
import pytest
import torch

import long_context_tsa_b200 as T
from oracle import paged_oracle as PO

from .paged_util import DEV, TORCH, Layer, host64

pytestmark = pytest.mark.gpu

LENS = {
    "one": [(1, 1)],
    "decode": [(1, 1), (15, 1), (16, 1), (17, 1), (128, 1), (129, 1), (300, 1), (1500, 1)],
    "verify": [(40, 8), (9, 3), (7, 7), (333, 5), (128, 2), (1025, 8), (12, 0)],
    "prompt": [(200, 200), (1, 1), (127, 127), (128, 128), (129, 129), (31, 31)],
    "chunks": [(513, 130), (64, 1), (900, 77), (31, 0), (700, 256), (260, 257), (40, 4)],
}
CACHES = [("bf16", None), ("bf16", "int8"), ("bf16", "e4m3"), ("f32", None), ("f32", "int8"), ("f32", "e4m3")]


def attend(c, q, fill=7.0):
    out = c.packed(c.Hq, random=False, fill=fill)
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    assert T.tsa_check_status(c.ws) == 0
    return out


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("D,Hkv,G,page,layout", [(128, 2, 4, 16, "tokens"), (64, 1, 16, 32, "heads"), (128, 4, 1, 64, "gaps"),
                                                 (64, 2, 2, 128, "tokens"), (128, 1, 8, 256, "heads")])
def test_matches_oracle(dtype, cache, lens, D, Hkv, G, page, layout):
    c = Layer(LENS[lens], Hkv=Hkv, G=G, D=D, dtype=dtype, cache=cache, page=page, layout=layout, pad=2, first=1, seed=D + page)
    q = c.packed(c.Hq)
    out = attend(c, q)
    c.check(out, q)
    assert (out[c.starts[-1]:] == 7.0).all() and (out[:1] == 7.0).all()  # rows of no sequence


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("n", [1, 3, 100])
def test_long_cache_and_large_logits(dtype, cache, n):
    # Logits of a spread that moves the running maximum often; keys of growing size at the end.
    c = Layer([(5000, n)], Hkv=1, G=4, D=128, dtype=dtype, cache=cache, page=64, seed=3, scale=0.4)
    q = c.packed(4)
    c.check(attend(c, q), q)


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("n", [1, 5, 140])
def test_hidden_rows_may_hold_anything(dtype, cache, n):
    # Behind the length: NaN and infinities in pages and scales.  Among the new tokens: value rows that are not
    # finite, seen by the later tokens only; keys that would give a NaN logit to the earlier ones.
    lens = [(150, n), (141, min(n, 141)), (300, 1)]
    c = Layer(lens, Hkv=2, G=2, D=64, dtype=dtype, cache=cache, page=32, seed=4)
    for s, (length, _) in enumerate(lens):
        pg, slot = int(c.table[s, (length - 1) // 32]), (length - 1) % 32
        for t in (c.k_pages, c.v_pages):
            if c.quantised:
                t.view(torch.uint8)[pg, :, slot + 1:] = 0x7F  # NaN in e4m3, 127 in int8
            else:
                t[pg, :, slot + 1:] = float("inf")
                t[pg, :, slot + 1:, ::3] = float("nan")
        if c.quantised:
            for t in (c.k_scales, c.v_scales):
                t[pg, :, slot + 1:] = float("nan")
    q = c.packed(c.Hq)
    clean = attend(c, q)
    c.check(clean, q)
    if n < 5:
        return
    hit = c.starts[0] + n - 3  # sequence 0: the third from the end has an infinite value, the last a NaN key
    for back, pages, scales, x in ((3, c.v_pages, c.v_scales, float("inf")), (1, c.k_pages, c.k_scales, float("nan"))):
        pos = lens[0][0] - back
        pg, slot = int(c.table[0, pos // 32]), pos % 32
        if c.quantised:
            scales[pg, :, slot] = x
        else:
            pages[pg, :, slot, 5] = x
    out = attend(c, q)
    assert torch.equal(out[:hit], clean[:hit]) and torch.equal(out[n:], clean[n:])
    seen = out[hit:n - 1].float()
    assert not torch.isfinite(seen[..., 5]).any()
    if not c.quantised:
        assert torch.isinf(seen[..., 5]).all() and (seen[..., 5] > 0).all()
        other = [d for d in range(64) if d != 5]
        assert torch.equal(out[hit:n - 1][..., other], clean[hit:n - 1][..., other])
    assert torch.isnan(out[n - 1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,at", [(3, 0), (6, 2), (8, 7), (100, 0), (140, 131), (300, 257)])
def test_an_infinite_value_among_the_first_keys(dtype, n, at):
    c = Layer([(n, n)], Hkv=1, G=4, D=64, dtype=dtype, page=16, seed=n)
    q = c.packed(4)
    want = attend(c, q)
    c.v_pages[int(c.table[0, at // 16]), 0, at % 16, 9] = -float("inf")
    got = attend(c, q)
    want[at:, :, 9] = -float("inf")
    assert torch.equal(got, want)


@pytest.mark.parametrize("cache", [None, "int8"])
@pytest.mark.parametrize("n", [1, 100])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(cache, n):
    c = Layer([(3000, n)] * 3, Hkv=2, G=4, D=128, cache=cache, page=64)
    q = c.packed(8)
    out = c.packed(8, random=False)
    T.tsa_debug_set_wait_limit(1)
    try:
        for _ in range(3):
            T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
            assert T.tsa_check_status(c.ws) in (0, 5)  # a single poll may also find the copy landed
    finally:
        T.tsa_debug_set_wait_limit(0)
    c.check(attend(c, q), q)


@pytest.mark.parametrize("dtype,cache", CACHES)
def test_length_below_new_tokens_gives_zeros_to_rows_without_keys(dtype, cache):
    c = Layer([(60, 40), (33, 1)], Hkv=2, G=2, D=64, dtype=dtype, cache=cache, page=16)
    q = c.packed(c.Hq)
    want = attend(c, q)
    c.seq_len[0] = 10
    out = c.packed(c.Hq, random=False, fill=7.0)
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    assert T.tsa_check_status(c.ws) == 6
    assert (out[:30] == 0).all() and torch.isfinite(out[:40]).all() and torch.equal(out[40:], want[40:])


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("bf16", "int8"), ("f32", "e4m3")])
def test_equal_calls_give_equal_bits_and_do_not_depend_on_max_new_or_the_workspace(dtype, cache):
    c = Layer([(3000, 1), (77, 1), (1500, 6)], Hkv=2, G=4, D=128, dtype=dtype, cache=cache, page=64)
    q = c.packed(c.Hq)
    first = attend(c, q)
    c.ws[2048:].fill_(0xFF)  # only what tsa_workspace_init zeroes has to be zero
    for _ in range(3):
        assert torch.equal(attend(c, q), first)
    c.desc.max_new = 400
    c.ws = T.alloc_paged_workspace(c.desc)
    c.check(attend(c, q), q)


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("news", [(40, 40), (40, 1), (12, 30)])
def test_captured_chunks_equal_eager_ones(dtype, cache, news):
    c = Layer([(500, news[0]), (333, news[1]), (70, 0)], Hkv=2, G=4, D=128, dtype=dtype, cache=cache, page=32, pad=1)
    q, k, v = c.packed(8), c.packed(2), c.packed(2)
    out = c.packed(8, random=False, fill=7.0)
    T.tsa_cache_write(c.desc, c.cache, k, v, c.ws)
    T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.tsa_cache_write(c.desc, c.cache, k, v, c.ws)
        T.tsa_attend_paged(c.desc, c.cache, q, out, c.ws)
    for _ in range(3):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=c.g).to(t.dtype))
        out.fill_(7.0)
        graph.replay()
        assert T.tsa_check_status(c.ws) == 0
        c.check(out, q)
        got = out.clone()
        assert torch.equal(attend(c, q), got)


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("bf16", "e4m3"), ("f32", None)])
@pytest.mark.parametrize("n", [1, 60])
def test_shared_pages_broadcast_queries_and_sizes_off_the_powers_of_two(dtype, cache, n):
    # Three KV heads, pages of 1024; two sequences whose first pages are the same and one that repeats a page;
    # the same query for every head and for every token.
    c = Layer([(2500, n), (2200, n), (1100, n)], Hkv=3, G=2, D=64, dtype=dtype, cache=cache, page=1024, seed=8)
    c.table[1, :2] = c.table[0, :2]
    c.table[2, 1] = c.table[2, 0]
    c.table_dev.copy_(c.table)
    one = c.packed(1)
    q = one.expand(c.rows, 6, 64)
    c.check(attend(c, q), q)
    q = one[:1].expand(c.rows, 6, 64)
    assert q.stride(0) == 0 and q.stride(1) == 0
    c.check(attend(c, q), q)


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("total,n", [(700, 130), (700, 1), (129, 129), (193, 100), (65, 40)])
def test_a_maximum_that_grows_with_every_step(dtype, cache, total, n):
    # Each key tile's largest logit passes the one before by more than the reference tolerates, to the last step.
    c = Layer([(total, total)], Hkv=1, G=4, D=64, dtype=dtype, cache=cache, page=32, scale=1.0, seed=7)
    k, v = c.packed(1), c.packed(1)
    k[..., 0] = (torch.arange(total, device=DEV) * 0.035).to(k.dtype)[:, None]
    T.tsa_cache_write(c.desc, c.cache, k, v, c.ws)
    c.lens, c.starts, c.rows = [(total, n)], [0, n], n
    c.token_start.copy_(torch.tensor(c.starts))
    c.finish()
    q = c.packed(4) * 0.25
    q[..., 0] = 4.0
    c.check(attend(c, q), q)


@pytest.mark.parametrize("dtype,cache", CACHES)
def test_more_new_tokens_than_max_new_says(dtype, cache):
    c = Layer([(300, 150), (40, 40)], Hkv=1, G=4, D=128, dtype=dtype, cache=cache, page=16)
    c.desc.max_new = 1
    c.ws = T.alloc_paged_workspace(c.desc)
    q = c.packed(4)
    c.check(attend(c, q), q)


@pytest.mark.parametrize("dtype,cache", CACHES)
def test_no_new_tokens_at_all(dtype, cache):
    for most in (1, 100):
        c = Layer([(5, 0), (9, 0)], Hkv=2, G=2, D=64, dtype=dtype, cache=cache, page=16, pad=2)
        c.desc.max_new = most
        c.ws = T.alloc_paged_workspace(c.desc)
        c.ws[2048:].fill_(0xFF)
        assert (attend(c, c.packed(4)) == 7.0).all()
        k = c.packed(2)
        before = c.k_pages.clone()
        T.tsa_cache_write(c.desc, c.cache, k, k, c.ws)
        out = c.packed(2, random=False, fill=7.0)
        T.tsa_cache_read(c.desc, c.cache, out, out, c.ws)
        assert T.tsa_check_status(c.ws) == 0 and (out == 7.0).all() and torch.equal(c.k_pages.view(torch.uint8), before.view(torch.uint8))


@pytest.mark.parametrize("cache", [None, "int8"])
def test_chunks_on_two_streams_at_once(cache):
    cs = [Layer([(3000 + 500 * i, 300), (700, 1)], Hkv=2, G=4, D=128, cache=cache, page=64, seed=i) for i in range(2)]
    qs = [c.packed(8) for c in cs]
    outs = [c.packed(8, random=False) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(20):
        for c, q, o, st in zip(cs, qs, outs, streams):
            T.tsa_attend_paged(c.desc, c.cache, q, o, c.ws, stream=st)
    torch.cuda.synchronize()
    for c, q, o in zip(cs, qs, outs):
        assert T.tsa_check_status(c.ws) == 0
        c.check(o, q)


@pytest.mark.parametrize("dtype,cache", CACHES)
def test_many_chunk_shapes_again_and_again(dtype, cache):
    # Segments of one to many steps, cut at every place: barriers' phases run through all their orders.
    g = np.random.default_rng(1)
    for trial in range(12):
        lens = []
        for _ in range(int(g.integers(1, 7))):
            n = int(g.integers(1, 1400))
            lens.append((n, int(g.integers(1, min(n, 400) + 1))))
        G = int(2 ** g.integers(0, 5))
        c = Layer(lens, Hkv=int(g.integers(1, 4)), G=G, D=int(g.choice([64, 128])), dtype=dtype, cache=cache,
                  page=int(2 ** g.integers(4, 9)), seed=trial)
        q = c.packed(c.Hq)
        out = attend(c, q)
        c.check(out, q)
        for _ in range(5):
            assert torch.equal(attend(c, q), out)


def test_captured_calls_follow_lengths_tables_and_new_rows():
    lens = [(100, 1), (40, 1), (260, 1)]
    c = Layer(lens, Hkv=2, G=4, D=128, cache="int8", page=16, spare=20)
    c.width += 2
    c.table = torch.cat([c.table, torch.full((3, 2), -1, dtype=torch.int32)], 1)
    c.table_dev = c.table.to(DEV)
    c.finish()
    k, v, q = c.packed(2), c.packed(2), c.packed(8)
    out = c.packed(8, random=False)
    args = (c.desc, c.cache)
    T.tsa_cache_write(*args, k, v, c.ws)
    T.tsa_attend_paged(*args, q, out, c.ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.tsa_cache_write(*args, k, v, c.ws)
        T.tsa_attend_paged(*args, q, out, c.ws)
    free = [p for p in range(c.n_pages) if p not in set(c.table[c.table >= 0].tolist())]
    for step in range(30):
        c.lens = [(n + 1, 1) for n, _ in c.lens]
        for s, (n, _) in enumerate(c.lens):
            if (n - 1) % 16 == 0:
                c.table[s, (n - 1) // 16] = free.pop()
        c.table_dev.copy_(c.table)
        c.seq_len += 1
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=c.g).to(t.dtype))
        graph.replay()
        if step % 7 == 0:
            assert T.tsa_check_status(c.ws) == 0
            c.check(out, q)


def test_two_streams_with_a_workspace_each():
    cs = [Layer([(2000 + 100 * i, 1), (500, 1)], Hkv=2, G=4, D=128, cache=None if i else "int8", page=64, seed=i) for i in range(2)]
    qs = [c.packed(8) for c in cs]
    outs = [c.packed(8, random=False) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(20):
        for c, q, o, st in zip(cs, qs, outs, streams):
            T.tsa_attend_paged(c.desc, c.cache, q, o, c.ws, stream=st)
    torch.cuda.synchronize()
    for c, q, o in zip(cs, qs, outs):
        assert T.tsa_check_status(c.ws) == 0
        c.check(o, q)


@pytest.mark.parametrize("cache,n", [(None, 1), (None, 200), ("int8", 1), ("int8", 200)])
def test_pools_of_more_than_4_gib(cache, n):
    # One pool of 2^32 + bytes of which only the last pages are used.
    esz = 1 if cache else 2
    pages = (1 << 32) // (8 * 64 * 128 * esz) + 40
    c = Layer([(1900, n)], Hkv=8, G=1, D=128, cache=cache, page=64, seed=6)
    used = c.n_pages
    big = {}
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        t = getattr(c, name)
        if t is not None:
            big[name] = torch.empty((pages,) + t.shape[1:], dtype=t.dtype, device=DEV)
            big[name][-used:] = t
    small, q = c, c.packed(8)
    want = attend(c, q)
    c.check(want, q)
    c.n_pages = pages
    c.table_dev = torch.where(c.table_dev >= 0, c.table_dev + pages - used, c.table_dev)
    for name, t in big.items():
        setattr(c, name, t)
    c.finish()
    assert torch.equal(attend(c, q), want)
    k, v = c.packed(8), c.packed(8)
    T.tsa_cache_write(c.desc, c.cache, k, v, c.ws)
    ko, vo = c.packed(8, random=False), c.packed(8, random=False)
    T.tsa_cache_read(c.desc, c.cache, ko, vo, c.ws)
    assert T.tsa_check_status(c.ws) == 0
    if cache is None:
        assert torch.equal(ko, k) and torch.equal(vo, v)
    else:
        codes, sc = PO.quantise(host64(k), cache)
        want_k = torch.from_numpy((codes.astype(np.float32) * sc[..., None])).to(TORCH["bf16"])
        assert torch.equal(ko.cpu(), want_k)


def test_many_sequences():
    g = np.random.default_rng(0)
    lens = [(int(g.integers(1, 60)), 1) for _ in range(1024)]
    c = Layer(lens, Hkv=1, G=2, D=64, page=16)
    q = c.packed(2)
    c.check(attend(c, q), q)


@pytest.mark.parametrize("dtype,cache", CACHES)
def test_a_prompt_in_chunks_then_tokens_then_the_sparse_layer(dtype, cache):
    """The calls as a server makes them: a prompt written and attended in chunks beside another sequence's single
    tokens, a few generated tokens, and the cached prefix read back for the sparse attention of this library."""
    Hkv, G, D, page, total = 2, 4, 64, 32, 300
    dt = TORCH[dtype]
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(2, total, Hkv, D, generator=g).to(dt) for _ in range(2))
    q = torch.randn(2, total, Hkv * G, D, generator=g).to(dt)
    c = Layer([(total, 1), (total, 1)], Hkv=Hkv, G=G, D=D, dtype=dtype, cache=cache, page=page)  # for its pools and tables
    lens = [0, 0]
    for new in [(130, 1), (1, 1), (0, 100), (100, 7), (1, 1), (1, 1)]:
        lens = [a + b for a, b in zip(lens, new)]
        starts = [0, new[0], new[0] + new[1]]
        c.lens, c.starts, c.rows = list(zip(lens, new)), starts, sum(new)
        c.seq_len.copy_(torch.tensor(lens))
        c.token_start.copy_(torch.tensor(starts))
        c.finish()
        part = lambda t: torch.cat([t[s, lens[s] - new[s]:lens[s]] for s in range(2)]).to(DEV)
        T.tsa_cache_write(c.desc, c.cache, part(k), part(v), c.ws)
        qq = part(q)
        out = torch.empty_like(qq)
        T.tsa_attend_paged(c.desc, c.cache, qq, out, c.ws)
        assert T.tsa_check_status(c.ws) == 0
        c.check(out, qq)
    # Sequence 0 back in the layout of the sparse path: [1, Hkv, L, D].
    L = lens[0]
    kb, vb = (torch.empty(1, Hkv, L, D, dtype=dt, device=DEV) for _ in range(2))
    rd = T.make_paged_desc(L, 1, Hkv * G, Hkv, D, dt, TORCH[c.kind], page, c.n_pages, c.width, L)
    rc = T.PagedCache(c.k_pages, c.v_pages, c.table_dev[:1], c.seq_len[:1], torch.tensor([0, L], dtype=torch.int32, device=DEV), c.k_scales, c.v_scales)
    T.tsa_cache_read(rd, rc, kb[0].transpose(0, 1), vb[0].transpose(0, 1), T.alloc_paged_workspace(rd))
    if not c.quantised:
        assert torch.equal(kb[0].cpu(), k[0, :L].transpose(0, 1)) and torch.equal(vb[0].cpu(), v[0, :L].transpose(0, 1))
    qb = q[0, :L].transpose(0, 1).contiguous()[None].to(DEV)
    desc = T.desc_for(qb, kb)
    ws = T.alloc_workspace(desc, 16)
    sparse = torch.empty_like(qb)
    T.tsa_forward(desc, qb, kb, vb, 16, [L] * Hkv, sparse, ws)  # every token kept: dense attention
    assert T.tsa_check_status(ws) == 0
    all_new = Layer([(L, L)], Hkv=Hkv, G=G, D=D, dtype=dtype, page=page)
    dense = torch.empty(L, Hkv * G, D, dtype=dt, device=DEV)
    T.tsa_cache_write(all_new.desc, all_new.cache, kb[0].transpose(0, 1), vb[0].transpose(0, 1), all_new.ws)
    T.tsa_attend_paged(all_new.desc, all_new.cache, qb[0].transpose(0, 1), dense, all_new.ws)
    all_new.check(dense, qb[0].transpose(0, 1))
    all_new.check(sparse[0].transpose(0, 1), qb[0].transpose(0, 1))
