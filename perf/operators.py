"""Cases over the paged key/value cache: appending to it, reading it back and attending over it.

The cache of one layer is a pool of pages.  ``k_pages`` and ``v_pages`` are
``[n_pages, Hkv, page_size, D]`` in the layer's type, or in 8 bits (``int8`` or
``float8_e4m3fn``) with one float32 scale for each token and head in
``k_scales`` / ``v_scales`` ``[n_pages, Hkv, page_size]``.  Row ``s`` of
``page_table`` lists the pages of sequence ``s``, ``seq_len[s]`` is its length
with the new tokens, and its new tokens are the rows ``token_start[s]`` to
``token_start[s + 1]`` of the packed activations: the last ones of the
sequence.

Three operators, each reached through the package's own calls:

append  ``tsa_cache_write`` then ``tsa_cache_read`` of the same tokens: the
        values that the cache now stands for.
read    ``tsa_cache_read`` of whole sequences (what the score and the selected
        attention of a prompt work on).
attend  ``tsa_attend_paged``: the new tokens' attention over everything that
        the cache holds up to their own positions.
"""

import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "int8": 1, "e4m3": 1}
QMAX = {"int8": 127.0, "e4m3": 448.0}


def listed():
    layer = {"Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16"}  # the benchmark's attention layer
    return [
        # One decoding step of 64 conversations: a token each, where the launch counts.
        {"name": "append-64x1-int8", "op": "append", "seqs": 64, "len": 8192, "new": 1, "ragged": True, "pad": 0, "cache": "int8", "page": 16, "heads_first": False, **layer},
        # A prompt of the 8K workload written at once, from the layer's [heads, tokens, D] layout.
        {"name": "append-8192-e4m3", "op": "append", "seqs": 1, "len": 8192, "new": 8192, "ragged": False, "pad": 0, "cache": "e4m3", "page": 64, "heads_first": True, **layer},
        # The 128K workload's keys and values.
        {"name": "append-131072-int8", "op": "append", "seqs": 1, "len": 131072, "new": 131072, "ragged": False, "pad": 0, "cache": "int8", "page": 128, "heads_first": False, **layer},
        # Reading a shared prefix back in 32 bits, three sequences of odd lengths.
        {"name": "read-3x32767-int8-f32", "op": "read", "seqs": 3, "len": 32767, "new": 0, "ragged": True, "pad": 5, "cache": "int8", "page": 32, "heads_first": False, **layer, "dtype": "f32"},
        # The whole 128K prompt, as the score and the selected attention read it.
        {"name": "read-131072-e4m3", "op": "read", "seqs": 1, "len": 131072, "new": 0, "ragged": False, "pad": 0, "cache": "e4m3", "page": 64, "heads_first": True, **layer},
        # One conversation's next token at a short length: latency.
        {"name": "decode-1x511-bf16", "op": "attend", "seqs": 1, "len": 511, "new": 1, "ragged": False, "pad": 0, "cache": "bf16", "page": 16, "heads_first": False, **layer},
        # A step of a batch of conversations of any length, padded to a captured batch size.
        {"name": "decode-64x8192-bf16", "op": "attend", "seqs": 61, "len": 8192, "new": 1, "ragged": True, "pad": 3, "cache": "bf16", "page": 64, "heads_first": False, **layer},
        # The next tokens of four 128K contexts.
        {"name": "decode-4x131072-int8", "op": "attend", "seqs": 4, "len": 131072, "new": 1, "ragged": False, "pad": 0, "cache": "int8", "page": 128, "heads_first": False, **layer},
        # Checking up to eight proposed tokens a conversation.
        {"name": "verify-16x8-e4m3", "op": "attend", "seqs": 16, "len": 32768, "new": 8, "ragged": True, "pad": 2, "cache": "e4m3", "page": 32, "heads_first": False, **layer},
        # The 8K workload's prompt without a prefix (every layer that keeps all tokens).
        {"name": "chunk-8192-bf16", "op": "attend", "seqs": 1, "len": 8192, "new": 8192, "ragged": False, "pad": 0, "cache": "bf16", "page": 64, "heads_first": True, **layer},
        # The last chunk of a 128K prompt over what is cached, an odd number of tokens.
        {"name": "chunk-1023-131071-int8", "op": "attend", "seqs": 1, "len": 131071, "new": 1023, "ragged": False, "pad": 1, "cache": "int8", "page": 128, "heads_first": False, **layer},
        # The tiny fp32 reference layer, as a batch of ragged prompts.
        {"name": "chunk-5x256-f32", "op": "attend", "seqs": 5, "len": 256, "new": 256, "ragged": True, "pad": 0, "cache": "f32", "page": 16, "heads_first": False, "Hq": 4, "Hkv": 4, "D": 64, "dtype": "f32"},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))

    while True:
        op = rng.choice(["append", "append", "read", "attend", "attend", "attend"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        c = {"op": op, "seqs": spread(1, 96), "len": spread(1, 131072), "new": 0, "ragged": rng.random() < 0.7, "pad": rng.choice([0, 0, 1, 7]),
             "cache": rng.choice([dtype, "int8", "e4m3"]), "page": rng.choice([16, 32, 64, 128, 256]), "heads_first": rng.random() < 0.3,
             "Hkv": rng.choice([1, 2, 4, 8]), "D": rng.choice([64, 128, 128]), "dtype": dtype}
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 8, 16] if c["Hkv"] < 8 else [1, 2, 4])
        if op == "append":
            c["new"] = spread(1, c["len"])
        if op == "attend":
            c["new"] = rng.choice([1, spread(1, min(c["len"], 32)), spread(1, min(c["len"], 8192))])
        tokens = c["seqs"] * (c["new"] if op == "append" else c["len"]) * c["Hkv"] * c["D"]
        if tokens > 131072 * 8 * 128 or c["seqs"] * c["len"] * c["Hkv"] * c["D"] > 4 * 131072 * 8 * 128:
            continue
        if op == "attend":
            pairs = c["seqs"] * c["Hq"] * c["new"] * c["len"]
            if pairs > (1 << 32 if dtype == "bf16" else 1 << 30):
                continue
        return c


def lengths(case):
    """(length, new tokens) of every sequence: a function of the case alone."""
    r = random.Random("%d %d %d" % (case["seqs"], case["len"], case["new"]))
    got = []
    for s in range(case["seqs"]):
        whole = s == 0 or not case["ragged"]
        n = case["len"] if whole else max(1, round(case["len"] ** r.random()) if r.random() < 0.3 else r.randint(1, case["len"]))
        new = n if case["op"] == "read" else min(n, case["new"] if whole else r.randint(1, case["new"]))
        got.append((n, new))
    return got


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 13)
    lens = lengths(case)
    S, H, D, ps = case["seqs"], case["Hkv"], case["D"], case["page"]
    dt, ct = DTYPES[case["dtype"]], DTYPES[case["cache"]]
    need = [(n + ps - 1) // ps for n, _ in lens]
    pages, width = sum(need) + 3, max(need) + 1
    # The pages of a running server: in no order, and some of them free.
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([sum(need[:s]) for s in range(S)], device=dev)
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col[None, :]).clamp_max(pages - 1)
    table = torch.where(col[None, :] < torch.tensor(need, device=dev)[:, None], order[at], torch.zeros_like(order[at])).contiguous()
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    used, rows = starts[-1], starts[-1] + case["pad"]
    gain = 1.0 + 3.0 * (torch.rand(2, H, 1, D, generator=g, device=dev) > 0.97)  # a few channels are larger, as in trained layers

    def acts(heads, fill):
        shape = (heads, rows, D) if case["heads_first"] else (rows, heads, D)
        x = torch.randn(shape, generator=g, device=dev) if fill else torch.zeros(shape, device=dev)
        x = x.to(dt)
        return x.transpose(0, 1) if case["heads_first"] else x

    def pool(kv):
        if case["op"] == "append":
            codes = torch.zeros(pages, H, ps, D, device=dev).to(ct)
            return codes, torch.zeros(pages, H, ps, device=dev)
        codes = torch.empty(pages, H, ps, D, dtype=ct, device=dev)
        scales = torch.zeros(pages, H, ps, device=dev)
        for lo in range(0, pages, 2048):
            x = torch.randn(min(2048, pages - lo), H, ps, D, generator=g, device=dev) * gain[kv]
            if case["cache"] in QMAX:
                a = x.abs().amax(-1) / QMAX[case["cache"]]
                x = x / a[..., None]
                x = x.round() if case["cache"] == "int8" else x.clamp(-448, 448)
                scales[lo:lo + 2048] = a
            codes[lo:lo + 2048] = x.to(ct)
        return codes, scales

    st = {"case": case, "used": used, "page_table": table,
          "seq_len": torch.tensor([n for n, _ in lens], dtype=torch.int32, device=dev),
          "token_start": torch.tensor(starts, dtype=torch.int32, device=dev)}
    st["k_pages"], st["k_scales"] = pool(0)
    st["v_pages"], st["v_scales"] = pool(1)
    if case["cache"] not in QMAX:
        st["k_scales"] = st["v_scales"] = None
    if case["op"] == "attend":
        st["q"], st["out"] = acts(case["Hq"], True), acts(case["Hq"], False)
    else:
        if case["op"] == "append":
            st["k"] = (acts(H, True) * gain[0, :, 0]).to(dt)
            st["v"] = (acts(H, True) * gain[1, :, 0]).to(dt)
        st["k_out"], st["v_out"] = acts(H, False), acts(H, False)
    if own:  # what a serving program makes once: the shape, the cache's handle and the workspace
        import long_context_tsa_b200 as T

        st["desc"] = T.make_paged_desc(n_tokens=rows, n_seqs=S, Hq=case["Hq"], Hkv=H, D=D, dtype=dt, cache_dtype=ct, page_size=ps, n_pages=pages,
                                       max_pages=width, max_new=max(n for _, n in lens))
        st["cache"] = T.PagedCache(st["k_pages"], st["v_pages"], st["page_table"], st["seq_len"], st["token_start"], st["k_scales"], st["v_scales"])
        st["ws"] = T.alloc_paged_workspace(st["desc"])
    return st


def run(state):
    if own:
        return _own(state)
    return _attend(state) if state["case"]["op"] == "attend" else _append(state)


def _own(st):
    import long_context_tsa_b200 as T

    if st["case"]["op"] == "attend":
        T.tsa_attend_paged(st["desc"], st["cache"], st["q"], st["out"], st["ws"])
        return st["out"]
    if st["case"]["op"] == "append":
        T.tsa_cache_write(st["desc"], st["cache"], st["k"], st["v"], st["ws"])
    T.tsa_cache_read(st["desc"], st["cache"], st["k_out"], st["v_out"], st["ws"])
    return {"k": st["k_out"], "v": st["v_out"]}


# ------------------------------------------------------------------ the plain forms


def _places(st):
    """Sequence, index among its new tokens, page and slot of every packed token that belongs to one."""
    t = torch.arange(st["used"], device="cuda")
    start, ps = st["token_start"].long(), st["case"]["page"]
    s = torch.searchsorted(start[1:], t, right=True)
    i = t - start[s]
    pos = st["seq_len"].long()[s] - (start[s + 1] - start[s]) + i
    return s, i, st["page_table"][s, pos // ps].long(), pos % ps


def _codes(x, kind):
    """The 8-bit values of rows x: x * qmax / max|x| rounded to the nearest, ties to even, and the row's scale max|x| / qmax."""
    a = x.abs().amax(-1, keepdim=True).float()
    t = x.double() * QMAX[kind] / torch.where(a > 0, a, torch.ones_like(a)).double()  # 64 bits: values next to a rounding border
    if kind == "e4m3":
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
        t = torch.round(t / step) * step
    else:
        t = torch.round(t)
    return t.float().to(DTYPES[kind]), (a / QMAX[kind])[..., 0]


def _append(st):
    case = st["case"]
    s, i, page, slot = _places(st)
    if case["op"] == "append":
        for x, pages, scales in ((st["k"], st["k_pages"], st["k_scales"]), (st["v"], st["v_pages"], st["v_scales"])):
            x = x[:st["used"]]
            if case["cache"] in QMAX:
                x, a = _codes(x, case["cache"])
                scales[page, :, slot] = a
            if case["cache"] == "e4m3":
                x, pages = x.view(torch.uint8), pages.view(torch.uint8)
            pages[page, :, slot] = x
    for pages, scales, out in ((st["k_pages"], st["k_scales"], st["k_out"]), (st["v_pages"], st["v_scales"], st["v_out"])):
        out[:st["used"]] = _values(pages, scales, page, slot).to(out.dtype)
    return {"k": st["k_out"], "v": st["v_out"]}


def _values(pages, scales, page, slot):
    """float32 values [..., Hkv, D] of the cache at these places."""
    raw = pages.view(torch.uint8)[page, :, slot].view(pages.dtype) if pages.dtype == torch.float8_e4m3fn else pages[page, :, slot]
    x = raw.float()
    return x if scales is None else x * scales[page, :, slot][..., None]


def _attend(st):
    case, ps = st["case"], st["case"]["page"]
    S, H, D, L = case["seqs"], case["Hkv"], case["D"], case["len"]
    G = case["Hq"] // H
    start, total = st["token_start"].long(), st["seq_len"].long()
    n = start[1:] - start[:-1]
    N = min(case["new"], L)
    pos = torch.arange(L, device="cuda")
    there = pos[None, :] < total[:, None]
    page = torch.where(there, st["page_table"][:, pos // ps].long(), 0)
    slot = (pos % ps)[None, :].expand(S, L)
    k = _values(st["k_pages"], st["k_scales"], page, slot).permute(0, 2, 3, 1)  # [S, H, D, L]
    v = (_values(st["v_pages"], st["v_scales"], page, slot) * there[..., None, None]).permute(0, 2, 1, 3)
    i = torch.arange(N, device="cuda")
    q = st["q"][(start[:-1, None] + i).clamp_max(st["used"] - 1)].float()  # [S, N, Hq, D]
    q = q.reshape(S, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, N * G, D)
    x = torch.matmul(q, k).mul_(D ** -0.5)
    sees = pos[None, None, :] <= (total - n)[:, None, None] + i[None, :, None]  # [S, N, L]
    sees = sees[:, None, :, None, :].expand(S, 1, N, G, L).reshape(S, 1, N * G, L)
    x = x.masked_fill_(~sees, float("-inf"))
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    y = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    y = y.reshape(S, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(S, N, H * G, D)
    s, j, _, _ = _places(st)
    st["out"][:st["used"]] = y[s, j].to(st["out"].dtype)
    return st["out"]


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    lens = lengths(case)
    used, row = sum(n for _, n in lens), case["Hkv"] * case["D"]
    held = BYTES[case["cache"]] * row + (4 * case["Hkv"] if case["cache"] in QMAX else 0)  # bytes of one cached token's K or V
    if case["op"] == "attend":
        pairs = sum(new * n - new * (new - 1) // 2 for n, new in lens)
        return {"bytes": 2 * used * case["Hq"] * case["D"] * BYTES[case["dtype"]] + 2 * held * sum(n for n, _ in lens), "flops": 4 * case["Hq"] * case["D"] * pairs}
    moved = 2 * used * (held + row * BYTES[case["dtype"]])
    return {"bytes": moved * (2 if case["op"] == "append" else 1), "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    H, D, ps = case["Hkv"], case["D"], case["page"]
    G = case["Hq"] // H
    out = {}

    def held(name, s, n):
        """[Hkv, n, D]: sequence s's cached values, page by page."""
        pages = st["page_table"][s, :(n + ps - 1) // ps].long()
        raw = st[name + "_pages"]
        x = (raw.view(torch.uint8)[pages].view(raw.dtype) if case["cache"] == "e4m3" else raw[pages]).double()
        if case["cache"] in QMAX:
            x = x * st[name + "_scales"][pages].double().unsqueeze(-1)
        return x.transpose(0, 1).reshape(H, -1, D)[:, :n]

    at = 0
    if case["op"] != "attend":
        for name in ("k", "v"):
            y = torch.zeros(st["used"] + case["pad"], H, D, dtype=torch.float64, device="cuda")
            if case["op"] == "append":
                x = st[name][:st["used"]].double()
                if case["cache"] in QMAX:
                    top = x.abs().amax(-1, keepdim=True)
                    u = (x.abs() * QMAX[case["cache"]]) / top
                    if case["cache"] == "e4m3":
                        ulp = torch.ldexp(torch.ones_like(u), (torch.frexp(u).exponent - 4).clamp_min(-9))
                    else:
                        ulp = torch.ones_like(u)
                    low = torch.floor(u / ulp)
                    rest = u / ulp - low
                    up = (rest > 0.5) | ((rest == 0.5) & (low % 2 == 1))
                    x = torch.sign(x) * (low + up.double()) * ulp * top / QMAX[case["cache"]]
                y[:st["used"]] = x
            else:
                at = 0
                for s, (n, _) in enumerate(lengths(case)):
                    y[at:at + n] = held(name, s, n).transpose(0, 1)
                    at += n
            out[name] = y
        return out
    y = torch.zeros(st["used"] + case["pad"], H * G, D, dtype=torch.float64, device="cuda")
    for s, (n, new) in enumerate(lengths(case)):
        k, v = held("k", s, n), held("v", s, n)
        for lo in range(0, new, 256):
            m = min(256, new - lo)
            q = st["q"][at + lo:at + lo + m].double().reshape(m, H, G, D)
            late = torch.arange(n, device="cuda")[None, :] > (n - new + lo + torch.arange(m, device="cuda"))[:, None]
            for h in range(H):
                z = (q[:, h].reshape(m * G, D) @ k[h].T / D ** 0.5).reshape(m, G, n).masked_fill_(late[:, None, :], float("-inf"))
                y[at + lo:at + lo + m, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v[h]
        at += new
    return y
