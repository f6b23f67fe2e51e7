"""Inputs for the paged-cache tests: pools in shuffled pages, ragged sequences, packed rows with strides."""

import numpy as np
import torch

import long_context_tsa_b200 as T
from oracle import paged_oracle as PO

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DEV = "cuda"


def host64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def strided(rows, heads, D, dtype, layout, fill=0.0):
    """[rows, heads, D] of one of three layouts: contiguous, heads first, or with gaps between heads and tokens."""
    dt = TORCH[dtype]
    if layout == "heads":
        return torch.full((heads, rows, D), fill, dtype=dt, device=DEV).transpose(0, 1)
    if layout == "gaps":
        return torch.full((rows, heads + 1, D + 16), fill, dtype=dt, device=DEV)[:, :heads, :D]
    return torch.full((rows, heads, D), fill, dtype=dt, device=DEV)


class Layer:
    """A cache of sequences of the given (length, new tokens), filled with random rows."""

    def __init__(self, lens, Hkv=2, G=4, D=128, dtype="bf16", cache=None, page=16, layout="tokens", pad=0, seed=0, scale=0.0,
                 spare=2, first=0, scale_spread=1.0):
        self.lens, self.Hkv, self.Hq, self.D, self.dtype, self.page, self.layout = lens, Hkv, Hkv * G, D, dtype, page, layout
        self.kind = cache or dtype
        self.quantised = self.kind in PO.QMAX
        g = torch.Generator().manual_seed(seed)
        self.g = g
        need = [-(-n // page) for n, _ in lens]
        self.n_pages = sum(need) + spare
        self.width = max(max(need), 1) + 1
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32)  # entries that must not be read
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        starts = [first]
        for _, n in lens:
            starts.append(starts[-1] + n)
        self.starts, self.rows = starts, max(starts[-1] + pad, 1)
        self.scale = scale
        shape = (self.n_pages, Hkv, page, D)
        self.k_scales = self.v_scales = None
        pools = []
        for kv in range(2):
            x = torch.randn(shape, generator=g)
            if self.quantised:
                x = x * torch.exp(scale_spread * torch.randn(shape[:3] + (1,), generator=g))
                codes, sc = PO.quantise(x.numpy(), self.kind)
                codes = torch.from_numpy(codes)
                pools.append((codes.view(TORCH[self.kind]).to(DEV), torch.from_numpy(sc).to(DEV)))
            else:
                pools.append((x.to(TORCH[self.kind]).to(DEV), None))
        (self.k_pages, self.k_scales), (self.v_pages, self.v_scales) = pools
        self.seq_len = torch.tensor([n for n, _ in lens], dtype=torch.int32, device=DEV)
        self.token_start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.table_dev = self.table.to(DEV)
        self.finish()

    def finish(self):
        self.desc = T.make_paged_desc(self.rows, len(self.lens), self.Hq, self.Hkv, self.D, TORCH[self.dtype], TORCH[self.kind], self.page,
                                      self.n_pages, self.width, max(max(n for _, n in self.lens), 1), self.scale)
        self.cache = T.PagedCache(self.k_pages, self.v_pages, self.table_dev, self.seq_len, self.token_start, self.k_scales, self.v_scales)
        self.ws = T.alloc_paged_workspace(self.desc)

    def packed(self, heads, random=True, fill=0.0):
        t = strided(self.rows, heads, self.D, self.dtype, self.layout, fill)
        if random:
            t.copy_(torch.randn((self.rows, heads, self.D), generator=self.g).to(TORCH[self.dtype]))
        return t

    def values(self, which):
        """[n_pages, Hkv, page, D] in fp64: what the pool stands for."""
        pages, scales = (self.k_pages, self.k_scales) if which == "k" else (self.v_pages, self.v_scales)
        if not self.quantised:
            return host64(pages)
        codes = pages.view(torch.uint8).cpu().numpy() if self.kind == "e4m3" else pages.cpu().numpy()
        with np.errstate(all="ignore"):
            return PO.code_value(codes, self.kind) * scales.cpu().numpy().astype(np.float64)[..., None]

    def oracle(self, q, bounds=None):
        """fp64 result; rows of no sequence hold NaN."""
        out = np.full((self.rows, self.Hq, self.D), np.nan)
        return PO.attend(host64(q), self.values("k"), self.values("v"), self.table.numpy(), [n for n, _ in self.lens], self.starts,
                         self.scale if self.scale > 0 else self.D ** -0.5, out, bounds)

    def check(self, got, q, rows=None):
        """got against the fp64 result.  The bound, with u = 2^-8 for bf16 and 2^-24 for f32:
        u |out|    the result's rounding
        bf16:      u A for the probabilities' rounding (8-bit pools: with the value row's scale in them; codes are exact)
                   8-bit pools of single tokens and short runs: the product of probability and scale is an f16 number
                   whose subnormals round by at most 2^-25 of the unit.  The unit is at least 2^-6 / 2 times the
                   largest scale so far, the sum of the probabilities at least 1 (the largest is, against its
                   reference), so n keys are off by at most n 2^-25 2^-5 max |v| together: n 2^-30 max |v|
        (n + D + 64) 2^-23 (A + |out|) + (D + 8) 2^-23 B   fp32 sums over n keys and D products, exponentials
        (twice the unit roundoff for every operation: tensor cores truncate)."""
        bd = {}
        want = self.oracle(q, bd)
        A, B, W = bd["A"], bd["B"], np.abs(want)
        bf16 = self.dtype == "bf16"
        u = 2.0 ** -8 if bf16 else 2.0 ** -24
        n = max(n for n, _ in self.lens)
        tol = u * W + (n + self.D + 64) * 2.0 ** -23 * (A + W) + (self.D + 8) * 2.0 ** -23 * B
        if bf16:
            tol = tol + u * A
            if self.quantised:
                tol = tol + n * 2.0 ** -30 * np.nanmax(np.abs(self.values("v")))
        sel = np.zeros(self.rows, bool)
        sel[self.starts[0]:self.starts[-1]] = True
        if rows is not None:
            sel &= np.isin(np.arange(self.rows), rows)
        g = host64(got)
        assert np.isfinite(g[sel]).all()
        err = np.abs(g - want)[sel]
        worst = (err / (tol[sel] + 1e-30)).max() if err.size else 0.0
        assert worst <= 1.0, f"worst error {worst:.2f} of the bound, max abs {err.max():.3e}"
