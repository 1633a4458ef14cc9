"""Shared by the paged-cache GPU tests: seeded caches mirrored into the fp64 oracle, and derived tolerances."""
from __future__ import annotations

import numpy as np
import torch

import oracle.paged_oracle as po
from compressed_draft_kv_gb300 import capi

DEV = torch.device("cuda:0")
E4M3 = torch.float8_e4m3fn


def np64(x):
    return x.detach().to("cpu").double().numpy()


class Cache:
    """A paged cache on the GPU and, on demand, the oracle's copy of it."""

    def __init__(self, kv_cap, hkv, d, page, dtype, seed=0, spare=2, gap=0, fill=True, first_page=0):
        """kv_cap: tokens each sequence's table covers; gap: unused pages between two pages of the same array."""
        g = torch.Generator().manual_seed(seed)
        per = [-(-max(1, x) // page) for x in kv_cap]
        n = sum(per) + spare + first_page
        self.page, self.hkv, self.d, self.e4 = page, hkv, d, dtype == "e4m3"
        perm = torch.randperm(n - first_page, generator=g).to(torch.int32) + first_page
        self.table = torch.full((len(per), max(per) + 1), -7, dtype=torch.int32)    # unused entries are no page ids
        at = 0
        for b, x in enumerate(per):
            self.table[b, :x] = perm[at:at + x]
            at += x
        gd = torch.Generator(device=DEV).manual_seed(seed)
        shape = (n, hkv, page, d)
        made = []
        for _ in range(2):
            big = torch.empty((n, 1 + gap) + shape[1:], dtype=torch.uint8 if self.e4 else torch.bfloat16, device=DEV)
            x = big[:, 0]
            if fill:
                if self.e4:
                    x.copy_((torch.randn(shape, generator=gd, device=DEV) * 70).clamp(-448, 448).to(E4M3).view(torch.uint8))
                else:
                    x.copy_(torch.randn(shape, generator=gd, device=DEV))
            made.append(x)
        self.k, self.v = made
        self.ks = self.vs = None
        if self.e4:
            self.ks, self.vs = (torch.exp2(torch.randint(-9, -4, (n, hkv), generator=gd, device=DEV).float()) for _ in range(2))
        self.dev_table = self.table.to(DEV)
        self.c = capi.masw_paged_cache(self.k, self.v, self.dev_table, self.ks, self.vs)

    def values(self, x):
        return np64(x.contiguous().view(E4M3)) if self.e4 else np64(x)

    def mirror(self):
        return {"k": self.values(self.k), "v": self.values(self.v),
                "k_scale": None if self.ks is None else np64(self.ks), "v_scale": None if self.vs is None else np64(self.vs)}


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def starts(n, first=0):
    return [first] + [first + int(x) for x in np.cumsum(n)]


def tables(n_pos, rot, theta=10000.0):
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def check_attention(cache, table, kv_len, row_start, q, o, lse, window=0, scale=None):
    """Tolerances.  Scores: fp32 sums of D products (each partial sum rounded: D 2^-24 of the sum of magnitudes, taken
    as 2^-16) and Q as two e4m3 terms (2^-14 of the largest |q| of its rows times the sum of |k|).  An error e of a
    score changes a weight by the factor 1 + e.  Weights enter P V rounded to at most 2^-8 relative (bf16's half
    step; the e4m3 terms are finer), so each output element is off by at most (2^-8 + 2 e) of the weighted mean of
    |v|, plus its own rounding, 2^-8 relative in bf16."""
    qn = np64(q)
    want_o, want_l, mean_abs, qk, kk = po.attention(cache, table, kv_len, row_start, qn, window, scale)
    r0, r1 = row_start[0], row_start[-1]
    got_o, got_l = np64(o)[r0:r1], np64(lse)[r0:r1]
    want_o, want_l = want_o[r0:r1], want_l[r0:r1]
    qmax = np.abs(qn[np.isfinite(qn)]).max() if qn.size else 0.0
    e = qk[r0:r1] * 2.0 ** -16 + kk[r0:r1] * qmax * 2.0 ** -14
    tol = np.abs(want_o) * 2.0 ** -8 + (2.0 ** -8 + 2 * e[..., None]) * mean_abs[r0:r1] + 1e-30
    same = np.isnan(want_o) & np.isnan(got_o)
    bad = ~((np.abs(got_o - want_o) <= tol) | same)
    assert not bad.any(), (np.argwhere(bad)[:5], got_o[bad][:5], want_o[bad][:5])
    empty = np.isneginf(want_l)
    assert (np.isneginf(got_l) == empty).all()
    tol_l = np.where(empty, 0, e + 2.0 ** -18 * (1 + np.abs(np.where(empty, 0, want_l))))
    bad = ~((np.abs(np.where(empty, 0, got_l) - np.where(empty, 0, want_l)) <= tol_l) | (np.isnan(want_l) & np.isnan(got_l)))
    assert not bad.any(), (np.argwhere(bad)[:5], got_l[bad][:5], want_l[bad][:5])
