"""Shared by the tests of include/mla_chunk.h: a paged cache of any format with
the float64 values of its rows, garbage in every slot that holds none."""
import numpy as np
import torch

from oracle import layer as L

ROW = {"bf16": 1152, "fp8": 594, "fp4": 324}


def kind(m, kv):
    return {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0, "fp4": m.MLA_KV_FP4_E2M1_E8M0}[kv]


def put(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


class Paged:
    """Caches of requests of `lens` rows in shuffled pages."""

    def __init__(self, rng, lens, page, kv, spare=3, extra_pages=0):
        self.lens, self.page, self.kv = np.asarray(lens), page, kv
        batch = len(lens)
        pages = -(-self.lens // page)
        self.max_pages = int(max(1, pages.max(initial=1) + extra_pages))
        self.num_pages = int(pages.sum()) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((batch, self.max_pages), 0x40000000, dtype=np.int32)   # never read behind a request's pages
        for b, first in enumerate(np.cumsum(pages) - pages):
            self.table[b, :pages[b]] = order[first:first + pages[b]]
        slots = self.num_pages * page
        if kv == "bf16":
            rows = torch.from_numpy(rng.standard_normal((slots, 576), dtype=np.float32)).to(torch.bfloat16)
            self.raw = rows.view(torch.int16).numpy().view(np.uint16)
            garbage = np.uint16(0x7FC0)
        else:
            codes = 576 if kv == "fp8" else 288
            self.raw = rng.integers(0, 256, (slots, ROW[kv]), dtype=np.uint8)
            if kv == "fp8":
                self.raw[:, :codes] &= 0xBF                     # magnitudes below 2 before the scale
            self.raw[:, codes:] = 124 + self.raw[:, codes:] % 4
            garbage = np.uint8(0xFF)                            # NaN codes and NaN scales
        self.slots = [self.table[b, np.arange(n) // page] * page + np.arange(n) % page
                      for b, n in enumerate(self.lens)]
        dead = np.ones(slots, dtype=bool)
        dead[np.concatenate(self.slots) if batch else []] = False
        self.raw[dead] = garbage
        self.dead = dead
        self.cache = put(self.raw.view(np.int16) if kv == "bf16" else self.raw)

    def rows(self, b):
        """Request b's rows [T, 576] in float64."""
        return L.gather_rows(self.raw, self.slots[b], self.kv)

    def problem(self, m, heads=1, **kw):
        return m.make_problem(len(self.lens), 1, heads, self.page, self.num_pages, self.max_pages,
                              kv_dtype=kind(m, self.kv), **kw)
