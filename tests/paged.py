"""Caches in pages for the tests: a table of scattered pages over pools that hold NaN wherever no row lies."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def i32(values):
    return torch.tensor(np.asarray(values, np.int32), device="cuda")


class Paged:
    """Sequences of `lens` rows in pages of `page`; rows [nkv, len, hd] of each in k and v."""

    def __init__(self, lens, nkv, hd, page, dtype, seed=1, spare=3, width=None):
        g, host = gen(seed), np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.lens, self.nkv, self.hd, self.page, self.pages = list(lens), nkv, hd, page, sum(need) + spare
        order = host.permutation(self.pages).astype(np.int32)
        width = max(max(need), 1) if width is None else width
        table, at = np.full((len(lens), width), -1, np.int32), 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.free, self.table_host, self.table, self.lengths = order[at:], table, i32(table), i32(lens)
        self.kp, self.vp = (torch.full((self.pages, nkv, page, hd), float("nan"), device="cuda", dtype=dtype) for _ in range(2))
        self.k = [randn(g, nkv, n, hd, dtype=dtype) for n in lens]
        self.v = [randn(g, nkv, n, hd, dtype=dtype) for n in lens]
        for b in range(len(lens)):
            self.put(b, self.kp, self.k[b])
            self.put(b, self.vp, self.v[b])

    def at(self, b, n=None):
        """(page, row in the page) of the first n rows of sequence b."""
        rows = torch.arange(self.lens[b] if n is None else n, device="cuda")
        return self.table[b].long()[rows // self.page], rows % self.page

    def put(self, b, pool, rows):
        page, row = self.at(b, rows.shape[1])
        pool[page, :, row] = rows.transpose(0, 1)

    def get(self, b, pool, n=None):
        page, row = self.at(b, n)
        return pool[page, :, row].transpose(0, 1)
