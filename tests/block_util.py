"""Shared helpers of the tests of the cache with a scale per block of tokens and head."""
import numpy as np

from oracle import blocks

from gpu_util import host, torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class BlockCache:
    """A cache of random contents; order "phd": slots before heads, "hpd": heads before slots
    and rows padded."""

    def __init__(self, q, rng, pages, page, block, heads, dim, fmt, order="phd", scale=(0.01, 0.03)):
        self.fmt, self.page, self.block = fmt, page, block
        c = rng.integers(0, 256, size=(pages, page, heads, dim), dtype=np.uint8)
        if fmt == "e4m3":
            c = np.where(c & 127 == 127, 5, c).astype(np.uint8)
        s = rng.uniform(*scale, size=(pages, page // block, heads)).astype(np.float32)
        if order == "phd":
            self.codes, self.scales = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
        else:
            self.codes = torch.zeros((pages, heads, page, dim + 16), dtype=torch.uint8,
                                     device="cuda")[..., :dim].transpose(1, 2)
            self.scales = torch.zeros((pages, heads, page // block + 1), device="cuda")[..., :page // block].transpose(1, 2)
            self.codes.copy_(torch.from_numpy(c))
            self.scales.copy_(torch.from_numpy(s))
        self.h = q.make_kv_blocks(self.codes, self.scales, fmt)

    def host(self):
        return host(self.codes), host(self.scales).astype(np.float64)


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def scattered(rng, lengths, page, spare=3, width=None):
    """(table as lists, pages): the sequences' pages in random order over the cache."""
    need = [blocks.pages_of(n, page) for n in lengths]
    pages = max(sum(need) + spare, 1)
    order = rng.permutation(pages)
    width = max(need + [1]) if width is None else width
    table, at = [], 0
    for n in need:
        table.append([int(p) for p in order[at:at + n]] + [-1] * (width - n))
        at += n
    return table, pages


def starts_of(counts):
    return [0] + [int(v) for v in np.cumsum(counts)]
