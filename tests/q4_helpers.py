"""Cases of the 4-bit cache: those of attention_helpers with their pools coded."""
import numpy as np

from attention_helpers import case, host
from oracle import q4_ref


def q4_case(torch, *args, **kw):
    """attention_helpers.case with q4 pools: k, v are the values that their
    codes stand for (so its reference and bound apply), k4, v4 the pools."""
    return coded(torch, case(torch, *args, **kw))


def coded(torch, c):
    for n in ("k", "v"):
        code, scale = q4_ref.encode(host(c[n]), c["dtype"])
        c[n + "4"] = torch.from_numpy(q4_ref.pack(code, scale)).cuda()
        c[n] = torch.from_numpy(q4_ref.decode(code, scale)).to(c["q"].dtype).cuda()
    return c


def scale_byte(pool, page, head, row, group):
    """View of one scale byte of a pool."""
    pages, heads, size, width = pool.shape
    dim = width * 32 // 17
    flat = pool.view(pages, -1)
    at = heads * size * dim // 2 + (head * size + row // 16 * 16) * (dim // 32) + group * 16 + row % 16
    return flat[page, at:at + 1]


def junk_rows(torch, pool, page, head_rows, rng, scale=None):
    """Rows of a page (all heads) with any codes and scales (or one scale)."""
    pages, heads, size, width = pool.shape
    dim = width * 32 // 17
    flat = pool.view(pages, -1)
    codes = flat[:, :heads * size * dim // 2].view(pages, heads, size, dim // 2)
    scales = flat[:, heads * size * dim // 2:].view(pages, heads, size // 16, dim // 32, 16)
    for r in head_rows:
        codes[page, :, r] = torch.from_numpy(rng.integers(0, 256, (heads, dim // 2), dtype=np.uint8)).cuda()
        if scale is None:
            scales[page, :, r // 16, :, r % 16] = torch.from_numpy(rng.integers(0, 256, (heads, dim // 32), dtype=np.uint8)).cuda()
        else:
            scales[page, :, r // 16, :, r % 16] = scale
