"""Plain 64-bit attention over a paged cache, inputs for it, and how far a result may be from it."""

import math

import torch


def rows_of(pool, table, n):
    """The first n rows of a sequence (NaN where the table names no page)."""
    page = pool.shape[1]
    ids = table[:-(-n // page)].long()
    rows = pool[ids.clamp(0, pool.shape[0] - 1)].double()
    rows[(ids < 0) | (ids >= pool.shape[0])] = math.nan
    return rows.reshape(-1, pool.shape[2])[:n]


def attention(q, cache, pages, seqs, window=0, scale=None, comp=None, comp_pages=None, ratio=0, start0=0):
    """(out, sum of the weights times the rows' magnitudes) of each token; seqs: (new, length) of each sequence, the
    first one's tokens from start0 on.  Tokens of no sequence: NaN."""
    d = q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    size = out.clone()
    at = start0
    for s, (new, length) in enumerate(seqs):
        x = rows_of(cache, pages[s], length)
        y = rows_of(comp, comp_pages[s], length // ratio) if ratio else None
        for i in range(new):
            t = length - new + i
            lo = max(0, t + 1 - window) if window else 0
            k = x[lo:max(t + 1, 0)]
            if ratio:
                k = torch.cat([k, y[:max(t + 1, 0) // ratio]])
            if k.shape[0] == 0:
                out[at + i] = size[at + i] = 0.0
                continue
            p = torch.softmax(q[at + i].double() @ k.T * scale, dim=-1)
            out[at + i], size[at + i] = p @ k, p @ k.abs()
        at += new
    return out, size


def pool(gen, rows_per_seq, page, d, first=None, spare=3, fill=math.nan):
    """A bfloat16 pool and table: the rows first[s] .. rows_per_seq[s] - 1 of each sequence normal values, everything
    else `fill`; pages in no order, those that hold no such row not listed (-1)."""
    first = first or [0] * len(rows_per_seq)
    need = [(f // page, -(-r // page)) for f, r in zip(first, rows_per_seq)]
    total = sum(b - a for a, b in need) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(need), max([b for _, b in need] + [1])), -1, dtype=torch.int32, device="cuda")
    rows = torch.full((total, page, d), fill, dtype=torch.bfloat16, device="cuda")
    at = 0
    for s, (a, b) in enumerate(need):
        if b <= a:
            continue
        ids = order[at:at + b - a]
        at += b - a
        table[s, a:b] = ids
        flat = rows[ids.long()].view(-1, d)
        lo, hi = first[s] - a * page, rows_per_seq[s] - a * page
        flat[lo:hi] = torch.randn(hi - lo, d, generator=gen, device="cuda").bfloat16()
        rows[ids.long()] = flat.view(-1, page, d)
    return rows, table


def starts(seqs, start0=0):
    at = [start0]
    for new, _ in seqs:
        at.append(at[-1] + new)
    return torch.tensor(at, dtype=torch.int32, device="cuda"), torch.tensor([m for _, m in seqs], dtype=torch.int32, device="cuda")


def assert_close(got, want, size):
    """Each probability is rounded to bfloat16, by 2^-8 of it at most, so the weighted sum by 2^-8 of the weighted
    magnitudes; the result is rounded once more, by 2^-8 of it.  Everything in float (logits of at most a few thousand
    steps of 2^-23 of their terms, exponentials, sums) stays below 2^-11 of the magnitudes."""
    tol = (2.0 ** -8 + 2.0 ** -11) * size + 2.0 ** -8 * want.abs() + 1e-30
    bad = ~((got.double() - want).abs() <= tol) & ~(got.isnan() & want.isnan())
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got.double() - want).abs() / tol)[bad].max()))
