"""The page pool's operators in plain Python (whole numbers and copies), one sequence and one page
after another.  Every function takes numpy arrays, leaves them alone and returns new ones and the
error bits."""
from __future__ import annotations

import numpy as np

BLOCK = 128
BAD_PAGE, BAD_SEQLEN, NO_PAGE, BAD_PARENT = 0x1, 0x2, 0x10, 0x20


def blocks(n):
    return -(-int(n) // BLOCK)


def extend(refs, table, lens, new):
    refs, table, lens = refs.copy(), table.copy(), lens.copy()
    free = [p for p in range(len(refs)) if refs[p] == 0]
    err = upto = 0
    given = []
    for b in range(len(lens)):
        L, n = int(lens[b]), int(new[b])
        if L < 0 or n < 0 or L + n > table.shape[1] * BLOCK:
            err |= BAD_SEQLEN
            continue
        need = blocks(L + n) - blocks(L)
        upto += need
        if need and upto > len(free):
            err |= NO_PAGE
            continue
        for i in range(need):
            page = free[upto - need + i]
            table[b, blocks(L) + i] = page
            given.append(page)
        lens[b] = L + n
    refs[given] = 1
    return refs, table, lens, err


def fork(refs, table, lens, parents, buffers=()):
    """buffers: list of (array [P, ...], token axis or None), changed in place."""
    n, width = len(parents), table.shape[1]
    refs, out, out_lens = refs.copy(), np.full((n, width), -1, np.int32), np.zeros(n, np.int32)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    P, err, taken = len(refs), 0, 0
    for i, p in enumerate(int(x) for x in parents):
        if p == -1:
            continue
        if p < -1 or p >= len(lens):
            err |= BAD_PARENT
            continue
        L = int(lens[p])
        if L < 0 or L > width * BLOCK:
            err |= BAD_SEQLEN
            continue
        full, tail = divmod(L, BLOCK)
        out_lens[i] = L
        for j in range(full):
            page = int(table[p, j])
            if 0 <= page < P:
                out[i, j] = page
                refs[page] += 1
            else:
                err |= BAD_PAGE
        if not tail:
            continue
        src = int(table[p, full])
        if not 0 <= src < P:
            err |= BAD_PAGE
        elif taken >= len(free):
            err |= NO_PAGE
            out_lens[i] = full * BLOCK
        else:
            page = free[taken]
            taken += 1
            refs[page] = 1
            out[i, full] = page
            for data, axis in buffers:
                if axis is None:
                    data[page] = data[src]
                else:
                    sel = (slice(None),) * (axis - 1) + (slice(0, tail),)
                    data[page][sel] = data[src][sel]
    return refs, out, out_lens, err


def free(refs, pages, counts=None):
    refs, err = refs.copy(), 0
    for r, row in enumerate(pages):
        n = len(row) if counts is None else int(counts[r])
        if n < 0 or n > len(row):
            err |= BAD_SEQLEN
            continue
        for page in row[:n].tolist():
            if page == -1:
                continue
            if not 0 <= page < len(refs) or refs[page] <= 0:
                err |= BAD_PAGE
            else:
                refs[page] -= 1
    return refs, err


def compact(refs, table, lens, buffers=()):
    P, err = len(refs), 0
    used = [p for p in range(P) if refs[p] != 0]
    n = len(used)
    page_map = np.full(P, -1, np.int32)
    page_map[used] = used
    holes = [p for p in range(n) if refs[p] == 0]
    for src, dst in zip([p for p in used if p >= n], holes, strict=True):
        page_map[src] = dst
        for data, _ in buffers:
            data[dst] = data[src]
    out_refs = np.zeros_like(refs)
    out_refs[page_map[used]] = refs[used]
    out = np.full_like(table, -1)
    for b in range(len(lens)):
        m = table.shape[1]
        if 0 <= lens[b] <= m * BLOCK:
            m = blocks(lens[b])
        else:
            err |= BAD_SEQLEN
        for j in range(m):
            page = int(table[b, j])
            if 0 <= page < P:
                out[b, j] = page_map[page]
            if out[b, j] < 0 and page != -1:
                err |= BAD_PAGE
    return out_refs, out, page_map, n, err
