"""The paged cache's update (dlrm_seq_pages.h) user by user, in Python: test infrastructure only."""
from __future__ import annotations

import numpy as np


def update(table, lengths, free, free_count, page, off, n, leave=None):
    """What dlrm_seq_pages_update leaves: (table, lengths, free, free_count, slots, refused), of copies.  slots where
    nothing is written: -7."""
    table, lengths, free = table.copy(), lengths.copy(), free.copy()
    top, width = int(free_count), table.shape[1]
    slots, refused = np.full(n, -7, np.int64), 0
    for b in range(len(lengths)):
        if leave is not None and leave[b]:
            have = -(-int(lengths[b]) // page)
            free[top:top + have] = table[b, :have]
            table[b, :have] = -1
            top, lengths[b] = top + have, 0
    wanted, stack = 0, top
    for b in range(len(lengths)):
        held, new = int(lengths[b]), int(off[b + 1]) - int(off[b])
        have = -(-held // page)
        want = -(-(held + new) // page) - have
        wide = held + new <= width * page
        wanted += want if wide else 0
        if not wide or (want and wanted > stack):
            refused += 1
            slots[off[b]:off[b + 1]] = -1
            continue
        for c in range(want):
            top -= 1
            table[b, have + c] = free[top]
        at = held + np.arange(new)
        slots[off[b]:off[b + 1]] = table[b, at // page].astype(np.int64) * page + at % page
        lengths[b] = held + new
    return table, lengths, free, top, slots, refused
