"""csa_cache_copy in plain numpy, from its definition."""
import numpy as np

BAD_INDEX, CAPACITY = 0x4, 0x2


def copy_slots(src, src_n, dst, dst_n, src_slot, dst_slot, keep=None, max_blocks=None, same=False):
    """src / dst: lists of planes [batch, cap, row]. Returns (new dst planes, new dst_n, status bits)."""
    out, out_n, status = [p.copy() for p in dst], np.array(dst_n).copy(), 0
    batch, cap = dst[0].shape[:2]
    for i, (s, d) in enumerate(zip(src_slot, dst_slot)):
        if not 0 <= d < batch or s >= len(src_n) or d in list(dst_slot[:i]):
            status |= BAD_INDEX
            continue
        others = [x for j, x in enumerate(src_slot) if j != i]
        if same and d in others and not (s == d and keep is None):
            status |= BAD_INDEX
            continue
        rows = []
        if s >= 0:
            filled = min(max(int(src_n[s]), 0), src[0].shape[1])
            rows = list(range(filled))
            if keep is not None:
                rows, last = [], -1
                for e in keep[i]:
                    if e < 0:
                        break
                    if e >= filled or e <= last:
                        status |= BAD_INDEX
                        break
                    rows.append(int(e))
                    last = e
            if max_blocks is not None:
                rows = rows[:max(int(max_blocks[i]), 0)]
        if len(rows) > cap:
            status |= CAPACITY
            continue
        for p, q in zip(src, out):
            q[d, :len(rows)] = p[s, rows]
        out_n[d] = len(rows)
    return out, out_n, status
