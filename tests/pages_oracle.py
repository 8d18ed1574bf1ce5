"""The paged-cache bookkeeping written out from its definition in plain
Python, one sequence and one page at a time."""
import numpy as np

INT32_MAX = 2 ** 31 - 1


def pages(tokens, page_size):
    return -(-tokens // page_size)


def build(prefix, new, held, table, stack, free, page_size, num_rows):
    """Returns (table, row_starts, slot_map, counts, free, status names)."""
    table = np.array(table, np.int64)
    B, max_pages = table.shape
    num_pages = len(stack)
    starts, slots, counts, status = [0], np.full(num_rows, -1, np.int64), [], []
    pool_ok = 0 <= free <= num_pages
    asked, left = 0, free
    for b in range(B):
        L, n, h = int(prefix[b]), int(new[b]), int(held[b])
        begin = starts[-1]
        end = begin + max(n, 0)
        starts.append(end)
        valid = (L >= 0 and n >= 0 and L + n <= max_pages * page_size and end <= num_rows
                 and 0 <= h <= max_pages and h >= pages(L, page_size))
        if not valid:
            counts.append(h)
            status.append("BAD_INPUT")
            continue
        need = max(0, pages(L + n, page_size) - h)
        asked += need
        served = need == 0 or (pool_ok and asked <= free)
        for j in range(need):
            table[b, h + j] = stack[free - 1 - (asked - need + j)] if served else -1
        counts.append(h + need if served else h)
        if served and need:
            left = free - asked
        bad = not served and not pool_ok
        if served:
            for i in range(n):
                pg = int(table[b, (L + i) // page_size])
                if 0 <= pg < num_pages:
                    slots[begin + i] = pg * page_size + (L + i) % page_size
            for j in range(L // page_size, pages(L + n, page_size)):
                bad = bad or not 0 <= table[b, j] < num_pages
            bad = bad or any(not 0 <= table[b, h + j] < num_pages for j in range(need))
        else:
            bad = bad or any(not 0 <= table[b, j] < num_pages
                             for j in range(L // page_size, min(h, pages(L + n, page_size))))
        status.append("BAD_INPUT" if bad else "OK" if served else "NO_PAGES")
    return table, np.minimum(starts, INT32_MAX), slots, np.array(counts), left, status


def release(keep, held, table, stack, free, page_size):
    """Returns (stack, counts, free, status names)."""
    table, stack = np.asarray(table), np.array(stack, np.int64)
    max_pages, num_pages = table.shape[1], len(stack)
    pool_ok = 0 <= free <= num_pages
    given, left, counts, status = 0, free, [], []
    for b in range(len(keep)):
        k, h = int(keep[b]), int(held[b])
        if k < 0 or h < pages(k, page_size) or h > max_pages:
            counts.append(h)
            status.append("BAD_INPUT")
            continue
        kept = pages(k, page_size)
        back = h - kept
        given += back
        if back and not (pool_ok and free + given <= num_pages):
            counts.append(h)
            status.append("BAD_INPUT")
            continue
        for j in range(back):
            stack[free + given - back + j] = table[b, kept + j]
        if back:
            left = free + given
        counts.append(kept)
        status.append("OK")
    return stack, np.array(counts), left, status
