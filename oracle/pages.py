"""Oracle of the page bookkeeping (CPU, plain loops): what a ring of free pages
hands to the sequences of a step, and what comes back.

TEST INFRASTRUCTURE.  "In-flight Batching", §KV Cache 管理的协同优化: pages of 16
tokens, a block table per sequence, pages freed when a request finishes.
"""
from __future__ import annotations

import numpy as np


def assign(q_len, context_len, ring, head, tail, block_table, page_size=16):
    """(cu_q_len, block_table, slots, head) of a step; None when the free pages
    are too few."""
    ring, table = np.asarray(ring), np.array(block_table)
    cu, slots = [0], []
    for s, (q, c) in enumerate(zip(q_len, context_len)):
        q, c = int(q), int(c)
        for pos in range(c - q, c):
            if pos % page_size == 0:
                if head == tail:
                    return None
                table[s, pos // page_size] = ring[head % len(ring)]
                head += 1
            slots.append(int(table[s, pos // page_size]) * page_size + pos % page_size)
        cu.append(cu[-1] + q)
    return np.array(cu, np.int32), table, np.array(slots, np.int64), head


def release(lengths, ring, head, tail, block_table, page_size=16):
    """(ring, tail) after the sequences with lengths > 0 gave their pages back."""
    ring = np.array(ring)
    for s, n in enumerate(lengths):
        for lp in range(-(-int(n) // page_size)):
            if tail - head >= len(ring):
                return None
            ring[tail % len(ring)] = block_table[s][lp]
            tail += 1
    return ring, tail
