"""Which block each slot of the scan's table holds, and which neighbour it waits for, run on the host (CPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
B = 128


@pytest.fixture(scope="module")
def table():
    out = os.path.join(ROOT, "tests", "_build", "seq_search.so")
    os.makedirs(os.path.dirname(out), exist_ok=True)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "gated_delta_rule_29_gb300", "csrc"), "-o", out,
                    os.path.join(ROOT, "tests", "c", "seq_search.cpp")], check=True)
    fn = ctypes.CDLL(out).seq_search_table
    fn.restype, fn.argtypes = None, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]

    def rows(cu, T, backward):
        cu = np.asarray(cu, dtype=np.int64)
        out = np.zeros((T // B + len(cu) - 1, 6), dtype=np.int64)
        fn(cu.ctypes.data, len(cu) - 1, T, backward, out.ctypes.data)
        return out
    return rows


def check_waits(rows, T, N, backward):
    """Blocks lie inside the batch; a block that waits has the block it waits for in the slot beside it, which leaves
    it something; and the slots that it may look back over are in the table."""
    toward = 1 if backward else -1
    for slot, (seq, c, count, start, order, last) in enumerate(rows):
        if seq < 0:
            continue
        assert 0 <= seq < N and 0 <= start and start + count <= T and count <= B, slot
        if order > 0:
            assert 0 <= slot + toward * order < len(rows), slot
            other = rows[slot + toward]
            assert other[0] == seq and other[1] == c + toward and not other[5], (slot, rows[slot], other)


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("N", [1, 2, 32, 33, 40, 200, 1024, 1025, 3000])
def test_valid_boundaries(table, N, backward):
    """Every block of every sequence is in its own slot, and waits for its neighbour unless it begins the chain."""
    rng = np.random.default_rng(N)
    for kind in range(6):
        lens = rng.integers(0, (5, 900, 300, 200, 129, 2)[kind], N)
        lens[rng.integers(0, N)] = 700
        cu = np.concatenate([[0], np.cumsum(lens)])
        T = int(cu[-1])
        rows = table(cu, T, backward)
        check_waits(rows, T, N, backward)
        want = np.full((T // B + N, 6), -1)
        for i, L in enumerate(lens):
            blocks = max(1, -(-int(L) // B))
            for c in range(blocks):
                order = blocks - 1 - c if backward else c
                want[cu[i] // B + i + c] = i, c, min(B, L - c * B), cu[i] + c * B, order, order == blocks - 1
        have = want[:, 0] >= 0
        assert np.array_equal(rows[have], want[have]) and (rows[~have, 0] == -1).all()


@pytest.mark.parametrize("backward", [0, 1])
def test_invalid_boundaries_wait_for_nothing_that_is_not_there(table, backward):
    # 40 sequences of 300 tokens, one of which begins 512 tokens too early: slot 66 holds block 3 of sequence 21, behind
    # the last block of sequence 19
    cu = 300 * np.arange(41)
    cu[21] = cu[20] - 512
    check_waits(table(cu, 12000, backward), 12000, 40, backward)
    rng = np.random.default_rng(5)
    for k in range(400):
        N = int(rng.integers(33, 300))
        T = int(rng.integers(N, 40000))
        cu = rng.integers(-200, T + 200, N + 1) if k % 2 else np.sort(rng.integers(0, T + 1, N + 1))
        for _ in range(int(rng.integers(1, 4))):
            cu[rng.integers(0, N + 1)] = rng.integers(0, T + 1)
        check_waits(table(cu, T, backward), T, N, backward)
