"""Drafted tokens that are given back while a sliding window releases blocks: what is left of a
sequence can always be attended to (host only)."""
import random

import pytest

from paged_kv_cache_90_gb300.block_manager import BlockAllocator, BlockManager


def readable(m, sid, window):
    """Every position that a decode with `window` reads has a block."""
    s = m.seqs[sid]
    for pos in range(max(0, s.length - window), s.length):
        assert s.slot(pos, m.bs) >= 0


def test_a_window_that_would_reach_released_blocks_is_refused():
    """100 tokens, ten of them drafted, in blocks of 16 with a window of 32: blocks 0 to 3 are
    released (positions 68 on are read); with 90 tokens the window starts in block 3."""
    m = BlockManager(BlockAllocator(8, 16))
    m.add_sequence("a", 100)
    assert m.release_outside_window("a", 32) == [0, 1, 2, 3]
    before = list(m.seqs["a"].blocks)
    for length in (90, 95, 64, 1, 0):
        with pytest.raises(ValueError):
            m.truncate("a", length)
        assert m.seqs["a"].length == 100 and m.seqs["a"].blocks == before
    m.check_structure()
    for length in (99, 96):   # the window of 96 tokens starts at position 64, block 4's first
        m.truncate("a", length)
        readable(m, "a", 32)
    with pytest.raises(ValueError):
        m.truncate("a", 95)
    m.fork("a", "b")   # the child's window is its parent's
    with pytest.raises(ValueError):
        m.truncate("b", 95)
    m.check_structure()


def test_drafted_tokens_keep_the_blocks_that_a_shorter_sequence_reads():
    m = BlockManager(BlockAllocator(8, 16))
    m.add_sequence("a", 100)
    assert m.release_outside_window("a", 32, drafted=10) == [0, 1, 2]
    m.truncate("a", 90)
    readable(m, "a", 32)
    with pytest.raises(ValueError):
        m.truncate("a", 79)   # a window from position 47 on, in block 2
    assert m.release_outside_window("a", 32) == []
    with pytest.raises(ValueError):
        m.release_outside_window("a", 32, drafted=-1)
    m.check_structure()


@pytest.mark.parametrize("seed", range(8))
def test_speculative_steps_with_a_window(seed):
    """Steps that draft tokens, release what the window has left and give some back."""
    rng = random.Random(seed)
    bs, window, most = rng.choice((2, 4, 8, 16, 32)), rng.randint(1, 70), rng.randint(1, 24)
    m = BlockManager(BlockAllocator(200, bs))
    m.add_sequence("a", rng.randint(1, 150))
    for _ in range(60):
        drafted = rng.randint(0, most)
        for _ in range(drafted):
            m.append_token("a")
        m.release_outside_window("a", window, drafted=drafted)
        m.truncate("a", m.seqs["a"].length - rng.randint(0, drafted))
        readable(m, "a", window)
        m.append_token("a")
        readable(m, "a", window)
        m.check_structure()
        s = m.seqs["a"]   # no more is kept than a step's drafted tokens ask for
        assert s.released >= max(0, s.length - 1 - most - window) // bs
