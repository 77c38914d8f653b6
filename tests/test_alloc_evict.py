"""pa_alloc_evict against a plain model of the allocator's rules."""
import numpy as np
import pytest

from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pa_build.build()


def table(a, seq, width=16):
    return [int(x) for x in a.export([seq], width)[0][0] if x >= 0]


def status(fn, *args):
    with pytest.raises(binding.PaError) as e:
        fn(*args)
    return e.value.status


def test_blocks_behind_the_cut_are_freed_in_order():
    a = binding.Allocator(10, 8)
    a.alloc(1, 61)
    a.evict(1, 20)
    assert table(a, 1) == [0, 1, 2] and a.seq_info(1)[0] == 20
    assert list(a.free_list()) == [8, 9, 3, 4, 5, 6, 7]
    slot, cow = a.append_slot(1)
    assert slot == 2 * 8 + 4 and cow is None
    a.evict(1, 16)
    assert table(a, 1) == [0, 1]
    assert a.append_slot(1)[0] == 8 * 8
    a.evict(1, 0)
    assert table(a, 1) == [] and a.stats()["used_blocks"] == 0
    assert a.append_slot(1)[0] % 8 == 0


def test_shared_blocks_are_replaced_and_stay_with_the_others():
    a = binding.Allocator(9, 8)
    a.alloc(1, 30)
    a.fork(1, 2)
    assert table(a, 2) == [0, 1, 2, 3]
    a.append_slot(2)                               # copies block 3 to 4
    assert table(a, 2) == [0, 1, 2, 4]
    a.evict(2, 13)
    assert table(a, 2) == [5, 6] and table(a, 1) == [0, 1, 2, 3]
    assert [a.block_ref(b) for b in range(9)] == [1, 1, 1, 1, 0, 1, 1, 0, 0]
    assert list(a.free_list()) == [7, 8, 4]
    a.free(1)
    a.free(2)
    assert sorted(a.free_list()) == list(range(9))


def test_no_room_for_replacements_changes_nothing():
    a = binding.Allocator(5, 8)
    a.alloc(1, 32)
    a.fork(1, 2)
    before = (table(a, 1), table(a, 2), list(a.free_list()), a.stats())
    assert status(a.evict, 2, 16) == 2             # two shared blocks stay, one block is free
    assert (table(a, 1), table(a, 2), list(a.free_list()), a.stats()) == before
    a.evict(2, 8)
    assert table(a, 2) == [4]


def test_equal_length_changes_nothing_and_refusals():
    a = binding.Allocator(8, 8)
    a.alloc(1, 20)
    a.fork(1, 2)
    a.evict(2, 20)
    assert table(a, 2) == table(a, 1) == [0, 1, 2]
    assert status(a.evict, 1, 21) == 1 and status(a.evict, 1, -1) == 1 and status(a.evict, 9, 0) == 3
    a.set_swap_pool(4)
    a.swap_out(2)
    assert status(a.evict, 2, 4) == 1


def test_prefix_cache_entries_of_rewritten_blocks_are_dropped():
    a = binding.Allocator(12, 4)
    prompt = list(range(16))
    assert a.alloc_prompt(1, prompt) == 0
    a.evict(1, 6)                                  # blocks 0, 1 stay and are rewritten; 2, 3 keep their content
    assert a.prefix_stats()["entries"] == 2
    assert a.alloc_prompt(2, prompt) == 0          # the prefix's first block is gone
    assert not set(table(a, 1)) & set(table(a, 2))
    # tokens appended to a cut sequence are not registered
    n = a.prefix_stats()["registered"]
    for t in range(8):
        a.append_token(1, t)
    assert a.prefix_stats()["registered"] == n


def test_shared_prefix_blocks_stay_cached():
    a = binding.Allocator(12, 4)
    prompt = list(range(8))
    a.alloc_prompt(1, prompt)
    a.alloc_prompt(2, prompt + [50, 51, 52, 53, 54])
    a.evict(2, 7)
    assert table(a, 1) == [0, 1] and not set(table(a, 2)) & {0, 1}
    assert a.alloc_prompt(3, prompt) == 8


def test_random_walks_keep_the_counts():
    rng = np.random.default_rng(7)
    a = binding.Allocator(64, 8)
    lens, nxt = {}, 0
    for _ in range(600):
        op = rng.integers(4)
        try:
            if op == 0 or not lens:
                a.alloc(nxt, int(rng.integers(1, 60)))
                lens[nxt] = a.seq_info(nxt)[0]
                nxt += 1
            elif op == 1:
                s = int(rng.choice(list(lens)))
                a.fork(s, nxt)
                lens[nxt] = lens[s]
                nxt += 1
            elif op == 2:
                s = int(rng.choice(list(lens)))
                n = int(rng.integers(0, lens[s] + 1))
                cut = n < lens[s]
                a.evict(s, n)
                lens[s] = n
                if cut:
                    assert all(a.block_ref(b) == 1 for b in table(a, s))
            else:
                s = int(rng.choice(list(lens)))
                a.free(s)
                del lens[s]
        except binding.PaError as e:
            assert e.status == 2
            for s in list(lens)[:3]:
                a.free(s)
                del lens[s]
        ref = np.zeros(64, int)
        for s, n in lens.items():
            t = table(a, s)
            assert len(t) == -(-n // 8) and a.seq_info(s)[0] == n
            for b in t:
                ref[b] += 1
        assert [a.block_ref(b) for b in range(64)] == ref.tolist()
        assert sorted(a.free_list()) == [b for b in range(64) if ref[b] == 0]
