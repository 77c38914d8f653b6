"""Evictions of several sequences for one move: no block that the move writes for one of them is in
another's old table, whatever they share and however few blocks are free."""
import os

import numpy as np
import pytest

from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build

OOM, INVALID, NOT_FOUND = 2, 1, 3
W = 32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pa_build.build()


def tables(a, seqs):
    return [[int(x) for x in row if x >= 0] for row in a.export(list(seqs), W)[0]]


def status(fn, *args):
    with pytest.raises(binding.PaError) as e:
        fn(*args)
    return e.value.status


def state(a, seqs):
    return (tables(a, seqs), [a.seq_info(s)[0] for s in seqs], list(a.free_list()), a.stats(), a.prefix_stats())


def check_move(old, new, cut):
    """What pa_compact_tokens asks of the tables of a call."""
    for i in range(len(old)):
        if not cut[i]:
            assert new[i] == old[i]
            continue
        for j, b in enumerate(new[i]):
            assert b not in old[i] or old[i][j] == b
            for k in range(len(old)):
                assert k == i or (b not in old[k] and b not in new[k]), (i, k, b)


def evict(a, batch, seqs, lens):
    if batch:
        a.evict_batch(seqs, lens)
    else:
        for s, n in zip(seqs, lens):
            a.evict(s, n)


@pytest.mark.parametrize("batch", [False, True])
def test_the_last_holder_of_a_block_does_not_write_it_either(batch):
    """Two forks of 90 tokens, both at 96, cut to 64: after the first one's cut the second is the only
    holder of the blocks that the first one's old table is still to be read by."""
    a = binding.Allocator(80, 8)
    a.alloc(0, 90)
    a.fork(0, 1)
    for _ in range(6):
        a.append_batch([0, 1])
    old = tables(a, (0, 1))
    assert old[0][:11] == old[1][:11] and old[0][11] != old[1][11]
    evict(a, batch, [0, 1], [64, 64])
    check_move(old, tables(a, (0, 1)), (True, True))
    used = sum(tables(a, (0, 1)), [])
    assert len(set(used)) == 16 and sorted(used + list(a.free_list())) == list(range(80))


@pytest.mark.parametrize("batch", [False, True])
def test_blocks_dropped_by_one_are_not_given_to_another(batch):
    """12 blocks of 8: sequence 1 drops three, sequence 2 shares its two blocks and one block is free."""
    a = binding.Allocator(9, 8)
    a.alloc(1, 48)
    a.alloc(2, 16)
    a.fork(2, 3)
    before = state(a, (1, 2, 3))
    if batch:
        assert status(a.evict_batch, [1, 2], [24, 15]) == OOM
        assert state(a, (1, 2, 3)) == before
        a.evict_batch([1], [24])
    else:
        a.evict(1, 24)
    cut = state(a, (1, 2, 3))
    assert cut[2] == [8, 3, 4, 5]                  # four free, three of them still to be read
    assert status(a.evict, 2, 15) == OOM and state(a, (1, 2, 3)) == cut
    a.evict_batch([], [])                          # the move has been launched
    old = tables(a, (2,))
    a.evict(2, 15)
    assert tables(a, (2, 3)) == [[8, 3], old[0]]


@pytest.mark.parametrize("hand_out", [
    lambda a: a.append_slot(9), lambda a: a.append_batch([9]), lambda a: a.append_token(9, 5),
    lambda a: a.alloc(9, 3), lambda a: a.alloc_prompt(10, []), lambda a: a.swap_in(8)])
def test_calls_that_hand_out_slots_end_a_run_of_evictions(hand_out):
    a = binding.Allocator(10, 8)
    a.set_swap_pool(2)
    a.alloc_prompt(9, [1, 2])
    a.alloc(8, 0)
    a.swap_out(8)
    a.alloc(1, 48)
    a.alloc(2, 16)
    a.fork(2, 3)
    a.evict(1, 24)                                 # one free block more, three that are still to be read
    assert status(a.evict, 2, 15) == OOM
    hand_out(a)
    a.evict(2, 15)
    assert tables(a, (2,))[0][1] in (3, 4, 5, 9)


def test_other_calls_do_not_and_freed_blocks_can_be_taken():
    a = binding.Allocator(10, 8)
    a.set_swap_pool(4)
    a.alloc(1, 48)
    a.alloc(2, 16)
    a.fork(2, 3)
    a.alloc(4, 16)
    old = tables(a, (1, 2))
    a.evict(1, 24)
    assert status(a.evict, 2, 15) == OOM
    assert status(a.alloc, 5, 8 * 9) == OOM        # a refused call ends nothing
    assert status(a.evict, 2, 15) == OOM
    a.fork(4, 6)
    a.free(6)
    a.swap_out(4)                                  # its two blocks lie behind those that 1 dropped
    assert list(a.free_list()) == [3, 4, 5, 8, 9]
    a.evict(2, 15)
    assert tables(a, (2,))[0] == [8, 9] and list(a.free_list()) == [3, 4, 5]
    check_move(old, tables(a, (1, 2)), (True, True))


def test_one_that_shares_with_a_cut_one_is_replaced_too_when_the_others_are_gone():
    a = binding.Allocator(12, 8)
    a.alloc(1, 24)
    a.fork(1, 2)
    a.fork(1, 3)
    old = tables(a, (1, 2))
    a.evict(1, 0)                                  # drops all three, which 2 and 3 keep
    a.free(3)
    assert [a.block_ref(b) for b in old[1]] == [1, 1, 1]
    a.evict(2, 9)
    check_move(old, tables(a, (1, 2)), (True, True))
    assert tables(a, (2,))[0] == [3, 4] and list(a.free_list()) == [5, 6, 7, 8, 9, 10, 11, 0, 1, 2]
    a.append_slot(2)
    a.evict(2, 8)                                  # a new run: in place
    assert tables(a, (2,))[0] == [3]


def test_equal_lengths_in_a_batch_change_nothing_of_theirs():
    a = binding.Allocator(12, 8)
    a.alloc(1, 24)
    a.fork(1, 2)
    a.alloc(3, 5)
    old = tables(a, (1, 2, 3))
    a.evict_batch([1, 2, 3], [24, 10, 5])
    new = tables(a, (1, 2, 3))
    check_move(old, new, (False, True, False))
    assert new[1] == [4, 5] and [a.seq_info(s)[0] for s in (1, 2, 3)] == [24, 10, 5]


def test_refusals_change_nothing():
    a = binding.Allocator(12, 8)
    a.set_swap_pool(4)
    a.alloc(1, 24)
    a.alloc(2, 10)
    a.alloc(3, 10)
    a.swap_out(3)
    before = state(a, (1, 2))
    for seqs, lens, want in (([1, 2], [8, 11], INVALID), ([1, 2], [8, -1], INVALID), ([1, 1], [8, 8], INVALID),
                             ([1, 7], [8, 8], NOT_FOUND), ([1, 3], [8, 8], INVALID)):
        assert status(a.evict_batch, seqs, lens) == want and state(a, (1, 2)) == before
    with pytest.raises(ValueError):
        a.evict_batch([1, 2], [8])
    lib = binding.load()
    assert lib.pa_alloc_evict_batch(None, None, None, 0) == lib.pa_alloc_evict_batch(a._h, None, None, -1) == INVALID
    assert lib.pa_alloc_evict_batch(a._h, None, None, 1) == INVALID
    assert lib.pa_alloc_evict_batch(a._h, None, None, 0) == 0


def model_cut(ref, left, run, free, tab, lens, seqs, cuts, bs, whole):
    """The rules in plain lists: whole = the cuts of one evict_batch.  True, or False for no room."""
    todo = []
    r, l, f, t = dict(ref), dict(left), list(free), {s: list(tab[s]) for s in tab}
    for s, n in zip(seqs, cuts):
        if n == lens[s]:
            continue
        stay = -(-n // bs)
        fresh = [j for j in range(stay) if r[t[s][j]] > 1 or l.get(t[s][j]) == run]
        usable = [b for b in f if l.get(b) != run]
        if len(fresh) > len(usable):
            return False
        for j in fresh:
            b = t[s][j]
            t[s][j] = usable.pop(0)
            f.remove(t[s][j])
            r[t[s][j]] = 1
            r[b] -= 1
            l[b] = run
            if r[b] == 0:
                f.append(b)
        for b in t[s][stay:]:
            r[b] -= 1
            l[b] = run
            if r[b] == 0:
                f.append(b)
        t[s] = t[s][:stay]
        todo.append((s, n))
    ref.update(r)
    left.update(l)
    free[:] = f
    tab.update(t)
    lens.update(todo)
    return True


@pytest.mark.parametrize("seed", range(12))
def test_random_forks_and_cuts(seed):
    rng = np.random.default_rng(seed)
    bs, N = 8, int(rng.choice([24, 40, 200]))
    a = binding.Allocator(N, bs)
    refused = cuts = 0
    for turn in range(60):
        live, nxt = [], 100 * turn
        for _ in range(int(rng.integers(1, 4))):
            n = int(rng.integers(1, 60))
            if a.stats()["free_blocks"] < -(-n // bs):
                break
            a.alloc(nxt, n)
            live.append(nxt)
            nxt += 1
            for _ in range(int(rng.integers(0, 4))):
                a.fork(int(rng.choice(live)), nxt)
                live.append(nxt)
                nxt += 1
        for s in list(live):
            for _ in range(int(rng.integers(0, 6))):
                try:
                    a.append_slot(s)
                except binding.PaError:
                    break
        a.evict_batch([], [])
        old = dict(zip(live, tables(a, live)))
        lens = {s: a.seq_info(s)[0] for s in live}
        was = dict(lens)
        free = [int(b) for b in a.free_list()]
        ref = {b: a.block_ref(b) for b in range(N)}
        seqs = [int(s) for s in rng.permutation(live)][: int(rng.integers(1, len(live) + 1))]
        to = [int(rng.integers(0, lens[s] + 1)) for s in seqs]
        tab, left = {s: list(old[s]) for s in live}, {}
        done = []
        if turn % 2:
            want = model_cut(ref, left, 1, free, tab, lens, seqs, to, bs, True)
            if want:
                a.evict_batch(seqs, to)
                done = seqs
            else:
                assert status(a.evict_batch, seqs, to) == OOM
                refused += 1
        else:
            for s, n in zip(seqs, to):
                if model_cut(ref, left, 1, free, tab, lens, [s], [n], bs, False):
                    a.evict(s, n)
                    done.append(s)
                else:
                    assert status(a.evict, s, n) == OOM
                    refused += 1
                others = [x for x in live if x not in seqs]
                if others and rng.integers(4) == 0:          # in between, a sequence ends
                    x = int(rng.choice(others))
                    a.free(x)
                    live.remove(x)
                    for b in tab.pop(x):
                        ref[b] -= 1
                        if ref[b] == 0:
                            free.append(b)
                    lens.pop(x)
        cuts += len(done)
        new = dict(zip(live, tables(a, live)))
        assert new == tab and {s: a.seq_info(s)[0] for s in live} == lens
        assert [int(b) for b in a.free_list()] == free and {b: a.block_ref(b) for b in range(N)} == ref
        check_move([old[s] for s in done], [new[s] for s in done], [lens[s] < was[s] for s in done])
        for s in done:                                       # nor is anything written that another one holds
            if lens[s] < was[s]:
                assert all(ref[b] == 1 for b in new[s])
        for s in live:
            a.free(s)
        assert sorted(a.free_list()) == list(range(N))
    assert cuts > 60 and (N > 24 or refused > 0)


def test_the_readme_cuts_a_batch_with_a_sequence_within_its_budget():
    """README.md's lines between the choice and the move, run as they stand."""
    text = open(os.path.join(os.path.dirname(pa_build.PKG), "README.md"), encoding="utf-8").read()
    lines = text[text.index("old_tables, "): text.index("pa.pa_compact_tokens(")]
    a = binding.Allocator(40, 8)
    for s, n in ((5, 100), (3, 20), (8, 64)):
        a.alloc(s, n)
    a.fork(5, 6)
    scope = dict(alloc=a, seq_ids=[5, 3, 6, 8], max_blocks=16, keep=64, np=np)
    exec(lines, scope)
    assert list(scope["new_lens"]) == [64, 20, 64, 64]
    old, new = ([[int(x) for x in row if x >= 0] for row in scope[t]] for t in ("old_tables", "new_tables"))
    check_move(old, new, (True, False, True, False))
