"""The two warps that check V tiles in window attention (csrc/pa_check.h says which takes which),
as a model of their barriers on the CPU: every order in which the copies, the products and the
two warps can go on, over rings of four and eight slots.

A barrier's wait names a parity and returns where the phase of that parity is complete, as the
hardware's does: a warp that falls two phases behind waits for one that is over."""
import ctypes
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_94_gb300", "csrc")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """check_slot and check_warp as the kernel compiles them."""
    d = tmp_path_factory.mktemp("check")
    src, lib = str(d / "check.cpp"), str(d / "check.so")
    with open(src, "w") as f:
        f.write('#include "pa_check.h"\n'
                'extern "C" unsigned slot(unsigned n, unsigned s) { return pa::check_slot(n, s); }\n'
                'extern "C" unsigned warp(unsigned n) { return pa::check_warp(n); }\n')
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib])
    return ctypes.CDLL(lib)


def stuck_orders(masked, slots, waits, takes, slot_of):
    """Orders that end before every tile had its products. masked[n]: tile n is checked.
    waits(w, n): warp w waits until tile n has landed; takes(w, n): and then checks it."""
    T = len(masked)
    work = [[n for n in range(T) if masked[n] and waits(w, n)] for w in (0, 1)]

    def landings(slot, copied):  # phases that are complete on the slot's barrier
        return sum(1 for n in range(copied) if masked[n] and slot_of(n) == slot)

    def moves(state):
        copied, done, at, checked = state
        if copied < T:  # a tile is copied once the products of the last one in its slot are done
            last = [n for n in range(copied) if slot_of(n) == slot_of(copied)]
            if not last or done > last[-1]:
                yield (copied + 1, done, at, checked)
        if done < copied and (not masked[done] or checked >> done & 1):
            yield (copied, done + 1, at, checked)
        for w in (0, 1):
            if at[w] == len(work[w]):
                continue
            n = work[w][at[w]]
            passed = sum(1 for m in work[w][:at[w]] if slot_of(m) == slot_of(n))
            if landings(slot_of(n), copied) % 2 != passed % 2:
                nxt = (at[0] + (w == 0), at[1] + (w == 1))
                yield (copied, done, nxt, checked | (1 << n if takes(w, n) else 0))

    stuck, seen, todo = [], set(), [(0, 0, (0, 0), 0)]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        after = list(moves(state))
        todo += after
        if not after and (state[1] < T or state[2] != (len(work[0]), len(work[1]))):
            stuck.append(state)
    return stuck


@pytest.mark.parametrize("slots", [4, 8])
def test_a_slot_belongs_to_one_warp(rule, slots):
    owner = {}
    for n in itertools.chain(range(100), range(2 ** 32 - 50, 2 ** 32)):
        s = rule.slot(ctypes.c_uint(n), slots)
        assert s < slots and s % 2 == 1
        assert owner.setdefault(s, rule.warp(ctypes.c_uint(n))) == rule.warp(ctypes.c_uint(n))
    assert set(owner.values()) == {0, 1}


@pytest.mark.parametrize("slots", [4, 8])
def test_no_order_gets_stuck(rule, slots):
    T = 2 * slots
    for mask in itertools.product((0, 1), repeat=8):
        masked = [mask[n % 8] for n in range(T)]
        mine = lambda w, n: rule.warp(n) == w  # noqa: E731
        assert not stuck_orders(masked, slots, mine, mine, lambda n: rule.slot(n, slots))


def test_the_model_finds_a_warp_that_falls_behind():
    """Tiles dealt out one by one, both warps waiting for each: with four slots the other warp's
    tile lets the slot be filled twice before this one has looked."""
    masked = [1] * 8
    slot = lambda n: (2 * n + 1) % 4  # noqa: E731
    both = lambda w, n: True  # noqa: E731
    assert stuck_orders(masked, 4, both, lambda w, n: n % 2 == w, slot)
