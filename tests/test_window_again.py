"""Rows that the sliding-window kernel (csrc/attn_window.cu) computes again, on
the CPU: its roles with output warps that note items, and a taker that asks for
no more once one has; the lists' length holds, every item is done, and which keys
a step holds for a row that does not see them."""
import random

import pytest

from test_window_schedule import Item, Run, configurations

AGAIN = 4  # entries of an output warp's list


class Noting(Run):
    """Four output warps, each of which notes some items; items behind the last one posted are left."""

    def __init__(self, items, ring, notes):
        super().__init__(items, ring)
        self.notes = notes                  # [quarter] -> items (by object) to note
        self.lists = [[] for _ in range(4)]
        self.freed_o = [[0, 0] for _ in range(4)]
        self.end = None

    def next_items(self, who):
        self.read[who] = n = 0
        while True:
            yield lambda: self.posted > n
            self.read[who] = n + 1
            if self.end is not None and n >= self.end:
                return
            yield self.items[n]
            n += 1

    def taker(self):
        have, n = True, 0
        while True:
            yield lambda: n < 2 or all(r >= n - 1 for r in self.read.values())
            if not have:
                self.end = n
            self.posted = n + 1
            if not have:
                return
            yield lambda: self.want > n
            have = not any(self.lists) and n + 1 < len(self.items)
            n += 1

    def output(self, quarter):
        n = [0, 0]
        for x in self.each(f"output{quarter}"):
            if callable(x):
                yield x
                continue
            for i in range(2):
                if x[0].steps(i):
                    yield lambda: self.l[i] > n[i] and self.o_full[i] > n[i]
                    n[i] += 1
                    self.freed_o[quarter][i] += 1
                    self.o_free[i] = min(f[i] for f in self.freed_o)
            yield lambda: True              # the row is noted some time after O is free
            if id(x[0]) in self.notes[quarter]:
                self.lists[quarter].append(x[0])
                assert len(self.lists[quarter]) <= AGAIN

    def finish(self, rng):
        roles = {"producer": self.producer(), "mma0": self.mma(0), "mma1": self.mma(1), "softmax0": self.softmax(0),
                 "softmax1": self.softmax(1), **{f"output{q}": self.output(q) for q in range(4)}}
        waits = {r: next(g, None) for r, g in roles.items()}
        roles["taker"] = self.taker()
        waits["taker"] = next(roles["taker"])
        slow = rng.choice([None] + [r for r in roles])  # a role that runs only when no other can
        while any(w is not None for w in waits.values()):
            able = [r for r, w in waits.items() if w is not None and w()]
            if not able:
                return False
            r = rng.choice([x for x in able if x != slow] or able)
            waits[r] = next(roles[r], None)
        return True


@pytest.mark.parametrize("ring", [5, 8])
def test_the_lists_hold_every_note_and_every_item_is_done(ring):
    rng = random.Random(3)
    longest = 0
    for N, _, window, sinks in configurations(5, 120):
        lens = [rng.choice([N, rng.randint(0, N)]) for _ in range(rng.randint(1, 4))]
        todo = [Item(N, n, window, sinks, pair) for n in lens for pair in reversed(range((N + 255) // 256))]
        todo = [w for w in todo if w.nt > 0 or rng.random() < 0.5][:12]
        share = rng.choice([0.1, 1.0])
        notes = [{id(w) for w in todo if w.nt > 0 and rng.random() < share} for _ in range(4)]
        ctas = 0
        while todo:                         # a CTA that has stopped leaves the others to the next
            run = Noting(todo, ring, notes)
            assert run.finish(rng), (N, lens, window, sinks, ring)
            assert run.end >= 1
            done, todo = todo[:run.end], todo[run.end:]
            for q in range(4):
                assert [id(w) for w in run.lists[q]] == [id(w) for w in done if id(w) in notes[q]]
                longest = max(longest, len(run.lists[q]))
            ctas += 1
        assert ctas == 1 or any(notes)
    assert longest == AGAIN                 # no shorter list would do


def test_only_masked_steps_hold_keys_that_a_row_does_not_see():
    """The steps that are searched for bad values in V: of the others a tile's rows see every key."""
    for N, n, window, sinks in configurations(11, 200):
        for pair in range((N + 255) // 256):
            w = Item(N, n, window, sinks, pair)
            for i in range(2):
                p0 = w.q0 + 128 * i
                diagonal = 2 * (w.ns + p0 // 128 - w.t0)
                whole = 0
                if w.window > 0 and p0 + 128 > w.window:
                    whole = int((p0 + 128 - w.window - 128 * (w.t0 - w.ns) + 63) / 64)
                for u in w.steps(i):
                    if u >= diagonal or w.sinks // 64 <= u < whole:
                        continue
                    k0 = w.key0(u)
                    for p in (p0, min(p0 + 127, n - 1)):
                        for j in (k0, k0 + 63):
                            assert j <= p and (w.window == 0 or p - j < w.window or j < w.sinks)


# ---------------------------------------------------------------- the order of the items
def order(B, Hq, Hkv, N, D):
    """(head, first row) of each item, as the launch and win_item have them, and the heads of a group."""
    heads, pairs = B * Hq, -(-N // 256)
    groups = (heads * N * D * 4 // (Hq // Hkv) + (32 << 20) - 1) >> 25
    groups = min(max(groups, 1), heads)
    group = -(-heads // groups)
    out = []
    for idx in range(heads * pairs):
        g, at = divmod(idx, group * pairs)
        here = min(group, heads - g * group)
        pair, h = divmod(at, here)
        out.append((g * group + h, 256 * (pairs - 1 - pair)))
    return out, group


@pytest.mark.parametrize("B,Hq,Hkv,N,D", [(1, 11, 11, 8192, 128), (4, 32, 32, 4096, 128), (1, 32, 8, 8192, 128),
                                          (3, 7, 1, 20000, 64), (2, 5, 5, 100000, 128), (1, 1, 1, 1, 64),
                                          (1, 3, 3, 70000, 128), (7, 13, 13, 2500, 64)])
def test_every_item_comes_once_and_a_group_at_a_time(B, Hq, Hkv, N, D):
    items, group = order(B, Hq, Hkv, N, D)
    heads, pairs = B * Hq, -(-N // 256)
    assert sorted(items) == [(h, 256 * p) for h in range(heads) for p in range(pairs)]
    assert [h // group for h, _ in items] == sorted(h // group for h, _ in items)
    for g in range(-(-heads // group)):     # a group's heaviest rows first
        rows = [q0 for h, q0 in items if h // group == g]
        assert rows == sorted(rows, reverse=True)
