"""The schedule of the sliding-window kernel (csrc/attn_window.cu) on the CPU: the
items and steps as the kernel computes them cover every visible key once and no
unmasked step holds a hidden one; and its roles (taker, TMA producer, two MMA
issuers, two softmax warpgroups, output), run as coroutines that block where the
kernel waits, always finish, whatever the lengths, windows and sinks are."""
import random

import numpy as np
import pytest

STEP = 64


class Item:
    """win_item and WinSteps of one (head, pair of row tiles)."""

    def __init__(self, N, n, window, sinks, pair):
        if window >= N or sinks >= N:
            window = 0
        if window == 0:
            sinks = 0
        self.n, self.window, self.sinks, self.q0 = n, window, sinks, 256 * pair
        lead = self.q0 - window + 1
        self.t0 = lead // 128 if window > 0 and lead > 0 else 0
        if sinks > 128 * self.t0:
            self.t0 = 0
        self.ns = -(-sinks // 128) if self.t0 > 0 else 0
        self.nt = 0 if self.q0 >= n else self.ns + self.q0 // 128 - self.t0 + (2 if self.q0 + 128 < n else 1)
        self.narrow = self.ns - 1 if self.ns > 0 and sinks - 128 * (self.ns - 1) <= STEP else -1

    def steps(self, i):
        """(first, steps in order) of row tile i, as halves of key tiles."""
        q0 = self.q0 + 128 * i
        lead = q0 - self.window + 1
        tile = lead // 128 if self.t0 > 0 and lead > 0 else 0
        lo = 2 * (self.ns + tile - self.t0) + (1 if self.t0 > 0 and lead - 128 * tile >= STEP else 0)
        sink = -(-self.sinks // STEP) if self.ns > 0 else -1
        if q0 >= self.n:
            return []
        end = 2 * (self.ns + q0 // 128 - self.t0) + (1 if self.n - q0 <= STEP else 2)
        u, out = (0 if self.ns > 0 else lo), []
        while u != end:
            out.append(u)
            assert len(out) < 10000 and 0 <= u < 2 * self.nt
            u = lo if u + 1 == sink else u + 1
        return out

    def key0(self, u):
        return STEP * u + (128 * (self.t0 - self.ns) if u >= 2 * self.ns else 0)


def configurations(seed, count):
    rng = random.Random(seed)
    for _ in range(count):
        N = rng.choice([rng.randint(1, 300), rng.randint(200, 1500)])
        n = rng.choice([N, rng.randint(0, N)])
        window = rng.choice([0, 1, rng.randint(1, N), rng.randint(1, 200)])
        sinks = rng.choice([0, 0, rng.randint(0, 20), rng.randint(0, 300), 64, 65, 128, 129])
        yield N, n, window, sinks


def test_steps_cover_the_visible_keys_once():
    for N, n, window, sinks in configurations(0, 400):
        for pair in range((N + 255) // 256):
            w = Item(N, n, window, sinks, pair)
            for i in range(2):
                p0 = w.q0 + 128 * i
                p = np.arange(p0, min(p0 + 128, n))
                seen = np.zeros((len(p), N + 256), dtype=int)
                for u in w.steps(i):
                    k0 = w.key0(u)
                    j = np.arange(k0, k0 + STEP)
                    visible = (j <= p[:, None]) & ((window == 0) | (p[:, None] - j < window) | (j < sinks))
                    masked = k0 + STEP - 1 > p0 or (w.window > 0 and p0 + 128 - w.window > k0 and w.sinks - k0 < STEP)
                    # as the kernel has it, by the step's number
                    diagonal = 2 * (w.ns + p0 // 128 - w.t0)
                    whole = 0
                    if w.window > 0 and p0 + 128 > w.window:
                        whole = int((p0 + 128 - w.window - 128 * (w.t0 - w.ns) + STEP - 1) / STEP)
                    assert masked == (u >= diagonal or w.sinks // STEP <= u < whole)
                    assert masked or visible.all(), (N, n, window, sinks, pair, i, u)
                    # a narrow tile holds its first 64 keys alone
                    assert u >> 1 != w.narrow or u & 1 == 0
                    seen[:, k0:k0 + STEP] += visible
                j = np.arange(N + 256)
                want = (j <= p[:, None]) & ((window == 0) | (p[:, None] - j < window) | (j < sinks))
                assert (seen == want).all(), (N, n, window, sinks, pair, i)


class Run:
    """The roles over a list of items; `ring` slots of K and V."""

    def __init__(self, items, ring):
        self.items, self.R = items, ring
        self.full = 0                       # ring slots filled, in order
        self.freed = [set(), set()]         # slots that each row tile released
        self.q_full, self.q_last = [0, 0], [0, 0]
        self.s, self.p, self.l, self.o_full, self.o_free = [0, 0], [0, 0], [0, 0], [0, 0], [0, 0]
        self.posted, self.want = 0, 0
        self.read = {}                      # reader -> items read

    def may_fill(self, x):
        return x < self.R or all(x - self.R in f for f in self.freed)

    def next_items(self, who):
        self.read[who] = 0
        for n in range(len(self.items) + 1):
            yield lambda: self.posted > n
            self.read[who] = n + 1
            if n < len(self.items):
                yield self.items[n]

    def taker(self):
        for n in range(len(self.items) + 1):
            yield lambda: n < 2 or all(r >= n - 1 for r in self.read.values())
            self.posted = n + 1
            if n < len(self.items):
                yield lambda: self.want > n

    def each(self, who):
        """The items as they can be read: yields conditions, then (item,) tuples."""
        for x in self.next_items(who):
            yield x if callable(x) else (x,)

    def producer(self):
        nq = [0, 0]
        for x in self.each("producer"):
            if callable(x):
                yield x
                continue
            w, = x
            if w.nt == 0:
                self.want += 1
            for j in range(w.nt):
                if j == max(0, w.nt - 4):
                    self.want += 1
                for half in range(2):
                    yield lambda: self.may_fill(self.full)
                    self.full += 1
                    if j == 0 and half == 0:
                        for i in range(2):
                            if w.steps(i):
                                yield lambda: self.q_last[i] >= nq[i]
                                nq[i] += 1
                                self.q_full[i] += 1

    def mma(self, i):
        base = s_qk = s_pv = n_items = 0
        for x in self.each(f"mma{i}"):
            if callable(x):
                yield x
                continue
            w, = x
            steps = w.steps(i)
            at = [0, 0]                     # key tile of K, of V

            def skip(kind, to):
                while at[kind] < to:
                    slot = 2 * (base + at[kind]) + kind
                    yield lambda: self.full > slot
                    self.freed[i].add(slot)
                    at[kind] += 1

            def ready(kind):
                yield lambda: self.full > 2 * (base + at[kind]) + kind

            def done(k):                    # with step k's key tile
                return k + 1 == len(steps) or steps[k + 1] >> 1 != steps[k] >> 1

            def release(kind, k):
                if done(k):
                    self.freed[i].add(2 * (base + at[kind]) + kind)

            def leave(kind, k):
                if done(k):
                    at[kind] += 1
                    yield from skip(kind, w.nt if k + 1 == len(steps) else steps[k + 1] >> 1)

            if not steps:
                for j in range(1, w.nt + 1):
                    yield from skip(0, j)
                    yield from skip(1, j)
                base += w.nt
                continue
            yield from skip(0, steps[0] >> 1)
            yield from skip(1, steps[0] >> 1)
            yield lambda: self.q_full[i] > n_items
            c = 0

            def qk():
                nonlocal c, s_qk
                yield from ready(0)
                assert at[0] == steps[c] >> 1
                s_qk += 1
                self.s[i] += 1
                release(0, c)
                if c + 1 == len(steps):
                    self.q_last[i] += 1
                c += 1
                yield from leave(0, c - 1)

            while c < min(2, len(steps)):
                yield from qk()
            yield lambda: self.o_free[i] >= n_items
            for d in range(len(steps)):
                yield from ready(1)
                assert at[1] == steps[d] >> 1
                yield lambda: self.p[i] > s_pv
                release(1, d)
                if d + 1 == len(steps):
                    self.o_full[i] += 1
                if c < len(steps):
                    yield from qk()
                s_pv += 1
                assert s_qk <= s_pv + 2
                yield from leave(1, d)
            n_items += 1
            base += w.nt

    def softmax(self, i):
        step = n = 0
        for x in self.each(f"softmax{i}"):
            if callable(x):
                yield x
                continue
            steps = x[0].steps(i)
            if not steps:
                continue
            for _ in steps:
                yield lambda: self.s[i] > step
                step += 1
                self.p[i] += 1
            yield lambda: self.o_free[i] >= n
            self.l[i] += 1
            n += 1

    def output(self):
        n = [0, 0]
        for x in self.each("output"):
            if callable(x):
                yield x
                continue
            for i in range(2):
                if x[0].steps(i):
                    yield lambda: self.l[i] > n[i] and self.o_full[i] > n[i]
                    n[i] += 1
                    self.o_free[i] += 1

    def finish(self, rng):
        roles = {"producer": self.producer(), "mma0": self.mma(0), "mma1": self.mma(1), "softmax0": self.softmax(0),
                 "softmax1": self.softmax(1), "output": self.output()}
        waits = {r: next(g, None) for r, g in roles.items()}
        roles["taker"] = self.taker()
        waits["taker"] = next(roles["taker"])
        while any(w is not None for w in waits.values()):
            able = [r for r, w in waits.items() if w is not None and w()]
            if not able:
                return False
            r = rng.choice(able)
            waits[r] = next(roles[r], None)
        return True


@pytest.mark.parametrize("ring", [5, 8])
def test_the_roles_always_finish(ring):
    rng = random.Random(7)
    for N, _, window, sinks in configurations(1, 250):
        lens = [rng.choice([N, 0, rng.randint(0, N)]) for _ in range(rng.randint(1, 3))]
        items = [Item(N, n, window, sinks, pair) for n in lens for pair in reversed(range((N + 255) // 256))]
        if rng.random() < 0.5:              # items without rows are passed over unless their rows are zeroed
            items = [w for w in items if w.nt > 0]
        rng.shuffle(items)
        assert Run(items[:8], ring).finish(rng), (N, lens, window, sinks, ring)


def test_a_row_tile_that_released_every_k_before_its_v_would_not_finish():
    """The model sees a schedule that waits for itself: an item of four key tiles, in the ring of five slots,
    whose second row tile is empty and releases all of K before any V."""
    class Bad(Run):
        def mma(self, i):
            if i == 0:
                yield from super().mma(0)
                return
            for x in self.each("mma1"):
                if callable(x):
                    yield x
                    continue
                for kind in range(2):
                    for j in range(x[0].nt):
                        yield lambda: self.full > 2 * j + kind
                        self.freed[1].add(2 * j + kind)

    item = Item(577, 577, 383, 0, 2)
    assert item.nt == 4 and not item.steps(1)
    assert not Bad([item], 5).finish(random.Random(0))
    assert Run([item], 5).finish(random.Random(0))
