"""The pipeline of the tree kernel for many query rows, on the host, in every order its roles may run.

The kernel's warps meet at barriers that complete one phase after another; a wait names a
phase by its parity alone, so it is right only while the barrier is at most one phase past
the one that is waited for. A GPU run meets one order of the roles, that in which V tiles
come early; here the roles are run as small programs against barriers of that kind, the
order drawn at random with one role held back as long as any other can go on, and every
buffer remembers which tile it holds. Which barrier a tile's scores and weights use, and its
phase, are the kernel's own (ring_attn_debug_tree_barriers).

A run must end (no order leaves every role waiting) and each product must meet its own
tile's queries, weights and values. The rule with two weight barriers for three score
buffers must fail here: the check has teeth.
"""
import random

import pytest

from sequence_exact_attention_ring_b200 import binding as B

GROUPS = 2  # row groups (a softmax warp of each set per group)


@pytest.fixture(scope="module")
def lib():
    from sequence_exact_attention_ring_b200 import build
    build.build()
    return B.load()


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):  # the phase of this parity has completed
        return self.phase % 2 != parity


class Stuck(Exception):
    pass


class Kernel:
    """One CTA over `parts` (tile counts). Roles are generators that yield a condition to wait for."""

    def __init__(self, fmt, D, parts, moves, weights=None):
        self.parts, self.moves, self.mx = parts, moves, fmt != B.CACHE_BF16
        self.rule = lambda t: B.ring_attn_debug_tree_barriers(fmt, D, t)
        self.weights = weights or (lambda t: self.rule(t)[4:6])
        self.bufs, self.raw = self.rule(0)[:2]
        n = lambda k, c: [Bar(c) for _ in range(k)]
        self.k_full, self.v_full, self.k_free, self.v_free = (n(2, 1) for _ in range(4))
        self.s_full, self.p_ready = n(self.bufs, 1), n(max(self.bufs, 2), GROUPS)
        self.q_ready, self.o_done = Bar(2 * GROUPS), Bar(1)
        self.pair, self.maxima = n(GROUPS, 2), [n(2, 1) for _ in range(GROUPS)]
        self.raw_full, self.raw_free = n(self.raw, 1), n(self.raw, 2)
        self.raw_seen = [n(self.raw, 1), n(self.raw, 1)]
        self.k_tile, self.v_tile, self.raw_tile = [None] * 2, [None] * 2, [None] * self.raw
        self.scores = [None] * self.bufs                     # tile whose scores a buffer holds
        self.p = [[None] * GROUPS for _ in range(self.bufs)]  # tile whose weights it holds
        self.o = [[] for _ in range(GROUPS)]                 # tiles that O holds
        self.s_m = [[None, None] for _ in range(GROUPS)]
        self.pipe = []                                       # products and commits, in order
        self.results = []
        self.tiles = sum(parts)

    # -------------------------------------------------------------- roles
    def issuer(self):
        t0 = 0
        for part, count in enumerate(self.parts):
            def issue_s(t):
                yield lambda: self.k_full[t & 1].done(t >> 1 & 1)
                self.pipe.append(lambda: self.product_s(t))
                bar = self.s_full[self.rule(t)[2]]
                self.pipe.append(bar.arrive)
                self.pipe.append(self.k_free[t & 1].arrive)
            yield lambda: self.q_ready.done(part & 1)
            for n in range(min(self.bufs, count)):
                yield from issue_s(t0 + n)
            for n in range(count):
                t = t0 + n
                yield lambda: self.v_full[t & 1].done(t >> 1 & 1)
                at, phase = self.weights(t)
                yield lambda: self.p_ready[at].done(phase)
                self.pipe.append(lambda t=t, first=n == 0: self.product_o(t, first))
                self.pipe.append(self.v_free[t & 1].arrive)
                if n + 1 == count:
                    self.pipe.append(self.o_done.arrive)
                if n + self.bufs < count:
                    yield from issue_s(t + self.bufs)
            t0 += count

    def product_s(self, t):
        assert self.k_tile[t & 1] == t, f"scores of tile {t} from K of {self.k_tile[t & 1]}"
        buf = t % self.bufs
        self.scores[buf], self.p[buf] = t, [None] * GROUPS

    def product_o(self, t, first):
        assert self.v_tile[t & 1] == t, f"tile {t} with V of {self.v_tile[t & 1]}"
        assert self.p[t % self.bufs] == [t] * GROUPS, f"tile {t} with weights of {self.p[t % self.bufs]}"
        for g in range(GROUPS):
            self.o[g] = [t] if first else self.o[g] + [t]

    def tensor_pipe(self):
        done = 0
        total = sum(5 * n for n in self.parts) + len(self.parts)  # two products and three commits a tile, one a part
        while done < total:
            yield lambda: bool(self.pipe)
            self.pipe.pop(0)()
            done += 1

    def fetch(self):
        for t in range(self.tiles):
            yield lambda: self.raw_free[t % self.raw].done((t // self.raw & 1) ^ 1)
            self.raw_tile[t % self.raw] = t
            self.raw_full[t % self.raw].arrive()

    def look(self, kv):
        for t in range(self.tiles):
            yield lambda: self.raw_full[t % self.raw].done(t // self.raw & 1)
            assert self.raw_tile[t % self.raw] == t
            self.raw_seen[kv][t % self.raw].arrive()

    def fill(self, kv):
        tile = self.v_tile if kv else self.k_tile
        full, free = (self.v_full, self.v_free) if kv else (self.k_full, self.k_free)
        for t in range(self.tiles):
            if self.mx:
                slot, phase = t % self.raw, t // self.raw & 1
                yield lambda: self.raw_seen[0][slot].done(phase)
                yield lambda: self.raw_seen[1][slot].done(phase)
                yield lambda: self.raw_full[slot].done(phase)
            yield lambda: free[t & 1].done((t >> 1 & 1) ^ 1)
            tile[t & 1] = t
            if self.mx:
                assert self.raw_tile[slot] == t
                full[t & 1].arrive()
                self.raw_free[slot].arrive()
            elif t > 0:  # reported once the next tile's copies are under way
                full[(t - 1) & 1].arrive()
        if not self.mx:
            full[(self.tiles - 1) & 1].arrive()

    def softmax(self, g, hh):
        t0 = 0
        for part, count in enumerate(self.parts):
            self.q_ready.arrive()
            self.pair[g].arrive()
            yield lambda: self.pair[g].done(0)
            for n in range(count):
                t = t0 + n
                if t & 1 != hh:
                    continue
                buf = t % self.bufs
                at, phase = self.rule(t)[2:4]
                yield lambda: self.s_full[at].done(phase)
                assert self.scores[buf] == t, f"tile {t} reads scores of {self.scores[buf]}"
                yield lambda: True
                if n > 0:
                    yield lambda: self.maxima[g][hh ^ 1].done((t - 1) >> 1 & 1)
                    assert self.s_m[g][hh ^ 1] == t - 1
                self.s_m[g][hh] = t
                self.maxima[g][hh].arrive()
                yield lambda: True
                assert self.scores[buf] == t
                self.p[buf][g] = t
                if n > 0 and self.moves(t):
                    yield lambda: self.v_free[(t - 1) & 1].done((t - 1) >> 1 & 1)
                    assert self.o[g] == list(range(t0, t)), f"tile {t} rescales O of {self.o[g]}"
                self.p_ready[self.weights(t)[0]].arrive()
            self.pair[g].arrive()
            yield lambda: self.pair[g].done(1)
            yield lambda: self.o_done.done(part & 1)
            assert self.o[g] == list(range(t0, t0 + count))
            self.results.append((part, g, hh))
            t0 += count

    # ---------------------------------------------------------- execution
    def run(self, rng, slow):
        roles = {"issuer": self.issuer(), "pipe": self.tensor_pipe(), "fill K": self.fill(0), "fill V": self.fill(1)}
        if self.mx:
            roles.update({"fetch": self.fetch(), "look K": self.look(0), "look V": self.look(1)})
        roles.update({f"softmax {g} {hh}": self.softmax(g, hh) for g in range(GROUPS) for hh in range(2)})
        waits = {name: next(role, None) for name, role in roles.items()}
        while any(w is not None for w in waits.values()):
            ready = [name for name, w in waits.items() if w is not None and w()]
            if not ready:
                raise Stuck(sorted(name for name, w in waits.items() if w is not None))
            name = rng.choice([x for x in ready if not x.startswith(slow)] or ready)
            waits[name] = next(roles[name], None)
        assert len(self.results) == 2 * GROUPS * len(self.parts)


FORMS = [(f, D) for f in (B.CACHE_BF16, B.CACHE_MXFP8, B.CACHE_MXFP4) for D in (64, 128)]
SLOW = ["fill V", "fill K", "fetch", "look V", "issuer", "pipe", "softmax 0", "softmax 1 1", "none"]


@pytest.mark.parametrize("slow", SLOW)
@pytest.mark.parametrize("fmt,D", FORMS)
def test_every_order_ends_with_every_tile_in_its_place(lib, fmt, D, slow):
    for seed in range(6):
        rng = random.Random(seed)
        parts = [rng.randrange(1, 14) for _ in range(4)]
        moves = (lambda t: False, lambda t: True, lambda t: (t * 7 + seed) % 3 == 0)[seed % 3]
        Kernel(fmt, D, parts, moves).run(rng, slow)


@pytest.mark.parametrize("fmt", [B.CACHE_BF16, B.CACHE_MXFP8, B.CACHE_MXFP4])
def test_two_weight_barriers_for_three_score_buffers_get_stuck(lib, fmt):
    with pytest.raises(Stuck):
        for seed in range(20):
            Kernel(fmt, 64, [9, 8], lambda t: False, lambda t: (t & 1, t >> 1 & 1)).run(random.Random(seed), "fill V")


def test_scores_and_weights_use_a_barrier_per_buffer(lib):
    for fmt, D in FORMS:
        bufs = B.ring_attn_debug_tree_barriers(fmt, D, 0)[0]
        for t in range(3 * bufs):
            _, _, s_at, s_phase, p_at, p_phase = B.ring_attn_debug_tree_barriers(fmt, D, t)
            assert (s_at, s_phase) == (p_at, p_phase) == (t % bufs, t // bufs % 2)


def test_refusals(lib):
    for args in ((3, 64, 0), (-1, 64, 0), (B.CACHE_BF16, 64, -1), (B.CACHE_BF16, 96, 0)):
        with pytest.raises(B.RingAttnError):
            B.ring_attn_debug_tree_barriers(*args)
