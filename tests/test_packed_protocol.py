"""A model of the packed forward kernel's per-CTA barrier protocol (csrc/packed_fwd.cu), run under
random schedules, in the manner of test_pipeline_protocol.py: the roles, waits, arrivals and parity
formulas of the kernel with the data reduced to labels.  It checks that every wait sees its barrier
at the awaited phase (blocks) or one past it (passes), that nothing deadlocks, that every read finds
the label it expects and every slot is written only after its last reader, and that the planted
mistakes are caught: one ring of an odd number of slots for K and V (a slot then has two waiters
that each miss the other's phases), no read barrier for the (max, sum) slots, and a Q tile reloaded
without waiting for the S products.

One lane quadrant is modelled: two softmax warps (a row's two threads) and one epilogue warp.
"""
import random

import pytest

from tests.test_pipeline_protocol import Bar, ProtocolError


class Packed:
    def __init__(self, items, stages, nb, rng, mistake=None):
        self.items, self.S, self.NB, self.rng, self.mistake = items, stages, nb, rng, mistake
        self.bars, self.res, self.readers = {}, {}, {}
        self.queue = {"s": [], "pv": []}  # MMAs of each issuer, in order
        self.loads = []                   # TMA loads in flight
        self.pair = [0, 0]                # arrivals at the softmax pair's barrier, per warp
        for name, count in (("Q", 1), ("QE", 1), ("OFULL", 1), ("OFREE", 1), ("ML0", 1), ("ML1", 1), ("MR0", 1), ("MR1", 1)):
            self.bars[name] = Bar(name, count)
        for k in range(nb):
            self.bars[f"S{k}"], self.bars[f"P{k}"], self.bars[f"PV{k}"] = Bar("S", 1), Bar("P", 2), Bar("PV", 1)
        for s in range(2 * stages + 1):
            for n in ("KF", "KE", "VF", "VE"):
                self.bars[f"{n}{s}"] = Bar(n, 1)

    # slots of tile j's K and V: (full, empty, phase)
    def k_slot(self, j):
        if self.mistake == "odd ring":
            e, n = 2 * j, 2 * self.S - 1
            return f"KF{e % n}", f"KE{e % n}", e // n
        return f"KF{j % self.S}", f"KE{j % self.S}", j // self.S

    def v_slot(self, j):
        if self.mistake == "odd ring":
            e, n = 2 * j + 1, 2 * self.S - 1
            return f"KF{e % n}", f"KE{e % n}", e // n
        return f"VF{j % self.S}", f"VE{j % self.S}", j // self.S

    def put(self, name, label):
        if self.readers.get(name, 0):
            raise ProtocolError(f"{name} written over while being read")
        self.res[name] = label

    def expect(self, name, label):
        if self.res.get(name) != label:
            raise ProtocolError(f"{name} holds {self.res.get(name)}, expected {label}")

    def tiles(self):
        jg = 0
        for k, n in enumerate(self.items):
            for j in range(n):
                yield k, j, jg
                jg += 1

    # ---- roles
    def load_k(self):
        for k, j, jg in self.tiles():
            if j == 0:
                if k > 0 and self.mistake != "no QE":
                    yield "wait", "QE", k - 1
                self.loads.append(("Qtile", ("Q", k), "Q"))
            full, empty, phase = self.k_slot(jg)
            if phase > 0:
                yield "wait", empty, phase - 1
            self.loads.append((full, ("K", jg), full))
            yield ("step",)

    def load_v(self):
        for _, _, jg in self.tiles():
            full, empty, phase = self.v_slot(jg)
            if phase > 0:
                yield "wait", empty, phase - 1
            self.loads.append((full, ("V", jg), full))
            yield ("step",)

    def s_issuer(self):
        for k, j, jg in self.tiles():
            if j == 0:
                yield "wait", "Q", k
            full, empty, phase = self.k_slot(jg)
            yield "wait", full, phase
            if jg >= self.NB:
                yield "wait", f"PV{jg % self.NB}", jg // self.NB - 1
            done = [f"S{jg % self.NB}", empty] + (["QE"] if j == self.items[k] - 1 else [])
            self.queue["s"].append(([("Qtile", ("Q", k)), (full, ("K", jg))], (f"buf{jg % self.NB}", ("S", jg)), done))
            yield ("step",)

    def pv_issuer(self):
        for k, j, jg in self.tiles():
            full, empty, phase = self.v_slot(jg)
            yield "wait", full, phase
            yield "wait", f"P{jg % self.NB}", jg // self.NB
            if j == 0 and k > 0:
                yield "wait", "OFREE", k - 1
            done = [f"PV{jg % self.NB}", empty] + (["OFULL"] if j == self.items[k] - 1 else [])
            need = [(full, ("V", jg)), (f"buf{jg % self.NB}", ("P", jg, 3))] + ([("O", (k, j))] if j else [])
            self.queue["pv"].append((need, ("O", (k, j + 1)), done))
            yield ("step",)

    def softmax(self, hf):
        jg = 0
        for k, n in enumerate(self.items):
            for j in range(n):
                b = f"buf{jg % self.NB}"
                yield "wait", f"S{jg % self.NB}", jg // self.NB
                if self.res.get(b) not in (("S", jg), ("P", jg, 1 << (1 - hf))):
                    raise ProtocolError(f"{b} holds {self.res.get(b)} for S({jg})")
                if j == n - 1:  # the last tile's zeros behind the sequence's last key
                    full, _, phase = self.v_slot(jg)
                    yield "wait", full, phase
                    self.expect(full, ("V", jg))
                yield "pair", hf  # no half row's sum has grown too large
                old = self.res[b]
                self.res[b] = ("P", jg, (old[2] if old[0] == "P" else 0) | 1 << hf)
                yield ("step",)
                if j > 0 and jg % 3 == 0:  # now and then the row is rescaled
                    yield "wait", f"PV{(jg - 1) % self.NB}", (jg - 1) // self.NB
                    self.expect("O", (k, j))
                yield "arrive", f"P{jg % self.NB}"
                jg += 1
            yield "pair", hf
            if hf == 0:
                if k > 1 and self.mistake != "no MR":
                    yield "wait", f"MR{k & 1}", (k >> 1) - 1
                self.put(f"ml{k & 1}", ("ml", k))
                yield "arrive", f"ML{k & 1}"
            yield "pair", hf

    def epilogue(self):
        for k, n in enumerate(self.items):
            yield "wait", f"ML{k & 1}", k >> 1
            yield "wait", "OFULL", k
            self.expect(f"ml{k & 1}", ("ml", k))
            self.expect("O", (k, n))
            yield ("step",)
            self.expect("O", (k, n))
            if k % 2:  # a whole item: the slot is free before O is read
                yield "arrive", f"MR{k & 1}"
            yield "arrive", "OFREE"
            yield ("step",)
            if not k % 2:  # a cut one: the slot serves as scratch until the parts are joined
                self.expect(f"ml{k & 1}", ("ml", k))
                yield "arrive", f"MR{k & 1}"

    # ---- scheduler
    def ready(self, req):
        if req[0] == "wait":
            bar, phase = self.bars[req[1]], req[2]
            # a parity wait passes when the barrier's current phase has the other parity
            passes = (bar.completed & 1) != (phase & 1)
            if passes and bar.completed < phase + 1:
                raise ProtocolError(f"{req[1]}: waiting for phase {phase} passes at {bar.completed}")
            if bar.completed > phase + 1:
                raise ProtocolError(f"{req[1]}: waiting for phase {phase}, already at {bar.completed}")
            return passes
        if req[0] == "pair":
            return self.pair[1 - req[1]] >= self.pair[req[1]]
        return True

    def run(self):
        roles = [self.load_k(), self.load_v(), self.s_issuer(), self.pv_issuer(), self.softmax(0), self.softmax(1), self.epilogue()]
        pending = {i: None for i in range(len(roles))}
        live = set(pending)

        def advance(i):
            try:
                pending[i] = next(roles[i])
                if pending[i][0] == "pair":
                    self.pair[pending[i][1]] += 1
            except StopIteration:
                live.discard(i)

        for i in list(live):
            advance(i)
        slow = self.rng.choice([*range(len(roles)), "load", "mma"])
        while live or self.loads or self.queue["s"] or self.queue["pv"]:
            acts = [("role", i) for i in live if self.ready(pending[i])]
            acts += [("load", i) for i in range(len(self.loads))]
            acts += [("mma", q) for q in self.queue if self.queue[q]]
            if not acts:
                raise ProtocolError("deadlock: " + ", ".join(str(pending[i]) for i in live))
            # one role (or the MMAs, or the loads) of the run lags behind wherever others can go on
            fast = [x for x in acts if x != ("role", slow) and x[0] != slow]
            what, i = self.rng.choice(fast if fast and self.rng.random() < 0.95 else acts)
            if what == "role":
                if pending[i][0] == "arrive":
                    self.bars[pending[i][1]].arrive()
                advance(i)
            elif what == "load":
                name, label, bar = self.loads.pop(i)
                self.put(name, label)
                self.bars[bar].arrive()
            else:
                need, (out, label), done = self.queue[i].pop(0)
                for name, want in need:
                    self.expect(name, want)
                self.res[out] = label
                for b in done:
                    self.bars[b].arrive()


# (stages, S buffers) of head dims 64, 128 and 256
CONFIGS = [(4, 3), (3, 3), (2, 2)]


@pytest.mark.parametrize("stages,nb", CONFIGS)
def test_protocol_is_sound(stages, nb):
    for seed in range(150):
        rng = random.Random(seed)
        items = [rng.choice([1, 1, 2, 3, 7]) for _ in range(rng.randrange(1, 9))]
        Packed(items, stages, nb, rng).run()


@pytest.mark.parametrize("mistake", ["odd ring", "no MR", "no QE"])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for seed in range(150):
        rng = random.Random(seed)
        items = [rng.choice([1, 1, 2, 3, 7]) for _ in range(8)]
        try:
            Packed(items, 3, 3, rng, mistake).run()
        except ProtocolError:
            caught += 1
    assert caught >= 10, caught
