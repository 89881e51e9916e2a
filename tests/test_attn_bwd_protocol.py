"""Model check of the gradient kernel's barrier protocol (host only, no GPU).

The kernel (svg2_attn_bwd.cu) has two kinds of unit, both with two resident tiles and two streamed ones (T1: Q or K,
T2: dO or V) of three stages and one:

* producers fill T1(j), T2(j) into stage j % stages and arrive on t1_full / t2_full; they wait on t1_empty / t2_empty
  before they reuse a stage;
* the MMA thread issues S(j) = R1 T1(j)^T and dP(j) = R2 T2(j)^T, and the products that read P and dS from tensor
  memory in two chunks each: dV += P T2 (key unit) and dK or dQ += dS T1.  The tensor core runs them in issue order;
* eight warps read S, write P over it (key unit), read dP and write dS over it, chunk by chunk.

As in test_attn_protocol.py the agents are Python generators run under many seeded random interleavings; a parity wait
passes only while the awaited phase is complete and not overtaken, and at every read the model checks that the place
holds the tile the schedule intends.  The model restates the protocol, not the code."""
import random

import pytest

from tests.test_attn_protocol import Bar, ProtocolError, check

WARPS, PRODUCERS = 8, 3


class Unit:
    def __init__(self, T, key, rng, stages, one_s_slot=False):
        self.T, self.key, self.rng = T, key, rng
        self.slots = 1 if key or one_s_slot else 2  # S slots (one_s_slot: the planted fault of a query unit)
        two = lambda n: [Bar(n), Bar(n)]  # noqa: E731
        self.stages = stages
        self.t_full = [[Bar(PRODUCERS) for _ in range(n)] for n in stages]
        self.t_empty = [[Bar(1) for _ in range(n)] for n in stages]
        self.s_full, self.dp_full, self.o_full = two(1), Bar(1), Bar(1)
        self.p_full, self.ds_full = two(WARPS), two(WARPS)
        self.smem = [[[None] * PRODUCERS for _ in range(n)] for n in stages]  # [operand][stage][producer]
        self.s = [[None] * WARPS for _ in range(2)]     # what each warp finds in its part of an S slot
        self.dp = [None] * WARPS
        self.p = [[None, None] for _ in range(WARPS)]   # chunks of P and dS written
        self.ds = [[None, None] for _ in range(WARPS)]
        self.applied = {"dV": 0, "acc": 0}
        self.queue, self.copies = [], []

    def run_tc(self):
        op = self.queue.pop(0)
        if op[0] == "commit":
            op[1].arrive()
        elif op[0] in ("S", "dP"):
            kind, j = op
            o = 0 if kind == "S" else 1
            at = self.smem[o][j % self.stages[o]]
            check(all(x == j for x in at), f"{kind}({j}) read {at}")
            for w in range(WARPS):
                if kind == "S":
                    self.s[j % self.slots][w] = j
                    if self.key:
                        self.p[w] = [None, None]
                else:
                    self.dp[w], self.ds[w] = j, [None, None]
        else:
            kind, j, c = op  # dV reads P and T2, the other accumulator dS and T1
            o, src = (1, self.p) if kind == "dV" else (0, self.ds)
            at = self.smem[o][j % self.stages[o]]
            check(all(x == j for x in at), f"{kind}({j}) read {at}")
            check(all(x[c] == j for x in src), f"{kind}({j}) chunk {c} read {src}")
            check(self.applied[kind] == 2 * j + c, f"{kind}({j}) chunk {c} out of order")
            self.applied[kind] += 1

    def run_copy(self):
        o, st, w, j = self.copies.pop(self.rng.randrange(len(self.copies)))
        self.smem[o][st][w] = j
        self.t_full[o][st].arrive()

    def wait(self, bar, phase):
        return lambda: bar.done(phase & 1)

    def producer(self, w):
        for j in range(self.T):
            for o in range(2):
                st, fill = j % self.stages[o], j // self.stages[o]
                if fill:
                    yield self.wait(self.t_empty[o][st], fill - 1)
                self.smem[o][st][w] = "landing"
                self.copies.append((o, st, w, j))
                yield None

    def mma(self):
        q, T, key = self.queue, self.T, self.key
        commit = lambda b: q.append(("commit", b))  # noqa: E731
        if T == 0:
            return
        S1, S2 = self.stages
        yield self.wait(self.t_full[0][0], 0)
        q.append(("S", 0))
        commit(self.s_full[0])
        yield self.wait(self.t_full[1][0], 0)
        q.append(("dP", 0))
        commit(self.dp_full)
        if not key:
            commit(self.t_empty[1][0])
        for j in range(T):
            more = j + 1 < T
            if key:
                for c in range(2):
                    yield self.wait(self.p_full[c], j)
                    q.append(("dV", j, c))
                commit(self.t_empty[1][j % S2])
            if more:
                yield self.wait(self.t_full[0][(j + 1) % S1], (j + 1) // S1)
                q.append(("S", j + 1))
                commit(self.s_full[0 if key else (j + 1) & 1])
            for c in range(2):
                yield self.wait(self.ds_full[c], j)
                q.append(("acc", j, c))
            commit(self.t_empty[0][j % S1])
            if more:
                yield self.wait(self.t_full[1][(j + 1) % S2], (j + 1) // S2)
                q.append(("dP", j + 1))
                commit(self.dp_full)
                if not key:
                    commit(self.t_empty[1][(j + 1) % S2])
        commit(self.o_full)

    def softmax(self, w):
        for j in range(self.T):
            yield self.wait(self.s_full[0], j) if self.key else self.wait(self.s_full[j & 1], j >> 1)
            for c in range(2):
                check(self.s[j % self.slots][w] == j, f"warp {w} read S {self.s[j % self.slots][w]} for tile {j}")
                yield None
                if self.key:
                    self.p[w][c] = j
                    self.p_full[c].arrive()
                    yield None
            yield self.wait(self.dp_full, j)
            for c in range(2):
                check(self.dp[w] == j, f"warp {w} read dP {self.dp[w]} for tile {j}")
                self.ds[w][c] = j
                yield None
                self.ds_full[c].arrive()
                yield None
        if self.T > 0:
            yield self.wait(self.o_full, 0)
            check(self.applied["acc"] == 2 * self.T, f"epilogue saw {self.applied}")
            check(not self.key or self.applied["dV"] == 2 * self.T, f"epilogue saw {self.applied}")


def run_schedule(T, key, seed, stages, **kw):
    rng = random.Random(seed)
    k = Unit(T, key, rng, stages, **kw)
    agents = {f"producer{w}": k.producer(w) for w in range(PRODUCERS)}
    agents["mma"] = k.mma()
    agents.update({f"softmax{w}": k.softmax(w) for w in range(WARPS)})
    waiting = {n: None for n in agents}
    for _ in range(100000):
        runnable = [n for n in agents if waiting[n] is None or waiting[n]()]
        runnable += ["tc"] * bool(k.queue) + ["copy"] * bool(k.copies)
        if not runnable:
            if agents:
                raise ProtocolError(f"deadlock: {sorted(agents)} wait forever")
            return
        n = rng.choice(runnable)
        if n == "tc":
            k.run_tc()
        elif n == "copy":
            k.run_copy()
        else:
            try:
                waiting[n] = next(agents[n])
            except StopIteration:
                del agents[n], waiting[n]
    raise ProtocolError("schedule did not finish")


@pytest.mark.parametrize("key,stages", [(True, (3, 1)), (False, (3, 1)), (True, (2, 2)), (False, (2, 2))])
@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 5, 9])
def test_protocol_has_no_deadlock_or_hazard(T, key, stages):
    for seed in range(120):
        run_schedule(T, key, seed, stages)


def test_the_model_sees_a_query_unit_without_its_second_s_slot():
    """S(j+1) is issued before dS(j) is handed over: in one slot it would overwrite an S(j) still being read."""
    hazards = 0
    for seed in range(200):
        try:
            run_schedule(4, False, seed, (3, 1), one_s_slot=True)
        except ProtocolError as e:
            hazards += "read S" in str(e)
    assert hazards > 0
