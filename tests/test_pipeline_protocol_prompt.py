"""Race detection for the barrier protocol of the paged prompts kernel, whose CTAs
run tile after tile (CPU, a model of the protocol, not of the arithmetic); the
barrier model and the checks are those of the prefill protocol test.

Roles of one CTA: the key producer (also finds the tiles and loads their queries),
the value producer, two Q.K^T issuers (even and odd blocks), the P.V issuer, and
per quarter of the rows a decider and an exponential warp (two quarters here; a
tile may fill one).  Rings run on from tile to tile: block g is the CTA's g-th.
"""
import random

import pytest

from tests.test_pipeline_protocol import Bar, ProtocolError

NQ, NR, NS, NV, NDEC = 2, 4, 3, 2, 4


def simulate_prompt(tiles, seed, PK=3, o_wait=True, q_wait=True, key_slot_of_tile=True,
                    dense_read=True):
    """tiles: (keep, rescale, dense, quarters with rows).  Raises ProtocolError."""
    rng = random.Random(seed)
    B = {}

    def bar(name, count=1):
        B[name] = Bar(name, count)

    for i in range(2):
        bar(("tile_full", i)), bar(("tile_empty", i), 4 + 2 * NQ)
        bar(("q_full", i)), bar(("l_full", i), NQ)
    for i in range(NR):
        bar(("ready", i), 2), bar(("qk_done", i))
    for i in range(NV):
        bar(("v_full", i)), bar(("v_empty", i))
    for i in range(NS):
        bar(("p_full", i), NQ), bar(("pv_done", i))
        B[("ready", i)].arrive()  # S buffers free at first
    for i in range(NDEC):
        bar(("dec_full", i)), bar(("dec_read", i), 2 + NQ)

    slot, qst, kst, vst = [None] * 2, [None] * 2, [None] * PK, [None] * NV
    sbuf, dec = [None] * NS, [None] * NDEC
    sums = [None] * NQ
    o_tile, o_count, left = [None], [0], [0] * len(tiles)  # left: warps whose epilogue is over
    votes, meets = {}, {}
    pipe, tma = [], []
    active = [2 * t[3] for t in tiles]

    def wait(name, phase):
        if name == "until":
            return phase()
        b = B[name]
        ok = (b.n % 2) != (phase % 2)
        if ok and b.n <= phase:
            raise ProtocolError(f"{name}: wait for phase {phase} passed after {b.n} phases")
        if not ok and b.n > phase:
            raise ProtocolError(f"{name}: phase {phase} completed but the parity wait blocks")
        return ok

    def expect(cond, msg):
        if not cond:
            raise ProtocolError(msg)

    def load(store, i, value, name):
        store[i] = None
        B[name].arrive(tx=1)

        def land():
            store[i] = value
            B[name].complete_tx(1)
        tma.append(land)

    def keys():
        g = 0
        for it, (keep, _, _, _) in enumerate(tiles):
            s = it & 1
            if it >= 2 and q_wait:
                yield ("wait", ("tile_empty", s), (it >> 1) - 1)
            expect(it < 2 or left[it - 2] == active[it - 2],
                   f"queries of tile {it} overwrite those of {it - 2} under its epilogue")
            slot[s] = it
            B[("tile_full", s)].arrive()
            load(qst, s, it, ("q_full", s))
            yield None
            for _ in keep:
                if g >= PK:
                    f = g - PK if key_slot_of_tile else g - NR
                    if f >= 0:
                        yield ("wait", ("qk_done", f % NR), f // NR)
                load(kst, g % PK, g, ("ready", g % NR))
                g += 1
                yield None
        it = len(tiles)
        if it >= 2:
            yield ("wait", ("tile_empty", it & 1), (it >> 1) - 1)
        slot[it & 1] = "end"
        B[("tile_full", it & 1)].arrive()

    def tiles_of():
        """(it, first block of the tile, the tile), after its set-up is there."""
        g = 0
        for it, t in enumerate(tiles):
            yield it, g, t
            g += len(t[0])

    def read_dec(g):
        d = dec[g % NDEC]
        expect(d is not None and d[0] == g, f"decision slot {g % NDEC} holds {d}, not block {g}")
        B[("dec_read", g % NDEC)].arrive()
        return d[1]

    def enter(it):
        expect(slot[it & 1] == it, f"tile slot {it & 1} holds {slot[it & 1]}, not {it}")

    def values():
        vi = 0
        for it, g0, (keep, _, dense, _) in tiles_of():
            yield ("wait", ("tile_full", it & 1), it >> 1)
            enter(it)
            for g in range(g0, g0 + len(keep)):
                if not dense:
                    yield ("wait", ("dec_full", g % NDEC), g // NDEC)
                    if not read_dec(g):
                        continue
                if vi >= NV:
                    yield ("wait", ("v_empty", vi % NV), vi // NV - 1)
                load(vst, vi % NV, g, ("v_full", vi % NV))
                vi += 1
                yield None
            B[("tile_empty", it & 1)].arrive()

    def scores(mine):
        for it, g0, (keep, _, _, _) in tiles_of():
            yield ("wait", ("tile_full", it & 1), it >> 1)
            enter(it)
            yield ("wait", ("q_full", it & 1), it >> 1)
            for g in range(g0, g0 + len(keep)):
                if g % 2 != mine:
                    continue
                yield ("wait", ("ready", g % NR), g // NR)
                expect(sbuf[g % NS] is None, f"Q.K^T of block {g} overwrites S: {sbuf[g % NS]}")
                sbuf[g % NS] = ("writing", g)

                def done(g=g, it=it):
                    expect(kst[g % PK] == g, f"Q.K^T of block {g} read key tile {kst[g % PK]}")
                    expect(qst[it & 1] == it, f"Q.K^T of tile {it} read queries {qst[it & 1]}")
                    sbuf[g % NS] = g
                    B[("qk_done", g % NR)].arrive()
                pipe.append(done)
                yield None
            B[("tile_empty", it & 1)].arrive()

    def pv():
        kc = 0
        for it, g0, (keep, _, _, _) in tiles_of():
            yield ("wait", ("tile_full", it & 1), it >> 1)
            enter(it)
            first = True
            for g in range(g0, g0 + len(keep)):
                yield ("wait", ("dec_full", g % NDEC), g // NDEC)
                if not read_dec(g):
                    continue
                if first and it and o_wait:
                    yield ("wait", ("tile_empty", (it - 1) & 1), (it - 1) >> 1)
                yield ("wait", ("p_full", kc % NS), kc // NS)
                yield ("wait", ("v_full", kc % NV), kc // NV)
                expect(not first or it == 0 or left[it - 1] == active[it - 1],
                       f"P.V of tile {it} overwrites O under the epilogue of {it - 1}")
                expect(sbuf[g % NS] == g and vst[kc % NV] == g, f"P.V of block {g}: operands")
                if first:
                    o_tile[0], o_count[0] = it, 0

                def done(g=g, kc=kc):
                    expect(vst[kc % NV] == g, f"P.V of block {g} read values {vst[kc % NV]}")
                    sbuf[g % NS] = None
                    o_count[0] += 1
                    B[("v_empty", kc % NV)].arrive()
                    B[("ready", (g + NS) % NR)].arrive()
                    B[("pv_done", kc % NS)].arrive()
                pipe.append(done)
                kc += 1
                first = False
                yield None
            B[("tile_empty", it & 1)].arrive()

    def epilogue(it, q, keep):
        expect(sums[q] == it, f"row sums of tile {sums[q]}, not {it}")
        n = sum(keep)
        expect(n == 0 or (o_tile[0] == it and o_count[0] == n), f"epilogue of tile {it} reads O early")
        left[it] += 1
        B[("tile_empty", it & 1)].arrive()

    def decider(q):
        for it, g0, (keep, _, dense, nq) in tiles_of():
            yield ("wait", ("tile_full", it & 1), it >> 1)
            meets[it] = meets.get(it, 0) + 1
            yield ("wait", "until", lambda it=it: meets[it] == NQ)
            enter(it)
            if q >= nq:
                B[("tile_empty", it & 1)].arrive()
                continue
            for c, k in enumerate(keep):
                g = g0 + c
                yield ("wait", ("qk_done", g % NR), g // NR)
                expect(sbuf[g % NS] == g, f"decider reads S {sbuf[g % NS]} for block {g}")
                votes[g] = votes.get(g, 0) + 1
                yield ("wait", "until", lambda g=g, nq=nq: votes[g] == nq)
                if q != (c % NQ if nq == NQ else 0):
                    continue
                if not k:
                    sbuf[g % NS] = None
                    B[("ready", (g + NS) % NR)].arrive()
                if g >= NDEC:
                    yield ("wait", ("dec_read", g % NDEC), g // NDEC - 1)
                dec[g % NDEC] = (g, k)
                B[("dec_full", g % NDEC)].arrive()
                if dense and dense_read:
                    B[("dec_read", g % NDEC)].arrive()
                yield None
            yield ("wait", ("l_full", it & 1), it >> 1)
            epilogue(it, q, keep)

    def exponential(q):
        kc = 0
        for it, g0, (keep, rescale, _, nq) in tiles_of():
            yield ("wait", ("tile_full", it & 1), it >> 1)
            enter(it)
            kc0 = kc
            for c in range(len(keep)):
                g = g0 + c
                yield ("wait", ("dec_full", g % NDEC), g // NDEC)
                if not read_dec(g):
                    continue
                if q < nq:
                    expect(sbuf[g % NS] == g, f"exponentials read S {sbuf[g % NS]} for block {g}")
                    if rescale[c] and kc > kc0:
                        yield ("wait", ("pv_done", (kc - 1) % NS), (kc - 1) // NS)
                        expect(o_tile[0] == it and o_count[0] >= kc - kc0, "O rescaled early")
                B[("p_full", kc % NS)].arrive()
                kc += 1
                yield None
            if q >= nq:
                B[("l_full", it & 1)].arrive()
                B[("tile_empty", it & 1)].arrive()
                continue
            if kc > kc0:
                yield ("wait", ("pv_done", (kc - 1) % NS), (kc - 1) // NS)
            sums[q] = it
            B[("l_full", it & 1)].arrive()
            yield ("wait", ("l_full", it & 1), it >> 1)
            epilogue(it, q, keep)

    roles = {"K": keys(), "V": values(), "QK0": scores(0), "QK1": scores(1), "PV": pv()}
    for q in range(NQ):
        roles[f"D{q}"], roles[f"E{q}"] = decider(q), exponential(q)
    pending = {n: None for n in roles}
    live = set(roles)
    while live or pipe or tma:
        runnable = [n for n in live if pending[n] is None or wait(pending[n][1], pending[n][2])]
        choices = sorted(runnable) + (["pipe"] if pipe else []) + (["tma"] if tma else [])
        if not choices:
            raise ProtocolError(f"deadlock: { {n: pending[n] for n in live} }")
        pick = rng.choice(choices)
        if pick == "pipe":
            pipe.pop(0)()
        elif pick == "tma":
            tma.pop(rng.randrange(len(tma)))()
        else:
            try:
                pending[pick] = next(roles[pick])
            except StopIteration:
                live.discard(pick)
                pending[pick] = None
    expect(left == active, f"epilogues: {left} of {active}")


def _run_many(runs, **kw):
    rng = random.Random(7)
    for run in range(runs):
        tiles = []
        for _ in range(rng.choice([1, 2, 5, 9])):
            n, frac, dense = rng.choice([1, 2, 3, 7, 12]), rng.choice([0.0, 0.4, 0.9]), rng.random() < 0.4
            keep = [dense or c == 0 or rng.random() >= frac for c in range(n)]
            if not dense and rng.random() < 0.1:
                keep[0] = False  # a first block that no row sees
            tiles.append((keep, [rng.random() < 0.2 for _ in keep], dense, rng.choice([1, 2, 2])))
        simulate_prompt(tiles, run, **kw)


def test_prompt_protocol_has_no_parity_race_or_deadlock():
    _run_many(400)


def test_the_wait_for_o_is_implied():
    """P.V's wait for the last tile's epilogue: every warp that reads O is past it
    before it decides on or exponentiates a block of the next tile."""
    _run_many(400, o_wait=False)


@pytest.mark.parametrize("fault", [dict(q_wait=False), dict(key_slot_of_tile=False),
                                   dict(dense_read=False)])
def test_model_catches(fault):
    """Self-checks of the model: queries loaded over a tile's rows on their way
    out, three key tiles freed as four would be, and a dense tile's decisions that
    nobody reads in the value producer's place."""
    with pytest.raises(ProtocolError):
        _run_many(400, **fault)
