"""Models of the barrier protocols of the paged-cache kernels, checked over random interleavings
(tests/mbarrier_model.py gives the machine; tests/test_fwd_protocol_model.py says what such a model is).

A CTA walks pieces of units; here a piece is the number of its tiles. Each model has the kernel's waits, arrivals and
commits, with copies, MMAs and commits completing at random times, and checks: no deadlock, no buffer reloaded before
its readers have completed, no MMA before its operands are there, no operand or accumulator overwritten while it is
read, and with waits that run out at random: every role ends and no copy is left in flight. A planted mistake must be
found in each. Keys and values are copied by one or two producers, which arrive on the same barriers; so is Q, or by the first alone.

decode   fa_paged_decode.cu: K and V rings of their own lengths, two Q buffers, S and P double buffered, O per piece
         double buffered; the softmax waits for V itself in a unit's last tile, whose rows past the last key it zeroes.
chunk    fa_paged_chunk.cu: two query tiles, one Q buffer; stage t of the ring holds V of tile t and K of tile t + 1; the
         last tile's V comes on a barrier of its own and the copying warp completes the stage after zeroing rows.
weights  fa_paged_weights.cu: K and Q rings, four S buffers, the groups in turn; with many rows two issuers in turn, and a
         last group adds the groups' sums, double buffered, to the weights.
"""

import random

from mbarrier_model import Machine


def tiles_of(pieces):
    """[(piece, tile within it, last of the piece)] in order."""
    return [(p, k, k + 1 == n) for p, n in enumerate(pieces) for k in range(n)]


def finish(M, roles, issued):
    """Runs the roles, then, after an abort, the exit's wait for the copies in flight: issued() names the barriers of
    copies that were issued, with the parity of their last phases."""
    def drain():
        if M.aborted:
            for name, parity in issued():
                while not M.B[name].passes(parity):
                    yield (name, parity)
            M.need(not M.loads, "the CTA exits with copies in flight")
        yield None
    return M.run(roles, final=drain), M.errors


def last_phases(M, name, counts, bufs):
    """Barrier and parity of the last copy into each of `bufs` buffers, after counts[p] copies by producer p; the arrivals
    of a producer that stopped before the other are made here."""
    n = max(counts)
    out = []
    for i in range(max(0, n - bufs), n):
        bar = name if name in M.B else f"{name}{i % bufs}"
        for c in counts:
            if c <= i:
                M.B[bar].arrive()
        out.append((bar, (i // bufs) & 1))
    return out


def landed(M, prods, *what):
    """Every producer's part of a copy has landed."""
    return all((*what, h) in M.done for h in range(prods))


# ----------------------------------------------------------------------------- decode


def decode(pieces, ks, vs, seed, abort_p=0.0, skip_pv_wait=False, one_p=False, groups=1, prods=1):
    """groups: softmax groups, each with an equal part of every tile's rows."""
    M = Machine(seed, abort_p)
    done, need = M.done, M.need
    T = tiles_of(pieces)
    for i in range(2):
        for n in ("qe", "sf", "pv"):
            M.bar(f"{n}{i}", 1)
        M.bar(f"qf{i}", prods)
        for n in ("of", "p"):
            M.bar(f"{n}{i}", groups)
    for i in range(ks):
        M.bar(f"kf{i}", prods), M.bar(f"ke{i}", 1)
    for i in range(vs):
        M.bar(f"vf{i}", prods), M.bar(f"ve{i}", 1)
    count = {n: [0] * prods for n in "qkv"}
    has = lambda *what: landed(M, prods, *what)

    def producer(h):
        run = True
        for t, (p, k, _) in enumerate(T):
            if k == 0:
                if run and p >= 2:
                    run = yield from M.wait(f"qe{p % 2}", (p // 2 - 1) & 1)
                run = run and not M.aborted
                if run:
                    for u in range(len(T)):
                        need(T[u][0] != p - 2 or ("S", u) in done, f"Q of piece {p - 2} overwritten before S({u})")
                    M.load(f"qf{p % 2}", 1, ("Q", p, h))
                    count["q"][h] = p + 1
            for x, n, reader in (("k", ks, "S"), ("v", vs, "PV")):
                if run and t >= n:
                    run = yield from M.wait(f"{x}e{t % n}", (t // n - 1) & 1)
                run = run and not M.aborted
                if run:
                    need(t < n or (reader, t - n) in done, f"{x} of tile {t - n} overwritten before {reader}")
                    M.load(f"{x}f{t % n}", 1, (x, t, h))
                    count[x][h] = t + 1
            yield None

    def issuer():
        run = True

        def issue_s(t, run):
            p, k, last = T[t]
            if run and k == 0:
                run = yield from M.wait(f"qf{p % 2}", (p // 2) & 1)
            if run:
                run = yield from M.wait(f"kf{t % ks}", (t // ks) & 1)
            if run:
                need(has("Q", p) and has("k", t), f"S({t}) before its operands")
                need(t < 2 or ("P", t - 2) in done, f"S({t}) over S({t - 2}) before it was read")
                M.mma("i", ("S", t))
                M.commit("i", f"sf{t & 1}"), M.commit("i", f"ke{t % ks}")
                if last:
                    M.commit("i", f"qe{p % 2}")
            return run
        if T:
            run = yield from issue_s(0, run)
        for t, (p, k, _) in enumerate(T):
            if t + 1 < len(T):
                run = yield from issue_s(t + 1, run)
            if run:
                run = yield from M.wait("p0" if one_p else f"p{t & 1}", t & 1 if one_p else (t >> 1) & 1)
            if run:
                run = yield from M.wait(f"vf{t % vs}", (t // vs) & 1)
            if run and k == 0 and p >= 2:
                run = yield from M.wait(f"of{p & 1}", ((p >> 1) - 1) & 1)
            if run:
                need(has("v", t) and ("P", t) in done, f"PV({t}) before its operands")
                need(k > 0 or p < 2 or ("O", p - 2) in done, f"PV({t}) over O of piece {p - 2} before it was read")
                M.mma("i", ("PV", t))
                M.commit("i", f"ve{t % vs}"), M.commit("i", f"pv{t & 1}")
            yield None

    parts = {}

    def part_done(what):  # the groups' parts of P(t), or of the read of a piece's O
        parts[what] = parts.get(what, 0) + 1
        if parts[what] == groups:
            done.add(what)

    def softmax(g):
        run = True
        r, r2 = random.Random(seed + 1 + g), random.Random(seed + 5)
        for t, (p, k, last) in enumerate(T):
            if run:
                run = yield from M.wait(f"sf{t & 1}", (t >> 1) & 1)
            if run:
                need(("S", t) in done, f"S({t}) read before it completed")
            if k > 0 and r.random() < 0.2:  # the reference max is raised: O is rescaled
                if run:
                    run = yield from M.wait(f"pv{(t - 1) & 1}", ((t - 1) >> 1) & 1)
                need(not run or ("PV", t - 1) in done, f"O rescaled at {t} before PV({t - 1})")
            if run:  # no wait: PV(t - 2) was issued before S(t)
                need(t < 2 or ("PV", t - 2) in done, f"P({t}) over P({t - 2}) before PV read it")
            if last and r2.random() < 0.7:  # the unit's last tile: V's rows past the last key become 0
                if run:
                    run = yield from M.wait(f"vf{t % vs}", (t // vs) & 1)
                need(not run or (has("v", t) and ("PV", t) not in done), f"V({t}) zeroed at the wrong time")
            yield None
            if run:
                part_done(("P", t))
                M.B["p0" if one_p else f"p{t & 1}"].arrive()
            if last:
                if run and not skip_pv_wait:
                    run = yield from M.wait(f"pv{t & 1}", (t >> 1) & 1)
                need(not run or ("PV", t) in done, f"O read before PV({t})")
                if run:
                    part_done(("O", p))
                    M.B[f"of{p & 1}"].arrive()

    def issued():
        return [x for n, c in (("q", 2), ("k", ks), ("v", vs)) for x in last_phases(M, f"{n}f", count[n], c)]
    return finish(M, {**{f"prod{h}": producer(h) for h in range(prods)}, "mma": issuer(),
                      **{f"soft{g}": softmax(g) for g in range(groups)}}, issued)


def pieces_for(seed):
    r = random.Random(seed * 7919)
    return [r.choice([1, 1, 2, r.randint(1, 9)]) for _ in range(r.randint(0, 6))]


RINGS = [(3, 3), (3, 2), (2, 2), (4, 4)]


def test_decode_has_no_deadlock_or_hazard():
    for seed in range(2500):
        res, errs = decode(pieces_for(seed), *RINGS[seed % 4], seed, groups=(1, 2, 4)[seed % 3], prods=1 + seed // 3 % 2)
        assert res == "ok" and not errs, (pieces_for(seed), RINGS[seed % 4], seed, res, errs[:3])


def test_decode_ends_after_waits_that_run_out():
    for seed in range(1500):
        res, errs = decode(pieces_for(seed), *RINGS[seed % 4], seed, abort_p=0.02, groups=(1, 2, 4)[seed % 3], prods=1 + seed // 3 % 2)
        assert res == "ok" and not errs, (pieces_for(seed), RINGS[seed % 4], seed, res, errs[:3])


def test_decode_model_finds_a_missing_wait():
    assert any(decode(pieces_for(s), 3, 3, s, skip_pv_wait=True)[1] for s in range(500))
    # One barrier for both buffers of P: its phase passes twice before the issuer looks.
    assert any(decode(pieces_for(s), 3, 3, s, one_p=True)[0] == "deadlock" for s in range(500))


# ----------------------------------------------------------------------------- chunk


def chunk(pieces, stages, seed, abort_p=0.0, early_q=False, prods=1, qprods=1):
    """pieces: (tiles, tiles query tile 0 sees, tiles query tile 1 sees, the last tile is the sequence's last)."""
    M = Machine(seed, abort_p)
    done, need = M.done, M.need
    T = tiles_of([n for n, *_ in pieces])
    sees = lambda x, t: t < len(T) and T[t][1] < pieces[T[t][0]][1 + x]
    M.bar("qf", qprods)
    for n in ("k0f", "tail"):
        M.bar(n, prods)
    for n in ("qe", "k0e"):
        M.bar(n, 1)
    for i in range(stages):
        M.bar(f"f{i}", prods + 1), M.bar(f"e{i}", 1)  # f: the copies, and P of tile 0 (128 threads, modelled as one arrival)
    M.bar("p1", 1)
    for x in (0, 1):
        for n in ("sf", "od", "of"):
            M.bar(f"{n}{x}", 1)
    count = {n: [0] * (qprods if n == "q" else prods) for n in ("q", "k0", "t", "tail")}
    needs_p0, p0_last = {}, [-1]
    has = lambda *what: landed(M, prods, *what)

    def producer(h):
        run = True
        if not T:
            return

        def copy_q(p, run):
            if h >= qprods:
                return run
            if run and p > 0 and not early_q:
                run = yield from M.wait("qe", (p - 1) & 1)
            run = run and not M.aborted
            if run:
                for u in range(len(T)):
                    for x in (0, 1):
                        need(T[u][0] != p - 1 or not sees(x, u) or (f"S{x}", u) in done, f"Q {p - 1} overwritten")
                M.load("qf", 1, ("Q", p, h))
                count["q"][h] = p + 1
            return run
        run = yield from copy_q(0, run)
        M.load("k0f", 1, ("K", 0, h))
        count["k0"][h] = 1
        tails = 0
        for t, (p, k, last) in enumerate(T):
            b = t % stages
            more = t + 1 < len(T)
            if run and t == stages - 1:
                run = yield from M.wait("k0e", 0)
            if run and t >= stages:
                run = yield from M.wait(f"e{b}", (t // stages - 1) & 1)
            run = run and not M.aborted
            if run:
                for x in (0, 1):
                    need(t < stages or not sees(x, t - stages) or (f"PV{x}", t - stages) in done, f"V {t} too early")
                    need(t + 1 < stages or not sees(x, t - stages + 1) or (f"S{x}", t - stages + 1) in done,
                         f"K {t + 1} too early")
                if h == 0:
                    needs_p0[b] = sees(0, t)
                    if not sees(0, t):
                        M.B[f"f{b}"].arrive()  # stands in for tile 0's softmax
                count["t"][h] = t + 1
                if not (last and pieces[p][3]):
                    M.expect(f"f{b}", 2 if more else 1)
                    M.copy(f"f{b}", 1, ("V", t, h))
                    if more:
                        M.copy(f"f{b}", 1, ("K", t + 1, h))
                    done.add(("clean", t, h))
                else:
                    M.B[f"f{b}"].tx += 1 if more else 0
                    M.load("tail", 1, ("V", t, h))
                    count["tail"][h] = tails + 1
                    if more:
                        M.copy(f"f{b}", 1, ("K", t + 1, h))
                    run = yield from M.wait("tail", tails & 1)
                    tails += 1
                    if run:
                        done.add(("clean", t, h))
                    M.B[f"f{b}"].arrive()
            if more and T[t + 1][1] == 0:
                run = yield from copy_q(T[t + 1][0], run)
            yield None

    def issuer():
        if not T:
            return
        np1, seen = 0, [0, 0]

        def issue_s(x, t):
            need(landed(M, qprods, "Q", T[t][0]) and has("K", t), f"S{x}({t}) before its operands")
            M.mma("i", (f"S{x}", t))
            M.commit("i", f"sf{x}")
        run = yield from M.wait("qf", 0)
        if run:
            run = yield from M.wait("k0f", 0)
        if run:
            for x in (0, 1):
                if sees(x, 0):
                    issue_s(x, 0)
            M.commit("i", "k0e")
            if T[0][2]:
                M.commit("i", "qe")
        for t, (p, k, last) in enumerate(T):
            if not run:
                break
            more, crosses = t + 1 < len(T), last
            run = yield from M.wait(f"f{t % stages}", (t // stages) & 1)
            for x in (0, 1):
                if not run:
                    break
                if sees(x, t):
                    if k == 0:
                        if seen[x] > 0:
                            run = yield from M.wait(f"of{x}", (seen[x] - 1) & 1)
                        seen[x] += 1
                    if run and x == 1:
                        run = yield from M.wait("p1", np1 & 1)
                        np1 += 1
                    if not run:
                        break
                    # (after an abort the stage is completed as it is; the product then runs on stale data)
                    need(M.aborted or (has("V", t) and has("clean", t)), f"PV{x}({t}) before V")
                    need((f"P{x}", t) in done, f"PV{x}({t}) before P")
                    M.mma("i", (f"PV{x}", t))
                    if k + 1 == min(pieces[p][0], pieces[p][1 + x]):
                        M.commit("i", f"od{x}")
                if more and not crosses and sees(x, t + 1):
                    issue_s(x, t + 1)
            if not run:
                break
            if crosses and more:
                run = yield from M.wait("qf", T[t + 1][0] & 1)
                if not run:
                    break
                for x in (0, 1):
                    if sees(x, t + 1):
                        issue_s(x, t + 1)
            if more and T[t + 1][2]:
                M.commit("i", "qe")
            M.commit("i", f"e{t % stages}")
            yield None

    def softmax(x):
        run, cnt, n = True, 0, 0
        for p, (tiles, *vis, _) in enumerate(pieces):
            mine = [t for t in range(len(T)) if T[t][0] == p and sees(x, t)]
            for t in mine:
                if run:
                    run = yield from M.wait(f"sf{x}", cnt & 1)
                cnt += 1
                if run:
                    need((f"S{x}", t) in done, f"S{x}({t}) read too early")
                    need(T[t][1] == 0 or (f"PV{x}", t - 1) in done, f"O{x} rescaled at {t} too early")
                yield None
                if run:
                    done.add((f"P{x}", t))
                    M.B[f"f{t % stages}" if x == 0 else "p1"].arrive()
                    if x == 0:
                        p0_last[0] = t
            if mine:
                if run:
                    run = yield from M.wait(f"od{x}", n & 1)
                n += 1
                need(not run or (f"PV{x}", mine[-1]) in done, f"O{x} read too early")
                if run:
                    M.B[f"of{x}"].arrive()

    def issued():
        out = [x for n in ("q", "k0", "tail") for x in last_phases(M, "tail" if n == "tail" else f"{n}f", count[n], 1)]
        n = max(count["t"])
        for t in range(max(0, n - stages), n):
            if not M.B[f"f{t % stages}"].passes((t // stages) & 1):
                if (count["t"][0] <= t or needs_p0[t % stages]) and p0_last[0] < t:
                    M.B[f"f{t % stages}"].arrive()  # the softmax arrival that never came, or its stand-in
        return out + last_phases(M, "f", count["t"], stages)
    return finish(M, {**{f"prod{h}": producer(h) for h in range(prods)}, "mma": issuer(), "s0": softmax(0),
                      "s1": softmax(1)}, issued)


def chunk_pieces(seed):
    r = random.Random(seed * 7919)
    out = []
    for n in pieces_for(seed):
        kind = r.random()
        v1 = n if kind < 0.7 else 0  # 0: no second query tile, or no key that it sees
        v0 = r.randint(0, n) if v1 else r.choice([n, n, 0 if n == 1 else n])
        out.append((n, v0, v1, r.random() < 0.5))
    return out


def test_chunk_has_no_deadlock_or_hazard():
    for seed in range(2500):
        res, errs = chunk(chunk_pieces(seed), (2, 4)[seed & 1], seed, prods=2, qprods=1 + seed // 2 % 2)
        assert res == "ok" and not errs, (chunk_pieces(seed), seed, res, errs[:3])


def test_chunk_ends_after_waits_that_run_out():
    for seed in range(1500):
        res, errs = chunk(chunk_pieces(seed), (2, 4)[seed & 1], seed, abort_p=0.02, prods=2, qprods=1 + seed // 2 % 2)
        assert res == "ok" and not errs, (chunk_pieces(seed), seed, res, errs[:3])


def test_chunk_model_finds_a_missing_wait():
    assert any(chunk(chunk_pieces(s), 2, s, early_q=True)[1] for s in range(500))


# ----------------------------------------------------------------------------- weights


def weights(pieces, few, seed, abort_p=0.0, no_sum_free=False, odd_ring=False, three=False, prods=1, qprods=1):
    """pieces: the query tiles of each key tile (few rows: one each, and every third begins another head)."""
    M = Machine(seed, abort_p)
    done, need = M.done, M.need
    T = tiles_of(pieces)
    G, kb, qb, sb, issuers = (3 if few or three else 4), (5 if few else 2), (2 if few else 4), 3 if odd_ring else 4, (1 if few else 2)
    head = lambda p: p % 3 == 0  # few rows: Q is copied where a head begins
    q_of = (lambda t: T[t][0] // 3) if few else (lambda t: t)
    for n, c in (("kf", kb), ("ke", kb), ("qf", qb), ("qe", qb), ("sf", sb), ("fr", sb)):
        for i in range(c):
            M.bar(f"{n}{i}", issuers if n == "ke" else prods if n == "kf" else qprods if n == "qf" else 1)
    for i in range(2):
        M.bar(f"sr{i}", G), M.bar(f"sx{i}", 1)
    count = {"k": [0] * prods, "q": [0] * qprods}
    has = lambda *what: landed(M, prods, *what)

    def producer(h):
        run = True

        def copy_q(q, run):
            if h >= qprods:
                return run
            if run and q >= qb:
                run = yield from M.wait(f"qe{q % qb}", (q // qb - 1) & 1)
            run = run and not M.aborted
            if run:
                need(all(("S", t) in done for t in range(len(T)) if q_of(t) == q - qb), f"Q {q - qb} overwritten")
                M.load(f"qf{q % qb}", 1, ("Q", q, h))
                count["q"][h] = q + 1
            return run
        for p, n in enumerate(pieces):
            if few and head(p):
                run = yield from copy_q(p // 3, run)
            if run and p >= kb:
                run = yield from M.wait(f"ke{p % kb}", (p // kb - 1) & 1)
            run = run and not M.aborted
            if run:
                need(all(("S", t) in done for t in range(len(T)) if T[t][0] == p - kb), f"K {p - kb} overwritten")
                M.load(f"kf{p % kb}", 1, ("K", p, h))
                count["k"][h] = p + 1
            if not few:
                for t in range(len(T)):
                    if T[t][0] == p:
                        run = yield from copy_q(t, run)
            yield None

    def issuer(me):  # with many rows two take the tiles in turn
        run = True
        for t, (p, k, last) in enumerate(T):
            if run and few and head(p):
                run = yield from M.wait(f"qf{p // 3 % qb}", (p // 3 // qb) & 1)
            if run and k == 0:
                run = yield from M.wait(f"kf{p % kb}", (p // kb) & 1)
            if few or (t & 1) == me:
                if run and not few:
                    run = yield from M.wait(f"qf{t % qb}", (t // qb) & 1)
                if run and t >= sb:
                    run = yield from M.wait(f"fr{t % sb}", (t // sb - 1) & 1)
                if not run:
                    break
                need(has("K", p) and landed(M, qprods, "Q", q_of(t)), f"S({t}) before its operands")
                need(t < sb or ("read", t - sb) in done, f"S({t}) over S({t - sb})")
                M.mma(f"i{me}", ("S", t))
                M.commit(f"i{me}", f"sf{t % sb}")
            if not run:
                break
            if last:
                M.commit(f"i{me}", f"ke{p % kb}")
                if few and t + 1 < len(T) and head(T[t + 1][0]):
                    M.commit(f"i{me}", f"qe{p // 3 % qb}")
            yield None

    def group(g):
        run = True
        for p in range(len(pieces)):
            for t in range(len(T)):
                if T[t][0] != p or t % G != g:
                    continue
                if run:
                    run = yield from M.wait(f"sf{t % sb}", (t // sb) & 1)
                need(not run or ("S", t) in done, f"S({t}) read too early")
                if run and not few:
                    M.B[f"qe{t % qb}"].arrive()
                yield None
                if run:
                    done.add(("read", t))
                    M.B[f"fr{t % sb}"].arrive()
            if not few:
                if run and p >= 2 and not no_sum_free:
                    run = yield from M.wait(f"sx{p & 1}", ((p >> 1) - 1) & 1)
                if run:
                    need(p < 2 or ("sum", p - 2) in done, f"the sums of piece {p - 2} overwritten")
                    M.B[f"sr{p & 1}"].arrive()
                yield None

    def adder():
        run = True
        for p in range(len(pieces)):
            if run:
                run = yield from M.wait(f"sr{p & 1}", (p >> 1) & 1)
            if run:
                done.add(("sum", p))
                M.B[f"sx{p & 1}"].arrive()
            yield None

    roles = {**{f"prod{h}": producer(h) for h in range(prods)}, "mma0": issuer(0), **{f"g{g}": group(g) for g in range(G)}}
    if not few:
        roles |= {"mma1": issuer(1), "add": adder()}

    def issued():
        return last_phases(M, "qf", count["q"], qb) + last_phases(M, "kf", count["k"], kb)
    return finish(M, roles, issued)


def weight_pieces(seed, few):
    return [1] * random.Random(seed).randint(0, 14) if few else pieces_for(seed)


def test_weights_has_no_deadlock_or_hazard():
    for seed in range(2500):
        few = bool(seed & 1)
        res, errs = weights(weight_pieces(seed, few), few, seed, prods=2, qprods=1 + seed // 2 % 2)
        assert res == "ok" and not errs, (weight_pieces(seed, few), few, seed, res, errs[:3])


def test_weights_ends_after_waits_that_run_out():
    for seed in range(1500):
        few = bool(seed & 1)
        res, errs = weights(weight_pieces(seed, few), few, seed, abort_p=0.02, prods=2, qprods=1 + seed // 2 % 2)
        assert res == "ok" and not errs, (weight_pieces(seed, few), few, seed, res, errs[:3])


def test_weights_model_finds_a_missing_wait():
    def faulty(s):
        try:
            return bool(weights(weight_pieces(s, False), False, s, no_sum_free=True)[1])
        except AssertionError:  # an arrival beyond a barrier's count
            return True
    assert any(faulty(s) for s in range(500))
    # Three S buffers between two issuers: each sees every other phase of a buffer, and a parity cannot tell it from
    # the one before.
    assert any(weights(weight_pieces(s, False), False, s, odd_ring=True)[1] for s in range(500))
    # Three groups between two issuers: a tile that is done does not mean that the one before it is, so a group may look
    # at a buffer two phases late.
    def early(s):
        try:
            return bool(weights(weight_pieces(s, False), False, s, three=True)[1])
        except AssertionError:
            return True
    assert any(early(s) for s in range(500))
