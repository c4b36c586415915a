"""Model of the barrier protocol of the few-row kernel over an 8-bit cache (fa_paged_fp8_few.cu), checked over random
interleavings; tests/mbarrier_model.py gives the machine and tests/test_paged_protocol_model.py says what such a model is.

Five kinds of roles: a warp that copies keys and codes, one that copies values and asks for Q (and splits it, or leaves that
to the softmax), one that issues S, one that issues P V, and the softmax groups. K and V have rings of their own lengths, codes
a longer one without a barrier of its own to empty it, S and P two buffers, Q two, O one, which no barrier frees: the first P of a
piece follows its group's read of the last piece's O. A planted mistake must be
found in each of the places that carry the protocol."""

import random

import pytest

from mbarrier_model import Machine
from test_paged_protocol_model import finish, tiles_of


def few8(pieces, ks, vs, seed, abort_p=0.0, soft=False, groups=1, cs=16, raise_p=0.2, skip=(), o_early=False):
    M = Machine(seed, abort_p)
    done, need = M.done, M.need
    T = tiles_of(pieces)
    for i in range(2):
        M.bar(f"qr{i}", 1)
        M.bar(f"qf{i}", groups if soft else 1)
        M.bar(f"qe{i}", 1 if "scales" in skip else 1 + groups)
        M.bar(f"sf{i}", 2)
        M.bar(f"p{i}", groups)
    for i in range(ks):
        M.bar(f"kf{i}", 2), M.bar(f"ke{i}", 1)
    for i in range(vs):
        M.bar(f"vf{i}", 1), M.bar(f"ve{i}", 1)
    issued = {"k": 0, "v": 0}
    rnd = random.Random(seed + 1)
    raises = {t for t in range(len(T)) if T[t][1] > 0 and rnd.random() < raise_p}  # the groups agree on them
    all_of = lambda *what: all((*what, g) in done for g in range(groups))  # noqa: E731

    def keys():
        run = True
        for t in range(len(T)):
            if run and t >= ks:
                run = yield from M.wait(f"ke{t % ks}", (t // ks - 1) & 1)
            run = run and not M.aborted
            if run:
                need(t < ks or ("S", t - ks) in done, f"K of tile {t - ks} overwritten before S")
                need(t < cs or all_of("P", t - cs), f"codes of tile {t - cs} overwritten before they were read")
                M.load(f"kf{t % ks}", 1, ("k", t))
                M.load(f"kf{t % ks}", 1, ("c", t))
                issued["k"] = t + 1
            yield None

    def values():
        run, piece, asked = True, 0, False

        def step():  # asks for Q of `piece`, or splits it
            nonlocal run, piece, asked
            if not asked:
                if run and piece >= 2:
                    run = yield from M.wait(f"qe{piece % 2}", (piece // 2 - 1) & 1)
                run = run and not M.aborted
                if run:
                    for u, (p, _, last) in enumerate(T):
                        need(p != piece - 2 or ("S", u) in done, f"Q of piece {p} overwritten before S({u})")
                        need(p != piece - 2 or not last or all_of("P", u), f"scales of piece {p} overwritten before tile {u}")
                    M.load(f"qr{piece % 2}", 1, ("raw", piece))
                if soft:
                    piece += 1
                else:
                    asked = True
                return
            if run:
                while ("raw", piece) not in done:  # (a wait for this warp's own copies: it always ends)
                    yield (f"qr{piece % 2}", (piece // 2) & 1)
                done.add(("Q", piece, 0))
                M.B[f"qf{piece % 2}"].arrive()
            asked = False
            piece += 1
        if T:
            yield from step()
        of = copied = 0
        for t, (p, _, last) in enumerate(T):
            if run and t >= vs:
                run = yield from M.wait(f"ve{t % vs}", (t // vs - 1) & 1)
            run = run and not M.aborted
            if run:
                need(t < vs or ("PV", t - vs) in done, f"V of tile {t - vs} overwritten before PV")
                M.load(f"vf{t % vs}", 1, ("v", t))
                issued["v"] = t + 1
            copied += 1
            due, more = of + 1 if last else of, int(copied > vs)
            while piece < len(pieces) and (piece <= due or (piece == of + 1 and more > 0)):
                if piece > due:
                    more -= 1
                yield from step()
            if last:
                of, copied = of + 1, 0
            yield None

    def scores():
        run = True
        for t, (p, k, last) in enumerate(T):
            if run and k == 0:
                run = yield from M.wait(f"qf{p % 2}", (p // 2) & 1)
            if run and t >= 2 and "s_wait" not in skip:
                run = yield from M.wait(f"ve{(t - 2) % vs}", ((t - 2) // vs) & 1)
            if run:
                run = yield from M.wait(f"kf{t % ks}", (t // ks) & 1)
            if run:
                need(all((("Q", p, g) in done) for g in range(groups if soft else 1)), f"S({t}) before Q")
                need(("k", t) in done and ("c", t) in done, f"S({t}) before its keys and codes")
                need(t < 2 or all_of("P", t - 2), f"S({t}) over S({t - 2}) before it was read")
                M.B[f"sf{t & 1}"].arrive()
                M.mma("s", ("S", t))
                M.commit("s", f"sf{t & 1}"), M.commit("s", f"ke{t % ks}")
                if last:
                    M.commit("s", f"qe{p % 2}")
            yield None

    def products():
        run = True
        for t, (p, k, _) in enumerate(T):
            if run:
                run = yield from M.wait(f"vf{t % vs}", (t // vs) & 1)
            if run:
                run = yield from M.wait(f"p{t & 1}", (t >> 1) & 1)
            if run:
                need(("v", t) in done and all_of("P", t), f"PV({t}) before its operands")
                need(k > 0 or p == 0 or all_of("O", p - 1), f"PV({t}) over O of piece {p - 1} before it was read")
                M.mma("p", ("PV", t))
                M.commit("p", f"ve{t % vs}")
            yield None

    def softmax(g):
        run, split = True, 0
        for t, (p, k, last) in enumerate(T):
            if soft:
                due = p + 1 if last and p + 1 < len(pieces) else p
                while split <= due:
                    if run:
                        run = yield from M.wait(f"qr{split % 2}", (split // 2) & 1)
                    if run:
                        need(("raw", split) in done, f"Q of piece {split} split before it arrived")
                        done.add(("Q", split, g))
                        M.B[f"qf{split % 2}"].arrive()
                    split += 1
            if run and k == 0:
                run = yield from M.wait(f"qf{p % 2}", (p // 2) & 1)
            if run:
                run = yield from M.wait(f"sf{t & 1}", (t >> 1) & 1)
            if run:
                need(("S", t) in done and ("c", t) in done, f"tile {t} read before it was there")
            if t in raises:
                if run:
                    run = yield from M.wait(f"ve{(t - 1) % vs}", ((t - 1) // vs) & 1)
                if run:
                    need(("PV", t - 1) in done, f"O rescaled for tile {t} while PV({t - 1}) adds to it")
            if run:
                need(t < 2 or ("PV", t - 2) in done, f"P({t}) over P({t - 2}) before PV had read it")
            if last and run:  # the rows past the last key
                run = yield from M.wait(f"vf{t % vs}", (t // vs) & 1)
            if run:
                done.add(("P", t, g))
                M.B[f"p{t & 1}"].arrive()
            if last:
                if run and "scales" not in skip:
                    M.B[f"qe{p % 2}"].arrive()
                if run and not o_early:
                    run = yield from M.wait(f"ve{t % vs}", (t // vs) & 1)
                if run and not o_early:
                    need(("PV", t) in done, f"O of piece {p} read before it was complete")
                    done.add(("O", p, g))
            yield None

    def in_flight():
        return [(f"{x}f{i % n}", (i // n) & 1) for x, n in (("k", ks), ("v", vs)) for i in range(max(0, issued[x] - n), issued[x])]

    roles = {"keys": keys(), "values": values(), "scores": scores(), "products": products()}
    roles.update({f"softmax{g}": softmax(g) for g in range(groups)})
    if abort_p:  # what a role asked for itself it also waits for
        return finish_loose(M, roles, in_flight)
    return finish(M, roles, in_flight)


def finish_loose(M, roles, issued):
    """finish(), with the Q copies left out of what must have landed at the exit: the warp that asked for them waits."""

    def drain():
        if M.aborted:
            for name, parity in issued():
                while not M.B[name].passes(parity):
                    yield (name, parity)
            M.need(not [x for x in M.loads if not x[0].startswith("qr")], "the CTA exits with copies in flight")
        yield None
    return M.run(roles, final=drain), M.errors


# (K ring, V ring, split by the softmax, groups): the kernels' own, at d = 128 and 64.
KERNELS = [(3, 2, False, 1), (5, 5, False, 1), (5, 5, True, 4), (8, 8, True, 4), (4, 3, True, 4), (6, 6, True, 4)]
SHARES = [[], [1], [5], [1, 1, 1, 1], [2, 1, 7], [9, 3, 1, 1, 6], [20, 4], [1, 12, 1, 2]]


@pytest.mark.parametrize("kernel", KERNELS)
def test_few8(kernel):
    ks, vs, soft, groups = kernel
    for i, pieces in enumerate(SHARES):
        for seed in range(25):
            r, errors = few8(pieces, ks, vs, 100 * i + seed, soft=soft, groups=groups)
            assert r == "ok" and not errors, (pieces, seed, r, errors[:3])


@pytest.mark.parametrize("kernel", KERNELS)
def test_few8_waits_that_run_out(kernel):
    """Every role ends, and the copies into the rings have landed at the exit."""
    ks, vs, soft, groups = kernel
    for i, pieces in enumerate(SHARES):
        for seed in range(25):
            r, errors = few8(pieces, ks, vs, 7000 + 100 * i + seed, abort_p=0.02, soft=soft, groups=groups)
            late = [e for e in errors if "in flight" in e or "deadlock" in e]
            assert r == "ok" and not late, (pieces, seed, r, late[:3])


def found(**kw):
    for pieces in ([9, 3, 1, 1, 6], [2, 1, 7, 2, 2], [30], [20, 4]):
        for seed in range(60):
            r, errors = few8(pieces, seed=seed, **kw)
            if r != "ok" or errors:
                return True
    return False


@pytest.mark.parametrize("kw", [
    dict(ks=3, vs=2, skip=("s_wait",)),                           # S does not wait for the scores and P of two tiles before
    dict(ks=5, vs=5, o_early=True, groups=2),                     # P of the next piece made before O is read
    dict(ks=5, vs=5, skip=("scales",)),                           # Q's scales overwritten while the softmax reads them
    dict(ks=8, vs=8, cs=9),                                       # a ring of codes no longer than the keys' and one
])
def test_planted_mistakes_are_found(kw):
    assert found(**kw)


def test_the_ring_of_codes_is_long_enough():
    """Codes of t overwrite those of t - 16 once S of t - kKStages is done, which P V of t - kKStages - 2 came before."""
    for ks in (3, 4, 5, 6, 8):
        assert 16 >= ks + 2
        for seed in range(20):
            r, errors = few8([40], ks, 8, seed, cs=ks + 2)
            assert r == "ok" and not errors, (ks, errors[:2])
