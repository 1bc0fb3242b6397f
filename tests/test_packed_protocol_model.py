"""Models of the barrier protocols of the packed attention's tensor-core kernels, run under random
timings on the CPU with every score warp by itself (some much slower than others): no deadlock,
and every tensor-core operation and every warp reads what it expects. Tensor-core operations run
in issue order and a commit completes when everything issued before it has; copies land in any
order. A barrier counts arrivals and nothing else: a warp that runs ahead may complete a phase in
the place of one that is late, which is what these models are there to find. How many barriers
the scores' arrivals are spread over is read from the source."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "video_diffusion_transformer_wan_b200", "csrc")


class Race(Exception):
    pass


class Bar:
    def __init__(self, count=1):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase ^= 1
            self.pending = self.count

    def ready(self, parity):
        return self.phase != parity & 1


def check(got, want, who):
    if got != want:
        raise Race(f"{who}: {got} in place of {want}")


class Machine:
    """Roles (generators; None is a wait or a delay), the tensor core's queue, copies in flight."""

    def __init__(self, seed):
        self.rnd = random.Random(seed)
        self.mma, self.copies, self.roles = [], [], []

    def issue(self, op):
        self.mma.append(op)

    def commit(self, bar):
        self.mma.append(bar.arrive)

    def copy(self, land):
        self.copies.append(land)

    def run(self, roles):
        # a role's speed differs up to 30 times from another's
        speed = [self.rnd.choice((1.0, 0.3, 0.03)) for _ in roles]
        live = list(roles)
        for _ in range(600000):
            if not live:
                break
            i = self.rnd.randrange(len(live))
            if self.rnd.random() < speed[roles.index(live[i])]:
                try:
                    next(live[i])
                except StopIteration:
                    live.pop(i)
            if self.copies and self.rnd.random() < 0.3:
                self.copies.pop(self.rnd.randrange(len(self.copies)))()
            if self.mma and self.rnd.random() < 0.5:
                self.mma.pop(0)()
        while self.mma:
            self.mma.pop(0)()
        return not live


def wait(bar, parity):
    while not bar.ready(parity):
        yield


WARPS = 8


def dq_slot(load):
    j = load >> 1
    return (3 + (j & 1), (j >> 1) & 1) if load & 1 else (j % 3, (j // 3) & 1)


def run_dq(n, seed, ds_bars):
    m = Machine(seed)
    kv_full, kv_empty = [Bar() for _ in range(5)], [Bar() for _ in range(5)]
    s_full, y_free, done = Bar(), Bar(WARPS), Bar()
    ds_full = [Bar(WARPS) for _ in range(ds_bars)]
    slot, S, Y, out = [None] * 5, [[None] * WARPS, [None] * WARPS], [None] * WARPS, []

    def ds_bar(j):
        return ds_full[j % ds_bars], (j // ds_bars) & 1

    def producer():
        for load in range(2 * n):
            s, ph = dq_slot(load)
            yield from wait(kv_empty[s], ph ^ 1)

            def land(s=s, load=load):
                slot[s] = load
                kv_full[s].arrive()
            m.copy(land)
            yield

    def mma():
        def scores(j):
            ks, kp = dq_slot(2 * j)
            vs, vp = dq_slot(2 * j + 1)
            yield from wait(kv_full[ks], kp)

            def s_op():
                check(slot[ks], 2 * j, "S")
                S[j & 1][:] = [("S", j)] * WARPS
            m.issue(s_op)
            yield from wait(kv_full[vs], vp)
            if j > 0:
                yield from wait(y_free, j - 1)

            def y_op():
                check(slot[vs], 2 * j + 1, "dP")
                Y[:] = [("dP", j)] * WARPS
            m.issue(y_op)
            m.commit(kv_empty[vs])
            m.commit(s_full)

        yield from scores(0)
        for j in range(n):
            if j + 1 < n:
                yield from scores(j + 1)
            yield from wait(*ds_bar(j))
            ks = dq_slot(2 * j)[0]

            def q_op(j=j, ks=ks):
                check(slot[ks], 2 * j, "dQ")
                check(S[j & 1], [("ds", j)] * WARPS, "dQ")
                out.append(j)
            m.issue(q_op)
            m.commit(kv_empty[ks])
            yield
        m.commit(done)
        yield from wait(done, 0)

    def warp(w):
        for j in range(n):
            yield from wait(s_full, j)
            check(S[j & 1][w], ("S", j), "scores")
            check(Y[w], ("dP", j), "scores")
            yield
            check(Y[w], ("dP", j), "scores")  # the reads take a while
            y_free.arrive()
            yield
            check(S[j & 1][w], ("S", j), "scores")
            S[j & 1][w] = ("ds", j)
            yield
            ds_bar(j)[0].arrive()
            yield
        yield from wait(done, 0)
        check(out, list(range(n)), "output")

    return m.run([producer(), mma()] + [warp(w) for w in range(WARPS)])


def run_dkv(n, seed, stages=4, stat_bufs=4):
    m = Machine(seed)
    q_full, q_empty = [Bar() for _ in range(stages)], [Bar() for _ in range(stages)]
    s_full, p_full, done = [Bar(), Bar()], [Bar(WARPS), Bar(WARPS)], Bar()
    st_full, st_empty = [Bar() for _ in range(stat_bufs)], [Bar(WARPS) for _ in range(stat_bufs)]
    slot, S, stats, out = [None] * stages, [[None] * WARPS, [None] * WARPS], [None] * stat_bufs, []

    def producer():
        for i in range(n):
            s = i % stages
            yield from wait(q_empty[s], (i // stages) ^ 1)

            def land(s=s, i=i):
                slot[s] = i
                q_full[s].arrive()
            m.copy(land)
            yield

    def stat_warp():
        for i in range(n):
            b = i % stat_bufs
            if i >= stat_bufs:
                yield from wait(st_empty[b], i // stat_bufs - 1)
            stats[b] = i
            yield
            st_full[b].arrive()
            yield

    def mma():
        def scores(i):
            s = i % stages
            yield from wait(q_full[s], i // stages)

            def op():
                check(slot[s], i, "scores")
                S[i & 1][:] = [("S", i)] * WARPS
            m.issue(op)
            m.commit(s_full[i & 1])

        for i in range(min(2, n)):
            yield from scores(i)
        for i in range(n):
            yield from wait(p_full[i & 1], i >> 1)

            def op(i=i):
                check(slot[i % stages], i, "products")
                check(S[i & 1], [("p", i)] * WARPS, "products")
                out.append(i)
            m.issue(op)
            m.commit(q_empty[i % stages])
            if i + 2 < n:
                yield from scores(i + 2)
            yield
        m.commit(done)
        yield from wait(done, 0)

    def warp(w):
        for i in range(n):
            yield from wait(st_full[i % stat_bufs], i // stat_bufs)
            yield from wait(s_full[i & 1], i >> 1)
            check(S[i & 1][w], ("S", i), "warp")
            check(stats[i % stat_bufs], i, "warp")
            yield
            check(stats[i % stat_bufs], i, "warp")
            st_empty[i % stat_bufs].arrive()
            yield
            check(S[i & 1][w], ("S", i), "warp")
            S[i & 1][w] = ("p", i)
            p_full[i & 1].arrive()
            yield
        yield from wait(done, 0)
        check(out, list(range(n)), "output")

    return m.run([producer(), stat_warp(), mma()] + [warp(w) for w in range(WARPS)])


def pos_k(j):
    return 0 if j == 0 else 2 * j - 1


def pos_v(j, n):
    return 2 * n - 1 if j == n - 1 else 2 * j + 2


def run_forward(pieces, seed, stages=5):
    """`pieces`: key tiles of the two query tiles of each piece; the last V tile of a piece with
    an odd number of them is ragged."""
    m, half = Machine(seed), 4
    q_full, q_empty, ragged, cleared = Bar(), Bar(), Bar(), Bar()
    kv_full, kv_empty = [Bar() for _ in range(stages)], [Bar() for _ in range(stages)]
    s_full, o_final = [Bar(), Bar()], [Bar(), Bar()]
    p_half, p_full = [Bar(half), Bar(half)], [Bar(half), Bar(half)]
    slot, q = [None] * stages, [None]
    S = [[None] * half, [None] * half]     # per warp of a query tile
    O = [None, None]
    clear = set()
    work = [(u, ns, max(ns)) for u, ns in enumerate(pieces) if max(ns) > 0]

    def is_ragged(n):
        return n & 1

    def producer():
        issued = 0
        for k, (u, ns, n) in enumerate(work):
            if k > 0:
                yield from wait(q_empty, k - 1)

            def land_q(u=u):
                q[0] = u
                q_full.arrive()
            m.copy(land_q)
            for ld in range(2 * n):
                s = issued % stages
                yield from wait(kv_empty[s], (issued // stages) ^ 1)
                is_v = ld == 2 * n - 1 or (ld > 0 and ld % 2 == 0)
                j = (n - 1 if ld == 2 * n - 1 else (ld >> 1) - 1) if is_v else (ld + 1) >> 1

                def land(s=s, what=("V" if is_v else "K", u, j)):
                    slot[s] = what
                    kv_full[s].arrive()
                m.copy(land)
                issued += 1
                yield

    def mma():
        base, rag = 0, 0
        seen = [0, 0]
        for k, (u, ns, n) in enumerate(work):
            def kv(pos):
                return wait(kv_full[pos % stages], pos // stages)

            def qk(t, j, s, u=u):
                def op():
                    check(slot[s], ("K", u, j), "scores")
                    check(q[0], u, "scores")
                    S[t][:] = [("S", u, j)] * half
                m.issue(op)
                m.commit(s_full[t])

            def pv(t, j, s, u=u, n=n, ns=ns):
                for part, bar in ((0, p_half[t]), (1, p_full[t])):
                    yield from wait(bar, seen[t])

                    def op(part=part):
                        check(slot[s], ("V", u, j), "product")
                        if j == n - 1 and is_ragged(n):
                            check(u in clear, True, "ragged values")
                        want = ("P", u, j) if part else None
                        for x in S[t]:
                            if part:
                                check(x, want, "product")
                            elif x not in (("H", u, j), ("P", u, j)):
                                raise Race(f"first part read {x}")
                        if part:
                            if j > 0:
                                check(O[t], (u, j), "sum")
                            elif isinstance(O[t], tuple) and O[t][1] != "read":
                                raise Race(f"{O[t]} was overwritten before it was read")
                            O[t] = (u, j + 1)
                    m.issue(op)
                seen[t] += 1

            yield from wait(q_full, k)
            for j in range(n):
                yield from kv(base + pos_k(j))
                if j > 0:
                    yield from kv(base + pos_v(j - 1, n))
                ks, vs = (base + pos_k(j)) % stages, (base + pos_v(j - 1, n)) % stages
                for t in range(2):
                    if 0 < j <= ns[t]:
                        yield from pv(t, j - 1, vs)
                        if j == ns[t]:
                            m.commit(o_final[t])
                    if j < ns[t]:
                        qk(t, j, ks)
                m.commit(kv_empty[ks])
                if j > 0:
                    m.commit(kv_empty[vs])
                yield
            m.commit(q_empty)
            pos = base + pos_v(n - 1, n)
            yield from kv(pos)
            if is_ragged(n):
                ragged.arrive()
                yield from wait(cleared, rag)
                rag += 1
            for t in range(2):
                if ns[t] == n:
                    yield from pv(t, n - 1, pos % stages)
                    m.commit(o_final[t])
            m.commit(kv_empty[pos % stages])
            base += 2 * n
            yield

    def clearing():
        rag = 0
        for u, ns, n in work:
            if is_ragged(n):
                yield from wait(ragged, rag)
                rag += 1
                clear.add(u)
                yield
                cleared.arrive()
                yield

    readers = [[0], [0]]

    def softmax(t, w):
        s_seen, o_seen = 0, 0
        for u, ns, n in work:
            for j in range(ns[t]):
                yield from wait(s_full[t], s_seen)
                s_seen += 1
                check(S[t][w], ("S", u, j), "softmax")
                if j > 0:
                    check(O[t], (u, j), "rescaling")
                yield
                S[t][w] = ("H", u, j)
                p_half[t].arrive()
                yield
                S[t][w] = ("P", u, j)
                p_full[t].arrive()
                yield
            if ns[t] > 0:
                yield from wait(o_final[t], o_seen)
                o_seen += 1
                check(O[t], (u, ns[t]), "output")
                yield
                check(O[t], (u, ns[t]), "output")
                readers[t][0] += 1
                if readers[t][0] % half == 0:
                    O[t] = (u, "read")
                yield

    return m.run([producer(), mma(), clearing()] + [softmax(t, w) for t in range(2) for w in range(half)])


def _ds_bars():
    text = open(os.path.join(CSRC, "attn_packed_bwd_tc.cu")).read()
    kernel = text[text.index("packed_dq_tc_kernel("):text.index("packed_dkv_tc_kernel(")]
    arrive = re.search(r"mbar_arrive\((&?ds_full[^;]*)\);", kernel).group(1)
    waits = re.search(r"mbar_wait_warp\((&?ds_full[^,]*), static_cast<uint32_t>\(([^;]*?)\), p\.err\)", kernel)
    if arrive == "ds_full":
        assert waits.groups() == ("ds_full", "j & 1")
        return 1
    assert arrive == "&ds_full[j & 1]" and waits.groups() == ("&ds_full[j & 1]", "(j >> 1) & 1")
    return 2


@pytest.mark.parametrize("n", [1, 2, 3, 4, 9, 17])
def test_queries_gradient(n):
    for seed in range(40):
        assert run_dq(n, seed, _ds_bars())


def test_model_finds_a_late_warp():
    """One barrier for all tiles' ds: a warp a tile ahead arrives in the place of a late one."""
    def races(seed):
        try:
            run_dq(9, seed, 1)
        except Race:
            return True
        return False
    assert any(races(seed) for seed in range(40))


@pytest.mark.parametrize("n", [1, 2, 3, 5, 12, 19])
def test_keys_gradient(n):
    for seed in range(30):
        assert run_dkv(n, seed)


@pytest.mark.parametrize("pieces", [[(1, 1)], [(3, 3)], [(4, 5), (1, 0), (0, 0), (0, 2), (6, 6)], [(1, 2)] * 5, [(2, 0), (7, 8), (1, 1)],
                                    [(0, 3), (3, 0), (5, 5)]])
def test_forward(pieces):
    for seed in range(30):
        assert run_forward(pieces, seed)


def test_float32_blocks_wait_for_copies_of_no_group():
    """A block whose rows see nothing (or no query sees its keys) copies its own rows and commits no
    group; what it waits for before it leaves has to cover those copies."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "attn_packed_simt.cu")).read())
    wait_all = re.search(r'void async_wait_all\(\) \{ asm volatile\("([^"]*)"', text).group(1)
    kernels = re.findall(r"packed_(?:fwd|dq|dkv)_kernel\(const PackedAttn p\) \{(.*?)\n\}", text, re.S)
    assert len(kernels) == 3
    for kernel in kernels:
        copies = len(re.findall(r"\n  load_async<D>\(s[qkov],", kernel))
        assert copies > 0
        pending = 0  # copies not waited for where the walk has no tile
        for line in (kernel[:kernel.index("st ^= 1) {")] + kernel[kernel.rindex("async_wait_all();"):]).splitlines():
            if "auto load" in line or "if (most > 0) load" in line or "if (n > 0) load" in line:
                continue
            if re.match(r"\s{2}load_async<D>\(s[qkov],", line):
                pending += 1
            if "async_wait_all();" in line and wait_all == "cp.async.wait_all;":
                pending = 0
        assert pending == 0
