"""The barrier protocol of the paged cache's tensor-core attention kernel, as a model
that runs its warps in random orders: the producer, the MMA warp, the tensor core,
two relays and the softmax warps, on the kernel's mbarriers (phases, parities) and
hardware barriers (counts). It looks for three things: a state in which nothing can
go on, a warp that arrives twice in one phase of a hardware barrier (the barrier then
opens without some other warp, which waits for good later), and data that is used
outside its turn. A wait may run out at any place: it gives up, and so do the others
when they see it, except those that stay in step (Wait.signal).

The kernel has to end in every such run. `steadfast=False` is a form whose relays and
MMA warp go on without waiting after a timeout; it gets stuck, which shows that the
model can tell."""
import random

import pytest


class Stuck(Exception):
    pass


class Model:
    def __init__(self, segs, poll_p, seed, fail=None, steadfast=True, warps=3):
        self.segs, self.n, self.poll_p, self.steadfast = segs, sum(segs), poll_p, steadfast
        self.rng = random.Random(seed)
        self.fail, self.count = fail, 0  # the fail-th time a wait has to wait, it gives up
        self.abort = False
        self.nw = warps
        self.first = [j == 0 for s in segs for j in range(s)]
        one = ["full%d%d" % (s, c) for s in (0, 1) for c in range(4)]
        one += ["empty%d%d" % (s, c) for s in (0, 1) for c in range(4)]
        one += ["sfull0", "sfull1", "pvdone"] + ["seg%d" % i for i in range(8)]
        one += ["info%d" % i for i in range(4)]
        self.mb = {k: [1, 1, 0] for k in one}  # expected, pending, phase
        for k in ("qfull", "ofree", "pfull"):
            self.mb[k] = [warps, warps, 0]
        self.hw = {k: (set(), [0]) for k in ("sready0", "sready1", "pvready0", "pvready1", "sfree0",
                                             "sfree1", "pready", "all", "vote")}
        self.tensor_queue, self.landing = [], []
        self.ended = set()
        # what the data's turns are checked with
        self.seg_at = [None] * 8
        self.info_at = [None] * 4

    # ------------------------------------------------------------- barriers
    def arrive(self, name):
        b = self.mb[name]
        b[1] -= 1
        if b[1] == 0:
            b[1], b[2] = b[0], b[2] + 1

    def done(self, name, parity):
        return (self.mb[name][2] & 1) != parity

    def hw_arrive(self, who, name):
        inside, phase = self.hw[name]
        if who in inside:
            raise Stuck("%s arrives twice at %s" % (who, name))
        inside.add(who)
        if len(inside) == (self.nw if name in ("all", "vote") else self.nw + 1):
            inside.clear()
            phase[0] += 1

    def hw_sync(self, who, name):
        at = self.hw[name][1][0]
        self.hw_arrive(who, name)
        while self.hw[name][1][0] == at:
            yield "hw"

    def wait(self, name, parity):
        """One of the kernel's bounded waits: True, or False after a timeout."""
        if self.done(name, parity):
            return True
        self.count += 1
        give_up = self.fail == self.count
        while True:
            if self.done(name, parity):
                return True
            if give_up and self.rng.random() < 0.3:
                self.abort = True
                return False
            if self.abort and self.rng.random() < 0.3:  # (seen at some later poll)
                return False
            yield "mb"

    def signal(self, name, parity, ok):
        """A wait that a timeout elsewhere does not end: its signal comes all the same."""
        if not self.steadfast:
            return ok and (yield from self.wait(name, parity))
        while not self.done(name, parity):
            yield "mb"
        return True

    def either(self, a, pa, b, pb):
        self.count += 1
        give_up = self.fail == self.count
        while True:
            if self.done(a, pa):
                return 1
            if self.done(b, pb):
                return 2
            if give_up and self.rng.random() < 0.3:
                self.abort = True
                return 0
            if self.abort and self.rng.random() < 0.3:
                return 0
            yield "mb"

    # ---------------------------------------------------------------- roles
    def producer(self):
        n, seg, planned, k = self.n, 1, 0, 0
        self.seg_at[0] = 0
        self.arrive("seg0")

        def plan():
            nonlocal planned, seg
            planned += 1
            if planned < n and self.first[planned]:
                self.seg_at[seg % 8] = seg
                self.arrive("seg%d" % (seg % 8))
                seg += 1

        plan()
        if n > 1:
            plan()
        ok, begun, last = True, 0, 0
        for i in range(n):
            if i + 2 < n:
                plan()
            begun, last = 0, i
            for c in range(4):
                if i >= 2:
                    ok = ok and (yield from self.wait("empty%d%d" % (i & 1, c), ((i >> 1) - 1) & 1))
                if ok:
                    self.landing.append("full%d%d" % (i & 1, c))
                    begun = c + 1
                yield
            if not ok:
                break
            if i == 0:
                self.info_at[0] = 0
                self.arrive("info0")
            if i + 1 < n:
                self.info_at[(i + 1) & 3] = i + 1
                self.arrive("info%d" % ((i + 1) & 3))
            yield
        if self.steadfast:  # no copy may be in flight at the end
            for c in range(4):
                j0 = max(last - (2 if begun == 0 else 1), 0)
                for j in range(j0, last + (c < begun)):
                    while not self.done("full%d%d" % (j & 1, c), (j >> 1) & 1):
                        yield "mb"
            assert not self.landing

    def mma(self):
        n, ok = self.n, True
        q = v = seg = left = 0
        while True:
            pv = v < q and (q == n or q - v == 2 or left == 0)
            if self.poll_p and not pv and v < q and ok:
                r = yield from self.either("full%d3" % (q & 1), (q >> 1) & 1, "pfull", v & 1)
                ok, pv = r != 0, r == 2
            if pv:
                i = v
                if self.poll_p:
                    ok = (yield from self.signal("pfull", i & 1, ok)) and ok
                else:
                    yield from self.hw_sync("mma", "pready")
                if self.first[i] and i > 0:
                    nth = sum(self.first[:i]) - 1
                    ok = ok and (yield from self.wait("ofree", nth & 1))
                if ok:
                    self.tensor_queue += ["empty%d%d" % (i & 1, c) for c in range(4)] + ["pvdone"]
                elif self.steadfast:
                    self.arrive("pvdone")
                v += 1
                if v == n:
                    return
            else:
                i = q
                if left == 0:
                    ok = ok and (yield from self.wait("seg%d" % (seg % 8), (seg >> 3) & 1))
                    if ok:
                        assert self.seg_at[seg % 8] == seg
                    left = self.segs[seg] if ok else n - q
                    ok = ok and (yield from self.wait("qfull", seg & 1))
                if i >= 2:
                    yield from self.hw_sync("mma", "sfree%d" % (i & 1))
                for c in range(4):
                    ok = ok and (yield from self.wait("full%d%d" % (i & 1, c), (i >> 1) & 1))
                if ok:
                    self.tensor_queue.append("sfull%d" % (i & 1))
                elif self.steadfast:
                    self.arrive("sfull%d" % (i & 1))
                q += 1
                left -= 1
                seg += left == 0
            yield

    def tensor(self):
        while self.tensor_queue or "mma" not in self.ended:
            if self.tensor_queue:
                self.arrive(self.tensor_queue.pop(0))
            yield "idle"

    def copies(self):
        while self.landing or "producer" not in self.ended:
            if self.landing:
                self.arrive(self.landing.pop(self.rng.randrange(len(self.landing))))
            yield "idle"

    def relay(self, pv):
        n, ok = self.n, True
        who = "relay_pv" if pv else "relay_s"
        for i in range(n):
            if pv:
                ok = (yield from self.signal("pvdone", i & 1, ok)) and ok
            else:
                if i == 0:
                    ok = ok and (yield from self.wait("info0", 0))
                if i + 1 < n:
                    ok = ok and (yield from self.wait("info%d" % ((i + 1) & 3), ((i + 1) >> 2) & 1))
                ok = (yield from self.signal("sfull%d" % (i & 1), (i >> 1) & 1, ok)) and ok
            self.hw_arrive(who, ("pvready%d" if pv else "sready%d") % (i & 1))
            yield

    def softmax(self, w):
        n, i, seg, lost_votes = self.n, 0, 0, self.lost_votes
        while True:
            more = seg < len(self.segs)
            if more:
                found = yield from self.wait("seg%d" % (seg % 8), (seg >> 3) & 1)
                lost_votes.setdefault(seg, []).append(not found)
                yield from self.hw_sync(w, "all")
                lost = any(lost_votes[seg])
                if not lost:
                    assert self.seg_at[seg % 8] == seg
                    self.arrive("qfull")
                    yield from self.hw_sync(w, "all")
            if seg > 0:
                yield from self.hw_sync(w, "pvready%d" % ((i - 1) & 1))
                yield from self.hw_sync(w, "vote")
                self.arrive("ofree")
            if not more:
                return
            if lost:
                while i < n:
                    yield from self.hw_sync(w, "sready%d" % (i & 1))
                    if i + 2 < n:
                        self.hw_arrive(w, "sfree%d" % (i & 1))
                    if not self.poll_p:
                        self.hw_arrive(w, "pready")
                    elif self.steadfast:
                        self.arrive("pfull")
                    yield from self.hw_sync(w, "pvready%d" % (i & 1))
                    i += 1
                return
            for k in range(self.segs[seg]):
                yield from self.hw_sync(w, "sready%d" % (i & 1))
                if not self.abort:
                    assert self.info_at[i & 3] == i
                if i + 2 < n:
                    self.hw_arrive(w, "sfree%d" % (i & 1))
                yield from self.hw_sync(w, "vote")
                if k > 0:
                    yield from self.hw_sync(w, "pvready%d" % ((i - 1) & 1))
                if self.poll_p:
                    self.arrive("pfull")
                else:
                    self.hw_arrive(w, "pready")
                i += 1
                yield
            seg += 1

    def run(self):
        self.lost_votes = {}
        roles = {"producer": self.producer(), "mma": self.mma(), "tensor": self.tensor(),
                 "copies": self.copies(), "relay_s": self.relay(False), "relay_pv": self.relay(True)}
        roles.update(("s%d" % w, self.softmax("s%d" % w)) for w in range(self.nw))
        slow = self.rng.choice(list(roles) + [None])  # one role may lag behind the others
        still = 0  # steps since something moved
        before = None
        while roles:
            names = list(roles)
            if slow in roles and len(names) > 1 and self.rng.random() < 0.9:
                names.remove(slow)
            k = self.rng.choice(names)
            try:
                next(roles[k])
            except StopIteration:
                del roles[k]
                self.ended.add(k)
            now = (len(roles), self.abort, self.count, len(self.tensor_queue), len(self.landing),
                   tuple((b[1], b[2]) for b in self.mb.values()),
                   tuple((len(s), p[0]) for s, p in self.hw.values()))
            still = still + 1 if now == before else 0
            before = now
            if still > 1500:
                raise Stuck("nothing moves: %s" % sorted(roles))


SEGMENTS = [[1], [2], [3], [7], [1, 1, 1], [2, 2], [3, 2], [1, 5, 1], [5, 1, 1, 4], [1] * 11, [2] * 6]


@pytest.mark.parametrize("poll_p", [False, True])
@pytest.mark.parametrize("segs", SEGMENTS)
def test_every_order_ends(segs, poll_p):
    for seed in range(12):
        m = Model(segs, poll_p, seed)
        m.run()
        assert not m.abort
        for s, p in m.hw.values():
            assert not s


@pytest.mark.parametrize("poll_p", [False, True])
@pytest.mark.parametrize("segs", SEGMENTS)
def test_every_order_ends_after_a_timeout(segs, poll_p):
    """Each of the first waits that has to wait runs out, in several orders."""
    ran_out = 0
    for fail in range(1, 15 * sum(segs) + 10, 1 + sum(segs) // 2):
        for seed in range(3):
            m = Model(segs, poll_p, 1000 * fail + seed, fail)
            m.run()
            ran_out += m.abort
            for s, p in m.hw.values():
                assert not s
    assert ran_out > 5


@pytest.mark.parametrize("poll_p", [False, True])
def test_the_model_sees_warps_that_run_ahead(poll_p):
    stuck = 0
    for fail in range(1, 30):
        for seed in range(4):
            try:
                Model([7], poll_p, 1000 * fail + seed, fail, steadfast=False).run()
            except Stuck:
                stuck += 1
    assert stuck > 0


def test_refusals_of_the_wait_self_test():
    from sparse_attention_prefill_dsa_b200 import build

    build.build()
    import sparse_attention_prefill_dsa_b200 as d

    at = 1 << 20  # an aligned, never dereferenced address
    batch = d.dsa_batch(at, at, at, 2, 4, 5, 0)

    def call(dc=512, dr=64, **over):
        c = d.dsa_cache(at, at, at, 64 * dc, 64 * dr, 10, 64, dc, dr)
        a = dict(q=at, n_heads=32, softmax_scale=0.04, window=0, n_sink=0, out=at, lse=None,
                 wait_cycles=1000, workspace=at, workspace_bytes=1 << 30, stream=0)
        a.update(over)
        return d.dsa_selftest_cache_wait(c, batch, **a)

    assert call(wait_cycles=-1) == d.DSA_ERR_DIMS
    assert call(dc=64, dr=16) == d.DSA_ERR_DIMS
    assert call(q=None) == d.DSA_ERR_NULL
    assert call(window=-1) == d.DSA_ERR_DIMS
    assert call(workspace_bytes=300) == d.DSA_ERR_WORKSPACE
