"""The order of the tensor-core walk's warp roles, on the CPU: each role's waits, reads, writes and arrivals, chunk by
chunk, as a graph.  An arrival comes before every wait for the phase that it completes; what a role does comes in its
program order.  Checked: the graph has no cycle (no role waits for ever), and whoever reads a buffer has read it
before it is written again, and after it was written.

The model is tied to the kernel's source: which barriers a role waits for and arrives on, and how many arrivals a
phase takes, are read from it."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "delta_rule_linear_efla_b200", "csrc",
                   "decay_tc.cu")
NS, GB, SLOTS = 3, 4, 8

# where a role's code begins, in the order of the source (the walk with output; None: the first pass alone)
SECTIONS = [("tma", "if (warp == W_TMA) {"), ("state_mma", "} else if (warp == W_STATE) {"),
            ("intra_mma", "} else if (OUT && warp == W_INTRA) {"), ("gate", "} else if (warp == W_GATE) {"),
            ("weight", "} else if (OUT ? wg == 0 : wg < 4) {"), (None, "} else if (!OUT && wg == 4) {"),
            ("mask", "} else if (OUT && wg == 1) {"), ("state", "} else if (OUT && wg == 2) {"),
            ("out", "} else if (OUT && (wg == 3 || wg == 4)) {"), (None, "    tc::tc_fence_before();\n    __syncthreads();\n    if (tid == 0 && abort_flag)")]


def code():
    """{role: its code}, without what only the first pass (no output) runs."""
    with open(SRC) as f:
        src = f.read()
    at = [src.index(start) for _, start in SECTIONS]
    assert at == sorted(at)
    out = {}
    for (role, _), a, b in zip(SECTIONS, at, at[1:]):
        if role:
            out[role] = "\n".join(line for line in src[a:b].split("\n") if "if (!OUT" not in line)
    return src, out


def steps(role, n, N, dots):
    """What a role does for chunk n, in order: ("wait" / "arrive", barrier, number of its phase), ("read" / "write", buffer, chunk).
    A buffer is named with its copy; a phase of one of several barriers is that of the chunk or batch it stands for."""
    def wait(bar, k):
        return [("wait", bar, k)] if k >= 0 else []

    def gate():
        return wait("gready", n // GB) if n % GB == 0 else []

    no1 = 1 if dots else 2
    last = n % GB == GB - 1
    tile = [("x%d" % (n % NS), n), ("y%d" % (n % NS), n), ("z%d" % (n % NS), n)]
    if role == "tma":
        return wait("free_s", n - NS) + [("write",) + t for t in tile] + [("arrive", "full", n)]
    if role == "state_mma":
        return (wait("full", n) + wait("s_ready", n) + wait("o_free", n - no1) +
                [("read",) + tile[0], ("read", "h", n), ("write", "o1_%d" % (n % no1), n), ("arrive", "o1done", n)] + wait("y_ready", n) +
                [("read",) + tile[2], ("read", "w%d" % (n % 2), n), ("read", "l", n)] +
                [("arrive", b, n) for b in ("d2done", "y_free", "l_free", "free_s")])
    if role == "intra_mma":  # the products P of chunk n + 1 before O2 of chunk n
        def p(m):
            s = m % NS
            return wait("full", m) + [("read", "x%d" % s, m), ("read", "y%d" % s, m), ("write", "p%d" % (m % 2), m), ("arrive", "pdone", m)]

        return ((p(0) if n == 0 else []) + (p(n + 1) if n + 1 < N else []) + wait("p_ready", n) + wait("o_free", n - 1) +
                [("read",) + tile[2], ("read", "dp", n), ("write", "o2", n)] + [("arrive", b, n) for b in ("o2done", "o2read", "free_s")])
    if role == "gate":
        if n % GB:
            return []
        b = n // GB
        return (wait("gfree", b - 2) + [("write", "slot%d" % (m % SLOTS), m) for m in range(n, min(n + GB, N))] + [("arrive", "gready", b)])
    slot = ("read", "slot%d" % (n % SLOTS), n)
    free = [("arrive", "gfree", n // GB)] if last else []
    if role == "weight":
        return (gate() + wait("full", n) + wait("y_free", n - 2) + [("read",) + tile[1], slot, ("write", "w%d" % (n % 2), n)] +
                wait("l_free", n - 1) + [("write", "l", n), ("arrive", "y_ready", n)] + free)
    if role == "mask":
        return (gate() + wait("pdone", n) + [slot, ("read", "p%d" % (n % 2), n)] + wait("o2done", n - 1) +
                [("write", "dp", n), ("arrive", "p_ready", n)])
    if role == "state":
        return wait("d2done", n - 1) + gate() + [slot, ("write", "h", n), ("arrive", "s_ready", n)]
    assert role == "out"
    load = wait("dread", n - 1) + [("write", "d", n), ("arrive", "dfull", n)] if dots else []
    use = wait("dfull", n) + [("read", "d", n), ("arrive", "dread", n)] if dots else []
    return (load + gate() + wait("o1done", n) + wait("o2read", n) + [("read", "o1_%d" % (n % no1), n), ("read", "o2", n), ("arrive", "o_free", n)] +
            [slot] + free + use)


ROLES = ("tma", "state_mma", "intra_mma", "gate", "weight", "mask", "state", "out")
WARPS = {"weight": 4, "mask": 4, "state": 4, "out": 8}


def graph(N, dots, drop=()):
    """(predecessors of every event, reads, writes); drop: (role, barrier) whose arrivals are left out."""
    events, arrivals = [], {}
    for role in ROLES:
        line = [(role, n, s) for n in range(N) for s in steps(role, n, N, dots) if (role, s[1]) not in drop or s[0] != "arrive"]
        events.append(line)
        for e in line:
            if e[2][0] == "arrive":
                arrivals.setdefault(e[2][1:], []).append(e)
    pred = {}
    for line in events:
        for i, e in enumerate(line):
            pred[e] = [line[i - 1]] if i else []
            if e[2][0] == "wait":
                pred[e] += arrivals[e[2][1:]]
    return pred


def before(pred):
    """The events that come before each event; fails on a cycle."""
    done, left, out = set(), dict(pred), {}
    order = {e: i for i, e in enumerate(pred)}
    while left:
        ready = [e for e, p in left.items() if all(x in done for x in p)]
        assert ready, "roles wait for one another"
        for e in ready:
            bits = 0
            for p in pred[e]:
                bits |= out[p] | 1 << order[p]
            out[e] = bits
            done.add(e)
            del left[e]
    return out, order


def hazards(N, dots, drop=()):
    pred = graph(N, dots, drop)
    out, order = before(pred)
    uses = {}
    for e in pred:
        if e[2][0] in ("read", "write"):
            uses.setdefault(e[2][1], {}).setdefault(e[2][2], {"read": [], "write": []})[e[2][0]].append(e)
    bad = []
    for buf, by in uses.items():
        chunks = sorted(by)
        for a in chunks:
            bad += [("read before written", buf, a, r[0]) for r in by[a]["read"] for w in by[a]["write"] if not out[r] >> order[w] & 1]
        for a, b in zip(chunks, chunks[1:]):
            bad += [("written over before read", buf, a, r[0]) for w in by[b]["write"] for r in by[a]["read"] + by[a]["write"]
                    if not out[w] >> order[r] & 1]
    return bad


@pytest.mark.parametrize("dots", [False, True])
def test_every_buffer_is_read_before_it_is_written_again(dots):
    for N in (1, 2, 4, 7, 8, 9, 25, 32):
        assert not hazards(N, dots)


def test_the_weights_must_release_their_slots():
    """The model sees a missing arrival: without the weight warps' on gfree, the last chunk of a batch is written over."""
    bad = hazards(25, False, drop={("weight", "gfree")})
    assert bad and {(x[0], x[3]) for x in bad} == {("written over before read", "weight")}
    assert all(b[2] % GB == GB - 1 for b in bad)


def test_the_model_is_the_source():
    src, roles = code()
    for role in ROLES:
        mine = [s for N in (25,) for n in range(N) for s in steps(role, n, N, True)]
        text = roles[role]
        waits = set(re.findall(r"(?<!mbar_)wait(?:_all)?\(&bars\.(\w+)", text)) | ({"gready"} if "wait_gate(" in text else set())
        assert waits == {s[1] for s in mine if s[0] == "wait"}, role
        arrives = set(re.findall(r"(?:mbar_arrive|mma_commit|warp_arrive|mbar_expect_tx)\(&bars\.(\w+)", text)) - {"drain"}
        if role == "state_mma":
            arrives -= {"pdone"}  # the first pass's
        assert arrives == {s[1] for s in mine if s[0] == "arrive"}, role


def test_arrivals_are_counted():
    """A phase of gfree takes one arrival from each warp that arrives on it."""
    src, roles = code()
    count = re.search(r"i < BARS_GATE \? \(OUT \? (\d+) : 16\)", src)
    assert count and int(count.group(1)) == sum(WARPS[r] for r in ROLES if r in WARPS and "mbar_arrive(&bars.gfree" in roles[r])


def test_no_role_waits_without_a_bound():
    """Once the roles' loops run, a warp that has given up and left meets the others again at the kernel's end only: no
    other barrier of the whole block or of a group, which waits for those that have left."""
    _, roles = code()
    for role, text in roles.items():
        assert not re.search(r"named_bar_sync|__syncthreads|bar\.sync|barrier\.", text), role
        for call in re.findall(r"tc::mbar_wait\(.*", text):  # what is in flight lands: bounded
            assert "budget" in call, (role, call)


def test_a_warp_gives_up_as_one():
    """The answer of a wait is the same in every lane: what follows takes whole warps."""
    with open(SRC) as f:
        src = f.read()
    wait = src[src.index("bool wait_longer("):src.index("// 16 lanes x 16 columns")]
    for call in re.findall(r".*try_wait\(addr.*", wait):
        assert "__all_sync(0xffffffffu, try_wait(addr, parity))" in call, call
    assert re.search(r"if \(__any_sync\(0xffffffffu, [^;]*\*abort_flag\)\) return false;", wait)
    assert wait.count("return false") == 1
