"""The pick of a row's best blocks (csrc/pick.cuh), run on the CPU thread by thread.

What a CTA finds in the workspace is sound unless a wait of the call ran into its
limit, or another call used the workspace meanwhile; then the selection is not
valid, but nothing may be written outside the row's own ids.  Such data cannot be
made on a GPU by a call that is allowed, so the device functions run here, on keys
and scores that do not agree with each other.
"""

import os
import random
import shutil
import struct
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
UNWRITTEN = -7


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("pick") / "pick")
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", exe, os.path.join(HERE, "pick_on_cpu.cpp")],
                   check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.returncode
        return [list(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


def order(f):
    """A float's key: its order as a whole number above 0."""
    if f != f:
        return 1
    u = struct.unpack("I", struct.pack("f", f + 0.0))[0]
    return ~u & 0xFFFFFFFF if u >> 31 else u | 1 << 31


def bits(f):
    return struct.unpack("I", struct.pack("f", f))[0]


def row(n_vis, take, first, last):
    need = 0 if take == n_vis else take - first - last
    return [n_vis, take, first, n_vis - last, need]


def wanted(n_vis, take, first, last, keys, ids):
    need = take - first - last
    best = sorted(range(len(ids)), key=lambda i: (-keys[i], ids[i]))[:need]
    return sorted(set(range(first)) | set(range(n_vis - last, n_vis)) | {ids[i] for i in best})


def scores_of(rnd, n, kind):
    if kind == "ties":
        return [float(rnd.randint(-2, 2)) for _ in range(n)]
    if kind == "near":
        return [1.0 + rnd.randint(0, 9) * 2.0 ** -23 for _ in range(n)]
    return [rnd.gauss(0, 100) for _ in range(n)]


@pytest.mark.parametrize("kind", ["ties", "near", "spread"])
@pytest.mark.parametrize("fill", [0, 255])
def test_sound_data_give_the_best(pick, kind, fill):
    rnd = random.Random(kind)
    cases, want = [], []
    for n_vis, take, first, last in ((30, 7, 1, 2), (500, 33, 0, 1), (3000, 200, 4, 9),
                                     (3000, 5, 2, 3), (70000, 40, 1, 1)):
        ids = list(range(first, n_vis - last))
        if n_vis > 5000:
            ids = sorted(rnd.sample(ids, 900))
        keys = [order(x) for x in scores_of(rnd, len(ids), kind)]
        want.append(wanted(n_vis, take, first, last, keys, ids))
        r = row(n_vis, take, first, last)
        # (with the limits as wide as a call may give them, and as narrow)
        for least, most in ((1, max(keys)), (min(keys), max(keys))):
            cases.append([0, *r, take, len(ids), least, most, fill, 2 * len(ids), *keys, *ids])
        if n_vis <= 5000:
            s = [0.0] * n_vis
            for i, x in zip(ids, scores_of(rnd, len(ids), kind)):
                s[i] = x
            want.append(wanted(n_vis, take, first, last, [order(s[i]) for i in ids], ids))
            cases.append([1, *r, take, 0, 0, 0, fill, n_vis, *map(bits, s)])
    got = pick(cases)
    want = iter(want)
    for c, g in zip(cases, got):
        take = c[2]
        if c[0] == 1 or c[8] == 1:
            w = next(want)
        assert g[:take] == w, (c[:12], g[:take], w)
        assert all(x == UNWRITTEN for x in g[take:])


def unsound(rnd):
    """Keys of which fewer than are needed lie within the limits."""
    n_vis, take, first, last = 900, 40, 1, 2
    n = 600
    ids = rnd.sample(range(first, n_vis - last), n)
    least, most = order(1.0), order(2.0)
    where = rnd.choice(["below", "just_below", "above", "split", "zero", "one_value"])
    if where == "below":
        keys = [order(rnd.uniform(-9, 0.9)) for _ in ids]
    elif where == "just_below":
        keys = [least - 1 - rnd.randint(0, 9) for _ in ids]
    elif where == "above":
        keys = [order(rnd.uniform(2.1, 1e30)) for _ in ids]
    elif where == "split":
        keys = [rnd.choice([order(0.5), order(1.5) if rnd.random() < 0.02 else order(3.0)])
                for _ in ids]
    elif where == "zero":
        keys = [0] * n
    else:
        keys = [order(1.5)] * 5 + [order(7.0)] * (n - 5)
    return n_vis, take, first, last, ids, keys, least, most


def test_keys_outside_their_limits_stay_in_the_row(pick):
    rnd = random.Random(5)
    cases = []
    for i in range(150):
        n_vis, take, first, last, ids, keys, least, most = unsound(rnd)
        fill = (0, 255, 0x7F, 1, rnd.randint(0, 255))[i % 5]
        cases.append([0, *row(n_vis, take, first, last), take, len(ids), least, most, fill,
                      2 * len(ids), *keys, *ids])
    for c, g in zip(cases, pick(cases)):
        take, n_vis = c[2], c[1]
        assert all(x == UNWRITTEN for x in g[take:]), c[:12]
        assert all(x == UNWRITTEN or 0 <= x < n_vis for x in g[:take])


def test_scores_that_change_stay_in_the_row(pick):
    rnd = random.Random(6)
    cases = []
    for kind in ("up", "level", "same", "nan"):
        for fill in (0, 255):
            n_vis, take, first, last = 700, 30, 2, 3
            a = [rnd.gauss(0, 1) for _ in range(n_vis)]
            b = {"up": [x + 100 for x in a], "level": [max(a)] * n_vis, "same": a,
                 "nan": [float("nan")] * n_vis}[kind]
            cases.append([2, *row(n_vis, take, first, last), take, 0, 0, 0, fill, 2 * n_vis,
                          *map(bits, a), *map(bits, b)])
    for c, g in zip(cases, pick(cases)):
        assert all(x == UNWRITTEN for x in g[c[2]:]), c[:12]


def test_areas_fit_what_is_launched(pick):
    """The places of a CTA's shared memory follow one another, the ids' bits in whole
    16-byte words, and end within the bytes of the launch, whatever the call."""
    rnd = random.Random(7)
    cases = []
    for n_vis in (1, 2, 127, 128, 129, 4096, 24576, 24577, 65536, 65537, 250001, 2 ** 29):
        for take in (1, 2, 33, 128, 1500, 2048):
            for n in {0, 1, n_vis // 2, n_vis - 1, rnd.randint(0, n_vis)}:
                cases += [(n_vis, take, n, 0, 0), (n_vis, take, n, 1, 0)]
            cases += [(n_vis, take, 0, 0, take << s) for s in range(4)]
    lines = pick([[3, n_vis, take, maxima, expected, 0, 0, n, 0, 0, 0, 0]
                  for n_vis, take, n, maxima, expected in cases])
    for (n_vis, take, n, maxima, expected), line in zip(cases, lines):
        key, ident, groups, reach, size, room, room_groups, room_reach, most, static = line
        assert key % 4 == 0 and 32 * key >= min(n_vis, 65536)
        assert min(room, room_groups, room_reach) >= 0
        assert ident == key + room and groups == ident + room and reach == groups + room_groups
        assert size == 4 * (reach + room_reach) <= most
        # Beside the kernels' own shared memory (at most this and two lists of 320).
        assert most + static + 2 * 320 * 4 <= 232448
        if maxima:
            assert room >= take and room_reach >= take
            assert room_groups == 0 if n == 0 else 0 < room_groups <= (n + 7) // 8


def test_no_read_only_loads_in_dependent_kernels():
    """The selection's kernels start before the kernel ahead of them has ended, so
    what it writes is not read-only for their lifetime: no load says that it is."""
    path = os.path.join(HERE, "..", "long_context_causal_gqa_gb300", "csrc")
    for name in ("select_blocks.cu", "pick.cuh", "pair_mma.cuh"):
        with open(os.path.join(path, name)) as f:
            text = f.read()
        assert not [w for w in ("__ldg", "global.nc", "__restrict__") if w in text], name
