"""GPU tests of attention over the 4-bit cache and of sliding windows with sinks.

Every output is held to window_reference.attend's bound, value by value.
"""

import random

import numpy as np
import pytest
import torch

import window_reference as ref
from cache_reference import E4M3

pytestmark = pytest.mark.gpu


class Tails:
    """A batch's caches (4-bit or E4M3) and queries, and the plain form over them."""

    def __init__(self, fp4, R, Hq, Hkv, D, page, lens, seed=0, max_ctx=None):
        self.fp4, self.R, self.Hq, self.Hkv, self.D, self.page = fp4, R, Hq, Hkv, D, page
        self.lens, self.B = list(lens), len(lens)
        self.max_ctx = max_ctx or max(max(lens), 1)
        rnd = np.random.default_rng(seed)
        stride = -(-self.max_ctx // page)
        pages = self.B * stride + 2
        self.tables = rnd.permutation(pages)[: self.B * stride].reshape(self.B, stride)
        self.ks, self.vs = 0.03125, 0.02
        self.k, self.v = (rnd.standard_normal((self.B, self.max_ctx, Hkv, D)) for _ in "kv")
        self.pages = pages
        self.q = rnd.standard_normal((self.B, R, Hq, D)).astype(np.float16)
        self.store()

    def store(self):
        """The caches, with NaN wherever no context reaches; k and v as stored."""
        D, page = self.D, self.page
        self.caches = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            if self.fp4:
                rows = ref.encode_rows((x / s).astype(np.float32))
                x[...] = ref.decode_rows(rows, D) * s
                c = np.full((self.pages, self.Hkv, page, 9 * D // 16), 0xFF, np.uint8)
            else:
                rows = torch.from_numpy(np.clip(x / s, -448, 448)).to(torch.float8_e4m3fn) \
                    .view(torch.uint8).numpy()
                x[...] = E4M3[rows] * s
                c = np.full((self.pages, page, self.Hkv, D), 0x7F, np.uint8)
            for b, n in enumerate(self.lens):
                t = np.arange(n)
                at = self.tables[b, t // page], t % page
                if self.fp4:
                    c[at[0], :, at[1]] = rows[b, :n]
                else:
                    c[at] = rows[b, :n]
            self.caches.append(c)

    def args(self, lens=None):
        dev = torch.device("cuda")
        one = lambda x: torch.tensor([x], dtype=torch.float32, device=dev)  # noqa: E731
        ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
        return [torch.from_numpy(self.q).to(dev), *(torch.from_numpy(c).to(dev) for c in self.caches),
                one(self.ks), one(self.vs), ints(self.tables), ints(lens or self.lens), self.max_ctx]

    def run(self, lib, window, sinks, scale, args=None, **kw):
        args = args or self.args()
        if self.fp4:
            return lib.paged_fp4(*args, scale=scale, window=window, sinks=sinks, **kw)
        return lib.paged_e4m3_window(*args, window, sinks=sinks, scale=scale, **kw)

    def check(self, out, window, sinks, scale, only=None):
        out = out.cpu().double().numpy()
        G = self.Hq // self.Hkv
        for b in range(self.B) if only is None else only:
            n = self.lens[b]
            see = ref.visible(range(n - self.R, n), n, window, sinks)
            for h in range(self.Hq):
                want, bound = ref.attend(self.q[b, :, h], self.k[b, :n, h // G],
                                         self.v[b, :n, h // G], see, scale)
                d = np.abs(out[b, :, h] - want)
                assert (d <= bound).all(), (b, h, float((d - bound).max()), float(d.max()))


TAILS = [
    # R, Hq, Hkv, D, page, lens, window, sinks
    (1, 6, 1, 256, 16, [1], 0, 0),
    (1, 6, 1, 256, 16, [0, 17, 128, 129, 0, 1000], 0, 0),
    (2, 6, 2, 128, 8, [1, 2, 3, 130, 777], 0, 0),
    (8, 6, 1, 256, 32, [5, 300, 2049], 0, 0),                  # 48 packed rows, one context short
    (5, 8, 4, 128, 64, [700, 64], 0, 0),
    (3, 12, 4, 256, 256, [513, 256, 255], 0, 0),
    (48, 4, 4, 128, 16, [60, 20], 0, 0),                       # one head a KV head, 48 rows
    (1, 64, 4, 128, 16, [333], 0, 0),
    (1, 6, 1, 256, 16, [1], 1, 0),
    (1, 6, 1, 256, 16, [0, 700, 129, 128], 1, 3),
    (1, 6, 1, 256, 16, [5000, 4096, 100], 1000, 4),
    (4, 6, 1, 256, 8, [3, 900, 513], 2, 1),                    # a window shorter than the rows
    (2, 16, 4, 128, 16, [640, 1500, 130], 129, 127),
    (2, 16, 4, 128, 128, [640, 1500, 130], 128, 128),
    (2, 16, 2, 128, 256, [640, 1500, 257], 127, 129),
    (3, 6, 1, 256, 64, [2000, 333], 500, 900),                 # sinks that reach far
    (1, 6, 2, 128, 16, [400, 50], 10 ** 6, 7),                 # a window longer than any context
    (7, 6, 1, 128, 16, [1024, 1025, 6], 256, 2 ** 31 - 1),     # sinks hold everything
    (6, 8, 1, 128, 32, [900, 901], 33, 5),                     # 48 packed rows
]


# (The E4M3 tails without a window are another entry point.)
@pytest.mark.parametrize("case,fp4", [(c, f) for c in TAILS for f in (True, False) if f or c[6]])
def test_tails(cuda_lib, case, fp4):
    R, Hq, Hkv, D, page, lens, window, sinks = case
    t = Tails(fp4, R, Hq, Hkv, D, page, lens, seed=R * 100 + len(lens) + window)
    scale = D ** -0.5
    args = t.args()
    out = t.run(cuda_lib, window, sinks, scale, args,
                out=torch.full(t.q.shape, float("nan"), dtype=torch.float16, device="cuda"))
    assert cuda_lib.device_error() == 0
    t.check(out, window, sinks, scale)
    assert torch.equal(out, t.run(cuda_lib, window, sinks, scale, args))


@pytest.mark.parametrize("fp4", [True, False])
def test_many_sequences(cuda_lib, fp4):
    """More sequences than SMs, many of them empty, and more units than cuts."""
    rnd = random.Random(5)
    lens = [rnd.choice([0, 0, 1, 40, 129, rnd.randint(1, 700)]) for _ in range(300)]
    t = Tails(fp4, 1, 4, 2, 128, 16, lens, seed=9)
    out = t.run(cuda_lib, 200, 3, 0.09)
    assert cuda_lib.device_error() == 0
    t.check(out, 200, 3, 0.09)


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("R,Hq,Hkv,D", [(2, 16, 2, 128), (3, 6, 1, 256), (4, 6, 1, 256)])
def test_wide_rows_of_many_sequences(cuda_lib, fp4, R, Hq, Hkv, D):
    """Two to four eights of packed rows, more sequences than a warp's lanes, cut anywhere."""
    rnd = random.Random(R)
    lens = [rnd.choice([0, 1, 2, 700, rnd.randint(1, 1500)]) for _ in range(70)]
    t = Tails(fp4, R, Hq, Hkv, D, 16, lens, seed=R)
    out = t.run(cuda_lib, 900, 5, 0.07)
    assert cuda_lib.device_error() == 0
    t.check(out, 900, 5, 0.07, only=range(0, 70, 3))


@pytest.mark.parametrize("fp4", [True, False])
def test_one_long_sequence_among_many(cuda_lib, fp4):
    """Its unit is cut into almost all ranges, while most are whole: more pieces than the
    join takes at a time."""
    t = Tails(fp4, 1, 2, 1, 128, 16, [3] * 40 + [30000] + [3] * 39, seed=4)
    out = t.run(cuda_lib, 29000, 2, 0.09)
    assert cuda_lib.device_error() == 0
    t.check(out, 29000, 2, 0.09)


def test_most_sequences(cuda_lib):
    lens = [(7 * b) % 50 for b in range(1024)]
    t = Tails(True, 1, 1, 1, 128, 8, lens, seed=2)
    out = t.run(cuda_lib, None, 0, 0.09)
    t.check(out, 0, 0, 0.09, only=[0, 1, 5, 511, 1000, 1022, 1023])
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("shape", ["ramp", "one key", "equal"])
def test_scores_that_move_the_reference(cuda_lib, shape, fp4):
    t = Tails(fp4, 2, 6, 1, 256, 16, [3000], seed=4)
    t.q[...] = np.float16(1) + np.arange(6)[:, None] * np.float16(0.125)
    s = np.zeros(3000)
    if shape == "ramp":
        s = (np.arange(3000) % 512) * 0.1
    elif shape == "one key":
        s[1234] = 30.0
    t.k[0, :, 0] = s[:, None] / 16 + 0.01 * t.k[0, :, 0]
    t.ks = 0.25 / 64 if fp4 else 0.01
    t.store()
    for window, sinks in ((0, 0), (2000, 130)):
        if window or fp4:
            t.check(t.run(cuda_lib, window, sinks, 1 / 16), window, sinks, 1 / 16)
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("fp4", [True, False])
def test_keys_no_row_sees_may_hold_anything(cuda_lib, fp4):
    t = Tails(fp4, 3, 6, 1, 256, 16, [1000, 500], seed=6)
    window, sinks = 150, 20
    args = t.args()
    clean = t.run(cuda_lib, window, sinks, 1 / 16, args)
    # NaN bytes in all of them, and table entries of whole unseen tiles out of range.
    for b, n in enumerate(t.lens):
        for p in range(sinks, n - 3 - window + 1):
            for c in args[1:3]:
                pg = t.tables[b, p // 16]
                (c[pg, :, p % 16] if fp4 else c[pg, p % 16]).fill_(0xFF)
    args[5][0, 8:48] = 10 ** 6          # tokens 128 .. 767: tiles 1 .. 5
    args[5][0, 63:] = -5                # behind the context's last page
    assert torch.equal(t.run(cuda_lib, window, sinks, 1 / 16, args), clean)
    assert cuda_lib.device_error() == 0


def test_a_nan_reaches_only_the_rows_that_see_it(cuda_lib):
    t = Tails(True, 4, 6, 2, 128, 16, [300, 140], seed=8)
    args = t.args()
    clean = t.run(cuda_lib, 100, 2, 0.1, args).clone()
    for cache in (1, 2):
        for key, rows in ((298, (2, 3)), (198, (0, 1))):   # row r sits at 296 + r, window 100
            kept = args[cache].clone()
            args[cache][t.tables[0, key // 16], 0, key % 16, 64:] = 0x7F
            out = t.run(cuda_lib, 100, 2, 0.1, args)
            bad = torch.zeros(2, 4, 6, dtype=torch.bool)
            bad[0, list(rows), :3] = True                  # the first KV head's queries
            bad = bad.cuda()
            assert torch.isnan(out[bad]).all(), (cache, key)
            assert torch.equal(out[~bad], clean[~bad]) or \
                (out[~bad].float() - clean[~bad].float()).abs().max() <= 2.0 ** -9
            args[cache].copy_(kept)
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("fp4", [True, False])
def test_bad_contexts_and_pages_are_flagged(cuda_lib, fp4):
    t = Tails(fp4, 2, 6, 1, 256, 16, [100, 90, 80], seed=3)
    args = t.args()
    args[6] = torch.tensor([101, -7, 80], dtype=torch.int32, device="cuda")
    out = t.run(cuda_lib, 64, 2, 1 / 16, args)
    assert cuda_lib.device_error() == cuda_lib.DEVERR_BAD_CTX_LEN
    t.check(out, 64, 2, 1 / 16, only=[0, 2])     # 101 counts as the bound, 100
    assert not out[1].any()
    args = t.args()
    args[5][0, 6] = t.pages                      # the last page of sequence 0
    args[1][0] = 0                               # page 0 is read in its place
    args[2][0] = 0
    out = t.run(cuda_lib, 64, 2, 1 / 16, args)
    assert cuda_lib.device_error() == cuda_lib.DEVERR_BAD_PAGE_ID
    t.check(out, 64, 2, 1 / 16, only=[b for b in (1, 2) if 0 not in t.tables[b]])
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("fp4", [True, False])
def test_replay_while_contexts_change(cuda_lib, fp4):
    """One captured graph over contexts from nothing to the bound, and eager calls
    between replays: the same bits.  A second graph shares the workspace."""
    t = Tails(fp4, 2, 6, 1, 256, 16, [600, 600], seed=11)
    args = t.args()
    out, other = (torch.zeros(t.q.shape, dtype=torch.float16, device="cuda") for _ in "ab")
    run = lambda o: t.run(cuda_lib, 300, 5, 1 / 16, args, out=o)  # noqa: E731
    run(out)
    graphs = []
    for o in (out, other):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(o)
    for lens in ((600, 600), (0, 1), (2, 0), (129, 600), (305, 431)):
        args[6].copy_(torch.tensor(lens))
        for g in graphs:
            g.replay()
        eager = run(None)
        assert torch.equal(out, eager) and torch.equal(other, eager)
        t.lens = list(lens)
        t.check(eager, 300, 5, 1 / 16)
    assert cuda_lib.device_error() == 0


def test_window_as_long_as_the_context_is_the_whole(cuda_lib):
    t = Tails(False, 2, 6, 1, 256, 16, [700, 333], seed=12)
    args = t.args()
    whole = cuda_lib.paged_e4m3_batch(*args, scale=1 / 16)
    got = cuda_lib.paged_e4m3_window(*args, 700, scale=1 / 16)
    # The same tiles; the splits may be fewer.
    assert (whole.float() - got.float()).abs().max() <= 2.0 ** -9
    f = Tails(True, 2, 6, 1, 256, 16, [700, 333], seed=12)
    a, b = (f.run(cuda_lib, w, 9, 1 / 16) for w in (None, 700))
    assert torch.equal(a, b)


def test_another_stream(cuda_lib):
    t = Tails(True, 1, 6, 1, 256, 16, [900], seed=13)
    args = t.args()
    want = t.run(cuda_lib, 100, 4, 1 / 16, args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = t.run(cuda_lib, 100, 4, 1 / 16, args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_binding_refuses(cuda_lib):
    t = Tails(True, 1, 6, 1, 256, 16, [90], seed=1)
    args = t.args()
    bad = [
        (0, args[0].float()), (0, args[0][:, :, :, :128].contiguous()), (1, args[1].int()),
        (1, args[1][..., :143].contiguous()), (2, args[2][:1]), (3, args[3].double()),
        (5, args[5].long()), (5, args[5][0]), (6, args[6].repeat(2)), (7, 97), (7, 2.5),
    ]
    for i, x in bad:
        a = list(args)
        a[i] = x
        with pytest.raises(cuda_lib.GQAError) as e:
            t.run(cuda_lib, 8, 0, 1 / 16, a)
        assert e.value.status in (cuda_lib.GQA_ERR_INVALID_ARG, cuda_lib.GQA_ERR_UNSUPPORTED), i
    for kw in (dict(window=-1), dict(sinks=-1), dict(window="x"), dict(scale=0.0),
               dict(out=args[0].float()), dict(out=args[0][0])):
        with pytest.raises(cuda_lib.GQAError):
            cuda_lib.paged_fp4(*args, **kw)
    q = torch.zeros(4, 6, 256, dtype=torch.float16, device="cuda")
    k = torch.zeros(8, 1, 256, dtype=torch.float16, device="cuda")
    for a in ((q.float(), k, k, 4), (q, k[:, :, :128].contiguous(), k, 4), (q, k, k[:7], 4),
              (q, k, k, 0), (q, k[:3], k[:3], 4), (q, k, k, None)):
        with pytest.raises(cuda_lib.GQAError):
            cuda_lib.prefill_window(*a)


# ---------------------------------------------------------------- the prefill

PREFILLS = [
    # Q, KV, Hq, Hkv, D, window, sinks
    (1, 1, 6, 1, 256, 1, 0),
    (1, 400, 6, 1, 256, 1, 0),
    (5, 9, 6, 1, 256, 3, 1),
    (100, 333, 6, 1, 256, 64, 0),
    (100, 333, 6, 1, 128, 64, 4),
    (256, 1024, 6, 1, 256, 128, 128),
    (257, 1025, 6, 2, 256, 129, 127),
    (300, 900, 8, 4, 128, 200, 129),
    (700, 700, 6, 1, 256, 100, 10),          # from the first token on
    (64, 2000, 6, 1, 256, 500, 1490),        # sinks that reach the window
    (64, 2000, 6, 1, 128, 500, 1400),        # ... and end just in front of it
    (200, 1500, 3, 3, 128, 1, 300),
    (333, 600, 6, 1, 256, 599, 0),
    (40, 600, 6, 1, 256, 250, 2 ** 31 - 1),
    (1000, 3000, 6, 1, 256, 700, 16),        # cut pair tiles
]


def prefill_inputs(Q, KV, Hq, Hkv, D, e4m3, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(Q, Hq, D, generator=g).half()
    k, v = (torch.randn(KV, Hkv, D, generator=g) for _ in "kv")
    if e4m3:
        k, v = ((x * 64).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        kf, vf = (E4M3[x.numpy()] / 64 for x in (k, v))
    else:
        k, v = k.half(), v.half()
        kf, vf = k.double().numpy(), v.double().numpy()
    return q, k, v, kf, vf


def run_prefill(lib, q, k, v, window, sinks, scale):
    dev = torch.device("cuda")
    if k.dtype == torch.uint8:
        s = torch.tensor([1 / 64], device=dev)
        return lib.prefill_e4m3_window(q.to(dev), k.to(dev), v.to(dev), s, s, window, sinks=sinks,
                                       scale=scale)
    return lib.prefill_window(q.to(dev), k.to(dev), v.to(dev), window, sinks=sinks, scale=scale)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", PREFILLS)
def test_prefill_window(cuda_lib, case, e4m3):
    Q, KV, Hq, Hkv, D, window, sinks = case
    q, k, v, kf, vf = prefill_inputs(Q, KV, Hq, Hkv, D, e4m3, Q + KV + window)
    scale = D ** -0.5
    out = run_prefill(cuda_lib, q, k, v, window, sinks, scale)
    assert cuda_lib.device_error() == 0
    assert torch.equal(out, run_prefill(cuda_lib, q, k, v, window, sinks, scale))
    got = out.cpu().double().numpy()
    rows = sorted(set(list(range(min(Q, 40))) + list(range(max(0, Q - 40), Q)) +
                      list(range(0, Q, 17))))
    see = ref.visible([KV - Q + r for r in rows], KV, window, sinks)
    for h in sorted({0, Hq // 2, Hq - 1}):
        want, bound = ref.attend(q[rows, h].numpy(), kf[:, h // (Hq // Hkv)],
                                 vf[:, h // (Hq // Hkv)], see, scale)
        d = np.abs(got[rows, h] - want)
        assert (d <= bound).all(), (h, float((d - bound).max()), float(d.max()))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hkv", [1, 2])
def test_prefill_never_reads_unseen_keys(cuda_lib, Hkv, e4m3):
    q, k, v, _, _ = prefill_inputs(130, 900, 6, Hkv, 128, e4m3, 5)
    clean = run_prefill(cuda_lib, q, k, v, 90, 7, 0.09)
    for x in (k, v):
        x[7:900 - 130 - 90 + 1] = 0x7F if e4m3 else float("nan")
    assert torch.equal(run_prefill(cuda_lib, q, k, v, 90, 7, 0.09), clean)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prefill_with_a_window_of_everything(cuda_lib, e4m3):
    q, k, v, _, _ = prefill_inputs(100, 500, 6, 1, 256, e4m3, 6)
    dev = torch.device("cuda")
    s = torch.tensor([1 / 64], device=dev)
    want = cuda_lib.prefill_e4m3(q.to(dev), k.to(dev), v.to(dev), s, s) if e4m3 else \
        cuda_lib.prefill(q.to(dev), k.to(dev), v.to(dev))
    for window in (500, 2 ** 31 - 1):
        assert torch.equal(run_prefill(cuda_lib, q, k, v, window, 3, 1 / 16), want)


def test_prefill_graph(cuda_lib):
    q, k, v, _, _ = prefill_inputs(300, 1500, 6, 1, 256, False, 7)
    dev = torch.device("cuda")
    q, k, v = q.to(dev), k.to(dev), v.to(dev)
    out = torch.zeros_like(q)
    want = cuda_lib.prefill_window(q, k, v, 400, sinks=4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.prefill_window(q, k, v, 400, sinks=4, out=out)
    g.replay()
    assert torch.equal(out, want)


# ---------------------------------------------------------------- together

def test_a_model_step_over_the_4_bit_cache(cuda_lib):
    """Two layers' worth of a serving step: a prompt written, its rows read back for a
    windowed prefill of its end, then tokens appended one by one and attended, with a
    window and without, from a fused projection."""
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(21)
    n, steps, page, D, Hq, Hkv = 300, 5, 16, 128, 4, 2
    total = n + steps
    qkv = torch.randn(total, Hq + 2 * Hkv, D, generator=g).half().to(dev)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pages = -(-total // page)
    kc, vc = (torch.full((pages, Hkv, page, 72), 0xFF, dtype=torch.uint8, device=dev) for _ in "kv")
    ks, vs = torch.tensor([0.02], device=dev), torch.tensor([0.03], device=dev)
    table = torch.randperm(pages, generator=g).int().to(dev).view(1, -1)
    freq = (1e4 ** (-torch.arange(32) / 32)).float().to(dev)
    w = (1 + 0.1 * torch.randn(D, generator=g)).half().to(dev)

    def write(a, b):
        ctx = torch.tensor([b], dtype=torch.int32, device=dev)
        return ctx, cuda_lib.cache_write_fp4(q[a:b], k[a:b], v[a:b], kc, vc, ks, vs, table, ctx,
                                             total, q_weight=w, k_weight=w, inv_freq=freq)

    def plain(qr, b, window, sinks):
        kd, vd = (ref.decode_rows(x.cpu().numpy()[table[0].cpu().numpy()], D) * float(s)
                  for x, s in ((kc, ks), (vc, vs)))
        kd, vd = (x.transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:b] for x in (kd, vd))
        r = qr.shape[0]
        see = ref.visible(range(b - r, b), b, window, sinks)
        for h in range(Hq):
            yield h, *ref.attend(qr[:, h].cpu().numpy(), kd[:, h // 2], vd[:, h // 2], see,
                                 D ** -0.5)

    ctx, qp = write(0, n)
    kd, vd = cuda_lib.cache_read_fp4(kc, vc, ks, vs, table, ctx, total, n)
    out = cuda_lib.prefill_window(qp[200:].contiguous(), kd, vd, 64, sinks=4, scale=D ** -0.5)
    for h, want, bound in plain(qp[200:], n, 64, 4):
        # The rows read back round by 2^-11 once more, K's through the scores.
        off = bound + 2.0 ** -10 * (1 + np.abs(want)) + 2.0 ** -11 * 8
        assert (np.abs(out[:, h].cpu().numpy() - want) <= off).all()
    for i in range(steps):
        ctx, qd = write(n + i, n + i + 1)
        for window, sinks in ((None, 0), (64, 4)):
            out = cuda_lib.paged_fp4(qd.view(1, 1, Hq, D), kc, vc, ks, vs, table, ctx, total,
                                     scale=D ** -0.5, window=window, sinks=sinks)[0]
            for h, want, bound in plain(qd, n + i + 1, window or 0, sinks):
                assert (np.abs(out[:, h].cpu().double().numpy() - want) <= bound).all()
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("Hkv,D", [(1, 256), (3, 128)])
def test_a_cache_beyond_32_bits(cuda_lib, Hkv, D):
    """Pages on both sides of 2^32 bytes: written, read back and attended as in a small
    cache."""
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(31)
    page, n = 16, 120
    a_page = Hkv * page * 9 * D // 16
    pages = 2 ** 32 // a_page + 9
    big = [torch.zeros(pages, Hkv, page, 9 * D // 16, dtype=torch.uint8, device=dev) for _ in "kv"]
    small = [torch.zeros(8, Hkv, page, 9 * D // 16, dtype=torch.uint8, device=dev) for _ in "kv"]
    k, v = (torch.randn(n, Hkv, D, generator=g).half().to(dev) for _ in "kv")
    q = torch.randn(1, 2, 2 * Hkv, D, generator=g).half().to(dev)
    s = torch.tensor([0.02], device=dev)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    got = []
    for (kc, vc), ids in ((big, [pages - 1, 0, pages - 3, 1, pages - 2, 2 ** 32 // a_page, 5,
                                2 ** 31 // a_page]),
                          (small, range(8))):
        table = torch.tensor([list(ids)], dtype=torch.int32, device=dev)
        cuda_lib.cache_write_fp4(None, k, v, kc, vc, s, s, table, lens, n)
        got.append(list(cuda_lib.cache_read_fp4(kc, vc, s, s, table, lens, n, n)) +
                   [cuda_lib.paged_fp4(q, kc, vc, s, s, table, lens, n, window=w, sinks=3)
                    for w in (None, 70)])
    assert got[0][0].any() and all(torch.equal(a, b) for a, b in zip(*got))
    assert cuda_lib.device_error() == 0


def test_calls_that_overlap_their_launches(cuda_lib):
    """Each call's launch overlaps the kernel in front, whose output it takes: a chain of all
    operators gives the same bits with a wait after every call and without any."""
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(41)
    n, page, D, Hq, Hkv, R = 1200, 16, 256, 6, 1, 2
    pages = n // page
    kv = torch.randn(n, 2 * Hkv, D, generator=g).half().to(dev)
    k, v = kv[:, :Hkv].contiguous(), kv[:, Hkv:].contiguous()
    s = torch.tensor([0.02], device=dev)
    table = torch.randperm(pages, generator=g).int().to(dev).view(1, -1)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    first = torch.randn(R, Hq, D, generator=g).half().to(dev)

    def chain(after):
        caches = [torch.zeros(pages, Hkv, page, 9 * D // 16, dtype=torch.uint8, device=dev)
                  for _ in "kv"]
        codes = [torch.zeros(pages, page, Hkv, D, dtype=torch.uint8, device=dev) for _ in "kv"]
        cuda_lib.cache_write_fp4(None, k, v, *caches, s, s, table, lens, n)
        cuda_lib.cache_write_e4m3(None, k, v, *codes, s, s, table, lens, n)
        x, seen = first, []
        for i in range(12):
            # The rows so far become queries and the last rows' keys of the next call.
            x = cuda_lib.cache_write_fp4(x, x[:, :1], x[:, 1:2], *caches, s, s, table, lens, n)
            after()
            x = cuda_lib.paged_fp4(x[None], *caches, s, s, table, lens, n, window=[None, 300][i % 2],
                                   sinks=i)[0]
            after()
            x = cuda_lib.paged_e4m3_window(x[None], *codes, s, s, table, lens, n, 500, sinks=3)[0]
            after()
            kd, vd = cuda_lib.cache_read_fp4(*caches, s, s, table, lens, n, n)
            after()
            x = cuda_lib.prefill_window(x, kd, vd, 400, sinks=i)
            after()
            x = cuda_lib.paged_e4m3(x, *codes, s, s, table[0], n)
            after()
            x = cuda_lib.prefill_window(x, kd, vd, 100) * 4
            seen.append(x)
        return torch.stack(seen)

    want = chain(torch.cuda.synchronize)
    assert torch.isfinite(want).all() and want.any()
    for _ in range(5):
        assert torch.equal(chain(lambda: None), want)
    assert cuda_lib.device_error() == 0
