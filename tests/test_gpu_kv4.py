"""The attention-side operators on the GPU against their 64-bit definitions
(tests/kv4_ref.py): rotary positions, the append to the paged 4-bit cache and
its read-back, and the attention, at the head layouts, lengths, pages and
masks where they can go wrong.

Tolerances.  Rotated values: one rounding (2^-24 of the value) and the
double arithmetic before it (2^-50 of the pair's magnitude for each turn of
the angle).  The cache: exact.  Attention: kv4_ref.attend."""

import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import gpu_pack, q8 as _q8, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    assert _q8().q8_device_supported(), "device is not gfx950"
    yield
    torch.cuda.synchronize()


@pytest.fixture(scope="module")
def q8():
    return _q8()


def i32(a):
    return to_dev(np.asarray(a, dtype=np.int32))


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def rotated_within(got, x, pos, freq, interleaved, amplitude):
    want = ref.rotate(x, pos, freq, interleaved, amplitude)
    turns = np.abs(np.asarray(pos, dtype=np.float64)) + 2
    big = np.abs(x).max() * 2 * amplitude
    tol = 2.0 ** -24 * np.abs(want) + 2.0 ** -50 * big * turns[:, None, None] + 2.0 ** -149
    return bool((np.abs(got.astype(np.float64) - want) <= tol).all())


# ------------------------------------------------------------------- rotary

ROTARY = [  # rows, heads, dim, rot, interleaved, scaling, x stride - width, y stride - width
    (16, 48, 128, 128, False, "none", 1024, 0),
    (1, 24, 64, 64, False, "none", 0, 0),
    (1, 1, 2, 2, True, "none", 0, 0),
    (3, 2, 6, 4, False, "linear", 1, 3),
    (7, 5, 96, 96, True, "ntk", 5, 0),
    (33, 3, 128, 96, True, "yarn", 7, 1),
    (19, 4, 80, 62, False, "bands", 0, 2),
    (5, 2, 1024, 1022, False, "none", 0, 0),
    (5, 2, 1024, 1024, True, "none", 0, 4),
    (300, 40, 128, 64, False, "yarn", 2048, 0),
    (1025, 9, 64, 64, True, "linear", 0, 0),
]


@pytest.mark.parametrize("rows,heads,dim,rot,inter,scaling,dx,dy", ROTARY)
def test_rotary(q8, rows, heads, dim, rot, inter, scaling, dx, dy):
    rng = np.random.default_rng(rows * 7 + dim)
    w = heads * dim
    x = rng.standard_normal((rows, w + dx), dtype=np.float32)
    pos = rng.integers(-1000, 200000, rows)
    pos[-1] = 2 ** 31 - 1
    freq, amp = q8.rotary_frequencies(rot, 1e6, scaling, 4.0, 8192.0)
    plan = q8.rotary_plan(rot, 1e6, inter, scaling, 4.0, 8192.0)
    X, Y = to_dev(x), torch.full((rows, w + dy), 7.25, device="cuda")
    q8.q8_rotary(X, Y, rows, w + dx, i32(pos), heads, dim, plan, y_stride=w + dy)
    y = host(Y)
    assert (y[:, w:] == 7.25).all()
    assert rotated_within(y[:, :w].reshape(rows, heads, dim), x[:, :w].reshape(rows, heads, dim), pos,
                          freq.numpy(), inter, amp)
    # in place: the same bits, the other columns untouched
    q8.q8_rotary(X, X, rows, w + dx, i32(pos), heads, dim, plan, y_stride=w + dx)
    xi = host(X)
    assert np.array_equal(xi[:, :w].view(np.uint32), y[:, :w].view(np.uint32))
    assert np.array_equal(xi[:, w:], x[:, w:])
    # a row alone: the same bits
    t = rows // 2
    one = torch.empty(1, w, device="cuda")
    q8.q8_rotary(to_dev(x[t:t + 1]), one, 1, w + dx, i32(pos[t:t + 1]), heads, dim, plan)
    assert np.array_equal(host(one)[0].view(np.uint32), y[t, :w].view(np.uint32))


def test_rotary_of_the_plain_kind_is_rope_multi(q8):
    """The unscaled half layout is q8_rope_multi's rotation, within the last
    bit of its own rounding (the two take their frequencies from different
    power functions)."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((16, 7168), dtype=np.float32)
    pos = rng.integers(0, 40000, 16)
    a, b = to_dev(x), to_dev(x)
    q8.q8_rope_multi(a, 16, 7168, i32(pos), 48, 128, 1e6)
    q8.q8_rotary(b, b, 16, 7168, i32(pos), 48, 128, q8.rotary_plan(128, 1e6), y_stride=7168)
    a, b = host(a).astype(np.float64), host(b).astype(np.float64)
    assert (np.abs(a - b) <= 2.0 ** -23 * np.abs(a) + 1e-9).all()


# ------------------------------------------------------------------- append

def random_cache(q8, rng, kv, dim, page, seqs, positions, fill=None):
    """A cache whose pages lie in no order; its memory filled with bytes of
    random garbage (or `fill`)."""
    most = -(-positions // page)
    pool = seqs * most + 2
    table = rng.permutation(pool)[:seqs * most].reshape(seqs, most)
    nbytes = q8.q8_kv4_page_bytes(kv, dim, page) * pool
    if fill is None:
        pages = torch.randint(0, 256, (nbytes,), dtype=torch.uint8, device="cuda")
    else:
        pages = torch.full((nbytes,), fill, dtype=torch.uint8, device="cuda")
    return q8.KV4Cache(pool, page, kv, dim, i32(table), pages=pages)


APPEND = [  # rows, seqs, query heads, kv heads, dim, rot, interleaved, page, extra stride
    (16, 16, 40, 8, 128, 128, False, 64, 0),
    (1, 1, 12, 12, 64, 64, False, 64, 0),
    (37, 3, 0, 2, 32, 32, True, 32, 3),
    (64, 5, 6, 3, 96, 62, False, 96, 1),
    (65, 2, 4, 1, 256, 128, True, 32, 0),
    (21, 4, 5, 5, 160, 0, False, 128, 5),
    (9, 2, 7, 1, 224, 224, False, 64, 2),
    (513, 3, 8, 2, 192, 96, False, 256, 0),
]


@pytest.mark.parametrize("rows,seqs,nq,kv,dim,rot,inter,page,extra", APPEND)
def test_append_then_read(q8, rows, seqs, nq, kv, dim, rot, inter, page, extra):
    rng = np.random.default_rng(rows + dim)
    span = -(-rows // seqs) + 100
    cache = random_cache(q8, rng, kv, dim, page, seqs, span)
    width = (nq + 2 * kv) * dim
    x = (rng.standard_normal((rows, width + extra)) * np.exp(2 * rng.standard_normal((rows, 1)))).astype(np.float32)
    where = rng.permutation(seqs * span)[:rows]  # distinct positions in any order
    seq, pos = where // span, where % span
    plan, freq = None, np.zeros(0)
    if rot:
        plan = q8.rotary_plan(rot, 1e4, inter)
        freq = q8.rotary_frequencies(rot, 1e4)[0].numpy()
    Q = torch.full((rows, nq * dim + 3), 2.5, device="cuda") if nq else None
    q8.q8_kv4_append(cache, to_dev(x), rows, width + extra, i32(seq), i32(pos), rotary=plan,
                     n_q_heads=nq, Q=Q, q_stride=nq * dim + 3)
    K, V = (torch.empty(rows, kv * dim, device="cuda") for _ in range(2))
    q8.q8_kv4_read(cache, i32(seq), i32(pos), rows, K, V)
    h = x[:, :width].reshape(rows, nq + 2 * kv, dim)
    turned = ref.rotate(h[:, :nq + kv], pos, freq, inter)
    want_k = ref.hold(turned[:, nq:].astype(np.float32))
    assert np.array_equal(host(K).reshape(rows, kv, dim), want_k)
    assert np.array_equal(host(V).reshape(rows, kv, dim), ref.hold(h[:, nq + kv:]))
    if nq:
        q = host(Q)
        assert (q[:, nq * dim:] == 2.5).all()
        assert rotated_within(q[:, :nq * dim].reshape(rows, nq, dim), h[:, :nq], pos, freq, inter, 1.0)
    # either output alone
    K2 = torch.empty_like(K)
    q8.q8_kv4_read(cache, i32(seq), i32(pos), rows, K2, None)
    assert torch.equal(K2, K)


def test_append_blocks_at_the_borders(q8):
    """Blocks on the scale rule's border, ties between codes, saturation,
    signs, zeros, subnormal and largest magnitudes, NaN and infinities."""
    rng = np.random.default_rng(11)
    rows, kv, dim = 256, 2, 64
    ties = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    x = rng.choice(ties, (rows, 2 * kv, dim)) * rng.choice([-1, 1], (rows, 2 * kv, dim))
    x = x * np.ldexp(1.0, rng.integers(-140, 122, (rows, 2 * kv, 1)))
    x = x.astype(np.float32)
    x[0] = 0.0
    x[1, :, 0] = 3.4028234e38
    x[2, 0, 5] = np.nan
    x[3, 1, 40] = np.inf
    x[4, 3, 33] = -np.inf
    x[5] = np.nextafter(np.float32(7), np.float32(8))
    x[6] = 7.0
    x[7] = np.nextafter(np.float32(7), np.float32(0))
    x[8] = 1e-45
    cache = random_cache(q8, rng, kv, dim, 32, 1, rows)
    seq, pos = i32(np.zeros(rows)), i32(np.arange(rows))
    q8.q8_kv4_append(cache, to_dev(x.reshape(rows, -1)), rows, 2 * kv * dim, seq, pos)
    K, V = (torch.empty(rows, kv * dim, device="cuda") for _ in range(2))
    q8.q8_kv4_read(cache, seq, pos, rows, K, V)
    want = ref.hold(x)
    assert np.array_equal(host(K).reshape(rows, kv, dim), want[:, :kv], equal_nan=True)
    assert np.array_equal(host(V).reshape(rows, kv, dim), want[:, kv:], equal_nan=True)
    # what the cache holds is held again unchanged
    again = random_cache(q8, rng, kv, dim, 64, 1, rows)
    q8.q8_kv4_append(again, torch.cat([K, V], 1).contiguous(), rows, 2 * kv * dim, seq, pos)
    K2, V2 = torch.empty_like(K), torch.empty_like(V)
    q8.q8_kv4_read(again, seq, pos, rows, K2, V2)
    assert np.array_equal(host(K2), host(K), equal_nan=True)
    assert np.array_equal(host(V2), host(V), equal_nan=True)


def test_rows_outside_the_cache(q8):
    """Idle rows and rows whose slot, position or page lies outside the cache
    write nothing and read as NaN; their queries are rotated all the same."""
    rng = np.random.default_rng(5)
    kv, dim, page = 2, 64, 32
    cache = random_cache(q8, rng, kv, dim, page, 3, 96, fill=0)
    cache.block_table[2, 1] = cache.n_pages
    cache.block_table[2, 2] = -1
    before = cache.pages.clone()
    seq = np.array([0, 0, -1, 3, 2, 2, 1, 2 ** 31 - 1])
    pos = np.array([-1, 96, 0, 0, 32, 95, 2 ** 31 - 1, 0])
    n = seq.size
    x = rng.standard_normal((n, (3 + 2 * kv) * dim), dtype=np.float32)
    Q = torch.empty(n, 3 * dim, device="cuda")
    q8.q8_kv4_append(cache, to_dev(x), n, x.shape[1], i32(seq), i32(pos),
                     rotary=q8.rotary_plan(dim), n_q_heads=3, Q=Q)
    assert torch.equal(cache.pages, before)
    freq = q8.rotary_frequencies(dim)[0].numpy()
    assert rotated_within(host(Q).reshape(n, 3, dim), x[:, :3 * dim].reshape(n, 3, dim), pos, freq, False, 1.0)
    K, V = (torch.zeros(n, kv * dim, device="cuda") for _ in range(2))
    q8.q8_kv4_read(cache, i32(seq), i32(pos), n, K, V)
    assert torch.isnan(K).all() and torch.isnan(V).all()


# ---------------------------------------------------------------- attention

class Step:
    """One attention call on a filled cache, and its definition."""

    def __init__(self, q8, dim, kv, group, tokens, page, lens, window=0, seed=0, scale=None,
                 positions=None, spread=1.0, extra=0, slots=None):
        self.q8, self.window, self.tokens, self.extra = q8, window, tokens, extra
        rng = self.rng = np.random.default_rng(seed + dim + 131 * kv + tokens)
        n = self.n_seq = len(lens)
        self.nq, self.kv, self.dim, self.group = kv * group, kv, dim, group
        self.scale = dim ** -0.5 if scale is None else scale
        n_slots = n + 2 if slots is None else slots
        self.cache = random_cache(q8, rng, kv, dim, page, n_slots, max(max(lens), 1))
        self.slot = rng.permutation(n_slots)[:n]
        self.k = [(spread * rng.standard_normal((L, kv, dim))).astype(np.float32) for L in lens]
        self.v = [rng.standard_normal((L, kv, dim)).astype(np.float32) for L in lens]
        for s, L in enumerate(lens):
            if L:
                self.put(s, np.arange(L), self.k[s], self.v[s])
        self.pos = np.array([[L - tokens + j for j in range(tokens)] for L in lens]
                            if positions is None else positions).reshape(n, tokens)
        self.seq = np.repeat(self.slot, tokens)
        self.q = rng.standard_normal((n * tokens, self.nq * dim + extra), dtype=np.float32)
        self.ws = q8.kv4_attend_workspace(self.cache, n, tokens, self.nq)

    def put(self, s, pos, k, v):
        rows = np.concatenate([k.reshape(len(pos), -1), v.reshape(len(pos), -1)], 1)
        self.q8.q8_kv4_append(self.cache, to_dev(rows.astype(np.float32)), len(pos), rows.shape[1],
                              i32(np.full(len(pos), self.slot[s])), i32(pos))

    def args(self, rows=None):
        rows = slice(None) if rows is None else rows
        return to_dev(self.q[rows]), i32(self.seq[rows]), i32(self.pos.reshape(-1)[rows])

    def run(self, ws=None, n_seq=None, seqs=None):
        """[rows, heads, dim]; seqs: a sublist of the sequences."""
        seqs = np.arange(self.n_seq) if seqs is None else np.asarray(seqs)
        rows = (seqs[:, None] * self.tokens + np.arange(self.tokens)).reshape(-1)
        q, seq, pos = self.args(rows)
        w = self.nq * self.dim
        o = torch.full((rows.size, w + self.extra), 3.5, device="cuda")
        self.q8.q8_kv4_attend(self.cache, q, len(seqs), self.tokens, self.nq, seq, pos, o,
                              self.ws if ws is None else ws, scale=self.scale, window=self.window,
                              q_stride=w + self.extra, o_stride=w + self.extra)
        o = host(o)
        assert (o[:, w:] == 3.5).all()
        return o[:, :w].reshape(-1, self.nq, self.dim)

    def want(self):
        n, t, g = self.n_seq, self.tokens, self.group
        O = np.zeros((n * t, self.nq, self.dim))
        tol = np.zeros_like(O)
        for s in range(n):
            k, v = ref.hold(self.k[s]), ref.hold(self.v[s])
            q = self.q[s * t:(s + 1) * t, :self.nq * self.dim].reshape(t, self.nq, self.dim)
            for h in range(self.kv):
                for j in range(g):
                    i = h * g + j
                    O[s * t:(s + 1) * t, i], tol[s * t:(s + 1) * t, i] = ref.attend(
                        q[:, i], k[:, h], v[:, h], self.pos[s], self.scale, self.window)
        return O, tol

    def check(self):
        got = self.run()
        want, tol = self.want()
        err = np.abs(got - want)
        assert np.isfinite(got).all()
        assert (err <= tol).all(), f"worst error / tolerance {np.max(err / np.maximum(tol, 1e-300)):.3g}"
        return got


ATTEND = [  # dim, kv heads, group, tokens, page, lengths, window
    (128, 8, 5, 1, 64, [1, 2, 31, 32, 33, 64, 65, 512], 0),
    (128, 2, 5, 1, 64, [513, 1023, 1025, 2048, 5000], 0),
    (64, 12, 1, 1, 64, [77], 0),
    (32, 3, 2, 1, 32, [100, 1], 0),
    (96, 5, 3, 1, 96, [95, 97, 700, 1500], 0),
    (128, 1, 8, 1, 32, [40, 3000], 0),
    (128, 1, 16, 1, 128, [600], 0),
    (128, 2, 17, 1, 64, [600, 33], 0),
    (64, 1, 71, 1, 64, [530], 0),
    (160, 2, 4, 1, 32, [555, 31], 0),
    (192, 1, 7, 1, 64, [800], 0),
    (224, 2, 3, 1, 64, [70], 0),
    (256, 2, 8, 1, 256, [1100, 255], 0),
    (128, 2, 5, 4, 64, [4, 35, 515, 1200], 0),
    (128, 1, 5, 64, 128, [700], 0),
    (64, 2, 2, 17, 32, [17, 600], 0),
    (256, 1, 2, 17, 64, [64, 530], 0),
    (96, 2, 7, 5, 32, [5, 70], 0),
    (128, 2, 4, 1, 64, [3, 100, 1500], 64),
    (128, 2, 4, 1, 64, [3, 100, 1500], 1),
    (64, 2, 3, 4, 32, [4, 100, 1500], 37),
    (96, 1, 2, 1, 96, [5000], 1024),
    (32, 1, 1, 1, 32, [70000], 0),
]


@pytest.mark.parametrize("dim,kv,group,tokens,page,lens,window", ATTEND)
def test_attend(q8, dim, kv, group, tokens, page, lens, window):
    Step(q8, dim, kv, group, tokens, page, lens, window).check()


@pytest.mark.parametrize("spread,scale", [(30.0, 0.1), (1e-3, 1.0), (8.0, 1.0)])
def test_attend_sharp_and_flat(q8, spread, scale):
    """Scores far apart (one position takes almost all the weight, maxima that
    grow from step to step) and nearly equal."""
    s = Step(q8, 128, 1, 5, 1, 64, [2000, 700], spread=spread, scale=scale)
    s.k[0] *= np.linspace(0, 1, 2000, dtype=np.float32)[:, None, None]
    s.put(0, np.arange(2000), s.k[0], s.v[0])
    s.check()


def test_attend_one_position_is_its_value(q8):
    s = Step(q8, 128, 2, 5, 1, 64, [1, 1])
    got = s.run()
    for i in range(2):
        want = np.repeat(ref.hold(s.v[i])[0], 5, 0)
        assert np.array_equal(got[i], want)


def test_attend_products_are_exact(q8):
    """Equal scores: the weights are exactly 1 and the outputs exact means of
    a power of two of values; and a score that needs all 24 bits of q."""
    s = Step(q8, 64, 1, 1, 1, 32, [64])
    s.k[0][:] = 0
    s.put(0, np.arange(64), s.k[0], s.v[0])
    v = ref.hold(s.v[0])[:, 0]
    # values share scales within a factor of a few: their sums are exact in fp32
    assert np.array_equal(s.run()[0, 0], (v.sum(0) / 64).astype(np.float32))
    # two positions whose scores differ in the last bits of q alone
    k = np.zeros((2, 1, 64), np.float32)
    k[0, 0, 0], k[1, 0, 1] = 4.0, 4.0
    s.put(0, np.arange(2), k, s.v[0][:2])
    s.pos[:] = 1
    s.q[:] = 0
    a = np.float32(4096.0)
    s.q[0, 0], s.q[0, 1] = np.nextafter(a, np.float32(1e9)), a   # differ by 2^-11
    s.scale = 64.0
    want = np.array([1 / (1 + np.exp(-0.125)), 1 / (1 + np.exp(0.125))]) @ v[:2]
    # scores of 2^20: their difference 0.125 is exact only if every product is
    assert np.abs(s.run()[0, 0] - want).max() <= 0.05 * np.abs(v[:2]).max()


@pytest.mark.parametrize("tokens,group", [(1, 5), (4, 5)])
def test_attend_idle_and_bad_rows(q8, tokens, group):
    lens = [700, 40, 600, 100, 70]
    s = Step(q8, 64, 2, group, tokens, 64, lens)
    good = s.run()
    t = tokens
    s.pos[0] = -1                       # an idle sequence
    s.seq[0:t] = -5                     # ... whatever its slot
    s.seq[1 * t:2 * t] = 99             # slot outside the table
    s.pos[2, -1] = s.cache.max_pages * 64  # position outside the cache
    s.cache.block_table[s.slot[3], 1] = s.cache.n_pages + 7  # a bad page among those read
    if t > 1:
        s.pos[4, 0] = -3                # idle row first: the others keep their sequence
        s.seq[4 * t] = -1
        s.seq[4 * t + 2] = (s.slot[4] + 1) % s.cache.n_slots   # a row of another slot
    got = s.run()
    assert (got[:t] == 0).all()
    assert np.isnan(got[t:2 * t]).all()
    assert np.isnan(got[3 * t - 1]).all()
    assert np.isnan(got[3 * t:4 * t]).all()
    assert np.array_equal(got[2 * t:3 * t - 1], good[2 * t:3 * t - 1]) or t == 1
    if t == 1:
        assert np.array_equal(got[4], good[4])
    else:
        want, tol = s.want()
        assert (got[4 * t] == 0).all() and np.isnan(got[4 * t + 2]).all()
        for j in (1, 3):
            assert (np.abs(got[4 * t + j] - want[4 * t + j]) <= tol[4 * t + j]).all()
    # every counter of the workspace is back at zero, and the call repeats
    assert not s.ws[:1 << 20].any()
    assert np.array_equal(s.run(), got, equal_nan=True)


def test_attend_nan_in_sight_and_out_of_sight(q8):
    """NaN keys and values: a row that sees them gives NaN (for values, in
    their 32 outputs); rows before them, and windows past them, do not."""
    s = Step(q8, 96, 2, 3, 8, 32, [50, 700])
    clean = s.run()
    bad_k, bad_v = s.k[0][46:47].copy(), s.v[0][46:47].copy()
    bad_k[0, 0, 3] = np.nan      # key head 0: position 46 of sequence 0
    bad_v[0, 1, 40] = np.inf     # value head 1, block 1
    s.put(0, [46], bad_k, bad_v)
    got = s.run()
    for j, p in enumerate(s.pos[0]):
        if p < 46:
            assert np.array_equal(got[j], clean[j])
        else:
            assert np.isnan(got[j, :3]).all()
            assert np.isnan(got[j, 3:, 32:64]).all()
            keep = np.r_[0:32, 64:96]
            assert np.array_equal(got[j, 3:][:, keep], clean[j, 3:][:, keep])
    assert np.array_equal(got[8:], clean[8:])
    # a NaN value block well inside, seen by every row: the unmasked steps
    s.put(1, [100], s.k[1][100:101], np.where(np.arange(96) < 32, np.nan, s.v[1][100:101]))
    got = s.run()[8:]
    assert np.isnan(got[:, :, :32]).all() and np.array_equal(got[:, :, 32:], clean[8:, :, 32:])
    # a window that starts after it
    s.window = 500
    assert np.isfinite(s.run()[8:]).all()


def test_attend_infinite_scores(q8):
    """Scores that overflow: -inf at some positions only loses them, at all
    of them gives NaN, +inf gives NaN."""
    s = Step(q8, 32, 1, 1, 1, 32, [40, 40, 40])
    big = np.zeros((40, 1, 32), np.float32)
    big[:, 0, 0] = 3e38
    one = big.copy()
    one[1:] = 0
    s.put(0, np.arange(40), one, s.v[0])
    s.put(1, np.arange(40), big, s.v[1])
    s.put(2, np.arange(40), one, s.v[2])
    s.q[:] = 0
    s.q[0, 0], s.q[1, 0], s.q[2, 0] = -1e10, -1e10, 1e10
    got = s.run()
    v = ref.hold(s.v[0])[1:, 0]
    assert np.abs(got[0, 0] - v.mean(0)).max() <= 2.0 ** -20 * np.abs(v).max()
    assert np.isnan(got[1]).all() and np.isnan(got[2]).all()


def test_attend_any_company(q8):
    """Sequences in any company and order; a call gives the same bits every
    time."""
    s = Step(q8, 128, 2, 5, 2, 64, [1300, 2, 90, 5000, 511, 513], seed=3)
    want, tol = (x.reshape(6, 2, 10, 128) for x in s.want())
    for order in ([0, 1, 2, 3, 4, 5], [5, 0, 3, 2, 1, 4], [3], [4, 1]):
        part = s.run(seqs=order).reshape(len(order), 2, 10, 128)
        assert (np.abs(part - want[order]) <= tol[order]).all()
        assert np.array_equal(s.run(seqs=order).reshape(part.shape), part)


@pytest.mark.parametrize("n,tokens", [(40, 1), (3, 20)])
def test_attend_more_than_runs_at_once(q8, n, tokens):
    """Batches with more steps than shares run at once: sequences laid end to
    end, cut where a share ends."""
    rng = np.random.default_rng(n)
    lens = rng.integers(tokens, 6000 if tokens == 1 else 9000, n).tolist()
    lens[1] = tokens
    s = Step(q8, 64, 4, 4, tokens, 32, lens, slots=n)
    got = s.check()
    assert np.array_equal(s.run(), got)
    assert not s.ws[:1 << 20].any()


def test_attend_many_sequences(q8):
    """More sequences than lanes of a wave, most of them short."""
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 60, 150).tolist()
    lens[70], lens[149] = 1800, 900
    Step(q8, 64, 2, 2, 1, 32, lens, slots=150).check()


def test_attend_workspace_serves_every_shape(q8):
    big = Step(q8, 128, 4, 5, 4, 64, [3000, 1000])
    shapes = [big, Step(q8, 64, 1, 3, 1, 32, [2000] * 3), Step(q8, 256, 1, 2, 1, 64, [1500])]
    alone = [s.run() for s in shapes]
    for i in (1, 0, 2, 0, 1):
        assert np.array_equal(shapes[i].run(ws=big.ws), alone[i])


def test_attend_strides_and_streams(q8):
    s = Step(q8, 128, 2, 5, 2, 64, [1300, 70], extra=3)
    want = s.check()
    st = torch.cuda.Stream()
    q, seq, pos = s.args()
    w = s.nq * s.dim
    o = torch.zeros(4, w + 3, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        q8.q8_kv4_attend(s.cache, q, 2, 2, s.nq, seq, pos, o, s.ws, q_stride=w + 3, o_stride=w + 3)
    st.synchronize()
    assert np.array_equal(host(o)[:, :w].reshape(want.shape), want)


def test_decode_step_in_a_graph(q8):
    """QKV projection, append with rotation and attention captured once and
    replayed with new activations and positions: every replay equals the
    eager step, with eager work in between."""
    rng = np.random.default_rng(21)
    K, nq, kv, dim, n = 256, 6, 2, 64, 3
    N = (nq + 2 * kv) * dim
    Wq = gpu_pack((0.05 * rng.standard_normal((N, K))).astype(np.float32))
    table = i32(rng.permutation(3 * 40).reshape(3, 40))
    plan = q8.rotary_plan(dim, 1e4)
    caches = [q8.KV4Cache(120, 32, kv, dim, table) for _ in range(2)]
    ws = [q8.kv4_attend_workspace(c, n, 1, nq) for c in caches]
    X, Xq = torch.empty(n, K, device="cuda"), q8.empty_act_slots(K)
    bi, seq, pos = i32([0, 1, 2]), i32([2, 0, 1]), i32([0, 0, 0])
    bufs = [[torch.empty(n, N, device="cuda"), torch.empty(n, nq * dim, device="cuda"),
             torch.zeros(n, nq * dim, device="cuda")] for _ in range(2)]

    def step(i):
        Y, Q, O = bufs[i]
        q8.q8_quantize_acts(X, n, K, Xq)
        q8.q8_matmul_narrow(Wq, Xq, bi, n, N, K, Y)
        q8.q8_kv4_append(caches[i], Y, n, N, seq, pos, rotary=plan, n_q_heads=nq, Q=Q)
        q8.q8_kv4_attend(caches[i], Q, n, 1, nq, seq, pos, O, ws[i])

    X.normal_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(0)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    third = 0
    for i in range(40):
        X.copy_(torch.randn(n, K, device="cuda"))
        idle = i % 3 == 1  # the third session skips a step now and then
        pos.copy_(i32([i, i, -1 if idle else third]))
        third += not idle
        graph.replay()
        step(1)
        torch.cuda.synchronize()
        assert torch.equal(bufs[0][2], bufs[1][2]), i
        assert torch.isfinite(bufs[0][2]).all()


def test_decode_attention_example():
    """The example runs, appends one position a step and stays finite."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decode_attention.py")
    spec = importlib.util.spec_from_file_location("decode_attention", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    out = mod.main(["--live", "3", "--context", "100", "--steps", "5"])
    assert out["finite"] and out["position"] == 100 + 5 + 1   # one step before the capture
