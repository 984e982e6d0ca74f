"""The 4-bit E2M1 cache on the GPU: the quantising write and the read bit-exact
against the oracle, attention within bounds that follow from its roundings.

Tolerance of the attention, per output element, with V the largest |value| the
row may read and X the row's largest scale * sum |q_d k_d| (natural units):
  * output rounded to bf16: 2^-8 |o|;
  * p rounded to f16, and normalised by the sum of what it became: each weight is
    off by at most 2^-11 relative, which moves a weighted average by at most
    2 * 2^-11 V;
  * fp32 accumulation of D products and the scaling of the score: (D + 4) 2^-23 X
    of the score, hence as much relative of each weight, twice that of V; the
    exponential (2^-22) and the sums (2^-20) are covered by rounding that up
    to (D + 8) 2^-23 (X + 8);
  * f16 subnormals: at most L 2^-25 / 2^7 of V.
The log-sum-exp is off by the score's error, the exponentials' and the sum's."""

import numpy as np
import pytest
import torch

import paged_kv_attention_17_gb300 as pkv
from oracle import e2m1, ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


class Batch:
    """A flat batch over an E2M1 cache whose slots outside the contexts hold any
    bytes at all, NaN scales among them."""

    def __init__(self, lens, hq, hkv, d, seed=0, ks=0.5, vs=0.3, causal=True, window=0, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d = lens, hq, hkv, d
        self.ks, self.vs, self.causal, self.window = ks, vs, causal, window
        self.scale = 1.0 / np.sqrt(d)
        counts = [-(-L // 16) for L, _ in lens]
        nb = sum(counts) + 3
        perm = rng.permutation(nb)
        self.width = max(counts + [1]) + 1
        self.table = np.full((len(lens), self.width), -7, dtype=np.int32)   # unread entries: bad ids
        at = 0
        for r, c in enumerate(counts):
            self.table[r, :c] = perm[at:at + c]
            at += c
        n = sum(k for _, k in lens)
        self.q = bf16(rng.standard_normal((n, hq, d)) * qscale)
        self.qsl = np.concatenate([[0], np.cumsum([k for _, k in lens])]).astype(np.int32)
        self.seq_lens = np.array([L for L, _ in lens], dtype=np.int32)
        caches, self.slots = [], [self.slot_range(r, 0, L) for r, (L, _) in enumerate(lens)]
        flat = np.concatenate(self.slots + [np.zeros(0, np.int64)]).astype(np.int64)
        for t in (ks, vs):
            c = rng.integers(0, 256, (nb, hkv, 9 * d), dtype=np.uint8)
            c[rng.random(c.shape) < 0.2] = 0x7F
            x = rng.standard_normal((len(flat), hkv, d)) * np.exp(0.5 * rng.standard_normal((1, hkv, d)))
            caches.append(e2m1.write(c, bf16(x).float().numpy(), flat, t) if len(flat) else c)
        self.k, self.v = caches
        self.mq, self.ms = max([k for _, k in lens]), max([L for L, _ in lens])

    def slot_range(self, r, a, b):
        p = np.arange(a, b)
        return self.table[r][p // 16].astype(np.int64) * 16 + p % 16

    def dev(self):
        f = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        return dict(q=self.q.to(DEV), k=f(self.k), v=f(self.v), qsl=f(self.qsl), lens=f(self.seq_lens),
                    table=f(self.table))

    def attend(self, t=None, splits=0, out=None, lse=None, workspace=None, flag=None, scale=None):
        t = t or self.dev()
        out = torch.empty_like(t["q"]) if out is None else out
        lse = torch.empty(t["q"].shape[:2], device=DEV) if lse is None else lse
        flag = torch.zeros(1, dtype=torch.int32, device=DEV) if flag is None else flag
        pkv.pkv_attention_varlen_e2m1(t["q"], t["k"], t["v"], out, t["qsl"], t["lens"], t["table"],
                                      self.mq, self.ms, self.scale if scale is None else scale,
                                      self.ks, self.vs, causal=self.causal, num_splits=splits,
                                      workspace=workspace, lse_out=lse, error_flag=flag,
                                      window=self.window)
        return out, lse, flag

    def oracle(self):
        """(o, lse, V, X) per row and head, in float64 over the decoded cache."""
        q = self.q.float().numpy().astype(np.float64)
        n = q.shape[0]
        o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
        top_v, top_x = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
        for r, (L, k) in enumerate(self.lens):
            K = e2m1.rows(self.k, self.slots[r], self.d, self.ks)
            V = e2m1.rows(self.v, self.slots[r], self.d, self.vs)
            pos = L - k + np.arange(k)
            j = np.arange(L)
            see = (j <= pos[:, None]) if self.causal else np.ones((k, L), bool)
            if self.window:
                see = see & (j > pos[:, None] - self.window)
            rows = slice(self.qsl[r], self.qsl[r + 1])
            for h in range(self.hq):
                g = h // (self.hq // self.hkv)
                s = np.where(see, self.scale * (q[rows, h] @ K[:, g].T), -np.inf)
                if not s.size:
                    continue
                m = s.max(1, keepdims=True)
                w = np.exp(s - m)
                o[rows, h] = (w @ V[:, g]) / w.sum(1, keepdims=True)
                lse[rows, h] = m[:, 0] + np.log(w.sum(1))
                top_v[rows, h] = np.abs(V[:, g]).max()
                top_x[rows, h] = (self.scale * (np.abs(q[rows, h]) @ np.abs(K[:, g]).T)).max(1)
        return o, lse, top_v, top_x

    def check(self, out, lse):
        o, l_ref, V, X = self.oracle()
        rel = (self.d + 8) * 2.0 ** -23 * (X + 8)
        err = np.abs(out.float().cpu().numpy().astype(np.float64) - o)
        tol = 2.0 ** -8 * np.abs(o) + ((2.0 ** -10 + 2 * rel + self.ms * 2.0 ** -32) * V)[..., None]
        assert (err <= tol).all(), (err - tol).max()
        got = lse.cpu().numpy().astype(np.float64)
        assert (np.abs(got - l_ref) <= rel + 2.0 ** -22 * np.abs(l_ref)).all()


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------
def special_rows(n, hkv, d, rng):
    x = rng.standard_normal((n, hkv, d)).astype(np.float32) * np.exp(2 * rng.standard_normal((n, hkv, 1))).astype(np.float32)
    flat = x.reshape(-1, 16)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=np.float32)
    edge = np.concatenate([mids, -mids])
    k = len(flat)
    flat[0] = 0
    flat[1 % k] = edge                                     # exact midpoints under a scale of 1
    flat[2 % k] = np.nextafter(edge, np.float32(0))
    flat[3 % k] = np.nextafter(edge, np.float32(100) * np.sign(edge))
    if k > 8:
        flat[4] = 1e-38
        flat[5] = np.float32(3e38) * np.sign(edge)
        flat[6, 3] = np.inf
        flat[6, 5] = -np.inf
        flat[7, 9] = np.nan
        flat[8] = 2.0 ** -9 * 6 / 2 * np.sign(edge)        # a scale halfway to E4M3's least
    return flat.reshape(n, hkv, d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, hkv, d", [(1, 1, 64), (1, 1, 128), (3, 2, 64), (5, 8, 128), (40, 3, 128),
                                       (333, 1, 64)])
@pytest.mark.parametrize("ks, vs", [(1.0, 0.5), (0.0375, 3.7), (1e-20, 1e25)])
def test_write_is_bit_exact_and_touches_nothing_else(dtype, n, hkv, d, ks, vs):
    rng = np.random.default_rng(n + d)
    kx, vx = special_rows(n, hkv, d, rng), special_rows(n, hkv, d, rng)[::-1].copy()
    nb = n // 16 + 3
    slots = rng.permutation(nb * 16)[:n].astype(np.int64)
    if n > 4:
        slots[2] = -1
        slots[4] = nb * 16 + 5
    k0, v0 = (rng.integers(0, 256, (nb, hkv, 9 * d), dtype=np.uint8) for _ in range(2))
    kt, vt = torch.from_numpy(kx).to(dtype), torch.from_numpy(vx).to(dtype)
    kc, vc = torch.from_numpy(k0).to(DEV), torch.from_numpy(v0).to(DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.pkv_write_e2m1(kt.to(DEV), vt.to(DEV), torch.from_numpy(slots).to(DEV), kc, vc, ks, vs,
                       error_flag=flag)
    want_k = e2m1.write(k0, kt.float().numpy(), slots, ks)
    want_v = e2m1.write(v0, vt.float().numpy(), slots, vs)
    assert np.array_equal(kc.cpu().numpy(), want_k)
    assert np.array_equal(vc.cpu().numpy(), want_v)
    assert flag.item() == (pkv.FLAG_BAD_SLOT if n > 4 else 0)


@pytest.mark.parametrize("t", [1.0, 0.7, 0.0123, 1.9999999, 3.0e-7, 5.5e11, 1e-30])
def test_write_divides_correctly_everywhere(t):
    """A million quotients of each kind: every block's scale and codes."""
    rng = np.random.default_rng(4)
    n, hkv, d = 1024, 8, 128
    x = (rng.standard_normal((n, hkv, d)) * t * np.exp2(rng.integers(-12, 9, (n, hkv, 1)))).astype(np.float32)
    x[::3, ::2] *= np.float32(0)                          # zeros of both signs
    x[1::7, :, ::5] = -0.0
    nb = n // 16
    cache = torch.zeros(nb, hkv, 9 * d, dtype=torch.uint8, device=DEV)
    other = torch.zeros_like(cache)
    dev = torch.from_numpy(x).to(DEV)
    pkv.pkv_write_e2m1(dev, dev, torch.arange(n, device=DEV), cache, other, t, 1.0)
    codes, scales = e2m1.quantize(x, t)
    want = e2m1.parts(cache.cpu().numpy(), d)
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(nb, 16, hkv, d // 2).transpose(0, 2, 1, 3)
    assert np.array_equal(want[0], packed)
    assert np.array_equal(want[1], scales.reshape(nb, 16, hkv, d // 16).transpose(0, 2, 1, 3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, hkv, d", [(1, 1, 64), (7, 3, 64), (50, 8, 128), (700, 2, 128)])
def test_read_is_exact(dtype, n, hkv, d):
    rng = np.random.default_rng(n)
    nb = 9
    cache = [rng.integers(0, 256, (nb, hkv, 9 * d), dtype=np.uint8) for _ in range(2)]
    slots = rng.integers(0, nb * 16, n).astype(np.int64)   # the same slot several times
    if n > 3:
        slots[1], slots[3] = -3, nb * 16
    dev = [torch.from_numpy(c).to(DEV) for c in cache]
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = [torch.full((n, hkv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    pkv.pkv_read_e2m1(*dev, torch.from_numpy(slots).to(DEV), *outs, 0.3, 1.7, error_flag=flag)
    ok = (slots >= 0) & (slots < nb * 16)
    for c, t, got in zip(cache, (0.3, 1.7), outs):
        want = torch.full((n, hkv, d), 7.0, dtype=torch.float64)
        want[torch.from_numpy(ok)] = torch.from_numpy(e2m1.rows(c, slots[ok], d, t))
        want = want.to(torch.float32).to(dtype)            # one rounding to fp32, one to the type
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=99.0), torch.nan_to_num(want, nan=99.0))
        assert torch.equal(got.cpu().isnan(), want.isnan())
    assert flag.item() == (pkv.FLAG_BAD_SLOT if n > 3 else 0)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
DECODE = [(1, 1), (16, 1), (17, 1), (33, 1), (300, 1), (513, 1)]


@pytest.mark.parametrize("hq, hkv, d", [(1, 1, 64), (4, 2, 64), (8, 2, 128), (32, 8, 128), (12, 1, 128),
                                        (16, 1, 64), (7, 1, 128), (40, 2, 128)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_decode_rows(hq, hkv, d, splits):
    b = Batch(DECODE, hq, hkv, d, seed=hq + d)
    out, lse, flag = b.attend(splits=splits)
    assert flag.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("hq, hkv, d", [(64, 4, 128), (64, 4, 64)])
def test_sixteen_row_tiles(hq, hkv, d, splits):
    # (batches that fill the device with 16-row tiles)
    b = Batch([(200 + 17 * r, 1 + r % 4) for r in range(24)], hq, hkv, d, seed=24)
    out, lse, flag = b.attend(splits=splits)
    assert flag.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[(4, 4), (20, 2), (35, 3), (5, 1)], [(900, 4), (0, 0), (129, 3)]])
@pytest.mark.parametrize("hq, hkv, d", [(8, 4, 64), (8, 2, 128), (16, 1, 128)])
@pytest.mark.parametrize("splits", [1, 4])
def test_tails(lens, hq, hkv, d, causal, splits):
    b = Batch(lens, hq, hkv, d, seed=3, causal=causal)
    out, lse, flag = b.attend(splits=splits)
    assert flag.item() == 0
    b.check(out, lse)


LONG = [(37, 37), (1, 1), (200, 5), (390, 133), (130, 3), (257, 257)]


@pytest.mark.parametrize("hq, hkv, d", [(2, 2, 64), (8, 2, 128), (12, 4, 64), (3, 1, 128), (16, 1, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_requests_among_decode_rows(hq, hkv, d, causal):
    b = Batch(LONG, hq, hkv, d, seed=5, causal=causal)
    out, lse, flag = b.attend()
    assert flag.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 128, 300, 5000])
@pytest.mark.parametrize("lens, d", [(DECODE + [(700, 4)], 128), (LONG, 128), (LONG, 64)])
def test_windows(window, lens, d):
    b = Batch(lens, 4, 2, d, seed=6, window=window)
    out, lse, flag = b.attend(splits=0)
    assert flag.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("window, causal, splits", [(100, True, 3), (20, False, 1), (200, False, 2),
                                                    (150, True, 4)])
def test_windows_with_splits_and_without_a_causal_limit(window, causal, splits):
    b = Batch(LONG + [(600, 1)], 8, 2, 128, seed=23, window=window, causal=causal)
    out, lse, flag = b.attend(splits=splits)
    assert flag.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("qscale", [0.0, 2.0 ** -60, 2.0 ** -8, 30.0])
@pytest.mark.parametrize("lens", [DECODE, LONG])
def test_query_magnitudes(qscale, lens):
    b = Batch(lens, 4, 1, 128, seed=7, qscale=qscale)
    out, lse, flag = b.attend()
    b.check(out, lse)


@pytest.mark.parametrize("lens", [[(40, 2)], [(40, 20)]])
def test_a_negative_scale_is_taken(lens):
    b = Batch(lens, 4, 2, 128, seed=8)
    out, lse, _ = b.attend(scale=-0.2)
    b.scale = -0.2
    o, l_ref, V, _ = b.oracle()
    assert np.abs(out.float().cpu().numpy() - o).max() <= (2.0 ** -8 + 2.0 ** -9) * V.max()


def poison(b, r, pos, kv_head, block, value=0x7F):
    slot = int(b.slot_range(r, pos, pos + 1)[0])
    at = 8 * b.d + (slot % 16) * (b.d // 16) + block
    b.v[slot // 16, kv_head, at] = value


@pytest.mark.parametrize("lens, pos", [([(50, 3)], 48), ([(300, 40)], 280), ([(600, 300)], 400),
                                       ([(600, 300)], 599)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [0x7F, 0xFF])
def test_a_nan_value_reaches_the_rows_that_see_it_alone(lens, pos, d, value):
    b = Batch(lens, 4, 2, d, seed=9)
    clean, _, _ = b.attend()
    poison(b, 0, pos, 1, 2, value)
    out, _, _ = b.attend()
    L, n = lens[0]
    rows = np.arange(n) + L - n
    nan = out.isnan().cpu().numpy()
    want = np.zeros_like(nan)
    want[rows >= pos, 2:, 32:48] = True
    assert np.array_equal(nan, want)
    assert torch.equal(out[rows < pos], clean[rows < pos])


def test_a_nan_before_the_window_is_not_seen():
    for n in (1, 3, 40):
        b = Batch([(300, n)], 4, 2, 128, seed=10, window=130)
        clean, _, _ = b.attend()
        poison(b, 0, 300 - n - 130, 1, 3)
        out, _, _ = b.attend()
        assert torch.equal(out, clean)


def test_nan_scores_make_nan_rows():
    b = Batch([(40, 1), (40, 1)], 4, 2, 128, seed=11)
    b.q[1] = float("nan")
    out, _, _ = b.attend(splits=1)
    assert not out[0].isnan().any() and out[1].isnan().all()


def test_one_key_gives_the_value():
    b = Batch([(1, 1)], 8, 2, 128, seed=12)
    out, lse, _ = b.attend()
    v = e2m1.rows(b.v, b.slots[0], 128, b.vs)[0]
    want = torch.from_numpy(np.repeat(v, 4, axis=0)).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(out[0].cpu(), want)


def test_bad_lengths_and_blocks_are_flagged():
    b = Batch([(30, 1), (20, 2)], 4, 2, 128, seed=13)
    t = b.dev()
    t["lens"][1] = 1                                       # fewer keys than new tokens
    _, _, flag = b.attend(t)
    assert flag.item() == pkv.FLAG_BAD_LENGTHS
    t = b.dev()
    t["lens"][0] = 16 * b.width + 1                        # past its table row
    assert b.attend(t)[2].item() & pkv.FLAG_BAD_LENGTHS
    t = b.dev()
    t["lens"][0] = 2 ** 31 - 1                             # and at the type's end
    assert b.attend(t)[2].item() & pkv.FLAG_BAD_LENGTHS
    long = Batch([(40, 30)], 4, 2, 128, seed=13)
    t = long.dev()
    for length in (2 ** 31 - 1, 16 * long.width + 1, 29, -5):
        t["lens"][0] = length
        assert long.attend(t)[2].item() & pkv.FLAG_BAD_LENGTHS
    t = b.dev()
    t["qsl"][1] = 5                                        # not nondecreasing, and past the tokens
    assert b.attend(t)[2].item() & pkv.FLAG_BAD_LENGTHS
    for bad in (-1, b.k.shape[0]):
        t = b.dev()
        t["table"][0, 1] = bad
        out, lse, flag = b.attend(t)
        assert flag.item() == pkv.FLAG_BAD_BLOCK
        torch.cuda.synchronize()


def test_rows_behind_the_last_sequence_are_left():
    b = Batch([(30, 1), (20, 2)], 4, 2, 128, seed=14)
    t = b.dev()
    t["q"] = torch.cat([t["q"], torch.full((5, 4, 128), float("nan"), device=DEV, dtype=torch.bfloat16)])
    out = torch.full_like(t["q"], 3.0)
    lse = torch.full(out.shape[:2], 5.0, device=DEV)
    for splits in (1, 2):
        b.attend(t, splits=splits, out=out, lse=lse)
        assert (out[3:] == 3.0).all() and (lse[3:] == 5.0).all()
        b.check(out[:3], lse[:3])


def test_split_counts_agree():
    b = Batch([(4000, 1), (777, 2)], 8, 2, 128, seed=15)
    outs = [b.attend(splits=s) for s in (1, 2, 7, 33, 64)]
    for out, lse, flag in outs:
        b.check(out, lse)


def test_long_context_past_32_bit_cache_offsets():
    # pages of 9216 bytes: block ids whose byte offsets pass 2^31 and 2^32
    hkv, d, L = 8, 128, 40
    nb = (1 << 32) // (hkv * 9 * d) + 64
    b = Batch([(L, 1)], 8, hkv, d, seed=16)
    t = b.dev()
    big = [torch.zeros(nb, hkv, 9 * d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    ids = [nb - 1, nb // 2 + 5, 3]
    for i, blk in enumerate(ids):
        for c, name in zip(big, ("k", "v")):
            c[blk] = t[name][int(b.table[0, i])]
    t["k"], t["v"] = big
    t["table"][0, :3] = torch.tensor(ids, dtype=torch.int32)
    out, lse, flag = b.attend(t)
    assert flag.item() == 0
    b.check(out, lse)
    slots = torch.tensor([ids[0] * 16 + 7, ids[1] * 16], device=DEV)
    got = [torch.empty(2, hkv, d, device=DEV) for _ in range(2)]
    pkv.pkv_read_e2m1(*big, slots, *got, b.ks, b.vs)
    want = e2m1.rows(b.k, b.slots[0][[7, 16]], d, b.ks).astype(np.float32)
    assert np.array_equal(got[0].cpu().numpy(), want)
    x = torch.randn(2, hkv, d, device=DEV)
    pkv.pkv_write_e2m1(x, x, slots, *big, b.ks, b.vs)
    pkv.pkv_read_e2m1(*big, slots, *got, b.ks, b.vs)
    codes, scales = e2m1.quantize(x.cpu().numpy(), b.ks)
    assert np.array_equal(got[0].cpu().numpy(), e2m1.values(codes, scales, b.ks).astype(np.float32))


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lens", [[(1, 1), (300, 1), (47, 1)], [(60, 4), (33, 3)], [(90, 60), (200, 1), (31, 31)]])
@pytest.mark.parametrize("hq, hkv, d", [(8, 2, 128), (6, 2, 64)])
def test_write_attend_read(lens, hq, hkv, d):
    b = Batch(lens, hq, hkv, d, seed=17)
    rng = np.random.default_rng(18)
    t = b.dev()
    new = np.concatenate([b.slot_range(r, L - n, L) for r, (L, n) in enumerate(lens)])
    kx, vx = (bf16(rng.standard_normal((len(new), hkv, d))) for _ in range(2))
    slots = torch.from_numpy(new).to(DEV)
    out, lse = torch.empty_like(t["q"]), torch.empty(t["q"].shape[:2], device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.pkv_write_attention_varlen_e2m1(kx.to(DEV), vx.to(DEV), slots, t["q"], t["k"], t["v"], out,
                                        t["qsl"], t["lens"], t["table"], b.mq, b.ms, b.scale, b.ks,
                                        b.vs, lse_out=lse, error_flag=flag)
    assert flag.item() == 0
    b.k = e2m1.write(b.k, kx.float().numpy(), new, b.ks)
    b.v = e2m1.write(b.v, vx.float().numpy(), new, b.vs)
    assert np.array_equal(t["k"].cpu().numpy(), b.k) and np.array_equal(t["v"].cpu().numpy(), b.v)
    b.check(out, lse)
    # the separate calls give the same bits
    t2 = b.dev()
    out2, lse2, _ = b.attend(t2)
    assert torch.equal(out2, out) and torch.equal(lse2, lse)
    # and the rows read back attend alike as a plain bf16 cache
    got = [torch.empty(len(new), hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pkv.pkv_read_e2m1(t["k"], t["v"], slots, *got, b.ks, b.vs)
    want = torch.from_numpy(e2m1.rows(b.k, new, d, b.ks)).float().bfloat16()
    assert torch.equal(got[0].cpu(), want)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("hq, hkv, d", [(8, 2, 128), (32, 2, 64)])
def test_the_fused_write_of_a_padded_step(hq, hkv, d, splits):
    """Decode steps store the rows in the attention kernel: padding rows (slot -1
    behind the last request), a slot outside the cache, blocks that begin with a
    new token, several row tiles and splits of one request."""
    lens = [(33, 1), (64, 4), (1, 1), (500, 2), (0, 0), (97, 3)]
    b = Batch(lens, hq, hkv, d, seed=21)
    rng = np.random.default_rng(22)
    new = np.concatenate([b.slot_range(r, L - n, L) for r, (L, n) in enumerate(lens)])
    n, pad = len(new), 3
    kx, vx = (bf16(rng.standard_normal((n + pad, hkv, d))) for _ in range(2))
    kx[0, 0, 3] = float("nan")                            # one row's block becomes NaN
    t = b.dev()
    t["q"] = torch.cat([t["q"], torch.ones(pad, hq, d, dtype=torch.bfloat16, device=DEV)])
    slots = np.concatenate([new, np.full(pad, -1)])
    out = torch.full_like(t["q"], 5.0)
    lse = torch.empty(t["q"].shape[:2], device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(sl):
        pkv.pkv_write_attention_varlen_e2m1(
            kx.to(DEV), vx.to(DEV), torch.from_numpy(sl).to(DEV), t["q"], t["k"], t["v"], out, t["qsl"],
            t["lens"], t["table"], b.mq, b.ms, b.scale, b.ks, b.vs, num_splits=splits, lse_out=lse,
            error_flag=flag)

    call(slots)
    assert flag.item() == 0
    b.k = e2m1.write(b.k, kx.float().numpy(), slots, b.ks)
    b.v = e2m1.write(b.v, vx.float().numpy(), slots, b.vs)
    assert np.array_equal(t["k"].cpu().numpy(), b.k) and np.array_equal(t["v"].cpu().numpy(), b.v)
    assert (out[n:] == 5.0).all()
    assert out[0, :hq // hkv].isnan().all() and not out[0, hq // hkv:].isnan().any()
    b.k[new[0] // 16] = 0                                 # (the oracle's check leaves that request out)
    b.v[new[0] // 16] = 0
    o, l_ref, V, X = b.oracle()
    got = out[1:n].float().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(o[1:]) + ((2.0 ** -10 + 2 * (d + 8) * 2.0 ** -23 * (X + 8)) * V)[1:, :, None]
    assert (np.abs(got - o[1:]) <= tol).all()
    # a slot outside the cache is reported, and nothing else changes
    bad = slots.copy()
    bad[1] = b.k.shape[0] * 16
    before = t["k"].clone()
    call(bad)
    assert flag.item() == pkv.FLAG_BAD_SLOT
    assert torch.equal(before, t["k"])


@pytest.mark.parametrize("lens", [[(300, 1), (47, 1)], [(290, 130), (200, 1)]])
def test_captured_and_replayed_on_another_stream(lens):
    b = Batch(lens, 8, 2, 128, seed=19)
    t = b.dev()
    want, lse_want, _ = b.attend(t)
    out, lse = torch.empty_like(want), torch.empty_like(lse_want)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = [torch.full((8 << 20,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for w in ws:                                       # two graphs, a workspace each
            o = torch.empty_like(want)
            b.attend(t, out=o, lse=lse, workspace=w, flag=flag)
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                b.attend(t, out=o, lse=lse, workspace=w, flag=flag)
            graphs.append(g)
            outs.append(o)
        for o in outs:
            o.zero_()
        for g in graphs * 3:
            g.replay()
    # eager calls on the default stream meanwhile
    for _ in range(3):
        b.attend(t, out=out, lse=torch.empty_like(lse))
    torch.cuda.synchronize()
    for o in outs + [out]:
        assert torch.equal(o, want)
    assert flag.item() == 0


@pytest.mark.parametrize("lens", [[(300, 1), (47, 1)], [(290, 130), (200, 1)]])
def test_a_stream_given_by_argument(lens):
    """Two streams at once, neither of them current, a workspace and rows of their own."""
    b = Batch(lens, 8, 2, 128, seed=20)
    t = b.dev()
    want, lse_want, _ = b.attend(t)
    n = want.shape[0]
    slots = torch.from_numpy(np.concatenate([b.slot_range(r, L - k, L) for r, (L, k) in enumerate(lens)])).to(DEV)
    read = [torch.empty(n, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pkv.pkv_read_e2m1(t["k"], t["v"], slots, read[0], read[1], b.ks, b.vs)
    runs = []
    for _ in range(2):
        runs.append((torch.cuda.Stream(), torch.empty_like(want), torch.empty_like(lse_want),
                     torch.empty(8 << 20, dtype=torch.uint8, device=DEV),
                     torch.zeros(1, dtype=torch.int32, device=DEV), [torch.empty_like(x) for x in read]))
    torch.cuda.synchronize()
    for _ in range(5):
        for side, out, lse, ws, flag, rows in runs:
            pkv.pkv_attention_varlen_e2m1(t["q"], t["k"], t["v"], out, t["qsl"], t["lens"], t["table"], b.mq,
                                          b.ms, b.scale, b.ks, b.vs, workspace=ws, lse_out=lse,
                                          error_flag=flag, stream=side)
            pkv.pkv_read_e2m1(t["k"], t["v"], slots, rows[0], rows[1], b.ks, b.vs, stream=side)
    for side, out, lse, _, flag, rows in runs:
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, lse_want) and flag.item() == 0
        assert torch.equal(rows[0], read[0]) and torch.equal(rows[1], read[1])


@pytest.mark.parametrize("inputs", ["stage", "mapped", "memcpy"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_graph_runner_steps(inputs, d):
    """Steps of several sizes through one runner: new rows in the cache bit-exact,
    outputs as the oracle's, padding untouched."""
    from paged_kv_attention_17_gb300.graphs import DecodeGraphRunner
    hq, hkv = 8, 2
    lens = [(40, 1), (1, 1), (700, 1), (17, 1), (128, 1)]
    b = Batch(lens, hq, hkv, d, seed=30)
    t = b.dev()
    runner = DecodeGraphRunner(t["k"], t["v"], hq, b.scale, b.width, 16 * b.width, max_batch=8,
                               sizes=[1, 4, 8], inputs=inputs, kv_scales=(b.ks, b.vs))
    rng = np.random.default_rng(31)
    for pick in ([0, 1, 2, 3, 4], [2], [4, 1, 0], [3, 2, 1, 0]):
        step = runner.begin(len(pick))
        kx, vx = (bf16(rng.standard_normal((len(pick), hkv, d))) for _ in range(2))
        slots = np.array([b.slot_range(r, b.lens[r][0] - 1, b.lens[r][0])[0] for r in pick])
        step.q.copy_(b.q[pick])
        step.k_new.copy_(kx)
        step.v_new.copy_(vx)
        step.slot_mapping.copy_(torch.from_numpy(slots))
        step.seq_lens.copy_(torch.from_numpy(b.seq_lens[pick]))
        step.block_table.copy_(torch.from_numpy(np.maximum(b.table[pick], 0)))
        runner.launch(step)
        out, flag = runner.result(step)
        assert flag == 0
        b.k = e2m1.write(b.k, kx.float().numpy(), slots, b.ks)
        b.v = e2m1.write(b.v, vx.float().numpy(), slots, b.vs)
        assert np.array_equal(t["k"].cpu().numpy(), b.k)
        assert np.array_equal(t["v"].cpu().numpy(), b.v)
        o, _, V, X = b.oracle()
        rel = (d + 8) * 2.0 ** -23 * (X + 8)
        tol = 2.0 ** -8 * np.abs(o) + ((2.0 ** -10 + 2 * rel + b.ms * 2.0 ** -32) * V)[..., None]
        assert (np.abs(out.float().numpy() - o[pick]) <= tol[pick]).all()


def test_the_runner_refuses_a_cache_without_scales_or_of_another_shape():
    from paged_kv_attention_17_gb300.graphs import DecodeGraphRunner
    cache = torch.zeros(4, 2, 9 * 64, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        DecodeGraphRunner(cache, cache.clone(), 4, 0.1, 4, 64, max_batch=1)
    bad = torch.zeros(4, 2, 9 * 64 + 1, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        DecodeGraphRunner(bad, bad.clone(), 4, 0.1, 4, 64, max_batch=1, kv_scales=(1.0, 1.0))


def test_bindings_refuse_wrong_tensors():
    b = Batch([(30, 1), (40, 1)], 4, 2, 128, seed=20)
    t = b.dev()
    ok = dict(t)
    for name, bad in [("q", t["q"].float()), ("q", t["q"][..., :64]), ("k", t["k"].cpu()),
                      ("k", t["k"][:, :, :1151]), ("v", t["v"][:, :1]), ("qsl", t["qsl"].long()),
                      ("lens", t["lens"].float()), ("table", t["table"][0]),
                      ("table", t["table"].t().contiguous().t())]:
        with pytest.raises((ValueError, TypeError)):
            b.attend({**ok, name: bad}, out=torch.empty_like(t["q"]))
    with pytest.raises((ValueError, TypeError)):
        b.attend(t, out=torch.empty(2, 4, 128, device=DEV))
    with pytest.raises(pkv.PkvError):
        b.attend(t, splits=4, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    x = torch.zeros(3, 2, 128, device=DEV)
    s = torch.zeros(3, dtype=torch.int64, device=DEV)
    for k, v, sl in [(x[:2], x, s), (x, x.double(), s), (x, x.transpose(0, 1), s), (x, x, s.int()),
                     (x.cpu(), x, s), (x[..., ::2], x, s)]:
        with pytest.raises((ValueError, TypeError)):
            pkv.pkv_write_e2m1(k, v, sl, t["k"], t["v"], 1.0, 1.0)
        with pytest.raises((ValueError, TypeError)):
            pkv.pkv_read_e2m1(t["k"], t["v"], sl, k, v, 1.0, 1.0)


def test_the_split_rule_on_this_device():
    """The rule of the header on this device's SM count, and a workspace sized by it
    suffices for the library's own choice."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for seqs, q, length, hq, hkv in [(1, 1, 8192, 32, 8), (1, 1, 1024, 32, 8), (1, 1, 500, 32, 8),
                                     (2, 1, 131072, 32, 8), (16, 3, 1027, 16, 1), (64, 1, 4096, 32, 8),
                                     (1, 900, 5000, 32, 8), (1, 1, 65536, 16, 1),
                                     (64, 4, 4000, 32, 8), (2, 2, 300, 128, 8)]:
        group = hq // hkv
        tokens = q if q <= 4 else 1
        blocks = -(-length // 16)
        full = seqs * hkv * -(-group * tokens // 16) * max(1, blocks // 32) > sms
        rows = 16 if group * tokens > 8 and full else 8
        units = seqs * hkv * -(-group * tokens // rows)
        s = max(1, min(blocks // 8, sms * 7 // 8 // units))
        if blocks > 64 * s:
            s = min(sms * (2 if rows == 8 else 1) // units, max(s, blocks // 32))
        s = min(s, 64)
        if s < 2 or blocks * (s - 1) < 48 * s:
            s = 1
        assert pkv.pkv_num_splits_e2m1(seqs, q, length, hq, hkv, 128) == s
