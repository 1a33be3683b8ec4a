"""GPU parity of the 4-bit paged key/value cache (fa_kv4_append, fa_kv4_read, fa_fwd_kv4)
against the fp64 oracle: every code, scale and value exactly, the attention within bounds
derived from its roundings.
"""
import numpy as np
import pytest

import oracle.kv4 as kv4
from io_aware_exact_24_b200.inputs import bf16_bits_to_f32, f32_to_bf16_bits, normal_bf16

from fa_testutil import SIXTEEN_ROWS, run_fa, to_device_bf16, to_host_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from io_aware_exact_24_b200.build import build
    build()


def ints(x, dtype=np.int32):
    import torch
    return None if x is None else torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype))).cuda()


class Cache:
    """A cache on the GPU whose unwritten rows hold the worst there is (codes of ones, scales NaN)."""

    def __init__(self, num_pages, H_kv, page_size, d, max_pages, table):
        import torch
        self.num_pages, self.H_kv, self.page_size, self.d, self.max_pages = num_pages, H_kv, page_size, d, max_pages
        self.table = None if table is None else np.asarray(table, np.int32)
        self.d_table = ints(table)
        shape = (num_pages, H_kv, page_size)
        new = lambda last, fill, t: torch.full((*shape, last), fill, dtype=t, device="cuda")
        self.k_codes, self.v_codes = new(d // 2, 255, torch.uint8), new(d // 2, 255, torch.uint8)
        self.k_scales = new(d // 32, float("nan"), torch.bfloat16)
        self.v_scales = self.k_scales.clone()

    @property
    def buffers(self):
        return self.k_codes, self.k_scales, self.v_codes, self.v_scales

    @property
    def sizes(self):
        return self.d, self.num_pages, self.page_size, self.max_pages

    def append(self, k, v, key_lens, new_lens=None):
        from io_aware_exact_24_b200 import fa_kv4_append
        B, H_kv, N, _ = k.shape
        fa_kv4_append(k, v, *self.buffers, self.d_table, ints(key_lens), ints(new_lens), B, H_kv, N, *self.sizes)

    def read(self, key_lens, N, first=None, B=None):
        import torch
        from io_aware_exact_24_b200 import fa_kv4_read
        B = len(key_lens)
        k = torch.full((B, self.H_kv, N, self.d), 7.0, dtype=torch.bfloat16, device="cuda")
        v = k.clone()
        fa_kv4_read(*self.buffers, self.d_table, ints(key_lens), ints(first), k, v, B, self.H_kv, N, *self.sizes)
        return k, v

    def host(self):
        """Codes [pages, H_kv, page_size, d] and scales (float64) of K and V."""
        out = []
        for c, s in ((self.k_codes, self.k_scales), (self.v_codes, self.v_scales)):
            out.append((kv4.unpack(c.cpu().numpy()), s.float().cpu().numpy().astype(np.float64)))
        return out

    def positions(self, b, L):
        """K and V values [H_kv, L, d] of positions 0..L-1 of sequence b, and which of them have a page."""
        (kc, ks), (vc, vs) = self.host()
        k, v = np.zeros((self.H_kv, L, self.d)), np.zeros((self.H_kv, L, self.d))
        there = np.zeros(L, bool)
        for j in range(L):
            at = kv4.place(j, b, self.table, self.page_size, self.max_pages, self.num_pages)
            if at is not None:
                there[j] = True
                k[:, j] = kv4.values(kc[at[0], :, at[1]], ks[at[0], :, at[1]])
                v[:, j] = kv4.values(vc[at[0], :, at[1]], vs[at[0], :, at[1]])
        return k, v, there


def tokens(B, H_kv, N, d, seed, sigma=1.0):
    bits = [normal_bf16((B, H_kv, N, d), seed, t, sigma) for t in (1, 2)]
    return [to_device_bf16(b) for b in bits], [bf16_bits_to_f32(b).astype(np.float64) for b in bits]


# ---------------------------------------------------------------- writing and reading back

# B, H_kv, N_new, d, page_size, max_pages, key_lens, new_lens, shuffled table
WRITES = [
    (1, 1, 1, 64, 16, 1, [1], None, False),
    (1, 1, 1, 128, 16, 3, [48], None, True),
    (3, 2, 1, 128, 32, 4, [1, 33, 128], None, True),
    (2, 3, 37, 64, 16, 5, [37, 80], None, True),              # runs over page ends
    (3, 5, 50, 128, 48, 2, [50, 20, 96], [50, 20, 7], True),  # padded batch; page size no power of two
    (2, 2, 9, 128, 16, 2, [4, 40], [9, 9], True),             # starts before 0; ends past the pages
    (2, 1, 6, 64, 64, 1, [0, 64], [0, 3], False),             # nothing new for one; dense cache
    (1, 2, 5, 128, 16, 2, [10], [9], True),                   # new_lens above N_new: clamped
    (1, 1, 130, 64, 16, 16, [256], None, True),
]


@pytest.mark.parametrize("B,H_kv,N,d,page,maxp,key_lens,new_lens,shuffled", WRITES)
def test_append_writes_the_tokens_and_nothing_else(B, H_kv, N, d, page, maxp, key_lens, new_lens, shuffled):
    import torch
    num_pages = B * maxp + 2
    rng = np.random.default_rng(5)
    table = rng.permutation(num_pages)[:B * maxp].reshape(B, maxp) if shuffled else None
    c = Cache(num_pages, H_kv, page, d, maxp, table)
    (k, v), host = tokens(B, H_kv, N, d, 11)
    c.append(k, v, key_lens, new_lens)
    torch.cuda.synchronize()
    want = [(np.full((num_pages, H_kv, page, d), 15, np.uint8), np.full((num_pages, H_kv, page, d // 32), np.nan))
            for _ in range(2)]
    for x, (codes, scales) in zip(host, want):
        qc, qs = kv4.quantise(x)
        for b in range(B):
            n_new = N if new_lens is None else min(N, new_lens[b])
            for n in range(n_new):
                at = kv4.place(key_lens[b] - n_new + n, b, table, page, maxp, num_pages)
                if at is not None:
                    codes[at[0], :, at[1]] = qc[b, :, n]
                    scales[at[0], :, at[1]] = qs[b, :, n]
    for (codes, scales), (wc, ws) in zip(c.host(), want):
        assert np.array_equal(codes, wc)
        assert np.array_equal(scales, ws, equal_nan=True)
    # reading back: what the cache holds, and zeros outside the sequence
    for first in (None, [-3] * B, [5] * B):
        kb, vb = c.read(key_lens, page * maxp + 7, first)
        kb, vb = to_host_f64(kb), to_host_f64(vb)
        for b in range(B):
            L = min(max(key_lens[b], 0), page * maxp)
            wk, wv, there = c.positions(b, L)
            f = 0 if first is None else first[b]
            for got, w in ((kb, wk), (vb, wv)):
                full = np.zeros((H_kv, page * maxp + 7, d))
                for n in range(full.shape[1]):
                    if 0 <= f + n < L and there[f + n]:
                        full[:, n] = w[:, f + n]
                assert np.array_equal(got[b], full, equal_nan=True)


def test_append_of_every_kind_of_value():
    """Groups of ties, equal pairs, tiny, huge and non-finite values get the oracle's codes and scales."""
    import torch
    d, N = 128, 4096
    rng = np.random.default_rng(6)
    x = np.empty((1, 1, N, d))
    for n in range(N):
        kind = n % 8
        m = np.ldexp(rng.integers(128, 256, d).astype(float), rng.integers(-12, 4, d)) * rng.choice([-1, 1], d)
        if kind == 1:
            m = rng.integers(-16, 17, d) * 2.0 ** -5             # many exact ties and equal pairs
        elif kind == 2:
            m *= 2.0 ** -112                                     # around the lower end
        elif kind == 3:
            m *= 2.0 ** 110                                      # around the upper end
        elif kind == 4:
            m = np.zeros(d)
            m[n % d] = -(2.0 ** (n % 20 - 10))
        elif kind == 5:
            m[n % d] = [np.nan, np.inf, -np.inf][n % 3]
        elif kind == 6:
            m = np.abs(m)
        x[0, 0, n] = m
    bits = f32_to_bf16_bits(np.nan_to_num(x, nan=0.0, posinf=1.0, neginf=1.0).astype(np.float32))
    bits = np.where(np.isnan(x), 0x7FC1, np.where(np.isposinf(x), 0x7F80, np.where(np.isneginf(x), 0xFF80, bits))).astype(np.uint16)
    host = bf16_bits_to_f32(bits).astype(np.float64)
    t = to_device_bf16(bits)
    c = Cache(1, 1, N, d, 1, None)
    c.append(t, t.clone(), [N])
    torch.cuda.synchronize()
    wc, ws = kv4.quantise(host)
    assert np.isnan(ws).sum() > 500 and (ws == 0).sum() > 100
    for codes, scales in c.host():
        assert np.array_equal(scales[0], ws[0], equal_nan=True)
        assert np.array_equal(codes[0], wc[0])


def test_bad_pages_are_skipped_and_read_as_zeros():
    import torch
    table = [[2, -1, 0], [7, 1, 1 << 30]]
    c = Cache(3, 2, 16, 64, 3, table)
    before = [b.clone() for b in c.buffers]
    (k, v), _ = tokens(2, 2, 48, 64, 12)
    c.append(k, v, [48, 48])
    torch.cuda.synchronize()
    # every page is written by exactly one of the named places
    assert not any(torch.isnan(s.float()).any() for s in (c.k_scales, c.v_scales))
    kb, vb = c.read([48, 48], 48)
    torch.cuda.synchronize()
    for got, x in ((kb, k), (vb, v)):
        for b, bad in ((0, [1]), (1, [0, 2])):
            for pg in range(3):
                part = got[b, :, pg * 16:(pg + 1) * 16]
                assert bool((part == 0).all()) == (pg in bad)
    assert before[0].shape == c.k_codes.shape


# ---------------------------------------------------------------- attention

def bounds(q, k, v, seen, scale, o, lse):
    """Largest |dO| [N, d] and |dLSE| [N] that the kernel's roundings allow, for one head.

    Scores: exact products of 8-bit numbers summed in 32 bits, d/16 tensor-core steps and the
    scale: (d/16 + 16 + 4) roundings of at most 2^-23 of the sum of magnitudes (truncating adds
    counted), and two more of the score itself in the exponent.  2^x: 2^-22.  A weight is rounded
    to bf16 and O divided by the sum of the rounded weights, so O moves by at most
    (2^-8 (1 + 2^-7) + weight error) times the mean distance of V from O; sums of n weights in 32
    bits by (n/16 + 40) 2^-23 of the mean magnitude; O rounds to bf16 once.  bf16 keeps 8
    significant bits: numbers of [1, 2) are 2^-7 apart, so a rounding is off by up to 2^-8.
    """
    n, d = q.shape[0], q.shape[1]
    eo, el = np.zeros((n, d)), np.zeros(n)
    for i in range(n):
        j = np.nonzero(seen[i])[0]
        if j.size == 0:
            continue
        s = scale * (k[j] @ q[i])
        mag = scale * (np.abs(k[j]) @ np.abs(q[i])).max()
        p = np.exp(s - lse[i])
        e_s = (d / 16 + 20) * 2.0 ** -23 * mag + 4 * 2.0 ** -23 * (np.abs(s).max() + abs(lse[i]) + 8) + 2.0 ** -21
        e_n = (j.size / 16 + 40) * 2.0 ** -23
        dist, size = p @ np.abs(v[j] - o[i]), p @ np.abs(v[j])
        eo[i] = (2.0 ** -8 * (1 + 2.0 ** -7) + 2 * e_s) * dist + 2 * e_n * size
        eo[i] += 2.0 ** -8 * (np.abs(o[i]) + eo[i])
        el[i] = e_s + e_n + 2.0 ** -22 * (abs(lse[i]) + 8)
    return eo, el


def run_kv4(c, q, key_lens, q_lens, scale, causal, window, workspace=None, stream=None):
    """fa_fwd_kv4 with guarded outputs; returns device tensors (o, lse) and whether the guards survived."""
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4, fa_fwd_kv4_workspace_size
    B, H, N, d = q.shape
    guard = 256
    o_buf = torch.full((q.numel() + 2 * guard,), -12345.0, dtype=torch.bfloat16, device="cuda")
    l_buf = torch.full((B * H * N + 2 * guard,), -777.0, dtype=torch.float32, device="cuda")
    o, lse = o_buf[guard:-guard].view(B, H, N, d), l_buf[guard:-guard].view(B, H, N)
    n = fa_fwd_kv4_workspace_size(B, H, c.H_kv, N, d)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    fa_fwd_kv4(q, *c.buffers, c.d_table, ints(key_lens), ints(q_lens), o, lse, B, H, c.H_kv, N, *c.sizes, scale, causal,
               window, ws, n, stream)
    torch.cuda.synchronize()
    ok = bool((o_buf[:guard] == -12345.0).all() and (o_buf[-guard:] == -12345.0).all()
              and (l_buf[:guard] == -777.0).all() and (l_buf[-guard:] == -777.0).all())
    return o, lse, ok


def check(c, q_bits, key_lens, q_lens, scale, causal, window, o, lse, heads=None, what=""):
    """Compare with the oracle, element by element, within the derived bounds."""
    q = bf16_bits_to_f32(q_bits).astype(np.float64)
    B, H, N, d = q.shape
    o, lse = to_host_f64(o), lse.cpu().numpy().astype(np.float64)
    top = c.max_pages * c.page_size
    worst = 0.0
    for b in range(B):
        L = min(max(int(key_lens[b]), 0), top)
        ql = N if q_lens is None else min(max(int(q_lens[b]), 0), N)
        k, v, there = c.positions(b, L)
        seen = kv4.visible_keys(N, ql, L, L, causal, window) & there[None, :]
        for h in (range(H) if heads is None else heads):
            kh, vh = k[h // (H // c.H_kv)], v[h // (H // c.H_kv)]
            ro, rl = kv4.attend(q[b, h], kh, vh, seen, scale)
            eo, el = bounds(q[b, h], kh, vh, seen, scale, ro, rl)
            empty = ~seen.any(1)
            assert np.all(np.isneginf(lse[b, h][empty])) and np.all(o[b, h][empty] == 0), f"{what}: empty rows"
            assert not np.signbit(o[b, h][empty]).any()
            nan = np.isnan(ro)
            assert np.array_equal(nan, np.isnan(o[b, h])), f"{what}: NaN"
            assert np.array_equal(np.isnan(rl), np.isnan(lse[b, h])), f"{what}: NaN in the LSE"
            fine = ~nan & ~empty[:, None]
            ratio = (np.abs(o[b, h] - ro)[fine] / np.maximum(eo[fine], 1e-30)).max(initial=0.0)
            live = ~empty & ~np.isnan(rl)
            lr = (np.abs(lse[b, h][live] - rl[live]) / el[live]).max(initial=0.0)
            assert ratio <= 1.0, f"{what}: b {b} h {h}: |dO| {ratio:.2f} of its bound"
            assert lr <= 1.0, f"{what}: b {b} h {h}: |dLSE| {lr:.2f} of its bound"
            worst = max(worst, ratio)
    return worst


def filled(B, H_kv, page, d, maxp, key_lens, seed, table="shuffled", sigma=1.0, edit=None):
    """A cache filled through fa_kv4_append; unwritten rows stay NaN."""
    num_pages = B * maxp + 1
    rng = np.random.default_rng(seed)
    t = rng.permutation(num_pages)[:B * maxp].reshape(B, maxp) if isinstance(table, str) else table
    c = Cache(num_pages, H_kv, page, d, maxp, t)
    L = max(1, max(min(max(n, 0), page * maxp) for n in key_lens))
    bits = [normal_bf16((B, H_kv, L, d), seed, i, sigma) for i in (1, 2)]
    if edit is not None:
        edit(*bits)
    k, v = (to_device_bf16(x) for x in bits)
    c.append(k, v, [L] * B)
    # what lies behind a sequence's length is made the worst there is again
    import torch
    worst = Cache(num_pages, H_kv, page, d, maxp, t)
    for b, n in enumerate(key_lens):
        for j in range(min(max(n, 0), page * maxp)):
            at = kv4.place(j, b, c.table, page, maxp, num_pages)
            if at is not None:
                for w, x in zip(worst.buffers, c.buffers):
                    w[at[0], :, at[1]] = x[at[0], :, at[1]]
    torch.cuda.synchronize()
    return worst


# B, H, H_kv, N_q, d, page_size, max_pages, key_lens, q_lens, causal, window
ATTEND = [
    (1, 1, 1, 1, 64, 16, 1, [1], None, False, -1),
    (1, 1, 1, 1, 128, 16, 1, [1], None, True, -1),
    (1, 1, 1, 1, 128, 16, 2, [17], None, False, -1),
    (2, 4, 2, 1, 128, 16, 20, [300, 0], None, False, -1),             # a sequence without keys
    (3, 6, 6, 1, 64, 32, 12, [129, 383, 1], None, True, -1),
    (1, 8, 1, 1, 128, 48, 20, [911], None, False, -1),                # 8 rows; pages of 48
    (1, 9, 1, 1, 64, 16, 20, [303], None, False, -1),                 # 9 rows: a second block of one
    (2, 24, 2, 1, 128, 64, 3, [100, 190], None, False, 50),
    (2, 2, 1, 5, 128, 16, 16, [250, 6], None, True, -1),
    (2, 4, 1, 5, 64, 16, 16, [250, 6], [5, 3], True, 20),             # ragged queries, window
    (3, 2, 2, 7, 128, 16, 4, [3, 40, 64], [7, 0, 2], True, -1),       # more queries than keys; none
    (1, 2, 1, 33, 128, 32, 8, [201], None, True, -1),
    (1, 4, 2, 40, 64, 32, 8, [201], None, True, 64),
    (2, 2, 1, 100, 128, 16, 8, [128, 100], [64, 100], True, -1),
    (2, 3, 3, 20, 64, 16, 8, [128, 90], None, False, 30),
    (1, 2, 2, 1, 128, 64, 40, [2500], None, False, 0),                # window 0: one key
    (1, 1, 1, 1, 128, 256, 16, [4096], None, False, -1),              # one head over many CTAs
    (1, 1, 1, 3, 64, 4096, 1, [4001], None, True, 3000),              # one page, window over many CTAs
    (40, 2, 2, 1, 64, 16, 4, list(range(1, 41)), None, False, -1),    # many short sequences
    (1, 1, 1, 128, 128, 32, 4, [128], None, True, -1),                # a whole prompt, few heads
    (1, 6, 2, 300, 64, 32, 40, [1111], None, True, 500),
    # many rows of many heads: the tensor-core tiles of 128 rows
    (4, 8, 8, 160, 128, 32, 12, [160, 300, 0, 371], [160, 100, 160, 7], True, -1),
    (4, 16, 8, 80, 64, 16, 30, [470, 80, 33, 200], None, True, 100),  # blocks that span heads; window
    (2, 64, 16, 70, 128, 48, 10, [470, 60], [70, 33], True, -1),
    (1, 32, 32, 200, 64, 64, 8, [201], None, False, -1),              # no causal mask
    (1, 40, 8, 129, 128, 128, 6, [700], None, True, 333),
    (1, 32, 32, 128, 128, 16, 8, [128], None, True, -1),              # whole prompts: one block of rows
    (64, 2, 2, 130, 64, 16, 13, [(37 * b) % 209 for b in range(64)], None, True, -1),
    # long keys of few heads: an item over many CTAs, merged in two levels
    (1, 8, 1, 1, 128, 32, 200, [6111], None, True, -1),
    (1, 3, 1, 1, 64, 16, 300, [4001], None, False, -1),
    (2, 13, 1, 1, 128, 16, 300, [4799, 3300], None, True, 4000),
    (3, 4, 2, 2, 64, 64, 60, [3833, 0, 3500], [2, 1, 1], True, -1),
    # many rows of few heads: the keys of a block in ranges, then joined
    (1, 8, 1, 5, 128, 32, 200, [6111], None, True, -1),
    (2, 4, 2, 33, 64, 16, 300, [4800, 129], [33, 20], True, -1),
    (3, 4, 2, 24, 128, 48, 70, [3300, 0, 50], None, False, -1),       # ranges without a key
    (1, 10, 5, 140, 64, 64, 40, [2222], [131], True, 700),            # ranges that windows leave out
    (1, 1, 1, 300, 128, 16, 160, [2500], None, True, -1),
    # room for much longer sequences and many heads: sixteen rows a block
    (8, 24, 8, 4, 128, 64, 128, [300, 0, 17, 2000, 129, 1, 777, 64], [4, 4, 0, 1, 3, 4, 4, 2], True, -1),
    (16, 16, 4, 4, 64, 16, 512, [(211 * b) % 1500 for b in range(16)], None, False, 100),
    (8, 64, 8, 2, 64, 48, 180, [5, 900, 48, 47, 2, 333, 1000, 96], None, True, -1),
    (8, 9, 9, 10, 128, 32, 256, [40, 1, 9, 10, 500, 128, 129, 127], None, True, 20),
]


@pytest.mark.parametrize("B,H,H_kv,N,d,page,maxp,key_lens,q_lens,causal,window", ATTEND)
def test_attention_matches_the_oracle(B, H, H_kv, N, d, page, maxp, key_lens, q_lens, causal, window):
    c = filled(B, H_kv, page, d, maxp, key_lens, 21)
    bits = normal_bf16((B, H, N, d), 22, 0)
    scale = float(np.float32(d ** -0.5))
    o, lse, guards = run_kv4(c, to_device_bf16(bits), key_lens, q_lens, scale, causal, window)
    assert guards
    heads = None if B * H * N < 2000 else sorted({0, H // 2, H - 1})
    check(c, bits, key_lens, q_lens, scale, causal, window, o, lse, heads=heads)


@pytest.mark.parametrize("sigma,scale", [(4.0, 0.5), (0.05, 1.0), (1.0, 30.0), (2.0 ** -60, 1.0)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,H_kv,N", [(3, 1, 2), (3, 1, 50), (16, 16, 150)])
def test_attention_on_steep_and_flat_scores(sigma, scale, d, H, H_kv, N):
    # steep: scores up to thousands, one key takes all; flat: every key counts alike
    key_lens = [700, 333]
    c = filled(2, H_kv, 16, d, 44, key_lens, 31, sigma=sigma)
    bits = normal_bf16((2, H, N, d), 32, 0, min(sigma, 4.0))
    o, lse, guards = run_kv4(c, to_device_bf16(bits), key_lens, None, scale, True, -1)
    assert guards
    check(c, bits, key_lens, None, scale, True, -1, o, lse, heads=None if H < 4 else [1], what=f"sigma {sigma}")


@pytest.mark.parametrize("H_kv,N", [(2, 1), (2, 20), (16, 65)])
def test_scores_that_grow_along_the_keys(H_kv, N):
    # every tile moves the reference max: all the rescaling there is
    def edit(k, v):
        ramp = np.linspace(0.0, 6.0, k.shape[2])[None, None, :, None]
        k[:] = f32_to_bf16_bits((0.01 * bf16_bits_to_f32(k) + ramp).astype(np.float32))
    c = filled(1, H_kv, 16, 128, 60, [960], 33, edit=edit)
    bits = f32_to_bf16_bits(np.ones((1, 4 * H_kv, N, 128), np.float32))
    o, lse, _ = run_kv4(c, to_device_bf16(bits), [960], None, 0.5, False, -1)
    check(c, bits, [960], None, 0.5, False, -1, o, lse, heads=[0, 2 * H_kv + 1])


@pytest.mark.parametrize("H_kv,N,rows", [(1, 3, 3), (1, 12, 24), (1, 40, 80), (32, 150, 150), (32, 100, 200), (4, 150, 300)])
@pytest.mark.parametrize("page", [16, 32])
def test_what_a_query_does_not_see_has_no_influence(H_kv, N, rows, page):
    # keys and values of the last tokens are NaN or infinite: the queries before them stay clean,
    # those that see them do not
    def edit(k, v):
        k[0, :, -2, 5] = 0x7FC0
        v[0, :, -1, 70] = 0x7F80
    key_lens = [200]
    c = filled(1, H_kv, page, 128, 13, key_lens, 34, edit=edit)
    bits = normal_bf16((1, H_kv * rows // N, N, 128), 35, 0)
    heads = [0] if H_kv == 1 else [0, H_kv * rows // N - 1]
    o, lse, _ = run_kv4(c, to_device_bf16(bits), key_lens, None, 0.09, True, -1)
    check(c, bits, key_lens, None, 0.09, True, -1, o, lse, heads=heads)
    import torch
    assert not torch.isnan(o[:, :, :N - 2].float()).any() and torch.isnan(o[:, :, N - 2:].float()).all()
    # behind a window too: an early poisoned value is out of sight of the last query
    def edit2(k, v):
        v[0, :, 190, 3] = 0xFF80
    c = filled(1, H_kv, page, 128, 13, key_lens, 34, edit=edit2)
    o, lse, _ = run_kv4(c, to_device_bf16(bits), key_lens, None, 0.09, True, 8)
    check(c, bits, key_lens, None, 0.09, True, 8, o, lse, heads=heads)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_poisoned_keys_and_missing_pages_with_sixteen_rows_a_block(d, page):
    import torch
    B, H_kv, N, n, pages = 8, 8, 12, 230, 8192 // page
    def edit(k, v):
        k[:, :, n - 2, 5] = 0x7FC0
        v[:, :, n - 1, 40] = 0x7F80
        v[:, :, 100, 9] = 0xFF80
    table = np.random.default_rng(45).permutation(B * pages).reshape(B, pages)
    lens = [n, n, n - 1, n - 2, 101, 100, 0, n]
    c = filled(B, H_kv, page, d, pages, [n] * B, 45, table=table, edit=edit)
    bits = normal_bf16((B, H_kv, N, d), 46, 0)
    q = to_device_bf16(bits)
    for window in (-1, 40):
        o, lse, _ = run_kv4(c, q, lens, None, 0.09, True, window)
        check(c, bits, lens, None, 0.09, True, window, o, lse, heads=[0, H_kv - 1], what=str(window))
    assert torch.isfinite(o[5].float()).all() and torch.isnan(o[0, :, -1].float()).all()
    table[:, 2] = -1
    c.table[...] = table
    c.d_table.copy_(ints(table))
    o, lse, _ = run_kv4(c, q, lens, [12, 5, 0, 12, 12, 12, 1, 1], 0.09, True, -1)
    check(c, bits, lens, [12, 5, 0, 12, 12, 12, 1, 1], 0.09, True, -1, o, lse, heads=[0, H_kv - 1])


@pytest.mark.parametrize("H,N", [(2, 1), (2, 3), (8, 30)])       # merged parts; ranges of keys
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_poisoned_keys_and_missing_pages_of_a_long_sequence(H, N, d, page):
    import torch
    def edit(k, v):
        k[0, :, -2, 5] = 0x7FC0
        v[0, :, -1, 40] = 0x7F80
    n = 5950
    pages = 6016 // page
    table = np.random.default_rng(39).permutation(pages)[None]
    c = filled(1, 1, page, d, pages, [n], 39, table=table, edit=edit)
    bits = normal_bf16((1, H, N, d), 40, 0)
    o, lse, _ = run_kv4(c, to_device_bf16(bits), [n], None, 0.09, True, -1)
    check(c, bits, [n], None, 0.09, True, -1, o, lse, heads=[0, H - 1])
    assert not torch.isnan(o[:, :, :max(0, N - 2)].float()).any() and torch.isnan(o[:, :, max(0, N - 2):].float()).any()
    table[0, pages // 5:pages // 2] = -1         # ranges without a page
    c.table[...] = table
    c.d_table.copy_(ints(table))
    for lens, window in (([n - 2], -1), ([n - 2], 3300), ([pages // 2 * page], 40)):
        o, lse, _ = run_kv4(c, to_device_bf16(bits), lens, None, 0.09, True, window)
        check(c, bits, lens, None, 0.09, True, window, o, lse, heads=[0, H - 1], what=str((lens, window)))


@pytest.mark.parametrize("H_kv,N", [(2, 3), (2, 30), (32, 75)])
def test_bad_pages_are_masked(H_kv, N):
    table = [[0, -1, 5, 2, 99, 1]]
    c = filled(1, H_kv, 16, 64, 6, [90], 36, table=table)
    bits = normal_bf16((1, 2 * H_kv, N, 64), 37, 0)
    heads = [0, 1, 2 * H_kv - 1]
    o, lse, _ = run_kv4(c, to_device_bf16(bits), [90], None, 0.125, True, -1)
    check(c, bits, [90], None, 0.125, True, -1, o, lse, heads=heads)
    o, lse, _ = run_kv4(c, to_device_bf16(bits), [5000], [2], 0.125, True, -1)     # length clamped to the pages
    check(c, bits, [5000], [2], 0.125, True, -1, o, lse, heads=heads)
    o, lse, _ = run_kv4(c, to_device_bf16(bits), [-3], None, 0.125, False, -1)
    check(c, bits, [-3], None, 0.125, False, -1, o, lse, heads=heads)


@pytest.mark.parametrize("N", [3, 300])
def test_a_cache_without_pages_is_empty(N):
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4, fa_fwd_kv4_workspace_size, fa_kv4_append, fa_kv4_read
    B, H, H_kv, d = 2, 4, 2, 64
    (k, v), _ = tokens(B, H_kv, N, d, 38)
    lens, none = ints([3, 3]), (None,) * 4
    for table, maxp in ((None, 0), (None, 4), (ints([[0] * 4] * B), 4)):
        fa_kv4_append(k, v, *none, table, lens, None, B, H_kv, N, d, 0, 16, maxp)
        kb, vb = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
        fa_kv4_read(*none, table, lens, None, kb, vb, B, H_kv, N, d, 0, 16, maxp)
        q = torch.ones((B, H, N, d), dtype=torch.bfloat16, device="cuda")
        o, lse = torch.full_like(q, 7.0), torch.full((B, H, N), 7.0, device="cuda")
        n = fa_fwd_kv4_workspace_size(B, H, H_kv, N, d)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        fa_fwd_kv4(q, *none, table, lens, None, o, lse, B, H, H_kv, N, d, 0, 16, maxp, 0.1, True, -1, ws, n)
        torch.cuda.synchronize()
        assert (kb == 0).all() and (vb == 0).all() and (o == 0).all() and torch.isneginf(lse).all()


def test_more_sequences_than_one_launch_takes():
    import torch
    B = 1500
    key_lens = [(7 * b) % 40 for b in range(B)]
    c = Cache(B, 1, 48, 64, 1, None)
    (k, v), _ = tokens(B, 1, 48, 64, 41)
    c.append(k, v, [48] * B)
    bits = normal_bf16((B, 2, 1, 64), 42, 0)
    o, lse, guards = run_kv4(c, to_device_bf16(bits), key_lens, None, 0.125, False, -1)
    assert guards
    check(c, bits, key_lens, None, 0.125, False, -1, o, lse)
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    import torch
    H_kv, page, d = 8, 1024, 128
    num_pages = (1 << 32) // (H_kv * page * d // 2) + 8      # codes of K alone exceed 2^32 bytes
    shape = (num_pages, H_kv, page)
    c = Cache(1, H_kv, page, d, 2, None)
    c.num_pages = num_pages
    c.k_codes = torch.empty((*shape, d // 2), dtype=torch.uint8, device="cuda")
    c.v_codes = torch.empty_like(c.k_codes)
    c.k_scales = torch.empty((*shape, d // 32), dtype=torch.bfloat16, device="cuda")
    c.v_scales = torch.empty_like(c.k_scales)
    c.table = np.array([[num_pages - 1, num_pages - 3]], np.int32)
    c.d_table = ints(c.table)
    (k, v), host = tokens(1, H_kv, 1100, d, 43)
    c.append(k, v, [1100])
    kb, vb = c.read([1100], 1100)
    torch.cuda.synchronize()
    for got, x in ((kb, host[0]), (vb, host[1])):
        assert np.array_equal(to_host_f64(got), kv4.values(*kv4.quantise(x)))
    bits = normal_bf16((1, 2 * H_kv, 1, d), 44, 0)
    o, lse, _ = run_kv4(c, to_device_bf16(bits), [1100], None, 0.088, False, -1)
    ks, vs = to_host_f64(kb), to_host_f64(vb)
    q = bf16_bits_to_f32(bits).astype(np.float64)
    seen = np.ones((1, 1100), bool)
    for h in (0, 7, 15):
        ro, rl = kv4.attend(q[0, h], ks[0, h // 2], vs[0, h // 2], seen, 0.088)
        eo, el = bounds(q[0, h], ks[0, h // 2], vs[0, h // 2], seen, 0.088, ro, rl)
        assert np.all(np.abs(to_host_f64(o)[0, h] - ro) <= eo)
        assert np.all(np.abs(lse.cpu().numpy()[0, h] - rl) <= el)


@pytest.mark.parametrize("H_kv,N", [(2, 1), (2, 5), (2, 40), (16, 70), (64, 4)])
def test_results_are_the_same_bits_each_time_and_on_another_stream(H_kv, N):
    import torch
    key_lens = [1900, 5, 777]
    c = filled(3, H_kv, 16, 128, 120, key_lens, 51)
    q = to_device_bf16(normal_bf16((3, 4 * H_kv, N, 128), 52, 0))
    o, lse, _ = run_kv4(c, q, key_lens, None, 0.09, True, -1)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        o2, lse2, _ = run_kv4(c, q, key_lens, None, 0.09, True, -1, stream=stream)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)


def test_a_decoding_loop_matches_the_dense_forward():
    """Append, read back and attend as a serving loop does: a prompt, then tokens one by one."""
    import torch
    B, H, H_kv, d, page, maxp = 2, 4, 2, 128, 16, 8
    prompt, steps = [70, 33], 4
    rng = np.random.default_rng(61)
    c = Cache(B * maxp, H_kv, page, d, maxp, rng.permutation(B * maxp).reshape(B, maxp))
    (k, v), _ = tokens(B, H_kv, max(prompt), d, 62)
    c.append(k, v, prompt, prompt)
    lens = list(prompt)
    for s in range(steps):
        (k1, v1), _ = tokens(B, H_kv, 1, d, 63 + s)
        lens = [n + 1 for n in lens]
        c.append(k1, v1, lens)
        bits = normal_bf16((B, H, 1, d), 80 + s, 0)
        o, lse, guards = run_kv4(c, to_device_bf16(bits), lens, None, 0.088, True, -1)
        assert guards
        check(c, bits, lens, None, 0.088, True, -1, o, lse, what=f"step {s}")
        # the dense forward on what is read back sees the same numbers (each within its own rounding)
        kb, vb = c.read(lens, max(lens))
        kd, vd = (x.repeat_interleave(H // H_kv, 1).contiguous().view(torch.int16).cpu().numpy().view(np.uint16) for x in (kb, vb))
        od, ld = run_fa(bits, kd, vd, 0.088, False, lens)
        assert np.abs(od - to_host_f64(o)).max() <= 2.0 ** -7 * np.abs(to_host_f64(vb)).max()
        assert np.abs(ld - lse.cpu().numpy()).max() <= 1e-4


@pytest.mark.parametrize("H,H_kv", [(4, 1), (16, 16)])
def test_captured_calls_replay_and_graphs_share_a_workspace(H, H_kv):
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4, fa_fwd_kv4_workspace_size, fa_kv4_append, fa_kv4_read
    B, d, page, maxp = 2, 64, 16, 100
    c = Cache(B * maxp, H_kv, page, d, maxp, None)
    (k, v), _ = tokens(B, H_kv, 1500, d, 71)
    c.append(k, v, [1500, 1500])
    lens = ints([900, 1400])
    (k1, v1), _ = tokens(B, H_kv, 1, d, 72)
    n = max(fa_fwd_kv4_workspace_size(B, H, H_kv, N, d) for N in (1, 5, 140))
    ws = torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
    graphs = []
    for N in (1, 5, 140):
        bits = normal_bf16((B, H, N, d), 73, 0)
        q = to_device_bf16(bits)
        o, lse = torch.empty_like(q), torch.empty((B, H, N), dtype=torch.float32, device="cuda")
        kb = torch.empty((B, H_kv, 3, d), dtype=torch.bfloat16, device="cuda")
        vb = torch.empty_like(kb)

        def step():
            fa_kv4_append(k1, v1, *c.buffers, None, lens, None, B, H_kv, 1, *c.sizes)
            fa_kv4_read(*c.buffers, None, lens, None, kb, vb, B, H_kv, 3, *c.sizes)
            fa_fwd_kv4(q, *c.buffers, None, lens, None, o, lse, B, H, H_kv, N, *c.sizes, 0.125, True, -1, ws, n)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append((graph, bits, o, lse, (q, kb, vb)))     # a graph's buffers live as long as it does
    for new in ([900, 1400], [17, 1500], [1500, 1], [1500, 1], [640, 641]):
        lens.copy_(ints(new))
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, bits, o, lse, _ in graphs:
            check(c, bits, new, None, 0.125, True, -1, o, lse, heads=[0, H - 1], what=str(new))


def test_long_sequences_of_few_heads_in_graphs_that_share_a_workspace():
    """Items over many CTAs, merged in two levels, and ranges of keys that are joined, as the
    sequence grows and shrinks under the captured calls."""
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4, fa_fwd_kv4_workspace_size
    H, d, page, maxp = 8, 128, 32, 200
    c = filled(1, 1, page, d, maxp, [6400], 74)
    lens = ints([6400])
    n = max(fa_fwd_kv4_workspace_size(1, H, 1, N, d) for N in (1, 2, 4, 30))
    ws = torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
    graphs = []
    for N in (1, 2, 4, 30):
        bits = normal_bf16((1, H, N, d), 75, 0)
        q = to_device_bf16(bits)
        o, lse = torch.empty_like(q), torch.empty((1, H, N), dtype=torch.float32, device="cuda")

        def step():
            fa_fwd_kv4(q, *c.buffers, c.d_table, lens, None, o, lse, 1, H, 1, N, *c.sizes, 0.0625, True, -1, ws, n)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append((graph, bits, o, lse, q))
    for new in ([6400], [17], [6001], [6001], [0], [1290], [6399]):
        lens.copy_(ints(new))
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, bits, o, lse, _ in graphs:
            check(c, bits, new, None, 0.0625, True, -1, o, lse, heads=[0, H - 1], what=str(new))


@pytest.mark.parametrize("H,N,keys", [(2, 8, 3000), (8, 1, 6000), (3, 20, 6000), (1, 150, 5000)])
def test_workspace_contents_do_not_matter_and_nothing_past_it_is_touched(H, N, keys):
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4_workspace_size
    key_lens = [keys]
    c = filled(1, 1, 64, 128, 100, key_lens, 91)
    q = to_device_bf16(normal_bf16((1, H, N, 128), 92, 0))
    n = fa_fwd_kv4_workspace_size(1, H, 1, N, 128)
    want = None
    for fill in (0, 0xFF, 0x7F):
        buf = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")
        o, lse, _ = run_kv4(c, q, key_lens, None, 0.09, True, -1, workspace=buf)
        assert bool((buf[n:] == fill).all())
        if want is not None:
            assert torch.equal(o.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])
        want = (o, lse)


def test_two_calls_at_once_and_one_workspace_for_unlike_shapes():
    """Calls on two streams with a workspace each, and calls in turn on one workspace, whose parts
    lie elsewhere for every shape."""
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4_workspace_size
    shapes = [(3, 8, 1, 64, [1500, 40, 900]), (2, 2, 3, 128, [700, 1999]), (1, 4, 20, 128, [2000]), (2, 16, 70, 64, [300, 500])]
    cases = []
    for i, (B, H_kv, N, d, key_lens) in enumerate(shapes):
        c = filled(B, H_kv, 32, d, 63, key_lens, 95 + i)
        q = to_device_bf16(normal_bf16((B, 2 * H_kv, N, d), 96 + i, 0))
        cases.append((c, q, key_lens, run_kv4(c, q, key_lens, None, 0.1, True, -1)))
    n = max(fa_fwd_kv4_workspace_size(q.shape[0], q.shape[1], c.H_kv, q.shape[2], q.shape[3]) for c, q, _, _ in cases)
    ws = torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda")
    for c, q, key_lens, (o, lse, _) in cases + cases[::-1] + cases:
        o2, lse2, _ = run_kv4(c, q, key_lens, None, 0.1, True, -1, workspace=ws)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    from io_aware_exact_24_b200 import fa_fwd_kv4
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for turn in range(6):
        for s, space in zip(streams, spaces):
            c, q, key_lens, want = cases[(turn + (s is streams[0])) % len(cases)]
            o, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
            lens = ints(key_lens)
            torch.cuda.current_stream().synchronize()
            fa_fwd_kv4(q, *c.buffers, c.d_table, lens, None, o, lse, q.shape[0], q.shape[1], c.H_kv, q.shape[2], *c.sizes, 0.1,
                       True, -1, space, n, s)
            outs.append((o, lse, want, lens))
    torch.cuda.synchronize()
    for o, lse, want, _ in outs:
        assert torch.equal(o.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])


def test_lengths_below_zero_are_empty():
    import torch
    c = Cache(4, 2, 16, 64, 2, None)
    (k, v), _ = tokens(2, 2, 5, 64, 97)
    c.append(k, v, [3, 9], [-1, -7])
    torch.cuda.synchronize()
    assert torch.isnan(c.k_scales.float()).all()          # nothing was written
    kb, vb = c.read([-1, -9], 4)
    bits = normal_bf16((2, 2, 3, 64), 98, 0)
    o, lse, _ = run_kv4(c, to_device_bf16(bits), [-1, 0], [-5, 3], 0.1, True, -1)
    assert (kb == 0).all() and (vb == 0).all() and (o == 0).all() and torch.isneginf(lse).all()


# ---------------------------------------------------------------- scales that the format has not

# bf16 bits: finite ones from 2^118 on, the first that overflows times 24, infinities, NaN
NO_SCALES = [0x7A80, 0xFB00, 0x7D2B, 0x7D80, 0x7F00, 0xFF00, 0x7F7F, 0x7F80, 0xFF80, 0x7FC0]


def bf16_of(bits):
    import torch
    return torch.tensor(np.array(bits, np.uint16).view(np.int16)).cuda().view(torch.bfloat16)


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,H_kv,N", [(1, 1, 1), (2, 2, 3), (4, 2, 12), (8, 4, 20), (32, 32, 150), (4, 1, 150)])
def test_rows_that_were_never_written_have_no_influence(H, H_kv, N, d, page):
    """A layer with a window appends the last tokens of a prompt alone: the rows before them, in the
    same page and the same tile, are whatever the memory held, and so are those behind the last token."""
    import torch
    n, window, B, maxp = 30 * page + 13, 7, 2, 32            # no query sees a position before n - N - window
    rand = torch.Generator(device="cuda")
    rand.manual_seed(107)
    bits = normal_bf16((B, H, N, d), 102, 0)
    q = to_device_bf16(bits)
    (k, v), _ = tokens(B, H_kv, N + window, d, 103)
    table = np.random.default_rng(104).permutation(B * maxp).reshape(B, maxp)
    for i, scale in enumerate(NO_SCALES):
        c = Cache(B * maxp, H_kv, page, d, maxp, table)
        for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
            codes.random_(generator=rand)
            scales[...] = bf16_of([scale])[0]
        c.append(k, v, [n, n], [N + window] * B)
        for causal, w in ((True, window), (False, window)):
            o, lse, guards = run_kv4(c, q, [n, n], None, 0.11, causal, w)
            assert guards
            assert not np.isnan(to_host_f64(o)).any() and np.isfinite(lse.cpu().numpy()).all(), hex(scale)
            if i < 2:
                check(c, bits, [n, n], None, 0.11, causal, w, o, lse, heads=sorted({0, H - 1}), what=hex(scale))


@pytest.mark.parametrize("H_kv,N", [(2, 1), (2, 12), (2, 20), (32, 150)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_a_scale_that_append_cannot_write_stands_for_nan(H_kv, N, d, page):
    """The queries that see such a group get NaN, in its channels where it is V's; the others do not."""
    import torch
    n = 9 * page + 5
    bits = normal_bf16((1, H_kv, N, d), 105, 0)
    q = to_device_bf16(bits)
    clean = filled(1, H_kv, page, d, 10, [n], 106)
    for what in ("k", "v"):
        # the largest below 2^118, and the largest of five bits.  The products of a scale of more bits
        # are not exact: 24 s is rounded by at most 2^-8 of it, and that is all that is left of a code 8
        for scale in NO_SCALES + [0x7A7F, 0x7A78]:
            number = scale not in NO_SCALES
            c = Cache(11, H_kv, page, d, 10, clean.table)
            for a, b in zip(c.buffers, clean.buffers):
                a.copy_(b)
            at, off = kv4.place(n - 1, 0, c.table, page, 10, 11)
            codes, scales = (c.k_codes, c.k_scales) if what == "k" else (c.v_codes, c.v_scales)
            codes[at, :, off] = 0x88                                  # every code stands for 0 * s
            scales[at, :, off, 1] = bf16_of([scale])[0]
            kb, vb = c.read([n], n)
            got = to_host_f64(kb if what == "k" else vb)[0, :, n - 1]
            assert np.isnan(got[:, 32:64]).all() != number and not np.isnan(got[:, :32]).any()
            if number:
                assert (np.abs(got[:, 32:64]) <= (24 * 2.0 ** 110 * 255 if scale == 0x7A7F else 0) * 2.0 ** -8).all()
            o, lse, _ = run_kv4(c, q, [n], None, 0.11, True, -1)
            if scale != 0x7A7F:
                check(c, bits, [n], None, 0.11, True, -1, o, lse, heads=[0, H_kv - 1], what=what + hex(scale))
            o = to_host_f64(o)
            assert not np.isnan(o[:, :, :-1]).any()
            assert np.isnan(o[:, :, -1, 32:64]).all() != number
    torch.cuda.synchronize()


# ---------------------------------------------------------------- calls that overlap

@pytest.mark.parametrize("B,H,H_kv,N,d,page,n", [(1, 4, 4, 1, 128, 16, 70), (2, 8, 4, 40, 64, 32, 300), (24, 8, 8, 1, 128, 64, 200),
                                                 (4, 16, 16, 150, 128, 16, 1500)])
def test_queued_calls_see_what_the_one_before_wrote(B, H, H_kv, N, d, page, n):
    """read, append of other values at the same positions, read, attend, many times without waiting
    on the host, and attention on what a read gave back: each call has the answers that it has alone."""
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4, fa_fwd_kv4_workspace_size, fa_kv4_append, fa_kv4_read
    maxp, turns, sets = -(-n // page), 30, 3
    table = ints(np.random.default_rng(111).permutation(B * maxp).reshape(B, maxp))
    lens, first = ints([n] * B), ints([n - N] * B)
    base, _ = tokens(B, H_kv, n, d, 112)
    new = [tokens(B, H_kv, N, d, 113 + i)[0] for i in range(sets)]
    q = [to_device_bf16(normal_bf16((B, H, N, d), 120 + i, 0)) for i in range(sets)]
    size = fa_fwd_kv4_workspace_size(B, H, H_kv, N, d)
    ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
    empty = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")

    def run(wait):
        c = Cache(B * maxp, H_kv, page, d, maxp, None)
        again = Cache(B * maxp, H_kv, page, d, maxp, None)
        out = [[empty(B, H_kv, N, d) for _ in range(4)] + [empty(B, H, N, d), empty(B, H, N, t=torch.float32)] for _ in range(turns)]
        torch.cuda.synchronize()
        done = torch.cuda.synchronize if wait else (lambda: None)
        fa_kv4_append(*base, *c.buffers, table, lens, None, B, H_kv, n, *c.sizes)
        for i, (k0, v0, k1, v1, o, lse) in enumerate(out):
            done()
            fa_kv4_read(*c.buffers, table, lens, first, k0, v0, B, H_kv, N, *c.sizes)
            done()
            fa_kv4_append(*new[i % sets], *c.buffers, table, lens, None, B, H_kv, N, *c.sizes)
            done()
            fa_kv4_read(*c.buffers, table, lens, first, k1, v1, B, H_kv, N, *c.sizes)
            done()
            # what was just read is written to another cache
            fa_kv4_append(k1, v1, *again.buffers, table, lens, None, B, H_kv, N, *again.sizes)
            done()
            fa_fwd_kv4(q[i % sets], *c.buffers, table, lens, None, o, lse, B, H, H_kv, N, *c.sizes, 0.1, True, -1, ws, size)
        torch.cuda.synchronize()
        return out + [list(c.buffers), list(again.buffers)]

    want = run(True)
    for got in (run(False), run(False)):
        for i, (g, w) in enumerate(zip(got, want)):
            for j, (a, b) in enumerate(zip(g, w)):
                a, b = (x.view(torch.int16) if x.dtype == torch.bfloat16 else x for x in (a, b))
                assert torch.equal(a, b), (i, j)
    for k0, k1, turn in ((want[i + 1][0], want[i][2], i) for i in range(turns - 1)):
        assert torch.equal(k0, k1), turn
        assert turn % sets == 0 or not torch.equal(k0, want[turn - 1][2])


def test_bad_pages_touch_no_other_page():
    """A page that two bad entries could be mistaken for, and every row behind the named ones, keep their bits."""
    import torch
    c = Cache(5, 2, 16, 64, 3, [[2, -1, 0], [5, 1, (1 << 31) - 1]])
    (k, v), _ = tokens(2, 2, 48, 64, 12)
    before = [b.clone() for b in c.buffers]
    c.append(k, v, [48, 48])
    torch.cuda.synchronize()
    named = {0: (0, 32), 2: (0, 0), 1: (1, 16)}              # page: sequence, its first token
    for got, was, x in zip(c.buffers, before, (k, k, v, v)):
        for page in range(5):
            same = torch.equal(got[page].view(torch.uint8), was[page].view(torch.uint8))
            assert same == (page not in named), page
    kb, vb = c.read([48, 48], 48)
    for got, x in ((kb, k), (vb, v)):
        back = kv4.values(*kv4.quantise(to_host_f64(x)))
        want = np.zeros_like(back)
        for b, at in named.values():
            want[b, :, at:at + 16] = back[b, :, at:at + 16]
        assert np.array_equal(to_host_f64(got), want)


def test_captured_calls_on_two_streams_that_fork_and_join():
    """K and V are made on a side stream, written there, and attended on another: each call has one or
    two predecessors of unlike kinds in the graph."""
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4, fa_fwd_kv4_workspace_size, fa_kv4_append, fa_kv4_read
    B, H, H_kv, N, d, page, maxp, n = 2, 8, 2, 5, 128, 16, 20, 300
    c = filled(B, H_kv, page, d, maxp, [n, n], 161)
    src = [tokens(B, H_kv, N, d, 162 + i)[0] for i in range(3)]
    bits = [normal_bf16((B, H, N, d), 170 + i, 0) for i in range(3)]
    k, v = (torch.empty_like(x) for x in src[0])
    q_src = [to_device_bf16(b) for b in bits]
    q, lens = torch.empty_like(q_src[0]), ints([n, n])
    feed = [x.clone() for x in (*src[0], q_src[0])]
    k1, v1 = torch.empty_like(k), torch.empty_like(v)
    o, lse = torch.empty_like(q), torch.empty((B, H, N), dtype=torch.float32, device="cuda")
    size = fa_fwd_kv4_workspace_size(B, H, H_kv, N, d)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            k.copy_(feed[0])
            v.copy_(feed[1])
            fa_kv4_append(k, v, *c.buffers, c.d_table, lens, None, B, H_kv, N, *c.sizes)
            fa_kv4_read(*c.buffers, c.d_table, lens, ints_first, k1, v1, B, H_kv, N, *c.sizes)
        torch.mul(feed[2], 1.0, out=q)
        main.wait_stream(side)
        fa_fwd_kv4(q, *c.buffers, c.d_table, lens, None, o, lse, B, H, H_kv, N, *c.sizes, 0.1, True, -1, ws, size)
    ints_first = ints([n - N] * B)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in (1, 2, 0, 1):
        for f, x in zip(feed, (*src[turn], q_src[turn])):
            f.copy_(x)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for got, x in ((k1, src[turn][0]), (v1, src[turn][1])):
            assert np.array_equal(to_host_f64(got), kv4.values(*kv4.quantise(to_host_f64(x))))
        check(c, bits[turn], [n, n], None, 0.1, True, -1, o, lse, heads=[0, H - 1], what=str(turn))


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("B,H,H_kv,N,d,page,maxp,key_lens", [
    (1, 8, 1, 5, 128, 32, 200, [6111]),                       # ranges of keys that are joined
    (2, 4, 2, 33, 64, 16, 300, [4800, 0]),                    # and a sequence without keys
    (4, 8, 8, 160, 128, 32, 40, [900, 1200, 0, 371]),
    (64, 2, 2, 130, 64, 16, 40, [(37 * b) % 609 for b in range(64)]),      # one CTA a block of rows
])
def test_a_wait_that_runs_out_leaves_nan_and_the_next_call_is_right(B, H, H_kv, N, d, page, maxp, key_lens):
    """With a wait limit of a few cycles the kernel for many rows winds down; no row has an answer that
    leaves keys out: it is the right one, bit for bit, or NaN.  The context stays usable."""
    import torch
    from io_aware_exact_24_b200 import (FA_ERR_DEVICE_TIMEOUT, FA_ERR_INVALID_ARG, FA_OK, fa_fwd_kv4_workspace_size,
                                        fa_get_device_status, fa_selftest_kv4_timeout)
    c = filled(B, H_kv, page, d, maxp, key_lens, 131)
    bits = normal_bf16((B, H, N, d), 132, 0)
    q, lens = to_device_bf16(bits), ints(key_lens)
    n = fa_fwd_kv4_workspace_size(B, H, H_kv, N, d)
    ws = torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda")      # (numbers, if taken for results)
    want = run_kv4(c, q, key_lens, None, 0.1, True, -1, workspace=ws)
    assert fa_get_device_status() == FA_OK
    for limit in (2, 2, 300, 3000):
        o, lse = torch.full_like(q, 3.0), torch.full((B, H, N), 3.0, device="cuda")
        st = fa_selftest_kv4_timeout(q, *c.buffers, c.d_table, lens, None, o, lse, B, H, H_kv, N, *c.sizes, 0.1, True, -1, ws, n, limit)
        assert st == FA_ERR_DEVICE_TIMEOUT if limit == 2 else st in (FA_ERR_DEVICE_TIMEOUT, FA_OK)
        assert fa_get_device_status() == FA_OK                # read and cleared by the call
        same = (o.view(torch.int16) == want[0].view(torch.int16)).all(-1) & (lse == want[1])
        lost = torch.isnan(o).all(-1) & torch.isnan(lse)
        assert (same | lost).all(), limit
        assert lost.any() == (st == FA_ERR_DEVICE_TIMEOUT)
        o2, lse2, guards = run_kv4(c, q, key_lens, None, 0.1, True, -1, workspace=ws)
        assert guards and torch.equal(o2.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse2, want[1])
    assert fa_selftest_kv4_timeout(q, *c.buffers, c.d_table, lens, None, o, lse, B, H, H_kv, 1, *c.sizes, 0.1, True, -1, ws, n,
                                   2) == FA_ERR_INVALID_ARG
    check(c, bits, key_lens, None, 0.1, True, -1, *want[:2], heads=[0, H - 1])


# ---------------------------------------------------------------- the ends of the range of V

@pytest.mark.parametrize("end", ["top", "bottom"])
@pytest.mark.parametrize("H,H_kv,N", [(1, 1, 1), (2, 1, 3), (16, 16, 1), (12, 2, 2), (8, 1, 8), (32, 32, 150), (4, 1, 150)])
@pytest.mark.parametrize("d,n", [(64, 700), (128, 3000)])
def test_values_at_the_ends_of_the_format(H, H_kv, N, d, n, end):
    """V up to 2^120, all keys alike or after a tile that leaves the reference max 7 octaves behind, and
    V down to 2^-107: O stays within the derived bound.

    At the bottom, sums keep multiples of 2^-149 at weights of at least 2^-16 for the largest, so besides
    the relative bounds O moves by (n/16 + 40) 2^-149 / 2^-16, and by 2^-134 where it rounds to a
    subnormal bf16 number."""
    page, maxp = 32, -(-n // 32)
    top = 2.0 ** 120 if end == "top" else 2.0 ** -107
    for lag in (False, True):
        def edit(k, v):
            x = bf16_bits_to_f32(k).astype(np.float64) * 0.01
            # scores of q = 1 are scale * sum of k: 0 for the first 128 keys, then 7 octaves above
            x[..., 0] += np.where(np.arange(n) < 128, 0.0, 7.0 * np.log(2.0)) if lag else 0.0
            k[:] = f32_to_bf16_bits(x.astype(np.float32))
            y = bf16_bits_to_f32(v).astype(np.float64)
            y = np.clip(y / 4.0, -1.0, 1.0) * top
            y[..., 5], y[..., 40] = top, -top                # and channels where all values are alike
            v[:] = f32_to_bf16_bits(y.astype(np.float32))
        c = filled(1, H_kv, page, d, maxp, [n], 141 + lag, edit=edit)
        q = np.ones((1, H, N, d))
        bits = f32_to_bf16_bits(q.astype(np.float32))
        o, lse, guards = run_kv4(c, to_device_bf16(bits), [n], None, 1.0, True, -1)
        assert guards
        o, lse = to_host_f64(o), lse.cpu().numpy().astype(np.float64)
        assert np.isfinite(o).all() and np.isfinite(lse).all()
        kk, vv, _ = c.positions(0, n)
        assert np.abs(vv).max() == top and np.isfinite(vv).all()
        seen = kv4.visible_keys(N, N, n, n, True, -1)
        for h in sorted({0, H - 1}):
            kh, vh = kk[h // (H // H_kv)], vv[h // (H // H_kv)]
            ro, rl = kv4.attend(q[0, h], kh, vh, seen, 1.0)
            eo, el = bounds(q[0, h], kh, vh, seen, 1.0, ro, rl)
            if end == "bottom":
                eo = eo + (n / 16 + 40) * 2.0 ** -133 + 2.0 ** -134
            assert (np.abs(o[0, h] - ro) <= eo).all(), (lag, h, (np.abs(o[0, h] - ro) / eo).max())
            assert (np.abs(lse[0, h] - rl) <= el).all()


# ---------------------------------------------------------------- tensors that do not fit

def test_tensors_that_do_not_fit_are_refused_and_nothing_is_touched():
    """int64 lengths, a slice of a wider table, one tensor for codes of K and V, tensors on the CPU."""
    import torch
    from io_aware_exact_24_b200 import fa_fwd_kv4, fa_fwd_kv4_workspace_size, fa_kv4_append, fa_kv4_read
    B, H, H_kv, N, d, page, maxp, num = 2, 2, 2, 3, 64, 16, 2, 8
    k = torch.zeros((B, H_kv, N, d), dtype=torch.bfloat16, device="cuda")
    kb, q, o = k.clone(), k.clone(), k.clone()
    lse = torch.zeros((B, H, N), device="cuda")
    codes = torch.full((num, H_kv, page, d // 2), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((num, H_kv, page, d // 32), 7.0, dtype=torch.bfloat16, device="cuda")
    size = fa_fwd_kv4_workspace_size(B, H, H_kv, N, d)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    good = dict(kc=codes, ks=scales, vc=codes.clone(), vs=scales.clone(), table=ints([[0, 1], [2, 3]]), lens=ints([3, 3]),
                new=ints([3, 3]), k=k, v=k.clone(), q=q, o=o, lse=lse, ws=ws)
    keep = {n: t.clone() for n, t in good.items()}

    def calls(**kw):
        a = good | kw
        cache = (a["kc"], a["ks"], a["vc"], a["vs"], a["table"], a["lens"])
        sizes = (d, num, page, maxp)
        return (lambda: fa_kv4_append(a["k"], a["v"], *cache, a["new"], B, H_kv, N, *sizes),
                lambda: fa_kv4_read(*cache, a["new"], a["k"], a["v"], B, H_kv, N, *sizes),
                lambda: fa_fwd_kv4(a["q"], *cache, a["new"], a["o"], a["lse"], B, H, H_kv, N, *sizes, 0.1, True, -1, a["ws"], size))
    wide = ints([[0, 1, 9, 9], [2, 3, 9, 9]])
    both = torch.zeros((num, H_kv, page, 2, d // 2), dtype=torch.uint8, device="cuda")
    every, attend = (0, 1, 2), (2,)
    for kw, which in ((dict(lens=ints([3, 3], np.int64)), every), (dict(new=ints([3, 3], np.int64)), every),
                      (dict(table=ints([[0, 1], [2, 3]], np.int64)), every), (dict(table=wide[:, :2]), every),
                      (dict(lens=ints([3, 3, 3, 3])[::2]), every), (dict(kc=both[..., 0, :], vc=both[..., 1, :]), every),
                      (dict(ks=scales.half()), every), (dict(vs=scales.float()), every), (dict(lens=ints([3, 3]).cpu()), every),
                      (dict(table=good["table"].cpu()), every), (dict(vc=codes.cpu()), every), (dict(k=k.half()), (0, 1)),
                      (dict(q=q.transpose(1, 2)), attend), (dict(lse=lse.double()), attend), (dict(lse=lse.cpu()), attend),
                      (dict(ws=ws.cpu()), attend), (dict(ws=torch.zeros(2 * size, dtype=torch.uint8, device="cuda")[::2]), attend)):
        for i in which:
            with pytest.raises(ValueError):
                calls(**kw)[i]()
    torch.cuda.synchronize()
    for n, t in good.items():
        assert torch.equal(t, keep[n]), n
    for call in calls():
        call()
    torch.cuda.synchronize()
    assert not torch.equal(codes, keep["kc"])


@pytest.mark.parametrize("H,H_kv,N", [(1, 1, 1), (3, 1, 4), (12, 2, 2), (32, 32, 150), (4, 1, 150)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("high", [12, 18, 23.5])
def test_large_scores_take_the_largest_key(H, H_kv, N, d, high):
    """Scores up to 2^high: O stays within V's range, and where the largest score leads the others by
    more than all roundings, e = (d/16 + 28) 2^-23 2^high in the natural exponent, and 30 besides, its
    value comes back (other weights sum to less than n e^-30 < 2^-30) and the LSE is it, within e."""
    n, page = 700, 32
    c = filled(1, H_kv, page, d, 22, [n], 191)
    bits = normal_bf16((1, H, N, d), 192, 0)
    q = bf16_bits_to_f32(bits).astype(np.float64)
    kk, vv, _ = c.positions(0, n)
    raw = np.stack([q[0, h] @ kk[h // (H // H_kv)].T for h in range(H)])               # [H, N, n]
    mag = np.stack([np.abs(q[0, h]) @ np.abs(kk[h // (H // H_kv)]).T for h in range(H)]).max()
    scale = float(np.float32(2.0 ** high / mag))
    o, lse, guards = run_kv4(c, to_device_bf16(bits), [n], None, scale, False, -1)
    assert guards
    o, lse = to_host_f64(o)[0], lse.cpu().numpy().astype(np.float64)[0]
    s = np.sort(scale * raw, -1)
    e = (d / 16 + 28) * 2.0 ** -23 * 2.0 ** high
    clear = s[..., -1] - s[..., -2] > 2 * e + 30
    assert clear.mean() > 0.5 or clear.size < 100
    for h in range(H):
        v = vv[h // (H // H_kv)]
        assert (np.abs(o[h]) <= np.abs(v).max(0) * (1 + 2.0 ** -7)).all()              # P's rounding and O's
        best = v[raw[h].argmax(-1)]
        assert (np.abs(o[h] - best)[clear[h]] <= 2.0 ** -8 * np.abs(best)[clear[h]] + 2.0 ** -25).all()
        assert (np.abs(lse[h] - s[h, :, -1])[clear[h]] <= e + 2.0 ** -20 * 2.0 ** high).all()


# ---------------------------------------------------------------- sixteen rows a block

@pytest.mark.parametrize("B,H,H_kv,N,d,page,maxp,window", SIXTEEN_ROWS)
def test_sixteen_rows_a_block(B, H, H_kv, N, d, page, maxp, window):
    """Ragged lengths and queries, windows, foreign scales in rows that no query sees, missing pages."""
    import torch
    top = page * maxp
    key_lens = [top if b == 0 else (53 * b) % top for b in range(B)]
    q_lens = [N if b % 3 else b % (N + 1) for b in range(B)]
    table = np.random.default_rng(151).permutation(B * maxp).reshape(B, maxp)
    c = Cache(B * maxp, H_kv, page, d, maxp, table)
    (k, v), _ = tokens(B, H_kv, top, d, 152)
    c.append(k, v, [top] * B)
    bits = normal_bf16((B, H, N, d), 153, 0)
    q = to_device_bf16(bits)
    for causal in (True, False):
        o, lse, guards = run_kv4(c, q, key_lens, q_lens, 0.1, causal, window)
        assert guards
        check(c, bits, key_lens, q_lens, 0.1, causal, window, o, lse, heads=[0, H - 1], what=str(causal))
    # rows behind the lengths, and those that all windows leave out, hold what was never written
    want = run_kv4(c, q, key_lens, None, 0.1, True, window)
    for scale in (0x7D80, 0xFF80, 0x7FC0):
        for b in range(0, B, max(1, B // 7)):
            for j in range(top):
                if j >= key_lens[b] or (window >= 0 and j < key_lens[b] - N - window):
                    for s in (c.k_scales, c.v_scales):
                        s[int(table[b][j // page]), :, j % page] = bf16_of([scale])[0]
        o, lse, _ = run_kv4(c, q, key_lens, None, 0.1, True, window)
        assert torch.equal(o.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1]), hex(scale)
    table[:, 1::3] = -1
    c.table[...] = table
    c.d_table.copy_(ints(table))
    o, lse, _ = run_kv4(c, q, key_lens, None, 0.1, True, window)
    check(c, bits, key_lens, None, 0.1, True, window, o, lse, heads=[0, H - 1], what="missing pages")


# ---------------------------------------------------------------- padding and shared pages

@pytest.mark.parametrize("H,H_kv,N", [(4, 2, 3), (2, 1, 40), (16, 16, 150)])
@pytest.mark.parametrize("fill", [0x7FC0, 0x7F80, 0xFF7F])
def test_padding_may_hold_anything_and_sequences_may_share_pages(H, H_kv, N, fill):
    """Tokens and queries behind a sequence's own are NaN, infinite or huge; the sequences after the
    first continue its pages (a common prefix), and one is the same as another."""
    import torch
    B, d, page, maxp, prefix = 4, 128, 16, 24, 160
    new = [N, N // 2, 1, 0]
    lens = [prefix + n for n in new]
    own = -(-N // page)
    table = np.full((B, maxp), -1)
    table[:, :prefix // page] = np.arange(prefix // page)[::-1]
    for b in range(B):
        table[b, prefix // page:prefix // page + own] = prefix // page + b * own + np.arange(own)
    c = Cache(prefix // page + B * own, H_kv, page, d, maxp, table)
    (k0, v0), _ = tokens(1, H_kv, prefix, d, 181)
    c.append(k0, v0, [prefix])                                # through the first sequence's pages
    (k, v), _ = tokens(B, H_kv, N, d, 182)
    bits = normal_bf16((B, H, N, d), 183, 0)
    for b in range(B):
        for x in (k, v):
            x[b, :, new[b]:] = bf16_of([fill])[0]
        bits[b, :, new[b]:] = fill
    c.append(k, v, lens, new)
    for causal, window in ((True, -1), (False, -1), (True, 30)):
        o, lse, guards = run_kv4(c, to_device_bf16(bits), lens, new, 0.1, causal, window)
        assert guards and torch.isfinite(o.float()).all()
        clean = np.where(np.arange(N)[None, None, :, None] < np.array(new)[:, None, None, None], bits, 0).astype(np.uint16)
        check(c, clean, lens, new, 0.1, causal, window, o, lse, heads=[0, H - 1], what=str((causal, window)))
    # the same sequence twice: the same answers
    c.table[1], same = table[0], to_device_bf16(bits)
    c.d_table.copy_(ints(c.table))
    same[1] = same[0]
    o, lse, _ = run_kv4(c, same, [lens[0], lens[0], *lens[2:]], [new[0], new[0], *new[2:]], 0.1, True, -1)
    assert torch.equal(o[0].view(torch.int16), o[1].view(torch.int16)) and torch.equal(lse[0], lse[1])
