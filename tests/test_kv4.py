"""CPU tests of the 4-bit key/value cache: the format's oracle against hand-worked groups and
its own properties, and the refusals of the entry points (no GPU touched)."""
import os
import re

import numpy as np
import pytest

import oracle.kv4 as kv4
from io_aware_exact_24_b200 import binding
from io_aware_exact_24_b200.build import build
from io_aware_exact_24_b200.inputs import bf16_bits_to_f32, f32_to_bf16_bits, normal_bf16

from fa_testutil import SIXTEEN_ROWS


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


# ---------------------------------------------------------------- the format

def test_a_hand_worked_group():
    # m = -4: s = 0.5 (16 * 2^-5); codes are x / 0.5 + 8, 3.6 -> 7.2 -> 15 and +4 -> 8 clamps to 15
    x = np.zeros(32)
    x[:6] = [-4.0, 4.0 - 2 ** -6, 3.6, 0.25, 0.75, -0.26]
    codes, s = kv4.quantise(x)
    assert s[0] == 0.5
    # 0.25 / 0.5 and 0.75 / 0.5 are ties: to the even 0 and 2
    assert list(codes[:7]) == [0, 15, 15, 8, 10, 7, 8]
    assert list(kv4.values(codes, s)[:6]) == [-4.0, 3.5, 3.5, 0.0, 1.0, -0.5]


def test_the_sign_of_the_scale_follows_the_extreme_value():
    x = np.zeros(32)
    x[3], x[9] = 6.0, -6.0
    codes, s = kv4.quantise(x)                  # an equal pair: the positive one sets the sign
    assert s[0] == -0.75 and codes[3] == 0 and codes[9] == 15
    codes, s = kv4.quantise(-np.abs(x))
    assert s[0] == 0.75 and codes[3] == 0 and codes[9] == 0


@pytest.mark.parametrize("m,s", [(1.0, -0.125), (255 / 128, -0.25), (131 / 128, -0.125 * 16 / 16),
                                 (133 / 128, -0.125 * 17 / 16), (132 / 128, -0.125 * 16 / 16),
                                 (140 / 128, -0.125 * 18 / 16), (-140 / 128, 0.125 * 18 / 16)])
def test_scales_round_to_five_bits_ties_to_even(m, s):
    # |m| * 128 = 131 .. 133 stand 3/8, 4/8 (a tie: down to the even 16) and 5/8 between 16 and 17;
    # 140 is the tie between 17 and 18; 255 rounds up into the next power of two
    x = np.zeros(32)
    x[5] = m
    assert kv4.scale_of(x) == s


def test_values_are_bf16_numbers_and_near():
    x = bf16_bits_to_f32(normal_bf16((64, 128), 3, 0)).astype(np.float64)
    codes, s = kv4.quantise(x)
    y = kv4.values(codes, s)
    assert np.array_equal(bf16_bits_to_f32(f32_to_bf16_bits(y.astype(np.float32))).astype(np.float64), y)
    step = np.abs(np.repeat(s, 32, axis=-1))
    # half a step, or up to 1.25 steps next to the value opposite to the extreme one
    assert np.all(np.abs(x - y) <= np.where(np.abs(x) > 7.5 * step, 1.25, 0.5) * step)
    assert np.array_equal(kv4.unpack(kv4.pack(codes)), codes)


def test_a_product_with_a_near_reciprocal_rounds_as_the_quotient():
    # what the kernels rely on: an 8-bit over a 5-bit significand is k + 1/2 or at least 2^-9 from
    # it, so x * (1/s), with 1/s off by an ulp or two, on a grid of 2^-11, ties where x / s does
    x, s, e = np.meshgrid(np.arange(128, 256), np.arange(16, 32), np.arange(-9, 1), indexing="ij")
    x = x * 2.0 ** e
    quotient = x / s
    keep = quotient <= 8.25
    off = np.abs(quotient - np.floor(quotient) - 0.5)[keep]
    assert off[off > 0].min() == 2.0 ** -9
    near = (1.0 / s).astype(np.float32)
    for steps in (-2, -1, 0, 1, 2):
        inv = near.copy()
        for _ in range(abs(steps)):
            inv = np.nextafter(inv, np.float32(np.sign(steps) * 4), dtype=np.float32)
        for sign in (1, -1):
            on_grid = np.rint((6144.0 + sign * x * inv.astype(np.float64)) * 2048.0) / 2048.0
            assert np.array_equal(np.rint(on_grid - 6144.0)[keep], np.rint(sign * quotient)[keep])


@pytest.mark.parametrize("bad,want", [(np.nan, "nan"), (np.inf, "nan"), (-np.inf, "nan"), (2.0 ** 121, "nan"),
                                      (2.0 ** -108, "zero"), (2.0 ** 120, "value"), (2.0 ** -107, "value")])
def test_ends_of_the_range(bad, want):
    x = np.zeros((1, 64))
    x[0, 7] = bad
    y = kv4.values(*kv4.quantise(x))
    assert np.all(y[0, 32:] == 0)               # the other group does not notice
    if want == "nan":
        assert np.all(np.isnan(y[0, :32]))
    elif want == "zero":
        assert np.all(y[0, :32] == 0)
    else:
        assert y[0, 7] == bad


@pytest.mark.parametrize("s,nan", [(2.0 ** 117, False), (2.0 ** 118 - 2.0 ** 110, False), (2.0 ** 118, True), (-2.0 ** 124, True),
                                   (np.inf, True), (-np.inf, True), (np.nan, True)])
def test_scales_that_the_format_has_not(s, nan):
    # the largest that a group can have is 2^117 (of 2^120); of foreign ones, 2^118 is the first to stand for NaN
    y = kv4.values(np.arange(16, dtype=np.uint8).repeat(2)[None], np.array([[s]]))
    assert np.all(np.isnan(y)) if nan else np.array_equal(y[0], (np.arange(16).repeat(2) - 8.0) * s)


def bf16_round(x):
    """float64 to the bf16 numbers, ties to even, past 2^128 - 2^119 to infinity."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        m, e = np.frexp(x)
        e = np.maximum(e, -125)                  # subnormal numbers are multiples of 2^-133
        y = np.ldexp(np.rint(np.ldexp(x, 8 - e)), e - 8)
    y = np.where(np.isfinite(x), y, x)
    return np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, x), y)


def test_the_arithmetic_of_the_codes_gives_the_format():
    # what the kernels compute, each step rounded to bf16: t = 1024 s, z = t - 131/128 t (-24 s, or
    # NaN from |s| = 2^118 on, where t is infinite), and (16 + c) s + z
    bits = np.arange(1 << 16, dtype=np.uint16)
    with np.errstate(all="ignore"):
        s = bf16_bits_to_f32(bits).astype(np.float64)
        t = bf16_round(s * 1024.0)
        z = bf16_round(t * (-131.0 / 128.0) + t)
        got = [bf16_round((16.0 + c) * s + z) for c in range(16)]
    five = np.isfinite(s) & (bits & 7 == 0) & (np.abs(s) >= 2.0 ** -110) & (np.abs(s) <= 2.0 ** 117)   # what append writes
    assert five.sum() == 2 * (227 * 16 + 1)
    for c in range(16):
        nan = ~(np.abs(s) < 2.0 ** 118)
        assert np.array_equal(np.isnan(got[c]), nan)
        assert np.array_equal(got[c][five], (c - 8) * s[five])
        assert np.all(np.isfinite(got[c][~nan]))


def test_attend_ignores_what_a_query_does_not_see():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 64)), rng.normal(size=(9, 64)), rng.normal(size=(9, 64))
    seen = kv4.visible_keys(3, 3, 7, 9, True, 2)
    assert seen.tolist() == [[j in r for j in range(9)] for r in ((2, 3, 4), (3, 4, 5), (4, 5, 6))]
    o, lse = kv4.attend(q, k, v, seen, 0.125)
    k[[0, 1, 7, 8]] = np.nan
    v[[0, 1, 7, 8]] = np.inf
    o2, lse2 = kv4.attend(q, k, v, seen, 0.125)
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)
    for i, r in enumerate(((2, 3, 4), (3, 4, 5), (4, 5, 6))):
        p = np.exp(0.125 * k[list(r)] @ q[i])
        np.testing.assert_allclose(o[i], p @ v[list(r)] / p.sum(), rtol=1e-12)
        np.testing.assert_allclose(lse[i], np.log(p.sum()), rtol=1e-12)
    assert kv4.visible_keys(4, 2, 7, 7, False, -1).sum(1).tolist() == [7, 7, 0, 0]
    assert kv4.visible_keys(5, 5, 2, 4, True, -1).sum(1).tolist() == [0, 0, 0, 1, 2]


def test_places():
    assert kv4.place(-1, 0, None, 16, 2, 9) is None and kv4.place(32, 0, None, 16, 2, 9) is None
    assert kv4.place(17, 3, None, 16, 2, 9) == (7, 1) and kv4.place(17, 4, None, 16, 2, 9) is None
    assert kv4.place(17, 0, [[4, 9]], 16, 2, 9) is None and kv4.place(15, 0, [[4, 9]], 16, 2, 9) == (4, 15)
    assert kv4.place(15, 0, [[-1, 9]], 16, 2, 9) is None


# ---------------------------------------------------------------- launches that overlap

def test_kernels_that_overlap_the_one_before_load_nothing_as_read_only():
    # their blocks may be resident while the kernel before still writes what they will read: the
    # non-coherent path is for memory that nobody writes during a kernel's lifetime
    csrc = os.path.join(os.path.dirname(binding.__file__), "csrc")
    for name in sorted(f for f in os.listdir(csrc) if f.startswith("fa_kv4") and f.endswith(".cuh")):
        code = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, name)).read())
        assert not re.search(r"__ldg\s*\(|\.nc\b|__restrict__", code), name
        # and each begins by waiting for it: nothing of its parameters' memory is touched before
        for kernel in re.findall(r"__global__[^{]*?(\w+_kernel)\(", code):
            body = code[code.index(kernel + "("):]
            before = body[:body.index("after_previous();")]
            assert not re.search(r"p\.(q|k|v|o|lse|part|part_ml|words|key_lens|\w+_codes|\w+_scales)\b|tma_load|cp_async16", before), kernel


# ---------------------------------------------------------------- the choice of a kernel

# B, H_kv, rows a head (the queries), keys, d, window, and us measured on one B200 of the kernel for
# few rows with 8 and with 16 rows a block, and of the one for many rows
MEASURED = [
    (8, 8, 20, 16, 128, -1, 6.1, 8.1, 8.1),
    (8, 8, 512, 16, 128, -1, 40.3, 42.6, 17),
    (64, 32, 20, 16, 128, -1, 56.2, 81.2, 106.4),
    (64, 32, 512, 1, 128, -1, 1190.6, 1336.7, 441.8),
    (64, 32, 200, 16, 64, -1, 367.6, 381.3, 202.5),
    (8, 8, 4096, 64, 128, -1, 327.9, 314.5, 115.8),
    (8, 8, 4096, 64, 64, -1, 252.2, 211.8, 103.7),
    (256, 1, 64, 64, 128, -1, 45.1, 29.2, 16.7),
    (8, 32, 200, 1, 128, -1, 58.3, 69.5, 31.7),
    (8, 32, 9, 128, 128, -1, 9.9, 7.7, 14.8),
    (100, 1, 300, 60, 128, -1, 95.8, 65.7, 22.3),
    (100, 1, 700, 5, 64, -1, 180.6, 113.3, 33.5),
    (100, 1, 24, 60, 128, -1, 8.9, 10.2, 8.8),
    (125, 8, 100, 60, 128, -1, 149.4, 158.1, 58.6),
    (125, 8, 40, 60, 64, -1, 45.1, 47.5, 50.5),
    (75, 2, 300, 260, 128, -1, 155.9, 133.2, 40.9),
    (37, 4, 10, 260, 64, -1, 15.8, 18.8, 11),
    (1, 8, 20, 700, 128, -1, 10.2, 13.1, 12.2),
    (1, 8, 256, 700, 128, -1, 19.3, 16.6, 14.3),
    (8, 8, 20, 700, 128, -1, 13.7, 16.3, 16.7),
    (8, 8, 256, 700, 64, -1, 47.5, 39.7, 13.7),
    (16, 32, 20, 700, 64, -1, 35.7, 38.2, 48.5),
    (1, 2, 9, 131072, 128, -1, 30.6, 51.3, 44.8),
    (1, 2, 16, 131072, 64, -1, 24.4, 39.1, 34.9),
    (1, 8, 20, 8192, 128, -1, 19, 19.9, 15.9),
    (1, 8, 1024, 8192, 128, -1, 261.2, 173.6, 58.5),
    (8, 8, 20, 4096, 128, -1, 36.5, 35.8, 33.4),
    (8, 8, 64, 4096, 128, -1, 78, 56.6, 34.4),
    (8, 8, 256, 4096, 128, -1, 267.9, 183.5, 52),
    (8, 32, 16, 2048, 128, -1, 46.5, 39, 55),
    (2, 8, 16, 32768, 128, -1, 46.9, 40.7, 49.7),
    (1, 8, 16, 8192, 128, -1, 18.1, 23.4, 15.8),
    (8, 8, 64, 2048, 64, -1, 31.9, 26.7, 17.7),
    (16, 4, 20, 8192, 128, 2048, 26.4, 27.7, 27.3),
    (8, 8, 512, 8192, 128, 16, 43.4, 43.2, 21.3),
    (1, 8, 512, 8192, 64, 64, 9.5, 7.4, 10.9),
    (64, 8, 20, 8192, 128, 128, 29, 37.9, 41.3),
    (8, 8, 64, 8192, 128, 100, 12.3, 14.3, 10.1),
]


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    import ctypes
    import subprocess
    at = tmp_path_factory.mktemp("rule")
    (at / "rule.cc").write_text("""
        #include "fa_kv4_rule.h"
        extern "C" int choose(int B, int H_kv, long long R, int N_q, int d, long long keys, int window, int sms, int *splits) {
            const fa::kv4::Choice c = fa::kv4::choose(B, H_kv, R, N_q, d, keys, window, sms);
            *splits = c.splits;
            return c.many ? 128 : c.rows_a_block;
        }""")
    csrc = os.path.join(os.path.dirname(binding.__file__), "csrc")
    subprocess.run(["g++", "-O1", "-Wall", "-Werror", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error",
                    "-shared", "-fPIC", "-I", csrc, "-o", str(at / "rule.so"), str(at / "rule.cc")], check=True)
    fn = ctypes.CDLL(str(at / "rule.so")).choose
    i32, i64 = ctypes.c_int, ctypes.c_longlong
    fn.argtypes = [i32, i32, i64, i32, i32, i64, i32, i32, ctypes.POINTER(i32)]

    def choose(B, H_kv, R, N_q, d, keys, window=-1, sms=148):
        splits = i32()
        return fn(B, H_kv, R, N_q, d, keys, window, sms, ctypes.byref(splits)), splits.value
    return choose


@pytest.mark.parametrize("B,H_kv,R,keys,d,window,us8,us16,many", MEASURED)
def test_the_choice_of_a_kernel_is_near_the_quickest(rule, B, H_kv, R, keys, d, window, us8, us16, many):
    kind, splits = rule(B, H_kv, R, R, d, -(-keys // 64) * 64, window)
    us = {8: us8, 16: us16, 128: many}
    if R <= 16:
        us.pop(128)
    assert us[kind] <= 1.3 * min(us.values())
    assert 1 <= splits <= max(1, 148 // (-(-R // 128) * B * H_kv))


@pytest.mark.parametrize("B,H,H_kv,N,d,page,maxp,window", SIXTEEN_ROWS)
def test_calls_with_sixteen_rows_a_block(rule, B, H, H_kv, N, d, page, maxp, window):
    assert rule(B, H_kv, H // H_kv * N, N, d, page * maxp, window)[0] == 16      # what the GPU tests of these rely on


def test_the_choice_of_a_kernel_at_the_ends_of_what_it_is_given(rule):
    for B in (1, 65535):
        for H_kv in (1, 65535):
            for R in (1, 8, 9, 17, 1 << 30):
                for keys in (0, 16, 1 << 30):
                    for window in (-1, 0, 1 << 30):
                        for d in (64, 128):
                            kind, splits = rule(B, H_kv, R, R, d, keys, window)
                            assert kind in (8, 16, 128) and 1 <= splits <= 148
                            assert kind != 128 or R > 16
                            assert splits == 1 or B * H_kv * R <= 148 * 128


# ---------------------------------------------------------------- refusals

P = 1 << 20   # a fake, suitably aligned address: validation must fail before it is used
INVALID, UNSUPPORTED, MISALIGNED = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_ERR_MISALIGNED


def append(k=P, v=P, kc=P, ks=P, vc=P, vs=P, table=P, key_lens=P, lens=P, B=1, H_kv=1, N=1, d=64, num_pages=4,
           page_size=16, max_pages=4):
    return binding.fa_kv4_append(k, v, kc, ks, vc, vs, table, key_lens, lens, B, H_kv, N, d, num_pages, page_size,
                                 max_pages, stream=0, check=False)


def read(k=P, v=P, kc=P, ks=P, vc=P, vs=P, table=P, key_lens=P, lens=P, B=1, H_kv=1, N=1, d=64, num_pages=4,
         page_size=16, max_pages=4):
    return binding.fa_kv4_read(kc, ks, vc, vs, table, key_lens, lens, k, v, B, H_kv, N, d, num_pages, page_size,
                               max_pages, stream=0, check=False)


def fwd(q=P, o=P, lse=P, kc=P, ks=P, vc=P, vs=P, table=P, key_lens=P, lens=P, B=1, H=2, H_kv=1, N=1, d=64,
        num_pages=4, page_size=16, max_pages=4, scale=0.125, causal=0, window=-1, ws=P, ws_bytes=1 << 40):
    return binding.fa_fwd_kv4(q, kc, ks, vc, vs, table, key_lens, lens, o, lse, B, H, H_kv, N, d, num_pages, page_size,
                              max_pages, scale, causal, window, ws, ws_bytes, stream=0, check=False)


SHARED = [
    (dict(d=32), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(B=-1), INVALID), (dict(H_kv=-1), INVALID), (dict(N=-1), INVALID), (dict(num_pages=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(page_size=-16), INVALID),
    (dict(page_size=24), INVALID), (dict(page_size=8), INVALID),
    (dict(page_size=1 << 20, max_pages=(1 << 10) + 1), UNSUPPORTED),
    (dict(B=70000), UNSUPPORTED),
    (dict(key_lens=None), INVALID), (dict(kc=None), INVALID), (dict(ks=None), INVALID), (dict(vc=None), INVALID),
    (dict(vs=None), INVALID),
    (dict(kc=P + 8), MISALIGNED), (dict(ks=P + 2), MISALIGNED), (dict(vc=P + 4), MISALIGNED), (dict(vs=P + 8), MISALIGNED),
    (dict(table=P + 2), MISALIGNED), (dict(key_lens=P + 1), MISALIGNED), (dict(lens=P + 3), MISALIGNED),
]
TOKENS = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=P + 8), MISALIGNED), (dict(v=P + 2), MISALIGNED),
          (dict(H_kv=65536), UNSUPPORTED), (dict(B=65535, H_kv=65535), UNSUPPORTED),
          (dict(N=(1 << 30) + 1), UNSUPPORTED)]
FWD = [
    (dict(H=3, H_kv=2), INVALID), (dict(H=-2), INVALID), (dict(H=65536), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=1e-46), INVALID),
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(ws=None), INVALID),
    (dict(q=P + 8), MISALIGNED), (dict(o=P + 4), MISALIGNED), (dict(lse=P + 2), MISALIGNED), (dict(ws=P + 128), MISALIGNED),
    (dict(ws_bytes=1024), INVALID), (dict(N=1 << 30, H=8), UNSUPPORTED),
    (dict(H=4096, H_kv=4096, page_size=1 << 20, max_pages=1 << 10), UNSUPPORTED),
]


@pytest.mark.parametrize("call,kw,code",
                         [(c, kw, code) for c in (append, read) for kw, code in SHARED + TOKENS]
                         + [(fwd, kw, code) for kw, code in SHARED + FWD],
                         ids=lambda x: x.__name__ if callable(x) else str(x))
def test_refusals_come_before_any_cuda_call(lib, call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("call", [append, read, fwd])
@pytest.mark.parametrize("kw", [dict(B=0), dict(N=0), dict(B=0, kc=None, key_lens=None, table=None)], ids=str)
def test_empty_problems_are_noops(lib, call, kw):
    assert call(**kw) == binding.FA_OK


def test_no_heads_is_a_noop(lib):
    assert append(H_kv=0) == read(H_kv=0) == fwd(H=0) == fwd(H=0, H_kv=0) == binding.FA_OK
    assert fwd(H=2, H_kv=0) == INVALID


def test_without_a_gpu_valid_calls_report_no_device(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("would launch on fake addresses")
    for call in (append, read, fwd):
        assert call() == binding.FA_ERR_NO_DEVICE
        assert call(table=None, lens=None) == binding.FA_ERR_NO_DEVICE
        assert call(num_pages=0, kc=None, ks=None, vc=None, vs=None) == binding.FA_ERR_NO_DEVICE


def test_selftest_timeout_argument_errors(lib):
    def f(limit=2, H=2, N=200, **kw):
        a = dict(B=1, H_kv=1, num_pages=4, page_size=1024, max_pages=4, key_lens=P, ws=P) | kw
        return binding.fa_selftest_kv4_timeout(P, P, P, P, P, P, a["key_lens"], P, P, P, a["B"], H, a["H_kv"], N, 64, a["num_pages"],
                                               a["page_size"], a["max_pages"], 0.125, 1, -1, a["ws"], 1 << 40, limit, stream=0)
    for kw in (dict(limit=0), dict(limit=(1 << 32) + 1), dict(B=0), dict(N=0), dict(H=0), dict(key_lens=None), dict(ws=None),
               dict(H_kv=3)):
        assert f(**kw) == INVALID, kw
    if not has_gpu():
        assert f() == binding.FA_ERR_NO_DEVICE


def has_gpu():
    import torch
    return torch.cuda.is_available()


def test_arguments_become_the_same_call(lib):
    """The marshalling module and ctypes hand the library the same values (B = 0: nothing is done)."""
    import ctypes
    import torch
    t = torch.zeros(64, dtype=torch.uint8)
    # (the table is only taken as an address)
    assert append(table=t, key_lens=None, B=0) == append(table=t.data_ptr(), key_lens=None, B=0) == binding.FA_OK
    for kw in ({}, dict(d=96), dict(ws_bytes=16), dict(q=P + 2), dict(N=0), dict(scale=-1), dict(window=7, causal=1, H=0)):
        a = dict(q=P, o=P, lse=P, kc=P, ks=P, vc=P, vs=P, table=P, key_lens=P, lens=P, B=1, H=2, H_kv=1, N=1, d=64,
                 num_pages=4, page_size=16, max_pages=4, scale=0.125, causal=0, window=-1, ws=P, ws_bytes=1 << 40) | kw
        if torch.cuda.is_available() and not kw:
            continue
        st = lib.fa_fwd_kv4(a["q"], a["kc"], a["ks"], a["vc"], a["vs"], a["table"], a["key_lens"], a["lens"], a["o"], a["lse"],
                            a["B"], a["H"], a["H_kv"], a["N"], a["d"], a["num_pages"], a["page_size"], a["max_pages"],
                            ctypes.c_float(a["scale"]), a["causal"], a["window"], a["ws"], a["ws_bytes"], None)
        assert fwd(**kw) == st
    for bad in (dict(q="x"), dict(B=1.5j), dict(B=1 << 40), dict(scale="y"), dict(ws_bytes=-1)):
        with pytest.raises((TypeError, OverflowError)):
            fwd(**bad)
    assert fwd(B=np.int64(0), scale=np.float32(0.5)) == binding.FA_OK


def test_tensors_elsewhere_are_refused(lib):
    import torch
    t = torch.zeros(64, dtype=torch.uint8)
    for call, kw in ((append, dict(k=t)), (append, dict(v=t)), (append, dict(kc=t)), (read, dict(k=t)), (read, dict(kc=t)),
                     (fwd, dict(q=t)), (fwd, dict(o=t)), (fwd, dict(kc=t))):
        with pytest.raises(ValueError, match="device"):
            call(B=0, **kw)

    class Elsewhere:                            # a tensor of another device, and one that is not contiguous
        def __init__(self, device, contiguous):
            self.device, self.contiguous = device, contiguous

        def get_device(self):
            return self.device

        def is_contiguous(self):
            return self.contiguous

        def data_ptr(self):
            return P

    here = torch.cuda.current_device() if torch.cuda.is_available() else 0
    for call, kw in ((append, "k"), (append, "v"), (read, "k"), (read, "v"), (fwd, "q"), (fwd, "o")):
        assert call(B=0, **{kw: Elsewhere(here, True)}) == binding.FA_OK
        with pytest.raises(ValueError, match="device"):
            call(B=0, **{kw: Elsewhere(here + 1, True)})
        with pytest.raises(ValueError, match="contiguous"):
            call(B=0, **{kw: Elsewhere(here, False)})


def test_other_entry_points_do_without_the_marshalling_module(lib):
    import subprocess
    import sys
    code = """
import sys
sys.modules["io_aware_exact_24_b200._fastcall"] = None          # as if it had not been built
import io_aware_exact_24_b200 as fa
P = 1 << 20
assert fa.fa_fwd(P, P, P, P, P, 0, 1, 8, 8, 64, 0.125, 0, None, 0) == fa.FA_OK
assert fa.binding.fa_fwd(P, P, P, P, P, 1, 1, 8, 8, 96, 0.125, 0, None, 0, False) == fa.FA_ERR_UNSUPPORTED
assert fa.fa_fwd_kv4_workspace_size(1, 1, 1, 1, 64) > 0
for _ in range(2):
    try:
        fa.fa_kv4_append(P, P, P, P, P, P, P, P, P, 0, 1, 1, 64, 4, 16, 4, 0)
    except ImportError as e:
        assert "_fastcall" in str(e)
    else:
        raise AssertionError("no error")
"""
    root = os.path.dirname(os.path.dirname(binding.__file__))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)


def test_the_library_is_built_where_the_marshalling_module_cannot_be(tmp_path, monkeypatch, capfd):
    from io_aware_exact_24_b200 import build as module
    monkeypatch.setattr(module, "FAST_OUT", str(tmp_path / "_fastcall.so"))
    for cc in ("false", str(tmp_path / "no_such_compiler")):
        (tmp_path / "_fastcall.so").write_text("of older sources")
        os.utime(tmp_path / "_fastcall.so", (1, 1))
        monkeypatch.setenv("CC", cc)
        assert module.build() == module.OUT
        assert "4-bit cache calls are not available" in capfd.readouterr().err
        assert not (tmp_path / "_fastcall.so").exists()


TYPES = dict(k="bfloat16", v="bfloat16", q="bfloat16", o="bfloat16", lse="float32", kc="uint8", vc="uint8", ks="bfloat16",
             vs="bfloat16", table="int32", key_lens="int32", lens="int32", ws=None)


class Tensor:
    """What the marshalling looks at."""

    def __init__(self, dtype, device=0, contiguous=True):
        self.dtype, self.device, self.contiguous = dtype, device, contiguous

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return P


@pytest.mark.parametrize("call,name", [(c, n) for c, names in ((append, "k v"), (read, "k v"), (fwd, "q o lse ws"))
                                       for n in (names + " kc ks vc vs table key_lens lens").split()])
def test_every_tensor_is_looked_at(lib, call, name):
    import torch
    here = torch.cuda.current_device() if torch.cuda.is_available() else 0
    dtype = getattr(torch, TYPES[name] or "uint8")
    # d = 96 is refused by the library, so that nothing is launched where all is well
    assert call(d=96, **{name: Tensor(dtype, here)}) == UNSUPPORTED
    with pytest.raises(ValueError, match="device"):
        call(d=96, **{name: torch.zeros(64, dtype=dtype)})                     # on the CPU
    with pytest.raises(ValueError, match="device"):
        call(d=96, **{name: Tensor(dtype, here + 1)})
    with pytest.raises(ValueError, match="contiguous"):
        call(d=96, **{name: Tensor(dtype, here, False)})
    for other in (torch.int64, torch.float16, torch.float32, torch.bfloat16, torch.int32, torch.uint8):
        if other != dtype and TYPES[name] is not None:
            with pytest.raises(ValueError, match="expected"):
                call(d=96, **{name: Tensor(other, here)})
    with pytest.raises(TypeError):
        call(d=96, **{name: "x"})


def test_workspace_size(lib):
    n = binding.fa_fwd_kv4_workspace_size(3, 8, 2, 1, 128)
    assert n > 0 and n % 256 == 0
    assert binding.fa_fwd_kv4_workspace_size(3, 8, 2, 5, 128) > 0
    for bad in ((0, 8, 2, 1, 128), (3, 8, 3, 1, 128), (3, 8, 0, 1, 128), (3, 8, 2, 0, 128), (3, 8, 2, 1, 96), (3, -8, 2, 1, 64)):
        assert binding.fa_fwd_kv4_workspace_size(*bad) == 0
