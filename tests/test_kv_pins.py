"""The cache's reference against hand-computed values, and the calls' refusals (CPU)."""
import numpy as np
import pytest

from oracle import kv
from variable_precision_weight_b200 import build, synth


@pytest.fixture(scope="module")
def fl():
    build.build()
    from variable_precision_weight_b200 import fl as mod
    return mod


def test_quantise_by_hand():
    x = np.zeros((4, 64))
    x[0, :4] = [127, -127, 63.5, 0.5]        # scale 1: ties to even
    x[1, :3] = [2.0, -1.0, 2.0 / 254]        # 127, -63.5 -> -64, 0.5 -> 0
    x[3, 0] = np.inf
    code, scale = kv.quantise(x)
    assert code[0, :4].tolist() == [127, -127, 64, 0]
    assert code[1, :3].tolist() == [127, -64, 0]
    assert scale[0] == 1.0 and scale[1] == np.float32(2.0) / np.float32(127.0)
    assert scale[2] == 0 and not code[2].any()
    assert np.isnan(scale[3]) and not code[3].any()


def test_fp32_quotient_gives_the_exact_code():
    """rint(127 x / a) in fp32 (one exact product, one rounded division) equals the exact one for
    bf16 x and a: every 8-bit significand pair, exponents up to nine binades apart."""
    sig = np.arange(128, 256, dtype=np.float64)
    for e in range(0, 10):
        x, a = np.meshgrid(sig * 2.0 ** -e, sig)
        ok = x <= a
        f = np.rint((x.astype(np.float32) * np.float32(127)) / a.astype(np.float32))
        num, den = (127 * x * 2 ** 9).astype(np.int64), (a * 2 ** 9).astype(np.int64)
        fl2, rem2 = num // den, num % den
        want = fl2 + ((2 * rem2 > den) | ((2 * rem2 == den) & (fl2 % 2 == 1)))
        assert np.array_equal(f[ok].astype(np.int64), want[ok]), e


def test_layout_by_hand():
    assert kv.element_place(128, "k", 0, 0) == (0, 0)
    assert kv.element_place(128, "k", 0, 1) == (2, 0)       # odd dims in the upper half of the word
    assert kv.element_place(128, "k", 0, 2) == (0, 1)
    assert kv.element_place(128, "k", 2, 0) == (8, 0)
    assert kv.element_place(128, "k", 1, 16) == (16 * 5, 0)
    assert kv.element_place(128, "k", 4, 64) == (16 * 32 * 3, 0)
    assert kv.element_place(64, "v", 0, 8) == (0, 1)
    assert kv.element_place(64, "v", 1, 0) == (2, 0) and kv.element_place(64, "v", 2, 0) == (1, 0)
    assert kv.element_place(64, "v", 17, 3) == (16 * (12 + 1) + 2, 0)
    for D in (64, 128):
        kv.places(D, "k"), kv.places(D, "v")                 # every place used once


@pytest.mark.parametrize("D", [64, 128])
def test_record_round_trip(D):
    g = np.random.default_rng(D)
    rec = g.integers(0, 256, kv.record_bytes(D), dtype=np.uint8)
    k, v = g.integers(-127, 128, (2, 64, D)).astype(np.int8)
    for j in g.permutation(64):
        kv.write_token(rec, D, j, k[j], 1.0, v[j], 2.0)
    kk, vv, _ = kv.read_record(rec, D, 4)
    assert np.array_equal(kk, k) and np.array_equal(vv, 2.0 * v)
    kk, vv, _ = kv.read_record(rec, D, 2)
    assert np.abs(kk - k).max() <= 8 and np.abs(vv - 2.0 * v).max() <= 16
    kk, _, _ = kv.read_record(rec, D, 0)
    assert not kk.any()


def test_attention_by_hand():
    k = np.zeros((3, 64))
    v = np.arange(3 * 64, dtype=np.float64).reshape(3, 64)
    k[1, 0] = np.log(3.0)
    q = np.zeros((2, 64))
    q[:, 0] = 1.0
    lv, sc = np.full(3, 4), np.zeros((2, 3), np.float32)
    out, _ = kv.attention(q, k, v, lv, sc, np.array([1, 2]), 1.0, 0, 0)
    assert np.allclose(out[0], (v[0] + 3 * v[1]) / 4) and np.allclose(out[1], (v[0] + 3 * v[1] + v[2]) / 5)
    out, _ = kv.attention(q, k, v, lv, sc, np.array([1, 2]), 1.0, 1, 0)      # window 1: itself
    assert np.allclose(out[1], v[2])
    out, _ = kv.attention(q, k, v, lv, sc, np.array([1, 2]), 1.0, 1, 1)      # and the first token
    assert np.allclose(out[1], (v[0] + v[2]) / 2)
    out, _ = kv.attention(q, k, v, np.zeros(3), sc, np.array([1, 2]), 1.0, 0, 0)
    assert not out.any()


def _status(fl, fn, *args):
    with pytest.raises(fl.FlError) as e:
        fn(*args)
    return e.value.status


def test_byte_counts(fl):
    assert fl.fl_kv_page_bytes(8, 128) == 8 * kv.record_bytes(128) == 8 * 16896
    assert fl.fl_kv_page_bytes(8, 64) == 8 * 8704
    assert fl.fl_kv_page_bytes(8, 96) == 0 and fl.fl_kv_page_bytes(0, 64) == 0 and fl.fl_kv_page_bytes(257, 64) == 0
    for bad in ((0, 16, 8, 128, 1), (1025, 16, 8, 128, 1), (1, 12, 8, 128, 1), (1, 8 * 33, 8, 128, 1),
                (1, 16, 8, 80, 1), (1, 16, 8, 128, 0), (1, 0, 8, 128, 1)):
        assert fl.fl_attn_workspace_bytes(*bad) == 0, bad


def test_refusals(fl):
    ARG, SHAPE, ALIGN = -1, -2, -4
    s0 = 0

    def cache(pages=16, num=4, heads=2, dim=64):
        return fl.kv_cache(pages, num, heads, dim)

    def batch(table=16, lens=16, start=16, n=2, blocks=3, rows=8, new=4):
        return fl.kv_batch(table, lens, start, n, blocks, rows, new)

    calls = [lambda c, b, p=16, s=128: fl.fl_kv_append(c, b, p, s, 16, 128, s0),
             lambda c, b, p=16, s=128: fl.fl_kv_append(c, b, 16, 128, p, s, s0),
             lambda c, b, p=16, s=128: fl.fl_kv_read(c, b, None, p, s, 16, 128, s0),
             lambda c, b, p=16, s=128: fl.fl_kv_read(c, b, None, 16, 128, p, s, s0),
             lambda c, b, p=16, s=128: fl.fl_attn_paged(c, b, None, p, s, 2, 0.1, 0, 0, 16, 128, 16, 1 << 30, s0),
             lambda c, b, p=16, s=128: fl.fl_attn_paged(c, b, None, 16, 128, 2, 0.1, 0, 0, p, s, 16, 1 << 30, s0)]
    for call in calls:
        for c, want in ((cache(pages=None), ARG), (cache(pages=24), ALIGN), (cache(num=0), SHAPE),
                        (cache(heads=0), SHAPE), (cache(heads=257), SHAPE), (cache(dim=96), SHAPE),
                        (cache(dim=256), SHAPE)):
            assert _status(fl, call, c, batch()) == want
        for b, want in ((batch(table=None), ARG), (batch(lens=None), ARG), (batch(table=18), ALIGN),
                        (batch(lens=17), ALIGN), (batch(start=18), ALIGN), (batch(n=0), SHAPE), (batch(n=1025), SHAPE),
                        (batch(blocks=0), SHAPE), (batch(blocks=1 << 24), SHAPE), (batch(new=0), SHAPE),
                        (batch(new=9), SHAPE), (batch(start=None, n=9, new=1), SHAPE), (batch(rows=0, new=0), SHAPE),
                        (batch(rows=1 << 23, new=(1 << 22) + 1), SHAPE)):
            assert _status(fl, call, cache(), b) == want
        assert _status(fl, call, cache(), batch(), None) == ARG
        assert _status(fl, call, cache(), batch(), 24) == ALIGN
        assert _status(fl, call, cache(), batch(), 16, 120) == SHAPE
        assert _status(fl, call, cache(), batch(), 16, 132) == SHAPE
        assert _status(fl, call, cache(), batch(), 16, -128) == SHAPE

    def attn(heads=2, scale=0.1, window=0, sinks=0, ws=16, ws_bytes=1 << 30, stride=128 * 40):
        return fl.fl_attn_paged(cache(), batch(), None, 16, stride, heads, scale, window, sinks, 16, stride, ws,
                                ws_bytes, s0)

    for kw in (dict(heads=0), dict(heads=3), dict(heads=66), dict(heads=-2)):
        assert _status(fl, lambda kw=kw: attn(**kw)) == SHAPE, kw
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(sinks=-1)):
        assert _status(fl, lambda kw=kw: attn(**kw)) == ARG, kw


@pytest.mark.parametrize("scale", [1.7e35, -1.7e35, 2e38, 3.4e38, -3.4e38])
def test_scale_beyond_the_kernels_range_is_refused(fl, scale):
    """Above 2^117 (1.66e35) the codes' factor times scale log2(e) is no longer finite in fp32."""
    c, b = fl.kv_cache(16, 4, 2, 64), fl.kv_batch(16, 16, 16, 2, 3, 8, 4)
    assert _status(fl, lambda: fl.fl_attn_paged(c, b, None, 16, 128, 2, scale, 0, 0, 16, 128, 16, 1 << 30, 0)) == -1
