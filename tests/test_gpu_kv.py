"""The paged key/value cache and its attention on the GPU against the 64-bit reference, through the C-ABI.

Cache bytes and read-back values are compared bit for bit. An attention output may be off by the
bound that oracle.kv.attention derives: half a bf16 step on the output and on every probability
times its value's scale (2^-8 relative each), and fp32 sums of the scores' and the outputs'
lengths."""
import numpy as np
import pytest

from oracle import kv
from variable_precision_weight_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_precision_weight_b200 import build
    build.build()
    from variable_precision_weight_b200 import fl
    torch.cuda.set_device(0)
    return torch, fl


def dev(torch, a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def f64(bits):
    return synth.bf16_bits_to_f32(np.asarray(bits).view(np.uint16)).astype(np.float64)


class Case:
    """A cache with random content (every slot of every page holds a quantised token), and a batch."""

    def __init__(self, torch, fl, lens, news, kvh, D, seed, spare=2, width=None, rows=None, max_new=None,
                 levels=None, spread=1.0):
        g = np.random.default_rng(seed)
        self.torch, self.fl, self.g, self.kvh, self.D = torch, fl, g, kvh, D
        self.lens, self.news = list(lens), list(news)
        blocks = [-(-n // 64) for n in lens]
        self.num_pages = sum(blocks) + spare
        self.width = width or max(blocks + [1])
        order = g.permutation(self.num_pages)
        self.table = np.full((len(lens), self.width), -7, np.int32)       # entries nobody needs are rubbish
        at = 0
        for i, b in enumerate(blocks):
            self.table[i, :b] = order[at:at + b]
            at += b
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.rows = rows or int(self.start[-1]) or 1
        self.max_new = max_new or max(max(news), 1)
        self.levels = None if levels is None else g.choice(levels, size=self.table.shape).astype(np.uint8)
        rec = kv.record_bytes(D)
        self.pages = g.integers(0, 256, (self.num_pages, kvh, rec), dtype=np.uint8)
        sc = np.abs(g.standard_normal((self.num_pages, kvh, 128))).astype(np.float32) * np.float32(spread / 80) + \
            np.float32(0.004)
        self.pages[:, :, :512] = sc.view(np.uint8).reshape(self.num_pages, kvh, 512)
        self.upload()

    def upload(self):
        t = self.torch
        self.d_pages, self.d_table = dev(t, self.pages), dev(t, self.table)
        self.d_lens, self.d_start = dev(t, np.array(self.lens, np.int32)), dev(t, self.start)
        self.d_levels = None if self.levels is None else dev(t, self.levels)
        self.cache = self.fl.kv_cache(self.d_pages, self.num_pages, self.kvh, self.D)
        self.batch = self.fl.kv_batch(self.d_table, self.d_lens, self.d_start, len(self.lens), self.width, self.rows,
                                      self.max_new)

    def workspace(self, heads):
        n = self.fl.fl_attn_workspace_bytes(len(self.lens), heads, self.kvh, self.D, self.max_new)
        assert n > 0
        return self.torch.zeros(n, dtype=self.torch.uint8, device="cuda"), n

    def q(self, heads, gain=1.0):
        return synth.f32_to_bf16_bits((gain * self.g.standard_normal((self.rows, heads, self.D))).astype(np.float32))

    def attend(self, q, heads, scale, window=0, sinks=0, ws=None, out=None, stream=None):
        t = self.torch
        d_q = dev(t, q)
        d_out = t.full((self.rows, heads, self.D), 77, dtype=t.int16, device="cuda") if out is None else out
        ws, n = ws or self.workspace(heads)
        w = heads * self.D
        self.fl.fl_attn_paged(self.cache, self.batch, self.d_levels, d_q, w, heads, scale, window, sinks, d_out, w, ws,
                              n, stream)
        t.cuda.synchronize()
        assert not ws[:2048].any()                                        # the counters are zero again
        return d_out.cpu().numpy().view(np.uint16)

    def check(self, got, q, heads, scale, window=0, sinks=0, skip=()):
        gr = heads // self.kvh
        worst = 0.0
        for i, (n, new) in enumerate(zip(self.lens, self.news)):
            if i in skip or new == 0:
                continue
            rows = slice(int(self.start[i]), int(self.start[i + 1]))
            pos = np.arange(n - new, n)
            for h in range(self.kvh):
                k, v, lv, sc = kv.gather(self.pages, self.table[i], None if self.levels is None else self.levels[i], n,
                                         self.D, h)
                for x in range(h * gr, (h + 1) * gr):
                    ref, tol = kv.attention(f64(q[rows, x]), k, v, lv, sc, pos, np.float32(scale), window, sinks)
                    err = np.abs(f64(got[rows, x]) - ref)
                    assert np.all(err <= tol), (i, x, float((err / tol).max()))
                    worst = max(worst, float((err / tol).max()))
        return worst

    def untouched(self, got, fill=77):
        """Rows outside every sequence keep what they held."""
        live = np.zeros(self.rows, bool)
        live[:self.start[-1]] = True
        assert np.all(got[~live] == fill)


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,news,kvh", [
    ([1], [1], 1), ([64], [64], 2), ([65], [1], 3), ([64], [1], 1), ([130], [130], 1), ([70], [9], 2),
    ([200, 0, 63, 129, 1], [137, 0, 2, 129, 1], 2), ([300, 300], [299, 1], 1)])
def test_append_bit_exact(env, D, lens, news, kvh):
    torch, fl = env
    c = Case(torch, fl, lens, news, kvh, D, seed=D + sum(lens), rows=sum(news) + 2)
    k, v = (synth.bf16_normal((c.rows, kvh, D), D, sum(lens), x) for x in (1, 2))
    k[0, 0, :] = 0                                                        # an all-zero head
    k[-3:, :, :4] = synth.f32_to_bf16_bits(np.array([127, -63.5, 0.5, 1.5], np.float32))   # ties
    fl.fl_kv_append(c.cache, c.batch, dev(torch, k), kvh * D, dev(torch, v), kvh * D)
    fl.fl_device_status()
    want = c.pages.copy()
    for i, (n, new) in enumerate(zip(lens, news)):
        for x in range(new):
            p, r = n - new + x, c.start[i] + x
            for h in range(kvh):
                (kc, ks), (vc, vs) = kv.quantise(f64(k[r, h])), kv.quantise(f64(v[r, h]))
                kv.write_token(want[c.table[i, p // 64], h], D, p % 64, kc, ks, vc, vs)
    assert np.array_equal(c.d_pages.cpu().numpy(), want)


def test_append_strided_rows_and_non_finite(env):
    """k and v inside one fused projection's rows; a row with an infinity or NaN is stored as scale NaN."""
    torch, fl = env
    kvh, D = 2, 64
    c = Case(torch, fl, [40], [30], kvh, D, seed=3)
    x = synth.bf16_normal((30, 4 * kvh * D + 8), 3, 1)
    x[5, kvh * D + 3] = 0x7F80                                            # k row 5, head 0: infinity
    x[6, 3 * kvh * D + D + 1] = 0xFFC1                                    # v row 6, head 1: NaN
    d = dev(torch, x)
    w = kvh * D
    fl.fl_kv_append(c.cache, c.batch, d[:, w:], x.shape[1], d[:, 3 * w:], x.shape[1])
    fl.fl_device_status()
    got = c.d_pages.cpu().numpy()
    for r in range(30):
        for h in range(kvh):
            rec = got[c.table[0, 0], h]
            sc = rec[:512].view(np.float32).reshape(2, 64)[:, 10 + r]
            ks, vs = (kv.quantise(f64(x[r, m * w + h * D:m * w + (h + 1) * D]))[1] for m in (1, 3))
            assert np.array_equal(sc, [ks, vs], equal_nan=True), (r, h)
            assert np.isnan(sc[0]) == (r == 5 and h == 0) and np.isnan(sc[1]) == (r == 6 and h == 1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,news,levels", [
    ([1], [1], None), ([64, 65, 128], [64, 65, 1], None), ([500], [499], (0, 1, 2, 3, 4, 9)),
    ([77, 0, 300], [3, 0, 211], (2, 4)), ([129], [100], (2,))])
def test_read_bit_exact(env, D, lens, news, levels):
    torch, fl = env
    kvh = 2
    c = Case(torch, fl, lens, news, kvh, D, seed=7 + D, levels=levels, rows=sum(news) + 1)
    ko, vo = (torch.full((c.rows, kvh * D + 16), 55, dtype=torch.int16, device="cuda") for _ in "kv")
    fl.fl_kv_read(c.cache, c.batch, c.d_levels, ko, kvh * D + 16, vo, kvh * D + 16)
    fl.fl_device_status()
    ko, vo = ko.cpu().numpy().view(np.uint16), vo.cpu().numpy().view(np.uint16)
    assert np.all(ko[:, kvh * D:] == 55) and np.all(vo[:, kvh * D:] == 55)
    assert np.all(ko[c.start[-1]:] == 55)
    for i, (n, new) in enumerate(zip(lens, news)):
        for h in range(kvh):
            k, v, _, _ = kv.gather(c.pages, c.table[i], None if levels is None else c.levels[i], n, D, h)
            for got, ref in ((ko, k), (vo, v)):
                want = synth.f32_to_bf16_bits(ref[n - new:].astype(np.float32))
                have = got[c.start[i]:c.start[i + 1], h * D:(h + 1) * D]
                assert np.array_equal(have, want), (i, h)


# ------------------------------------------------------------------ attention

SHAPES = [  # kv heads, group, D
    (1, 1, 64), (2, 2, 128), (2, 4, 64), (1, 3, 128), (1, 7, 64), (1, 8, 128), (1, 32, 64)]


@pytest.mark.parametrize("kvh,group,D", SHAPES)
@pytest.mark.parametrize("lens,news", [
    ([1], [1]), ([64], [1]), ([65], [2]), ([1000], [1]), ([3, 700, 64, 129], [1, 1, 1, 1]), ([40, 0, 333], [8, 0, 5]),
    ([517], [16])])
def test_attend_short_chunks(env, kvh, group, D, lens, news):
    torch, fl = env
    heads = kvh * group
    c = Case(torch, fl, lens, news, kvh, D, seed=group + sum(lens), rows=sum(news) + 3)
    q = c.q(heads)
    got = c.attend(q, heads, D ** -0.5)
    fl.fl_device_status()
    c.check(got, q, heads, D ** -0.5)
    c.untouched(got)


@pytest.mark.parametrize("kvh,group,D", [(2, 2, 128), (2, 4, 64), (1, 3, 64), (1, 1, 128)])
@pytest.mark.parametrize("lens,news", [([150], [150]), ([300], [129]), ([64], [64]), ([257, 1, 90, 40], [200, 1, 33, 40]),
                                       ([1100], [70]), ([513], [65])])
@pytest.mark.parametrize("levels", [None, (2, 4)])
def test_attend_prompt_chunks(env, kvh, group, D, lens, news, levels):
    torch, fl = env
    heads = kvh * group
    c = Case(torch, fl, lens, news, kvh, D, seed=group + sum(news), rows=sum(news) + 5, levels=levels)
    q = c.q(heads)
    got = c.attend(q, heads, D ** -0.5)
    fl.fl_device_status()
    c.check(got, q, heads, D ** -0.5)
    c.untouched(got)


@pytest.mark.parametrize("kvh,group,D", [(1, 1, 64), (2, 2, 128), (1, 8, 64), (1, 32, 128)])
@pytest.mark.parametrize("rows", [31, 32, 33, 127, 128, 129, 255, 256, 257, 384, 385, 511, 512, 513])
def test_attend_row_counts(env, kvh, group, D, rows):
    """Query rows per key/value head around the kernels' limits and the tiles' sizes, alone and among others."""
    torch, fl = env
    heads, new = kvh * group, max(1, rows // group)
    for lens, news in (([new + 700], [new]), ([new, 90, new + 130], [new, 1, max(1, new - 1)])):
        c = Case(torch, fl, lens, news, kvh, D, seed=rows + group, rows=sum(news) + 2, levels=(2, 4, 4, 0))
        q = c.q(heads)
        got = c.attend(q, heads, D ** -0.5)
        fl.fl_device_status()
        c.check(got, q, heads, D ** -0.5)
        c.untouched(got)


@pytest.mark.parametrize("kvh,group,D,n,new", [(1, 1, 64, 9000, 40), (1, 1, 64, 9000, 200), (2, 2, 128, 6000, 130),
                                                 (1, 4, 64, 5000, 65)])
def test_attend_chunk_cut_into_many_pieces(env, kvh, group, D, n, new):
    """One tile of rows whose keys are spread over most of the GPU, and joined."""
    torch, fl = env
    heads = kvh * group
    c = Case(torch, fl, [n], [new], kvh, D, seed=n, levels=(2, 4))
    q = c.q(heads, 2.0)
    for window, sinks in ((0, 0), (3000, 70)):
        got = c.attend(q, heads, 0.1, window, sinks)
        fl.fl_device_status()
        c.check(got, q, heads, 0.1, window, sinks)
        assert np.array_equal(c.attend(q, heads, 0.1, window, sinks), got)


@pytest.mark.parametrize("lens,news", [
    ([6000, 300, 300, 300], [200, 290, 290, 290]),                  # one long tile per head among short ones
    ([400 + 97 * i for i in range(20)], [63 + i for i in range(20)]),   # more tiles than the GPU has SMs
    ([1500, 64, 700], [600, 64, 33])])
def test_attend_chunks_in_equal_ranges(env, lens, news):
    """Tiles of unequal lengths, cut anywhere by equal ranges of steps."""
    torch, fl = env
    c = Case(torch, fl, lens, news, 8, 64, seed=sum(news), rows=sum(news) + 4, levels=(2, 4))
    q = c.q(8)
    got = c.attend(q, 8, 0.125)
    fl.fl_device_status()
    c.check(got, q, 8, 0.125)
    c.untouched(got)
    assert np.array_equal(c.attend(q, 8, 0.125), got)


def test_chunk_sized_call_with_fewer_tokens(env):
    """max_new sizes the launch only: one token, or none, in calls sized for a chunk."""
    torch, fl = env
    for lens, news in (([300], [1]), ([1], [1]), ([0], [0]), ([300, 77], [1, 5]), ([300, 77], [0, 0])):
        c = Case(torch, fl, lens, news, 2, 64, seed=3, rows=300, max_new=300)
        q = c.q(4)
        got = c.attend(q, 4, 0.1)
        fl.fl_device_status()
        c.check(got, q, 4, 0.1)
        c.untouched(got)


def test_two_streams_with_their_own_workspaces(env):
    torch, fl = env
    cs = [Case(torch, fl, [2500, 800], [300, 1], 2, 128, seed=21), Case(torch, fl, [3000], [2], 2, 128, seed=22)]
    qs = [c.q(4) for c in cs]
    want = [c.attend(q, 4, 0.1) for c, q in zip(cs, qs)]
    streams = [torch.cuda.Stream() for _ in cs]
    spaces = [c.workspace(4) for c in cs]
    d_q = [dev(torch, q) for q in qs]
    outs = [[torch.zeros((c.rows, 4, 128), dtype=torch.int16, device="cuda") for _ in range(4)] for c in cs]
    torch.cuda.synchronize()
    for r in range(4):
        for c, q, s, (ws, n), o in zip(cs, d_q, streams, spaces, outs):
            fl.fl_attn_paged(c.cache, c.batch, None, q, 512, 4, 0.1, 0, 0, o[r], 512, ws, n, s)
    torch.cuda.synchronize()
    fl.fl_device_status()
    for w, o in zip(want, outs):
        for x in o:
            assert np.array_equal(x.cpu().numpy().view(np.uint16), w)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 0), (64, 4), (65, 64), (200, 65), (100, 5000), (5000, 4),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("new", [1, 7, 150])
def test_attend_window_and_sinks(env, window, sinks, new):
    torch, fl = env
    kvh, heads, D = 2, 4, 64
    c = Case(torch, fl, [900, 151, 333], [new, new, 1], kvh, D, seed=window % 1000 + new, levels=(2, 4, 4))
    q = c.q(heads)
    got = c.attend(q, heads, 0.2, window, sinks)
    fl.fl_device_status()
    c.check(got, q, heads, 0.2, window, sinks)


@pytest.mark.parametrize("levels", [(0,), (0, 2, 4), (0, 0, 0, 4), (1, 3), (2,), (0, 255)])
@pytest.mark.parametrize("new", [1, 10, 140])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_levels_and_empty_rows(env, levels, new, D):
    """Blocks at every level; queries whose every block is ZERO give exact zeros."""
    torch, fl = env
    kvh, heads = 2, 4
    c = Case(torch, fl, [700, 140, 64 * 3], [new, new, new], kvh, D, seed=len(levels) + new, levels=levels)
    q = c.q(heads)
    got = c.attend(q, heads, D ** -0.5, 30 if new == 10 else 0, 0)
    fl.fl_device_status()
    c.check(got, q, heads, D ** -0.5, 30 if new == 10 else 0, 0)
    if levels == (0,):
        assert not got.any()


@pytest.mark.parametrize("new", [1, 5, 130])
def test_unseen_keys_have_no_influence(env, new):
    """Slots behind the last token, keys after a query, and ZERO blocks hold NaN and infinite scales."""
    torch, fl = env
    kvh, heads, D = 2, 4, 128
    c = Case(torch, fl, [330], [new], kvh, D, seed=11, levels=(4,))
    c.levels[0, 1] = 0
    c.upload()
    q = c.q(heads)
    clean = c.attend(q, heads, 0.09)
    c.check(clean, q, heads, 0.09)
    sc = c.pages[:, :, :512].view(np.float32).reshape(c.num_pages, kvh, 2, 64)
    poison = np.where(np.arange(64) % 2, np.nan, np.inf).astype(np.float32)
    sc[c.table[0, 1]] = poison                                    # the ZERO block
    sc[c.table[0, 330 // 64], :, :, 330 % 64:] = poison[330 % 64:]  # behind the last token
    unused = sorted(set(range(c.num_pages)) - set(c.table[0].tolist()))
    sc[unused] = np.nan
    c.upload()
    assert np.array_equal(c.attend(q, heads, 0.09), clean)
    # the newest token poisoned: only its own query sees it
    sc[c.table[0, 329 // 64], :, :, 329 % 64] = np.nan
    c.upload()
    got = c.attend(q, heads, 0.09)
    assert np.array_equal(got[:new - 1], clean[:new - 1]) and np.isnan(f64(got[new - 1])).all()


def test_nan_query_stays_in_its_row(env):
    torch, fl = env
    for new in (9, 140):
        c = Case(torch, fl, [200], [new], 2, 64, seed=new)
        q = c.q(4)
        clean = c.attend(q, 4, 0.1)
        q2 = q.copy()
        q2[3, 2, 5] = 0x7FC0
        got = c.attend(q2, 4, 0.1)
        hit = np.zeros(got.shape[:2], bool)
        hit[3, 2] = True
        assert np.isnan(f64(got[hit])).all() and np.array_equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("scale,gain", [(0.0, 1.0), (-0.3, 1.0), (30.0, 3.0), (1e-30, 1.0)])
@pytest.mark.parametrize("new", [3, 140])
def test_scales(env, scale, gain, new):
    """Flat, negative and very sharp softmax (one key takes all)."""
    torch, fl = env
    c = Case(torch, fl, [500], [new], 1, 64, seed=5, levels=(2, 4))
    q = c.q(2, gain)
    c.check(c.attend(q, 2, scale), q, 2, scale)


def test_new_start_omitted(env):
    """One new token per sequence without new_start; an empty sequence's row keeps what it held."""
    torch, fl = env
    lens = [5, 0, 300, 64]
    c = Case(torch, fl, lens, [1, 0, 1, 1], 2, 64, seed=2, rows=6, max_new=1)
    c.batch = fl.kv_batch(c.d_table, c.d_lens, None, 4, c.width, c.rows, 1)
    q = c.q(4)
    got = c.attend(q, 4, 0.1)
    fl.fl_device_status()
    full = q.copy()
    for i in (0, 2, 3):
        for h in range(2):
            k, v, lv, sc = kv.gather(c.pages, c.table[i], None, lens[i], 64, h)
            for x in (2 * h, 2 * h + 1):
                ref, tol = kv.attention(f64(full[i:i + 1, x]), k, v, lv, sc, np.array([lens[i] - 1]), np.float32(0.1), 0, 0)
                assert np.all(np.abs(f64(got[i, x]) - ref[0]) <= tol[0])
    assert np.all(got[[1, 4, 5]] == 77)
    k = synth.bf16_normal((6, 2, 64), 2, 9)
    fl.fl_kv_append(c.cache, c.batch, dev(torch, k), 128, dev(torch, k), 128)
    ko, vo = (torch.full((6, 2, 64), 55, dtype=torch.int16, device="cuda") for _ in "kv")
    fl.fl_kv_read(c.cache, c.batch, None, ko, 128, vo, 128)
    fl.fl_device_status()
    ko = ko.cpu().numpy().view(np.uint16)
    assert np.all(ko[[1, 4, 5]] == 55) and torch.equal(vo.cpu(), torch.from_numpy(ko.view(np.int16)))
    code, sc = kv.quantise(f64(k))
    want = synth.f32_to_bf16_bits(sc[..., None] * code.astype(np.float32))
    assert np.array_equal(ko[[0, 2, 3]], want[[0, 2, 3]])


def test_strides_and_output_over_query(env):
    """Queries inside wider rows; the output may be the query buffer."""
    torch, fl = env
    for new in (4, 150):
        heads, D = 4, 64
        c = Case(torch, fl, [260], [new], 2, D, seed=new)
        wide = synth.bf16_normal((new, heads * D + 24), 9, new)
        q = wide[:, 8:8 + heads * D].reshape(new, heads, D)
        d = dev(torch, wide)
        ws, n = c.workspace(heads)
        stride = heads * D + 24
        fl.fl_attn_paged(c.cache, c.batch, None, d[:, 8:], stride, heads, 0.1, 0, 0, d[:, 8:], stride, ws, n)
        fl.fl_device_status()
        out = d.cpu().numpy().view(np.uint16)
        assert np.array_equal(out[:, :8], wide[:, :8]) and np.array_equal(out[:, 8 + heads * D:], wide[:, 8 + heads * D:])
        c.check(out[:, 8:8 + heads * D].reshape(new, heads, D), q, heads, 0.1)


def test_shared_prefix_pages(env):
    """Two sequences whose first blocks are the same pages."""
    torch, fl = env
    c = Case(torch, fl, [400, 380], [3, 3], 2, 64, seed=8)
    c.table[1, :4] = c.table[0, :4]
    c.upload()
    q = c.q(4)
    c.check(c.attend(q, 4, 0.125), q, 4, 0.125)


def test_equal_bits_and_reused_workspace(env):
    """Calls of different shapes in a row on one workspace; the same call gives the same bits."""
    torch, fl = env
    cs = [Case(torch, fl, [3000, 70], [2, 2], 2, 128, seed=1), Case(torch, fl, [4100], [1], 2, 128, seed=2),
          Case(torch, fl, [700], [300], 2, 128, seed=3)]
    qs = [c.q(4) for c in cs]
    n = max(c.workspace(4)[1] for c in cs)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    first = [c.attend(q, 4, 0.1, ws=(ws, n)) for c, q in zip(cs, qs)]
    for c, q, f in zip(cs, qs, first):
        c.check(f, q, 4, 0.1)
    for _ in range(3):
        for c, q, f in zip(cs, qs, first):
            assert np.array_equal(c.attend(q, 4, 0.1, ws=(ws, n)), f)


def test_bad_device_data_is_reported(env):
    """Page indices, lengths and row ranges that the host cannot see: the block or sequence is left out."""
    torch, fl = env
    c = Case(torch, fl, [200, 100, 130], [2, 2, 2], 2, 64, seed=4)
    q = c.q(4)
    c.table[0, 1] = c.num_pages                                   # one past the last page
    c.upload()
    got = c.attend(q, 4, 0.1)
    with pytest.raises(fl.FlError) as e:
        fl.fl_device_status()
    assert e.value.status == -1 and "page" in str(e.value)
    fl.fl_device_status()
    c.check(got, q, 4, 0.1)                                       # the reference reads that block as ZERO
    for call in ("append", "read"):
        x = torch.zeros((6, 2, 64), dtype=torch.int16, device="cuda")
        before = c.d_pages.clone()
        c.d_lens.copy_(torch.tensor([128, 100, 130], dtype=torch.int32))   # its new tokens lie in that block
        if call == "append":
            fl.fl_kv_append(c.cache, c.batch, x, 128, x, 128)
        else:
            fl.fl_kv_read(c.cache, c.batch, None, x, 128, x.clone(), 128)
        with pytest.raises(fl.FlError):
            fl.fl_device_status()
        if call == "read":
            assert torch.equal(before, c.d_pages)
    c = Case(torch, fl, [200, 100, 130], [2, 2, 2], 2, 64, seed=4)
    for lens, start in (([-1, 100, 130], [0, 2, 4, 6]), ([64 * c.width + 1, 100, 130], [0, 2, 4, 6]),
                        ([1, 100, 130], [0, 2, 4, 6]), ([2 ** 31 - 1, 100, 130], [0, 2, 4, 6]),
                        ([200, 100, 130], [0, 0, 4, 6]), ([200, 100, 130], [-2, 2, 4, 6]),
                        ([200, 100, 130], [0, 2, 4, 7]), ([200, 100, 130], [5, 2, 4, 6])):
        c.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        bad = [i for i in range(3) if not (0 <= lens[i] <= 64 * c.width and 0 <= start[i] <= start[i + 1] <= 6 and
                                           start[i + 1] - start[i] <= min(2, lens[i]))]
        got = c.attend(q, 4, 0.1)
        with pytest.raises(fl.FlError) as e:
            fl.fl_device_status()
        assert e.value.status == -1 and "sequence" in str(e.value), (lens, start)
        keep = (c.start, c.lens)
        ok = [i for i in range(3) if i not in bad]
        assert ok
        for i in ok:
            c.lens, c.start = lens, np.array(start, np.int32)
            c.check(got, q, 4, 0.1, skip=[x for x in range(3) if x != i or start[i + 1] - start[i] != 2])
        c.start, c.lens = keep


def test_captured_calls_follow_device_lengths(env):
    """Append, read and attention captured once; replayed after lens, rows and table change."""
    torch, fl = env
    kvh, heads, D = 2, 4, 64
    c = Case(torch, fl, [300, 200, 100], [2, 60, 1], kvh, D, seed=6, rows=80, max_new=64, width=6)
    k, v = (dev(torch, synth.bf16_normal((80, kvh, D), 6, x)) for x in (1, 2))
    q = c.q(heads)
    d_q, d_out = dev(torch, q), torch.full((80, heads, D), 77, dtype=torch.int16, device="cuda")
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    ws, n = c.workspace(heads)
    w = heads * D

    def calls(s=None):
        fl.fl_kv_append(c.cache, c.batch, k, kvh * D, v, kvh * D, s)
        fl.fl_kv_read(c.cache, c.batch, None, ko, kvh * D, vo, kvh * D, s)
        fl.fl_attn_paged(c.cache, c.batch, None, d_q, w, heads, 0.1, 0, 0, d_out, w, ws, n, s)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        calls()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            calls()
    for lens, news in (([300, 200, 100], [2, 60, 1]), ([310, 70, 384], [10, 64, 0]), ([0, 384, 1], [0, 1, 1])):
        c.lens, c.news = lens, news
        c.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        c.table = np.random.default_rng(sum(lens)).permutation(c.num_pages * 2)[:18].reshape(3, 6).astype(np.int32)
        used = [(i, b) for i in range(3) for b in range(-(-lens[i] // 64))]
        for x, (i, b) in enumerate(used):
            c.table[i, b] = x % c.num_pages if len(used) <= c.num_pages else x
        if len(used) > c.num_pages:
            pytest.fail("the test's cache is too small")
        c.d_table.copy_(torch.from_numpy(c.table))
        c.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.d_start.copy_(torch.from_numpy(c.start))
        d_out.fill_(77)
        graph.replay()
        fl.fl_device_status()
        c.pages = c.d_pages.cpu().numpy()
        got = d_out.cpu().numpy().view(np.uint16)
        c.check(got, q, heads, 0.1)
        c.untouched(got)
    del graph


def test_run_together_a_speculation_window(env):
    """A prompt, then draft steps that read the cache at 4 bits and write their own keys, and one
    verification call over the window at 8 bits, all on one cache, each against the reference."""
    torch, fl = env
    kvh, heads, D, prompt, K = 2, 4, 64, 137, 5
    width = 4
    c = Case(torch, fl, [prompt + K], [prompt], kvh, D, seed=12, width=width, rows=prompt, max_new=prompt)
    g = np.random.default_rng(99)
    w, kw = heads * D, kvh * D
    four = torch.full((1, width), 2, dtype=torch.uint8, device="cuda")
    allk, allv = (synth.bf16_normal((prompt + K, kvh, D), 12, x) for x in (1, 2))
    allq = synth.bf16_normal((prompt + K, heads, D), 12, 3)
    d_k, d_v, d_q = dev(torch, allk), dev(torch, allv), dev(torch, allq)
    out = torch.zeros((prompt + K, heads, D), dtype=torch.int16, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    nbytes = fl.fl_attn_workspace_bytes(1, heads, kvh, D, prompt)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")

    def step(first, n, levels, append):
        lens.fill_(first + n)
        start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        b = fl.kv_batch(c.d_table, lens, start, 1, width, n, n)
        if append:
            fl.fl_kv_append(c.cache, b, d_k[first:], kw, d_v[first:], kw)
        fl.fl_attn_paged(c.cache, b, levels, d_q[first:], w, heads, 0.125, 0, 0, out[first:], w, ws, nbytes)
        torch.cuda.synchronize()
        return out[first:first + n].cpu().numpy().view(np.uint16).copy()

    got = {"prompt": step(0, prompt, None, True)}
    for t in range(K):
        got[t] = step(prompt + t, 1, four, True)
    got["verify"] = step(prompt, K, None, False)
    fl.fl_device_status()
    pages = c.d_pages.cpu().numpy()
    for name, first, n, level in [("prompt", 0, prompt, 4), ("verify", prompt, K, 4)] + [(t, prompt + t, 1, 2) for t in range(K)]:
        for h in range(kvh):
            k, v, lv, sc = kv.gather(pages, c.table[0], [level] * width, first + n, D, h)
            for x in (2 * h, 2 * h + 1):
                ref, tol = kv.attention(f64(allq[first:first + n, x]), k, v, lv, sc, np.arange(first, first + n),
                                        np.float32(0.125), 0, 0)
                assert np.all(np.abs(f64(got[name][:, x]) - ref) <= tol), (name, x)
    code, s = kv.quantise(f64(allk))
    k, _, _, _ = kv.gather(pages, c.table[0], None, prompt + K, D, 1)
    assert np.array_equal(k, s[:, 1, None].astype(np.float64) * code[:, 1])


def test_many_sequences(env):
    """1024 sequences, most of them empty or short; and lengths that leave most CTAs idle."""
    torch, fl = env
    g = np.random.default_rng(1)
    lens = [int(x) for x in np.where(g.random(1024) < 0.7, 0, g.integers(1, 90, 1024))]
    news = [min(1, n) for n in lens]
    c = Case(torch, fl, lens, news, 1, 64, seed=77)
    q = c.q(2)
    c.check(c.attend(q, 2, 0.125), q, 2, 0.125)
    fl.fl_device_status()


def test_pages_beyond_32_bit_offsets(env):
    """A cache of more than 2^32 bytes: tokens in its last pages are written, read and attended to."""
    torch, fl = env
    kvh, D = 8, 128
    per = fl.fl_kv_page_bytes(kvh, D)
    num = (1 << 32) // per + 40
    pages = torch.empty(num * per, dtype=torch.uint8, device="cuda")
    assert num * per > 1 << 32
    table = torch.tensor([[num - 1, num - 17, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    cache, b = fl.kv_cache(pages, num, kvh, D), fl.kv_batch(table, lens, start, 1, 3, 150, 150)
    k, v = synth.bf16_normal((150, kvh, D), 4, 1), synth.bf16_normal((150, kvh, D), 4, 2)
    q = synth.bf16_normal((150, 16, D), 4, 3)
    fl.fl_kv_append(cache, b, dev(torch, k), kvh * D, dev(torch, v), kvh * D)
    ko, vo = torch.zeros((150, kvh, D), dtype=torch.int16, device="cuda"), torch.zeros((150, kvh, D), dtype=torch.int16, device="cuda")
    fl.fl_kv_read(cache, b, None, ko, kvh * D, vo, kvh * D)
    out = torch.zeros((150, 16, D), dtype=torch.int16, device="cuda")
    n = fl.fl_attn_workspace_bytes(1, 16, kvh, D, 150)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    fl.fl_attn_paged(cache, b, None, dev(torch, q), 16 * D, 16, D ** -0.5, 0, 0, out, 16 * D, ws, n)
    fl.fl_device_status()
    (kc, ks), (vc, vs) = kv.quantise(f64(k)), kv.quantise(f64(v))
    assert np.array_equal(ko.cpu().numpy().view(np.uint16), synth.f32_to_bf16_bits(ks[..., None] * kc.astype(np.float32)))
    assert np.array_equal(vo.cpu().numpy().view(np.uint16), synth.f32_to_bf16_bits(vs[..., None] * vc.astype(np.float32)))
    for h in (0, 7):
        kk, vv = ks[:, h, None].astype(np.float64) * kc[:, h], vs[:, h, None].astype(np.float64) * vc[:, h]
        sc = np.stack([ks[:, h], vs[:, h]])
        for x in (2 * h, 2 * h + 1):
            ref, tol = kv.attention(f64(q[:, x]), kk, vv, np.full(150, 4), sc, np.arange(150), np.float32(D ** -0.5), 0, 0)
            assert np.all(np.abs(f64(out[:, x].cpu().numpy()) - ref) <= tol)


# ------------------------------------------------------------------ the calls at their edges

@pytest.mark.parametrize("D", [64, 128])
def test_append_over_all_magnitudes(env, D):
    """Rows from the smallest subnormal to the largest finite bf16: the formula's codes and scales, and
    the values read back at eight and at four bits."""
    torch, fl = env
    kvh, top = 2, 0x7F7F
    n = 262                                                               # maxima of 2^-134 .. 2^127
    c = Case(torch, fl, [n], [n], kvh, D, seed=D, levels=(2, 4))
    g = np.random.default_rng(D)
    with np.errstate(over="ignore"):
        x = (g.uniform(-1, 1, (2, n, kvh, D)) * 2.0 ** np.arange(-134, 128)[:, None, None]).astype(np.float32)
    bits = synth.f32_to_bf16_bits(x)
    bits = np.where((bits & 0x7FFF) > top, (bits & 0x8000) | top, bits).astype(np.uint16)
    bits[:, -1, 0, :4] = [top, top | 0x8000, 0x7C00, 0x0001]              # the largest, both signs, and the smallest
    any_ = g.integers(0, 1 << 16, (2, n, D)).astype(np.uint16)            # any finite pattern
    bits[:, ::3, 1] = np.where((any_ & 0x7F80) == 0x7F80, 0x4000, any_)[:, ::3]
    k, v = bits
    fl.fl_kv_append(c.cache, c.batch, dev(torch, k), kvh * D, dev(torch, v), kvh * D)
    ko, vo = (torch.zeros((n, kvh, D), dtype=torch.int16, device="cuda") for _ in "kv")
    fl.fl_kv_read(c.cache, c.batch, c.d_levels, ko, kvh * D, vo, kvh * D)
    fl.fl_device_status()
    want = c.pages.copy()
    for p in range(n):
        for h in range(kvh):
            (kc, ks), (vc, vs) = kv.quantise(f64(k[p, h])), kv.quantise(f64(v[p, h]))
            kv.write_token(want[c.table[0, p // 64], h], D, p % 64, kc, ks, vc, vs)
    assert np.array_equal(c.d_pages.cpu().numpy(), want)
    for h in range(kvh):
        kk, vv, _, _ = kv.gather(want, c.table[0], c.levels[0], n, D, h)
        for got, ref in ((ko, kk), (vo, vv)):
            assert np.array_equal(got[:, h].cpu().numpy().view(np.uint16), synth.f32_to_bf16_bits(ref.astype(np.float32)))


def needed_blocks(n, new, width, window, sinks):
    """Blocks that hold a key some new token sees."""
    key, pos = np.arange(64 * width)[:, None], np.arange(n - new, n)[None, :]
    see = key <= pos
    if window:
        see &= (pos - key < window) | (key < sinks)
    return see.any(axis=1).reshape(width, 64).any(axis=1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,news", [([1500], [300]), ([1500, 900, 700], [300, 1, 5]), ([1500, 200], [1, 3])])
@pytest.mark.parametrize("window,sinks", [(100, 0), (65, 1), (192, 64), (300, 70), (1000, 130), (64, 200), (1, 0)])
def test_pages_outside_the_window_may_be_gone(env, D, lens, news, window, sinks):
    """Blocks that no new token sees have no page any more: nothing is reported, nothing changes."""
    torch, fl = env
    c = Case(torch, fl, lens, news, 2, D, seed=window + sinks)
    for i, (n, new) in enumerate(zip(lens, news)):
        c.table[i, ~needed_blocks(n, new, c.width, window, sinks)] = (-1, c.num_pages)[i % 2]
    c.upload()
    q = c.q(8)
    got = c.attend(q, 8, D ** -0.5, window, sinks)
    fl.fl_device_status()
    c.check(got, q, 8, D ** -0.5, window, sinks)


@pytest.mark.parametrize("new", [1, 10, 300])
@pytest.mark.parametrize("lens", [[700], [700, 500]])
def test_zero_blocks_need_no_page(env, lens, new):
    """A block at level ZERO is not read, so its table entry may be anything."""
    torch, fl = env
    kvh, D = 2, 64
    c = Case(torch, fl, lens, [new] * len(lens), kvh, D, seed=new, levels=(0, 2, 4))
    c.levels[:, -1] = c.levels[:, 0] = 0
    c.levels[:, 1] = 4
    c.table[c.levels == 0] = -1
    c.upload()
    q = c.q(4)
    got = c.attend(q, 4, 0.125)
    fl.fl_device_status()
    c.check(got, q, 4, 0.125)
    ko, vo = (torch.full((c.rows, kvh * D), 55, dtype=torch.int16, device="cuda") for _ in "kv")
    fl.fl_kv_read(c.cache, c.batch, c.d_levels, ko, kvh * D, vo, kvh * D)
    fl.fl_device_status()
    for i, n in enumerate(lens):
        for h in range(kvh):
            k, v, _, _ = kv.gather(c.pages, c.table[i], c.levels[i], n, D, h)
            for got, ref in ((ko, k), (vo, v)):
                have = got[c.start[i]:c.start[i + 1], h * D:(h + 1) * D].cpu().numpy().view(np.uint16)
                assert np.array_equal(have, synth.f32_to_bf16_bits(ref[n - new:].astype(np.float32)))


def test_every_pending_error_is_named(env):
    """A wait that ran out is not lost behind bad arguments, nor one kernel's report behind another's."""
    torch, fl = env
    fl.fl_device_status()

    def pending(*calls):
        for call in calls:
            call()
        with pytest.raises(fl.FlError) as e:
            fl.fl_device_status()
        fl.fl_device_status()                                             # every word was cleared
        return e.value.status, str(e.value)

    def case(news, page=False, seq=False):
        c = Case(torch, fl, [700, 400], news, 2, 64, seed=6)
        if page:
            c.table[0, 0] = c.num_pages
        if seq:
            c.lens[1] = -1
        c.upload()
        return c

    def attend(c):
        ws, n = c.workspace(4)
        q = torch.zeros((c.rows, 256), dtype=torch.int16, device="cuda")
        fl.fl_attn_paged(c.cache, c.batch, None, q, 256, 4, 0.1, 0, 0, q, 256, ws, n)
        return ws

    def read(c):
        x = torch.zeros((c.rows, 128), dtype=torch.int16, device="cuda")
        fl.fl_kv_read(c.cache, c.batch, None, x, 128, torch.zeros_like(x), 128)

    for news in ([2, 2], [300, 300]):
        status, text = pending(fl.fl_selftest_wait_timeout, lambda: attend(case(news, page=True)))
        assert status == -7 and "self-test" in text and "attention: a page" in text, text
        status, text = pending(lambda: attend(case(news, page=True, seq=True)))
        assert status == -1 and "attention: a page" in text and "attention: a sequence" in text, text
        status, text = pending(lambda: attend(case(news, page=True)), lambda: read(case([2, 2], seq=True)))
        assert status == -1 and "attention: a page" in text and "cache append or read: a sequence" in text, text
    status, text = pending(lambda: attend(case([2, 2], page=True)), lambda: attend(case([300, 300], seq=True)))
    assert status == -1 and "attention: a page" in text and "attention: a sequence" in text, text


@pytest.mark.parametrize("new", [2, 300])
@pytest.mark.parametrize("exp", [-117, 117])
def test_largest_scales(env, new, exp):
    """scale at the largest that is taken, over keys as small; and the reverse."""
    torch, fl = env
    c = Case(torch, fl, [500], [new], 2, 64, seed=5, levels=(2, 4))
    sc = c.pages[:, :, :512].view(np.float32).reshape(c.num_pages, 2, 2, 64)
    sc[:, :, 0] *= np.float32(2.0) ** -exp
    c.upload()
    q = c.q(4, 0.1)
    got = c.attend(q, 4, 2.0 ** exp)
    fl.fl_device_status()
    c.check(got, q, 4, 2.0 ** exp)


def attend_counted(c, q, heads, scale, *rest):
    """c.attend, and the counters of both kernels are zero behind it."""
    ws, n = c.workspace(heads)
    got = c.attend(q, heads, scale, *rest, ws=(ws, n))
    assert not ws[:4096].any()
    return got


def test_half_tiles_before_whole_tiles(env):
    """Equal ranges in which tiles of at most 128 rows (one of the kernel's two halves has nothing to do for many
    steps) are followed by tiles of 129 to 256."""
    torch, fl = env
    kvh, D = 16, 64
    lens, news = [1300, 260] * 5, [100, 200] * 5
    c = Case(torch, fl, lens, news, kvh, D, seed=31, levels=(2, 4))
    q = c.q(kvh)
    got = attend_counted(c, q, kvh, 0.125)
    fl.fl_device_status()
    c.check(got, q, kvh, 0.125, skip=range(3, 9))
    for _ in range(3):
        assert np.array_equal(attend_counted(c, q, kvh, 0.125), got)


@pytest.mark.parametrize("kvh,group,D,lens,news", [
    (1, 1, 64, [9000], [300]), (2, 2, 128, [6000], [140]), (2, 4, 64, [5000, 70], [100, 1]), (8, 1, 64, [3000, 900], [290, 257]),
    (8, 1, 64, [400 + 97 * i for i in range(20)], [63 + i for i in range(20)])])
def test_joined_chunks_leave_the_counters_at_zero(env, kvh, group, D, lens, news):
    """Tiles cut into parts, and cut anywhere by equal ranges, on the chunk kernel (more than 256 rows in some sequence)."""
    torch, fl = env
    heads = kvh * group
    c = Case(torch, fl, lens, news, kvh, D, seed=sum(lens), levels=(2, 4))
    q = c.q(heads)
    for window, sinks in ((0, 0), (700, 70)):
        got = attend_counted(c, q, heads, 0.1, window, sinks)
        fl.fl_device_status()
        c.check(got, q, heads, 0.1, window, sinks, skip=range(2, len(lens) - 1))
        assert np.array_equal(attend_counted(c, q, heads, 0.1, window, sinks), got)


@pytest.mark.parametrize("n_seqs", [1, 3])
def test_captured_chunks_follow_device_lengths(env, n_seqs):
    """The chunk kernel (alone, and behind the other) captured once; replayed after lens, rows and table change."""
    torch, fl = env
    kvh, heads, D, rows, width = 2, 4, 64, 640, 12
    lens, news = [700, 300, 100][:n_seqs], [300, 290, 1][:n_seqs]
    c = Case(torch, fl, lens, news, kvh, D, seed=6, rows=rows, max_new=300, width=width, spare=30)
    q = c.q(heads)
    w = heads * D
    d_q, d_out = dev(torch, q), torch.full((rows, heads, D), 77, dtype=torch.int16, device="cuda")
    ws, n = c.workspace(heads)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        fl.fl_attn_paged(c.cache, c.batch, None, d_q, w, heads, 0.1, 0, 0, d_out, w, ws, n, st)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            fl.fl_attn_paged(c.cache, c.batch, None, d_q, w, heads, 0.1, 0, 0, d_out, w, ws, n, st)
    for r, (lens, news) in enumerate((([700, 300, 100], [300, 290, 1]), ([300, 768, 384], [300, 40, 300]), ([1, 0, 130], [1, 0, 0]),
                                      ([650, 129, 64], [33, 129, 64]), ([0, 0, 0], [0, 0, 0]), ([768, 5, 600], [257, 5, 70]))):
        c.lens, c.news = lens[:n_seqs], news[:n_seqs]
        c.start = np.concatenate([[0], np.cumsum(c.news)]).astype(np.int32)
        order = np.random.default_rng(r).permutation(c.num_pages)
        c.table[:] = -5
        at = 0
        for i, x in enumerate(c.lens):
            c.table[i, :-(-x // 64)] = order[at:at + -(-x // 64)]
            at += -(-x // 64)
        c.d_table.copy_(torch.from_numpy(c.table))
        c.d_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        c.d_start.copy_(torch.from_numpy(c.start))
        d_out.fill_(77)
        graph.replay()
        fl.fl_device_status()
        assert not ws[:4096].any()
        got = d_out.cpu().numpy().view(np.uint16)
        c.check(got, q, heads, 0.1)
        c.untouched(got)
    del graph


def test_bad_device_data_of_chunks_is_reported(env):
    """What test_bad_device_data_is_reported asks, of sequences that the chunk kernel takes."""
    torch, fl = env
    good = ([700, 400, 450], [0, 300, 305, 600])
    c = Case(torch, fl, good[0], [300, 5, 295], 2, 64, seed=14)
    q = c.q(4)
    c.check(attend_counted(c, q, 4, 0.1), q, 4, 0.1)
    fl.fl_device_status()
    for seq, block, page in ((0, 3, c.num_pages), (2, 0, -1), (2, 7, 2 ** 31 - 1)):
        keep = int(c.table[seq, block])
        c.table[seq, block] = page
        c.upload()
        got = attend_counted(c, q, 4, 0.1)
        with pytest.raises(fl.FlError) as e:
            fl.fl_device_status()
        assert e.value.status == -1 and "page" in str(e.value)
        c.check(got, q, 4, 0.1)                                   # the reference reads that block as ZERO
        c.table[seq, block] = keep
    c.upload()
    for lens, start in (([-1, 400, 450], good[1]), ([64 * c.width + 1, 400, 450], good[1]), ([299, 400, 450], good[1]),
                        ([700, 400, 2 ** 31 - 1], good[1]), (good[0], [0, 300, 305, 601]), (good[0], [0, 300, 299, 594]),
                        ([700, 400, 294], good[1])):
        c.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.d_start.copy_(torch.tensor(start, dtype=torch.int32))
        got = attend_counted(c, q, 4, 0.1)
        with pytest.raises(fl.FlError) as e:
            fl.fl_device_status()
        assert e.value.status == -1 and "sequence" in str(e.value), (lens, start)
        fl.fl_device_status()
        bad = [not (0 <= lens[i] <= 64 * c.width and 0 <= start[i] <= start[i + 1] <= 600 and
                    start[i + 1] - start[i] <= min(300, lens[i])) for i in range(3)]
        assert any(bad)
        for i in range(3):
            if start[i:i + 2] != good[1][i:i + 2]:
                continue
            if bad[i]:
                assert np.all(got[good[1][i]:good[1][i + 1]] == 77)
            else:
                c.check(got, q, 4, 0.1, skip=[x for x in range(3) if x != i])


def test_append_leaves_bad_blocks_and_sequences_out(env):
    """A page index or length out of range: that block or sequence is not written, all others are, byte for byte."""
    torch, fl = env
    kvh, D = 2, 64
    for what in ("page", "sequence"):
        c = Case(torch, fl, [200, 100, 130], [80, 100, 2], kvh, D, seed=4)
        if what == "page":
            c.table[0, 2] = c.num_pages
        else:
            c.lens[2] = 64 * c.width + 1
        c.upload()
        k, v = (synth.bf16_normal((c.rows, kvh, D), 4, x) for x in (1, 2))
        fl.fl_kv_append(c.cache, c.batch, dev(torch, k), kvh * D, dev(torch, v), kvh * D)
        with pytest.raises(fl.FlError) as e:
            fl.fl_device_status()
        assert e.value.status == -1 and what in str(e.value)
        want = c.pages.copy()
        for i, (n, new) in enumerate(zip(c.lens, c.news)):
            for x in range(new):
                p, r = n - new + x, c.start[i] + x
                if n > 64 * c.width or c.table[i, p // 64] >= c.num_pages:
                    continue
                for h in range(kvh):
                    (kc, ks), (vc, vs) = kv.quantise(f64(k[r, h])), kv.quantise(f64(v[r, h]))
                    kv.write_token(want[c.table[i, p // 64], h], D, p % 64, kc, ks, vc, vs)
        assert np.array_equal(c.d_pages.cpu().numpy(), want)


@pytest.mark.parametrize("kvh,n_seqs,rows", [(8, 3, 169), (8, 3, 170), (8, 3, 171), (8, 4, 127), (8, 4, 128), (8, 4, 129),
                                             (4, 5, 204), (4, 5, 205), (9, 7, 64), (9, 7, 65), (9, 7, 66)])
def test_attend_row_counts_of_several_sequences(env, kvh, n_seqs, rows):
    """Row counts around the kernels' limit where it lies between 64 and 256."""
    torch, fl = env
    c = Case(torch, fl, [rows + 50 + 40 * i for i in range(n_seqs)], [rows, 1] + [rows - 3 * i for i in range(2, n_seqs)], kvh, 64,
             seed=rows, levels=(2, 4, 4, 0))
    q = c.q(kvh)
    got = attend_counted(c, q, kvh, 0.125)
    fl.fl_device_status()
    c.check(got, q, kvh, 0.125, skip=range(3, n_seqs))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 4)])
def test_sequences_shared_by_both_kernels(env, D, window, sinks):
    """One call whose sequences of 65 to 256 rows divide by how many blocks they see; and a table wider than they need."""
    torch, fl = env
    kvh = 8
    lens, news = [300, 620, 900, 1500, 230, 2100, 66, 64], [200, 130, 256, 70, 65, 256, 64, 64]
    for width in (None, 4096):
        c = Case(torch, fl, lens, news, kvh, D, seed=D + window, levels=(2, 4), rows=sum(news) + 3, width=width)
        q = c.q(kvh)
        got = attend_counted(c, q, kvh, 0.1, window, sinks)
        fl.fl_device_status()
        c.check(got, q, kvh, 0.1, window, sinks, skip=(1, 4, 6))
        c.untouched(got)
        assert np.array_equal(attend_counted(c, q, kvh, 0.1, window, sinks), got)


@pytest.mark.parametrize("n,new,width", [(2000, 128, None), (300, 128, 40000), (20000, 256, None), (30000, 100, 469), (90, 65, 30000)])
def test_one_sequence_between_the_kernels(env, n, new, width):
    """One sequence of 65 to 256 rows: short and long contexts, under tables that allow more."""
    torch, fl = env
    c = Case(torch, fl, [n], [new], 4, 64, seed=n, levels=(2, 4), width=width)
    q = c.q(4)
    got = attend_counted(c, q, 4, 0.125)
    fl.fl_device_status()
    c.check(got, q, 4, 0.125)
