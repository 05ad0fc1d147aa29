"""mxq_attn against the 64-bit reference: the three cache types, lengths from
0 to a few thousand, ragged batches, windows and sinks, pages of every kind,
masked NaNs, rows that see nothing, refused data, offsets past 32 bits,
streams and graphs.

Tolerances.  A weight exp(s - m) is rounded to 16 bits (2^-9 relative, half an
ulp of BF16) before it multiplies its row, the output once more to BF16: with
A = sum_j w_j |k_j| >= |out| the two stay within 2^-8 * A.  The scores come
from FP32 sums of D exact products; their error, at most 2^-19 of
sabs = sm_scale * sum_d |q_d k_d|, moves weights and lse by as much
relatively, twice for the numerator and denominator.
"""

import numpy as np
import pytest
import torch

import attn_ref as ref
import workloads as W

pytestmark = pytest.mark.gpu

SCALE8 = 0.0371


@pytest.fixture(scope="module")
def mxq():
    import mxfp8_block_scaled_inv_gb300 as m
    from mxfp8_block_scaled_inv_gb300 import build

    build.build()
    m.lib()
    return m


class Problem:
    """A seeded batch: nq[b] new tokens on top of lens[b] keys each."""

    def __init__(self, nq, lens, H, D, cache, page=64, window=0, sinks=0, seed=0, q_std=1.0, kv_std=1.0,
                 spare=3, num_slots=None):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.nq, self.lens, self.H, self.D, self.cache, self.page = nq, lens, H, D, cache, page
        self.window, self.sinks = window, sinks
        B, T = len(lens), sum(nq)
        self.pages = max(1, -(-max(lens) // page))
        total = B * self.pages + spare
        self.num_slots = num_slots or total * page
        self.bt = rng.permutation(total)[:B * self.pages].astype(np.int32).reshape(B, self.pages)
        self.q_start = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.q = W.bf16_normal((T, H, D), seed=seed + 1, std=q_std)
        kv = W.f32_normal((total * page, D), seed=seed + 2, std=kv_std)
        self.sf = None
        if cache == "bf16":
            self.kv = kv.bfloat16()
            self.rows = self.kv.double().numpy()
        elif cache == "e4m3":
            self.kv = (kv / SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.rows = ref.e4m3_values(self.kv.numpy()) * np.float64(np.float32(SCALE8))
        else:
            codes, sf = ref.encode_e2m1(kv.numpy())
            self.kv, self.sf = torch.from_numpy(codes), torch.from_numpy(sf)
            self.rows = ref.e2m1_values(codes, sf)

    def slots(self, b, j):
        j = np.asarray(j)
        return self.bt[b, j // self.page].astype(np.int64) * self.page + j % self.page

    def poison(self, slots):
        """Makes rows NaN in the stored form (the reference never reads masked rows)."""
        slots = np.asarray(slots)
        if self.cache == "bf16":
            self.kv[slots] = float("nan")
        elif self.cache == "e4m3":
            self.kv[slots] = 0x7F
        else:
            self.sf[slots] = 0xFF
        self.rows[slots] = np.nan

    def run(self, mxq, scale=None, lse=True, **kw):
        d = "cuda"
        self.err = torch.zeros(1, dtype=torch.int32, device=d)
        lse = torch.full((self.q.shape[0], self.H), 7.0, device=d) if lse else None
        out = mxq.mxq_attn(self.q.to(d), self.kv.to(d), torch.from_numpy(self.bt).to(d),
                           torch.tensor(self.lens, dtype=torch.int32, device=d),
                           q_start=torch.from_numpy(self.q_start).to(d), page_size=self.page,
                           window=self.window, sinks=self.sinks, sm_scale=scale,
                           kv_scale=torch.tensor([SCALE8], device=d) if self.cache == "e4m3" else None,
                           cache_sf=None if self.sf is None else self.sf.to(d), lse=lse,
                           err_flag=self.err, **kw)
        torch.cuda.synchronize()
        return out, lse

    def want(self, scale=None, bad_pages=()):
        return ref.attention(self.q.double().numpy(), self.rows, self.bt, self.page, self.q_start, self.lens,
                             self.window, self.sinks, scale or self.D ** -0.5, bad_pages)


def check(out, lse, want, rows=slice(None)):
    o, l, A, sabs = (x[rows] for x in want)
    got = out.double().cpu().numpy()[rows]
    ds = 2.0 ** -19 * sabs
    tol = A * (2.0 ** -8 + 2 * ds[..., None]) + 1e-30
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - o) / tol)
    assert worst <= 1.0, f"out: {worst:.3f} of the tolerance"
    if lse is not None:
        g = lse.double().cpu().numpy()[rows]
        empty = np.isinf(l)
        assert np.array_equal(np.isneginf(g), empty)
        e = np.abs(g[~empty] - l[~empty]) / (ds[~empty] + 2.0 ** -22 * np.abs(l[~empty]) + 1e-6)
        assert e.size == 0 or e.max() <= 1.0, f"lse: {e.max():.3f} of the tolerance"


CACHES = ["bf16", "e4m3", "e2m1"]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("H,D", [(1, 64), (16, 512), (64, 512), (3, 192), (128, 128), (20, 320)])
def test_decode(mxq, cache, H, D):
    """One new token for sequences of 1 to 1000 keys, lengths around every tile edge."""
    lens = [1, 2, 15, 16, 17, 64, 127, 128, 129, 255, 257, 1000]
    p = Problem([1] * len(lens), lens, H, D, cache, seed=100 + H)
    out, lse = p.run(mxq)
    check(out, lse, p.want())
    assert int(p.err.item()) == 0


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (16, 16), (100, 3), (128, 4), (300, 17), (5000, 4)])
def test_decode_window(mxq, cache, window, sinks):
    """Windows from one key to more than the context, sinks inside, next to and far from the window."""
    lens = [1, 3, 20, 128, 131, 140, 700]
    p = Problem([1] * len(lens), lens, 16, 256, cache, page=32, window=window, sinks=sinks, seed=200 + window)
    out, lse = p.run(mxq)
    check(out, lse, p.want())


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("H,D", [(64, 512), (5, 128), (12, 192), (100, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
def test_ragged_chunks(mxq, cache, H, D, window, sinks):
    """Chunks of 0, 1, 2, 17 and 70 new tokens with and without a prefix: tiles end inside a token, a
    page and a sequence."""
    nq, lens = [17, 0, 1, 70, 2, 40], [17, 33, 200, 150, 500, 41]
    p = Problem(nq, lens, H, D, cache, page=48, window=window, sinks=sinks, seed=300 + H)
    out, lse = p.run(mxq)
    check(out, lse, p.want())


@pytest.mark.parametrize("cache", CACHES)
def test_long_keys_few_rows(mxq, cache):
    """The keys of one row are split over CTAs: 9000 keys, then the joined result; the tail of the weights
    is flat and one first key dominates."""
    p = Problem([1, 1], [9000, 5], 8, 512, cache, page=16, seed=400)
    first = p.slots(0, 0)
    if cache == "bf16":
        p.kv[first] = (p.q[0, 0].float() * 0.4).bfloat16()
        p.rows[first] = p.kv[first].double().numpy()
    out, lse = p.run(mxq)
    check(out, lse, p.want())


@pytest.mark.parametrize("page", [16, 48, 128, 1024])
def test_page_sizes(mxq, page):
    p = Problem([3, 1], [1000, 777], 16, 128, "e4m3", page=page, window=333, sinks=5, seed=500 + page)
    out, lse = p.run(mxq)
    check(out, lse, p.want())


@pytest.mark.parametrize("cache", CACHES)
def test_large_scores(mxq, cache):
    """Scores in the hundreds: the running maximum grows by far more than one step, both ways."""
    p = Problem([2, 5], [600, 300], 8, 256, cache, seed=600, q_std=8.0, kv_std=3.0)
    out, lse = p.run(mxq)
    check(out, lse, p.want())
    p = Problem([4], [700], 16, 128, cache, seed=601)
    out, lse = p.run(mxq, scale=2.5)
    check(out, lse, p.want(scale=2.5))
    out, lse = p.run(mxq, scale=-1.5)
    # A negative scale: the same as negated queries under the positive one.
    check(out, lse, ref.attention(-p.q.double().numpy(), p.rows, p.bt, p.page, p.q_start, p.lens, 0, 0, 1.5))


@pytest.mark.parametrize("cache", CACHES)
def test_rows_that_see_nothing(mxq, cache):
    """Fewer keys than new tokens: the first of them see no key (out 0, lse -inf); a length of zero."""
    p = Problem([6, 3, 2], [2, 0, 2], 12, 128, cache, seed=700)
    out, lse = p.run(mxq)
    w = p.want()
    check(out, lse, w)
    assert (out.float().cpu().numpy()[np.isinf(w[1])] == 0).all()
    assert np.isinf(w[1]).sum() == (4 + 3) * 12


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("H", [4, 64])
def test_masked_nans_reach_nothing(mxq, cache, H):
    """NaN rows past the lengths, before the window (sinks kept), in pages of nobody, and in keys that only
    later tokens of the same tile see."""
    nq, lens = [1, 30, 1], [201, 90, 17]
    p = Problem(nq, lens, H, 128, cache, page=32, window=50, sinks=2, seed=800)
    used = set()
    for b in range(3):
        first = max(0, lens[b] - nq[b] - 50 + 1)
        used |= set(p.slots(b, np.arange(first, lens[b])).tolist()) | set(p.slots(b, np.arange(2)).tolist())
    p.poison([s for s in range(p.rows.shape[0]) if s not in used])
    out, lse = p.run(mxq)
    check(out, lse, p.want())
    # The last key of the chunk: only its last token sees it.
    p.poison(p.slots(1, [lens[1] - 1]))
    out, lse = p.run(mxq)
    w = p.want()
    last = 1 + 30 - 1
    keep = [t for t in range(sum(nq)) if t != last]
    check(out, lse, w, keep)
    assert torch.isnan(out[last].float()).all() and torch.isnan(lse[last]).all()


def test_infinite_keys(mxq):
    """+-infinity in a masked row changes nothing; in a visible one it makes the rows that see it NaN."""
    p = Problem([1, 8], [40, 70], 16, 64, "bf16", page=16, window=20, seed=900)
    p.kv[p.slots(0, [3])] = float("inf")
    p.kv[p.slots(1, [0, 5])] = float("-inf")
    out, lse = p.run(mxq)
    p.rows[p.slots(0, [3])] = np.nan
    check(out, lse, p.want())
    p.kv[p.slots(1, [60]), 7] = float("inf")
    out, lse = p.run(mxq)
    assert torch.isfinite(out[0].float()).all() and torch.isnan(out[1:].float()).all()


def test_block_table_outside_the_cache(mxq):
    """Pages that are negative or past the cache hide their keys and set MXQ_DEVERR_SLOT."""
    p = Problem([1, 2], [100, 90], 16, 128, "e4m3", page=16, seed=1000)
    p.bt[0, 2] = -1
    p.bt[1, 1] = p.num_slots // 16
    bad = {-1, p.num_slots // 16}
    out, lse = p.run(mxq)
    check(out, lse, p.want(bad_pages=bad))
    assert int(p.err.item()) == mxq.MXQ_DEVERR_SLOT


def test_lengths_outside_the_table(mxq):
    """A length past the table is clamped to its reach, a negative one to zero; MXQ_DEVERR_LENGTH."""
    p = Problem([1, 1, 1], [64, 64, 30], 8, 128, "bf16", page=32, seed=1100)
    p.lens = [1000, -5, 30]
    out, lse = p.run(mxq)
    assert int(p.err.item()) == mxq.MXQ_DEVERR_LENGTH
    p.lens = [64, 0, 30]
    check(out, lse, p.want())


def test_tokens_of_no_sequence_are_not_written(mxq):
    p = Problem([3, 2], [50, 60], 4, 64, "bf16", seed=1200)
    p.q_start = np.array([0, 3, 4], dtype=np.int32)
    out = torch.full(p.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    out, lse = p.run(mxq, out=out)
    assert (out[4].float() == 5.0).all() and (lse[4] == 7.0).all()
    p.nq = [3, 1]
    check(out, lse, p.want(), slice(0, 4))


@pytest.mark.parametrize("cache", ["bf16", "e2m1"])
def test_offsets_past_32_bits(mxq, cache):
    """Rows beyond 2^32 bytes into the cache (a cache of 4.5 GiB)."""
    D, page = 512, 64
    row = 1024 if cache == "bf16" else 256
    num = (9 << 29) // row // page * page
    p = Problem([1, 4], [300, 100], 16, D, cache, page=page, seed=1300)
    n = p.rows.shape[0]
    shift = num - n
    dev = "cuda"
    big = torch.empty((num, p.kv.shape[1]), dtype=p.kv.dtype, device=dev)
    big[shift:] = p.kv.to(dev)
    sf = None
    if p.sf is not None:
        sf = torch.empty((num, D // 32), dtype=torch.uint8, device=dev)
        sf[shift:] = p.sf.to(dev)
    want = p.want()
    p.bt += shift // page
    p.kv, p.sf = big, sf
    out, lse = p.run(mxq)
    check(out, lse, want)


def test_default_arguments_and_no_lse(mxq):
    """One token per sequence without q_start; no lse."""
    p = Problem([1] * 5, [3, 40, 64, 65, 200], 8, 128, "bf16", page=64, seed=1400)
    d = "cuda"
    out = mxq.mxq_attn(p.q.to(d), p.kv.to(d), torch.from_numpy(p.bt).to(d),
                       torch.tensor(p.lens, dtype=torch.int32, device=d))
    check(out, None, p.want())


def test_same_inputs_same_bits(mxq):
    p = Problem([1, 1, 20], [5000, 3000, 700], 64, 512, "e4m3", seed=1500)
    a, la = p.run(mxq)
    for _ in range(3):
        b, lb = p.run(mxq)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)


def test_streams_and_graphs(mxq):
    """A side stream, two calls in a row on it with workspaces of their own, and a captured graph."""
    p = Problem([1] * 4, [2000, 900, 30, 4], 16, 512, "bf16", window=600, sinks=4, seed=1600)
    want = p.want()
    d = "cuda"
    q, kv, bt = p.q.to(d), p.kv.to(d), torch.from_numpy(p.bt).to(d)
    lens = torch.tensor(p.lens, dtype=torch.int32, device=d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kw = dict(page_size=p.page, window=p.window, sinks=p.sinks)
    with torch.cuda.stream(s):
        a = mxq.mxq_attn(q, kv, bt, lens, **kw)
        b = mxq.mxq_attn(q, kv, bt, lens, **kw)
    s.synchronize()
    check(a, None, want)
    check(b, None, want)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mxq.mxq_attn(q, kv, bt, lens, out=out, **kw)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    check(out, None, want)


def test_binding_refuses(mxq):
    """Wrong types, shapes and strides raise before anything is launched."""
    p = Problem([1, 1], [40, 64], 8, 128, "bf16", seed=1700)
    d = "cuda"
    q, kv, bt = p.q.to(d), p.kv.to(d), torch.from_numpy(p.bt).to(d)
    lens = torch.tensor(p.lens, dtype=torch.int32, device=d)
    good = dict(q=q, cache=kv, block_table=bt, seq_lens=lens)
    for bad in (dict(q=q.float()), dict(q=q.transpose(0, 1)), dict(cache=kv.float()), dict(cache=kv[:, :64]),
                dict(block_table=bt.long()), dict(seq_lens=lens[:1]), dict(seq_lens=lens.long()),
                dict(page_size=24), dict(window=-1), dict(sinks=-1), dict(sm_scale=float("nan")),
                dict(lse=torch.zeros(2, 8, dtype=torch.float64, device=d)),
                dict(out=torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=d)),
                dict(q=q[:, :, :32].contiguous(), cache=kv[:, :32].contiguous()),
                dict(cache=kv.view(torch.uint8)[:, :128].contiguous()),  # E4M3 without its scale
                dict(cache_sf=torch.zeros(3, 3, dtype=torch.uint8, device=d))):
        with pytest.raises(mxq.MxqError):
            mxq.mxq_attn(**{**good, **bad})
    assert mxq.mxq_watchdog_read() == 0
