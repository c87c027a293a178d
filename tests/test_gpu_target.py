"""GPU parity of the target's verification pass against oracle/target.py: the
paged cache (append, read), its attention and the logit rules.

Appended values and counts are compared bit for bit; attention within a bound
derived from its roundings (attention_bound); logit rules within one rounding
to bf16 of a value computed in fp32.
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
dev = "cuda"
U32 = 2.0**-24
U16 = 2.0**-11
UB = 2.0**-8  # bf16: half a step, relative


@pytest.fixture(scope="module")
def D():
    import block_diffusion_speculative_tap_gb300 as D

    return D


def f64(t):
    return t.detach().double().cpu().numpy()


class Setup:
    """A paged cache with streams of given committed lengths and rows; slots that no
    row sees (other pages, the rest of a last page) hold NaN."""

    def __init__(self, D, rows, lens, nkv=2, d=128, page=16, fp4=False, seed=0, depth=None, extra_rows=0, status=False):
        g = torch.Generator().manual_seed(seed)
        self.g, self.D = g, D
        self.rows, self.lens, self.nkv, self.d, self.page, self.fp4 = rows, lens, nkv, d, page, fp4
        S, T = len(rows), sum(rows)
        need = [-(-(c + n) // page) for c, n in zip(lens, rows)]
        n_pages = sum(need) + 2
        perm = torch.randperm(n_pages, generator=g)
        cols = max(1, max(need)) + 1
        table = torch.full((S, cols), -7, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = perm[at : at + n].to(torch.int32)
            at += n
        self.table = table.to(dev)
        start = np.concatenate([[0], np.cumsum(rows)])
        self.start = start
        self.T = T + extra_rows
        self.k_val = [self.normal(c + n, nkv, d) for c, n in zip(lens, rows)]
        self.v_val = [self.normal(c + n, nkv, d) for c, n in zip(lens, rows)]
        w = d // 2 if fp4 else d
        dt = torch.uint8 if fp4 else torch.bfloat16
        pool = lambda: torch.full((n_pages, nkv, page, w), 255 if fp4 else float("nan"), dtype=dt)
        scale = lambda: torch.full((n_pages, nkv, page, d // 16), 0x7F, dtype=torch.uint8) if fp4 else None
        k, v, ks, vs = pool(), pool(), scale(), scale()
        for s in range(S):
            for vals, x, sc in ((self.k_val, k, ks), (self.v_val, v, vs)):
                c = torch.arange(lens[s] + rows[s])
                pg, sl = table[s, c // page].long(), c % page
                if fp4:
                    codes, byte = O.quantise_fp4(f64(vals[s]))
                    x[pg, :, sl] = torch.from_numpy(codes[..., 0::2] | (codes[..., 1::2] << 4))
                    sc[pg, :, sl] = torch.from_numpy(byte)
                    vals[s] = torch.from_numpy(O.fp4_values(codes, byte)).to(torch.bfloat16)
                else:
                    x[pg, :, sl] = vals[s]
        self.status = torch.zeros(1, dtype=torch.int32, device=dev) if status else None
        to = lambda t: t.to(dev) if t is not None else None
        self.k, self.v, self.ks, self.vs = to(k), to(v), to(ks), to(vs)
        self.cache = D.PagedCache(self.k, self.v, self.table, self.ks, self.vs, status=self.status)
        self.depth = depth
        dp = torch.tensor(depth + [0] * extra_rows, dtype=torch.int32, device=dev) if depth is not None else None
        self.batch = D.Rows(torch.tensor(start, dtype=torch.int32, device=dev),
                            torch.tensor(lens, dtype=torch.int32, device=dev), self.T, max(max(rows), 1), dp)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g).to(torch.bfloat16)

    def positions(self, s):
        at = self.start[s]
        return [self.lens[s] + (self.depth[at + j] if self.depth is not None else j) for j in range(self.rows[s])]

    def drop(self, seen):
        """NaN into the slots of stream s that are not in seen[s]."""
        for s, keep in enumerate(seen):
            for c in range(self.lens[s] + self.rows[s]):
                if c in keep:
                    continue
                pg, sl = int(self.table[s, c // self.page]), c % self.page
                if self.fp4:
                    self.ks[pg, :, sl] = 0x7F
                    self.vs[pg, :, sl] = 0x7F
                else:
                    self.k[pg, :, sl] = float("nan")
                    self.v[pg, :, sl] = float("nan")


def attention_bound(out, mass, spread, n_slots, d, fp4):
    """What the GPU's output may be off, for weights w, A = sum w |v| and B = the
    largest sum_d scale |q_d k_d| of a slot.
    - A score is an fp32 sum of d exact products (4-bit pages: queries in fp16
      over a power of two, off by 2^-25 of the row's largest, at most 2 * 2^-25
      of B * d), scaled: off by (d + 4) * u32 * B at most, twice that for a
      truncating adder; a softmax weight is then off by twice that, relative.
    - exp2 by the special function unit: 2^-21 relative; the scaled argument's
      rounding: u32 of the largest argument, under 2 B / ln 2, in the exponent.
    - a weight enters the product rounded to bf16 (fp16): UB (U16) relative;
      fp16 weights below 2^-14 of 2^7 are off by 2^-32 of the largest.
    - the output's and the sum's fp32 additions: (n + 16) u32 each, twice that
      for a truncating adder.
    - the output is rounded to bf16: UB |out|."""
    B = spread[..., None]
    ds = 2 * (d + 4) * U32 * B + 4 * U32 * B / np.log(2) + (d * 2.0**-24 * B if fp4 else 0.0)
    rel = (U16 if fp4 else UB) + 2 * ds + 2.0**-20 + 4 * (n_slots + 16) * U32
    tiny = n_slots * 2.0**-24 * np.maximum(np.abs(out), mass) if fp4 else 0.0
    return UB * np.abs(out) * (1 + 2 * rel) + mass * rel * (1 + UB) + tiny + 1e-30


def check_attention(setup, q, nq, mode, window=0, sinks=0, tree=None, scale=None, mask=None, out=None):
    got = setup.cache.attend(setup.batch, q, window=window, sinks=sinks, mask=mask if mask is not None else mode,
                             scale=scale, out=out)
    torch.cuda.synchronize()
    for s, (n, C) in enumerate(zip(setup.rows, setup.lens)):
        if n == 0:
            continue
        at = slice(setup.start[s], setup.start[s] + n)
        want, mass, spread = O.paged_attention(f64(q[at]), f64(setup.k_val[s]), f64(setup.v_val[s]), C, mode, window,
                                               sinks, setup.positions(s), tree[s] if tree is not None else None, scale)
        bound = attention_bound(want, mass, spread, C + n, setup.d, setup.fp4)
        err = np.abs(f64(got[at]) - want)
        assert np.all(err <= bound), (s, float((err / bound).max()), np.argwhere(~(err <= bound))[:4])
    return got


def tree_of(n):
    parent = [-1] + [(i - 1) // 2 if i < 7 else i - 4 for i in range(1, n)]
    depth = [0] * n
    for i in range(1, n):
        depth[i] = depth[parent[i]] + 1
    return O.tree_mask(parent), depth


def words_of(masks):
    """Rows of bits, one block of rows a stream, as int32 words."""
    W = max((m.shape[1] + 31) // 32 for m in masks)
    out = []
    for m in masks:
        bits = np.zeros((m.shape[0], W * 32), dtype=np.uint64)
        bits[:, : m.shape[1]] = m
        w = (bits.reshape(m.shape[0], W, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
        out.append(w.astype(np.uint32).view(np.int32))
    return torch.from_numpy(np.concatenate(out)).to(dev)


SHAPES = [
    # rows, committed, kv heads, heads a kv head
    ([1], [0], 1, 1),
    ([1], [37], 2, 4),
    ([1, 1, 1, 1, 1], [0, 1, 15, 300, 129], 2, 8),
    ([3, 0, 5], [40, 9, 0], 1, 3),
    ([16, 16], [100, 511], 2, 5),
    ([7, 33, 0, 1], [64, 200, 5, 700], 1, 6),
    ([130], [70], 1, 2),
    ([45, 90], [0, 150], 1, 12),
]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_causal_attention(D, shape, d, fp4):
    rows, lens, nkv, G = SHAPES[shape]
    page = (16, 32, 64, 128)[(shape + d // 32) % 4]
    st = Setup(D, rows, lens, nkv, d, page, fp4, seed=shape)
    q = st.normal(st.T, nkv * G, d).to(dev)
    check_attention(st, q, nkv * G, "causal")


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (16, 3), (33, 40), (64, 4), (100, 1000), (4096, 7)])
@pytest.mark.parametrize("rows,lens,G", [([1, 1], [200, 31], 4), ([16, 2], [333, 0], 8), ([70], [190], 9)])
def test_windows_and_sinks_with_nan_outside(D, rows, lens, G, window, sinks, fp4):
    """Slots that no row sees hold NaN (in their scales, for 4-bit pages)."""
    st = Setup(D, rows, lens, 2, 64 if G == 4 else 128, 32, fp4, seed=window)
    q = st.normal(st.T, 2 * G, st.d).to(dev)
    st.drop([{c for c in range(C + n) for j in range(n)
              if O.sees(C, n, j, c, "causal", window, sinks, [C + i for i in range(n)])}
             for n, C in zip(rows, lens)])
    check_attention(st, q, 2 * G, "causal", window, sinks)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (20, 6)])
@pytest.mark.parametrize("rows,lens,G", [([3], [5], 1), ([15, 31], [40, 0], 4), ([93], [130], 8)])
def test_block_mode(D, rows, lens, G, window, sinks, fp4):
    st = Setup(D, rows, lens, 1, 128, 64, fp4, seed=window)
    q = st.normal(st.T, G, 128).to(dev)
    check_attention(st, q, G, "block", window, sinks)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2, 0), (3, 5), (40, 2)])
@pytest.mark.parametrize("n,lens,G", [(5, [3, 0], 2), (31, [70, 33], 1), (33, [64, 127], 4), (93, [100], 6)])
def test_tree_mode(D, n, lens, G, window, sinks, fp4):
    """Trees by mask and depth, at committed lengths where the rows' bits straddle
    tiles; windows shorter than the tree is deep cut ancestors off."""
    mask, depth = tree_of(n)
    S = len(lens)
    st = Setup(D, [n] * S, lens, 1, 64 if n == 33 else 128, 16, fp4, seed=n, depth=depth * S)
    q = st.normal(st.T, G, st.d).to(dev)
    check_attention(st, q, G, "tree", window, sinks, [mask] * S, mask=words_of([mask] * S))


@pytest.mark.parametrize("n", [4, 40])
def test_rows_that_see_nothing_are_zero(D, n):
    """Mask words of zero and a window of one: nothing of the context, nothing of the block."""
    st = Setup(D, [n], [50], 1, 128, 16, depth=[1] * n)
    q = st.normal(n, 8, 128).to(dev)
    mask = np.zeros((n, n), dtype=bool)
    mask[n - 1, 0] = True  # only the last row sees a slot
    got = check_attention(st, q, 8, "tree", 1, 0, [mask], mask=words_of([mask]))
    assert not got[: n - 1].any() and got[n - 1].any()
    # no committed slots at all
    st = Setup(D, [n], [0], 1, 128, 16)
    none = np.zeros((n, n), dtype=bool)
    out = st.cache.attend(st.batch, q, mask=words_of([none]))
    assert not out.any()


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("n,C,G", [(1, 9000, 4), (16, 5000, 5), (600, 700, 2), (300, 2100, 4)])
def test_long_contexts_split_over_ctas(D, n, C, G, fp4):
    """Few streams and long caches: slices are joined from the workspace."""
    st = Setup(D, [n, 1], [C, 40], 1, 128, 64, fp4, seed=C)
    q = st.normal(st.T, G, 128).to(dev)
    # rows are many: the oracle looks at a few of them, with the others' slots in place
    got = st.cache.attend(st.batch, q)
    torch.cuda.synchronize()
    for j in sorted({0, n // 3, n - 1}):
        k, v = f64(st.k_val[0][: C + j + 1]), f64(st.v_val[0][: C + j + 1])
        want, mass, spread = O.paged_attention(f64(q[j : j + 1]), k, v, C + j, "causal", 0, 0, [C + j])
        bound = attention_bound(want, mass, spread, C + n, 128, fp4)
        assert np.all(np.abs(f64(got[j : j + 1]) - want) <= bound), j


@pytest.mark.parametrize("scale_q", [1e-30, 1.0, 1e4, 3e38])
def test_query_magnitudes_over_4_bit_pages(D, scale_q):
    """Queries beyond fp16's range: a power of two a row keeps them. scale undoes the
    magnitude, so the scores are ordinary."""
    st = Setup(D, [2, 20], [50, 60], 1, 128, 32, True, seed=2)
    q = (torch.randn(st.T, 4, 128, generator=st.g).clamp(-0.9, 0.9) * scale_q).to(torch.bfloat16).to(dev)
    check_attention(st, q, 4, "causal", scale=float(np.float32(min(128**-0.5 / scale_q, 1e37))))


def test_large_scores(D):
    """Scores of thousands: one slot takes a row's whole weight, nothing overflows."""
    for n in (2, 24):
        st = Setup(D, [n], [300], 1, 128, 32, seed=8)
        q = (st.normal(n, 4, 128) * 64).to(dev)
        got = st.cache.attend(st.batch, q, scale=1.0)
        k, v = f64(st.k_val[0]), f64(st.v_val[0])
        for j in range(n):
            x = k[: 301 + j, 0] @ f64(q[j]).T  # [slots, heads]
            for h in range(4):
                order = np.sort(x[:, h])
                if order[-1] - order[-2] > 60:  # everything else is under 2^-86 of it
                    assert np.array_equal(f64(got[j, h]), v[x[:, h].argmax(), 0])
        assert torch.isfinite(got).all()


def test_strides_and_rows_behind_the_batch(D):
    """Queries read in place from a fused projection; rows past the last stream and
    the gaps of a strided output stay as they were."""
    for n in (2, 19):
        st = Setup(D, [n, 1], [33, 64], 2, 64, 16, seed=1, extra_rows=3)
        fused = torch.randn(st.T, 10, 64, generator=st.g).to(torch.bfloat16).to(dev)
        q = fused[:, 1:9]
        dst = torch.full((st.T, 16, 64), 7.0, dtype=torch.bfloat16, device=dev)
        out = dst[:, 4:12]
        check_attention(st, q, 8, "causal", out=out)
        assert (dst[n + 1 :] == 7).all() and (dst[:, :4] == 7).all() and (dst[:, 12:] == 7).all()


def test_same_bits_again_and_on_another_stream(D):
    for n, fp4 in ((1, False), (16, True), (40, False)):
        st = Setup(D, [n] * 3, [700, 33, 256], 2, 128, 64, fp4, seed=n)
        q = st.normal(st.T, 8, 128).to(dev)
        first = st.cache.attend(st.batch, q)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            other = st.cache.attend(st.batch, q)
        again = st.cache.attend(st.batch, q)
        torch.cuda.synchronize()
        assert torch.equal(first, again) and torch.equal(first, other)


@pytest.mark.parametrize("n", [1, 16])
def test_captured_calls_follow_later_lengths(D, n):
    """Two graphs over one cache, replayed as the committed lengths grow."""
    st = Setup(D, [n, n], [100, 400], 2, 128, 16, seed=3)
    q = st.normal(st.T, 8, 128).to(dev)
    st.cache.attend(st.batch, q)
    torch.cuda.synchronize()
    outs, graphs = [], []
    for window in (0, 24):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(st.cache.attend(st.batch, q, window=window, sinks=4))
        graphs.append(g)
    for lens in ([100, 400], [3, 399], [0, 17]):
        st.batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for window, out in zip((0, 24), outs):
            assert torch.equal(out, st.cache.attend(st.batch, q, window=window, sinks=4)), (lens, window)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("n,G", [(1, 4), (16, 4), (40, 8)])
def test_output_over_the_queries(D, n, G, fp4):
    st = Setup(D, [n] * 2, [3000, 70], 2, 128, 64, fp4, seed=n)
    q = st.normal(st.T, 2 * G, 128).to(dev)
    want = st.cache.attend(st.batch, q)
    got = q.clone()
    assert st.cache.attend(st.batch, got, out=got) is got
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [1, 16, 40])
def test_calls_at_once_on_two_streams(D, n):
    """Eager calls and captured ones of one cache, on two streams at the same time."""
    st = Setup(D, [n] * 2, [3000, 900], 2, 128, 64, seed=n)
    q = st.normal(st.T, 8, 128).to(dev)
    windows = (0, 600)
    want = [st.cache.attend(st.batch, q, window=w).clone() for w in windows]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(25):
        for i, w in enumerate(windows):
            with torch.cuda.stream(sides[i]):
                outs[i].append(st.cache.attend(st.batch, q, window=w))
    torch.cuda.synchronize()
    graphs = []
    for i, w in enumerate(windows):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs[i].append(st.cache.attend(st.batch, q, window=w))
        graphs.append(g)
    for _ in range(25):
        for side, g in zip(sides, graphs):
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(o, w) for o in got)


@pytest.mark.parametrize("rows,lens,nkv,G", [
    ([1] * 70, [(37 * i) % 211 for i in range(70)], 2, 2),  # more streams than a warp's lanes
    ([3] * 40, [(97 * i) % 900 for i in range(40)], 1, 6),
    ([1, 2], [2900, 10], 40, 1),                            # more kv heads than lanes, split streams
    ([20, 1], [1500, 3000], 40, 2),
])
@pytest.mark.parametrize("fp4", [False, True])
def test_many_streams_and_many_heads(D, rows, lens, nkv, G, fp4):
    st = Setup(D, rows, lens, nkv, 64, 16, fp4, seed=len(rows))
    check_attention(st, st.normal(st.T, nkv * G, 64).to(dev), nkv * G, "causal", window=400, sinks=3)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (90, 5), (300, 0), (900, 200)])
@pytest.mark.parametrize("rows,lens,nkv,G", [([700, 5, 333], [1000, 900, 0], 1, 3), ([97], [2000], 2, 8), ([1025], [0], 1, 1),
                                             ([16, 15], [800, 3000], 1, 1)])
@pytest.mark.parametrize("depths", [False, True])
def test_prompt_chunks(D, rows, lens, nkv, G, window, sinks, depths):
    """Rows of several tiles, whose tiles see more and more (or a window that moves on
    through the chunk itself), split over CTAs."""
    depth = [j + (j * 7) % 5 for n in rows for j in range(n)] if depths else None
    st = Setup(D, rows, lens, nkv, 64, 32, seed=sum(rows), depth=depth)
    check_attention(st, st.normal(st.T, nkv * G, 64).to(dev), nkv * G, "causal", window, sinks)


@pytest.mark.parametrize("n", [1, 6])
def test_rows_far_under_the_bound(D, n):
    """A padded batch: max_rows and the buffers are for many more rows than there are."""
    st = Setup(D, [n, 0, n], [300, 5, 1100], 2, 128, 32, seed=n, extra_rows=700)
    st.batch = D.Rows(st.batch.row_start, st.batch.lens, st.T, 700)
    q = torch.full((st.T, 8, 128), float("nan"), dtype=torch.bfloat16, device=dev)
    q[: 2 * n] = st.normal(2 * n, 8, 128).to(dev)
    out = torch.full_like(q, 7.0)
    check_attention(st, q, 8, "causal", out=out)
    assert (out[2 * n :] == 7).all()


@pytest.mark.parametrize("n", [1, 9])
def test_streams_that_share_pages(D, n):
    """A common prompt: the committed pages of one stream in another's table."""
    st = Setup(D, [n, n], [128, 128], 2, 64, 16, seed=n)
    st.table[1, :8] = st.table[0, :8]
    st.k_val[1][:128], st.v_val[1][:128] = st.k_val[0][:128], st.v_val[0][:128]
    check_attention(st, st.normal(st.T, 8, 64).to(dev), 8, "causal")


def test_threads_on_one_stream(D):
    """Two threads' calls on one stream, in whatever order their launches come."""
    import threading

    setups = [Setup(D, [n] * 2, [3000, 900], 2, 128, 64, seed=n) for n in (16, 40)]
    qs = [st.normal(st.T, 8, 128).to(dev) for st in setups]
    want = [st.cache.attend(st.batch, q).clone() for st, q in zip(setups, qs)]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(100):
            got[i].append(setups[i].cache.attend(setups[i].batch, qs[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert len(outs) == 100 and all(torch.equal(o, w) for o in outs)


def test_a_workspace_that_grows(D):
    """Small, large and small calls again, eager and captured, one behind the other."""
    small, large = (Setup(D, [n], [2000], 2, 128, 64, seed=n) for n in (1, 60))
    q0, q1 = small.normal(1, 8, 128).to(dev), large.normal(60, 8, 128).to(dev)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = small.cache.attend(small.batch, q0)
        b = large.cache.attend(large.batch, q1)
        c = small.cache.attend(small.batch, q0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d = large.cache.attend(large.batch, q1)
        e = small.cache.attend(small.batch, q0)
    for _ in range(3):
        g.replay()
        f = large.cache.attend(large.batch, q1)
        torch.cuda.synchronize()
        assert torch.equal(a, c) and torch.equal(a, e) and torch.equal(b, d) and torch.equal(b, f)


def test_numbers_past_32_bits_are_refused(D):
    st = Setup(D, [1], [20], 2, 64, 16)
    q = st.normal(1, 4, 64).to(dev)
    for bad in (dict(window=1 << 32), dict(window=(1 << 32) + 5), dict(window=4, sinks=1 << 31)):
        with pytest.raises(ValueError):
            st.cache.attend(st.batch, q, **bad)
    for n, m in ((1 << 32, 1), (1, 1 << 32), (-(1 << 32), 1)):
        with pytest.raises(ValueError):
            D.Rows(st.batch.row_start, st.batch.lens, n, m)


def test_bad_tables_and_rows_are_flagged_and_never_followed(D):
    """A needed slot without a page, lengths past the table, descending row_start:
    status bits, rows of other streams unharmed."""
    for n in (1, 24):
        st = Setup(D, [n, n], [100, 60], 1, 64, 16, seed=4, status=True)
        q = st.normal(st.T, 4, 64).to(dev)
        good = st.cache.attend(st.batch, q)
        assert int(st.status) == 0
        for bad in (-1, 10**6):
            keep = int(st.table[0, 2])
            st.table[0, 2] = bad
            out = st.cache.attend(st.batch, q)
            assert int(st.status) == 8 and torch.equal(out[n:], good[n:]), bad
            st.status.zero_()
            k = st.normal(st.T, 1, 64).to(dev)
            st.table[0, 2] = keep
            st.table[0, 100 // 16] = bad
            before = st.k.clone()
            st.cache.append(st.batch, k, k)
            st.cache.read(st.batch)
            assert int(st.status) == 8
            mine = [int(p) for p in st.table[1] if p >= 0]
            other = [p for p in range(st.k.shape[0]) if p not in mine and p not in [int(x) for x in st.table[0]]]
            same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))
            assert same(st.k[other], before[other])
            st.status.zero_()
            st = Setup(D, [n, n], [100, 60], 1, 64, 16, seed=4, status=True)
        st.batch.lens.copy_(torch.tensor([10**8, -5], dtype=torch.int32))
        st.cache.attend(st.batch, q)
        assert int(st.status) & 16
        st.status.zero_()
        st.batch.lens.copy_(torch.tensor([100, 60], dtype=torch.int32))
        st.batch.row_start.copy_(torch.tensor([0, 5 * n, -3], dtype=torch.int32))
        st.cache.attend(st.batch, q)
        assert int(st.status) & 16


# ---------------------------------------------------------------- append and read


def rope_table(n, d, theta=1e6):
    a = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    return torch.stack([a.cos(), a.sin()], -1).float()


def rotate32(x, rope, pos):
    """The documented fp32 operations, each rounded."""
    cs = rope[torch.as_tensor(pos)].to(x.device)[:, None]
    c, s = cs[..., 0], cs[..., 1]
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(torch.bfloat16)


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("rows,lens,nkv,nq", [([1], [0], 1, 1), ([2, 0, 19], [15, 8, 130], 2, 6), ([16], [4090], 8, 40),
                                              ([3] * 40, list(range(40)), 1, 2)])
def test_append_and_read(D, rows, lens, nkv, nq, d, fp4):
    page = 16 if d == 64 else 64
    st = Setup(D, rows, lens, nkv, d, page, fp4, seed=d, extra_rows=2)
    rope = rope_table(max(lens) + max(rows), d)
    qkv = torch.randn(st.T, nq + 2 * nkv, d, generator=st.g).to(torch.bfloat16).to(dev)
    q, k, v = qkv[:, :nq], qkv[:, nq : nq + nkv], qkv[:, nq + nkv :]
    before = [t.clone() if t is not None else None for t in (st.k, st.v, st.ks, st.vs)]
    q_out = torch.full((st.T, nq, d), 5.0, dtype=torch.bfloat16, device=dev)
    st.cache.append(st.batch, k, v, rope.to(dev), q=q, q_out=q_out)
    pos = [c + j for c, n in zip(lens, rows) for j in range(n)]
    T = sum(rows)
    assert torch.equal(bits(q_out[:T]), bits(rotate32(q[:T], rope, pos))) and (q_out[T:] == 5).all()
    # the formula in 64 bits, within the rounding to bf16 and the three of fp32
    c, s = f64(rope[torch.as_tensor(pos)][:, None]).transpose(3, 0, 1, 2)
    h = d // 2
    a, b = f64(q[:T])[..., :h], f64(q[:T])[..., h:]
    for got, x, y, sg in ((f64(q_out[:T])[..., :h], a, b, -1.0), (f64(q_out[:T])[..., h:], b, a, 1.0)):
        want, room = x * c + sg * y * s, (np.abs(x * c) + np.abs(y * s)) * 2 * U32
        assert np.all(np.abs(got - want) <= UB * (np.abs(want) + room) + room)
    want_k, want_v = rotate32(k[:T], rope, pos).cpu(), v[:T].cpu()
    if fp4:
        # a midpoint of codes is hit exactly here: bits of the oracle's quantiser
        packed = [O.quantise_fp4(f64(x)) for x in (want_k, want_v)]
        want_k, want_v = (torch.from_numpy(O.fp4_values(*p)).to(torch.bfloat16) for p in packed)
    got_k, got_v = st.cache.read(st.batch)
    assert torch.equal(got_k[:T].cpu(), want_k) and torch.equal(got_v[:T].cpu(), want_v)
    # exactly the rows' slots have changed
    after = [st.k, st.v, st.ks, st.vs]
    at = 0
    touched = torch.zeros(st.k.shape[0], page, dtype=torch.bool)
    for i, (n, C) in enumerate(zip(rows, lens)):
        for j in range(n):
            pg, sl = int(st.table[i, (C + j) // page]), (C + j) % page
            touched[pg, sl] = True
            if fp4:
                for x, sc, (codes, byte) in ((st.k, st.ks, packed[0]), (st.v, st.vs, packed[1])):
                    want = torch.from_numpy(codes[at + j][..., 0::2] | (codes[at + j][..., 1::2] << 4))
                    assert torch.equal(x[pg, :, sl].cpu(), want)
                    assert torch.equal(sc[pg, :, sl].cpu(), torch.from_numpy(byte[at + j]))
        at += n
    for x, y in zip(before, after):
        if x is not None:
            m = ~touched.to(dev)
            assert torch.equal(bits(x.transpose(1, 2)[m]), bits(y.transpose(1, 2)[m]))


def test_append_without_rotation_with_depths_and_in_place(D):
    depth = [0, 1, 1, 2]
    st = Setup(D, [4], [9], 2, 64, 16, depth=depth, status=True)
    k, v, q = (st.normal(4, 2, 64).to(dev) for _ in range(3))
    assert st.cache.append(st.batch, k, v) is None
    got_k, got_v = st.cache.read(st.batch)
    assert torch.equal(got_k, k) and torch.equal(got_v, v)
    rope = rope_table(12, 64)
    want = rotate32(q, rope, [9 + x for x in depth])
    st.cache.append(st.batch, k, v, rope.to(dev), q=q, q_out=q)
    assert torch.equal(bits(q), bits(want)) and int(st.status) == 0
    assert torch.equal(bits(st.cache.read(st.batch)[0]), bits(rotate32(k, rope, [9 + x for x in depth])))
    # a position past the table of angles: flagged, the row left alone
    st.cache.append(st.batch, v, v, rope[:11].contiguous().to(dev))
    assert int(st.status) == 16
    assert torch.equal(bits(st.cache.read(st.batch)[0][3]), bits(rotate32(k, rope, [9 + x for x in depth])[3]))


def test_quantised_specials(D):
    """Infinities and NaN clamp; a group under the least scale becomes zeros; signs of zeros stay."""
    st = Setup(D, [1], [0], 1, 32, 16, True)
    k = torch.zeros(1, 1, 32, dtype=torch.bfloat16)
    k[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0])
    k[0, 0, 16:18] = torch.tensor([2.0**-12, -(2.0**-12)])
    st.cache.append(st.batch, k.to(dev), k.to(dev))
    got = st.cache.read(st.batch)[0][0, 0].float().cpu()
    assert got[:4].tolist() == [2688.0, -2688.0, 2688.0, 0.0]
    assert not got[16:].any()


def test_slots_past_four_gigabytes(D):
    """Offsets of 64 bits: pages at the end of a pool of more than 2^32 bytes."""
    n_pages, nkv, page, d = 20000, 8, 128, 128
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 12 GB of pools")
    k = torch.empty(n_pages, nkv, page, d, dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    table = torch.tensor([[n_pages - 1, 17, n_pages - 2]], dtype=torch.int32, device=dev)
    cache = D.PagedCache(k, v, table)
    for n in (300, 1):  # a prompt, then a token, over the same slots
        lens = torch.tensor([0 if n == 300 else 300], dtype=torch.int32, device=dev)
        batch = D.Rows(torch.tensor([0, n], dtype=torch.int32, device=dev), lens, n, n)
        g = torch.Generator().manual_seed(n)
        new = [torch.randn(n, nkv, d, generator=g).to(torch.bfloat16).to(dev) for _ in range(2)]
        cache.append(batch, *new)
        assert torch.equal(cache.read(batch)[1], new[1])
        if n == 300:
            hist = new
        q = torch.randn(n, nkv, d, generator=g).to(torch.bfloat16).to(dev)
        out = cache.attend(batch, q)
        j = n - 1
        kk, vv = (f64(torch.cat([a, b]) if n == 1 else a) for a, b in zip(hist, new))
        want, mass, spread = O.paged_attention(f64(q[j:]), kk, vv, len(kk) - 1, "causal", 0, 0, [len(kk) - 1])
        assert np.all(np.abs(f64(out[j:]) - want) <= attention_bound(want, mass, spread, len(kk), d, False))


# ---------------------------------------------------------------- logit rules


@pytest.mark.parametrize("S,N,V,tree", [(1, 1, 8, False), (2, 16, 2048, False), (3, 5, 2056, True), (2, 40, 4104, True),
                                        (1, 3, 151936, False)])
def test_logit_rules(D, S, N, V, tree):
    g = np.random.default_rng(V + N)
    x = torch.from_numpy(g.standard_normal((S, N, V)) * 4).to(torch.bfloat16)
    x[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0])[: min(4, V)]
    counts = np.zeros((S, V), dtype=np.uint16)
    hist = g.integers(0, V, size=(S, 60))
    for s in range(S):
        O.count_tokens(counts[s], hist[s, :30], False)
        O.count_tokens(counts[s], hist[s, 20:], True)
    tokens = np.where(g.random((S, N)) < 0.5, g.integers(0, min(V, 30), size=(S, N)), hist[:, :1])
    tokens[:, -1] = -1 if N > 2 else tokens[:, -1]  # an id outside the vocabulary counts nowhere
    if tree:
        mask, _ = tree_of(N)
    else:
        mask = np.tril(np.ones((N, N), dtype=bool))
    rep, freq, pres = (g.uniform(lo, hi, S).astype(np.float32) for lo, hi in ((0.8, 2), (-0.2, 1), (-0.5, 1)))
    nb = [0, 37, 600][:S] if S > 1 else [5]
    ids = [np.concatenate([g.integers(-2, V + 3, size=n - n // 3), g.integers(0, min(V, 6), size=n // 3)]) for n in nb]
    vals = [g.standard_normal(n).astype(np.float32) for n in nb]
    allowed = g.random((S, N, V)) < 0.7
    words = (V + 31) // 32
    pad = np.zeros((S, N, words * 32), dtype=np.uint64)
    pad[..., :V] = allowed
    gram = (pad.reshape(S, N, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(dt).to(dev)
    kw = dict(
        counts=t(counts.view(np.int16), torch.int16), tokens=t(tokens, torch.int32),
        node_mask=words_of([mask] * S).view(S, N, -1) if tree else None,
        repetition=t(rep, torch.float32), frequency=t(freq, torch.float32), presence=t(pres, torch.float32),
        bias=(t(np.concatenate([[0], np.cumsum(nb)]), torch.int32), t(np.concatenate(ids), torch.int32),
              t(np.concatenate(vals), torch.float32)),
        grammar=t(gram, torch.int32),
    )
    xd = x.to(dev)
    got = D.logit_rules(xd, **kw)
    part = D.logit_rules(xd, counts=kw["counts"], presence=kw["presence"])
    same = D.logit_rules(xd)
    assert torch.equal(bits(same), bits(xd))
    place = xd.clone()
    assert D.logit_rules(place, **kw, out=place) is place and torch.equal(bits(place), bits(got))
    for s in range(S):
        for n in range(N):
            path = [tokens[s, m] for m in range(1, N) if mask[n, m]]
            xs = f64(x[s, n])
            for res, want in (
                (got, O.logit_rules(xs, counts[s], path, rep[s], freq[s], pres[s], list(zip(ids[s], vals[s])),
                                    allowed[s, n])),
                (part, O.logit_rules(xs, counts[s], [], presence=pres[s])),
            ):
                y = f64(res[s, n])
                assert np.array_equal(np.isneginf(want), np.isneginf(y))
                fin = np.isfinite(want)
                assert np.array_equal(y[~fin], want[~fin])
                # fp32 steps: each within u32 of the magnitudes it adds (the count's products,
                # the biases one by one), then half a step of bf16
                size = np.abs(xs) * 3 + (np.abs(freq[s]) * 100 + np.abs(pres[s]))
                for i, b in zip(ids[s], vals[s]):
                    if 0 <= i < V:
                        size[i] += (len(ids[s]) + 1) * abs(b)
                room = 4 * U32 * size[fin]
                assert np.all(np.abs(y[fin] - want[fin]) <= UB * (np.abs(want[fin]) + room) + room)


def test_token_counts(D):
    V, S = 64, 3
    g = np.random.default_rng(9)
    want = np.zeros((S, V), dtype=np.uint16)
    want[1, 5] = 32766
    counts = torch.from_numpy(want.copy().view(np.int16)).to(dev)
    n = [0, 5000, 77]
    toks = g.integers(-2, V + 2, size=sum(n)).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(n)])
    for prompt in (False, True):
        part = toks if not prompt else toks[:5007]
        st = start if not prompt else np.minimum(start, 5007)
        D.token_counts(counts, torch.from_numpy(part).to(dev),
                       torch.from_numpy(st.astype(np.int32)).to(dev), prompt=prompt)
        for s in range(S):
            O.count_tokens(want[s], part[st[s] : st[s + 1]], prompt)
    assert np.array_equal(counts.cpu().numpy().view(np.uint16), want)
    assert want[1, 5] & 0x7FFF == 32767  # saturated
    rows = np.full((S, 16), -1, dtype=np.int32)  # as verification writes them
    rows[0, :3] = [7, 7, 63]
    rows[2, :1] = 0
    D.token_counts(counts, torch.from_numpy(rows).to(dev))
    for s in range(S):
        O.count_tokens(want[s], rows[s], False)
    assert np.array_equal(counts.cpu().numpy().view(np.uint16), want)


def test_rules_of_more_streams_than_a_grid_axis_holds(D):
    S, V = 65600, 8
    g = torch.Generator().manual_seed(4)
    x = torch.randn(S, 1, V, generator=g).to(torch.bfloat16).to(dev)
    counts = torch.randint(0, 3, (S, V), generator=g).to(torch.int16).to(dev)
    presence = torch.randn(S, generator=g).to(dev)
    got = D.logit_rules(x, counts=counts, presence=presence)
    want = torch.where(counts[:, None] > 0, x.float() - presence[:, None, None], x.float()).to(torch.bfloat16)
    assert torch.equal(got, want)


# ---------------------------------------------------------------- the pass as it is used


class ToyTarget:
    """One attention layer over the paged cache between a table of projections by token
    and a linear head, rows as one batch: what the operators are between."""

    def __init__(self, D, V, nq, nkv, d, S, fp4, seed):
        g = torch.Generator().manual_seed(seed)
        self.D, self.nq, self.nkv, self.d, self.S = D, nq, nkv, d, S
        self.qkv = torch.randn(V, nq + 2 * nkv, d, generator=g).to(torch.bfloat16).to(dev)
        self.head = (torch.randn(V, nq * d, generator=g) * 0.2).to(dev)
        self.rope = rope_table(256, d).to(dev)
        table = torch.randperm(S * 8, generator=g).to(torch.int32).view(S, 8).to(dev)
        z = lambda n, dt: torch.zeros(S * 8, nkv, 32, n, dtype=dt, device=dev)
        if fp4:
            b = torch.uint8
            self.cache = D.PagedCache(z(d // 2, b), z(d // 2, b), table, z(d // 16, b), z(d // 16, b))
        else:
            self.cache = D.PagedCache(z(d, torch.bfloat16), z(d, torch.bfloat16), table)

    def rows(self, n, lens, depth=None):
        start = torch.arange(self.S + 1, dtype=torch.int32, device=dev) * n
        return self.D.Rows(start, torch.tensor(lens, dtype=torch.int32, device=dev), self.S * n, n, depth)

    def score(self, tokens, batch, mask="causal"):
        x = self.qkv[tokens.long().view(-1)]
        q = self.cache.append(batch, x[:, self.nq : self.nq + self.nkv], x[:, self.nq + self.nkv :], self.rope,
                              q=x[:, : self.nq])
        a = self.cache.attend(batch, q, window=40, sinks=2, mask=mask)
        return (a.flatten(1).float() @ self.head.T).to(torch.bfloat16).view(self.S, -1, self.head.shape[0])


def only(tokens, V):
    """Grammar words that allow one token a row: tokens [S, N]."""
    S, N = tokens.shape
    allowed = np.zeros((S * N, V), dtype=bool)
    allowed[np.arange(S * N), tokens.cpu().numpy().reshape(-1)] = True
    return words_of([allowed]).view(S, N, -1)


@pytest.mark.parametrize("fp4", [False, True])
def test_verification_rounds_equal_token_by_token(D, fp4):
    """A drafted block scored at once gives the scores that its tokens give one at a
    time, so does a draft tree along its branches, under penalties that count each
    row's own path; under a grammar, verification commits what it allows.

    Two runs of the attention differ by at most twice its bound: under
    4 * UB * max |v| an output (a weight's and the output's rounding on each side;
    the fp32 terms are far below the slack of |v|'s maximum), which the head sums;
    each side's scores are then rounded to bf16, divided by or multiplied with the
    repetition penalty, and rounded again."""
    S, V, C0 = 2, 512, 20
    g = torch.Generator().manual_seed(12)
    toy = ToyTarget(D, V, 8, 2, 64, S, fp4, 5)
    draw = lambda *s: torch.randint(0, V, s, generator=g, dtype=torch.int32).to(dev)
    prompt, plan = draw(S, C0), draw(S, 17)
    anchor = plan[:, 0].contiguous()
    toy.score(prompt, toy.rows(C0, [0, 0]))
    counts = torch.zeros(S, V, dtype=torch.int16, device=dev)
    D.token_counts(counts, prompt, prompt=True)
    D.token_counts(counts, anchor[:, None].contiguous())
    rules = dict(repetition=torch.full((S,), 1.3, device=dev), presence=torch.full((S,), 0.4, device=dev))
    # token by token
    solo_counts, solo = counts.clone(), []
    for i in range(16):
        lg = toy.score(plan[:, i : i + 1], toy.rows(1, [C0 + i] * S))
        solo.append(D.logit_rules(lg, solo_counts, **rules))
        if i < 15:
            D.token_counts(solo_counts, plan[:, i + 1 : i + 2].contiguous())
    solo = torch.cat(solo, 1)
    vmax = float(toy.qkv[:, toy.nq + toy.nkv :].abs().max()) * (1 + 2.0**-4)  # 4-bit values may round up
    off = 4 * UB * vmax * toy.head.abs().sum(1).double()

    def close(x, y):
        room = (off + 2 * UB * y.double().abs()) * 1.3 + 2 * UB * (y.double().abs() + off)
        err = (x.double() - y.double()).abs()
        assert bool((err <= room).all()), float((err / room).max())
        return float(err.max())

    # the block at once
    block = plan[:, :16].contiguous()
    raw = toy.score(block, toy.rows(16, [C0] * S))
    lg = D.logit_rules(raw, counts, tokens=block, **rules)
    close(lg, solo)
    # under a grammar that follows the plan, with one drafted token off it
    draft = block[:, 1:].clone()
    draft[0, 9] = (draft[0, 9] + 1) % V
    lg = D.logit_rules(raw, counts, tokens=block, grammar=only(plan[:, 1:17], V), **rules)
    accept, tokens = D.verify_greedy(draft.contiguous(), lg)
    assert accept.tolist() == [9, 15]
    assert tokens[0, :11].tolist() == plan[0, 1:11].tolist() + [-1] and tokens[1].tolist() == plan[1, 1:].tolist()
    after = D.token_counts(counts.clone(), tokens)
    want = D.token_counts(solo_counts.clone(), plan[:, 16:17].contiguous())
    assert torch.equal(after[1], want[1])
    # a tree whose first branch is the plan
    widths = [2, 2, 1]
    cand = torch.zeros(S, 15, 2, dtype=torch.int32, device=dev)
    cand[..., 0] = plan[:, 1:16]
    cand[..., 1] = (cand[..., 0] + 7) % V
    toks, parents, depths, mask = D.tree_build(anchor, cand.view(S * 15, 2).contiguous(), widths)
    N = toks.shape[1]
    raw = toy.score(toks, toy.rows(N, [C0] * S, depths.view(-1)), mask=mask.view(S * N, -1))
    lg = D.logit_rules(raw, counts, tokens=toks, node_mask=mask, **rules)
    branch = [0]
    for _ in widths:
        branch.append(parents[0].tolist().index(branch[-1]))
    close(lg[:, branch], solo[:, : len(branch)])
    follow = plan[:, 1:].gather(1, depths.long())
    lg = D.logit_rules(raw, counts, tokens=toks, node_mask=mask, grammar=only(follow, V), **rules)
    accept, out, node = D.tree_verify(toks, lg, widths)
    assert accept.tolist() == [3, 3] and node.tolist() == [branch[-1]] * S
    assert torch.equal(out[:, :4], plan[:, 1:5])
