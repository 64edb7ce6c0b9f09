"""GPU parity of the entry points for beam search over a paged fp8 K/V cache against plain
implementations: appended rows byte for byte against the oracle's encoder, attention against its formula in 64
bits, selections, page tables and copies exactly; then whole steps against a search over dense caches."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BAD_INDEX, BAD_PAGE, NO_PAGE, BAD_VALUE = 1, 2, 16, 32


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_kv_cache_fp8_gb300 as k
    return k


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def host(t):
    return t.cpu().numpy()


def scratch(n):
    """A workspace of n bytes whose contents are no zeros."""
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda")


def new_planes(kv, rows, d, code=0x7F, scale=float("nan")):
    """Planes that hold NaN codes and scales wherever nothing is written."""
    return dict(k=torch.full((kv, rows, d), code, dtype=torch.uint8, device="cuda"), k_scale=torch.full((kv, rows), scale, device="cuda"),
                v=torch.full((kv, rows, d), code, dtype=torch.uint8, device="cuda"), v_scale=torch.full((kv, rows), scale, device="cuda"))


def graphed(step):
    """`step` captured into a graph (after a run of it on a side stream)."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    return g


# --- the append ----------------------------------------------------------------------------------

def encoded(orc, x):
    """x [rows, kv, d] -> codes [kv, rows, d], scales [kv, rows] as the oracle encodes each row of a head."""
    n, kv, d = x.shape
    c, s = orc.encode_fp8(np.ascontiguousarray(x.reshape(n * kv, d)))
    return c.reshape(n, kv, d).transpose(1, 0, 2), s.reshape(n, kv).T


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,kv,layout", [(1, 1, "plain"), (37, 3, "fused"), (130, 8, "fused"), (77, 2, "heads first"), (3001, 5, "plain")])
def test_append_bytes(kvq, orc, d, bf16, rows, kv, layout):
    g = np.random.default_rng(d + rows + bf16)
    x = g.standard_normal((2, rows, kv, d)).astype(np.float32) * np.exp(g.uniform(-9, 9, (2, rows, kv, 1))).astype(np.float32)
    x[0, 0] = 0.0                                            # a zero row
    if rows > 20:
        x[:, 5] *= np.float32(2.0**-110)                     # scales at the ends of the range
        x[:, 6] *= np.float32(2.0**100)
        x[1, 7, :, 1:] = 0.0
        x[:, 8, 0] = np.float32(-0.0)
    t = dev(x)
    if bf16:
        t = t.bfloat16()
        x = host(t.float())
    if layout == "fused":
        fused = torch.empty(rows, 3 * kv + 1, d, dtype=t.dtype, device="cuda")
        fused[:, 1:1 + kv], fused[:, 1 + 2 * kv:] = t[0], t[1]
        k, v = fused[:, 1:1 + kv], fused[:, 1 + 2 * kv:]
    elif layout == "heads first":
        k, v = (y.transpose(0, 1).contiguous().transpose(0, 1) for y in t)
    else:
        k, v = t[0], t[1]
    pool = rows + 50
    slot = g.permutation(pool)[:rows].astype(np.int32)
    if rows > 20:
        slot[[3, 19]] = -1, -7
        slot[11] = pool                                      # outside the pool: skipped, and flagged
    pl, st = new_planes(kv, pool, d), i32(1)
    kvq.kvq_append_kv8(k, v, dev(slot), pl, st)
    torch.cuda.synchronize()
    assert st.item() == (BAD_PAGE if rows > 20 else 0)
    ok = (slot >= 0) & (slot < pool)
    for i, name in enumerate(("k", "v")):
        codes, scales = encoded(orc, x[i])
        want = np.full((kv, pool, d), 0x7F, np.uint8), np.full((kv, pool), np.nan, np.float32)
        want[0][:, slot[ok]], want[1][:, slot[ok]] = codes[:, ok], scales[:, ok]
        assert np.array_equal(host(pl[name]), want[0])
        assert np.array_equal(host(pl[name + "_scale"]).view(np.uint32), want[1].view(np.uint32))


@pytest.mark.parametrize("d,rows,kv,layout", [(64, 15001, 13, "fused"), (128, 12003, 9, "plain"), (256, 19990, 3, "fused")])
@pytest.mark.parametrize("bf16", [False, True])
def test_append_bytes_of_many_rows(kvq, orc, d, bf16, rows, kv, layout):
    """As many that a warp takes a dozen vectors or more in turn."""
    test_append_bytes(kvq, orc, d, bf16, rows, kv, layout)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bf16", [False, True])
def test_append_what_is_no_number(kvq, d, bf16):
    """Rows with infinities and NaNs, rows near the type's largest and smallest: the bytes of kvq_encode_fp8."""
    rows, kv = 24, 2
    x = np.random.default_rng(d).standard_normal((2, rows, kv, d)).astype(np.float32)
    x[:, 0, :, 3] = np.inf
    x[:, 1, :, d - 1] = -np.inf
    x[:, 2, :, 0], x[:, 2, :, 9] = np.inf, -np.inf
    x[:, 3, :, 5] = np.nan
    x[:, 4] = np.nan
    x[:, 5, :, 5], x[:, 5, :, 6] = np.nan, np.inf
    x[:, 6, :, 7] = 3.3e38
    x[:, 7] *= np.float32(1e-38)
    x[:, 8] = 0.0
    x[:, 8, :, 1] = np.float32(2.0**-133)
    x[:, 9] = 0.0
    x[:, 9, :, 1] = np.nan
    t = dev(x)
    t = t.bfloat16() if bf16 else t
    pl, slot = new_planes(kv, rows, d), torch.arange(rows, dtype=torch.int32, device="cuda")
    kvq.kvq_append_kv8(t[0], t[1], slot, pl)
    for i, name in enumerate(("k", "v")):
        flat = t[i].float().reshape(rows * kv, d).contiguous()
        codes, scales = torch.zeros(rows * kv, d, dtype=torch.uint8, device="cuda"), torch.zeros(rows * kv, device="cuda")
        kvq.kvq_encode_fp8(flat, codes, scales)
        torch.cuda.synchronize()
        assert np.array_equal(host(pl[name]), host(codes).reshape(rows, kv, d).transpose(1, 0, 2))
        got, want = host(pl[name + "_scale"]), host(scales).reshape(rows, kv).T
        assert np.array_equal(got, want, equal_nan=True) and np.isposinf(got[:, 0]).all()


def test_append_nothing(kvq):
    pl = new_planes(2, 16, 64)
    x = torch.zeros(0, 2, 64, device="cuda")
    kvq.kvq_append_kv8(x, x, i32(0), pl)
    torch.cuda.synchronize()
    assert bool((pl["k"] == 0x7F).all())


# --- the decode ----------------------------------------------------------------------------------

def values(pl, name, rows, dtype=torch.float64):
    return pl[name].view(torch.float8_e4m3fn)[:, rows].to(dtype) * pl[name + "_scale"][:, rows, None].to(dtype)


def decode_ref(pl, q, lens, rows_of, window, scale):
    """out, lse in 64 bits, and two bounds of each head: on |score error| / 2^-24 and sum of p |v| (the largest over dims)."""
    n, H, d = q.shape
    kv = pl["k"].shape[0]
    G = H // kv
    out = torch.zeros(n, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda")
    size = torch.zeros(n, H, dtype=torch.float64, device="cuda")
    mass = torch.zeros(n, H, d, dtype=torch.float64, device="cuda")
    for s in range(n):
        L = int(lens[s])
        pos = np.arange(max(0, L - window) if window else 0, L)
        rows = rows_of(s, pos)
        rows = torch.from_numpy(rows[rows >= 0]).cuda()
        if rows.numel() == 0:
            continue
        K, V = values(pl, "k", rows), values(pl, "v", rows)
        qs = q[s].double().view(kv, G, d)
        x = qs @ K.transpose(1, 2) * scale
        lse[s] = torch.logsumexp(x, 2).flatten()
        p = torch.softmax(x, 2)
        out[s], mass[s] = (p @ V).view(H, d), (p @ V.abs()).view(H, d)
        # the terms of a score, and the score itself (its scaling by fp32 factors and log2 e)
        size[s] = ((qs.abs() @ K.abs().transpose(1, 2)) * abs(scale)).amax(2).flatten()
    return out, lse, size, mass


def check_decode(out, lse, ref, d, rows):
    o, l, size, mass = ref
    # a score is a sum of d products in fp32 (each addition within 2^-23 of the terms: the tensor cores may
    # truncate), then three factors; a probability's relative error is at most the score's on both sides of the quotient,
    # and 2^-21 for the hardware's exponentials and the sums
    ds = (d + 8) * 2.0**-23 * size
    dp = torch.expm1(2 * ds) + 2.0**-21
    assert bool(((lse.double() - l).abs() <= ds + 2.0**-22 * l.abs() + 2.0**-21)[l > -math.inf].all())
    assert bool((lse[l == -math.inf] == -math.inf).all())
    # weights: binary16, half a step is 2^-11 of the weight, or 2^-25 of the largest weight of their part of the rows (whose
    # codes reach 448, as every row's do); then the output's bfloat16, 2^-8 of it
    bar = (dp[..., None] + 2.0**-11) * mass + rows * 2.0**-25 * mass.amax(2, keepdim=True) * d
    bar = bar + 2.0**-8 * (o.abs() + bar) + 1e-38
    err = (out.double() - o).abs()
    assert bool((err <= bar).all()), float((err / bar).max())


class Cache:
    """Random sequences in a pool whose other rows hold NaNs."""

    def __init__(self, lens, kv, d, page, seed, stride=0, spread=1.5):
        g = np.random.default_rng(seed)
        n = len(lens)
        self.lens, self.page = np.asarray(lens, np.int32), page
        if page:
            pages = [-(-int(x) // page) for x in lens]
            perm = g.permutation(sum(pages) + 4).astype(np.int32)
            self.table = np.full((n, max(pages) + 2), -1, np.int32)
            o = 0
            for s, k in enumerate(pages):
                self.table[s, :k] = perm[o:o + k]
                o += k
            self.pool = (sum(pages) + 4) * page
        else:
            self.stride = stride or int(max(lens))
            self.table, self.pool = None, self.stride * n
        self.pl = new_planes(kv, self.pool, d)
        held = np.concatenate([self.rows_of(s, np.arange(int(x))) for s, x in enumerate(lens)]).astype(np.int64)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        at = torch.from_numpy(held).cuda()
        for name in ("k", "v"):
            mag = torch.exp(torch.empty(kv, len(held), 1, device="cuda").uniform_(-spread, spread, generator=gen))
            x = torch.randn(kv, len(held), d, device="cuda", generator=gen) * mag
            s = x.abs().amax(2) / 448.0
            self.pl[name][:, at] = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            self.pl[name + "_scale"][:, at] = s

    def rows_of(self, s, pos):
        if not self.page:
            return s * self.stride + pos
        return self.table[s, pos // self.page].astype(np.int64) * self.page + pos % self.page

    def problem(self, kvq, q, window=0, max_seq_len=None, scale=None, lens=None, table=None):
        table = self.table if table is None else table
        most = int(self.lens.max()) if max_seq_len is None else max_seq_len
        return kvq.make_kv8_problem(
            seq_len=dev(self.lens if lens is None else lens), q=q, sm_scale=1 / math.sqrt(q.shape[2]) if scale is None else scale,
            max_seq_len=most, cache=self.pl, block_table=None if table is None else dev(table), page_size=self.page,
            seq_stride_rows=0 if self.page else self.stride, window=window)


def queries(n, H, d, seed, size=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(n, H, d, device="cuda", generator=gen) * size).bfloat16()


def decode(kvq, p, st=None, want_lse=True):
    out = torch.full((p.n_seq, p.n_qh, p.cache.head_dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.n_seq, p.n_qh), float("nan"), device="cuda") if want_lse else None
    kvq.kvq_kv8_decode(p, out, lse, scratch(kvq.kvq_kv8_decode_workspace(p)), st)
    torch.cuda.synchronize()
    return out, lse


CASES = [
    # lens, kv heads, group, page, window
    ([1], 1, 1, 0, 0), ([2, 0, 1], 2, 4, 16, 0), ([15, 16, 17, 31, 33], 1, 8, 16, 0), ([127, 128, 129, 130], 2, 7, 64, 0),
    ([300, 5, 0, 1000], 3, 9, 40, 0), ([4097], 1, 16, 64, 0), ([700, 650], 2, 17, 8, 0), ([2048, 100], 1, 40, 100, 0),
    ([513, 512], 8, 3, 0, 0), ([9000], 2, 4, 1, 0), ([1000, 64, 63, 65], 2, 5, 64, 64), ([5000, 3], 1, 12, 48, 1),
    ([777, 2000, 31], 4, 2, 7, 1500), ([40000], 1, 8, 128, 0), ([20000, 1, 12345, 0, 777], 2, 8, 64, 9999),
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,kv,group,page,window", CASES)
def test_decode(kvq, d, lens, kv, group, page, window):
    c = Cache(lens, kv, d, page, seed=sum(lens) + d)
    q = queries(len(lens), kv * group, d, 5 + d)
    st = i32(1)
    p = c.problem(kvq, q, window)
    out, lse = decode(kvq, p, st)
    assert st.item() == 0
    ref = decode_ref(c.pl, q, lens, c.rows_of, window, 1 / math.sqrt(d))
    check_decode(out, lse, ref, d, min(4096, max(lens)))
    again, lse2 = decode(kvq, p)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)      # the same bits


@pytest.mark.parametrize("n,kv,most,d,page", [(3, 8, 1000, 128, 16), (9, 8, 700, 64, 24), (16, 8, 1020, 128, 64), (30, 8, 512, 256, 16),
                                              (60, 7, 150, 64, 0), (2, 1, 4000, 128, 16), (50, 8, 130, 128, 32), (100, 8, 3000, 64, 16)])
def test_decode_batches_of_short_sequences(kvq, n, kv, most, d, page):
    """Units of one to a few places: clusters of every size, and more units than CTAs."""
    g = np.random.default_rng(n + most)
    lens = g.integers(0, most + 1, n)
    lens[0], lens[-1] = most, 0
    c = Cache(lens, kv, d, page, n + d)
    q = queries(n, 3 * kv, d, n)
    out, lse = decode(kvq, c.problem(kvq, q))
    check_decode(out, lse, decode_ref(c.pl, q, lens, c.rows_of, 0, 1 / math.sqrt(d)), d, most)


@pytest.mark.parametrize("lens,page,window", [([700, 90, 1300], 16, 300), ([700, 90, 1300], 20, 300), ([30000, 5], 64, 5000), ([5000, 4100], 48, 1)])
def test_decode_window_over_freed_pages(kvq, lens, page, window):
    """Pages that lie ahead of the window as a whole may be gone; nothing is flagged."""
    c = Cache(lens, 2, 128, page, window)
    q = queries(len(lens), 6, 128, page)
    table = c.table.copy()
    for s, L in enumerate(lens):
        table[s, :max(0, L - window) // page] = -1
    st = i32(1)
    out, lse = decode(kvq, c.problem(kvq, q, window, table=table), st)
    assert st.item() == 0
    check_decode(out, lse, decode_ref(c.pl, q, lens, c.rows_of, window, 1 / math.sqrt(128)), 128, max(lens))


@pytest.mark.parametrize("most", [2000, 100000, 1 << 30])
def test_decode_generous_bound(kvq, most):
    """A bound far above every length: the outcome is that of a close one, up to the parts' order."""
    lens = [1500, 0, 3, 700]
    c = Cache(lens, 2, 64, 16, 5)
    q = queries(4, 10, 64, 6)
    out, lse = decode(kvq, c.problem(kvq, q, max_seq_len=most))
    check_decode(out, lse, decode_ref(c.pl, q, lens, c.rows_of, 0, 1 / 8), 64, 1500)


@pytest.mark.parametrize("d,heads,L", [(64, 4096, 100), (128, 1000, 700), (256, 333, 50), (64, 24, 5000)])
def test_decode_many_heads_of_one(kvq, d, heads, L):
    """One KV head for all query heads: more blocks of heads than CTAs."""
    lens = [L, L // 2]
    c = Cache(lens, 1, d, 16, heads)
    q = queries(2, heads, d, L)
    out, lse = decode(kvq, c.problem(kvq, q))
    check_decode(out, lse, decode_ref(c.pl, q, lens, c.rows_of, 0, 1 / math.sqrt(d)), d, L)


def test_decode_many_sequences(kvq):
    g = np.random.default_rng(0)
    lens = g.integers(0, 90, 1500)
    c = Cache(lens, 2, 64, 16, 1)
    q = queries(1500, 8, 64, 2)
    out, lse = decode(kvq, c.problem(kvq, q))
    check_decode(out, lse, decode_ref(c.pl, q, lens, c.rows_of, 0, 1 / 8), 64, 90)


@pytest.mark.parametrize("d,page", [(128, 16), (64, 24), (256, 0)])
def test_decode_lengths_are_clamped(kvq, d, page):
    c = Cache([500, 400, 300], 2, d, page, 3, stride=600)
    q = queries(3, 8, d, 4)
    out, lse = decode(kvq, c.problem(kvq, q, max_seq_len=350, lens=np.array([500, 2**31 - 1, -5], np.int32)))
    check_decode(out, lse, decode_ref(c.pl, q, [350, 350, 0], c.rows_of, 0, 1 / math.sqrt(d)), d, 350)
    out, lse = decode(kvq, c.problem(kvq, q, max_seq_len=0))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_decode_strided_queries_without_lse(kvq):
    c = Cache([100, 1700], 2, 128, 32, 6)
    fused = queries(2, 12, 128, 7)
    q = fused[:, 2:10]                                       # the heads of a fused projection's output
    out, _ = decode(kvq, c.problem(kvq, q), want_lse=False)
    ref = decode_ref(c.pl, q, [100, 1700], c.rows_of, 0, 1 / math.sqrt(128))
    plain, _ = decode(kvq, c.problem(kvq, q.contiguous()))
    assert torch.equal(out, plain)
    check_decode(out, ref[1].float(), ref, 128, 1700)


@pytest.mark.parametrize("lens,page", [([200, 333], 16), ([200, 333], 12), ([9000, 7333], 16), ([9000, 7333], 20)])
def test_decode_bad_pages(kvq, lens, page):
    c = Cache(lens, 2, 128, page, 8)
    q = queries(2, 8, 128, 9)
    table = c.table.copy()
    table[0, 3], table[1, 0], table[1, -4] = -1, c.pool // page, 2**31 - 1
    st = i32(1)
    out, lse = decode(kvq, c.problem(kvq, q, table=table), st)
    assert st.item() == BAD_PAGE
    bad = {(0, 3), (1, 0), (1, table.shape[1] - 4)}
    rows_of = lambda s, pos: np.array([-1 if (s, int(t) // page) in bad else int(c.rows_of(s, t)) for t in pos], np.int64)
    check_decode(out, lse, decode_ref(c.pl, q, lens, rows_of, 0, 1 / math.sqrt(128)), 128, max(lens))
    # a table too short for the lengths, and one without any page
    out, lse = decode(kvq, c.problem(kvq, q, table=np.ascontiguousarray(c.table[:, :5])), st)
    check_decode(out, lse, decode_ref(c.pl, q, [5 * page] * 2, c.rows_of, 0, 1 / math.sqrt(128)), 128, 5 * page)
    out, lse = decode(kvq, c.problem(kvq, q, table=np.full_like(c.table, -1)), st)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_decode_ranges(kvq):
    """Scales and queries near the ends of their ranges, zero rows, one row that outweighs all others."""
    L, d = 900, 128
    for case, (ks, vs, qs, scale) in enumerate([(1e-30, 1e30, 1e28, 0.09), (1e25, 1e-30, 1e-27, 0.09), (1.0, 1e-36, 1.0, 0.09),
                                                (1.0, 1.0, 1.0, 0.0), (1.0, 1.0, 1.0, -0.2), (4.0, 1.0, 4.0, 0.3)]):
        c = Cache([L, 17], 2, d, 64, 20 + case)
        c.pl["k_scale"] *= ks
        c.pl["v_scale"] *= vs
        q = queries(2, 12, d, 30 + case, qs)
        rows = torch.from_numpy(c.rows_of(0, np.arange(0, L, 7))).cuda()
        c.pl["v_scale"][0, rows] = 0.0
        c.pl["v"][0, rows] = 0
        c.pl["k_scale"][1, rows] = 0.0
        c.pl["k"][1, rows] = 0
        out, lse = decode(kvq, c.problem(kvq, q, scale=scale))
        check_decode(out, lse, decode_ref(c.pl, q, [L, 17], c.rows_of, 0, scale), d, L)
    # every V row of a head zero
    c = Cache([333], 2, d, 64, 40)
    c.pl["v_scale"][1] = 0.0
    c.pl["v"][1] = 0
    q = queries(1, 8, d, 41)
    out, lse = decode(kvq, c.problem(kvq, q))
    check_decode(out, lse, decode_ref({**c.pl, "v": c.pl["v"], "v_scale": torch.nan_to_num(c.pl["v_scale"])}, q, [333], c.rows_of, 0,
                                      1 / math.sqrt(d)), d, 333)
    assert bool((out[0, 4:] == 0).all())


@pytest.mark.parametrize("lens", [[900, 17], [20000, 300]])
@pytest.mark.parametrize("ks,qs,scale", [(1e34, 1e-34, 0.09), (1e-34, 1e34, 0.09), (1e36, 1e-37, 0.5), (1e36, 1e-39, 50.0), (1e-37, 1e37, 0.09),
                                         (1e30, 1e-19, 1e-12), (1e-30, 3e37, 1e-9), (1e-36, 1e19, 1e16), (1.0, 1e-36, 1e19)])
def test_decode_score_ranges(kvq, lens, ks, qs, scale):
    """Scores of ordinary size whose factors are near the ends of fp32, queries that are subnormal among them."""
    d = 128
    c = Cache(lens, 2, d, 64, 90, spread=0.5)
    c.pl["k_scale"] *= ks
    q = queries(2, 12, d, 91, qs)
    out, lse = decode(kvq, c.problem(kvq, q, scale=scale))
    check_decode(out, lse, decode_ref(c.pl, q, lens, c.rows_of, 0, scale), d, 32)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[900, 17], [40000, 300], [3, 1]])
@pytest.mark.parametrize("vs", [1e37, 1e-36])
def test_decode_value_ranges(kvq, d, lens, vs):
    """V rows near the ends of fp32: sums over the rows pass its largest, the weighted means do not."""
    c = Cache(lens, 2, d, 64, 95, spread=0.5)
    c.pl["v_scale"] *= vs
    q = queries(2, 12, d, 96)
    out, lse = decode(kvq, c.problem(kvq, q))
    assert bool(out.isfinite().all())
    check_decode(out, lse, decode_ref(c.pl, q, lens, c.rows_of, 0, 1 / math.sqrt(d)), d, 32)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1, 3], [900, 17], [40000, 300]])
def test_decode_equal_scores_of_any_size(kvq, d, lens):
    """Rows of one K, whose scores are equal to the last bit: the output is the mean of V however large the scores are."""
    c = Cache(lens, 2, d, 64, 130, spread=2.0)
    rows = torch.from_numpy(np.concatenate([c.rows_of(s, np.arange(L)) for s, L in enumerate(lens)])).cuda()
    for name in ("k", "k_scale"):
        c.pl[name][:, rows] = c.pl[name][:, rows[:1]]
    for size in (1.0, 1e3, 1e5, 1e7, 1e10, 1e20, 1e30, 1e36):
        q = queries(2, 6, d, 131, size)
        out, lse = decode(kvq, c.problem(kvq, q))
        o, l, _, mass = decode_ref(c.pl, torch.zeros_like(q), lens, c.rows_of, 0, 1.0)
        # weights: 2^-11 of each, or 2^-25 of the largest; 2^-20 for exponentials, sums and scales; the output's bfloat16
        bar = (2.0**-11 + 2.0**-20) * mass + 4096 * 2.0**-25 * mass.amax(2, keepdim=True)
        bar = bar + 2.0**-8 * (o.abs() + bar)
        assert bool(((out.double() - o).abs() <= bar).all()), (size, float(((out.double() - o).abs() / bar).max()))
        x = (q.double().view(2, 2, 3, d) * values(c.pl, "k", rows[:1]).view(1, 2, 1, d)).sum(3).view(2, 6) / math.sqrt(d)
        n = torch.tensor(lens, dtype=torch.float64, device="cuda").log()[:, None]
        size_of = (q.double().abs().view(2, 2, 3, d) * values(c.pl, "k", rows[:1]).abs().view(1, 2, 1, d)).sum(3).view(2, 6) / math.sqrt(d)
        assert bool(((lse.double() - x - n).abs() <= (d + 8) * 2.0**-23 * size_of + 2.0**-22 * (x + n).abs() + 2.0**-20).all()), size


@pytest.mark.parametrize("d,lens", [(64, [900, 17]), (128, [900, 17]), (128, [20000, 300]), (256, [5000, 1])])
def test_decode_heads_of_every_size(kvq, d, lens):
    """Heads of one KV head whose queries are 2^250 apart, one of them zero."""
    c = Cache(lens, 2, d, 64, 110, spread=0.5)
    size = torch.tensor([1.0, 1e-39, 1e20, 0.0, 1e37, 1e-30, 1.0], device="cuda").repeat(2)
    q = (queries(2, 14, d, 111).float() * size[:, None]).bfloat16()
    out, lse = decode(kvq, c.problem(kvq, q))
    check_decode(out, lse, decode_ref(c.pl, q, lens, c.rows_of, 0, 1 / math.sqrt(d)), d, 32)
    one = size == 1.0
    q[:, ~one] = 0.0
    out2, lse2 = decode(kvq, c.problem(kvq, q))
    assert torch.equal(out[:, one], out2[:, one]) and torch.equal(lse[:, one], lse2[:, one])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,page", [([900, 0, 17], 16), ([20000, 300, 1], 64), ([3000, 2], 20)])
def test_decode_extremes_of_many_heads(kvq, d, lens, page):
    """Twelve heads a KV head (two blocks of eight): queries of every size, infinities and NaNs, V rows near fp32's largest."""
    c = Cache(lens, 2, d, page, 140, spread=0.5)
    c.pl["v_scale"] *= 1e36
    n = len(lens)
    size = torch.tensor([1.0, 1e-39, 1e20, 0.0, 1.0, 1e37, 1e-30, 1.0, 1e-38, 1.0, 1e37, 1.0], device="cuda").repeat(2)
    q = (queries(n, 24, d, 141).float() * size[:, None]).bfloat16()
    clean, lse0 = decode(kvq, c.problem(kvq, q))
    assert bool(clean.isfinite().all())
    check_decode(clean, lse0, decode_ref(c.pl, q, lens, c.rows_of, 0, 1 / math.sqrt(d)), d, 32)
    bad = q.clone()
    bad[:, 4, 3], bad[:, 11, 0], bad[:, 21, d - 1] = math.inf, -math.inf, float("nan")
    hit = torch.zeros(24, dtype=torch.bool, device="cuda")
    hit[[4, 11, 21]] = True
    out, lse = decode(kvq, c.problem(kvq, bad))
    sees = dev(np.asarray(lens) > 0)
    assert bool(out[sees][:, hit].isnan().all()) and bool(lse[sees][:, hit].isnan().all())
    assert bool((out[~sees] == 0).all()) and bool((lse[~sees] == -math.inf).all())
    assert torch.equal(out[:, ~hit], clean[:, ~hit]) and torch.equal(lse[:, ~hit], lse0[:, ~hit])


def test_decode_many_small_weights(kvq):
    """One row takes most of the softmax, and 50000 rows far below it hold the rest together."""
    L, d = 50001, 64
    c = Cache([L], 1, d, 64, 50, spread=0.0)
    c.pl["k"].zero_()
    c.pl["k_scale"].fill_(1.0)
    c.pl["v"].fill_(0x7E)                                    # 448
    c.pl["v_scale"].fill_(1.0 / 448)
    at = int(c.rows_of(0, np.array([12345]))[0])
    q = torch.zeros(1, 4, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    for code, gap in ((0x58, 16.0), (0x5A, 20.0), (0x5C, 24.0)):         # e^-16 .. e^-24 each: 0.5 % to 2e-6 in all
        c.pl["k"][0, at, 0] = code
        c.pl["v"][0, at] = 0xFE                              # -448 where all the others have 448
        assert float(c.pl["k"].view(torch.float8_e4m3fn)[0, at, 0].float()) == gap
        out, lse = decode(kvq, c.problem(kvq, q, scale=1.0))
        check_decode(out, lse, decode_ref(c.pl, q, [L], c.rows_of, 0, 1.0), d, 4096)


@pytest.mark.parametrize("code,gap", [(0x54, 12.0), (0x56, 14.0), (0x58, 16.0)])
def test_decode_small_weights_of_a_part(kvq, code, gap):
    """A row of V = 0 takes most of the softmax, so that the output is what the rows far below it hold together; parts of many
    rows (64 sequences over the same pages: a warp has about 900 rows of a unit)."""
    n, kv, L, d, page = 64, 8, 4096, 64, 64
    pl = new_planes(kv, L, d)
    pl["k"].zero_()
    pl["v"].fill_(0x7E)                                      # 448
    pl["k_scale"].fill_(1.0)
    pl["v_scale"].fill_(1.0 / 448)
    at = 1234
    pl["k"][:, at, 0] = code
    pl["v"][:, at] = 0
    q = torch.zeros(n, kv, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    table = torch.arange(L // page, dtype=torch.int32, device="cuda").repeat(n, 1)
    p = kvq.make_kv8_problem(seq_len=i32(n, fill=L), q=q, sm_scale=1.0, max_seq_len=L, cache=pl, block_table=table, page_size=page)
    out, lse = decode(kvq, p)
    total = 1.0 + (L - 1) * math.exp(-gap)
    want = (L - 1) * math.exp(-gap) / total
    # the rows of the heavy row's part: a warp's quarter of the unit at most.  Their weights are within 2^-25 of the heavy one
    # (half a step of binary16's subnormals) or 2^-11 of themselves; scores, in log2 at most 24, are rounded three times (the
    # scale, two products), on both sides of the quotient: 6 24 2^-24 ln 2 < 2^-17, with the exponentials and sums; then the
    # output's bfloat16
    part = L // 4
    bar = want * (2.0**-11 + 2.0**-17) + part * 2.0**-25 / total
    bar += 2.0**-8 * (want + bar)
    # (without the small weights of the heavy row's part: some head's has three quarters of that at least, as a cut falls every 27
    # places of 128 rows and a unit has 32)
    assert 0.75 * part * math.exp(-gap) / total > bar
    assert float((out.double() - want).abs().max()) <= bar
    # log2 of the sum is added to the score and the whole scaled by ln 2: five roundings of 2^-24 and the constant's 2^-25; the
    # sum itself within 2^-20
    assert float((lse.double() - gap - math.log(total)).abs().max()) <= 5.5 * 2.0**-24 * (gap + 1) + 2.0**-20


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,kv,group,page,window", [([300, 5, 0, 1000], 3, 9, 40, 0), ([4097], 1, 16, 64, 0), ([9000], 2, 4, 1, 0),
                                                       ([777, 2000, 31], 4, 2, 7, 1500), ([40000], 1, 8, 128, 0), ([4000] * 70, 4, 3, 64, 0)])
def test_decode_rounding_of_weights(kvq, d, lens, kv, group, page, window):
    """Outputs against what the roundings allow and no more: a weight's 2^-11, or 2^-25 of the largest of its part."""
    c = Cache(lens, kv, d, page, seed=d)
    q = queries(len(lens), kv * group, d, 120 + d)
    out, _ = decode(kvq, c.problem(kvq, q, window))
    o, _, size, mass = decode_ref(c.pl, q, lens, c.rows_of, window, 1 / math.sqrt(d))
    # As in check_decode, but for the small weights: each is within 2^-25 of the largest of its part, and that one's row, whose
    # largest code is 448, has its share in `mass`, so that the part's rows lose 2^-25 of the largest over the dims each
    dp = torch.expm1(2 * (d + 8) * 2.0**-23 * size) + 2.0**-21
    bar = (dp[..., None] + 2.0**-11) * mass + min(4096, max(lens)) * 2.0**-25 * mass.amax(2, keepdim=True)
    bar = bar + 2.0**-8 * (o.abs() + bar) + 1e-38
    assert bool(((out.double() - o).abs() <= bar).all()), float(((out.double() - o).abs() / bar).max())


@pytest.mark.parametrize("lens", [[700, 20], [9000, 5001]])
def test_decode_nan_queries_stay_in_their_head(kvq, lens):
    c = Cache(lens, 2, 128, 64, 60)
    q = queries(2, 16, 128, 61)
    clean, lse0 = decode(kvq, c.problem(kvq, q))
    bad = q.clone()
    bad[0, 3, 5], bad[1, 8, 0], bad[1, 15, 127] = float("nan"), math.inf, -math.inf
    out, lse = decode(kvq, c.problem(kvq, bad))
    hit = torch.zeros(2, 16, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[1, 8] = hit[1, 15] = True
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], lse0[~hit])


@pytest.mark.parametrize("lens,kv,page", [([900, 300], 2, 16), ([40000, 0, 1], 2, 64), ([9000, 5001, 77], 1, 20)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_heads_do_not_touch_each_other(kvq, d, lens, kv, page):
    """A head's bits are the same whatever the others hold: zeros, large queries, a NaN."""
    c = Cache(lens, kv, d, page, 100 + d)
    n, H = len(lens), 6 * kv
    q = queries(n, H, d, 101)
    clean, lse0 = decode(kvq, c.problem(kvq, q))
    keep = torch.ones(H, dtype=torch.bool, device="cuda")
    keep[1] = keep[H - 1] = False
    for x in (0.0, 30.0, float("nan")):
        other = q.clone()
        other[:, ~keep] = queries(n, 2, d, 102) * x
        out, lse = decode(kvq, c.problem(kvq, other))
        assert torch.equal(out[:, keep], clean[:, keep]) and torch.equal(lse[:, keep], lse0[:, keep]), x


@pytest.mark.parametrize("lens,kv,page,window", [([1, 0, 2], 2, 16, 0), ([1, 1], 3, 0, 0), ([300, 0, 200], 2, 16, 1), ([700, 90], 1, 20, 3),
                                                 ([1] * 700, 2, 16, 0), ([40000, 0, 1], 2, 64, 0)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_infinite_queries(kvq, d, lens, kv, page, window):
    """A head that holds an infinity gets NaN also where every visible row's score is -inf (one element's codes of one
    sign), on a cluster and on the line; its neighbours keep their bits."""
    c = Cache(lens, kv, d, page, 80 + d)
    c.pl["k"][:, :, 5] = 0x38                                # 1.0, in every row
    n, H = len(lens), 6 * kv
    q = queries(n, H, d, 81)
    clean, lse0 = decode(kvq, c.problem(kvq, q, window))
    bad, hit = q.clone(), torch.zeros(n, H, dtype=torch.bool, device="cuda")
    for s in {0, n // 2, n - 1}:
        bad[s, 1, 5], bad[s, H - 1, 5] = -math.inf, math.inf
        hit[s, 1] = hit[s, H - 1] = True
    out, lse = decode(kvq, c.problem(kvq, bad, window))
    sees = dev(np.asarray(lens) > 0)[:, None].expand(n, H)
    assert bool(out[hit & sees].isnan().all()) and bool(lse[hit & sees].isnan().all())
    assert bool((out[~sees] == 0).all()) and bool((lse[~sees] == -math.inf).all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], lse0[~hit])


def test_decode_far_rows(kvq):
    """A pool whose rows lie behind 2^32 bytes."""
    d, page = 256, 64
    n_pages = (1 << 32) // (page * d) + 40
    pl = dict(k=torch.empty(1, n_pages * page, d, dtype=torch.uint8, device="cuda"), k_scale=torch.empty(1, n_pages * page, device="cuda"),
              v=torch.empty(1, n_pages * page, d, dtype=torch.uint8, device="cuda"), v_scale=torch.empty(1, n_pages * page, device="cuda"))
    L = 250
    table = np.array([[n_pages - 1, 3, n_pages - 17, n_pages - 2]], np.int32)
    pos = np.arange(L)
    slot = (table[0][pos // page].astype(np.int64) * page + pos % page)
    x = torch.randn(2, L, 1, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    kvq.kvq_append_kv8(x[0], x[1], dev(slot.astype(np.int32)), pl)
    q = queries(1, 8, d, 2)
    p = kvq.make_kv8_problem(seq_len=i32(1, fill=L), q=q, sm_scale=1 / 16, max_seq_len=L, cache=pl, block_table=dev(table), page_size=page)
    out, lse = decode(kvq, p)
    check_decode(out, lse, decode_ref(pl, q, [L], lambda s, t: slot[t], 0, 1 / 16), d, L)


@pytest.mark.parametrize("long", [3000, 20000])
def test_decode_streams_and_graph(kvq, long):
    """Two problems on two streams at once, and a replayed graph after the lengths have changed."""
    cs = [Cache([long, 100], 2, 128, 64, 70), Cache([long - 500, 1, 9], 4, 64, 16, 71)]
    qs = [queries(2, 16, 128, 72), queries(3, 4, 64, 73)]
    ps = [c.problem(kvq, q) for c, q in zip(cs, qs)]
    want = [decode(kvq, p) for p in ps]
    ws = [scratch(kvq.kvq_kv8_decode_workspace(p)) for p in ps]
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, w, (o, l), s in zip(ps, ws, outs, streams):
            with torch.cuda.stream(s):
                kvq.kvq_kv8_decode(p, o, l, w)
    torch.cuda.synchronize()
    for (o, l), (o2, l2) in zip(outs, want):
        assert torch.equal(o, o2) and torch.equal(l, l2)
    p, w, (o, l) = ps[0], ws[0], outs[0]
    g = graphed(lambda: kvq.kvq_kv8_decode(p, o, l, w))
    p._keep[0].copy_(torch.tensor([1234, 0], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check_decode(o, l, decode_ref(cs[0].pl, qs[0], [1234, 0], cs[0].rows_of, 0, 1 / math.sqrt(128)), 128, 1234)


# --- the selection -------------------------------------------------------------------------------

def beam_ref(x, score, fin, n_out, eos, pad):
    """x [R, B, V] fp32 as numpy; -> score, token, parent, finished, whether a beam was refused."""
    R, B, V = x.shape
    out = np.full((R, n_out), -np.inf), np.full((R, n_out), -1), np.full((R, n_out), -1), np.zeros((R, n_out), int)
    refused = False
    for r in range(R):
        val, beam, logit, token, done = [], [], [], [], []
        for b in range(B):
            s = score[r, b]
            if not s < np.inf:
                refused = True
                continue
            if s == -np.inf:
                continue
            if fin is not None and fin[r, b]:
                val.append(np.array([np.float64(s)])), logit.append(np.zeros(1)), token.append(np.zeros(1, int))
                beam.append(np.array([b])), done.append(np.ones(1, int))
                continue
            row = x[r, b].astype(np.float64)
            if not (row < np.inf).all():
                refused = True
                continue
            t = np.flatnonzero(row > -np.inf)
            if len(t) == 0:
                continue
            # the differences first: m + log(sum) of logits near 3e38 rounds to m even in 64 bits, and a constant row's
            # values, score - log(vocab), would come out as 0
            d = row[t] - row[t].max()
            val.append(d + (np.float64(s) - math.log(np.exp(d).sum()))), logit.append(row[t] + 0.0), token.append(t)
            beam.append(np.full(len(t), b)), done.append(np.zeros(len(t), int))
        if not val:
            continue
        val, beam, logit, token, done = (np.concatenate(a) for a in (val, beam, logit, token, done))
        order = np.lexsort((token, -logit, beam, -val))[:n_out]
        k = len(order)
        out[0][r, :k] = val[order]
        out[1][r, :k] = np.where(done[order] == 1, pad, token[order])
        out[2][r, :k] = r * B + beam[order]
        out[3][r, :k] = (done[order] == 1) | ((token[order] == eos) & (eos >= 0)) | ((done[order] == 1) & (pad == eos))
    return (*out, refused)


def select(kvq, x, score, fin, n_out, eos=2, pad=0, ld=None, status=None):
    R, B, V = x.shape
    if ld:
        wide = torch.full((R, B, ld), float("nan"), dtype=x.dtype, device="cuda")
        wide[..., :V] = x
        x = wide[..., :V]
    out = [torch.full((R, n_out), float("nan"), device="cuda"), *(i32(R, n_out, fill=-9) for _ in range(3))]
    p = kvq.make_beam_problem(logits=x, score=score, finished=fin, out_score=out[0], out_token=out[1], out_parent=out[2],
                              out_finished=out[3], eos=eos, pad=pad)
    st = i32(1)
    kvq.kvq_beam_select(p, scratch(kvq.kvq_beam_select_workspace(p)), st)
    torch.cuda.synchronize()
    return out, st.item()


def check_select(kvq, x, score, fin=None, n_out=4, eos=2, pad=0, ld=None):
    x, score = dev(x) if isinstance(x, np.ndarray) else x, dev(score)
    got, st = select(kvq, x, score, None if fin is None else dev(fin.astype(np.int32)), n_out, eos, pad, ld)
    want = beam_ref(host(x.float()), host(score), fin, n_out, eos, pad)
    for name, g, w in zip(("token", "parent", "finished"), got[1:], want[1:4]):
        assert np.array_equal(host(g), w), name
    s, w = host(got[0]).astype(np.float64), want[0]
    assert np.array_equal(s == -np.inf, w == -np.inf)
    fine = w > -np.inf
    # the exponentials are fp32 (2^-22 each), the argument's factor within 2^-25 of log2 e over distances up to 100
    # that count, and the value is rounded to fp32
    assert np.all(np.abs(s[fine] - w[fine]) <= 2.0**-24 * np.abs(w[fine]) + 2.0**-21 + 100 * 2.0**-25)
    assert st == (BAD_VALUE if want[4] else 0)


@pytest.mark.parametrize("R,B,V,K,bf16,ld", [
    (1, 1, 1, 1, False, None), (1, 4, 7, 4, False, None), (2, 3, 1000, 5, True, 1001), (1, 4, 32000, 8, False, None),
    (3, 8, 50257, 16, True, None), (2, 5, 2049, 128, False, 2052), (1, 64, 513, 64, True, 520), (40, 2, 300, 4, True, None),
    (2, 64, 40000, 128, True, None), (70, 8, 9001, 16, False, None), (1, 2, 200003, 3, True, 200008),
])
def test_select(kvq, R, B, V, K, bf16, ld):
    g = np.random.default_rng(R + B + V)
    x = dev((g.standard_normal((R, B, V)) * 3).astype(np.float32))
    x = x.bfloat16() if bf16 else x
    score = (-10 * g.random((R, B))).astype(np.float32)
    check_select(kvq, x, score, None, K, ld=ld)
    fin = g.random((R, B)) < 0.3
    score[g.random((R, B)) < 0.2] = -np.inf
    drop = dev(g.random((R, B, V)) < 0.6)
    check_select(kvq, x.masked_fill(drop, -math.inf), score, fin, K, eos=min(2, V - 1), pad=-3, ld=ld)


@pytest.mark.parametrize("V", [100, 5000, 70000])
@pytest.mark.parametrize("K", [1, 6, 64])
@pytest.mark.parametrize("R", [1, 30])
def test_select_ties(kvq, V, K, R):
    """Equal logits go to the lowest token, equal values to the lowest beam: constant rows, few levels, zeros of both signs."""
    g = np.random.default_rng(V + K)
    B = 4
    zero = np.zeros((R, B), np.float32)
    check_select(kvq, np.full((R, B, V), 1.5, np.float32), zero, None, K, eos=-1)
    x = np.repeat(g.integers(0, 3, (R, 1, V)), B, 1).astype(np.float32)
    check_select(kvq, x, zero, None, K)
    x = np.where(g.random((R, B, V)) < 0.5, np.float32(-0.0), np.float32(0.0))
    check_select(kvq, x, zero, np.arange(B)[None, :].repeat(R, 0) == 2, K)
    ramp = np.broadcast_to(np.arange(V, dtype=np.float32) / V, (R, B, V)).copy()
    check_select(kvq, ramp, zero, None, K)
    check_select(kvq, ramp[..., ::-1].copy(), zero, None, K)


@pytest.mark.parametrize("V,ld", [(101, None), (4099, None), (50257, None), (50257, 50264), (20000, 20003), (7, None), (33001, 33006)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("R", [3, 60])
def test_select_equal_beams(kvq, R, V, ld, bf16):
    """Beams of equal scores and logits, their rows beginning at any place: the lowest beam's candidate stands first."""
    g = np.random.default_rng(V)
    B = 8
    x = dev(np.repeat((g.standard_normal((R, 1, V)) * 3).astype(np.float32), B, 1))
    x = x.bfloat16() if bf16 else x
    score = np.repeat(-7 * g.random((R, 1)), B, 1).astype(np.float32)
    check_select(kvq, x, score, None, min(V, 20 if R == 3 else 16), ld=ld)


@pytest.mark.parametrize("bf16,ld,K", [(False, 20000, 16), (False, 20001, 7), (True, 20000, 3), (True, 20003, 16), (True, 20008, 13)])
def test_select_long_rows(kvq, bf16, ld, K):
    """Many rows of several pieces a warp: random, sorted both ways, few levels, empty stretches, and values of no use."""
    g = np.random.default_rng(ld + K)
    B, V = 5, 20000
    kinds = [(g.standard_normal((B, V)) * 3) for _ in range(60)]
    kinds[1:13:3] = [np.sort(k, 1) for k in kinds[1:13:3]]
    kinds[2:14:3] = [np.sort(k, 1)[:, ::-1] for k in kinds[2:14:3]]
    kinds[15] = np.zeros((B, V))
    kinds[16] = g.integers(0, 3, (B, V))
    kinds[17] = np.where(np.arange(V) < 19000, -np.inf, kinds[17])
    kinds[18] = np.where(np.arange(V) > 50, -np.inf, kinds[18])
    kinds[19] = np.where(g.random((B, V)) < 0.9997, -np.inf, kinds[19])     # (fewer than K, some of them)
    kinds[20] = np.full((B, V), -np.inf)
    kinds[21][2, 19999] = np.nan
    kinds[22][1, 4100] = np.inf
    kinds[23] = np.where(g.random((B, V)) < 0.9, -1e9, kinds[23])           # a mask's filler
    kinds[24] = np.where(np.arange(V) // 4096 % 2 == 0, -3.0e38, kinds[24])
    kinds[25] = kinds[25] + np.arange(V) * 2.0                              # from below 2^13 to above it
    kinds[26] = np.cumsum(np.ones((B, V)), 1) * 0.01
    x = dev(np.stack(kinds).astype(np.float32))
    x = x.bfloat16() if bf16 else x
    score = (-10 * g.random((60, B))).astype(np.float32)
    fin = (g.random((60, B)) < 0.2).astype(int)
    score[g.random((60, B)) < 0.1] = -np.inf
    check_select(kvq, x, score, fin, K, ld=ld)


def test_select_edges(kvq):
    g = np.random.default_rng(4)
    R, B, V = 6, 4, 3000
    x = (g.standard_normal((R, B, V)) * 2).astype(np.float32)
    x[0, 1, 77] = np.nan
    x[0, 2, 5] = np.inf
    x[1] = -np.inf                                           # nothing left at all
    x[2, :, 3:] = -np.inf                                    # fewer candidates than places
    x[3, 0] = 1e35 * x[3, 0]                                 # far above the others, finite
    x[3, 1] = np.float32(3.0e38)
    x[3, 2] *= 1e-30
    x[4, 0, 0] = 200.0                                       # all the probability on one token
    score = (-10 * g.random((R, B))).astype(np.float32)
    score[5] = [np.nan, np.inf, -np.inf, -1.0]
    fin = np.zeros((R, B), int)
    fin[0, 3] = 5
    fin[1, 2] = 1
    check_select(kvq, x, score, fin, 16)
    check_select(kvq, x[1:2], score[1:2], None, 4)
    # a NaN in a finished beam's row, or in a dead one's, is not read
    x, score, fin = x[:1].copy(), score[:1].copy(), np.array([[0, 1, 1, 0]])
    score[0, 0] = -np.inf
    x[0, 0] = np.nan
    check_select(kvq, x, score, fin, 3, eos=0, pad=0)


def test_select_far_apart(kvq):
    """Logits and scores whose plain sums or differences pass fp32's largest, while the values do not."""
    g = np.random.default_rng(6)
    R, B, V = 4, 3, 2500
    x = (g.standard_normal((R, B, V)) * 2).astype(np.float32)
    score = np.zeros((R, B), np.float32)
    x[0] += np.float32(3.0e38) * np.array([1, -1, 1], np.float32)[:, None]
    score[0] = -3.0e38, -2.9e38, -3.3e38
    x[1] = -3.0e38                                           # (further from the largest than fp32 reaches)
    x[1, :, :6] = np.array([3.0, 2.99, 2.98, 2.97, 2.96, 2.95], np.float32) * np.float32(1e38)
    score[1] = -1, -2, -3
    x[2, 0] *= 1e-30
    score[2] = -1000
    score[3] = 3.0e38, -3.0e38, 1e30
    check_select(kvq, x, score, None, 8, eos=-1)


@pytest.mark.parametrize("V", [3000, 40000])
@pytest.mark.parametrize("R", [1, 30])
def test_select_large_logits(kvq, V, R):
    """Rows around levels of any size and sign, a mask's filler among them: sums are of differences.  (A request a row: values
    of rows of different levels that would tie exactly differ by the exponentials' 2^-22.)"""
    g = np.random.default_rng(V)
    for levels in ([3e4, -3e4, 1e6, -1e6], [2e6, -2e6, 1e9, -1e9], [1e10, -1e10, 1e13, -1e13], [1e25, -1e25, 9e29, -3.4028235e38]):
        at = np.array(levels, np.float32).repeat(R)[:, None, None]
        x = np.broadcast_to(at, (4 * R, 1, V)).copy()         # nothing but the level
        check_select(kvq, x, np.zeros((4 * R, 1), np.float32), None, 6, eos=-1)
        far = np.abs(at) < 1e30
        step = np.maximum(np.spacing(np.where(far, np.abs(at), 1)), np.float32(0.125))
        x = np.where(far, at + step * g.integers(-9, 1, x.shape).astype(np.float32), at).astype(np.float32)
        check_select(kvq, x, (-5 * g.random((4 * R, 1))).astype(np.float32), None, 6, eos=-1)


@pytest.mark.parametrize("V", [4000, 128000])
@pytest.mark.parametrize("level", [0.0, 5.3, -300.7, 9000.0, 3e6])
def test_select_sum_of_a_far_tail(kvq, V, level):
    """One token above all others, which lie at one distance, so that their exponentials' errors add up."""
    for far in (0.7, 3.3, 5.01, 7.77, 9.7, 11.1, 12.3, 13.9):
        x = np.full((1, 1, V), np.float32(level - far), np.float32)
        x[0, 0, 77] = level
        (out, token, _, _), st = select(kvq, dev(x), dev(np.zeros((1, 1), np.float32)), None, 1, eos=-1)
        D = float(x[0, 0, 77]) - float(x[0, 0, 0])
        tail = (V - 1) * math.exp(-D)
        # A term: its argument in log2, and the rest of the factor log2 e, are rounded to 2^-24 of the distance each, twice more
        # where warps and chunks are brought to one maximum, whose exponentials are within 2^-22; the instruction's 2^-22 and
        # some additions within 2^-24 besides.  Then the value's fp32.
        bar = 2.0**-20 + tail / (1 + tail) * D * 2.0**-22 + 2.0**-24 * math.log1p(tail)
        assert st == 0 and token.item() == 77
        assert abs(out.item() + math.log1p(tail)) <= bar, far


@pytest.mark.parametrize("V", [1, 3000, 70000])
@pytest.mark.parametrize("bf16", [False, True])
def test_select_forced_tokens(kvq, V, bf16):
    """Beams with one token left: its value is the score, to the last bit, and equal ones come in the order of the beams."""
    g = np.random.default_rng(V)
    R, B = 40, 8
    x = torch.full((R, B, V), -math.inf, device="cuda")
    token = torch.from_numpy(g.integers(0, V, (R, B, 1))).cuda()
    level = torch.from_numpy((g.standard_normal((R, B, 1)) * np.exp(g.uniform(-5, 12, (R, B, 1)))).astype(np.float32)).cuda()
    x.scatter_(2, token, level)
    x = x.bfloat16() if bf16 else x
    score = (-20 * g.random((R, B))).astype(np.float32)
    score[:R // 2] = score[:R // 2, :1]
    (out, tok, parent, _), st = select(kvq, x, dev(score), None, B, eos=-1)
    order = np.argsort(-score, axis=1, kind="stable")
    assert st == 0 and np.array_equal(host(out), np.take_along_axis(score, order, 1))
    assert np.array_equal(host(parent), order + np.arange(R)[:, None] * B)
    assert np.array_equal(host(tok), np.take_along_axis(host(token)[..., 0], order, 1))


def test_select_beams_at_different_levels(kvq):
    """Constant rows at levels far apart, whose values tie exactly: beams in either order (their sums are of fp32
    exponentials), each beam's tokens from its lowest on."""
    for V in (3000, 40000):
        for levels in ([3e4, -3e4, 1e6, -1e6], [0.0, 1.5, -7.25, 1e13], [1e25, -1e25, 9e29, -3.4e38]):
            x = np.broadcast_to(np.array(levels, np.float32)[None, :, None], (1, 4, V)).copy()
            (out, token, parent, _), st = select(kvq, dev(x), dev(np.zeros((1, 4), np.float32)), None, 10, eos=-1)
            assert st == 0
            assert np.abs(host(out).astype(np.float64) + math.log(V)).max() <= 2.0**-22 + 2.0**-24 * math.log(V)
            token, parent = host(token)[0], host(parent)[0]
            for b in range(4):
                mine = token[parent == b]
                assert np.array_equal(mine, np.arange(len(mine)))
            assert sum((parent == b).sum() for b in range(4)) == 10


def test_select_in_place_and_graph(kvq):
    """A loop of steps in a graph whose scores and finished flags are the step's own outputs."""
    g = np.random.default_rng(5)
    R, B, V, steps = 3, 4, 700, 6
    x = (g.standard_normal((steps, R, B, V)) * 2).astype(np.float32)
    x[..., 2] += 4.0                                         # the end is often among the best
    score = np.zeros((R, B), np.float32)
    score[:, 1:] = -np.inf
    fin = np.zeros((R, B), int)
    logits, d_score, d_fin = dev(x[0]), dev(score), i32(R, B)
    token, parent = i32(R, B), i32(R, B)
    p = kvq.make_beam_problem(logits=logits, score=d_score, finished=d_fin, out_score=d_score, out_token=token, out_parent=parent,
                              out_finished=d_fin, eos=2, pad=1)
    ws = scratch(kvq.kvq_beam_select_workspace(p))
    graph = graphed(lambda: kvq.kvq_beam_select(p, ws))
    d_score.copy_(dev(score))
    d_fin.zero_()
    for k in range(steps):
        logits.copy_(dev(x[k]))
        graph.replay()
        torch.cuda.synchronize()
        want = beam_ref(x[k], score, fin, B, 2, 1)
        assert np.array_equal(host(token), want[1]) and np.array_equal(host(parent), want[2])
        assert np.array_equal(host(d_fin), want[3])
        score, fin = host(d_score), want[3]
        assert np.allclose(score, want[0], rtol=0, atol=1e-5)
    assert fin.any()


@pytest.mark.parametrize("R,B,V", [(1, 4, 900), (24, 8, 20000)])
def test_select_queued_steps_in_place(kvq, R, B, V):
    """Steps in place, one behind the other without a wait of the host, give the bits of steps one by one."""
    gen = torch.Generator(device="cuda").manual_seed(R)
    steps = 50
    x = torch.randn(steps, R, B, V, device="cuda", generator=gen).bfloat16()
    x[..., 2] += 3.0
    runs = []
    for one_by_one in (True, False, False):
        score, fin, token, parent = torch.zeros(R, B, device="cuda"), i32(R, B), i32(steps, R, B), i32(steps, R, B)
        ps = [kvq.make_beam_problem(logits=x[k], score=score, finished=fin, out_score=score, out_token=token[k], out_parent=parent[k],
                                    out_finished=fin, eos=2, pad=1) for k in range(steps)]
        ws = scratch(kvq.kvq_beam_select_workspace(ps[0]))
        torch.cuda.synchronize()
        for p in ps:
            kvq.kvq_beam_select(p, ws)
            if one_by_one:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        runs.append((score, fin, token, parent))
    for run in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], run))


# --- page forks ----------------------------------------------------------------------------------

def fork_ref(parent, keep, table, held, free, n_free, lens, page, n_pages):
    """One call, sequence by sequence; table, held, free and lens are updated.  -> copies, n_free, status"""
    n, mp = table.shape
    st = 0
    h = np.clip(held, 0, mp)
    if (h != held).any() or not 0 <= n_free <= n_pages:
        st |= BAD_INDEX
    n_free = min(max(n_free, 0), n_pages)
    old, old_lens = table.copy(), lens.copy()
    new, new_len = [], []
    for s in range(n):
        p = int(parent[s])
        if not -1 <= p < n:
            st |= BAD_INDEX
            p = -1
        if p < 0:
            new.append([]), new_len.append(0)
            continue
        L = int(old_lens[p])
        if L < 0:
            st, L = st | BAD_INDEX, 0
        if L > int(h[p]) * page:
            st, L = st | BAD_PAGE, int(h[p]) * page
        if keep is not None:
            L = min(L, max(int(keep[s]), 0))
        row = [int(x) for x in old[p, :-(-L // page)]]
        if any(not 0 <= x < n_pages for x in row):
            st |= BAD_PAGE
        new.append([x if 0 <= x < n_pages else -1 for x in row]), new_len.append(L)
    for s in range(n):
        if any(not 0 <= int(x) < n_pages for x in old[s, :h[s]]):
            st |= BAD_PAGE
    whole = {x for r, L in zip(new, new_len) for x in r[:L // page]}
    keeper, copies = {}, []
    for s in range(n):
        if new_len[s] % page and new[s][-1] >= 0:
            x = new[s][-1]
            if x in whole or x in keeper:
                copies.append(s)
            else:
                keeper[x] = s
    was = {int(x) for s in range(n) for x in old[s, :h[s]] if 0 <= x < n_pages}
    stack = [int(x) for x in free[:n_free]]
    for x in sorted(was - whole - set(keeper), reverse=True):
        if len(stack) < n_pages:
            free[len(stack)] = x
            stack.append(x)
        else:
            st |= BAD_PAGE
    done = []
    for s in copies:
        if not stack:
            st |= NO_PAGE
            new_len[s] -= new_len[s] % page
            new[s] = new[s][:-1]
            continue
        x = stack.pop()
        done.append((new[s][-1], x, new_len[s] % page))
        new[s][-1] = x
    for s in range(n):
        for e in range(max(len(new[s]), int(h[s]), -(-new_len[s] // page))):
            table[s, e] = new[s][e] if e < len(new[s]) else -1
        held[s], lens[s] = len(new[s]), new_len[s]
    return done, len(stack), st


class Forks:
    """The state of a pool on the device beside the plain one's."""

    def __init__(self, kvq, n, max_pages, n_pages, page, seed):
        self.kvq, self.page, self.n_pages, self.g = kvq, page, n_pages, np.random.default_rng(seed)
        self.table, self.held, self.lens = np.full((n, max_pages), -1, np.int32), np.zeros(n, np.int32), np.zeros(n, np.int32)
        self.free, self.n_free = self.g.permutation(n_pages).astype(np.int32), n_pages
        self.d = dict(block_table=dev(self.table), n_held=dev(self.held), free_list=dev(self.free), n_free=i32(1, fill=n_pages),
                      seq_len=dev(self.lens))
        self.lists = dict(copy_src=i32(n, fill=-7), copy_dst=i32(n, fill=-7), copy_rows=i32(n, fill=-7), n_copy=i32(1, fill=-7))

    def push(self):
        for k, v in (("block_table", self.table), ("n_held", self.held), ("free_list", self.free), ("seq_len", self.lens)):
            self.d[k].copy_(dev(v))
        self.d["n_free"].fill_(self.n_free)

    def grow(self, new, page_plan=True):
        """kvq_resize_pages of every sequence by new[s] tokens; -> the slots, packed."""
        n = len(self.lens)
        new = np.asarray(new, np.int32)
        seq_len, start, slots, st = i32(n), i32(n + 1), i32(int(new.sum()) + 1), i32(1)
        self.kvq.kvq_resize_pages(self.kvq.make_page_plan(
            keep_len=dev(self.lens), n_new=dev(new), seq_len=seq_len, tok_start=start, slot_map=slots, page_size=self.page,
            **{k: self.d[k] for k in ("block_table", "n_held", "free_list", "n_free")}), st)
        torch.cuda.synchronize()
        self.d["seq_len"].copy_(seq_len)
        self.pull()
        return host(slots)[:-1], st.item()

    def pull(self):
        self.table, self.held, self.free, self.lens = (host(self.d[k]).copy() for k in ("block_table", "n_held", "free_list", "seq_len"))
        self.n_free = int(self.d["n_free"].item())

    def fork(self, parent, keep=None, status=None):
        parent = np.asarray(parent, np.int32)
        keep = None if keep is None else np.asarray(keep, np.int32)
        p = self.kvq.make_fork_plan(parent=dev(parent), keep_len=None if keep is None else dev(keep), page_size=self.page, **self.d,
                                    **self.lists)
        st = i32(1)
        self.kvq.kvq_fork_pages(p, scratch(self.kvq.kvq_fork_pages_workspace(p)), st)
        torch.cuda.synchronize()
        copies, self.n_free, want = fork_ref(parent, keep, self.table, self.held, self.free, self.n_free, self.lens, self.page, self.n_pages)
        assert st.item() == want if status is None else st.item() == want == status
        for k, v in (("block_table", self.table), ("n_held", self.held), ("free_list", self.free), ("seq_len", self.lens)):
            assert np.array_equal(host(self.d[k]), v), k
        assert self.d["n_free"].item() == self.n_free and self.lists["n_copy"].item() == len(copies)
        n = len(parent)
        for k, name in enumerate(("copy_src", "copy_dst", "copy_rows")):
            assert np.array_equal(host(self.lists[name]), [c[k] for c in copies] + [-1] * (n - len(copies))), name
        return copies


@pytest.mark.parametrize("n,max_pages,n_pages,page,tokens", [
    (1, 1, 1, 1, 1), (4, 8, 64, 16, 60), (8, 40, 400, 16, 500), (64, 9, 900, 5, 30), (300, 30, 20000, 64, 1500),
    (1030, 5, 9000, 3, 9), (2, 3000, 7000, 4, 9000), (40, 600, 200000, 8, 4000),
    (5000, 3, 20000, 4, 9), (512, 16, 8192, 2, 20), (513, 16, 8192, 2, 20), (4097, 2, 8193, 3, 5),
])
def test_fork_steps(kvq, n, max_pages, n_pages, page, tokens):
    f = Forks(kvq, n, max_pages, n_pages, page, n + page)
    g = f.g
    f.grow(g.integers(0, tokens + 1, n))
    for step in range(6):
        if step == 2:
            parent = np.full(n, int(g.integers(0, n)))       # all from one
        elif step == 4:
            parent = np.arange(n)                            # everyone stays
        else:
            parent = g.integers(-1, n, n)
        keep = None if step % 2 == 0 else g.integers(-2, tokens + 5, n)
        f.fork(parent, keep)
        # every page is in the list, or held; a partial last page has one owner
        held = [int(x) for s in range(n) for x in f.table[s, :f.held[s]]]
        assert set(held) | set(f.free[:f.n_free].tolist()) == set(range(n_pages)) and not set(held) & set(f.free[:f.n_free].tolist())
        last = [int(f.table[s, f.held[s] - 1]) for s in range(n) if f.lens[s] % page]
        assert all(held.count(x) == 1 for x in last[:50])
        f.grow(g.integers(0, 3, n) * (f.lens + 2 < max_pages * page))
    f.fork(np.full(n, -1))
    assert f.n_free == n_pages and sorted(f.free.tolist()) == list(range(n_pages)) and not f.held.any()


def test_fork_without_pages(kvq):
    """A list that runs out: the sequences from there on lose their last page's rows."""
    f = Forks(kvq, 6, 4, 5, 4, 1)
    f.grow([11, 0, 0, 0, 0, 3])
    assert f.n_free == 1
    f.fork([0, 0, 0, 0, 5, 5], status=NO_PAGE)
    assert f.lens.tolist() == [11, 11, 8, 8, 3, 0] and f.n_free == 0
    f.fork([0, -1, 2, 3, 4, 4], status=0)                    # the page given back is the one that is wanted
    assert f.lens.tolist() == [11, 0, 8, 8, 3, 3]


def test_fork_bad_inputs(kvq):
    f = Forks(kvq, 6, 5, 30, 4, 2)
    f.grow([9, 3, 20, 0, 7, 1])
    f.fork([0, 9, -2, 2, 4, 5], status=BAD_INDEX)
    f.lens[0], f.lens[4] = -3, 10
    f.push()
    f.fork([0, 0, 4, 3, 4, 4], status=BAD_INDEX | BAD_PAGE)
    f = Forks(kvq, 4, 5, 30, 4, 3)
    f.grow([9, 18, 20, 5])
    f.table[0, 1], f.table[1, 4], f.table[2, 0] = -1, 30, 2**31 - 1
    f.push()
    f.fork([0, 1, 2, 1], status=BAD_PAGE)
    f = Forks(kvq, 3, 5, 30, 4, 4)
    f.grow([9, 18, 20])
    f.held[0], f.held[2], f.n_free = -1, 9, 31
    f.push()
    f.fork([1, 1, 1], status=BAD_INDEX | BAD_PAGE)           # (no room in the list for what is given back)


def test_fork_longest(kvq):
    """A length of 2^31 - 1 rows, of a table that lists its pages many times."""
    page, n_pages = 1 << 20, 100
    f = Forks(kvq, 2, 2100, n_pages, page, 6)
    f.table[0] = np.arange(2100) % 90
    f.held[0], f.lens[0] = 2100, 2**31 - 1
    f.free[:10], f.n_free = np.arange(90, 100), 10
    f.push()
    assert len(f.fork([0, 0], status=0)) == 2 and f.held.tolist() == [2048, 2048] and f.lens.tolist() == [2**31 - 1] * 2


def test_forks_of_several_threads(kvq):
    """Plans of several sizes (and amounts of shared memory) called at once by threads with a stream each."""
    import threading
    sizes = [(8, 1000, 8000, 4), (8, 400, 5000, 4), (600, 20, 60000, 4), (600, 20, 20000, 4)]
    errors = []

    def run(size, seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                n, most, pages, page = size
                f = Forks(kvq, n, most, pages, page, seed)
                f.grow(f.g.integers(0, 60, n))
                parent = dev(np.arange(n, dtype=np.int32))
                p = kvq.make_fork_plan(parent=parent, page_size=page, **f.d, **f.lists)
                ws = scratch(kvq.kvq_fork_pages_workspace(p))
                torch.cuda.current_stream().synchronize()
                for _ in range(300):
                    kvq.kvq_fork_pages(p, ws)
                torch.cuda.current_stream().synchronize()
                assert np.array_equal(host(f.d["block_table"]), f.table) and np.array_equal(host(f.d["seq_len"]), f.lens)
        except BaseException as e:                           # noqa: B036 (raised below)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(s, i)) for i, s in enumerate(sizes)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_fork_in_a_graph(kvq):
    """A replayed fork reads what the device holds then."""
    f = Forks(kvq, 8, 20, 300, 8, 5)
    f.grow(f.g.integers(1, 100, 8))
    parent = dev(np.arange(8, dtype=np.int32))
    p = kvq.make_fork_plan(parent=parent, page_size=8, **f.d, **f.lists)
    ws = scratch(kvq.kvq_fork_pages_workspace(p))
    g = graphed(lambda: kvq.kvq_fork_pages(p, ws))
    for _ in range(5):
        par = f.g.integers(-1, 8, 8).astype(np.int32)
        parent.copy_(dev(par))
        g.replay()
        torch.cuda.synchronize()
        copies, f.n_free, _ = fork_ref(par, None, f.table, f.held, f.free, f.n_free, f.lens, 8, 300)
        assert np.array_equal(host(f.d["block_table"]), f.table) and np.array_equal(host(f.d["free_list"]), f.free)
        assert np.array_equal(host(f.d["seq_len"]), f.lens) and f.lists["n_copy"].item() == len(copies)


# --- compaction and copies -----------------------------------------------------------------------

def pool_planes(n_rows, seed, kv=3, d=64):
    """Planes of every kind, their bytes at random: MLA, fp8 K/V, a q4_0 pool, odd rows."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=gen)
    f32 = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    return [dict(lat=u8(n_rows, 512), lat_scale=f32(n_rows), rope=u8(n_rows, 64), rope_scale=f32(n_rows)),
            dict(k=u8(kv, n_rows, d), k_scale=f32(kv, n_rows), v=u8(kv, n_rows, d), v_scale=f32(kv, n_rows)),
            u8(n_rows, 2, 144), u8(n_rows, 7), u8(n_rows * 6)[:n_rows * 5].view(n_rows, 5), f32(n_rows, 3), f32(n_rows, 1, 2, 2100)]


def all_planes(kvq, caches):
    return [x for c in caches for x in kvq._pool_planes(c)]


def run_copies(kvq, caches, page, src, dst, rows, n_copy=None):
    src, dst, rows = (np.asarray(x, np.int32) for x in (src, dst, rows))
    want = []
    for t, axis in all_planes(kvq, caches):
        w = host(t).copy()
        v = w if axis else w[None]
        b = v.copy()
        for s, d, r in list(zip(src, dst, rows))[:n_copy]:
            r = min(max(int(r), 0), page)
            if s >= 0 and d >= 0 and (max(int(s), int(d)) + 1) * page <= b.shape[1]:
                b[:, d * page:d * page + r] = v[:, s * page:s * page + r]
        want.append(b if axis else b[0])
    st = i32(1)
    c = kvq.make_page_copy(caches=caches, page_size=page, copy_src=dev(src), copy_dst=dev(dst), copy_rows=dev(rows),
                           n_copy=i32(1, fill=len(src) if n_copy is None else n_copy))
    kvq.kvq_copy_pages(c, st)
    torch.cuda.synchronize()
    for (t, _), w in zip(all_planes(kvq, caches), want):
        assert np.array_equal(host(t).view(np.uint8), w.view(np.uint8))
    return st.item()


@pytest.mark.parametrize("page", [1, 3, 16, 64, 100])
def test_copies(kvq, page):
    g = np.random.default_rng(page)
    pages = 40
    caches = pool_planes(pages * page, page)
    ids = g.permutation(pages)
    rows = g.integers(0, page + 1, 20)
    rows[:3] = page, 1, page + 9
    assert run_copies(kvq, caches, page, ids[:20], ids[20:], rows) == 0
    assert run_copies(kvq, caches, page, ids[:20], ids[20:], rows[::-1], n_copy=7) == 0
    assert run_copies(kvq, caches, page, ids[:20], ids[20:], rows, n_copy=-3) == 0
    assert run_copies(kvq, caches, page, [-1, 3, 5], [4, -1, 6], [page, page, page]) == 0
    assert run_copies(kvq, caches, page, [pages, 3, 5, 2], [4, 2**31 - 1, pages, 9], [page] * 4) == BAD_PAGE
    assert run_copies(kvq, caches, page, [], [], []) == 0
    assert run_copies(kvq, [caches[0]], page, [8], [9], [page], n_copy=99) == 0      # more than the list holds


def compact_ref(table, held, n_pages, page, most):
    n, mp = table.shape
    h = np.clip(held, 0, mp)
    st = BAD_INDEX if (h != held).any() else 0
    mine = np.arange(mp)[None] < h[:, None]
    ok = mine & (table >= 0) & (table < n_pages)
    if (mine & ~ok).any():
        st |= BAD_PAGE
    used = np.zeros(n_pages, bool)
    used[table[ok]] = True
    u = int(used.sum())
    hole, move = np.flatnonzero(~used[:u]), u + np.flatnonzero(used[u:])
    to = np.arange(n_pages + 1)
    to[move] = hole
    new = np.where(ok, to[np.where(ok, table, 0)], -1)
    free = np.full(n_pages, -1)
    free[:n_pages - u] = np.arange(n_pages - 1, u - 1, -1)
    lists = [np.concatenate([x, np.full(most - len(move), -1)]) for x in (move, hole, np.full(len(move), page))]
    return new, free, u, lists, len(move), st


def check_compact(kvq, table, held, n_pages, page, most=None, in_place=False):
    most = n_pages // 2 if most is None else most
    d_table, d_held = dev(table), dev(held)
    new = d_table if in_place else i32(*table.shape, fill=-7)
    free, n_free, n_used = i32(n_pages, fill=-7), i32(1, fill=-7), i32(1, fill=-7)
    lists = dict(copy_src=i32(most, fill=-7), copy_dst=i32(most, fill=-7), copy_rows=i32(most, fill=-7), n_copy=i32(1, fill=-7))
    p = kvq.make_compact_plan(block_table=d_table, n_held=d_held, new_table=new, free_list=free, n_free=n_free, n_used=n_used,
                              page_size=page, **lists)
    st = i32(1)
    kvq.kvq_compact_pages(p, scratch(kvq.kvq_compact_pages_workspace(p)), st)
    torch.cuda.synchronize()
    want, w_free, u, w_lists, moved, w_st = compact_ref(table, held, n_pages, page, most)
    assert st.item() == w_st
    assert np.array_equal(host(new), want) and np.array_equal(host(free), w_free)
    assert (n_free.item(), n_used.item(), lists["n_copy"].item()) == (n_pages - u, u, moved)
    for name, w in zip(("copy_src", "copy_dst", "copy_rows"), w_lists):
        assert np.array_equal(host(lists[name]), w), name
    if not in_place:
        assert np.array_equal(host(d_table), table)
    return lists, want


@pytest.mark.parametrize("n,n_pages,used,in_place", [
    (1, 1, 1, False), (3, 2, 1, False), (4, 64, 30, True), (5, 100, 100, False), (5, 100, 0, True), (60, 5000, 2600, False),
    (2000, 30000, 9000, True), (7, 300001, 120000, False), (3, 1000, 999, True),
])
def test_compact(kvq, n, n_pages, used, in_place):
    g = np.random.default_rng(n + n_pages)
    cut = np.sort(g.integers(0, used + 1, n - 1))
    held = np.diff(np.concatenate([[0], cut, [used]])).astype(np.int32)
    perm = g.permutation(n_pages).astype(np.int32)
    table = np.full((n, int(held.max()) + 3), -1, np.int32)
    o = 0
    for s in range(n):
        table[s, :held[s]] = perm[o:o + held[s]]
        o += held[s]
    for s in range(1, n, 3):                                 # shared pages
        k = min(held[s], held[s - 1]) // 2
        table[s, :k] = table[s - 1, :k]
    check_compact(kvq, table, held, n_pages, 16, most=None if n % 2 else n_pages // 2 + 5, in_place=in_place)


def test_plans_of_nothing(kvq):
    """No sequences, no pages, or neither."""
    check_compact(kvq, np.zeros((0, 4), np.int32), np.zeros(0, np.int32), 20, 16)
    check_compact(kvq, np.full((3, 4), -1, np.int32), np.zeros(3, np.int32), 0, 16)
    check_compact(kvq, np.zeros((0, 4), np.int32), np.zeros(0, np.int32), 0, 16)
    f = Forks(kvq, 3, 4, 0, 16, 1)
    assert f.fork([2, 0, -1], status=0) == []
    f = Forks(kvq, 0, 4, 5, 16, 1)
    kvq.kvq_fork_pages(kvq.make_fork_plan(parent=i32(0), page_size=16, **f.d, **f.lists))
    torch.cuda.synchronize()
    assert f.d["n_free"].item() == 5 and np.array_equal(host(f.d["free_list"]), f.free) and f.lists["n_copy"].item() == -7


def test_two_streams(kvq):
    """Appends, selections and compactions of two problems at once, each over and over on a stream of its own."""
    def append(i):
        pl, rows = new_planes(4, 5000, 128), 3000 + 1000 * i
        gen = torch.Generator(device="cuda")
        gen.manual_seed(i)
        k, v = (torch.randn(rows, 4, 128, device="cuda", generator=gen).bfloat16() for _ in range(2))
        slot = torch.randperm(5000, device="cuda", generator=gen)[:rows].int()
        return lambda: kvq.kvq_append_kv8(k, v, slot, pl), list(pl.values())

    def select(i):
        R, B, V, K = 20, 4, 30000 + 77 * i, 8
        gen = torch.Generator(device="cuda")
        gen.manual_seed(i)
        x = torch.randn(R, B, V, device="cuda", generator=gen)
        out = [torch.zeros(R, K, device="cuda"), i32(R, K), i32(R, K)]
        p = kvq.make_beam_problem(logits=x, score=torch.randn(R, B, device="cuda", generator=gen), out_score=out[0], out_token=out[1],
                                  out_parent=out[2])
        ws = scratch(kvq.kvq_beam_select_workspace(p))
        return lambda: kvq.kvq_beam_select(p, ws), out

    def compact(i):
        n, n_pages = 50, 9000 + 60000 * i
        g = np.random.default_rng(i)
        table = g.permutation(n_pages)[:n * 60].reshape(n, 60).astype(np.int32)
        out = [i32(n, 60), i32(n_pages), i32(1), i32(1), *(i32(n_pages // 2) for _ in range(3)), i32(1)]
        p = kvq.make_compact_plan(block_table=dev(table), n_held=dev(g.integers(0, 61, n).astype(np.int32)), new_table=out[0], free_list=out[1],
                                  n_free=out[2], n_used=out[3], page_size=16, copy_src=out[4], copy_dst=out[5], copy_rows=out[6],
                                  n_copy=out[7])
        ws = scratch(kvq.kvq_compact_pages_workspace(p))
        return lambda: kvq.kvq_compact_pages(p, ws), out

    for make in (append, select, compact):
        calls, outs = zip(*(make(i) for i in range(2)))
        want = []
        for call, out in zip(calls, outs):
            call()
            torch.cuda.synchronize()
            want.append([t.clone() for t in out])
            for t in out:
                t.zero_()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(40):
            for call, s in zip(calls, streams):
                with torch.cuda.stream(s):
                    call()
        torch.cuda.synchronize()
        for out, ref in zip(outs, want):
            for t, r in zip(out, ref):
                same = t.view(torch.int32) if t.dtype == torch.float32 else t
                assert torch.equal(same, r.view(torch.int32) if r.dtype == torch.float32 else r) or make is append
        if make is append:                                   # (rows without a slot keep what was there)
            for out, ref in zip(outs, want):
                for t, r in zip(out, ref):
                    written = (r != 0x7F) if r.dtype == torch.uint8 else ~r.isnan()
                    assert bool((t == r)[written].all())


def test_compact_bad_inputs(kvq):
    table = np.array([[5, -1, 9, 3], [7, 10, 2**31 - 1, 0], [1, 2, 4, 6]], np.int32)
    check_compact(kvq, table, np.array([4, 3, 9], np.int32), 10, 4)
    check_compact(kvq, table, np.array([0, -1, 2], np.int32), 10, 4, in_place=True)


def test_compacted_cache_decodes_alike(kvq):
    """Attention over a cache gives the same bits after its pages were compacted."""
    lens = [700, 33, 0, 1200, 64]
    c = Cache(lens, 2, 128, 32, 90)
    n_pages = c.pool // 32
    q = queries(5, 8, 128, 91)
    want = decode(kvq, c.problem(kvq, q))
    gap = np.sort(np.random.default_rng(1).permutation(3 * n_pages)[:n_pages])      # a larger, fragmented pool
    pl = new_planes(2, 3 * c.pool, 128)
    rows = torch.from_numpy((gap[:, None] * 32 + np.arange(32)).reshape(-1)).cuda()
    for k in pl:
        pl[k][:, rows] = c.pl[k]
    table = np.where(c.table >= 0, gap[np.maximum(c.table, 0)], -1).astype(np.int32)
    held = np.array([-(-x // 32) for x in lens], np.int32)
    lists, new = check_compact(kvq, table, held, 3 * n_pages, 32)
    kvq.kvq_copy_pages(kvq.make_page_copy(caches=[pl], page_size=32, **lists))
    c.pl = pl
    got = decode(kvq, c.problem(kvq, q, table=new.astype(np.int32)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# --- whole steps ---------------------------------------------------------------------------------

class Toy:
    """A small model of one attention layer: embeddings, projections, logits."""

    def __init__(self, V, H, kv, d, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        m = 128
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.emb, self.wqkv, self.wo = r(V, m), r(m, (H + 2 * kv) * d) / math.sqrt(m), r(H * d, V) * 3 / math.sqrt(H * d)
        self.H, self.kv, self.d = H, kv, d

    def rows(self, tokens):
        x = (self.emb[tokens] @ self.wqkv).bfloat16().view(len(tokens), self.H + 2 * self.kv, self.d)
        return x[:, :self.H], x[:, self.H:self.H + self.kv], x[:, self.H + self.kv:]


def fp8_rows(orc, x):
    """The rows [n, kv, d] that the oracle's encoder keeps of x, as numbers (torch's quotient by a number is a product)."""
    codes, scales = encoded(orc, host(x.float()))
    c = dev(codes).view(torch.float8_e4m3fn).double() * dev(scales)[..., None].double()
    return c.transpose(0, 1)


@pytest.mark.parametrize("as_graph", [False, True])
def test_beam_search(kvq, orc, as_graph):
    """Prompts, then steps of resize, append, decode, selection, fork and copies over a paged cache (two layers' planes
    share its tables), against a search whose beams each hold a dense cache of their own."""
    V, H, kv, d, page, R, B, steps = 301, 8, 2, 64, 8, 3, 4, 20
    model = Toy(V, H, kv, d, 7)
    n, n_pages, most = R * B, 120, 64
    g = np.random.default_rng(8)
    prompts = [torch.from_numpy(g.integers(3, V, int(x))).cuda() for x in (17, 8, 30)]
    pl, other = new_planes(kv, n_pages * page, d), new_planes(kv, n_pages * page, d)
    f = Forks(kvq, n, most // page, n_pages, page, 9)
    lens = np.zeros(n, np.int32)
    lens[::B] = [len(p) for p in prompts]
    slots, st = f.grow(lens)
    assert st == 0
    _, k, v = model.rows(torch.cat(prompts))
    for c in (pl, other):
        kvq.kvq_append_kv8(k, v, dev(slots), c)
    copy = kvq.make_page_copy(caches=[pl, other], page_size=page, **f.lists)
    f.fork(np.arange(n) // B * B)                            # the prompt's beam fans out
    kvq.kvq_copy_pages(copy)

    seq_len, start, slot, ones = f.d["seq_len"], i32(n + 1), i32(n), i32(n, fill=1)
    old_len = seq_len.clone()
    score, fin = torch.full((R, B), -math.inf, device="cuda"), i32(R, B)
    score[:, 0] = 0.0
    token, parent = torch.cat([p[-1:].repeat(B) for p in prompts]).int().view(R, B), i32(R, B)
    q, out = torch.zeros(n, H, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, H, d, dtype=torch.bfloat16, device="cuda")
    logits, status = torch.zeros(R, B, V, device="cuda"), i32(1)
    plan = kvq.make_page_plan(keep_len=old_len, n_new=ones, seq_len=seq_len, tok_start=start, slot_map=slot, page_size=page,
                              **{k: f.d[k] for k in ("block_table", "n_held", "free_list", "n_free")})
    dp = kvq.make_kv8_problem(seq_len=seq_len, q=q, sm_scale=1 / 8, max_seq_len=most, cache=pl, block_table=f.d["block_table"], page_size=page)
    bp = kvq.make_beam_problem(logits=logits, score=score, finished=fin, out_score=score, out_token=token, out_parent=parent,
                               out_finished=fin, eos=2, pad=1)
    fp = kvq.make_fork_plan(parent=parent.view(n), page_size=page, **f.d, **f.lists)
    ws = [scratch(w) for w in (kvq.kvq_kv8_decode_workspace(dp), kvq.kvq_beam_select_workspace(bp), kvq.kvq_fork_pages_workspace(fp))]

    def step():
        old_len.copy_(seq_len)
        kvq.kvq_resize_pages(plan, status)
        qk, k, v = model.rows(token.view(n).long())
        q.copy_(qk)
        for c in (pl, other):
            kvq.kvq_append_kv8(k, v, slot, c, status)
        kvq.kvq_kv8_decode(dp, out, None, ws[0], status)
        torch.matmul(out.float().view(n, -1), model.wo, out=logits.view(n, V))
        logits[..., 2] += 0.5
        kvq.kvq_beam_select(bp, ws[1], status)
        kvq.kvq_fork_pages(fp, ws[2], status)
        kvq.kvq_copy_pages(copy, status)

    # the dense search: every beam's own rows as numbers
    dense = [[fp8_rows(orc, model.rows(p)[i + 1]) for i in range(2)] for p in prompts for _ in range(B)]
    history = [[] for _ in range(n)]
    if as_graph:
        keep = [t.clone() for t in (seq_len, score, fin, token, parent, *(f.d[k] for k in f.d))]
        planes = [{k: t.clone() for k, t in c.items()} for c in (pl, other)]
        graph = graphed(step)
        for t, w in zip((seq_len, score, fin, token, parent, *(f.d[k] for k in f.d)), keep):
            t.copy_(w)
        for c, w in zip((pl, other), planes):
            for k in c:
                c[k].copy_(w[k])
    for _ in range(steps):
        before = (score.clone(), fin.clone(), token.clone())
        graph.replay() if as_graph else step()
        torch.cuda.synchronize()
        assert status.item() == 0
        qk, k, v = model.rows(before[2].view(n).long())
        rows = [fp8_rows(orc, k), fp8_rows(orc, v)]
        dense = [[torch.cat([dense[s][i], rows[i][s:s + 1]]) for i in range(2)] for s in range(n)]
        for s in range(n):                                   # the attention of this step, over the beam's own rows
            K, V_ = (x.transpose(0, 1) for x in dense[s])
            x = qk[s].double().view(kv, H // kv, d) @ K.transpose(1, 2) / 8
            p = torch.softmax(x, 2)
            o, mass = (p @ V_).view(H, d), (p @ V_.abs()).view(H, d)
            # (scores here are below 2^7 in their terms' sum: 2^-10 covers their part, as in check_decode)
            bar = 2.0**-8 * o.abs() + (2.0**-9 + 2.0**-10) * mass.amax(1, keepdim=True)
            assert bool(((out[s].double() - o).abs() <= bar).all())
        want = beam_ref(host(logits), host(before[0]), host(before[1]), B, 2, 1)
        assert np.array_equal(host(token), want[1]) and np.array_equal(host(parent), want[2]) and np.array_equal(host(fin), want[3])
        up = want[2].reshape(n)
        dense = [dense[u] for u in up]
        history = [history[u] + [int(t)] for u, t in zip(up, want[1].reshape(n))]
        assert host(seq_len).tolist() == [len(x[0]) for x in dense]
        table, held = host(f.d["block_table"]), host(f.d["n_held"])
        for c in (pl, other):                                # every beam's rows, through its table
            for s in range(n):
                pos = np.arange(len(dense[s][0]))
                at = torch.from_numpy(table[s, pos // page].astype(np.int64) * page + pos % page).cuda()
                for name, x in zip(("k", "v"), dense[s]):
                    assert torch.equal(values(c, name, at).transpose(0, 1), x)
        pages = {int(x) for s in range(n) for x in table[s, :held[s]]}
        free = host(f.d["free_list"])[:f.d["n_free"].item()].tolist()
        assert len(pages) + len(free) == n_pages and not pages & set(free)
    assert len({tuple(h) for h in history}) > R              # beams of a request differ


@pytest.mark.parametrize("d,page", [(64, 0), (128, 0), (256, 16), (128, 48), (64, 20)])
def test_decode_rows_behind_the_pool(kvq, d, page):
    """A pool cut short: rows (without a table) or whole pages that it no longer holds are skipped, and flagged."""
    c = Cache([400, 300], 2, d, page, 95)
    cut = c.pool - 37
    pl = {k: t[:, :cut].contiguous() for k, t in c.pl.items()}
    q = queries(2, 8, d, 96)
    p = kvq.make_kv8_problem(seq_len=dev(c.lens), q=q, sm_scale=1 / math.sqrt(d), max_seq_len=400, cache=pl, page_size=page,
                             block_table=None if c.table is None else dev(c.table), seq_stride_rows=0 if page else c.stride)
    st = i32(1)
    out, lse = decode(kvq, p, st)

    def rows_of(s, pos):
        r = c.rows_of(s, pos)
        last = (r // page + 1) * page - 1 if page else r
        return np.where(last < cut, r, -1)
    lost = any((rows_of(s, np.arange(int(n))) < 0).any() for s, n in enumerate(c.lens))
    assert st.item() == (BAD_PAGE if lost else 0)
    check_decode(out, lse, decode_ref(pl, q, c.lens, rows_of, 0, 1 / math.sqrt(d)), d, 400)
