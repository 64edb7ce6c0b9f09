"""GPU parity of the entry points for drafted tokens against plain implementations: page
tables and accepted rows exactly, appended rows byte for byte against the oracle's encoders,
tree attention against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu
NO_PAGE, BAD_INDEX, BAD_PAGE = 16, 1, 2
ROW_BYTES = {1: 512, 2: 256, 4: 384, 5: 192}
BITS = {2: 4, 4: 6, 5: 3}


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


# --- page tables ---------------------------------------------------------------------------

def resize_ref(keep, new, table, held, free, n_free, page, n_pages, max_tokens):
    """One call, page by page (table, held and free are updated); -> seq_len, tok_start, slots,
    positions, n_free, status."""
    n, mp = table.shape
    status = 0
    keep0, new0, held0 = keep, new, held.copy()
    keep, new = np.maximum(keep, 0).astype(np.int64), np.maximum(new, 0).astype(np.int64)
    h = np.clip(held, 0, mp).astype(np.int64)
    if (keep0 < 0).any() or (new0 < 0).any() or (h != held0).any() or not 0 <= n_free <= n_pages:
        status |= BAD_INDEX
    n_free = min(max(n_free, 0), n_pages)
    start = np.concatenate([[0], np.cumsum(new)])
    need, ok = h.copy(), np.zeros(n, bool)
    for s in range(n):
        want = -(-(keep[s] + new[s]) // page)
        if keep[s] + new[s] > 2**31 - 1 or (new[s] > 0 and start[s + 1] > max_tokens):
            status |= BAD_INDEX
        elif keep[s] > h[s] * page:
            status |= BAD_PAGE
        elif want > mp:
            status |= NO_PAGE
        else:
            need[s], ok[s] = want, True
    stack = [int(x) for x in free[:n_free]]
    for s in reversed(range(n)):
        for e in reversed(range(int(need[s]), int(h[s]))):
            free[len(stack)] = table[s, e]
            stack.append(int(table[s, e]))
            table[s, e] = -1
    out = False
    seq_len = np.minimum(keep, h * page)
    for s in range(n):
        take = int(need[s] - h[s])
        if not ok[s]:
            continue
        if take > 0 and (out or take > len(stack)):
            out, ok[s] = True, False
            status |= NO_PAGE
            continue
        for e in range(int(h[s]), int(need[s])):
            table[s, e] = stack.pop()
        held[s] = need[s]
        seq_len[s] = keep[s] + new[s]
    slots, pos = np.full(max_tokens, -1), np.full(max_tokens, -1)
    for s in range(n):
        if ok[s]:
            for t in range(int(new[s])):
                p = int(keep[s]) + t
                pg = int(table[s, p // page])
                if 0 <= pg < n_pages:
                    slots[start[s] + t], pos[start[s] + t] = pg * page + p % page, p
                else:
                    status |= BAD_PAGE
    return seq_len, np.minimum(start, 2**31 - 1), slots, pos, len(stack), status


class Pages:
    """The allocator's state on the device beside the plain one's."""

    def __init__(self, kvq, n_seq, max_pages, n_pages, page, seed):
        g = np.random.default_rng(seed)
        self.kvq, self.page, self.n_pages = kvq, page, n_pages
        self.table = np.full((n_seq, max_pages), -1, np.int32)
        self.held = np.zeros(n_seq, np.int32)
        self.free = g.permutation(n_pages).astype(np.int32)
        self.n_free = n_pages
        self.d = [dev(self.table), dev(self.held), dev(self.free), i32(1, fill=n_pages)]

    def step(self, keep, new, max_tokens, positions=True, status=None):
        keep, new = np.asarray(keep, np.int32), np.asarray(new, np.int32)
        n = len(keep)
        seq_len, start = i32(n, fill=-7), i32(n + 1, fill=-7)
        slots, pos = i32(max_tokens, fill=-7), i32(max_tokens, fill=-7)
        st = i32(1)
        plan = self.kvq.make_page_plan(
            keep_len=dev(keep), n_new=dev(new), block_table=self.d[0], n_held=self.d[1], free_list=self.d[2],
            n_free=self.d[3], page_size=self.page, seq_len=seq_len, tok_start=start, slot_map=slots,
            tok_pos=pos if positions else None)
        self.kvq.kvq_resize_pages(plan, st)
        torch.cuda.synchronize()
        r_len, r_start, r_slots, r_pos, self.n_free, r_st = resize_ref(
            keep, new, self.table, self.held, self.free, self.n_free, self.page, self.n_pages, max_tokens)
        assert st.item() == r_st if status is None else st.item() == r_st == status
        for got, want in ((seq_len, r_len), (start, r_start), (slots, r_slots), (self.d[0], self.table),
                          (self.d[1], self.held), (self.d[2], self.free)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert np.array_equal(pos.cpu().numpy(), r_pos if positions else np.full(max_tokens, -7))
        assert self.d[3].item() == self.n_free
        return r_len


@pytest.mark.parametrize("n_seq,page,grow,tokens", [(1, 64, 1, 1), (1, 8, 5000, 5003), (7, 16, 40, 280), (300, 64, 30, 9000),
                                                   (1024, 1, 3, 3100), (1500, 48, 100, 150000), (2600, 16, 9, 4096),
                                                   (3000, 100, 2, 6000)])
def test_resize_grow_shrink_refuse(kvq, n_seq, page, grow, tokens):
    """A run of steps: admission, growth, roll-back, ends of sequences, an empty list."""
    g = np.random.default_rng(n_seq)
    per = -(-3 * grow // page)
    P = Pages(kvq, n_seq, per + 1, max(1, n_seq * per * 2 // 3), page, seed=page)
    lens = np.zeros(n_seq, np.int64)
    for step in range(6):
        new = g.integers(0, grow + 1, n_seq)
        if step == 2:                                     # roll back, and some sequences end
            lens = np.where(g.random(n_seq) < 0.3, 0, g.integers(0, lens + 1))
            new[:] = 0
        lens = P.step(lens, new, tokens, positions=step != 3)


def test_resize_undoes_a_step(kvq):
    P = Pages(kvq, 40, 12, 300, 16, seed=1)
    g = np.random.default_rng(2)
    lens = P.step(np.zeros(40), g.integers(0, 60, 40), 3000, status=0)
    before = [t.clone() for t in P.d]
    P.step(lens, g.integers(0, 60, 40), 3000, status=0)
    P.step(lens, np.zeros(40), 0, status=0)
    top = int(before[3].item())
    for got, want, upto in zip(P.d, before, (None, None, top, None)):
        assert torch.equal(got[:upto], want[:upto])


def test_resize_refusals_and_bad_lengths(kvq):
    """Every reason for a refusal in one batch, beside sequences that are served."""
    P = Pages(kvq, 8, 4, 12, 8, seed=3)
    P.step([0] * 8, [8, 9, 0, 1, 3, 0, 0, 0], 64, status=0)
    big = 2**31 - 1
    keep = [8, 17, -5, 1, 3, 2, 0, 0]     # 1: beyond its pages; 2: negative; 5: rows but no page
    new = [1, 1, 4, 32, big, 1, 0, -3]    # 3: table full; 4: length and tokens
    P.step(keep, new, 50)
    P.step([0] * 8, [0] * 8, 1, status=0)
    P.step([0] * 8, [32, 32, 32, 32, 0, 1, 0, 5], 200, status=NO_PAGE)     # the list runs out at sequence 3
    P.d[3].fill_(-4)
    P.n_free = -4
    P.step([0] * 8, [0, 0, 0, 40, 0, 0, 0, 0], 200, status=BAD_INDEX | NO_PAGE)


def test_resize_without_sequences_or_tokens(kvq):
    P = Pages(kvq, 1, 1, 4, 8, seed=4)
    for tokens in (0, 5, 9000):
        plan = kvq.make_page_plan(keep_len=i32(0), n_new=i32(0), block_table=i32(0, 1), n_held=i32(0),
                                  free_list=P.d[2], n_free=P.d[3], page_size=8, seq_len=i32(0),
                                  tok_start=i32(1, fill=9), slot_map=i32(tokens, fill=9))
        kvq.kvq_resize_pages(plan)
        torch.cuda.synchronize()
        assert plan._keep[7].tolist() == [0] and (plan._keep[8] == -1).all() and P.d[3].item() == 4


def test_resize_page_id_outside_the_pool(kvq):
    P = Pages(kvq, 2, 2, 6, 8, seed=5)
    P.free[5] = 77
    P.d[2][5] = 77
    P.step([0, 0], [9, 3], 16, status=BAD_PAGE)


# --- append --------------------------------------------------------------------------------

def encode_ref(orc, fmt, x, k, signs):
    lat, ls = orc.encode_fp8(x) if fmt == 1 else orc.encode_tq(x, signs, BITS[fmt])
    rope, rs = orc.encode_fp8(k)
    return dict(lat=lat, lat_scale=ls, rope=rope, rope_scale=rs)


def empty_planes(fmt, rows, fill=0xA5):
    return dict(lat=torch.full((rows, ROW_BYTES[fmt]), fill, dtype=torch.uint8, device="cuda"),
                lat_scale=torch.full((rows,), -3.0, device="cuda"),
                rope=torch.full((rows, 64), fill, dtype=torch.uint8, device="cuda"),
                rope_scale=torch.full((rows,), -3.0, device="cuda"))


@pytest.mark.parametrize("fmt", [1, 2, 4, 5])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows", [1, 7, 257, 3001])
def test_append_bytes_and_untouched_rows(kvq, orc, fmt, bf16, rows):
    """Byte-exact rows at their slots from strided inputs (one fused projection's output);
    rows without a slot are skipped and no other pool row changes."""
    g = np.random.default_rng(rows)
    pool = 2 * rows + 3
    data = W.fp8_tiny_rows(rows, seed=rows)
    both = torch.cat([dev(data.c), dev(data.k_rope)], 1)
    both = both.bfloat16() if bf16 else both
    x, k = both[:, :512], both[:, 512:]
    slot = g.permutation(pool)[:rows].astype(np.int32)
    if rows > 1:
        slot[g.random(rows) < 0.2] = -1
        slot[1] = -(2**31)
    if rows > 7:
        slot[5], slot[6] = pool, 2**31 - 1               # past the pool: skipped, flagged
    signs = W.sign_bits(3)
    planes, st = empty_planes(fmt, pool), i32(1)
    kvq.kvq_append_mla(x, k, dev(slot), fmt, dev(signs.view(np.int32)), planes, st)
    torch.cuda.synchronize()
    ref = encode_ref(orc, fmt, x.float().cpu().numpy(), k.float().cpu().numpy(), signs)
    want = {n: v.cpu().numpy() for n, v in empty_planes(fmt, pool).items()}
    go = (slot >= 0) & (slot < pool)
    for n in want:
        want[n][slot[go]] = ref[n][go]
        assert np.array_equal(planes[n].cpu().numpy().view(np.uint8), want[n].view(np.uint8)), n
    assert st.item() == (BAD_PAGE if rows > 7 else 0)


@pytest.mark.parametrize("bf16", [False, True])
def test_append_extreme_magnitudes(kvq, orc, bf16):
    """fp8 rows from the smallest normal numbers to 1e35: the quotients by the row's scale are IEEE ones
    at every scale, codes and scales byte for byte."""
    g = np.random.default_rng(0)
    mag = np.concatenate([10.0 ** np.arange(-37, 36, 1.0), [2.0**-81, 2.0**-82, 2.0**99, 2.0**98]]).astype(np.float32)
    x = (W.normal(g, (len(mag), 576)) * mag[:, None]).astype(np.float32)
    both = dev(x).bfloat16() if bf16 else dev(x)
    planes = empty_planes(1, len(mag))
    kvq.kvq_append_mla(both[:, :512], both[:, 512:], torch.arange(len(mag), dtype=torch.int32, device="cuda"), 1, None, planes)
    torch.cuda.synchronize()
    host = both.float().cpu().numpy()
    ref = encode_ref(orc, 1, np.ascontiguousarray(host[:, :512]), np.ascontiguousarray(host[:, 512:]), None)
    for key in ref:
        assert np.array_equal(planes[key].cpu().numpy().view(np.uint8), ref[key].view(np.uint8)), key


@pytest.mark.parametrize("bf16", [False, True])
def test_append_non_finite_rows_equal_encode_mla(kvq, bf16):
    """fp8 rows that hold NaNs, infinities or subnormals: still the bytes of kvq_encode_mla."""
    x = W.normal(np.random.default_rng(8), (40, 576)).astype(np.float32)
    for r in range(30):
        x[r, 17 * r % 512] = (np.nan, np.inf, -np.inf)[r % 3]
        x[r, 512 + r] = (np.inf, np.nan, -np.nan)[r % 3]
    x[5, :] = np.nan
    x[33:36] *= np.float32(1e-39)
    both = dev(x).bfloat16() if bf16 else dev(x)
    wide = both.float()
    a, b = empty_planes(1, 40), empty_planes(1, 40)
    kvq.kvq_encode_mla(wide[:, :512].contiguous(), wide[:, 512:].contiguous(), 1, None, a["lat"], a["lat_scale"], a["rope"], a["rope_scale"])
    kvq.kvq_append_mla(both[:, :512], both[:, 512:], torch.arange(40, dtype=torch.int32, device="cuda"), 1, None, b)
    torch.cuda.synchronize()
    for key in a:
        assert torch.equal(a[key].view(torch.uint8), b[key].view(torch.uint8)), key


@pytest.mark.parametrize("bf16", [False, True])
def test_append_every_quotient_equals_encode_mla(kvq, bf16):
    """fp8 rows whose largest element takes each of the 128 significands of bfloat16, at exponents from -70 to 90, beside
    elements of every significand, both signs and 18 binades, and beside zeros of both signs: the
    bytes of kvq_encode_mla, in which a negative zero is the code 0x80."""
    sig = np.arange(128, 256, dtype=np.float64)
    small = np.concatenate([sig * 2.0**-e for e in range(1, 19)])             # below the largest's binade
    small = np.concatenate([small, -small, [0.0, -0.0]])
    per = 510
    small = np.concatenate([small, np.full(-len(small) % per, -0.0)]).reshape(-1, per)
    rows = []
    for e in (-77, 0, 83):
        for top in sig:
            x = np.full((len(small), 576), -0.0)
            x[:, 0], x[:, 1:1 + per], x[:, 511], x[:, 512] = top, small, 0.0, -top
            x[:, 513:] = small[:, :63]
            rows.append(x * 2.0**e)
    x = np.concatenate(rows).astype(np.float32)
    n = len(x)
    wide = dev(x)
    both = wide.bfloat16() if bf16 else wide
    assert torch.equal(both.float().view(torch.int32), wide.view(torch.int32))                 # exact, signs of zeros included
    a, b = empty_planes(1, n), empty_planes(1, n)
    kvq.kvq_encode_mla(wide[:, :512].contiguous(), wide[:, 512:].contiguous(), 1, None, a["lat"], a["lat_scale"], a["rope"], a["rope_scale"])
    kvq.kvq_append_mla(both[:, :512], both[:, 512:], torch.arange(n, dtype=torch.int32, device="cuda"), 1, None, b)
    torch.cuda.synchronize()
    assert (a["lat"] == 0x80).any() and (a["rope"] == 0x80).any()
    for key in a:
        assert torch.equal(a[key].view(torch.uint8), b[key].view(torch.uint8)), key


def test_append_equals_encode_mla(kvq):
    """The bytes of kvq_encode_mla, at the identity and a reversed slot map; zero rows."""
    n = 600
    data = W.fp8_tiny_rows(n, seed=2)
    x, k, signs = dev(data.c), dev(data.k_rope), dev(W.sign_bits(2).view(np.int32))
    for fmt in (1, 2, 4, 5):
        a, b = empty_planes(fmt, n), empty_planes(fmt, n)
        kvq.kvq_encode_mla(x, k, fmt, signs, a["lat"], a["lat_scale"], a["rope"], a["rope_scale"])
        for slot in (torch.arange(n), torch.arange(n - 1, -1, -1)):
            slot = slot.int().cuda()
            kvq.kvq_append_mla(x, k, slot, fmt, signs, b)
            torch.cuda.synchronize()
            for key in a:
                assert torch.equal(b[key][slot.long()], a[key])


# --- tree attention ------------------------------------------------------------------------

U = 2.0**-8                       # half a step of bf16, relative


def random_tree(g, n):
    out = []
    for j in range(n):
        out.append((out[int(g.integers(0, j))] if j else 0) | 1 << j)
    return out


def masks_of(g, n_node, n_q, kind):
    """[n_seq][n_q] bit masks: "tree" (ancestors and self), "any" (any bits, some empty, some
    past the nodes), or None (a chain)."""
    if kind == "chain":
        return None
    m = np.zeros((len(n_node), n_q), np.uint64)
    for s, n in enumerate(n_node):
        rows = random_tree(g, n) if kind == "tree" else [int(x) for x in g.integers(0, 2**63, n, dtype=np.uint64)]
        for j, x in enumerate(rows):
            m[s, j] = 0 if kind == "any" and j % 3 == 1 else x
    return m


def tree_ref(orc, fmt, cache, signs, rows_of, lens, n_node, masks, q_lat, q_rope, sm_scale):
    """The formula in 64 bits, and per output row the error bounds of the packed form:
    (out, lse, worst [.., 512], norm [..]).  The packed form carries each weight in two e4m3
    digits: a relative error of at most 2^-4 2^-4 (half steps of both), or, where the second digit
    is subnormal, half of its step 2^-9 on a scale that holds the largest weight at 2^4 or more;
    every output is rounded to bf16."""
    n_seq, n_q, H, _ = q_lat.shape
    out, lse = np.zeros((n_seq, n_q, H, 512)), np.full((n_seq, n_q, H), -np.inf)
    worst, norm = np.zeros_like(out), np.zeros((n_seq, n_q, H))
    for s in range(n_seq):
        r, ok = rows_of(s)
        if fmt == 1:
            code, c = orc.decode_fp8(cache["lat"][r], np.ones(len(r), np.float32)), orc.decode_fp8(cache["lat"][r], cache["lat_scale"][r])
        else:
            c, _ = orc.decode_tq(cache["lat"][r], cache["lat_scale"][r], signs, 512, BITS[fmt])
            code = np.zeros_like(c)
        k = orc.decode_fp8(cache["rope"][r], cache["rope_scale"][r])
        ls = cache["lat_scale"][r].astype(np.float64)
        first = lens[s] - n_node[s]
        for j in range(n_node[s]):
            see = ok.copy()
            for t in range(n_node[s]):
                bit = t <= j if masks is None else (int(masks[s, j]) >> t) & 1
                see[first + t] &= bool(bit)
            if not see.any():
                continue
            x, kk, cd = c[see], k[see], code[see]
            sc = sm_scale * (q_lat[s, j].astype(np.float64) @ x.T + q_rope[s, j].astype(np.float64) @ kk.T)
            top = sc.max(1, keepdims=True)
            p = np.exp(sc - top)
            z = p.sum(1, keepdims=True)
            p /= z
            o = p @ x
            out[s, j] = o
            lse[s, j] = (top + np.log(z))[:, 0]
            # the weight of a code is p * scale; floor of its two digits
            floor = 2.0**-14 * (p * ls[see]).max(1, keepdims=True)
            worst[s, j] = U * np.abs(o) + U * (p @ np.abs(x)) + floor * np.abs(cd).sum(0)
            var = (U * o)**2 + U**2 * (p**2 @ x**2) + floor**2 * (cd**2).sum(0)
            norm[s, j] = np.sqrt(var.sum(1) / 3.0)
    return out, lse, worst, norm


def make_cache(orc, fmt, rows, seed, signs):
    data = W.magnitude_rows(rows, seed=seed, lo=1e-2, hi=10.0)
    return encode_ref(orc, fmt, data.c, data.k_rope, signs)


def run_tree(kvq, *, fmt, cache, signs, lens, n_node, masks, q_lat, q_rope, table=None, page=0, stride=0, impl=0,
             max_len=None, sm_scale=float(W.SM_SCALE), pass_nodes=True, kernel=None):
    p = kvq.make_tree_problem(
        seq_len=dev(np.asarray(lens, np.int32)), n_node=dev(np.asarray(n_node, np.int32)) if pass_nodes else None,
        mask=None if masks is None else dev(masks.view(np.int64)), q_lat=q_lat, q_rope=q_rope, sm_scale=sm_scale,
        max_seq_len=max(lens) if max_len is None else max_len, fmt=fmt,
        cache={k: v if torch.is_tensor(v) else dev(v) for k, v in cache.items()},
        signs=dev(signs.view(np.int32)), block_table=None if table is None else dev(table), page_size=page,
        seq_stride_rows=stride, impl=impl)
    if kernel is not None:
        assert kvq.kvq_mla_tree_decode_kernel(p) == kernel
    n_seq, n_q, H, _ = q_lat.shape
    ws = torch.full((kvq.kvq_mla_tree_decode_workspace(p),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((n_seq, n_q, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n_seq, n_q, H), float("nan"), device="cuda")
    st = i32(1)
    kvq.kvq_mla_tree_decode(p, out, lse, ws, st)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), st.item()


def check_tree(got, ref):
    (out, lse, _), (r_out, r_lse, worst, norm) = got, ref
    empty = np.isneginf(r_lse)
    assert np.all(out[empty] == 0) and np.all(np.isneginf(lse[empty]))
    assert np.isfinite(out).all()
    err = np.abs(out - r_out)
    # fp32 scores and sums on top: 1e-4 of the largest output of the row, as kvq_mla_decode's
    slack = 1e-4 * np.abs(r_out).max(-1, keepdims=True)
    assert np.all(err <= worst + slack), f"worst element {np.max((err - worst)[~empty])}"
    # independent roundings: the row's error norm is close to its root mean square; twice that
    got_norm = np.sqrt((err**2).sum(-1))
    assert np.all(got_norm <= 2 * norm + np.sqrt(512) * slack[..., 0]), \
        f"row norm {np.max(got_norm[~empty] / norm[~empty])} of its rms"
    assert np.allclose(lse[~empty], r_lse[~empty], rtol=2e-6, atol=1e-4)


def queries(n_seq, n_q, H, seed):
    q = W.queries(n_seq, n_q, H, seed=seed)
    return dev(q.q_lat).bfloat16(), dev(q.q_rope).bfloat16()


def contiguous(lens, stride):
    return lambda s: (s * stride + np.arange(lens[s]), np.ones(lens[s], bool))


def paged(lens, page, g, spare=1):
    n = [max(1, -(-x // page)) for x in lens]
    perm = g.permutation(sum(n) + spare).astype(np.int32)
    table = np.full((len(lens), max(n) + 1), -1, np.int32)
    o = 0
    for s, k in enumerate(n):
        table[s, :k] = perm[o:o + k]
        o += k

    def rows_of(s):
        t = np.arange(lens[s])
        return table[s, t // page].astype(np.int64) * page + t % page, np.ones(lens[s], bool)
    return table, (sum(n) + spare) * page, rows_of


FORMS = [(1, 1), (1, 2), (2, 2), (4, 2), (5, 2)]          # (format, form)


@pytest.mark.parametrize("fmt,impl", FORMS)
@pytest.mark.parametrize("T,n,H,kind", [(1, 1, 1, "chain"), (2, 2, 16, "tree"), (5, 4, 3, "any"), (64, 64, 2, "tree"),
                                        (127, 7, 9, "tree"), (128, 8, 8, "chain"), (129, 1, 64, "any"),
                                        (193, 64, 1, "any"), (700, 13, 5, "tree"), (1500, 5, 30, "chain")])
def test_tree_shapes(kvq, orc, fmt, impl, T, n, H, kind):
    g = np.random.default_rng(T + n)
    signs = W.sign_bits(T)
    cache = make_cache(orc, fmt, T + 3, T, signs)
    masks = masks_of(g, [n], n, kind)
    ql, qr = queries(1, n, H, T)
    got = run_tree(kvq, fmt=fmt, cache=cache, signs=signs, lens=[T], n_node=[n], masks=masks, q_lat=ql, q_rope=qr,
                   impl=impl, kernel=impl)
    ref = tree_ref(orc, fmt, cache, signs, contiguous([T], 0), [T], [n], masks, ql.float().cpu().numpy(),
                   qr.float().cpu().numpy(), float(W.SM_SCALE))
    assert got[2] == 0
    check_tree(got, ref)


@pytest.mark.parametrize("fmt,impl,page", [(1, 1, 64), (1, 1, 8), (1, 1, 48), (1, 1, 256), (1, 0, 20), (1, 2, 64),
                                           (2, 0, 16), (5, 0, 33)])
@pytest.mark.parametrize("H", [4, 40])
def test_tree_ragged_pages_padding(kvq, orc, fmt, impl, page, H):
    """A ragged batch over a paged pool: sequences of length 0 and of fewer rows than nodes,
    padded nodes whose queries are NaN, masks with empty rows."""
    lens = [300, 0, 1, 777, 3, 128, 64, 1025]
    n_node = [9, 5, 1, 0, 6, 12, 12, 7]
    n_q = 12
    g = np.random.default_rng(page)
    signs = W.sign_bits(1)
    table, rows, rows_of = paged(lens, page, g)
    cache = make_cache(orc, fmt, rows, page, signs)
    eff = [min(a, b) for a, b in zip(n_node, lens)]
    masks = masks_of(g, eff, n_q, "any")
    ql, qr = queries(len(lens), n_q, H, 5)
    for s, n in enumerate(eff):
        ql[s, n:], qr[s, n:] = float("nan"), float("inf")
    got = run_tree(kvq, fmt=fmt, cache=cache, signs=signs, lens=lens, n_node=n_node, masks=masks, q_lat=ql, q_rope=qr,
                   table=table, page=page, impl=impl)
    ref = tree_ref(orc, fmt, cache, signs, rows_of, lens, eff, masks, ql.float().cpu().numpy(),
                   qr.float().cpu().numpy(), float(W.SM_SCALE))
    assert got[2] == 0
    check_tree(got, ref)


@pytest.mark.parametrize("n_seq,n,H,T,page,kind", [(2, 16, 33, 2400, 64, "tree"), (1, 64, 50, 1100, 0, "any"),
                                                   (40, 4, 64, 700, 16, "tree"), (3, 7, 129, 3001, 128, "chain")])
def test_tree_full_tiles(kvq, orc, n_seq, n, H, T, page, kind):
    """Problems large enough for tiles of 64 query rows: units split among CTAs, several units a
    CTA, more units than CTAs; ragged lengths and nodes; the same bits at a second call."""
    g = np.random.default_rng(T)
    signs = W.sign_bits(T)
    lens = [T] + [int(x) for x in g.integers(1, T + 1, n_seq - 1)]
    n_node = [min(int(x), L) for x, L in zip([n] + list(g.integers(1, n + 1, n_seq - 1)), lens)]
    if page:
        table, rows, rows_of = paged(lens, page, g)
    else:
        table, rows, rows_of = None, n_seq * T, contiguous(lens, T)
    cache = make_cache(orc, 1, rows, T, signs)
    masks = masks_of(g, n_node, n, kind)
    ql, qr = queries(n_seq, n, H, T)
    runs = [run_tree(kvq, fmt=1, cache=cache, signs=signs, lens=lens, n_node=n_node, masks=masks, q_lat=ql, q_rope=qr,
                     table=table, page=page, stride=T, impl=1) for _ in range(2)]
    ref = tree_ref(orc, 1, cache, signs, rows_of, lens, n_node, masks, ql.float().cpu().numpy(),
                   qr.float().cpu().numpy(), float(W.SM_SCALE))
    assert runs[0][2] == 0
    check_tree(runs[0], ref)
    assert np.array_equal(runs[0][0], runs[1][0]) and np.array_equal(runs[0][1], runs[1][1])


@pytest.mark.parametrize("impl", [1, 2])
def test_tree_many_short_sequences(kvq, orc, impl):
    """More sequences than a CTA has threads, lengths from 0 to 200."""
    n_seq, n_q, H, cap = 1500, 2, 3, 200
    g = np.random.default_rng(3)
    signs = W.sign_bits(1)
    lens = [int(x) for x in g.integers(0, cap + 1, n_seq)]
    n_node = [min(int(x), L) for x, L in zip(g.integers(0, n_q + 1, n_seq), lens)]
    cache = make_cache(orc, 1, 4096, 3, signs)
    starts = g.integers(0, 4096 // 8, (n_seq, cap // 8)).astype(np.int32)        # pages of 8, shared freely
    masks = masks_of(g, n_node, n_q, "tree")
    ql, qr = queries(n_seq, n_q, H, 2)

    def rows_of(s):
        t = np.arange(lens[s])
        return starts[s, t // 8].astype(np.int64) * 8 + t % 8, np.ones(lens[s], bool)
    got = run_tree(kvq, fmt=1, cache=cache, signs=signs, lens=lens, n_node=n_node, masks=masks, q_lat=ql, q_rope=qr,
                   table=starts, page=8, impl=impl, max_len=cap)
    ref = tree_ref(orc, 1, cache, signs, rows_of, lens, n_node, masks, ql.float().cpu().numpy(),
                   qr.float().cpu().numpy(), float(W.SM_SCALE))
    assert got[2] == 0
    check_tree(got, ref)


@pytest.mark.parametrize("impl", [1, 2])
def test_tree_missing_pages(kvq, orc, impl):
    """A page id of -1, one past the pool and a table that is too short: those rows are skipped and
    flagged, whatever lies in the buffers."""
    lens, page = [400, 400, 100], 16
    g = np.random.default_rng(8)
    signs = W.sign_bits(1)
    table, rows, _ = paged(lens, page, g)
    cache = make_cache(orc, 1, rows, 3, signs)
    table[0, 3], table[0, 24], table[1, 7] = -1, -1, rows // page + 5
    table = np.ascontiguousarray(table[:, :24])           # rows 384 .. 399 have no entry
    n_q, H = 6, 11
    n_node = [6, 6, 6]
    masks = masks_of(g, n_node, n_q, "tree")
    ql, qr = queries(3, n_q, H, 6)

    def rows_of(s):
        t = np.arange(lens[s])
        pg = np.where(t // page < 24, table[s, np.minimum(t // page, 23)], -1)
        r = pg.astype(np.int64) * page + t % page
        ok = (pg >= 0) & (r < rows)
        return np.where(ok, r, 0), ok
    got = run_tree(kvq, fmt=1, cache=cache, signs=signs, lens=lens, n_node=n_node, masks=masks, q_lat=ql, q_rope=qr,
                   table=table, page=page, impl=impl)
    ref = tree_ref(orc, 1, cache, signs, rows_of, lens, n_node, masks, ql.float().cpu().numpy(),
                   qr.float().cpu().numpy(), float(W.SM_SCALE))
    assert got[2] == BAD_PAGE
    check_tree(got, ref)


# 20 heads run in tiles of 32 query rows, 640 in tiles of 64
SIZES = pytest.mark.parametrize("impl,H", [(1, 20), (1, 640), (2, 20)])


@SIZES
def test_tree_unused_rows_and_unwritten_codes(kvq, orc, impl, H):
    """Rows behind a sequence, and rows that a node does not see, may hold NaN codes and scales; the code
    S.1111.111 in a row that is seen reads as 0."""
    T, n_q = 999, 5
    g = np.random.default_rng(9)
    signs = W.sign_bits(1)
    cache = make_cache(orc, 1, T + 64, 4, signs)
    for i, key in enumerate(("lat", "rope")):
        mask, val = W.planted_codes(cache[key][:T].shape, 0.002, seed=5 + i)
        cache[key][:T] = np.where(mask, val, cache[key][:T])
    for key in ("lat", "rope"):
        cache[key][T:] = 0x7F
    for key in ("lat_scale", "rope_scale"):
        cache[key][T:] = np.nan
    masks = masks_of(g, [n_q], n_q, "tree")
    masks &= ~np.uint64(1 << 3)                           # nobody sees node 3, whose scales are not finite
    cache["lat_scale"][T - n_q + 3], cache["rope_scale"][T - n_q + 3] = np.inf, np.nan
    ql, qr = queries(1, n_q, H, 7)
    got = run_tree(kvq, fmt=1, cache=cache, signs=signs, lens=[T], n_node=[n_q], masks=masks, q_lat=ql, q_rope=qr, impl=impl)
    host = {k: v.copy() for k, v in cache.items()}
    for key in ("lat_scale", "rope_scale"):
        host[key][~np.isfinite(host[key])] = 0.0
    ref = tree_ref(orc, 1, host, signs, contiguous([T], 0), [T], [n_q], masks, ql.float().cpu().numpy(),
                   qr.float().cpu().numpy(), float(W.SM_SCALE))
    check_tree(got, ref)


@SIZES
def test_tree_scores_far_below_zero_beside_missing_pages(kvq, impl, H):
    """Scores of about -5e31, and every page but the last third missing, so that parts of the sequence have nothing to
    add: the rows that are there, all equal, are the output."""
    T, n_q, page = 20000, 4, 16
    pages = T // page
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    table[0, 2 * pages // 3:] = torch.arange(pages - 2 * pages // 3, dtype=torch.int32, device="cuda")
    rows = (pages - 2 * pages // 3) * page
    planes = dict(lat=torch.full((rows, 512), 0x38, dtype=torch.uint8, device="cuda"),            # 1.0
                  lat_scale=torch.ones(rows, device="cuda"),
                  rope=torch.zeros(rows, 64, dtype=torch.uint8, device="cuda"), rope_scale=torch.zeros(rows, device="cuda"))
    ql = torch.full((1, n_q, H, 512), -(2.0**100), dtype=torch.bfloat16, device="cuda")
    p = kvq.make_tree_problem(seq_len=i32(1, fill=T), q_lat=ql, q_rope=torch.zeros(1, n_q, H, 64, dtype=torch.bfloat16, device="cuda"),
                              sm_scale=float(W.SM_SCALE), max_seq_len=T, fmt=1, cache=planes, block_table=table, page_size=page, impl=impl)
    ws = torch.empty(kvq.kvq_mla_tree_decode_workspace(p), dtype=torch.uint8, device="cuda")
    out, lse, st = torch.empty(1, n_q, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n_q, H, device="cuda"), i32(1)
    kvq.kvq_mla_tree_decode(p, out, lse, ws, st)
    torch.cuda.synchronize()
    score = -512 * 2.0**100 * float(W.SM_SCALE)
    assert st.item() == BAD_PAGE
    # the mean of equal rows: off by a step of fp32 a row at most, 2^-24 * 7000, below the rounding's 2^-8
    assert (out == 1.0).all()
    assert torch.allclose(lse, torch.full_like(lse, score), rtol=2e-6, atol=0)


@SIZES
@pytest.mark.parametrize("case", ["large scores", "zero queries", "zero rows", "mixed magnitudes", "one row"])
def test_tree_score_ranges(kvq, orc, impl, H, case):
    """Scores far apart (one row takes everything; running maxima that climb by many powers of
    two), all equal, and rows of zero scale."""
    T, n_q = 900, 4
    g = np.random.default_rng(11)
    signs = W.sign_bits(1)
    scale = float(W.SM_SCALE)
    data = W.magnitude_rows(T, seed=1, lo=1e-3, hi=40.0) if case == "mixed magnitudes" else W.unit_rows(T, seed=1)
    if case == "zero rows":
        data.c[::2], data.k_rope[::3] = 0.0, 0.0
    if case == "large scores":                            # magnitudes rise along the sequence
        data.c *= np.linspace(0.1, 30.0, T, dtype=np.float32)[:, None]
    cache = encode_ref(orc, 1, data.c, data.k_rope, signs)
    masks = masks_of(g, [n_q], n_q, "tree")
    ql, qr = queries(1, n_q, H, 3)
    if case == "zero queries":
        ql, qr = ql * 0, qr * 0
    if case == "one row":
        ql = (ql.float() * 30).bfloat16()
    got = run_tree(kvq, fmt=1, cache=cache, signs=signs, lens=[T], n_node=[n_q], masks=masks, q_lat=ql, q_rope=qr, impl=impl)
    ref = tree_ref(orc, 1, cache, signs, contiguous([T], 0), [T], [n_q], masks, ql.float().cpu().numpy(),
                   qr.float().cpu().numpy(), scale)
    assert got[2] == 0
    check_tree(got, ref)


@pytest.mark.parametrize("impl", [1, 2])
def test_tree_strided_queries_stream_and_no_lse(kvq, orc, impl):
    """Queries that are slices of one projection's rows, on a stream of the caller's, without lse; a chain is a
    tree whose masks are the chain's."""
    T, n_q, H, n_seq = 500, 6, 12, 2
    signs = W.sign_bits(1)
    cache = {k: dev(v) for k, v in make_cache(orc, 1, n_seq * T, 2, signs).items()}
    ql, qr = queries(n_seq, n_q, H, 4)
    both = torch.cat([ql, qr, ql[..., :32]], -1)
    chain = np.array([[(2 << j) - 1 for j in range(n_q)]] * n_seq, np.uint64)
    outs = []
    side = torch.cuda.Stream()
    for masks, q1, q2 in ((None, ql, qr), (chain, both[..., :512], both[..., 512:576])):
        p = kvq.make_tree_problem(seq_len=i32(n_seq, fill=T), mask=None if masks is None else dev(masks.view(np.int64)),
                                  q_lat=q1, q_rope=q2, sm_scale=0.07, max_seq_len=T, fmt=1, cache=cache,
                                  seq_stride_rows=T, impl=impl)
        ws = torch.empty(kvq.kvq_mla_tree_decode_workspace(p), dtype=torch.uint8, device="cuda")
        out = torch.empty(n_seq, n_q, H, 512, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        kvq.kvq_mla_tree_decode(p, out, None, ws, stream=side.cuda_stream)
        side.synchronize()
        outs.append(out)
    assert torch.equal(outs[0], outs[1])


@SIZES
def test_tree_non_finite_queries(kvq, orc, impl, H):
    """A query row with an infinity or a NaN gets NaN and leaves the others alone."""
    T, n_q = 900, 4
    signs = W.sign_bits(1)
    cache = make_cache(orc, 1, T, 2, signs)
    ql, qr = queries(1, n_q, H, 4)
    bad = [(0, 0), (0, 5), (1, 3), (2, 18), (3, 7)]
    for i, (j, h) in enumerate(bad):
        (qr if i == 3 else ql)[0, j, h, 7 * i] = (float("inf"), float("nan"), float("-inf"))[i % 3]
    out, lse, st = run_tree(kvq, fmt=1, cache=cache, signs=signs, lens=[T], n_node=[n_q], masks=None, q_lat=ql, q_rope=qr,
                            stride=T, impl=impl)
    where = torch.zeros(1, n_q, H, dtype=torch.bool)
    for j, h in bad:
        where[0, j, h] = True
    ql[where.cuda()], qr[where.cuda()] = 0, 0
    ref = tree_ref(orc, 1, cache, signs, contiguous([T], T), [T], [n_q], None, ql.float().cpu().numpy(),
                   qr.float().cpu().numpy(), float(W.SM_SCALE))
    where = where.numpy()
    assert st == 0 and np.isnan(out[where]).all() and np.isnan(lse[where]).all()
    out[where], lse[where] = ref[0][where], ref[1][where]
    check_tree((out, lse, st), ref)


@pytest.mark.parametrize("H", [20, 640])
def test_tree_non_finite_queries_touch_no_other_row(kvq, orc, H):
    """NaNs and infinities in every eighth query row (the first of each group of rows that the packed form's warps
    share), beside codes that no encoder writes: the other rows have the bits that they have when these
    rows are zero."""
    T, n_q = 1300, 4
    signs = W.sign_bits(1)
    cache = make_cache(orc, 1, T, 2, signs)
    for i, key in enumerate(("lat", "rope")):
        mask, val = W.planted_codes(cache[key].shape, 2e-5, seed=5 + i)
        cache[key] = np.where(mask, val, cache[key])
    ql, qr = queries(1, n_q, H, 4)
    flat_l, flat_r = ql.view(-1, 512), qr.view(-1, 64)
    bad = torch.arange(0, n_q * H, 8, device="cuda")
    kw = dict(fmt=1, cache=cache, signs=signs, lens=[T], n_node=[n_q], masks=None, q_lat=ql, q_rope=qr, stride=T, impl=1)
    flat_l[bad], flat_r[bad] = 0, 0
    want = run_tree(kvq, **kw)
    for i, r in enumerate(bad.tolist()):
        (flat_r if i % 4 == 3 else flat_l)[r, 5 * i % 64] = (float("nan"), float("inf"), float("-inf"))[i % 3]
    got = run_tree(kvq, **kw)
    hit = np.zeros(n_q * H, bool)
    hit[::8] = True
    hit = hit.reshape(1, n_q, H)
    assert got[2] == want[2] == 0
    assert np.isnan(got[0][hit]).all() and np.isnan(got[1][hit]).all()
    assert np.array_equal(got[0][~hit], want[0][~hit]) and np.array_equal(got[1][~hit], want[1][~hit])


@pytest.mark.parametrize("n_seq,H", [(1, 16), (3, 200)])
def test_tree_waits_give_up_then_recover(kvq, orc, n_seq, H):
    """With the limit of the pipeline's waits cut to 200 ns the call still returns, sets KVQ_DEV_TIMEOUT and
    leaves rows that are NaN whole or right; with the default limit the next call is right again."""
    T, n_q = 5000, 4
    g = np.random.default_rng(6)
    signs = W.sign_bits(1)
    host = make_cache(orc, 1, n_seq * T, 7, signs)
    cache = {k: dev(v) for k, v in host.items()}
    masks = masks_of(g, [n_q] * n_seq, n_q, "tree")
    ql, qr = queries(n_seq, n_q, H, 8)
    kw = dict(fmt=1, cache=cache, signs=signs, lens=[T] * n_seq, n_node=[n_q] * n_seq, masks=masks, q_lat=ql, q_rope=qr,
              stride=T, impl=1)
    ref = tree_ref(orc, 1, host, signs, contiguous([T] * n_seq, T), [T] * n_seq, [n_q] * n_seq, masks,
                   ql.float().cpu().numpy(), qr.float().cpu().numpy(), float(W.SM_SCALE))
    assert kvq.lib().kvq_set_wait_limit_ns(200) == 0
    try:
        out, lse, st = run_tree(kvq, **kw)
    finally:
        assert kvq.lib().kvq_set_wait_limit_ns(0) == 0
    assert st & kvq.DEV_TIMEOUT
    gone = np.isnan(out).all(-1)
    assert gone.any() and np.array_equal(gone, np.isnan(lse)) and np.array_equal(gone, np.isnan(out).any(-1))
    out[gone], lse[gone] = ref[0][gone], ref[1][gone]
    check_tree((out, lse, st), ref)
    got = run_tree(kvq, **kw)
    assert got[2] == 0
    check_tree(got, ref)


@pytest.mark.parametrize("H", [20, 640])
def test_tree_moving_maxima_and_small_pages_repeat(kvq, orc, H):
    """Scores that rise tile after tile, so that the running maxima move in each, over pages of 8 rows, whose
    addresses the lanes of a warp look up for the thread that issues the copies: the formula's values,
    and the same bits at every call."""
    T, n_q, page = 2600, 4, 8
    g = np.random.default_rng(13)
    signs = W.sign_bits(1)
    data = W.unit_rows(T, seed=2)
    data.c *= np.linspace(0.1, 20.0, T, dtype=np.float32)[:, None]
    table, rows, rows_of = paged([T], page, g)
    r, _ = rows_of(0)
    enc = encode_ref(orc, 1, data.c, data.k_rope, signs)
    cache = {k: np.zeros((rows,) + v.shape[1:], v.dtype) for k, v in enc.items()}
    for k, v in enc.items():
        cache[k][r] = v
    masks = masks_of(g, [n_q], n_q, "tree")
    ql, qr = queries(1, n_q, H, 9)
    kw = dict(fmt=1, cache={k: dev(v) for k, v in cache.items()}, signs=signs, lens=[T], n_node=[n_q], masks=masks,
              q_lat=ql, q_rope=qr, table=table, page=page, impl=1)
    got = run_tree(kvq, **kw)
    ref = tree_ref(orc, 1, cache, signs, rows_of, [T], [n_q], masks, ql.float().cpu().numpy(), qr.float().cpu().numpy(),
                   float(W.SM_SCALE))
    assert got[2] == 0
    check_tree(got, ref)
    for _ in range(10):
        again = run_tree(kvq, **kw)
        assert np.array_equal(again[0], got[0]) and np.array_equal(again[1], got[1])


def heavy_tail_cache(T, seed):
    """fp8 rows with a common mean; rope keys whose element 0 is N(0,1) and whose elements 1, 2, 3 single out
    the first, a middle and the last row but eight (256 there, 0 elsewhere)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    c = rnd(1, 512) + rnd(T, 512)
    k = torch.zeros(T, 64, device="cuda")
    k[:, 0] = rnd(T)
    for i, t in enumerate((0, T // 2 + 5, T - 9)):
        k[t] = 0
        k[t, 1 + i] = 256.0
    ls, rs = c.abs().amax(1) / 448.0, k.abs().amax(1) / 448.0
    code = lambda x, s: (x / s.clamp(min=1e-30)[:, None]).to(torch.float8_e4m3fn)
    lat, rope = code(c, ls), code(k, rs)
    cache = dict(lat=lat.view(torch.uint8), lat_scale=ls, rope=rope.view(torch.uint8), rope_scale=rs)
    return cache, lat.double() * ls.double()[:, None], rope.double() * rs.double()[:, None]


@pytest.mark.parametrize("impl,n_q,many", [(1, 2, True), (1, 4, True), (1, 4, False), (2, 4, False)])
@pytest.mark.parametrize("T", [1000, 4096, 14001, 32768, 65536])
def test_tree_heavy_row_and_broad_tail(kvq, impl, n_q, many, T):
    """A long context as it is met: one row holds 0 to 99.9% of a query's weight, the rest is spread over all
    others, whose latents share a mean, so that lost or rounded weights of the tail add up instead of
    averaging out.  In tiles of 32 and 64 query rows, with a unit in one stretch (as many equal sequences as SMs,
    sharing their pages) and cut into many, and per query.

    Bounds, relative to the output's norm, none of which grows with T.  Rounding of the output: 2^-8 an
    element at most, so 2^-8 / sqrt(3) in the root mean square.  Weights of the heavy row and of a tail of equal
    weights may all be off the same way, by 2^-8 of themselves, but one of the two sets the scale and is exact, so the
    mixture is off by 2^-8 / 4 of the two parts' difference at most, 2^-9 of the output with a tail of at least its
    norm.  Below 2^-12 of the largest, weights are off by 2^-19 of it at random: sqrt(65536) 2^-19 = 2^-11.
    Together under 2^-8.  The share along the right direction, where the roundings of 512 elements
    average to 2^-8 / sqrt(3 512) each, six of them 2^-10.7: 2^-9 + 2^-10."""
    page, H, n_seq = 64, 16, torch.cuda.get_device_properties(0).multi_processor_count if many else 1
    cache, c, k = heavy_tail_cache(T, T + n_q)
    pad = -T % page
    cache = {key: torch.cat([v, v[:pad]]).contiguous() for key, v in cache.items()}
    scale = float(W.SM_SCALE)
    spread = [0.0, 0.3, 1.0, 2.5]                               # standard deviation of the tail's scores, in nats
    share = [0.0, 0.5, 0.9, 0.99, 0.999]
    ql = torch.zeros(n_q, H, 512, device="cuda")
    qr = torch.zeros(n_q, H, 64, device="cuda")
    for j in range(n_q):
        for h in range(H):
            i = H * j + h
            qr[j, h, 0] = spread[i % 4] / scale
            p = share[i % 5]
            tail = torch.logsumexp(scale * qr[j, h, 0].bfloat16().double() * k[:, 0], 0).item()
            for at in range(3):
                want = tail + np.log(p / (1 - p)) if p > 0 and at == i % 3 else 0.0
                qr[j, h, 1 + at] = want / (256.0 * scale)
    ql, qr = ql.bfloat16()[None].repeat(n_seq, 1, 1, 1), qr.bfloat16()[None].repeat(n_seq, 1, 1, 1)
    order = torch.randperm((T + pad) // page, generator=torch.Generator().manual_seed(T)).int().cuda()
    paged_cache = {}
    for key, v in cache.items():
        w = torch.empty_like(v).view(-1, page, *v.shape[1:])
        w[order.long()] = v.view(-1, page, *v.shape[1:])
        paged_cache[key] = w.view(v.shape)
    p = kvq.make_tree_problem(seq_len=i32(n_seq, fill=T), q_lat=ql, q_rope=qr, sm_scale=scale, max_seq_len=T, fmt=1,
                              cache=paged_cache, block_table=order[None].repeat(n_seq, 1), page_size=page, impl=impl)
    assert kvq.kvq_mla_tree_decode_kernel(p) == impl
    ws = torch.empty(kvq.kvq_mla_tree_decode_workspace(p), dtype=torch.uint8, device="cuda")
    out = torch.empty(n_seq, n_q, H, 512, dtype=torch.bfloat16, device="cuda")
    lse, st = torch.empty(n_seq, n_q, H, device="cuda"), i32(1)
    kvq.kvq_mla_tree_decode(p, out, lse, ws, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    worst = 0.0
    for j in range(n_q):
        L = T - n_q + j + 1
        sc = scale * (ql[0, j].double() @ c[:L].T + qr[0, j].double() @ k[:L].T)
        ref = torch.softmax(sc, 1) @ c[:L]
        got = out[:, j].double()
        assert torch.allclose(lse[:, j].double(), torch.logsumexp(sc, 1).expand(n_seq, H), rtol=2e-6, atol=1e-4)
        err = (got - ref).norm(dim=-1) / ref.norm(dim=-1)
        along = ((got * ref).sum(-1) / (ref * ref).sum(-1) - 1).abs()
        worst = max(worst, err.max().item())
        assert err.max() < 2.0**-8, f"node {j}: {err.max(0).values.tolist()}"
        assert along.max() < 2.0**-9 + 2.0**-10, f"node {j}: {along.max(0).values.tolist()}"
    print(f"worst |error| / |output| {worst:.5f}")


def test_tree_two_calls_at_once(kvq, orc):
    """Calls on two streams with their own workspaces do not touch one another."""
    T, n_q, H = 3000, 8, 64
    signs = W.sign_bits(1)
    cache = {k: dev(v) for k, v in make_cache(orc, 1, T, 9, signs).items()}
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for i in range(2):
        ql, qr = queries(1, n_q, H, 30 + i)
        p = kvq.make_tree_problem(seq_len=i32(1, fill=T), q_lat=ql, q_rope=qr, sm_scale=0.07, max_seq_len=T, fmt=1, cache=cache)
        ws = torch.empty(kvq.kvq_mla_tree_decode_workspace(p), dtype=torch.uint8, device="cuda")
        outs = [torch.empty(1, n_q, H, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        jobs.append((p, ws, outs))
    torch.cuda.synchronize()
    for p, ws, outs in jobs:
        kvq.kvq_mla_tree_decode(p, outs[0], None, ws)
    torch.cuda.synchronize()
    for _ in range(5):
        for (p, ws, outs), s in zip(jobs, streams):
            kvq.kvq_mla_tree_decode(p, outs[1], None, ws, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for _, _, outs in jobs:
        assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("fmt,impl", [(1, 1), (1, 2), (2, 2)])
def test_tree_graph_replays_new_lengths(kvq, orc, fmt, impl):
    """A captured call reads lengths, tables, masks and queries at replay; two captured calls
    that share a workspace may be replayed in turn."""
    page, n_q, H, cap = 64, 8, 16, 2000
    g = np.random.default_rng(12)
    signs = W.sign_bits(1)
    table, rows, _ = paged([cap, cap], page, g)
    host = make_cache(orc, fmt, rows, 6, signs)
    cache = {k: dev(v) for k, v in host.items()}
    sl, nn, tb = i32(2), i32(2), dev(table)
    mk = torch.zeros(2, n_q, dtype=torch.int64, device="cuda")
    graphs, outs = [], []
    problems = []
    for i in range(2):
        ql, qr = queries(2, n_q, H, 20 + i)
        problems.append((ql, qr, kvq.make_tree_problem(seq_len=sl, n_node=nn, mask=mk, q_lat=ql, q_rope=qr, sm_scale=0.07,
                                                       max_seq_len=cap, fmt=fmt, cache=cache, signs=dev(signs.view(np.int32)),
                                                       block_table=tb, page_size=page, impl=impl)))
    ws = torch.empty(kvq.kvq_mla_tree_decode_workspace(problems[0][2]), dtype=torch.uint8, device="cuda")
    for ql, qr, p in problems:
        out = torch.empty(2, n_q, H, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(2, n_q, H, device="cuda")
        kvq.kvq_mla_tree_decode(p, out, lse, ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            kvq.kvq_mla_tree_decode(p, out, lse, ws)
        graphs.append(gr)
        outs.append((out, lse))
    for lens, nodes in (([1999, 5], [8, 3]), ([64, 1300], [1, 8]), ([0, 2000], [8, 5])):
        eff = [min(a, b) for a, b in zip(nodes, lens)]
        masks = masks_of(g, eff, n_q, "tree")
        sl.copy_(torch.tensor(lens))
        nn.copy_(torch.tensor(nodes))
        mk.copy_(torch.from_numpy(masks.view(np.int64)))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for (ql, qr, _), (out, lse) in zip(problems, outs):
            def rows_of(s):
                t = np.arange(lens[s])
                return table[s, t // page].astype(np.int64) * page + t % page, np.ones(lens[s], bool)
            ref = tree_ref(orc, fmt, host, signs, rows_of, lens, eff, masks, ql.float().cpu().numpy(),
                           qr.float().cpu().numpy(), 0.07)
            check_tree((out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64), 0), ref)


def test_tree_empty_calls(kvq):
    planes = empty_planes(1, 64)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    for n_seq, max_len in ((0, 8), (3, 0)):
        p = kvq.make_tree_problem(seq_len=i32(n_seq, fill=5), q_lat=z(n_seq, 2, 4, 512), q_rope=z(n_seq, 2, 4, 64),
                                  sm_scale=0.1, max_seq_len=max_len, fmt=1, cache=planes, seq_stride_rows=8)
        ws = torch.empty(max(1, kvq.kvq_mla_tree_decode_workspace(p)), dtype=torch.uint8, device="cuda")
        out, lse = torch.ones_like(z(n_seq, 2, 4, 512)), torch.ones(n_seq, 2, 4, device="cuda")
        kvq.kvq_mla_tree_decode(p, out, lse, ws)
        torch.cuda.synchronize()
        assert (out == 0).all() and (lse == -float("inf")).all()


# --- accept --------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [1, 2, 4, 5])
@pytest.mark.parametrize("page", [0, 16, 25])
def test_accept_moves_rows(kvq, fmt, page):
    """Paths of every length; bad entries end a path; rows elsewhere keep their bytes."""
    g = np.random.default_rng(fmt + page)
    n_q, n_seq = 64, 9
    lens = [64, 200, 150, 3, 0, 90, 91, 92, 128]
    n_node = [64, 64, 10, 10, 4, 20, 20, 20, 33]
    path = np.full((n_seq, n_q), -9, np.int32)
    acc = [64, 20, 10, 2, 1, 0, 12, 12, 99]
    eff = [min(a, b) for a, b in zip(n_node, lens)]
    for s in range(n_seq):
        a = min(max(acc[s], 0), eff[s])
        path[s, :a] = np.sort(g.choice(eff[s], a, replace=False)) if a else []
    path[6, 5], path[7, 3] = path[6, 4], 20               # not larger; not a node
    if page:
        table, rows, rows_of = paged(lens, page, g)
    else:
        table, rows, rows_of = None, n_seq * 200, contiguous(lens, 200)
    host = dict(lat=g.integers(0, 256, (rows, ROW_BYTES[fmt]), dtype=np.uint8), lat_scale=g.random(rows, dtype=np.float32),
                rope=g.integers(0, 256, (rows, 64), dtype=np.uint8), rope_scale=g.random(rows, dtype=np.float32))
    planes = {k: dev(v) for k, v in host.items()}
    sl, st = dev(np.array(lens, np.int32)), i32(1)
    d = kvq.make_accept(seq_len=sl, n_node=dev(np.array(n_node, np.int32)), path=dev(path),
                        n_acc=dev(np.array(acc, np.int32)), new_len=sl, fmt=fmt, cache=planes,
                        block_table=None if table is None else dev(table), page_size=page, seq_stride_rows=200)
    kvq.kvq_accept_mla(d, st)
    torch.cuda.synchronize()
    want = {k: v.copy() for k, v in host.items()}
    want_len = []
    for s in range(n_seq):
        base, a = lens[s] - eff[s], min(max(acc[s], 0), eff[s])
        bad = [k for k in range(a) if not 0 <= path[s, k] < eff[s] or (k and path[s, k] <= path[s, k - 1])]
        a = min([a] + bad)
        r, _ = rows_of(s)
        for k in range(a):
            for key in want:
                want[key][r[base + k]] = host[key][r[base + path[s, k]]]
        want_len.append(base + a)
    assert sl.tolist() == want_len
    for key in want:
        assert np.array_equal(planes[key].cpu().numpy(), want[key]), key
    assert st.item() == BAD_INDEX


def test_accept_missing_page(kvq):
    planes = empty_planes(1, 64)
    planes["lat"][:] = torch.arange(64, device="cuda", dtype=torch.uint8)[:, None]
    table = dev(np.array([[0, -1, 2, 9]], np.int32))
    sl, st = i32(1, fill=32), i32(1)
    d = kvq.make_accept(seq_len=sl, path=dev(np.array([[0, 9, 17, 25] + [0] * 24], np.int32)), n_acc=i32(1, fill=4),
                        new_len=i32(1), fmt=1, cache=planes, block_table=table, page_size=8)
    before = planes["lat"].clone()
    kvq.kvq_accept_mla(d, st)                             # base 4: rows 4, 13 (no page), 21 -> 6, 29 (past the pool)
    torch.cuda.synchronize()
    before[6] = before[16 + 21 % 8]
    assert st.item() == BAD_PAGE and torch.equal(planes["lat"], before) and d._keep[4].tolist() == [8]


# --- a run of steps ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [1, 2])
def test_steps_together(kvq, orc, fmt):
    """Draft, append, attend, accept and roll back, step after step as a server does it, one captured
    graph a step replayed with the device's own lengths; the cache is checked against rows
    kept on the host, the attention against the formula."""
    n_seq, n_q, H, page, n_pages = 3, 6, 8, 16, 40
    g = np.random.default_rng(fmt)
    signs = W.sign_bits(4)
    d_signs = dev(signs.view(np.int32))
    planes = empty_planes(fmt, n_pages * page, fill=0)
    for k in ("lat_scale", "rope_scale"):
        planes[k].zero_()
    table, held, free, n_free = i32(n_seq, n_pages, fill=-1), i32(n_seq), dev(g.permutation(n_pages).astype(np.int32)), i32(1, fill=n_pages)
    keep, new, seq_len, start = i32(n_seq), i32(n_seq), i32(n_seq), i32(n_seq + 1)
    cap = 64
    slots, st = i32(cap), i32(1)
    x = torch.zeros(cap, 512, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(cap, 64, dtype=torch.bfloat16, device="cuda")
    mk = torch.zeros(n_seq, n_q, dtype=torch.int64, device="cuda")
    ql, qr = queries(n_seq, n_q, H, 1)
    path, acc = i32(n_seq, n_q), i32(n_seq)
    plan = kvq.make_page_plan(keep_len=keep, n_new=new, block_table=table, n_held=held, free_list=free, n_free=n_free,
                              page_size=page, seq_len=seq_len, tok_start=start, slot_map=slots)
    prob = kvq.make_tree_problem(seq_len=seq_len, n_node=new, mask=mk, q_lat=ql, q_rope=qr, sm_scale=0.07, max_seq_len=n_pages * page,
                                 fmt=fmt, cache=planes, signs=d_signs, block_table=table, page_size=page)
    ws = torch.empty(kvq.kvq_mla_tree_decode_workspace(prob), dtype=torch.uint8, device="cuda")
    out = torch.empty(n_seq, n_q, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n_seq, n_q, H, device="cuda")
    done = kvq.make_accept(seq_len=seq_len, n_node=new, path=path, n_acc=acc, new_len=keep, fmt=fmt, cache=planes,
                           block_table=table, page_size=page)

    def step():
        kvq.kvq_resize_pages(plan, st)
        kvq.kvq_append_mla(x, k, slots, fmt, d_signs, planes, st)
        kvq.kvq_mla_tree_decode(prob, out, lse, ws, st)
        kvq.kvq_accept_mla(done, st)

    # prompts: appended in one call, nothing attended
    prompt = [33, 1, 16]
    rows = [[] for _ in range(n_seq)]
    keep.zero_()
    new.copy_(torch.tensor(prompt))
    kvq.kvq_resize_pages(plan, st)
    hx = torch.randn(cap, 576).bfloat16()
    x.copy_(hx[:, :512])
    k.copy_(hx[:, 512:])
    kvq.kvq_append_mla(x, k, slots, fmt, d_signs, planes, st)
    o = 0
    for s, n in enumerate(prompt):
        rows[s] = [hx[o + t].float().numpy() for t in range(n)]
        o += n
    keep.copy_(seq_len)
    torch.cuda.synchronize()
    graph = None
    for it in range(5):
        n_new = [int(v) for v in g.integers(1, n_q + 1, n_seq)]
        masks = masks_of(g, n_new, n_q, "tree")
        new.copy_(torch.tensor(n_new))
        mk.copy_(torch.from_numpy(masks.view(np.int64)))
        hx = torch.randn(cap, 576).bfloat16()
        x.copy_(hx[:, :512])
        k.copy_(hx[:, 512:])
        paths = np.zeros((n_seq, n_q), np.int32)
        accepted = []
        for s, n in enumerate(n_new):
            node = int(g.integers(0, n))
            p = [t for t in range(n) if (int(masks[s, node]) >> t) & 1]        # the node and its ancestors
            paths[s, :len(p)] = p
            accepted.append(p)
        path.copy_(torch.from_numpy(paths))
        acc.copy_(torch.tensor([len(p) for p in accepted]))
        if it == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        o = 0
        lens = []
        for s, n in enumerate(n_new):
            drafted = [hx[o + t].float().numpy() for t in range(n)]
            o += n
            full = np.stack(rows[s] + drafted)
            lens.append(len(full))
            ref = tree_ref(orc, fmt, encode_ref(orc, fmt, np.ascontiguousarray(full[:, :512]), np.ascontiguousarray(full[:, 512:]), signs),
                           signs, lambda _: (np.arange(len(full)), np.ones(len(full), bool)), [len(full)], [n], masks[s:s + 1],
                           ql[s:s + 1].float().cpu().numpy(), qr[s:s + 1].float().cpu().numpy(), 0.07)
            check_tree((out[s:s + 1].float().cpu().numpy().astype(np.float64), lse[s:s + 1].cpu().numpy().astype(np.float64), 0), ref)
            rows[s] += [drafted[t] for t in accepted[s]]
        assert seq_len.tolist() == lens and keep.tolist() == [len(r) for r in rows]
        # the cache holds exactly the accepted rows
        t_host = table.cpu().numpy()
        for s in range(n_seq):
            full = np.stack(rows[s])
            want = encode_ref(orc, fmt, np.ascontiguousarray(full[:, :512]), np.ascontiguousarray(full[:, 512:]), signs)
            t = np.arange(len(full))
            r = t_host[s, t // page].astype(np.int64) * page + t % page
            for key in want:
                assert np.array_equal(planes[key].cpu().numpy()[r], want[key])
    # every sequence ends: all pages come back
    keep.zero_()
    new.zero_()
    kvq.kvq_resize_pages(plan, st)
    torch.cuda.synchronize()
    assert n_free.item() == n_pages and sorted(free.tolist()) == list(range(n_pages)) and (table == -1).all()
