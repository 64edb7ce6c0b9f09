"""The operators that serve drafted tokens over a paged, quantized MLA cache: their cases,
inputs, plain forms and costs.

  pages   a step of the page allocator: block tables and the slot map from request lengths,
          then the roll-back that returns the pages of the rejected tokens
  append  new MLA rows quantized and written at the pool rows of a slot map
  tree    absorbed latent attention of a tree of drafted tokens over the cache
  accept  the rows of the accepted path moved to the front of the draft

Every cache row is a 512-wide latent in its tier (fp8, or the rotated 4-bit tier) and a
64-wide rope key in fp8.
"""
import math

import numpy as np
import torch

own = False

D_LAT, D_ROPE = 512, 64
SM_SCALE = 1.0 / math.sqrt(192.0)
FMT_FP8, FMT_TQ4 = 1, 2
# the 16-level N(0,1) Lloyd-Max codebook of the rotated tier, in binary16 (positive half)
TQ4_HALF = [float.fromhex(h) for h in ("0x1.07p-3", "0x1.8d4p-2", "0x1.504p-1", "0x1.e28p-1", "0x1.418p+0",
                                       "0x1.9e4p+0", "0x1.08cp+1", "0x1.5dcp+1")]


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one draft step of a small batch: 8 sequences, 16 drafted tokens each
        dict(name="pages_step", op="pages", n_seq=8, new=16, keep=4000, page=64),
        # admission of a large batch of ragged prompts
        dict(name="pages_prompts", op="pages", n_seq=512, new=2048, keep=0, page=64),
        # the drafted tokens of a small batch (padded with -1 slots), fp32 rows as the codecs take
        dict(name="append_step", op="append", fmt=FMT_FP8, rows=61, bf16=False, page=64),
        # the prompts of a batch, bfloat16 rows as a model's projection writes them
        dict(name="append_prompt", op="append", fmt=FMT_FP8, rows=65536, bf16=True, page=64),
        # a chunk of a prompt into the rotated 4-bit tier
        dict(name="append_tq4", op="append", fmt=FMT_TQ4, rows=4099, bf16=True, page=16),
        # a short context and a small draft: latency
        dict(name="tree_small", op="tree", fmt=FMT_FP8, n_seq=1, nodes=4, heads=16, T=1024, ragged=False,
             page=0, chain=False),
        # a batch of trees at the 32768-row context of the decode benchmark, 64 heads
        dict(name="tree_batch", op="tree", fmt=FMT_FP8, n_seq=4, nodes=16, heads=64, T=32768, ragged=False,
             page=64, chain=False),
        # one long sequence, 128 heads, a short chain of drafted tokens
        dict(name="tree_long", op="tree", fmt=FMT_FP8, n_seq=1, nodes=5, heads=128, T=131072, ragged=False,
             page=64, chain=True),
        # the ragged batch: 32 sequences of 1024 to 65536 rows, trees of up to 32 nodes
        dict(name="tree_ragged", op="tree", fmt=FMT_FP8, n_seq=32, nodes=32, heads=64, T=65536, ragged=True,
             page=64, chain=False),
        # the rotated 4-bit tier, odd head count and small pages
        dict(name="tree_tq4", op="tree", fmt=FMT_TQ4, n_seq=2, nodes=9, heads=20, T=8190, ragged=True,
             page=16, chain=False),
        # after the verification of one small tree
        dict(name="accept_one", op="accept", fmt=FMT_FP8, n_seq=1, nodes=16, T=1000, page=0),
        # after the verification of a large batch of full trees, every plane moved
        dict(name="accept_batch", op="accept", fmt=FMT_FP8, n_seq=512, nodes=64, T=2048, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "append", "tree", "tree", "tree", "accept"])
    if op == "pages":
        return dict(op=op, n_seq=_log(rng, 1, 600), new=_log(rng, 1, 1700), keep=rng.choice([0, _log(rng, 1, 8000)]),
                    page=rng.choice([8, 16, 48, 64, 128]))
    if op == "append":
        fmt = rng.choice([FMT_FP8, FMT_FP8, FMT_TQ4])
        return dict(op=op, fmt=fmt, rows=_log(rng, 1, 60000 if fmt == FMT_FP8 else 8000), bf16=rng.random() < 0.5,
                    page=rng.choice([16, 64, 100]))
    if op == "accept":
        return dict(op=op, fmt=rng.choice([FMT_FP8, FMT_TQ4]), n_seq=_log(rng, 1, 400), nodes=rng.randint(2, 64),
                    T=_log(rng, 70, 2048), page=rng.choice([0, 16, 64, 100]))
    fmt = rng.choice([FMT_FP8, FMT_FP8, FMT_FP8, FMT_TQ4])
    c = dict(op=op, fmt=fmt, n_seq=_log(rng, 1, 24), nodes=_log(rng, 1, 64), heads=_log(rng, 2, 128),
             T=_log(rng, 64, 60000), ragged=rng.random() < 0.5, page=rng.choice([0, 16, 40, 64, 128]),
             chain=rng.random() < 0.3)
    most = 1 << 30 if fmt == FMT_FP8 else 32 * 64 * 32768   # query rows x cache rows
    while c["n_seq"] * c["nodes"] * c["heads"] * c["T"] > most:
        key = max(("n_seq", "nodes", "heads", "T"), key=lambda k: c[k] / dict(n_seq=1, nodes=2, heads=8, T=512)[k])
        c[key] = max(1, c[key] // 2)
    return c


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < D_LAT:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _codebook(dtype):
    up = torch.tensor(TQ4_HALF, dtype=dtype, device="cuda")
    return torch.cat([-up.flip(0), up])


def _lengths(case, g):
    if not case.get("ragged"):
        return [case["T"]] * case["n_seq"]
    return [int(x) for x in g.integers(max(1, case["T"] // 64), case["T"] + 1, case["n_seq"])]


def _table(lens, page, g):
    """Page ids in a random order, -1 past a sequence's pages; and the pool's row count."""
    n = [max(1, -(-int(x) // page)) for x in lens]
    perm = g.permutation(sum(n)).astype(np.int32)
    t = np.full((len(lens), max(n)), -1, np.int32)
    o = 0
    for s, k in enumerate(n):
        t[s, :k] = perm[o:o + k]
        o += k
    return t, sum(n) * page


def _random_cache(fmt, rows, gen):
    """Planes of `rows` rows: N(0,1) rows times a magnitude log-uniform in [1e-2, 10], quantized."""
    planes = dict(lat=torch.empty(rows, 512 if fmt == FMT_FP8 else 256, dtype=torch.uint8, device="cuda"),
                  lat_scale=torch.empty(rows, device="cuda"),
                  rope=torch.empty(rows, D_ROPE, dtype=torch.uint8, device="cuda"),
                  rope_scale=torch.empty(rows, device="cuda"))
    for a in range(0, rows, 65536):
        b = min(rows, a + 65536)
        mag = torch.exp(torch.empty(b - a, 1, device="cuda").uniform_(math.log(1e-2), math.log(10.0), generator=gen))
        c = torch.randn(b - a, D_LAT, device="cuda", generator=gen) * mag
        k = torch.randn(b - a, D_ROPE, device="cuda", generator=gen) * mag
        if fmt == FMT_FP8:
            s = c.abs().amax(1) / 448.0
            planes["lat"][a:b] = (c / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            planes["lat_scale"][a:b] = s
        else:                               # the rotation of a N(0,1) row is a N(0,1) row
            r = c.pow(2).sum(1).sqrt()
            cb = _codebook(torch.float32)
            code = torch.bucketize(c / (r[:, None] / math.sqrt(512.0)), (cb[1:] + cb[:-1]) / 2).to(torch.uint8)
            planes["lat"][a:b] = code[:, 0::2] | (code[:, 1::2] << 4)
            planes["lat_scale"][a:b] = r
        s = k.abs().amax(1) / 448.0
        planes["rope"][a:b] = (k / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        planes["rope_scale"][a:b] = s
    return planes


def _tree_masks(n_node, nodes, g):
    """Ancestor masks of random trees: node j hangs under an earlier node, bit k of mask j is
    set where node k is j or an ancestor of j."""
    out = np.zeros((len(n_node), nodes), np.uint64)
    for s, n in enumerate(n_node):
        for j in range(n):
            up = int(out[s, int(g.integers(0, j))]) if j else 0
            out[s, j] = np.uint64(up | (1 << j))
    return out.view(np.int64)


def _signs(g):
    return g.integers(0, 2, D_LAT)


def _sign_words(bits):
    w = np.zeros(D_LAT // 32, np.uint64)
    for i, b in enumerate(bits):
        w[i // 32] |= np.uint64(int(b)) << np.uint64(i % 32)
    return torch.from_numpy(w.astype(np.uint32).view(np.int32)).cuda()


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def prepare(case, seed):
    g = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "pages":
        n, ps = case["n_seq"], case["page"]
        keep = g.integers(case["keep"] // 2, case["keep"] + 1, n).astype(np.int32)
        new = g.integers((case["new"] + 1) // 2, case["new"] + 1, n).astype(np.int32)
        held = -(-keep // ps)
        most = -(-(case["keep"] + case["new"]) // ps)
        total, max_pages = n * most + 5, most + 3
        perm = g.permutation(total).astype(np.int32)
        table = np.full((n, max_pages), -1, np.int32)
        o = 0
        for s in range(n):
            table[s, :held[s]] = perm[o:o + held[s]]
            o += held[s]
        free = np.full(total, -1, np.int32)
        free[:total - o] = perm[o:]
        tokens = n * case["new"] + 7                      # a padded step: the last slots stay -1
        st.update(keep=_dev(keep), new=_dev(new), zero=_dev(np.zeros(n, np.int32)), table=_dev(table),
                  held=_dev(held.astype(np.int32)), free=_dev(free), n_free=_dev(np.array([total - o], np.int32)),
                  n_pages=total, max_tokens=tokens, n_seq=n, max_pages=max_pages)
        i32 = dict(dtype=torch.int32, device="cuda")
        for k in ("grow", "back"):
            st[k] = dict(seq_len=torch.empty(n, **i32), tok_start=torch.empty(n + 1, **i32),
                         slot_map=torch.empty(tokens if k == "grow" else 1, **i32),
                         tok_pos=torch.empty(tokens if k == "grow" else 1, **i32))
        if own:
            import quantized_kv_cache_fp8_gb300 as kvq
            kw = dict(block_table=st["table"], n_held=st["held"], free_list=st["free"], n_free=st["n_free"],
                      page_size=ps, keep_len=st["keep"])
            st["plan_grow"] = kvq.make_page_plan(n_new=st["new"], **st["grow"], **kw)
            st["plan_back"] = kvq.make_page_plan(n_new=st["zero"], **st["back"], **kw)
    elif op == "append":
        n, ps, fmt = case["rows"], case["page"], case["fmt"]
        pages = -(-n // ps) + 3
        rows = pages * ps
        ids = g.permutation(pages)[: -(-n // ps)]
        slot = (ids[:, None] * ps + np.arange(ps)[None, :]).reshape(-1)[:n].astype(np.int32)
        slot[g.random(n) < 0.03] = -1                     # tokens of refused sequences, padding
        mag = torch.exp(torch.empty(n, 1, device="cuda").uniform_(math.log(1e-2), math.log(10.0), generator=gen))
        x = torch.randn(n, D_LAT, device="cuda", generator=gen) * mag
        k = torch.randn(n, D_ROPE, device="cuda", generator=gen) * mag
        dt = torch.bfloat16 if case["bf16"] else torch.float32
        bits = _signs(g)
        # one row more than the pool: where the plain form puts the rows without a slot
        st.update(x=x.to(dt), k=k.to(dt), slot=_dev(slot), rows=rows, sign_words=_sign_words(bits),
                  sign=_dev(1.0 - 2.0 * bits).float(),
                  planes=dict(lat=torch.zeros(rows + 1, 512 if fmt == FMT_FP8 else 256, dtype=torch.uint8, device="cuda"),
                              lat_scale=torch.zeros(rows + 1, device="cuda"),
                              rope=torch.zeros(rows + 1, D_ROPE, dtype=torch.uint8, device="cuda"),
                              rope_scale=torch.zeros(rows + 1, device="cuda")))
        cb = _codebook(torch.float16)
        b = torch.arange(256, device="cuda")
        st["pairs"] = torch.stack([cb[b & 15], cb[b >> 4]], 1)      # the two centroids of a packed byte
    else:
        lens = _lengths(case, g)
        page = case["page"]
        n_node = [min(case["nodes"], L) if not case.get("ragged") else int(g.integers(1, min(case["nodes"], L) + 1))
                  for L in lens]
        if page:
            table, rows = _table(lens, page, g)
            st["table"] = _dev(table)
        else:
            rows = max(lens) * len(lens)
            st["table"] = None
        st.update(lens=lens, nodes=n_node, stride=max(lens), rows=rows,
                  seq_len=_dev(np.array(lens, np.int32)), n_node=_dev(np.array(n_node, np.int32)),
                  planes=_random_cache(case["fmt"], rows, gen))
        if op == "tree":
            bits = _signs(g)
            n, nq, H = case["n_seq"], case["nodes"], case["heads"]
            st.update(q_lat=torch.randn(n, nq, H, D_LAT, device="cuda", generator=gen).bfloat16(),
                      q_rope=torch.randn(n, nq, H, D_ROPE, device="cuda", generator=gen).bfloat16(),
                      sign_words=_sign_words(bits), sign=_dev(1.0 - 2.0 * bits).float(),
                      mask=None if case["chain"] else _dev(_tree_masks(n_node, nq, g)),
                      out=torch.empty(n, nq, H, D_LAT, dtype=torch.bfloat16, device="cuda"),
                      lse=torch.empty(n, nq, H, device="cuda"))
            if own:
                import quantized_kv_cache_fp8_gb300 as kvq
                st["problem"] = kvq.make_tree_problem(
                    seq_len=st["seq_len"], n_node=st["n_node"], mask=st["mask"], q_lat=st["q_lat"],
                    q_rope=st["q_rope"], sm_scale=SM_SCALE, max_seq_len=max(lens), fmt=case["fmt"],
                    cache=st["planes"], signs=st["sign_words"], block_table=st["table"], page_size=page,
                    seq_stride_rows=st["stride"])
                st["workspace"] = torch.empty(kvq.kvq_mla_tree_decode_workspace(st["problem"]), dtype=torch.uint8,
                                              device="cuda")
        else:
            n, nq = case["n_seq"], case["nodes"]
            path = np.zeros((n, nq), np.int32)
            acc = np.zeros(n, np.int32)
            for s in range(n):
                # the first drafted tokens as they stand, the rest from further down the tree
                a = int(g.integers(0, (n_node[s] + 1) // 2 + 1))
                i = int(g.integers(max(0, 2 * a - n_node[s]), a + 1))
                acc[s] = a
                path[s, :a] = np.concatenate([np.arange(i), a + np.sort(g.choice(n_node[s] - a, a - i, replace=False))])
            st.update(path=_dev(path), n_acc=_dev(acc), new_len=torch.empty(n, dtype=torch.int32, device="cuda"))
            if own:
                import quantized_kv_cache_fp8_gb300 as kvq
                st["accept"] = kvq.make_accept(
                    seq_len=st["seq_len"], n_node=st["n_node"], path=st["path"], n_acc=st["n_acc"],
                    new_len=st["new_len"], fmt=case["fmt"], cache=st["planes"], block_table=st["table"],
                    page_size=page, seq_stride_rows=st["stride"])
    return st


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _plain_resize(st, keep, new, out):
    """One call of the page allocator, every sequence at once."""
    ps, table, held, free, n_free = st["case"]["page"], st["table"], st["held"], st["free"], st["n_free"]
    n, mp, tokens = st["n_seq"], st["max_pages"], out["slot_map"].numel()
    need = (keep + new + ps - 1) // ps
    end = torch.cumsum(new, 0)
    out["tok_start"][0] = 0
    out["tok_start"][1:] = end
    fits = (need <= mp) & (end <= tokens) & (keep <= held * ps)
    give = torch.where(fits, (held - need).clamp(min=0), 0)
    take = torch.where(fits, (need - held).clamp(min=0), 0)
    col = torch.arange(mp, device="cuda")
    # pages given back, the last sequence's last page first
    total = give.sum()
    behind = total - torch.cumsum(give, 0)                        # given by later sequences
    s, p = torch.nonzero((col >= need[:, None]) & (col < held[:, None]) & fits[:, None], as_tuple=True)
    free[(n_free + behind[s] + (held[s] - 1 - p)).long()] = table[s, p]
    table[s, p] = -1
    have = n_free + total
    stop = torch.cumsum(take, 0)
    served = fits & ((take == 0) | (stop <= have))
    take = torch.where(served, take, 0)
    s, p = torch.nonzero((col >= held[:, None]) & (col < (held + take)[:, None]), as_tuple=True)
    table[s, p] = free[(have - 1 - ((stop - take)[s] + p - held[s])).long()]
    n_free.copy_(have - take.sum())
    out["seq_len"].copy_(torch.where(served, keep + new, torch.minimum(keep, held * ps)))
    held.copy_(torch.where(served, need, held))
    tok = torch.arange(tokens, device="cuda")
    s = torch.searchsorted(end, tok, right=True).clamp(max=n - 1)
    pos = keep[s] + tok - (end - new)[s]
    ok = (tok < end[-1]) & served[s]
    page = table[s, (pos // ps).clamp(0, mp - 1)]
    out["slot_map"].copy_(torch.where(ok, page * ps + pos % ps, -1))
    out["tok_pos"].copy_(torch.where(ok, pos, -1))


def _fwht(y):
    """Orthonormal up to 1/sqrt(512): the Walsh-Hadamard stages in ascending order."""
    h = 1
    while h < D_LAT:
        v = y.view(-1, D_LAT // (2 * h), 2, h)
        y = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2).reshape(-1, D_LAT)
        h *= 2
    return y


def _plain_append(st):
    fmt, pl = st["case"]["fmt"], st["planes"]
    x, k = st["x"].float(), st["k"].float()
    slot = torch.where(st["slot"] >= 0, st["slot"], st["rows"]).long()

    def fp8(v):
        s = v.abs().amax(1) / 448.0
        c = torch.where(s[:, None] > 0, v / s[:, None], 0.0)
        return c.to(torch.float8_e4m3fn).view(torch.uint8), s

    if fmt == FMT_FP8:
        lat, ls = fp8(x)
    else:
        cs = torch.tensor(1.0 / math.sqrt(512.0), device="cuda")
        y = _fwht(x * st["sign"]) * cs
        # the radius in 64 bits, rounded once: the codes next to a threshold depend on it
        ls = y.double().pow(2).sum(1).sqrt().float()
        cb = _codebook(torch.float32)
        u = torch.where(ls[:, None] > 0, y / (ls * cs)[:, None], 0.0)
        code = torch.where(ls[:, None] > 0, torch.bucketize(u, (cb[1:] + cb[:-1]) / 2, right=True), 0).to(torch.uint8)
        lat = code[:, 0::2] | (code[:, 1::2] << 4)
    rope, rs = fp8(k)
    pl["lat"][slot] = lat
    pl["lat_scale"][slot] = ls
    pl["rope"][slot] = rope
    pl["rope_scale"][slot] = rs


def _seq_rows(st, s, a, b):
    """Pool rows of the rows a .. b-1 of sequence s."""
    t = torch.arange(a, b, device="cuda")
    if st["table"] is None:
        return s * st["stride"] + t
    ps = st["case"]["page"]
    return st["table"][s, t // ps].long() * ps + t % ps


def _seq_values(st, s, dtype):
    """The latent and rope rows of sequence s as numbers (rotated tier: the rotated rows)."""
    r, pl = _seq_rows(st, s, 0, st["lens"][s]), st["planes"]
    if st["case"]["fmt"] == FMT_FP8:
        c = pl["lat"][r].view(torch.float8_e4m3fn).to(dtype) * pl["lat_scale"][r, None].to(dtype)
    else:
        b = pl["lat"][r]
        code = torch.stack([b & 15, b >> 4], 2).reshape(-1, D_LAT).long()
        c = _codebook(dtype)[code] * (pl["lat_scale"][r, None].to(dtype) / math.sqrt(512.0))
    k = pl["rope"][r].view(torch.float8_e4m3fn).to(dtype) * pl["rope_scale"][r, None].to(dtype)
    return c, k


def _visible(st, s, nq):
    """[node][cache row]: which rows the nodes of sequence s see."""
    L, n = st["lens"][s], st["nodes"][s]
    j = torch.arange(nq, device="cuda")[:, None]
    t = torch.arange(L, device="cuda")[None, :] - (L - n)
    bit = j >= t if st["mask"] is None else ((st["mask"][s][:, None] >> t.clamp(0, 63)) & 1) > 0
    return ((t < 0) | bit) & (j < n)


def _plain_tree(st):
    case, out, lse = st["case"], st["out"], st["lse"]
    nq, H = case["nodes"], case["heads"]
    had = _hadamard(torch.float32) / math.sqrt(512.0)
    for s in range(case["n_seq"]):
        c, k = _seq_values(st, s, torch.float32)
        q = st["q_lat"][s].float().view(nq * H, D_LAT)
        if case["fmt"] == FMT_TQ4:
            q = (q * st["sign"]) @ had
        sc = (q @ c.T + st["q_rope"][s].float().view(nq * H, D_ROPE) @ k.T) * SM_SCALE
        see = _visible(st, s, nq).repeat_interleave(H, 0)
        sc = torch.where(see, sc, -math.inf)
        m = sc.amax(1, keepdim=True)
        m = torch.where(m > -math.inf, m, 0.0)
        p = torch.exp(sc - m)
        tot = p.sum(1, keepdim=True)
        o = (p @ c) / torch.where(tot > 0, tot, 1.0)
        if case["fmt"] == FMT_TQ4:
            o = (o @ had) * st["sign"]
        out[s] = o.view(nq, H, D_LAT).bfloat16()
        lse[s] = (m + torch.log(tot)).view(nq, H)


def _plain_accept(st):
    n, nq, pl = st["case"]["n_seq"], st["case"]["nodes"], st["planes"]
    k = torch.arange(nq, device="cuda")[None, :]
    base = (st["seq_len"] - st["n_node"])[:, None]
    s = torch.arange(n, device="cuda")[:, None].expand(n, nq)

    def row(t):
        if st["table"] is None:
            return s * st["stride"] + t
        ps = st["case"]["page"]
        return st["table"][s, (t // ps).clamp(0, st["table"].shape[1] - 1)].long() * ps + t % ps

    go = k < st["n_acc"][:, None]
    src, dst = row(base + torch.where(go, st["path"], 0))[go], row(base + k)[go]
    for key in ("lat", "lat_scale", "rope", "rope_scale"):
        pl[key][dst] = pl[key][src]
    st["new_len"].copy_(st["seq_len"] - st["n_node"] + st["n_acc"])


def run(state):
    st = state
    op = st["case"]["op"]
    if own:
        import quantized_kv_cache_fp8_gb300 as kvq
    if op == "pages":
        if own:
            kvq.kvq_resize_pages(st["plan_grow"])
            kvq.kvq_resize_pages(st["plan_back"])
        else:
            _plain_resize(st, st["keep"], st["new"], st["grow"])
            _plain_resize(st, st["keep"], st["zero"], st["back"])
        return [st["table"], st["held"], st["n_free"], st["free"], st["grow"]["seq_len"], st["grow"]["tok_start"],
                st["grow"]["slot_map"], st["grow"]["tok_pos"], st["back"]["seq_len"]]
    if op == "append":
        rows = st["rows"]
        pool = {k: v[:rows] for k, v in st["planes"].items()}
        if own:
            kvq.kvq_append_mla(st["x"], st["k"], st["slot"], st["case"]["fmt"], st["sign_words"], pool)
        else:
            _plain_append(st)
        lat = pool["lat"].view(torch.float8_e4m3fn) if st["case"]["fmt"] == FMT_FP8 else \
            torch.index_select(st["pairs"], 0, pool["lat"].reshape(-1).int())
        return [lat, pool["lat_scale"], pool["rope"].view(torch.float8_e4m3fn), pool["rope_scale"]]
    if op == "tree":
        if own:
            kvq.kvq_mla_tree_decode(st["problem"], st["out"], st["lse"], st["workspace"])
        else:
            _plain_tree(st)
        return [st["out"], st["lse"]]
    if own:
        kvq.kvq_accept_mla(st["accept"])
    else:
        _plain_accept(st)
    pl = st["planes"]
    lat = pl["lat"].view(torch.float8_e4m3fn) if st["case"]["fmt"] == FMT_FP8 else pl["lat"]
    return [st["new_len"], lat, pl["lat_scale"], pl["rope"].view(torch.float8_e4m3fn), pl["rope_scale"]]


# ---------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "append":
        return [None, *_exact_append(case, seed)]
    if op != "tree" or case["fmt"] != FMT_FP8 and case["T"] * case["n_seq"] > 1 << 20:
        return None
    st = prepare(case, seed)
    nq, H, n = case["nodes"], case["heads"], case["n_seq"]
    if n * nq * H * case["T"] > 1 << 32:
        return None
    out = torch.zeros(n, nq, H, D_LAT, dtype=torch.float64, device="cuda")
    lse = torch.full((n, nq, H), -math.inf, dtype=torch.float64, device="cuda")
    turn = _hadamard(torch.float64) * st["sign"].double()[None, :] / math.sqrt(512.0)
    for s in range(n):
        c, k = _seq_values(st, s, torch.float64)
        if case["fmt"] == FMT_TQ4:
            c = c @ turn                     # every row rotated back: the definition's own order
        rows = torch.cat([c, k], 1)
        first = st["lens"][s] - st["nodes"][s]
        for j in range(st["nodes"][s]):
            seen = [t for t in range(st["nodes"][s])
                    if (t <= j if st["mask"] is None else (int(st["mask"][s, j]) >> t) & 1)]
            idx = torch.tensor([first + t for t in seen], dtype=torch.long, device="cuda")
            x = torch.cat([rows[:first], rows[idx]])
            q = torch.cat([st["q_lat"][s, j], st["q_rope"][s, j]], 1).double()
            sc = q @ x.T * SM_SCALE
            top = sc.max(1, keepdim=True).values
            w = torch.exp(sc - top)
            z = w.sum(1, keepdim=True)
            out[s, j] = (w / z) @ x[:, :D_LAT]
            lse[s, j] = (top + torch.log(z))[:, 0]
    return [out, lse]


def _exact_append(case, seed):
    """The scales and the rope values of the pool rows (a code next to a border has no value
    of its own in 64 bits, so the codes are left out)."""
    st = prepare(case, seed)
    x, k = st["x"].double(), st["k"].double()
    ls = torch.zeros(st["rows"], dtype=torch.float64, device="cuda")
    rs = torch.zeros_like(ls)
    for i, r in enumerate(st["slot"].tolist()):
        if r >= 0 and case["rows"] <= 8192:
            ls[r] = x[i].abs().max() / 448.0 if case["fmt"] == FMT_FP8 else x[i].norm()
            rs[r] = k[i].abs().max() / 448.0
    if case["rows"] > 8192:
        go = st["slot"] >= 0
        ls[st["slot"][go].long()] = x[go].abs().amax(1) / 448.0 if case["fmt"] == FMT_FP8 else x[go].norm(dim=1)
        rs[st["slot"][go].long()] = k[go].abs().amax(1) / 448.0
    return ls, None, rs


# ---------------------------------------------------------------------------------------
# costs
# ---------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "pages":
        n = case["n_seq"]
        pages = n * -(-(case["new"] * 3 // 4) // case["page"])
        # grow: lengths in, lengths, offsets, tables, slots and positions out; back: the pages return
        return dict(bytes=n * (12 + 12) * 2 + pages * 8 * 2 + (n * case["new"] + 7) * 8, flops=0)
    row = (512 if case["fmt"] == FMT_FP8 else 256) + 72
    if op == "append":
        return dict(bytes=case["rows"] * (576 * (2 if case["bf16"] else 4) + 4 + row),
                    flops=case["rows"] * (1152 if case["fmt"] == FMT_FP8 else 512 * 11))
    mean = 33 / 64 if case.get("ragged") else 1.0            # lengths are uniform between T/64 and T
    if op == "accept":
        return dict(bytes=case["n_seq"] * (case["nodes"] // 4) * (2 * row + 4), flops=0)
    nodes = (case["nodes"] + 1) / 2 if case.get("ragged") else case["nodes"]
    rows, q = case["n_seq"] * case["T"] * mean, case["n_seq"] * nodes * case["heads"]
    return dict(bytes=int(rows * row + q * (1152 + 1024 + 4)),
                flops=int(2 * (576 + 512) * q * case["T"] * mean))
