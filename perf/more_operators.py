"""The operators of beam search and parallel sampling over a paged fp8 K/V cache: their cases,
inputs, plain forms and costs.

  append   new K/V rows of a grouped-query model quantized to fp8 and written at the pool rows of
           a slot map
  decode   attention of one new token a sequence over that cache, through block tables
  beam     the best continuations over beams and vocabulary, with their parents
  fork     block tables after the beams' reordering: pages shared, copied and freed; and the copies
  compact  a fragmented pool's pages moved to its front: tables, free list and the copies

A K/V cache holds, for each KV head, its rows' e4m3 codes and one fp32 scale a row.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small batch (padded with -1 slots): K and V are slices of a fused projection
        dict(name="append_step", op="append", rows=37, n_kv=8, group=4, dim=128, bf16=True, page=64),
        # the prompts of a batch
        dict(name="append_prompt", op="append", rows=32768, n_kv=8, group=4, dim=128, bf16=True, page=64),
        # a single short sequence: latency
        dict(name="decode_one", op="decode", n_seq=1, T=1024, n_kv=8, group=4, dim=128, page=16, window=0, ragged=False),
        # one long sequence, eight query heads a KV head
        dict(name="decode_long", op="decode", n_seq=1, T=131072, n_kv=8, group=8, dim=128, page=64, window=0, ragged=False),
        # a ragged batch (an empty sequence in it) of 512 to 32768 rows, seven query heads a KV head
        dict(name="decode_ragged", op="decode", n_seq=64, T=32768, n_kv=4, group=7, dim=128, page=64, window=0, ragged=True),
        # wide heads without grouping behind a sliding window, odd lengths, no block table
        dict(name="decode_window", op="decode", n_seq=24, T=9001, n_kv=16, group=1, dim=256, page=0, window=4096, ragged=False),
        # four beams of one request
        dict(name="beam_small", op="beam", n_req=1, n_beam=4, vocab=32000, n_out=4, bf16=False),
        # a batch of requests, eight beams each, twice as many candidates as beams
        dict(name="beam_batch", op="beam", n_req=64, n_beam=8, vocab=128000, n_out=16, bf16=True),
        # the four beams of one request after a step
        dict(name="fork_small", op="fork", n_req=1, n_beam=4, T=1000, n_kv=8, dim=128, page=16),
        # a batch of requests' beams, long shared prompts
        dict(name="fork_batch", op="fork", n_req=64, n_beam=8, T=4096, n_kv=8, dim=128, page=64),
        # a small pool
        dict(name="compact_small", op="compact", n_pages=256, n_seq=8, n_kv=2, dim=64, page=16, used=0.5),
        # a large pool after many requests have come and gone
        dict(name="compact_large", op="compact", n_pages=16384, n_seq=128, n_kv=4, dim=128, page=64, used=0.6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _shrink(c, cost, most, least):
    """Halves the largest of a case's sizes until it costs no more than `most`."""
    while cost(c) > most:
        key = max(least, key=lambda k: c[k] / least[k])
        c[key] = max(1, c[key] // 2)
    return c


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "decode", "beam", "beam", "fork", "compact"])
    dim = rng.choice([64, 128, 128, 256])
    if op == "append":
        return _shrink(dict(op=op, rows=_log(rng, 1, 30000), n_kv=_log(rng, 1, 16), group=rng.randint(1, 8), dim=dim,
                            bf16=rng.random() < 0.7, page=rng.choice([16, 64, 100])),
                       lambda c: c["rows"] * c["n_kv"] * c["dim"] * (1 if c["bf16"] else 2), 1 << 25, dict(rows=64, n_kv=2))
    if op == "decode":
        T = _log(rng, 1, 60000)
        return _shrink(dict(op=op, n_seq=_log(rng, 1, 128), T=T, n_kv=_log(rng, 1, 16), group=_log(rng, 1, 20), dim=dim,
                            page=rng.choice([0, 8, 16, 40, 64, 100, 128]),
                            window=rng.choice([0, 0, 0, _log(rng, 1, 5000)]), ragged=rng.random() < 0.6),
                       lambda c: c["n_seq"] * c["T"] * c["n_kv"] * c["dim"], 1 << 27, dict(n_seq=2, T=256, n_kv=2))
    if op == "beam":
        B = rng.randint(1, 16)
        return _shrink(dict(op=op, n_req=_log(rng, 1, 64), n_beam=B, vocab=_log(rng, 500, 160000),
                            n_out=rng.choice([B, 2 * B]), bf16=rng.random() < 0.6),
                       lambda c: c["n_req"] * c["n_beam"] * c["vocab"] * (1 if c["bf16"] else 2), 1 << 26,
                       dict(n_req=1, vocab=4000))
    if op == "fork":
        return _shrink(dict(op=op, n_req=_log(rng, 1, 64), n_beam=rng.randint(2, 16), T=_log(rng, 20, 8000),
                            n_kv=_log(rng, 1, 8), dim=dim, page=rng.choice([8, 16, 64, 100])),
                       lambda c: c["n_req"] * (c["T"] + c["n_beam"] * 4 * c["page"]) * c["n_kv"] * c["dim"], 1 << 28,
                       dict(n_req=2, T=64, n_kv=2))
    return _shrink(dict(op=op, n_pages=_log(rng, 64, 16000), n_seq=_log(rng, 2, 200), n_kv=_log(rng, 1, 8), dim=dim,
                        page=rng.choice([8, 16, 64, 100]), used=round(rng.uniform(0.1, 0.9), 2)),
                   lambda c: c["n_pages"] * c["page"] * c["n_kv"] * c["dim"], 1 << 29, dict(n_pages=64, n_kv=2))


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def _table(lens, page, g, spare=3):
    """Page ids in a random order, -1 past a sequence's pages; and the pool's pages."""
    n = [-(-int(x) // page) for x in lens]
    total = sum(n) + spare
    perm = g.permutation(total).astype(np.int32)
    t = np.full((len(lens), max(1, max(n))), -1, np.int32)
    o = 0
    for s, k in enumerate(n):
        t[s, :k] = perm[o:o + k]
        o += k
    return t, total


def _random_cache(n_kv, rows, dim, gen):
    """Rows of N(0,1) elements, each row times a magnitude log-uniform in [0.1, 4], quantized."""
    planes = {}
    for x in ("k", "v"):
        codes = torch.empty(n_kv, rows, dim, dtype=torch.uint8, device="cuda")
        scale = torch.empty(n_kv, rows, device="cuda")
        for h in range(n_kv):
            for a in range(0, rows, 1 << 18):
                b = min(rows, a + (1 << 18))
                mag = torch.exp(torch.empty(b - a, 1, device="cuda").uniform_(math.log(0.1), math.log(4.0), generator=gen))
                v = torch.randn(b - a, dim, device="cuda", generator=gen) * mag
                s = v.abs().amax(1) / 448.0
                codes[h, a:b] = (v / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                scale[h, a:b] = s
        planes[x], planes[x + "_scale"] = codes, scale
    return planes


def _byte_cache(n_kv, rows, dim, gen):
    """A cache whose bytes are only moved: any finite codes."""
    planes = {}
    for x in ("k", "v"):
        planes[x] = torch.randint(0, 127, (n_kv, rows, dim), dtype=torch.uint8, device="cuda", generator=gen)
        planes[x + "_scale"] = torch.rand(n_kv, rows, device="cuda", generator=gen)
    return planes


def _prepare_append(case, g, gen):
    n, kv, d, ps = case["rows"], case["n_kv"], case["dim"], case["page"]
    pages = -(-n // ps) + 3
    ids = g.permutation(pages)[: -(-n // ps)]
    slot = (ids[:, None] * ps + np.arange(ps)[None, :]).reshape(-1)[:n].astype(np.int32)
    slot[g.random(n) < 0.03] = -1                             # tokens of refused sequences, padding
    heads = kv * (case["group"] + 2)
    x = torch.randn(n, heads, d, device="cuda", generator=gen)
    x *= torch.exp(torch.empty(n, heads, 1, device="cuda").uniform_(math.log(0.1), math.log(4.0), generator=gen))
    x = x.bfloat16() if case["bf16"] else x
    # one row more than the pool: where the plain form puts the rows without a slot
    rows = pages * ps
    planes = dict(k=torch.zeros(kv, rows + 1, d, dtype=torch.uint8, device="cuda"),
                  v=torch.zeros(kv, rows + 1, d, dtype=torch.uint8, device="cuda"),
                  k_scale=torch.zeros(kv, rows + 1, device="cuda"), v_scale=torch.zeros(kv, rows + 1, device="cuda"))
    return dict(k=x[:, heads - 2 * kv:heads - kv], v=x[:, heads - kv:], slot=_dev(slot), rows=rows, planes=planes)


def _prepare_decode(case, g, gen):
    n, T, kv, d, ps = case["n_seq"], case["T"], case["n_kv"], case["dim"], case["page"]
    lens = g.integers(max(1, T // 64), T + 1, n) if case["ragged"] else np.full(n, T)
    lens[0] = T
    if case["ragged"] and n >= 8:
        lens[n // 2] = 0
    st = dict(lens=_dev(lens.astype(np.int32)), most=T, stride=T)
    if ps:
        table, pages = _table(lens, ps, g)
        st["table"], rows = _dev(table), pages * ps
    else:
        st["table"], rows = None, n * T
    st["planes"] = _random_cache(kv, rows, d, gen)
    H = kv * case["group"]
    st["q"] = torch.randn(n, H, d, device="cuda", generator=gen).bfloat16()
    st["out"] = torch.empty(n, H, d, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty(n, H, device="cuda")
    st["scale"] = 1.0 / math.sqrt(d)
    if own:
        import quantized_kv_cache_fp8_gb300 as kvq
        st["problem"] = kvq.make_kv8_problem(
            seq_len=st["lens"], q=st["q"], sm_scale=st["scale"], max_seq_len=T, cache=st["planes"],
            block_table=st["table"], page_size=ps, seq_stride_rows=T, window=case["window"])
        st["workspace"] = torch.empty(kvq.kvq_kv8_decode_workspace(st["problem"]), dtype=torch.uint8, device="cuda")
    return st


def _prepare_beam(case, g, gen):
    R, B, V, K = case["n_req"], case["n_beam"], case["vocab"], case["n_out"]
    # logits with a few likely tokens; a third of the rows from a constrained vocabulary
    x = torch.randn(R, B, V, device="cuda", generator=gen) * 2.0
    x += torch.where(torch.rand(R, B, V, device="cuda", generator=gen) < 20.0 / V, 8.0, 0.0)
    masked = torch.rand(R, B, 1, device="cuda", generator=gen) < 0.33
    x.masked_fill_(masked & (torch.rand(R, B, V, device="cuda", generator=gen) < 0.5), -math.inf)
    score = -5.0 * torch.rand(R, B, device="cuda", generator=gen) - 20.0
    if R > 1:
        score[R // 2, 1:] = -math.inf                         # a request at its first step
    fin = (torch.rand(R, B, device="cuda", generator=gen) < 0.1).int()
    st = dict(logits=x.bfloat16() if case["bf16"] else x, score=score, finished=fin, out_score=torch.empty(R, K, device="cuda"),
              out_token=_i32(R, K), out_parent=_i32(R, K), out_finished=_i32(R, K), eos=2, pad=0)
    if own:
        import quantized_kv_cache_fp8_gb300 as kvq
        st["problem"] = kvq.make_beam_problem(
            logits=st["logits"], score=score, finished=fin, eos=2, pad=0, out_score=st["out_score"],
            out_token=st["out_token"], out_parent=st["out_parent"], out_finished=st["out_finished"])
        st["workspace"] = torch.empty(kvq.kvq_beam_select_workspace(st["problem"]), dtype=torch.uint8, device="cuda")
    return st


def _prepare_fork(case, g, gen):
    """Requests whose beams share a prompt; some beams (the survivors) have pages of their own behind it,
    each other beam is a copy of a survivor, with its own last page, as it is again after the step."""
    R, B, ps = case["n_req"], case["n_beam"], case["page"]
    n = R * B
    n_pages, max_pages = R * (case["T"] // ps) + 3 * n + 5, case["T"] // ps + 6
    parent, lens, rows_of = np.zeros(n, np.int32), np.zeros(n, np.int32), []
    for r in range(R):
        prompt = int(g.integers(case["T"] // 2, case["T"] + 1)) // ps      # shared pages
        L = prompt * ps + int(g.integers(1, 3 * ps + 1))
        alive = g.random(B) < 0.5
        alive[int(g.integers(0, B))] = True
        up = np.where(alive, np.arange(B), g.choice(np.flatnonzero(alive), B))
        parent[r * B:(r + 1) * B] = r * B + up
        lens[r * B:(r + 1) * B] = L
        rows_of.append((prompt, -(-L // ps), alive, up))
    table, held = np.full((n, max_pages), -1, np.int32), np.zeros(n, np.int32)
    ids = list(range(n_pages))
    # the pages that the step frees and hands out again: the lowest ids, in the beams' order
    for r, (prompt, need, alive, up) in enumerate(rows_of):
        for b in range(B):
            held[r * B + b] = need
            if not alive[b] and lens[r * B] % ps:
                table[r * B + b, need - 1] = ids.pop(0)
    ids = [ids[i] for i in g.permutation(len(ids))]
    for r, (prompt, need, alive, up) in enumerate(rows_of):
        first = [ids.pop() for _ in range(prompt)]
        for b in np.flatnonzero(alive):
            table[r * B + b, :need] = first + [ids.pop() for _ in range(need - prompt)]
        for b in np.flatnonzero(~alive):
            whole = lens[r * B] // ps
            table[r * B + b, :whole] = table[r * B + up[b], :whole]
    # survivors come before their copies, so that they keep their pages
    order = np.concatenate([r * B + np.argsort(~rows_of[r][2], kind="stable") for r in range(R)])
    place = np.argsort(order)
    parent, table, held = place[parent[order]].astype(np.int32), table[order], held[order]
    free = np.full(n_pages, -1, np.int32)
    free[:len(ids)] = sorted(ids, reverse=True)
    return dict(parent=_dev(parent), table=_dev(table), held=_dev(held), seq_len=_dev(lens), free=_dev(free),
                n_free=_i32(1, fill=len(ids)), src=_i32(n, fill=-1), dst=_i32(n, fill=-1), rows=_i32(n, fill=-1),
                n_copy=_i32(1), n_pages=n_pages, planes=_byte_cache(case["n_kv"], n_pages * ps, case["dim"], gen))


def _prepare_compact(case, g, gen):
    N, n, ps = case["n_pages"], case["n_seq"], case["page"]
    most = int(N * case["used"]) * 4 // n + 1
    share = g.random(n)
    held = np.minimum(share / share.sum() * N * case["used"], most).astype(np.int32)
    perm = g.permutation(N).astype(np.int32)
    table = np.full((n, most + 2), -1, np.int32)
    o = 0
    for s in range(n):
        table[s, :held[s]] = perm[o:o + held[s]]
        o += held[s]
    most = N // 2
    return dict(table=_dev(table), new_table=_i32(*table.shape), held=_dev(held), free=_i32(N), n_free=_i32(1),
                n_used=_i32(1), src=_i32(most), dst=_i32(most), rows=_i32(most), n_copy=_i32(1), n_pages=N,
                planes=_byte_cache(case["n_kv"], N * ps, case["dim"], gen))


def prepare(case, seed):
    g = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, ps = case["op"], case.get("page")
    make = dict(append=_prepare_append, decode=_prepare_decode, beam=_prepare_beam, fork=_prepare_fork,
                compact=_prepare_compact)[op]
    st = make(case, g, gen)
    st["case"] = case
    if own and op in ("fork", "compact"):
        import quantized_kv_cache_fp8_gb300 as kvq
        lists = dict(copy_src=st["src"], copy_dst=st["dst"], copy_rows=st["rows"], n_copy=st["n_copy"])
        if op == "fork":
            st["plan"] = kvq.make_fork_plan(parent=st["parent"], block_table=st["table"], n_held=st["held"], free_list=st["free"],
                                            n_free=st["n_free"], seq_len=st["seq_len"], page_size=ps, **lists)
            size = kvq.kvq_fork_pages_workspace(st["plan"])
        else:
            st["plan"] = kvq.make_compact_plan(block_table=st["table"], n_held=st["held"], new_table=st["new_table"],
                                               free_list=st["free"], n_free=st["n_free"], n_used=st["n_used"], page_size=ps,
                                               **lists)
            size = kvq.kvq_compact_pages_workspace(st["plan"])
        st["copy"] = kvq.make_page_copy(caches=[st["planes"]], page_size=ps, **lists)
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _fp8(v):
    s = v.abs().amax(-1) / 448.0
    c = torch.where(s[..., None] > 0, v / s[..., None], 0.0)
    return c.to(torch.float8_e4m3fn).view(torch.uint8), s


def _plain_append(st):
    slot = torch.where(st["slot"] >= 0, st["slot"], st["rows"]).long()
    kc, ks = _fp8(st["k"].float())
    vc, vs = _fp8(st["v"].float())
    pl = st["planes"]
    pl["k"][:, slot] = kc.transpose(0, 1)
    pl["v"][:, slot] = vc.transpose(0, 1)
    pl["k_scale"][:, slot] = ks.t()
    pl["v_scale"][:, slot] = vs.t()


def _rows_of(st):
    """The pool rows [sequence][position] of a decode problem, 0 where there is none."""
    t = torch.arange(st["most"], device="cuda")
    if st["table"] is None:
        return torch.arange(st["lens"].shape[0], device="cuda")[:, None] * st["stride"] + t
    ps = st["case"]["page"]
    return (st["table"][:, t // ps].long() * ps + t % ps).clamp(min=0)


def _values(pl, x, rows, dtype):
    """Rows of a plane pair as numbers: [sequence][KV head][position][dim]."""
    c = pl[x].view(torch.float8_e4m3fn)[:, rows].to(dtype) * pl[x + "_scale"][:, rows, None].to(dtype)
    return c.transpose(0, 1)


def _plain_decode(st):
    case, L = st["case"], st["lens"]
    n, kv, G, d = case["n_seq"], case["n_kv"], case["group"], case["dim"]
    t = torch.arange(st["most"], device="cuda")
    see = t < L[:, None]
    if case["window"]:
        see &= t >= (L - case["window"])[:, None]
    rows = _rows_of(st)
    q = st["q"].float().view(n, kv, G, d)
    s = torch.matmul(q, _values(st["planes"], "k", rows, torch.float32).transpose(2, 3)) * st["scale"]
    s = torch.where(see[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(s - m)
    tot = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _values(st["planes"], "v", rows, torch.float32)) / torch.where(tot > 0, tot, 1.0)
    st["out"].copy_(o.view(n, kv * G, d))
    st["lse"].copy_((m + torch.log(tot)).view(n, kv * G))


def _plain_beam(st):
    case = st["case"]
    R, B, V, K = case["n_req"], case["n_beam"], case["vocab"], case["n_out"]
    # candidates of different beams stand next to one another within an fp32 rounding: 64 bits
    x = st["logits"].double()
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    val = x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True)))
    val = torch.where(x > -math.inf, val + st["score"].double()[..., None], -math.inf)
    fin = st["finished"] != 0
    val = torch.where(fin[..., None], -math.inf, val)
    val[..., st["pad"]] = torch.where(fin, st["score"].double(), val[..., st["pad"]])
    val = val.view(R, B * V)
    kth = torch.topk(val, K, 1).values[:, -1:]
    tie = val == kth                                          # the lowest of those that tie for the last places
    more = val > kth
    take = more | (tie & (torch.cumsum(tie, 1) <= K - more.sum(1, keepdim=True)))
    at = torch.nonzero(take)[:, 1].view(R, K)
    v, order = torch.sort(torch.gather(val, 1, at), dim=1, descending=True, stable=True)
    at = torch.gather(at, 1, order)
    none = v == -math.inf
    beam, token = at // V, at % V
    ended = torch.gather(fin, 1, beam) | (token == st["eos"])
    st["out_score"].copy_(v)
    st["out_token"].copy_(torch.where(none, -1, token))
    st["out_parent"].copy_(torch.where(none, -1, beam + B * torch.arange(R, device="cuda")[:, None]))
    st["out_finished"].copy_(torch.where(none, False, ended))


def _plain_copy(st):
    """Every plane's rows of the listed copies."""
    ps, n = st["case"]["page"], st["src"].numel()
    row = torch.arange(ps, device="cuda")
    go = (torch.arange(n, device="cuda") < st["n_copy"])[:, None] & (row < st["rows"][:, None])
    src = (st["src"].long()[:, None] * ps + row)[go]
    dst = (st["dst"].long()[:, None] * ps + row)[go]
    pl = st["planes"]
    pl["k"][:, dst] = pl["k"][:, src]
    pl["v"][:, dst] = pl["v"][:, src]
    pl["k_scale"][:, dst] = pl["k_scale"][:, src]
    pl["v_scale"][:, dst] = pl["v_scale"][:, src]


def _list_copies(st, src, dst, rows):
    k = src.shape[0]
    st["src"].fill_(-1)[:k] = src.int()
    st["dst"].fill_(-1)[:k] = dst.int()
    st["rows"].fill_(-1)[:k] = rows.int()
    st["n_copy"].fill_(k)


def _plain_fork(st):
    ps, N, table, held, free = st["case"]["page"], st["n_pages"], st["table"], st["held"], st["free"]
    n, mp = table.shape
    me, col = torch.arange(n, device="cuda"), torch.arange(mp, device="cuda")
    par = st["parent"].long()
    up = par.clamp(min=0)
    length = torch.where(par >= 0, torch.minimum(st["seq_len"][up], held[up] * ps), 0)
    need = (length + ps - 1) // ps
    new = torch.where(col < need[:, None], table[up], -1)
    # page N stands for none
    whole = torch.where(col < (length // ps)[:, None], new, N).long()
    part = length % ps > 0
    last = torch.where(part, torch.gather(new, 1, (need - 1).clamp(min=0)[:, None].long())[:, 0], N).long()
    is_whole = torch.zeros(N + 1, dtype=torch.bool, device="cuda")
    is_whole[whole] = True
    keeper = torch.full((N + 1,), n, dtype=torch.long, device="cuda").scatter_reduce_(0, last, me, "amin")
    copy = part & (is_whole[last] | (keeper[last] != me))
    stays = is_whole
    stays[torch.where(copy, N, last)] = True
    was = torch.zeros(N + 1, dtype=torch.bool, device="cuda")
    was[torch.where(col < held[:, None], table, N).long()] = True
    freed = torch.nonzero((was & ~stays)[:N])[:, 0]
    have = st["n_free"] + freed.shape[0]
    free[(st["n_free"] + torch.arange(freed.shape[0], device="cuda")).long()] = freed.flip(0).int()
    who = torch.nonzero(copy)[:, 0]
    page = free[(have - 1 - torch.arange(who.shape[0], device="cuda")).long()]
    _list_copies(st, last[who], page, (length % ps)[who])
    new[who, (need - 1)[who].long()] = page
    st["n_free"].copy_(have - who.shape[0])
    table.copy_(new)
    held.copy_(need)
    st["seq_len"].copy_(length)


def _plain_compact(st):
    ps, N, table, held = st["case"]["page"], st["n_pages"], st["table"], st["held"]
    col = torch.arange(table.shape[1], device="cuda")
    mine = col < held[:, None]
    used = torch.zeros(N + 1, dtype=torch.bool, device="cuda")
    used[torch.where(mine, table, N).long()] = True
    used = used[:N]
    n_used = int(used.sum())
    hole = torch.nonzero(~used[:n_used])[:, 0]
    move = torch.nonzero(used[n_used:])[:, 0] + n_used
    to = torch.arange(N, device="cuda")
    to[move] = hole
    st["new_table"].copy_(torch.where(mine, to[table.clamp(min=0).long()], -1))
    st["free"].fill_(-1)[:N - n_used] = torch.arange(N - 1, n_used - 1, -1, dtype=torch.int32, device="cuda")
    st["n_free"].fill_(N - n_used)
    st["n_used"].fill_(n_used)
    _list_copies(st, move, hole, torch.full_like(move, ps))


def run(state):
    st = state
    op = st["case"]["op"]
    if own:
        import quantized_kv_cache_fp8_gb300 as kvq
    if op == "append":
        if own:
            pl = st["planes"]
            kvq.kvq_append_kv8(st["k"], st["v"], st["slot"], pl)
        else:
            _plain_append(st)
        # (the last row is where the plain form puts the rows without a slot)
        pool = {k: v[:, :st["rows"]] for k, v in st["planes"].items()}
        return [pool["k"].view(torch.float8_e4m3fn), pool["k_scale"], pool["v"].view(torch.float8_e4m3fn), pool["v_scale"]]
    if op == "decode":
        if own:
            kvq.kvq_kv8_decode(st["problem"], st["out"], st["lse"], st["workspace"])
        else:
            _plain_decode(st)
        return [st["out"], st["lse"]]
    if op == "beam":
        if own:
            kvq.kvq_beam_select(st["problem"], st["workspace"])
        else:
            _plain_beam(st)
        return [st["out_score"], st["out_token"], st["out_parent"], st["out_finished"]]
    if op == "fork":
        if own:
            kvq.kvq_fork_pages(st["plan"], st["workspace"])
            kvq.kvq_copy_pages(st["copy"])
        else:
            _plain_fork(st)
            _plain_copy(st)
        tables = [st["table"], st["held"], st["seq_len"], st["n_free"], st["free"]]
    else:
        if own:
            kvq.kvq_compact_pages(st["plan"], st["workspace"])
            kvq.kvq_copy_pages(st["copy"])
        else:
            _plain_compact(st)
            _plain_copy(st)
        tables = [st["new_table"], st["free"], st["n_free"], st["n_used"]]
    pl = st["planes"]
    return tables + [st["src"], st["dst"], st["rows"], st["n_copy"], pl["k"].view(torch.float8_e4m3fn), pl["k_scale"],
                     pl["v"].view(torch.float8_e4m3fn), pl["v_scale"]]


# ---------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None                                           # whole numbers, and bytes that are moved
    st = prepare(case, seed)
    if op == "append":
        # a code next to a border has no value of its own in 64 bits, so the codes are left out
        out = [None, None, None, None]
        go = torch.nonzero(st["slot"] >= 0)[:, 0]
        for i, x in ((1, "k"), (3, "v")):
            out[i] = torch.zeros(case["n_kv"], st["rows"], dtype=torch.float64, device="cuda")
            out[i][:, st["slot"][go].long()] = (st[x][go].double().abs().max(2).values / 448.0).T
        return out
    if op == "beam":
        R, B, V, K = case["n_req"], case["n_beam"], case["vocab"], case["n_out"]
        best = torch.full((R, K), -math.inf, dtype=torch.float64, device="cuda")
        for r in range(R):
            rows = []
            for b in range(B):
                s = st["score"][r, b].double()
                x = st["logits"][r, b].double()
                rows.append(s.view(1) if st["finished"][r, b] else s + x - torch.logsumexp(x, 0))
            v = torch.sort(torch.nan_to_num(torch.cat(rows), nan=-math.inf), descending=True).values[:K]
            best[r, :v.shape[0]] = v
        return [best, None, None, None]
    n, kv, G, d = case["n_seq"], case["n_kv"], case["group"], case["dim"]
    out = torch.zeros(n, kv * G, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, kv * G), -math.inf, dtype=torch.float64, device="cuda")
    pl = st["planes"]
    for s in range(n):
        L = int(st["lens"][s])
        a = max(0, L - case["window"]) if case["window"] else 0
        pos = np.arange(a, L)
        if L == 0:
            continue
        if st["table"] is None:
            rows = pos + s * st["stride"]
        else:
            rows = st["table"][s].cpu().numpy()[pos // case["page"]].astype(np.int64) * case["page"] + pos % case["page"]
        rows = torch.from_numpy(rows).cuda()
        for h in range(kv):
            K = pl["k"][h, rows].view(torch.float8_e4m3fn).double() * pl["k_scale"][h, rows].double()[:, None]
            V = pl["v"][h, rows].view(torch.float8_e4m3fn).double() * pl["v_scale"][h, rows].double()[:, None]
            w = st["q"][s, h * G:(h + 1) * G].double() @ K.T * st["scale"]
            z = torch.logsumexp(w, 1)
            out[s, h * G:(h + 1) * G] = torch.exp(w - z[:, None]) @ V
            lse[s, h * G:(h + 1) * G] = z
    return [out, lse]


# ---------------------------------------------------------------------------------------
# costs
# ---------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "append":
        n = case["rows"] * case["n_kv"] * 2
        return dict(bytes=n * (case["dim"] * (2 if case["bf16"] else 4) + case["dim"] + 4) + 4 * case["rows"], flops=2 * n * case["dim"])
    if op == "decode":
        T = case["T"]
        seen = case["n_seq"] * (min(T, case["window"]) if case["window"] else T)
        if case["ragged"]:                                    # lengths are uniform between T/64 and T, the first is T
            lens = [T / 64 + (T - T / 64) * (i + 0.5) / 64 for i in range(64)]
            mean = sum(min(x, case["window"] or x) for x in lens) / 64
            seen = (case["n_seq"] - 1) * mean + min(T, case["window"] or T)
            seen -= mean if case["n_seq"] >= 8 else 0
        H = case["n_kv"] * case["group"]
        return dict(bytes=int(seen * case["n_kv"] * 2 * (case["dim"] + 4) + case["n_seq"] * H * (4 * case["dim"] + 4)),
                    flops=int(seen * H * 4 * case["dim"]))
    if op == "beam":
        n = case["n_req"] * case["n_beam"]
        return dict(bytes=n * (case["vocab"] * (2 if case["bf16"] else 4) + 8) + case["n_req"] * case["n_out"] * 16,
                    flops=n * case["vocab"] * 4)              # maximum, difference, exponential, sum
    row = 2 * case["n_kv"] * (case["dim"] + 4)
    ps = case["page"]
    if op == "fork":
        n, need = case["n_req"] * case["n_beam"], case["T"] * 3 / 4 / ps + 2
        # tables read and written, half of the beams copy half a page
        return dict(bytes=int(n * (need * 8 + 16) + n / 2 * (ps / 2) * row * 2), flops=0)
    moved = case["n_pages"] * case["used"] * (1 - case["used"])
    held = case["n_pages"] * case["used"]
    return dict(bytes=int(held * 8 + (case["n_pages"] - held) * 4 + moved * (12 + ps * row * 2)), flops=0)
