"""The entry points for beam search over a paged fp8 K/V cache without a GPU: their argument errors
(nothing is launched), the workspaces, the struct layouts and the checks of the binding."""
import ctypes as C
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000            # a 64 KiB-aligned address that is never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_kv_cache_fp8_gb300 as k
    return k


def fill(struct, base, kw):
    for k, v in {**base, **kw}.items():
        setattr(struct, k, v)
    return struct


def cache(kvq, **kw):
    return fill(kvq.Kv8Cache(), dict(k=FAKE, k_scale=FAKE, v=FAKE, v_scale=FAKE, n_rows=4096, n_kv=4, head_dim=128), kw)


def test_append_kv8_argument_errors(kvq):
    def call(k=FAKE, kr=512, kh=128, v=FAKE, vr=512, vh=128, kind=1, rows=4, slot=FAKE, status=None, **kw):
        c = cache(kvq, **kw)
        return kvq.lib().kvq_append_kv8(k, kr, kh, v, vr, vh, kind, rows, slot, C.byref(c), status, None)
    assert kvq.lib().kvq_append_kv8(FAKE, 512, 128, FAKE, 512, 128, 1, 4, FAKE, None, None, None) == 1
    for bad in (dict(rows=-1), dict(kind=2), dict(head_dim=96), dict(n_kv=0), dict(n_kv=65536), dict(kh=127), dict(vh=64),
                dict(kr=-8), dict(vr=-8), dict(k=None), dict(v=None), dict(slot=None), dict(n_rows=-1)):
        assert call(**bad) == 1, bad
    # (a plane is a field of the same name as an argument)
    for name in ("k", "v", "k_scale", "v_scale"):
        c = cache(kvq)
        setattr(c, name, None)
        assert kvq.lib().kvq_append_kv8(FAKE, 512, 128, FAKE, 512, 128, 1, 4, FAKE, C.byref(c), None, None) == 1
        c = cache(kvq)
        setattr(c, name, FAKE + (8 if len(name) == 1 else 2))
        assert kvq.lib().kvq_append_kv8(FAKE, 512, 128, FAKE, 512, 128, 1, 4, FAKE, C.byref(c), None, None) == 4
    for bad in (dict(k=FAKE + 8), dict(v=FAKE + 8), dict(kr=516), dict(vr=516), dict(kh=132), dict(vh=132), dict(kind=0, kr=514),
                dict(slot=FAKE + 2), dict(status=FAKE + 1)):
        assert call(**bad) == 4, bad
    assert call(rows=0, k=None, v=None, slot=None) == 0


def kv8(kvq, c=None, **kw):
    base = dict(n_seq=3, n_qh=32, max_seq_len=65536, window=0, seq_len=FAKE, block_table=FAKE, max_pages=64, page_size=64,
                seq_stride_rows=0, cache=c or cache(kvq), q=FAKE, ldq=4096, sm_scale=0.1)
    return fill(kvq.Kv8Problem(), base, kw)


def test_kv8_decode_argument_errors(kvq):
    L = kvq.lib()

    def call(out=FAKE, lse=None, ws=None, n=0, status=None, **kw):
        return L.kvq_kv8_decode(C.byref(kv8(kvq, **kw)), out, lse, ws, n, status, None)
    assert L.kvq_kv8_decode(None, FAKE, None, None, 0, None, None) == 1
    for bad in (dict(n_seq=-1), dict(n_seq=65536), dict(n_qh=0), dict(n_qh=30), dict(n_qh=65540), dict(max_seq_len=-1),
                dict(max_seq_len=(1 << 30) + 1), dict(window=-1), dict(sm_scale=NAN), dict(sm_scale=INF), dict(max_pages=0),
                dict(page_size=0), dict(block_table=None, seq_stride_rows=-1), dict(seq_len=None), dict(q=None), dict(ldq=4088),
                dict(ldq=-8), dict(out=None), dict(c=cache(kvq, head_dim=96)), dict(c=cache(kvq, n_kv=0)),
                dict(c=cache(kvq, n_rows=-1)), dict(c=cache(kvq, v=None)), dict(c=cache(kvq, k_scale=None))):
        assert call(**bad) == 1, bad
    for bad in (dict(q=FAKE + 8), dict(ldq=4100), dict(c=cache(kvq, k=FAKE + 8)), dict(c=cache(kvq, v_scale=FAKE + 2)),
                dict(seq_len=FAKE + 2), dict(block_table=FAKE + 1), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(status=FAKE + 2)):
        assert call(**bad) == 4, bad
    need = L.kvq_kv8_decode_workspace(C.byref(kv8(kvq)))
    assert need > 0
    assert call() == 5 and call(ws=FAKE, n=need - 1) == 5 and call(ws=FAKE + 128, n=need) == 4
    assert call(n_seq=0, seq_len=None, q=None, out=None) == 0
    assert L.kvq_kv8_decode_workspace(C.byref(kv8(kvq, n_seq=0))) == 0
    assert L.kvq_kv8_decode_workspace(C.byref(kv8(kvq, max_seq_len=1024))) == 0        # short units need none
    assert L.kvq_kv8_decode_workspace(C.byref(kv8(kvq, n_qh=30))) == 0


def beam(kvq, **kw):
    base = dict(n_req=2, n_beam=4, vocab=1000, n_out=4, x_type=1, eos=2, pad=0, logits=FAKE, ld=1000, score=FAKE, finished=None,
                out_score=FAKE + 256, out_token=FAKE, out_parent=FAKE, out_finished=None)
    return fill(kvq.BeamProblem(), base, kw)


def test_beam_select_argument_errors(kvq):
    L = kvq.lib()

    def call(ws=None, n=0, status=None, **kw):
        return L.kvq_beam_select(C.byref(beam(kvq, **kw)), ws, n, status, None)
    assert L.kvq_beam_select(None, None, 0, None, None) == 1
    for bad in (dict(x_type=2), dict(n_req=-1), dict(n_req=65536), dict(n_beam=0), dict(n_beam=65), dict(n_out=0), dict(n_out=129),
                dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(eos=-2), dict(ld=999), dict(logits=None), dict(score=None),
                dict(out_score=None), dict(out_token=None), dict(out_parent=None), dict(n_out=8, out_score=FAKE),
                dict(n_out=8, finished=FAKE, out_finished=FAKE)):
        assert call(**bad) == 1, bad
    for bad in (dict(logits=FAKE + 1), dict(x_type=0, logits=FAKE + 2), dict(score=FAKE + 2), dict(finished=FAKE + 1),
                dict(out_token=FAKE + 2), dict(status=FAKE + 2)):
        assert call(**bad) == 4, bad
    need = L.kvq_beam_select_workspace(C.byref(beam(kvq)))
    assert need > 0 and call() == 5 and call(ws=FAKE, n=need - 1) == 5 and call(ws=FAKE + 64, n=need) == 4
    assert call(n_req=0, logits=None) == 0
    assert L.kvq_beam_select_workspace(C.byref(beam(kvq, n_beam=65))) == 0


def fork(kvq, **kw):
    base = dict(n_seq=4, max_pages=8, page_size=64, n_pages=100, parent=FAKE, keep_len=None, block_table=FAKE, n_held=FAKE + 64,
                free_list=FAKE, n_free=FAKE, seq_len=FAKE + 128, copy_src=FAKE, copy_dst=FAKE, copy_rows=FAKE, n_copy=FAKE)
    return fill(kvq.ForkPlan(), base, kw)


def compact(kvq, **kw):
    base = dict(n_seq=4, max_pages=8, page_size=64, n_pages=101, max_copy=50, block_table=FAKE, n_held=FAKE, new_table=FAKE,
                free_list=FAKE, n_free=FAKE, n_used=FAKE, copy_src=FAKE, copy_dst=FAKE, copy_rows=FAKE, n_copy=FAKE)
    return fill(kvq.CompactPlan(), base, kw)


@pytest.mark.parametrize("make,entry,arrays,own", [
    (fork, "kvq_fork_pages", ("parent", "block_table", "n_held", "free_list", "n_free", "seq_len", "copy_src", "copy_dst",
                              "copy_rows", "n_copy"),
     (dict(keep_len=FAKE + 128), dict(parent=FAKE + 128), dict(parent=FAKE + 64))),
    (compact, "kvq_compact_pages", ("block_table", "n_held", "new_table", "free_list", "n_free", "n_used", "copy_src", "copy_dst",
                                    "copy_rows", "n_copy"), (dict(max_copy=49),)),
])
def test_page_plan_argument_errors(kvq, make, entry, arrays, own):
    L = kvq.lib()
    run, size = getattr(L, entry), getattr(L, entry + "_workspace")

    def call(ws=None, n=0, status=None, **kw):
        return run(C.byref(make(kvq, **kw)), ws, n, status, None)
    assert run(None, None, 0, None, None) == 1
    for bad in (dict(n_seq=-1), dict(n_seq=65536), dict(max_pages=0), dict(max_pages=(1 << 20) + 1), dict(page_size=0),
                dict(n_pages=-1), dict(n_pages=1 << 26), *({name: None} for name in arrays), *own):
        assert call(**bad) == 1, bad
        assert size(C.byref(make(kvq, **bad))) == 0, bad
    for name in arrays:
        assert call(**{name: FAKE + 2}) == 4, name
    assert call(status=FAKE + 1) == 4
    need = size(C.byref(make(kvq)))
    assert need > 0 and call() == 5 and call(ws=FAKE, n=need - 1) == 5 and call(ws=FAKE + 32, n=need) == 4


@pytest.mark.parametrize("make,entry", [(fork, "kvq_fork_pages"), (compact, "kvq_compact_pages")])
def test_page_plans_of_the_largest_pools(kvq, make, entry):
    """The plans count pages in 32 bits, a list's pushes past its end among them: a pool of more than 2^29 pages, or a copy
    list of more than 2^30 entries, is refused."""
    L = kvq.lib()
    run, size = getattr(L, entry), getattr(L, entry + "_workspace")
    big = dict(page_size=1, **(dict(max_copy=1 << 30) if make is compact else {}))
    for pages in ((1 << 29) + 1, 1 << 30, (1 << 31) - 9000, (1 << 31) - 3, (1 << 31) - 1):
        p = make(kvq, n_pages=pages, **big)
        assert run(C.byref(p), None, 0, None, None) == 1 and size(C.byref(p)) == 0, pages
    p = make(kvq, n_pages=1 << 29, **big)
    # a byte of marks a page in the tables before and after, for each of 8 CTAs; or the pages' new numbers
    assert size(C.byref(p)) >= (16 << 29 if make is fork else 4 << 29) and run(C.byref(p), None, 0, None, None) == 5
    if make is compact:
        assert run(C.byref(make(kvq, max_copy=(1 << 30) + 1)), None, 0, None, None) == 1


def test_fork_of_nothing(kvq):
    none = dict(n_seq=0, parent=None, block_table=None, n_held=None, seq_len=None, copy_src=None, copy_dst=None, copy_rows=None)
    assert kvq.lib().kvq_fork_pages(C.byref(fork(kvq, **none)), None, 0, None, None) == 0


def test_copy_pages_argument_errors(kvq):
    L = kvq.lib()

    def call(plane=None, planes=1, status=None, **kw):
        p = (kvq.Plane * 64)()
        for i in range(64):
            fill(p[i], dict(base=FAKE, row_bytes=128, n_rows=1000, n_outer=2, outer_stride=128000), plane or {})
        base = dict(n_planes=planes, page_size=64, max_copy=4, copy_src=FAKE, copy_dst=FAKE, copy_rows=FAKE, n_copy=FAKE)
        d = fill(kvq.PageCopy(), base, kw)
        d.planes = C.cast(p, C.POINTER(kvq.Plane))
        return L.kvq_copy_pages(C.byref(d), status, None)
    assert L.kvq_copy_pages(None, None, None) == 1
    for bad in (dict(planes=0), dict(planes=65), dict(page_size=0), dict(max_copy=-1), dict(copy_src=None), dict(copy_dst=None),
                dict(copy_rows=None), dict(n_copy=None), dict(plane=dict(base=None)), dict(plane=dict(row_bytes=0)),
                dict(plane=dict(n_rows=-1)), dict(plane=dict(n_outer=0)), dict(plane=dict(outer_stride=127999)),
                dict(plane=dict(row_bytes=1 << 62, n_outer=1)), dict(plane=dict(n_outer=1 << 40)),
                dict(plane=dict(row_bytes=1 << 40, n_outer=1))):
        assert call(**bad) == 1, bad
    assert call(copy_src=FAKE + 2) == 4 and call(status=FAKE + 2) == 4
    assert call(max_copy=0, copy_src=None, n_copy=None) == 0


def test_injected_faults(kvq):
    L = kvq.lib()
    calls = dict(
        kvq_append_kv8=lambda: L.kvq_append_kv8(None, 0, 0, None, 0, 0, 0, 0, None, None, None, None),
        kvq_kv8_decode=lambda: L.kvq_kv8_decode(None, None, None, None, 0, None, None),
        kvq_beam_select=lambda: L.kvq_beam_select(None, None, 0, None, None),
        kvq_fork_pages=lambda: L.kvq_fork_pages(None, None, 0, None, None),
        kvq_compact_pages=lambda: L.kvq_compact_pages(None, None, 0, None, None),
        kvq_copy_pages=lambda: L.kvq_copy_pages(None, None, None))
    try:
        for name, call in calls.items():
            kvq.kvq_set_fault(f"{name}:6")
            assert call() == 6, name
    finally:
        kvq.kvq_set_fault(None)


@pytest.mark.parametrize("source", ["kvq_kv8.cu", "kvq_beam.cu", "kvq_fork.cu"])
def test_kernels_read_behind_the_wait(source):
    """A kernel that may start under the one before it reads no array ahead of its own wait: what earlier kernels wrote is
    visible to the threads that wait."""
    text = open(os.path.join(ROOT, "quantized_kv_cache_fp8_gb300", "csrc", source)).read()
    kernels = re.findall(r"__global__.*?(\w+_kernel)\((.*?)grid_dependency_wait\(\);", text, re.S)
    assert len(kernels) == text.count("__global__") > 0
    for name, ahead in kernels:
        assert "__global__" not in ahead, name               # (its own wait)
        assert not re.search(r"\b[ap]\.\w+(\.\w+)*\[|__ld\w+\(|atomic", ahead), name


def test_struct_layouts(kvq, tmp_path):
    """The ctypes mirrors have the size and the last field's offset that the C header gives."""
    pairs = [(kvq.Kv8Cache, "kvq_kv8_cache", "head_dim"), (kvq.Kv8Problem, "kvq_kv8_problem", "sm_scale"),
             (kvq.BeamProblem, "kvq_beam_problem", "out_finished"), (kvq.ForkPlan, "kvq_fork_plan", "n_copy"),
             (kvq.CompactPlan, "kvq_compact_plan", "n_copy"), (kvq.Plane, "kvq_plane", "outer_stride"),
             (kvq.PageCopy, "kvq_page_copy", "n_copy")]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvq.h"\nint main(void){' + "".join(
        f'printf("%zu %zu\\n", sizeof({c}), offsetof({c}, {f}));' for _, c, f in pairs) + "return 0;}\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    want = [x for s, _, f in pairs for x in (C.sizeof(s), getattr(s, f).offset)]
    assert [int(x) for x in got] == want


# --- the binding's own checks (host tensors: refused before anything is launched) ----------------

def planes(kv=2, rows=64, d=64):
    return dict(k=torch.zeros(kv, rows, d, dtype=torch.uint8), v=torch.zeros(kv, rows, d, dtype=torch.uint8),
                k_scale=torch.zeros(kv, rows), v_scale=torch.zeros(kv, rows))


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses(kvq):
    x = torch.zeros(3, 2, 64)
    good = dict(k=x, v=x, slot_map=i32(3), planes=planes())
    for bad in (dict(k=x.half(), v=x.half()), dict(v=x.bfloat16()), dict(v=x[:2]), dict(k=x[..., :32], v=x[..., :32]),
                dict(k=x[..., ::2], v=x[..., ::2]), dict(slot_map=i32(2)), dict(slot_map=torch.zeros(3)),
                dict(planes={**planes(), "v": planes()["v"][:, :32]}), dict(planes={**planes(), "k_scale": torch.zeros(2, 65)}),
                dict()):
        with pytest.raises(ValueError):
            kvq.kvq_append_kv8(**{**good, **bad})

    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    good = dict(seq_len=i32(2), q=q, sm_scale=1.0, max_seq_len=8, cache=planes(), block_table=i32(2, 3), page_size=16)
    p = kvq.make_kv8_problem(**good)
    assert (p.n_seq, p.n_qh, p.ldq, p.cache.n_kv, p.max_pages) == (2, 4, 256, 2, 3)
    for bad in (dict(q=q.float()), dict(q=q[:, ::2]), dict(q=q[..., :32]), dict(seq_len=i32(3)), dict(block_table=i32(3, 3))):
        with pytest.raises(ValueError):
            kvq.make_kv8_problem(**{**good, **bad})
    out = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for bad in (dict(out=out.float()), dict(out=out[:1]), dict(out=out, lse=torch.zeros(2, 3)), dict(out=out)):
        with pytest.raises(ValueError):
            kvq.kvq_kv8_decode(p, **bad)

    good = dict(logits=torch.zeros(2, 4, 50), score=torch.zeros(2, 4), out_score=torch.zeros(2, 8), out_token=i32(2, 8),
                out_parent=i32(2, 8), finished=i32(2, 4), out_finished=i32(2, 8))
    p = kvq.make_beam_problem(**good)
    assert (p.n_req, p.n_beam, p.vocab, p.n_out, p.ld, p.x_type) == (2, 4, 50, 8, 50, 0)
    assert kvq.make_beam_problem(**{**good, "logits": torch.zeros(2, 4, 64)[..., :50]}).ld == 64
    for bad in (dict(logits=torch.zeros(2, 4, 50).half()), dict(logits=torch.zeros(2, 4, 100)[..., ::2]),
                dict(logits=torch.zeros(2, 5, 50)[:, :4]), dict(score=torch.zeros(2, 5)), dict(out_token=i32(2, 7)),
                dict(finished=torch.zeros(2, 4, dtype=torch.bool))):
        with pytest.raises(ValueError):
            kvq.make_beam_problem(**{**good, **bad})
    with pytest.raises(ValueError):
        kvq.kvq_beam_select(p)

    lists = dict(copy_src=i32(4), copy_dst=i32(4), copy_rows=i32(4), n_copy=i32(1))
    good = dict(parent=i32(4), block_table=i32(4, 3), n_held=i32(4), free_list=i32(9), n_free=i32(1), seq_len=i32(4), page_size=16,
                **lists)
    p = kvq.make_fork_plan(**good)
    for name in ("parent", "n_held", "seq_len", "copy_src", "copy_dst", "copy_rows", "n_copy", "n_free"):
        with pytest.raises(ValueError):
            kvq.make_fork_plan(**{**good, name: i32(5)})
    with pytest.raises(ValueError):
        kvq.kvq_fork_pages(p)
    good = dict(block_table=i32(4, 3), n_held=i32(4), new_table=i32(4, 3), free_list=i32(9), n_free=i32(1), n_used=i32(1),
                page_size=16, **lists)
    p = kvq.make_compact_plan(**good)
    for bad in (dict(new_table=i32(4, 4)), dict(copy_dst=i32(5)), dict(n_used=i32(2)), dict(n_held=i32(3))):
        with pytest.raises(ValueError):
            kvq.make_compact_plan(**{**good, **bad})
    with pytest.raises(ValueError):
        kvq.kvq_compact_pages(p)
    d = kvq.make_page_copy(caches=[planes(), torch.zeros(64, 2, 144, dtype=torch.uint8)], page_size=16, **lists)
    got = [(p.row_bytes, p.n_rows, p.n_outer, p.outer_stride) for p in d._planes]
    assert got == [(64, 64, 2, 4096), (4, 64, 2, 256), (64, 64, 2, 4096), (4, 64, 2, 256), (288, 64, 1, 18432)]
    with pytest.raises(ValueError):
        kvq.make_page_copy(caches=[torch.zeros(64, 4).t()], page_size=16, **lists)
    with pytest.raises(ValueError):
        kvq.kvq_copy_pages(d)
