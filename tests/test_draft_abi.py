"""The entry points for drafted tokens without a GPU: their argument errors (nothing is
launched), the choice of the tree form, and the struct layouts of the binding."""
import ctypes as C
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000            # a 64 KiB-aligned address that is never dereferenced


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


def plan(kvq, **kw):
    base = dict(n_seq=4, max_pages=8, page_size=64, n_pages=100, max_tokens=64, keep_len=FAKE, n_new=FAKE + 64,
                block_table=FAKE, n_held=FAKE, free_list=FAKE, n_free=FAKE, seq_len=FAKE + 128, tok_start=FAKE,
                slot_map=FAKE, tok_pos=None)
    return fill(kvq.PagePlan(), base, kw)


def test_resize_pages_argument_errors(kvq):
    call = lambda **kw: kvq.lib().kvq_resize_pages(C.byref(plan(kvq, **kw)), None, None)
    assert kvq.lib().kvq_resize_pages(None, None, None) == 1
    for bad in (dict(n_seq=-1), dict(n_seq=65536), dict(max_pages=0), dict(max_pages=(1 << 20) + 1), dict(page_size=0), dict(n_pages=-1),
                dict(max_tokens=-1), dict(n_pages=1 << 26, page_size=64), dict(keep_len=None), dict(n_new=None),
                dict(block_table=None), dict(n_held=None), dict(free_list=None), dict(n_free=None),
                dict(seq_len=None), dict(tok_start=None), dict(slot_map=None), dict(seq_len=FAKE),
                dict(seq_len=FAKE + 64)):
        assert call(**bad) == 1, bad
    for bad in (dict(tok_pos=FAKE + 2), dict(slot_map=FAKE + 1), dict(n_free=FAKE + 3)):
        assert call(**bad) == 4, bad
    assert kvq.lib().kvq_resize_pages(C.byref(plan(kvq)), FAKE + 2, None) == 4


def test_append_mla_argument_errors(kvq):
    c = kvq.MlaCache(FAKE, FAKE, FAKE, FAKE, 100)

    def call(x=FAKE, ldx=512, k=FAKE, ldr=64, kind=0, rows=4, slot=FAKE, fmt=1, signs=FAKE, cache=c):
        return kvq.lib().kvq_append_mla(x, ldx, k, ldr, kind, rows, slot, fmt, signs,
                                        None if cache is None else C.byref(cache), None, None)
    assert call(fmt=3) == 3 and call(fmt=9) == 3
    for bad in (dict(rows=-1), dict(kind=2), dict(ldx=511), dict(ldr=63), dict(x=None), dict(k=None), dict(slot=None),
                dict(cache=None), dict(fmt=2, signs=None), dict(cache=kvq.MlaCache(FAKE, None, FAKE, FAKE, 100)),
                dict(cache=kvq.MlaCache(FAKE, FAKE, FAKE, FAKE, -1))):
        assert call(**bad) == 1, bad
    for bad in (dict(x=FAKE + 8), dict(ldx=514), dict(ldr=66), dict(kind=1, ldx=516), dict(slot=FAKE + 2),
                dict(cache=kvq.MlaCache(FAKE + 8, FAKE, FAKE, FAKE, 100)), dict(fmt=2, signs=FAKE + 1)):
        assert call(**bad) == 4, bad
    assert call(rows=0, x=None, slot=None, cache=None) == 0


def tree(kvq, **kw):
    base = dict(n_seq=2, n_q=16, n_heads=64, d_lat=512, d_rope=64, fmt=1, max_seq_len=4096, seq_len=FAKE,
                n_node=None, mask=FAKE, block_table=FAKE, max_pages=64, page_size=64,
                cache=kvq.MlaCache(FAKE, FAKE, FAKE, FAKE, 100000), signs=FAKE, q_lat=FAKE, q_rope=FAKE,
                ldq_lat=512, ldq_rope=64, sm_scale=0.07, impl=0)
    return fill(kvq.TreeProblem(), base, kw)


def test_tree_argument_errors(kvq):
    L = kvq.lib()

    def call(out=FAKE, lse=None, ws=None, n=0, **kw):
        return L.kvq_mla_tree_decode(C.byref(tree(kvq, **kw)), out, lse, ws, n, None, None)
    assert L.kvq_mla_tree_decode(None, FAKE, None, None, 0, None, None) == 1
    for bad in (dict(d_lat=256), dict(d_rope=32), dict(n_seq=-1), dict(n_seq=65536), dict(n_q=0), dict(n_q=65),
                dict(n_heads=0), dict(n_heads=1 << 20), dict(n_heads=(1 << 31) - 1), dict(max_seq_len=-1), dict(max_seq_len=(1 << 30) + 1), dict(impl=3),
                dict(impl=-1), dict(sm_scale=float("nan")), dict(sm_scale=float("inf")), dict(ldq_lat=504),
                dict(ldq_rope=56), dict(page_size=0), dict(max_pages=0), dict(block_table=None, seq_stride_rows=4000),
                dict(impl=1, page_size=20), dict(seq_len=None), dict(q_lat=None), dict(q_rope=None),
                dict(fmt=2, signs=None), dict(cache=kvq.MlaCache(FAKE, FAKE, None, FAKE, 10)), dict(out=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(fmt=3), dict(fmt=0), dict(fmt=2, impl=1)):
        assert call(**bad) == 3, bad
    for bad in (dict(q_lat=FAKE + 8), dict(ldq_lat=516), dict(ldq_rope=68), dict(mask=FAKE + 4), dict(out=FAKE + 8),
                dict(lse=FAKE + 2), dict(cache=kvq.MlaCache(FAKE + 8, FAKE, FAKE, FAKE, 10))):
        assert call(**bad) == 4, bad
    for kw in (dict(), dict(impl=2), dict(fmt=2), dict(page_size=20)):
        need = L.kvq_mla_tree_decode_workspace(C.byref(tree(kvq, **kw)))
        assert need > 0
        assert call(**kw) == 5
        assert call(ws=FAKE, n=need - 1, **kw) == 5
        assert call(ws=FAKE + 64, n=need, **kw) == 4
    assert L.kvq_mla_tree_decode_workspace(C.byref(tree(kvq, n_q=65))) == 0
    assert call(n_seq=0, seq_len=None, out=None) == 0


def test_tree_form(kvq):
    k = lambda **kw: kvq.kvq_mla_tree_decode_kernel(tree(kvq, **kw))
    assert k() == kvq.TREE_PACKED
    assert k(block_table=None, seq_stride_rows=4096) == kvq.TREE_PACKED
    assert k(page_size=8) == kvq.TREE_PACKED
    assert k(page_size=20) == kvq.TREE_PER_QUERY
    for fmt in (kvq.FMT_TQ3, kvq.FMT_TQ4, kvq.FMT_TQ6):
        assert k(fmt=fmt) == kvq.TREE_PER_QUERY
    assert k(impl=2) == kvq.TREE_PER_QUERY and k(impl=1) == kvq.TREE_PACKED
    with pytest.raises(kvq.KvqError) as e:
        k(fmt=kvq.FMT_TQ4, impl=1)
    assert e.value.status == 3


def test_accept_argument_errors(kvq):
    def call(**kw):
        base = dict(n_seq=2, n_q=16, fmt=1, seq_len=FAKE, n_node=None, path=FAKE, n_acc=FAKE, new_len=FAKE,
                    block_table=FAKE, max_pages=8, page_size=20, seq_stride_rows=0,
                    cache=kvq.MlaCache(FAKE, FAKE, FAKE, FAKE, 100))
        return kvq.lib().kvq_accept_mla(C.byref(fill(kvq.AcceptDesc(), base, kw)), None, None)
    assert kvq.lib().kvq_accept_mla(None, None, None) == 1
    assert call(fmt=3) == 3
    for bad in (dict(n_seq=-1), dict(n_q=0), dict(n_q=65), dict(page_size=0), dict(max_pages=0),
                dict(block_table=None, seq_stride_rows=-1), dict(seq_len=None), dict(path=None), dict(n_acc=None),
                dict(new_len=None), dict(cache=kvq.MlaCache(None, FAKE, FAKE, FAKE, 100))):
        assert call(**bad) == 1, bad
    assert call(cache=kvq.MlaCache(FAKE, FAKE, FAKE + 8, FAKE, 100)) == 4
    assert call(n_seq=0, seq_len=None) == 0


def test_accept_refuses_sequences_on_the_same_rows(kvq):
    """Without a block table and without a stride every sequence would move the same rows."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for n_seq, stride, reason in ((2, 0, b"bad paging sizes"), (1, 0, b"NULL pointer"), (2, 1, b"NULL pointer")):
        d = kvq.make_accept(seq_len=i32(n_seq), path=i32(n_seq, 3), n_acc=i32(n_seq), new_len=i32(n_seq), fmt=1,
                            cache=host_planes(512), seq_stride_rows=stride)
        d.cache.lat = None                    # the check behind it: nothing is launched
        assert kvq.lib().kvq_accept_mla(C.byref(d), None, None) == 1 and reason in kvq.lib().kvq_last_error()


def test_misaligned_arrays_are_refused(kvq):
    """Every 32-bit array that a kernel would read at a misaligned address."""
    L = kvq.lib()
    tree_call = lambda st=None, **kw: L.kvq_mla_tree_decode(C.byref(tree(kvq, **kw)), FAKE, None, None, 0, st, None)
    for bad in (dict(seq_len=FAKE + 2), dict(n_node=FAKE + 1), dict(block_table=FAKE + 3), dict(fmt=2, signs=FAKE + 2),
                dict(st=FAKE + 2)):
        assert tree_call(**bad) == 4, bad
    assert tree_call(signs=FAKE + 2) == 5                 # fp8: no signs; the workspace is missing
    base = dict(n_seq=2, n_q=16, fmt=1, seq_len=FAKE, n_node=FAKE, path=FAKE, n_acc=FAKE, new_len=FAKE, block_table=FAKE,
                max_pages=8, page_size=20, seq_stride_rows=0, cache=kvq.MlaCache(FAKE, FAKE, FAKE, FAKE, 100))
    for name in ("seq_len", "n_node", "path", "n_acc", "new_len", "block_table"):
        assert L.kvq_accept_mla(C.byref(fill(kvq.AcceptDesc(), base, {name: FAKE + 2})), None, None) == 4, name
    assert L.kvq_accept_mla(C.byref(fill(kvq.AcceptDesc(), base, {})), FAKE + 2, None) == 4
    c = kvq.MlaCache(FAKE, FAKE, FAKE, FAKE, 100)
    assert L.kvq_append_mla(FAKE, 512, FAKE, 64, 0, 4, FAKE, 1, None, C.byref(c), FAKE + 2, None) == 4


def test_faults_reach_the_new_entries(kvq):
    L = kvq.lib()
    calls = {"kvq_resize_pages": lambda: L.kvq_resize_pages(None, None, None),
             "kvq_append_mla": lambda: L.kvq_append_mla(None, 0, None, 0, 0, 0, None, 0, None, None, None, None),
             "kvq_mla_tree_decode": lambda: L.kvq_mla_tree_decode(None, None, None, None, 0, None, None),
             "kvq_accept_mla": lambda: L.kvq_accept_mla(None, None, None)}
    for name, f in calls.items():
        assert L.kvq_set_fault(f"{name}:7".encode()) == 0
        try:
            assert f() == 7
        finally:
            L.kvq_set_fault(None)


def test_binding_refuses_wrong_tensors(kvq):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    args = dict(keep_len=i32(3), n_new=i32(3), block_table=i32(3, 4), n_held=i32(3), free_list=i32(9),
                n_free=i32(1), page_size=16, seq_len=i32(3), tok_start=i32(4), slot_map=i32(8))
    kvq.make_page_plan(**args)
    for k, v in (("n_new", i32(2)), ("tok_start", i32(3)), ("n_held", torch.zeros(3)), ("tok_pos", i32(7)),
                 ("block_table", i32(3, 8)[:, ::2])):
        with pytest.raises(ValueError):
            kvq.make_page_plan(**{**args, k: v})
    q = torch.zeros(2, 3, 4, 576, dtype=torch.bfloat16)
    planes = dict(lat=torch.zeros(8, 512, dtype=torch.uint8), lat_scale=torch.zeros(8),
                  rope=torch.zeros(8, 64, dtype=torch.uint8), rope_scale=torch.zeros(8))
    args = dict(seq_len=i32(2), q_lat=q[..., :512], q_rope=q[..., 512:], sm_scale=1.0, max_seq_len=8, fmt=1,
                cache=planes)
    p = kvq.make_tree_problem(**args)
    assert (p.ldq_lat, p.ldq_rope) == (576, 576)                        # rows of one fused projection
    for k, v in (("q_lat", q[..., :512].float()), ("q_lat", q[:, :, ::2, :512]), ("q_rope", q[:, :2, :, 512:]),
                 ("mask", torch.zeros(2, 4, dtype=torch.int64)), ("mask", torch.zeros(2, 3, dtype=torch.int32)),
                 ("cache", {**planes, "lat": torch.zeros(8, 256, dtype=torch.uint8)}),
                 ("cache", {**planes, "rope_scale": torch.zeros(7)})):
        with pytest.raises(ValueError):
            kvq.make_tree_problem(**{**args, k: v})
    with pytest.raises(ValueError):
        kvq.kvq_append_mla(torch.zeros(4, 512), torch.zeros(4, 64).bfloat16(), i32(4), 1, None, planes)
    with pytest.raises(ValueError):
        kvq.kvq_append_mla(torch.zeros(4, 512), torch.zeros(4, 64), i32(3), 1, None, planes)


def test_binding_refuses_tensors_of_several_devices(kvq, monkeypatch):
    i32 = lambda *s, device="cpu": torch.zeros(*s, dtype=torch.int32, device=device)
    args = dict(keep_len=i32(3), n_new=i32(3), block_table=i32(3, 4), n_held=i32(3), free_list=i32(9),
                n_free=i32(1), page_size=16, seq_len=i32(3), tok_start=i32(4), slot_map=i32(8))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t.shape == (9,) else 0)
    with pytest.raises(ValueError, match="different devices"):
        kvq.make_page_plan(**args)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    p = kvq.make_page_plan(**args)
    with pytest.raises(ValueError, match="current device"):
        kvq.kvq_resize_pages(p)
    planes = dict(lat=torch.zeros(8, 512, dtype=torch.uint8), lat_scale=torch.zeros(8),
                  rope=torch.zeros(8, 64, dtype=torch.uint8), rope_scale=torch.zeros(8))
    with pytest.raises(ValueError, match="current device"):
        kvq.kvq_append_mla(torch.zeros(4, 512), torch.zeros(4, 64), i32(4), 1, None, planes)
    d = kvq.make_accept(seq_len=i32(2), path=i32(2, 3), n_acc=i32(2), new_len=i32(2), fmt=1, cache=planes)
    with pytest.raises(ValueError, match="current device"):
        kvq.kvq_accept_mla(d)
    q = torch.zeros(2, 3, 4, 576, dtype=torch.bfloat16)
    t = kvq.make_tree_problem(seq_len=i32(2), q_lat=q[..., :512], q_rope=q[..., 512:], sm_scale=1.0, max_seq_len=8, fmt=1,
                              cache=planes)
    with pytest.raises(ValueError, match="current device"):
        kvq.kvq_mla_tree_decode(t, torch.zeros(2, 3, 4, 512, dtype=torch.bfloat16), None, torch.zeros(4096, dtype=torch.uint8))


def host_planes(bytes_a_row):
    return dict(lat=torch.zeros(8, bytes_a_row, dtype=torch.uint8), lat_scale=torch.zeros(8),
                rope=torch.zeros(8, 64, dtype=torch.uint8), rope_scale=torch.zeros(8))


@pytest.mark.parametrize("bad", [torch.zeros(15, dtype=torch.int32), torch.zeros(16, dtype=torch.int16),
                                 torch.zeros(16), torch.zeros(32, dtype=torch.int32)[::2], torch.zeros(512, dtype=torch.int32)],
                         ids=["short", "int16", "float", "strided", "long"])
def test_binding_refuses_wrong_signs(kvq, bad):
    """The kernels read 16 words of signs: a tensor of fewer would be read past its end."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q = torch.zeros(2, 3, 4, 576, dtype=torch.bfloat16)
    args = dict(seq_len=i32(2), q_lat=q[..., :512], q_rope=q[..., 512:], sm_scale=1.0, max_seq_len=8)
    for fmt, width in ((kvq.FMT_TQ4, 256), (kvq.FMT_TQ6, 384), (kvq.FMT_TQ3, 192)):
        planes = host_planes(width)
        kvq.make_tree_problem(**args, fmt=fmt, cache=planes, signs=i32(16))
        with pytest.raises(ValueError, match="signs"):
            kvq.make_tree_problem(**args, fmt=fmt, cache=planes, signs=bad)
        with pytest.raises(ValueError, match="sign_bits"):
            kvq.kvq_append_mla(torch.zeros(4, 512), torch.zeros(4, 64), i32(4), fmt, bad, planes)


def calls_with_status(kvq):
    """The entry points on host tensors that pass every other check, as functions of dev_status."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    planes = host_planes(512)
    plan = kvq.make_page_plan(keep_len=i32(3), n_new=i32(3), block_table=i32(3, 4), n_held=i32(3), free_list=i32(9),
                              n_free=i32(1), page_size=16, seq_len=i32(3), tok_start=i32(4), slot_map=i32(8))
    done = kvq.make_accept(seq_len=i32(2), path=i32(2, 3), n_acc=i32(2), new_len=i32(2), fmt=1, cache=planes)
    q = torch.zeros(2, 3, 4, 576, dtype=torch.bfloat16)
    tree = kvq.make_tree_problem(seq_len=i32(2), q_lat=q[..., :512], q_rope=q[..., 512:], sm_scale=1.0, max_seq_len=8, fmt=1,
                                 cache=planes)
    out = torch.zeros(2, 3, 4, 512, dtype=torch.bfloat16)
    return [lambda st: kvq.kvq_resize_pages(plan, st),
            lambda st: kvq.kvq_append_mla(torch.zeros(4, 512), torch.zeros(4, 64), i32(4), 1, None, planes, st),
            lambda st: kvq.kvq_mla_tree_decode(tree, out, None, torch.zeros(4096, dtype=torch.uint8), st),
            lambda st: kvq.kvq_accept_mla(done, st)]


def test_binding_refuses_wrong_status(kvq, monkeypatch):
    for call in calls_with_status(kvq):
        for bad in (torch.zeros(1, dtype=torch.int16), torch.zeros(1), torch.zeros(0, dtype=torch.int32)):
            with pytest.raises(ValueError, match="dev_status"):
                call(bad)
    there = torch.zeros(1, dtype=torch.int32)
    real = torch.Tensor.get_device
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t is there else real(t))
    for call in calls_with_status(kvq):
        with pytest.raises(ValueError, match="different devices"):
            call(there)


def test_binding_refuses_host_tensors(kvq):
    """Nothing is launched on addresses of the host, whatever the stream."""
    for call in calls_with_status(kvq):
        with pytest.raises(ValueError, match="on the host"):
            call(None)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the host"):
        kvq.kvq_append_mla(torch.zeros(4, 512), torch.zeros(4, 64), i32(4), 1, None, host_planes(512), i32(1), stream=0)


def test_problems_keep_the_planes(kvq):
    """A problem holds the tensors whose addresses it carries, not the dictionary they came in."""
    import gc
    import weakref
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q = torch.zeros(2, 3, 4, 576, dtype=torch.bfloat16)
    for make in (lambda planes: kvq.make_accept(seq_len=i32(2), path=i32(2, 3), n_acc=i32(2), new_len=i32(2), fmt=1, cache=planes),
                 lambda planes: kvq.make_tree_problem(seq_len=i32(2), q_lat=q[..., :512], q_rope=q[..., 512:], sm_scale=1.0,
                                                      max_seq_len=8, fmt=1, cache=planes)):
        planes = host_planes(512)
        refs = {k: weakref.ref(v) for k, v in planes.items()}
        p = make(planes)
        for k in planes:
            planes[k] = None
        gc.collect()
        kept = {"lat": p.cache.lat, "lat_scale": p.cache.lat_scale, "rope": p.cache.rope, "rope_scale": p.cache.rope_scale}
        for k, ref in refs.items():
            assert ref() is not None and ref().data_ptr() == kept[k], k


def test_struct_layouts(kvq, tmp_path):
    structs = dict(kvq_page_plan=kvq.PagePlan, kvq_mla_tree_problem=kvq.TreeProblem, kvq_mla_accept_desc=kvq.AcceptDesc)
    lines = []
    for c, py in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvq.h"\nint main(void){' + "".join(lines) +
                   "return 0;}\n")
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for py in structs.values():
        want += [C.sizeof(py)] + [getattr(py, f).offset for f, _ in py._fields_]
    assert got == want
