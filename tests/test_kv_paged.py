"""The paged cache's index arithmetic and work split (plain host code of
csrc/kv_paged.cuh), and the host-side refusals of the norm, append and
attention entry points.  CPU only."""
import ctypes
import os
import random
import subprocess

import pytest

import nvfp4_w4a4_quantized_04_b200 as nv
from nvfp4_w4a4_quantized_04_b200 import build as nvbuild

SOURCE = r"""
#include "kv_paged.cuh"
using namespace nvfp4::kv;
extern "C" {
long long row_of(long long page, int heads, int ps, int head, int row) { return pool_row(page, heads, ps, head, row); }
int split(long long slot, long long pages, int ps, long long *page, int *row) {
  int64_t p = 0; bool ok = split_slot(slot, pages, ps, p, *row); *page = p; return ok;
}
int ok_page(int page, long long pages) { return page_ok(page, pages); }
long long visible(long long len, long long q, long long j, int causal) { return visible_keys(len, q, j, causal != 0); }
long long per(long long total, long long grid, long long least) { return steps_per_cta(total, grid, least); }
int slot_of(long long c, long long per, long long first) { return part_slot(c, per, first); }
void part_of(long long c, long long per, long long start, int fixed, int steps, int *lo, int *hi) {
  item_part(c, per, start, fixed, steps, *lo, *hi);
}
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv")
    (d / "k.cpp").write_text(SOURCE)
    so = d / "k.so"
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I" + nvbuild.CSRC, str(d / "k.cpp"),
                           "-o", str(so)])
    L = ctypes.CDLL(str(so))
    i64 = ctypes.c_longlong
    L.row_of.restype = L.visible.restype = L.per.restype = i64
    L.row_of.argtypes = [i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    L.split.argtypes = [i64, i64, ctypes.c_int, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_int)]
    L.ok_page.argtypes = [ctypes.c_int, i64]
    L.visible.argtypes = [i64, i64, i64, ctypes.c_int]
    L.per.argtypes = [i64, i64, i64]
    L.slot_of.argtypes = [i64, i64, i64]
    L.part_of.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                          ctypes.POINTER(ctypes.c_int)]
    return L


def test_slots_and_rows(host):
    page, row = ctypes.c_longlong(), ctypes.c_int()
    for ps in (16, 48, 64, 128):
        for pages in (0, 1, 7, 1 << 24):
            for slot in (-(1 << 62), -1, 0, 1, ps - 1, ps, pages * ps - 1, pages * ps, pages * ps + 1, 1 << 62):
                ok = host.split(slot, pages, ps, page, row)
                assert bool(ok) == (0 <= slot < pages * ps)
                if ok:
                    assert (page.value, row.value) == divmod(slot, ps)
    # every (page, head, row) has a row of its own inside the pool
    seen = {host.row_of(p, 3, 16, h, r) for p in range(5) for h in range(3) for r in range(16)}
    assert seen == set(range(5 * 3 * 16))
    # past 32 bits
    assert host.row_of((1 << 31) - 1, 1024, 128, 1023, 127) == ((1 << 31) - 1) * 1024 * 128 + 1023 * 128 + 127
    for page_id, pages, good in ((-1, 4, 0), (0, 4, 1), (3, 4, 1), (4, 4, 0), (-(1 << 31), 4, 0), (0, 0, 0)):
        assert bool(host.ok_page(page_id, pages)) == bool(good)


def test_visible_keys(host):
    for n in range(0, 9):
        for q in range(1, 6):
            for j in range(q):
                assert host.visible(n, q, j, 1) == max(0, n - (q - 1 - j))
                assert host.visible(n, q, j, 0) == n


@pytest.mark.parametrize("seed", range(20))
def test_work_split_covers_every_step_once(host, seed):
    """Walk the line of steps as the kernel's CTAs do: every step of every item
    is taken once, an item that several CTAs share has its parts in distinct
    workspace slots, and the joining kernel's arithmetic finds exactly those."""
    r = random.Random(seed)
    items, at = [], 0
    for _ in range(r.randrange(1, 40)):
        n = r.choice((0, 1, 2, 3, 5, 17, 100, 1000))
        if n:
            items.append((at, n))
            at += n
    total = at
    grid, least = r.choice((1, 2, 7, 148, 592)), r.choice((1, 4))
    per = host.per(total, grid, least)
    assert per >= least and per * grid >= total
    taken, slots, parts = set(), set(), {}
    for c in range(grid):
        pos, end = min(total, c * per), min(total, (c + 1) * per)
        while pos < end:
            first, n = next(i for i in items if i[0] <= pos < i[0] + i[1])
            stop = min(first + n, end)
            assert not taken & set(range(pos, stop))
            taken |= set(range(pos, stop))
            if not (pos == first and stop == first + n):
                key = (c, host.slot_of(c, per, first))
                assert key not in slots
                slots.add(key)
                parts.setdefault(first, []).append(key)
            pos = stop
    assert taken == set(range(total))
    for first, n in items:
        c0, c1 = first // per, (first + n - 1) // per
        want = [] if c0 == c1 else [(c, host.slot_of(c, per, first)) for c in range(c0, c1 + 1)]
        assert parts.get(first, []) == want


@pytest.mark.parametrize("seed", range(20))
def test_weighted_split_covers_every_step_once(host, seed):
    """The same for a line on which every item takes a fixed cost before its steps."""
    r = random.Random(100 + seed)
    fixed, items, at = r.choice((0, 1, 2, 5)), [], 0
    for _ in range(r.randrange(1, 60)):
        n = r.choice((1, 2, 3, 17, 100, 700))
        items.append((at, n))
        at += n + fixed
    grid = r.choice((1, 2, 7, 148))
    per = host.per(at, grid, 1)
    lo, hi = ctypes.c_int(), ctypes.c_int()
    parts, slots = {}, set()
    for c in range(grid):
        for start, n in items:
            host.part_of(c, per, start, fixed, n, lo, hi)
            inside = start < (c + 1) * per and start + fixed + n > c * per
            assert inside or lo.value >= hi.value
            if lo.value < hi.value:
                parts.setdefault(start, []).append((c, lo.value, hi.value))
                if hi.value - lo.value < n:
                    key = (c, host.slot_of(c, per, start))
                    assert key not in slots
                    slots.add(key)
    for start, n in items:
        got = parts[start]
        assert [p[1] for p in got] == [0] + [p[2] for p in got][:-1] and got[-1][2] == n
        assert [p[0] for p in got] == list(range((start + fixed) // per, (start + fixed + n - 1) // per + 1))


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return nv.load_library()


F = 1 << 20          # a pointer that is never dereferenced: the checks fail first


def _call(fn, names, base, **change):
    a = dict(base, **change)
    vals = [a[n] for n in names]
    return fn(*vals)


NORM = "x ld_x res ld_res rows K w eps ro ld_ro y fmt scale q sf layout st stream".split()
NORM_OK = dict(x=F, ld_x=256, res=F, ld_res=256, rows=4, K=256, w=F, eps=1e-6, ro=F, ld_ro=256, y=None, fmt=1, scale=F,
               q=F, sf=F, layout=1, st=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(K=24, ld_x=24), nv.ERR_UNSUPPORTED_SHAPE), (dict(K=0), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(K=65552, ld_x=65552, ld_res=65552, ld_ro=65552), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(K=32), nv.ERR_UNSUPPORTED_SHAPE), (dict(rows=-1), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(rows=1 << 31), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(ld_x=248), nv.ERR_INVALID_ARG), (dict(ld_x=260), nv.ERR_INVALID_ARG), (dict(ld_res=128), nv.ERR_INVALID_ARG),
    (dict(ld_ro=257), nv.ERR_INVALID_ARG), (dict(fmt=3), nv.ERR_INVALID_ARG), (dict(layout=2), nv.ERR_INVALID_ARG),
    (dict(eps=-1.0), nv.ERR_INVALID_ARG), (dict(eps=float("nan")), nv.ERR_INVALID_ARG),
    (dict(x=None), nv.ERR_INVALID_ARG), (dict(x=F + 2), nv.ERR_INVALID_ARG), (dict(w=None), nv.ERR_INVALID_ARG),
    (dict(scale=None), nv.ERR_INVALID_ARG), (dict(q=None), nv.ERR_INVALID_ARG), (dict(sf=None), nv.ERR_INVALID_ARG),
    (dict(q=F + 4), nv.ERR_INVALID_ARG), (dict(fmt=0), nv.ERR_INVALID_ARG), (dict(y=F + 8), nv.ERR_INVALID_ARG),
    (dict(rows=0, x=None, q=None, sf=None, scale=None), nv.OK)])
def test_norm_refusals(lib, change, want):
    assert _call(lib.nvfp4_add_rmsnorm_quantize, NORM, NORM_OK, **change) == want


APPEND = ("k ld_k v ld_v tokens heads D slots q ld_q hq qo ld_qo pos rope rr rot inter kgs vgs kq ks vq vs pages ps st "
          "stream").split()
APPEND_OK = dict(k=F, ld_k=512, v=F, ld_v=512, tokens=3, heads=4, D=128, slots=F, q=F, ld_q=1024, hq=8, qo=F, ld_qo=1024,
                 pos=F, rope=F, rr=100, rot=64, inter=0, kgs=F, vgs=F, kq=F, ks=F, vq=F, vs=F, pages=9, ps=64, st=None,
                 stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(D=48), nv.ERR_UNSUPPORTED_SHAPE), (dict(D=544, ld_k=4096, ld_v=4096), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(heads=0), nv.ERR_UNSUPPORTED_SHAPE), (dict(tokens=-1), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(ps=8), nv.ERR_UNSUPPORTED_SHAPE), (dict(ps=40), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(pages=-1), nv.ERR_UNSUPPORTED_SHAPE), (dict(rot=48), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(rot=160), nv.ERR_UNSUPPORTED_SHAPE), (dict(hq=0), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(inter=2), nv.ERR_INVALID_ARG), (dict(rope=None), nv.ERR_INVALID_ARG), (dict(rr=0), nv.ERR_INVALID_ARG),
    (dict(pos=None), nv.ERR_INVALID_ARG), (dict(ld_k=504), nv.ERR_INVALID_ARG), (dict(ld_v=516), nv.ERR_INVALID_ARG),
    (dict(ld_q=1016), nv.ERR_INVALID_ARG), (dict(qo=None), nv.ERR_INVALID_ARG), (dict(k=None), nv.ERR_INVALID_ARG),
    (dict(k=F + 8), nv.ERR_INVALID_ARG), (dict(slots=None), nv.ERR_INVALID_ARG), (dict(slots=F + 4), nv.ERR_INVALID_ARG),
    (dict(kgs=None), nv.ERR_INVALID_ARG), (dict(vq=None), nv.ERR_INVALID_ARG), (dict(kq=F + 8), nv.ERR_INVALID_ARG),
    (dict(ks=F + 1), nv.ERR_INVALID_ARG), (dict(vs=F + 8), nv.ERR_INVALID_ARG),
    (dict(tokens=0, k=None, v=None, q=None), nv.OK)])
def test_append_refusals(lib, change, want):
    assert _call(lib.nvfp4_kv_append, APPEND, APPEND_OK, **change) == want


ATTEND = ("q ld_q tokens offs maxq lens batch table maxp hq hkv D kq ks kgs vq vs vgs pages ps scale causal out dt lse ws "
          "st stream").split()
ATTEND_OK = dict(q=F, ld_q=1024, tokens=5, offs=F, maxq=4, lens=F, batch=2, table=F, maxp=10, hq=8, hkv=4, D=128, kq=F,
                 ks=F, kgs=F, vq=F, vs=F, vgs=F, pages=9, ps=64, scale=0.1, causal=1, out=F, dt=1, lse=None, ws=F, st=None,
                 stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(D=96), nv.ERR_UNSUPPORTED_SHAPE), (dict(D=512), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(batch=4097), nv.ERR_UNSUPPORTED_SHAPE), (dict(batch=-1), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(hq=6), nv.ERR_UNSUPPORTED_SHAPE), (dict(hkv=0), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(ps=24), nv.ERR_UNSUPPORTED_SHAPE), (dict(maxp=1 << 30), nv.ERR_UNSUPPORTED_SHAPE),
    (dict(maxp=-1), nv.ERR_UNSUPPORTED_SHAPE), (dict(dt=2), nv.ERR_INVALID_ARG), (dict(causal=2), nv.ERR_INVALID_ARG),
    (dict(scale=0.0), nv.ERR_INVALID_ARG), (dict(scale=float("nan")), nv.ERR_INVALID_ARG),
    (dict(ld_q=1000), nv.ERR_INVALID_ARG), (dict(ld_q=1028), nv.ERR_INVALID_ARG), (dict(maxq=0), nv.ERR_INVALID_ARG),
    (dict(offs=None), nv.ERR_INVALID_ARG), (dict(offs=None, maxq=1), nv.ERR_INVALID_ARG),
    (dict(q=None), nv.ERR_INVALID_ARG), (dict(lens=None), nv.ERR_INVALID_ARG), (dict(table=None), nv.ERR_INVALID_ARG),
    (dict(ws=None), nv.ERR_INVALID_ARG), (dict(ws=F + 16), nv.ERR_INVALID_ARG), (dict(out=F + 8), nv.ERR_INVALID_ARG),
    (dict(kq=None), nv.ERR_INVALID_ARG), (dict(vs=F + 8), nv.ERR_INVALID_ARG), (dict(kgs=None), nv.ERR_INVALID_ARG),
    (dict(batch=0, tokens=0, offs=F), nv.OK), (dict(tokens=0), nv.OK)])
def test_attention_refusals(lib, change, want):
    assert _call(lib.nvfp4_paged_attention, ATTEND, ATTEND_OK, **change) == want


def test_attention_workspace_size(lib):
    f = nv.nvfp4_paged_attention_workspace_size
    assert f(1, 1, 8, 4, 96) == 0 and f(0, 1, 8, 4, 128) == 0 and f(1, 1, 6, 4, 128) == 0 and f(1, 0, 8, 4, 128) == 0
    assert f(1, 1, 8, 4, 128) > 0 and f(1, 1, 8, 4, 128) % 256 == 0
    assert f(64, 4, 32, 4, 256) >= f(1, 1, 32, 4, 256)


def test_layer_refusals():
    """The Python layer names the argument before any device work."""
    torch = pytest.importorskip("torch")
    from nvfp4_w4a4_quantized_04_b200 import layer as L

    def u8(*s):
        return torch.zeros(s, dtype=torch.uint8)
    gs = torch.ones(1)
    with pytest.raises(ValueError, match="k_sf"):
        L.PagedKVCache(u8(2, 4, 16, 64), u8(2, 4, 16, 4), gs, u8(2, 4, 16, 64), u8(2, 4, 16, 8), gs)
    with pytest.raises(ValueError, match="k_gs"):
        L.PagedKVCache(u8(2, 4, 16, 64), u8(2, 4, 16, 8), gs.double(), u8(2, 4, 16, 64), u8(2, 4, 16, 8), gs)
    c = L.PagedKVCache(u8(2, 4, 16, 64), u8(2, 4, 16, 8), gs, u8(2, 4, 16, 64), u8(2, 4, 16, 8), gs)
    kv = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    for bad, match in ((dict(k=kv.float()), "k:"), (dict(k=kv[:, :2]), "heads"), (dict(v=kv[:2]), "v:"),
                       (dict(slots=slots.int()), "slots"), (dict(slots=slots[:2]), "slots"),
                       (dict(rope=torch.zeros(9, 64)), "positions"), (dict(rope=torch.zeros(9, 64).double()), "rope"),
                       (dict(q=kv.transpose(0, 1)), "q:"), (dict(q=kv, q_out=kv[:, :2]), "q_out")):
        with pytest.raises(ValueError, match=match):
            c.append(**dict(dict(k=kv, v=kv, slots=slots), **bad))
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    for bad, match in ((dict(q=q.half()), "q:"), (dict(seq_lens=lens.long()), "seq_lens"),
                       (dict(page_table=table[:1]), "page_table"), (dict(query_offsets=lens), "query_offsets"),
                       (dict(out=q.float()), "out"), (dict(lse=torch.zeros(2, 4)), "lse"),
                       (dict(ws=torch.zeros(16, dtype=torch.uint8)), "ws")):
        with pytest.raises(ValueError, match=match):
            c.attend(**dict(dict(q=q, seq_lens=lens, page_table=table), **bad))
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    for bad, match in ((dict(x=x.float()), "x:"), (dict(weight=w[:32]), "weight"), (dict(residual=x[:1]), "residual"),
                       (dict(residual_out=x[:, :32]), "residual_out"), (dict(q=u8(2, 32)), "q:"),
                       (dict(scale=gs), "scale"), (dict(y=x.float()), "y:")):
        with pytest.raises(ValueError, match=match):
            L.add_rmsnorm_e4m3(**dict(dict(x=x, weight=w), **bad))
    with pytest.raises(ValueError, match="global_scale"):
        L.add_rmsnorm_nvfp4(x, w, torch.ones(2))


def test_rope_table_is_computed_in_64_bits():
    torch = pytest.importorskip("torch")
    import math
    from nvfp4_w4a4_quantized_04_b200 import layer as L
    t = L.rope_table(262144, 32, 1e7, device="cpu")
    assert t.dtype == torch.float32 and tuple(t.shape) == (262144, 32)
    for p in (0, 1, 1000, 262143):
        for i in (0, 1, 7, 15):
            a = p * 1e7 ** (-2 * i / 32)
            # one rounding to fp32, plus the 64-bit angle's own error
            assert abs(t[p, i].item() - math.cos(a)) <= 2.0 ** -24 + 1e-9
            assert abs(t[p, 16 + i].item() - math.sin(a)) <= 2.0 ** -24 + 1e-9
