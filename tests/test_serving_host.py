"""The host side of the serving operators: which buffers a call writes through, and
what the layer refuses before a kernel could run.  CPU only: the library's calls are
recorded instead of made."""
import contextlib
import random

import pytest

torch = pytest.importorskip("torch")

from nvfp4_w4a4_quantized_04_b200 import layer as L  # noqa: E402
from tests._forms import choose_forms  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    """The library's entry points replaced by a record of their arguments."""
    seen = []

    def fake(name):
        return lambda *a, **k: seen.append((name, a))
    for name in ("nvfp4_quantize", "nvfp4_moe_quantize", "nvfp4_swiglu_quantize", "nvfp4_add_rmsnorm_quantize",
                 "nvfp4_kv_append", "nvfp4_paged_attention", "nvfp4_grouped_gemm_swiglu_nvfp4"):
        monkeypatch.setattr(L, name, fake(name))
    monkeypatch.setattr(L, "_on", lambda t: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return seen


def bf16(*shape):
    return torch.ones(shape, dtype=torch.bfloat16)


# where each entry point gets the global scales that it writes
GS = {"nvfp4_quantize": 8, "nvfp4_moe_quantize": 9, "nvfp4_swiglu_quantize": 6}


@pytest.mark.parametrize("again", ["quantize", "given", "grouped", "moe", "swiglu"])
def test_a_reused_output_never_writes_through_the_callers_scale(calls, again):
    """add_rmsnorm_nvfp4's output holds the model's calibrated scale.  A later
    quantization into the same buffers has scales of its own, one per group."""
    E, K = 4, 64
    scale = torch.full((1,), 0.25)
    offsets = torch.arange(0, E + 1, dtype=torch.int32) * 2
    p = L.empty_packed(8, K, E, offsets, device="cpu")
    got, _, _ = L.add_rmsnorm_nvfp4(bf16(8, K), bf16(K), scale, out=p)
    assert got is p and p.gs is scale
    if again == "quantize":
        L.quantize(bf16(8, K), out=p)
    elif again == "given":
        L.quantize(bf16(8, K), out=p, global_scale=torch.full((1,), 3.0))
        assert p.gs[0] == 3.0
    elif again == "grouped":
        L.quantize(bf16(8, K), offsets=offsets, num_groups=E, out=p)
    elif again == "moe":
        L.moe_quantize(bf16(8, K), torch.zeros(8, 1, dtype=torch.int32), offsets, E, out=p)
    else:
        L.swiglu_quantize(bf16(8, 2 * K), offsets, E, out=p)
    name, args = calls[-1]
    written = args[GS[name]]
    assert written.data_ptr() != scale.data_ptr() and scale[0] == 0.25
    assert written.numel() >= (1 if again in ("quantize", "given") else E) and written is p.gs
    # and the buffers serve the norm again
    L.add_rmsnorm_nvfp4(bf16(8, K), bf16(K), scale, out=p)
    assert p.gs is scale and scale[0] == 0.25


def test_an_output_with_too_few_scales_is_refused(calls):
    E, K = 4, 64
    offsets = torch.arange(0, E + 1, dtype=torch.int32) * 2
    p = L.empty_packed(8, K, E, offsets, device="cpu")
    p.gs = torch.empty(E - 1)
    for call in (lambda: L.quantize(bf16(8, K), offsets=offsets, num_groups=E, out=p),
                 lambda: L.moe_quantize(bf16(8, K), torch.zeros(8, 1, dtype=torch.int32), offsets, E, out=p),
                 lambda: L.swiglu_quantize(bf16(8, 2 * K), offsets, E, out=p)):
        with pytest.raises(ValueError, match="global scales"):
            call()
    assert not calls


def test_the_calibrated_scale_of_the_experts_is_not_written(calls):
    """grouped_gemm_swiglu_nvfp4's output holds the given scales, too."""
    E, K = 2, 64
    offsets = torch.arange(0, E + 1, dtype=torch.int32) * 4
    a = L.empty_packed(8, K, E, offsets, device="cpu")
    h_gs = torch.full((E,), 0.5)
    p = L.grouped_gemm_swiglu_nvfp4(a, L.empty_packed(2 * K * E, K, device="cpu"), 2 * K, h_gs)
    assert p.gs is h_gs
    L.swiglu_quantize(bf16(8, 2 * K), offsets, E, out=p)
    assert calls[-1][1][GS["nvfp4_swiglu_quantize"]].data_ptr() != h_gs.data_ptr()


# ---------------------------------------------------------------------------------------- attention
def cache(pages=4, heads=2, ps=16, D=64):
    def u8(*s):
        return torch.zeros(s, dtype=torch.uint8)
    gs = torch.ones(1)
    return L.PagedKVCache(u8(pages, heads, ps, D // 2), u8(pages, heads, ps, D // 16), gs,
                          u8(pages, heads, ps, D // 2), u8(pages, heads, ps, D // 16), gs)


def attend_args(counts=(3, 2), D=64):
    offsets = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32)
    return dict(q=bf16(sum(counts), 4, D), seq_lens=torch.full((2,), 9, dtype=torch.int32),
                page_table=torch.zeros(2, 2, dtype=torch.int32), query_offsets=offsets)


def test_query_offsets_without_max_query_are_refused(calls):
    """The kernels compute nothing for a sequence of more queries than max_query, so
    that a forgotten one would return memory as it was found."""
    a = attend_args()
    with pytest.raises(ValueError, match="max_query"):
        cache().attend(**a)
    assert not calls
    cache().attend(**a, max_query=3)
    cache().attend(**a, max_query=1)                 # said so: at most one each (the device reports it)
    cache().attend(a["q"][:2], a["seq_lens"], a["page_table"])
    assert [c[1][4] for c in calls] == [3, 1, 1]
    with pytest.raises(ValueError, match="max_query"):
        cache().attend(a["q"][:2], a["seq_lens"], a["page_table"], max_query=2)


def test_buffers_that_a_kernel_would_leave_are_refused(calls):
    """Workspaces and packed outputs with gaps, and status words that are not one 32-bit
    integer at least: a kernel takes them for dense and would write behind their ends."""
    a = attend_args()
    a["max_query"] = 3
    need = cache().workspace(2, 3, 4).numel()
    gaps = torch.empty(2 * need, dtype=torch.uint8)[::2]
    assert gaps.numel() >= need
    with pytest.raises(ValueError, match="ws"):
        cache().attend(**a, ws=gaps)
    x, w, gs = bf16(4, 64), bf16(64), torch.ones(1)
    kv = bf16(3, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64)
    for bad in (torch.zeros(1, dtype=torch.int8), torch.zeros(1, dtype=torch.int64), torch.zeros(0, dtype=torch.int32)):
        for call in (lambda: cache().attend(**a, dev_status=bad), lambda: cache().append(kv, kv, slots, dev_status=bad),
                     lambda: L.add_rmsnorm_e4m3(x, w, dev_status=bad), lambda: L.add_rmsnorm_nvfp4(x, w, gs, dev_status=bad)):
            with pytest.raises(ValueError, match="dev_status"):
                call()
    for name in ("q", "sf"):
        p = L.empty_packed(4, 64, device="cpu")
        t = getattr(p, name)
        wide = torch.empty(*t.shape[:-1], 2 * t.shape[-1], dtype=torch.uint8)
        for bad in (wide[..., ::2], t.view(torch.int8), t.float(), t[..., :t.shape[-1] // 2]):
            setattr(p, name, bad)
            with pytest.raises(ValueError, match="out"):
                L.add_rmsnorm_nvfp4(x, w, gs, out=p)
    assert not calls
    ok = torch.zeros(2, dtype=torch.int32)
    cache().attend(**a, ws=torch.empty(need, dtype=torch.uint8), dev_status=ok)
    L.add_rmsnorm_nvfp4(x, w, gs, dev_status=ok)
    assert len(calls) == 2


def test_what_a_cache_keeps_per_shape_is_bounded(calls):
    """A server's max_query and batch take many values; a cache that lives as long as
    the server does not keep one entry for each."""
    c, a = cache(), attend_args()
    for n in range(3, 3000):
        c.attend(**a, max_query=n)
    assert len(c._need) <= 256 and len(calls) == 2997


@pytest.mark.parametrize("group,cap", [(1, 8), (4, 8), (8, 8), (12, 16), (16, 16), (32, 32)])
def test_decode_sequences_beside_a_prompt_keep_their_form(group, cap):
    """A prompt in the batch does not draw single-query sequences of long contexts
    into the 128-row form, where a tile costs the same for 4 rows as for 128."""
    for decodes in (1, 32, 63):
        for prompt in (100, 2048, 8192):
            got = choose_forms(decodes + 1, decodes + prompt, prompt, group, 8, 16384)
            assert got[1] and got[0] >= group
            if prompt > 100:
                assert got == (cap, True)


def test_every_sequence_has_a_form():
    r = random.Random(3)
    for _ in range(20000):
        group, batch = r.choice((1, 2, 4, 5, 8, 16, 31, 32, 33, 64, 200)), r.choice((1, 2, 7, 64, 4096))
        max_query = r.choice((1, 2, 4, 9, 33, 2048))
        tokens = r.randrange(1, batch * max_query + 1)
        keys, heads = r.choice((0, 16, 1024, 65536, 1 << 20)), r.choice((1, 8))
        offsets = max_query > 1 or r.random() < 0.5
        if not offsets:
            tokens = batch
        cap, prefill = choose_forms(batch, tokens, max_query, group, heads, keys, offsets)
        most = min(max_query, tokens) * group
        assert cap in (0, 8, 16, 32) and (prefill or most <= cap)            # none is left over
        if cap and prefill:
            assert group <= cap and batch > 1 and offsets
        # one form where only one can have work, or where the other's launches cost more than they save
        if most <= 32:
            assert not prefill
        if group > 32 or not offsets:
            assert (cap == 0) == (group > 32) and prefill == (group > 32)
        if batch == 1 and most > 32:
            assert (cap, prefill) == (0, True)


def test_prompts_alone_and_few_rows_alone():
    assert choose_forms(64, 64, 1, 8, 4, 262144, False) == (8, False)        # decode
    assert choose_forms(64, 64, 1, 4, 8, 16384, False) == (8, False)
    assert choose_forms(32, 100, 4, 8, 4, 8192) == (32, False)               # verification
    assert choose_forms(32, 100, 2, 8, 4, 8192) == (16, False)
    assert choose_forms(1, 4096, 4096, 4, 8, 4096) == (0, True)              # a prompt
    assert choose_forms(2, 1024, 512, 4, 8, 512) == (0, True)                # short ones: no second pair of launches
    assert choose_forms(64, 256, 16, 8, 4, 16384) == (32, True)              # verification with a loose max_query
    assert choose_forms(64, 64, 16, 8, 4, 16384) == (8, True)
    assert choose_forms(1, 4, 64, 8, 4, 262144) == (32, False)               # fewer tokens than max_query says


def test_workspace_size_of_refused_shapes():
    """0 for what the attention refuses, also where the rows would pass 64 bits."""
    from nvfp4_w4a4_quantized_04_b200 import build, nvfp4_paged_attention_workspace_size as size
    build.build()
    assert size(1, 1 << 62, 8, 4, 128) == 0 and size(4096, 1 << 61, 64, 1, 256) == 0
    assert size(1, 0x7FFFFFFF // 8 + 1, 8, 4, 128) == 0
    assert size(1, 1, 8192, 4, 128) == 0
    assert size(1, 0x7FFFFFFF // 4096, 4096, 4096, 64) > 0


def test_workspace_sizes_are_those_of_the_caches_device(calls, monkeypatch):
    """The size depends on the SM count of the current device, so the cache's device is
    current while it is asked for."""
    inside, sizes = [], []

    @contextlib.contextmanager
    def on(t):
        inside.append(t)
        yield
        inside.pop()
    monkeypatch.setattr(L, "_on", on)
    monkeypatch.setattr(L, "_cuda", lambda t: True, raising=False)
    monkeypatch.setattr(L, "nvfp4_paged_attention_workspace_size", lambda *a: sizes.append(len(inside)) or 512)
    c = cache()
    c.workspace(2, 3, 4)
    c.attend(**attend_args(), max_query=3)
    assert sizes == [1, 1]


def test_in_place_outputs_of_another_stride_are_refused():
    """r may go where x or the residual is, and the rotated queries where the queries are,
    row by row: with another stride one row's output lies in a row still to be read."""
    import nvfp4_w4a4_quantized_04_b200 as nv
    from nvfp4_w4a4_quantized_04_b200 import build
    from tests.test_kv_paged import APPEND, APPEND_OK, F, NORM, NORM_OK
    build.build()
    lib = nv.load_library()
    far = 1 << 24                                     # never dereferenced: the checks fail first

    def norm(**change):
        a = dict(NORM_OK, x=F, res=2 * F, w=3 * F, ro=far, q=5 * F, sf=6 * F, scale=7 * F, **{})
        a.update(change)
        return lib.nvfp4_add_rmsnorm_quantize(*[a[n] for n in NORM])

    def append(**change):
        a = dict(APPEND_OK, q=F, qo=F)
        a.update(change)
        return lib.nvfp4_kv_append(*[a[n] for n in APPEND])
    assert norm(ro=F, ld_ro=264) == nv.ERR_INVALID_ARG
    assert norm(ro=F, ld_x=512) == nv.ERR_INVALID_ARG
    assert norm(ro=2 * F, ld_ro=264) == nv.ERR_INVALID_ARG
    assert append(ld_qo=2048) == nv.ERR_INVALID_ARG
    assert append(ld_q=2048) == nv.ERR_INVALID_ARG
