"""The serving operators at the ends of their ranges: values near the largest
and smallest that bf16 holds, scores far apart, bad global scales, buffers used
again, and batches that both forms of the attention share."""
import gc
import weakref

import numpy as np
import pytest

import oracle
from tests._forms import choose_forms
from tests._util import bf16_dev, to_dev, to_np
from tests.test_gpu_serving import FEW_ROWS, Case, bits_of, bf16_of, layer, nvmod, random_bf16, same, status_word, values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_w4a4_quantized_04_b200 import build
    build.build()


def bf16_full(x):
    """float64 -> the nearest bf16 (ties to even) as float64, subnormals and overflow included."""
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    r = np.rint(x / step) * step
    return np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, x), r)


# ---------------------------------------------------------------------------------------- norm
# r ~ 2^rows, w ~ 2^weights: the products r w leave fp32's range at either end while y is ordinary,
# the root leaves it, or y itself is a subnormal
@pytest.mark.parametrize("rows,weights,eps", [(126, 2, 1e-6), (120, 30, 1e-6), (100, 40, 1e-6), (126, 100, 0.0),
                                              (-60, -80, 0.0), (-120, -20, 0.0), (-130, 0, 0.0), (-128, -126, 0.0),
                                              (0, -127, 1e-6), (3, -131, 1e-6), (-80, 90, 1e-6), (-133, 30, 1e-30)])
@pytest.mark.parametrize("K", [64, 5120, 20480])
def test_norm_rounds_correctly_over_the_whole_range(rows, weights, eps, K):
    """y is within 2^-40 of the exact value before its one rounding, so it is the
    64-bit result's nearest bf16 unless that lies within 2^-40 of a border (about
    2^-31 per element of a bf16 with 8 bits).  Below 2^-100 max(1, |w|) the
    definition allows 2^-132 max(1, |w|) besides the rounding."""
    L = layer()
    rng = np.random.default_rng(1000 + rows + 7 * weights + K)
    T = 5
    x = bits_of(bf16_full(rng.uniform(1, 1.999, (T, K)) * rng.choice([-1, 1], (T, K)) * 2.0 ** rows))
    x[1, ::3] = bits_of(bf16_full(values(x[1, ::3]) * 2.0 ** -9))     # elements far below their row's largest
    x[2] = 0
    w = bits_of(bf16_full(rng.uniform(1, 1.999, K) * 2.0 ** weights))
    r = values(x)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        y64 = r * values(w) / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    y = bf16_full(y64)
    keep = [0, 1, 3, 4] + ([2] if eps else [])                        # 0 / 0 has no value
    yd = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    st = status_word()
    q, scale, _, _ = L.add_rmsnorm_e4m3(bf16_dev(x)[keep], bf16_dev(w), eps=eps, y=yd[:len(keep)], dev_status=st)
    got = to_np(yd)[:len(keep)]
    assert np.isfinite(y[keep]).all() and st.item() == 0
    low = np.abs(y64[keep]) < 2.0 ** -100 * np.maximum(1.0, np.abs(values(w)))
    same(np.where(low, 0.0, values(got)), np.where(low, 0.0, y[keep]))
    half = np.ldexp(0.5, np.maximum(np.frexp(y64[keep])[1] - 8, -133))
    assert (np.abs(values(got) - y64[keep]) <= half + 2.0 ** -132 * np.maximum(1.0, np.abs(values(w))))[low].all()
    amax = np.abs(values(got)).max(1).astype(np.float32)
    want = np.where(amax == 0, np.float32(1), np.maximum(amax / np.float32(448), np.float32(2.0 ** -126)))
    same(to_np(scale), want)


def test_norm_reports_what_overflows():
    """A y beyond bf16's range is inf and reported; its neighbours in the row are not disturbed."""
    L, nv = layer(), nvmod()
    x = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    w[3] = 3.0e38
    x[1, 3] = 8.0
    y, st = torch.empty_like(x), status_word()
    L.add_rmsnorm_e4m3(x[:1], w, y=y[:1], dev_status=st)
    assert st.item() == 0 and torch.isfinite(y[0]).all()
    L.add_rmsnorm_e4m3(x, w, y=y, dev_status=st)
    assert st.item() == nv.ERR_NONFINITE and torch.isinf(y[1, 3]) and torch.isfinite(y[1, :3]).all()
    assert torch.isfinite(y[0]).all()


# ---------------------------------------------------------------------------------------- attention
def test_a_captured_workspace_outlives_its_last_reference():
    """A graph points into the workspace; when the caller lets go of it, it must not
    go back to the allocator, whose cache the next capture empties."""
    c = Case(10, 256, 4, 8, 64, [3000, 500, 0], None, True)
    want = c.run()
    ws, out = c.cache.workspace(3, 1, 32), torch.zeros_like(c.q)
    c.run(ws=ws, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ws=ws, out=out)
    held = weakref.ref(ws)
    del ws
    gc.collect()
    assert held() is not None
    y = torch.zeros(1, device="cuda")
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        y.add_(1)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def one_key_case(D, queries, at, seed=4, hkv=2, group=4, n=700):
    """A case whose queries look at one element only, in which token `at` has the
    largest key of every head (72 times the head's scale; the others at most 20)."""
    c = Case(seed, D, hkv, group, 64, [n], queries, True)
    page, row = c.pages[0][at // 64], at % 64
    c.t["k_sf"][c.t["k_sf"] == 0] = 0x38
    c.t["k_sf"][page, :, row, 0] = 0x54                        # 12
    c.t["k_q"][page, :, row, 0] = 0x77                         # 6, 6
    c.t["k_q"][:, :, :, 0] &= 0x77                             # the element itself is not negative
    return c


def one_hot_queries(c, value):
    q = torch.zeros_like(c.q)
    q[..., 0] = value
    return q


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("queries", [None, [4], [40]])
@pytest.mark.parametrize("power", [12, 24, 27, 30, 60, 110])
def test_attention_scores_far_apart_give_the_largest_keys_value(D, queries, power):
    """Scores up to 2^118, beyond what fp32 resolves to units: the weights of all
    keys but one vanish, and the output is that key's value.  Its weight is rounded
    to f16 (2^-11) and the output to fp32."""
    L = layer()
    for at in (0, 333, 660):
        c = one_key_case(D, queries, at)
        q = one_hot_queries(c, 2.0 ** power)
        want, lse, mag = c.reference(q=q)
        ls = torch.zeros(c.q.shape[:2], device="cuda")
        out = c.run(q=q, out_dtype=L.OUT_F32, lse=ls)
        assert torch.isfinite(out).all()
        assert ((out.double() - want).abs() <= mag * (2.0 ** -11 + 2.0 ** -22)).all()
        assert ((ls - lse).abs() <= 2.0 ** -21 * lse.abs()).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("queries", [None, [4], [40]])
@pytest.mark.parametrize("power", [60, 110, 122])
def test_attention_scores_all_far_below_zero(D, queries, power):
    """All of a row's scores at -2^57 to -2^122: the least negative one wins, and the
    row is neither zeros nor without a sum.  Tolerances as above."""
    L = layer()
    for at in (0, 333, 660):
        c = one_key_case(D, queries, at)
        page, row = c.pages[0][at // 64], at % 64
        c.t["k_q"][:, :, :, 0] = 0x22                              # 1, 1
        c.t["k_sf"][:, :, :, 0] = 0x38                             # 1
        c.t["k_sf"][page, :, row, 0] = 0x30                        # 0.5
        q = one_hot_queries(c, -(2.0 ** power))
        want, lse, mag = c.reference(q=q)
        ls = torch.zeros(c.q.shape[:2], device="cuda")
        out = c.run(q=q, out_dtype=L.OUT_F32, lse=ls)
        assert ((out.double() - want).abs() <= mag * (2.0 ** -11 + 2.0 ** -22)).all()
        assert ((ls - lse).abs() <= 2.0 ** -21 * lse.abs()).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("queries", [None, [4, 3], [40, 1]])
def test_attention_reports_bad_global_scales(D, queries):
    """A scale of zero, below it, NaN or inf is reported, and the outputs are NaN
    rather than a plausible average of the values."""
    L, nv = layer(), nvmod()
    c = Case(12, D, 2, 4, 64, [200, 70], queries, True)
    good = c.run()
    for bad in (0.0, -0.5, float("nan"), float("inf")):
        for which in ("k_gs", "v_gs"):
            keep = getattr(c.cache, which)
            setattr(c.cache, which, torch.tensor([bad], device="cuda"))
            st = status_word()
            out = c.run(out_dtype=L.OUT_F32, dev_status=st)
            setattr(c.cache, which, keep)
            assert st.item() == nv.ERR_INVALID_ARG and torch.isnan(out).all()
    st = status_word()
    assert torch.equal(c.run(dev_status=st), good) and st.item() == 0
    # one so small that the scaled score is a subnormal is still good
    c.cache.k_gs = torch.tensor([1e-44], device="cuda")
    out = c.run(out_dtype=L.OUT_F32, dev_status=st)
    assert st.item() == 0 and torch.isfinite(out).all()


# ---------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("power,gain", [(-133, 1.0), (-128, 1.0), (-126, 1.0), (-110, 2.0 ** -20), (0, 2.0 ** -126),
                                        (120, 1.0), (127, 1.0), (126, 3.0), (100, 2.0 ** 30), (0, 1.0)])
def test_append_rounds_correctly_over_the_whole_range(power, gain, pairs):
    """Rotated queries and keys are the 64-bit result's nearest bf16, for values and
    tables whose products are subnormal in fp32 or leave its range (the products are
    exact in 64 bits, their sum is off by 2^-53, so that another bf16 would need a
    border within that)."""
    L = layer()
    rng = np.random.default_rng(2000 + power + int(pairs))
    T, heads, D, rot = 1000, 2, 64, 64
    with np.errstate(over="ignore"):
        x = bits_of(bf16_full(rng.standard_normal((T, heads, D)) * 2.0 ** power))
    x[np.isinf(values(x))] = 0x7F7F
    x[:40] = 0
    x[40:80, :, ::2] = 0
    pos = rng.integers(0, 5000, T).astype(np.int64)
    pos[:100] = 0
    table = L.rope_table(5000, rot) * gain
    tab = table.double().cpu().numpy()
    c, s = tab[pos, None, :rot // 2], tab[pos, None, rot // 2:]
    v, want = values(x), np.empty((T, heads, D))
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    want[..., a] = v[..., a] * c - v[..., b] * s
    want[..., b] = v[..., b] * c + v[..., a] * s
    with np.errstate(over="ignore"):
        want = bf16_full(want)
    gs = np.float32(min(max(2.0 ** power * gain / 300, 2.0 ** -100), 2.0 ** 100))
    g = torch.tensor([gs], device="cuda")
    cache = L.PagedKVCache.empty(63, 16, heads, D, g, g)
    st = status_word()
    xd = bf16_dev(x)
    got = cache.append(xd, xd, torch.arange(T, device="cuda"), q=xd, positions=to_dev(pos), rope=table, interleaved=pairs,
                       dev_status=st)
    same(values(to_np(got)), want)
    finite = np.isfinite(want)
    assert st.item() == (0 if finite.all() else nvmod().ERR_NONFINITE)
    blocks = finite.reshape(T, heads, D // 16, 16).all(-1)
    q_, sf_, _ = oracle.quantize(bits_of(np.where(finite, want, 0.0)).reshape(T * heads, D), global_scale=np.array([gs], np.float32))[:3]
    kq = to_np(cache.k_q.transpose(1, 2).reshape(-1, heads, D // 2)[:T].contiguous()).reshape(T, heads, D // 16, 8)
    ks = to_np(cache.k_sf.transpose(1, 2).reshape(-1, heads, D // 16)[:T].contiguous())
    same(kq, np.where(blocks[..., None], q_.reshape(T, heads, D // 16, 8), np.uint8(0)))
    same(ks, np.where(blocks, sf_.reshape(T, heads, D // 16), np.uint8(0)))


# ---------------------------------------------------------------------------------------- both forms in one call
MIXED = [
    # D, hkv, group, page, decode lengths (one query each), others (length, queries)
    (64, 2, 4, 16, [0, 1, 33, 4000, 17, 2500, 64, 700] * 5, [(900, 50)]),
    (128, 2, 4, 64, [0, 1, 33, 5000, 17, 2500, 64, 700] * 5, [(900, 50)]),
    (256, 2, 4, 32, [0, 1, 33, 3000, 17, 2500, 64, 700] * 5, [(900, 50)]),
    (128, 1, 8, 64, [6000, 0, 129, 1] * 10, [(3000, 300), (70, 70), (0, 40)]),
    (256, 1, 8, 64, [6000, 0, 129, 1] * 10, [(3000, 300), (20, 30)]),
    (64, 1, 16, 32, [6000, 31, 0, 1] * 12, [(2000, 129), (40, 3)]),
    (128, 1, 32, 48, [6000, 31, 0, 1] * 10, [(2000, 65), (40, 2)]),
    (256, 1, 12, 16, [3000, 31, 0, 2000] * 12, [(2000, 65), (40, 2), (1500, 3)]),
    (128, 2, 2, 16, [4000, 31, 0, 1] * 10, [(2000, 17), (40, 16), (900, 4), (900, 5)]),
]


@pytest.mark.parametrize("D,hkv,group,ps,decodes,others", MIXED)
@pytest.mark.parametrize("causal", [True, False])
def test_attention_batches_that_both_forms_share(D, hkv, group, ps, decodes, others, causal):
    """Long and short single-query sequences beside prompts: the rule sends work to
    both forms, and every row and sum is there."""
    half = len(decodes) // 2                          # the prompts in the middle and at the end
    lens = decodes[:half] + [n for n, _ in others[:1]] + decodes[half:] + [n for n, _ in others[1:]]
    counts = [1] * half + [q for _, q in others[:1]] + [1] * (len(decodes) - half) + [q for _, q in others[1:]]
    c = Case(sum(lens) + D, D, hkv, group, ps, lens, counts, causal)
    cap, prefill = choose_forms(len(lens), sum(counts), c.max_query, group, hkv, c.table.shape[1] * ps,
                                sms=torch.cuda.get_device_properties(0).multi_processor_count)
    assert prefill and any(n and q * group <= cap for n, q in zip(lens, counts)) and \
        any(n and q * group > cap for n, q in zip(lens, counts))
    want, lse, mag = c.reference()
    for dt, td in ((layer().OUT_F32, torch.float32), (layer().OUT_BF16, torch.bfloat16)):
        ls = torch.full(lse.shape, 5.0, dtype=torch.float32, device="cuda")
        out = torch.full(c.q.shape, float("nan"), dtype=td, device="cuda")
        st = status_word()
        c.run(out=out, out_dtype=dt, lse=ls, dev_status=st)
        assert st.item() == 0 and not torch.isnan(out).any()
        err = (out.double() - want).abs() - c.tolerance(want, mag, td)
        assert err.max().item() <= 0, err.max().item()
        empty = torch.isinf(lse)
        assert torch.equal(empty, torch.isinf(ls)) and (out[empty] == 0).all()
        assert ((ls - lse)[~empty].abs() <= 2e-4 + 2.0 ** -21 * lse[~empty].abs()).all()
        assert torch.equal(c.run(out_dtype=dt), out)


@pytest.mark.parametrize("D,hkv,group,lens,queries", [(64, 4, 4, [700], [700]), (128, 8, 4, [1500, 300], [1500, 80]),
                                                      (256, 2, 8, [1000, 90, 400], [300, 90, 40])])
def test_attention_prefill_waits_give_up_and_report(D, hkv, group, lens, queries):
    """A wait that runs out ends the kernel with a status, outside the rows' neighbours
    and with a context that stays usable: the next call is right again."""
    L, nv = layer(), nvmod()
    c = Case(30 + D, D, hkv, group, 64, lens, queries, True)
    T, H = c.q.shape[:2]
    want = c.run(out_dtype=L.OUT_F32)
    wide = torch.full((T + 8, H, D), 3.0, device="cuda")
    st = status_word()
    torch.cuda.synchronize()
    nv.nvfp4_gemm_set_wait_budget(1)
    try:
        c.run(out=wide[4:T + 4], out_dtype=L.OUT_F32, dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == nv.ERR_TIMEOUT
    finally:
        nv.nvfp4_gemm_set_wait_budget(0)
    assert (wide[:4] == 3).all() and (wide[T + 4:] == 3).all()
    st.zero_()
    assert torch.equal(c.run(out_dtype=L.OUT_F32, dev_status=st), want) and st.item() == 0


# ---------------------------------------------------------------------------------------- exact scores
def exact_scores(c, seed):
    """Queries of +-1, +-2 and keys of +-0.5, +-1, +-2: every partial sum of a score is
    a multiple of 0.5 below 2^11, exact in fp32.  Unused rows keep their garbage."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    used = c.t["k_sf"][..., :1] != 0xFF
    table = torch.tensor([1, 2, 4, 9, 10, 12], dtype=torch.uint8, device="cuda")
    nib = table[torch.randint(0, 6, (*c.t["k_q"].shape, 2), generator=g, device="cuda")]
    c.t["k_q"].copy_(torch.where(used, nib[..., 0] | nib[..., 1] << 4, c.t["k_q"]))
    c.t["k_sf"].copy_(torch.where(used, torch.full_like(c.t["k_sf"], 0x38), c.t["k_sf"]))
    c.kgs.fill_(1.0)
    sizes = torch.tensor([1.0, 2.0, -1.0, -2.0], device="cuda").to(torch.bfloat16)
    c.q.copy_(sizes[torch.randint(0, 4, c.q.shape, generator=g, device="cuda")])


PEAKED = [(D, hkv, group, ps, lens, queries, True) for D, hkv, group, ps, lens, queries in FEW_ROWS] + [
    (64, 2, 4, 32, [900, 333], None, True), (128, 2, 4, 32, [900, 333], None, True), (256, 2, 4, 32, [900, 333], None, True),
    (128, 8, 4, 64, [2048], [2048], True), (64, 8, 4, 32, [2048], [2048], True), (256, 4, 4, 64, [1500], [1500], True),
    (128, 2, 8, 128, [1500, 900, 1800], [700, 900, 1], True), (256, 1, 2, 64, [9000, 200], [130, 65], False),
    (64, 1, 16, 16, [130, 2000, 17], [2, 3, 17], False)]


@pytest.mark.parametrize("D,hkv,group,ps,lens,queries,causal", PEAKED)
@pytest.mark.parametrize("scale", [0.02, 0.3, 2.0])
def test_attention_of_exact_scores(D, hkv, group, ps, lens, queries, causal, scale):
    """From even weights to one key that takes all, with scores that carry no error into
    the softmax, so that a wrong maximum, rescale or join shows.  The tolerance: the
    scaling's roundings (factor, product, difference: 2^-21 of the largest score), the
    weights' f16 rounding (2^-11, or 2^-25 absolute against a maximum of 1 at least),
    exp2 (2^-22) and N/16 + 64 additions; the sum's logarithm has all but the f16 part."""
    L = layer()
    c = Case(sum(lens) + D, D, hkv, group, ps, lens, queries, causal)
    exact_scores(c, 77 + D)
    plain = c.q
    stretch = scale * D ** 0.5                                     # the reference scales by D^-0.5
    want, lse, mag = c.reference(q=plain.double() * stretch)
    ls = torch.full(lse.shape, 5.0, dtype=torch.float32, device="cuda")
    st = status_word()
    out = c.run(out_dtype=L.OUT_F32, softmax_scale=scale, lse=ls, dev_status=st)
    assert st.item() == 0 and not torch.isnan(out).any()
    n = max(lens)
    top = scale * 4 * D                                            # no score is larger
    top = min(top, scale * 2.1 * D ** 0.5 * 7)                     # nor, for these values, beyond 7 deviations
    ds = 2.0 ** -21 * top + 2.0 ** -22 + (n / 16 + 64) * 2.0 ** -24
    err = (out.double() - want).abs() - (mag * (2.0 ** -11 + 2 * ds) + n * 2.0 ** -25 * c.vmax + out.abs() * 2.0 ** -24)
    assert err.max().item() <= 0, err.max().item()
    empty = torch.isinf(lse)
    assert torch.equal(empty, torch.isinf(ls)) and (out[empty] == 0).all()
    assert ((ls - lse)[~empty].abs() <= ds + 2.0 ** -22 * lse[~empty].abs() + 2.0 ** -23).all()


# ---------------------------------------------------------------------------------------- into the GEMM
@pytest.mark.parametrize("rows,K,N", [(1, 256, 256), (70, 512, 256), (128, 256, 512), (300, 1024, 512)])
def test_norm_feeds_the_projection(rows, K, N):
    """The norm's output goes into the W4A4 GEMM as it is: the same result as that of the
    quantized y, whatever the buffers' padding rows held."""
    L = layer()
    torch.manual_seed(rows)
    x, r = (torch.randn(rows, K, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = (1 + 0.1 * torch.randn(K, device="cuda")).to(torch.bfloat16)
    wp = L.quantize((0.05 * torch.randn(N, K, device="cuda")).to(torch.bfloat16))
    gs = torch.tensor([6.0 / 2688], device="cuda")
    y = torch.empty_like(x)
    packed = L.empty_packed(rows, K)
    packed.q.fill_(0x7F)
    packed.sf.fill_(0x7F)                                          # NaN
    st = status_word()
    packed, _, _ = L.add_rmsnorm_nvfp4(x, w, gs, residual=r, out=packed, y=y, dev_status=st)
    got = L.grouped_gemm(packed, wp, N, L.OUT_F32, dev_status=st)
    want = L.grouped_gemm(L.quantize(y, global_scale=gs), wp, N, L.OUT_F32, dev_status=st)
    assert st.item() == 0 and torch.isfinite(got).all() and torch.equal(got, want)
    # the buffers again, with scales of their own: the calibrated one is as it was
    L.quantize(x, out=packed)
    assert gs.item() == np.float32(6.0 / 2688) and packed.gs is not gs
    assert torch.equal(L.grouped_gemm(packed, wp, N, L.OUT_F32), L.grouped_gemm(L.quantize(x), wp, N, L.OUT_F32))


# ---------------------------------------------------------------------------------------- captured
@pytest.mark.parametrize("D,hkv,group,lens,counts", [
    (128, 8, 4, [1500, 0, 900], [1500, 0, 300]),                                       # the prefill form
    (128, 2, 4, [4000, 33, 1, 2500] * 10 + [900], [1] * 40 + [60]),                    # both forms
    (256, 2, 4, [3000, 33, 1, 2500] * 10 + [900], [1] * 40 + [60]),
    (64, 4, 8, [6000, 33, 1, 700] * 10 + [900], [1] * 40 + [60])])
def test_attention_in_graphs_of_either_form_takes_new_lengths(D, hkv, group, lens, counts):
    """Captured once and replayed with other lengths, offsets and queries inside the
    captured sizes, on a padded batch whose last rows no sequence has, with pages that
    two sequences share: the same bits as a plain call."""
    c = Case(40 + D, D, hkv, group, 64, lens, counts, True)
    pad, T = 9, sum(counts)
    c.table[1] = c.table[0]                                        # a shared prefix
    q = torch.randn(T + pad, *c.q.shape[1:], device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = c.cache.workspace(len(lens), c.max_query, q.shape[1])
    st = status_word()

    def run(out, lse, ws):
        c.cache.attend(q, c.seq_lens, c.table, query_offsets=c.offsets, max_query=c.max_query, out=out, lse=lse, ws=ws,
                       dev_status=st)
    run(out, lse, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, lse, ws)
    for turn in range(3):
        q.copy_(torch.randn(q.shape, device="cuda"))
        if turn:
            less = [n if i % 3 else max(0, n - 17 * turn) for i, n in enumerate(lens)]
            less[1] = less[0]
            fewer = [max(0, n - turn) if i % 4 == 0 else n for i, n in enumerate(counts)]
            c.seq_lens.copy_(torch.tensor(less, dtype=torch.int32))
            c.offsets.copy_(torch.tensor([0] + list(np.cumsum(fewer)), dtype=torch.int32))
        out.fill_(3.0)
        lse.fill_(4.0)
        graph.replay()
        want, wl = torch.full_like(out, 3.0), torch.full_like(lse, 4.0)
        run(want, wl, None)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl) and st.item() == 0
        last = int(c.offsets[-1])
        assert (out[last:] == 3).all() and (lse[last:] == 4).all() and last < T + pad
        assert not torch.isnan(out).any()
