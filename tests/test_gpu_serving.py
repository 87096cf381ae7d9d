"""The serving operators around the paged NVFP4 cache on the GPU: residual +
RMS norm with a quantized output, rotated append, attention, against plain
64-bit forms and the oracle's encoder."""
import numpy as np
import pytest

import oracle
from tests._util import bf16_dev, to_dev, to_np, untile

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_w4a4_quantized_04_b200 import build
    build.build()


def layer():
    from nvfp4_w4a4_quantized_04_b200 import layer as L
    return L


def nvmod():
    import nvfp4_w4a4_quantized_04_b200 as nv
    return nv


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def bf16_of(x):
    """float64 -> the nearest bf16 (ties to even) as float64."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def bits_of(x):
    """bf16 values held in float64 -> their bits."""
    return (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def random_bf16(rng, *shape, scale=1.0):
    x = rng.standard_normal(shape) * scale
    x = np.where(rng.random(shape) < 0.002, 20 * x, x)
    return bits_of(bf16_of(x))


def same(a, b):
    """Arrays equal, with the first differences in the message rather than the arrays."""
    assert a.shape == b.shape and a.dtype == b.dtype, (a.shape, b.shape, a.dtype, b.dtype)
    at = np.argwhere(a != b)
    assert not len(at), (len(at), a.size, at[:4].tolist(), [(a[tuple(i)], b[tuple(i)]) for i in at[:4]])
    return True


# ---------------------------------------------------------------------------------------- norm
NORM_SHAPES = [(1, 16), (1, 64), (3, 64), (5, 192), (7, 1024), (64, 5120), (130, 2176), (2, 16384), (3, 16448), (2, 40000),
               (1, 65536)]


def norm_reference(x, res, w, eps):
    r = values(x)
    if res is not None:
        r = bf16_of(r + values(res))
    y = bf16_of(r * values(w) / np.sqrt((r * r).mean(1, keepdims=True) + eps))
    return r, y


@pytest.mark.parametrize("rows,K", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_is_correctly_rounded_in_every_format(rows, K, residual):
    """r and y bit for bit, and the codes and scales that the oracle (NVFP4) and
    the definition (E4M3) give for that y.  y is the correctly rounded value: its
    error before rounding is about 2^-40, so a different bf16 would need the exact
    value within 2^-40 of a rounding border (about 2^-31 per element)."""
    L, nv = layer(), nvmod()
    rng = np.random.default_rng(rows * 1000003 + K)
    x, w = random_bf16(rng, rows, K), random_bf16(rng, K)
    res = random_bf16(rng, rows, K, scale=3.0) if residual else None
    r, y = norm_reference(x, res, w, 1e-6)
    xd, wd, rd = bf16_dev(x), bf16_dev(w), bf16_dev(res) if residual else None
    gs = np.float32(max(np.abs(y).max(), 1e-3) / 2688 * 0.7)
    st = status_word()
    for layout in ((L.SF_ROWMAJOR, L.SF_MMA_TILED) if K % 64 == 0 else (L.SF_ROWMAJOR,)):
        yd = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
        p, ro, _ = L.add_rmsnorm_nvfp4(xd, wd, torch.tensor([gs], device="cuda"), residual=rd, layout=layout, y=yd,
                                       dev_status=st)
        assert same(to_np(ro), bits_of(r)) if residual else ro is xd
        same(values(to_np(yd)), y)
        q, sf, _ = oracle.quantize(to_np(yd), global_scale=np.array([gs], np.float32))[:3]
        same(to_np(p.q)[:rows], q)
        got = to_np(p.sf)
        got = untile(got, (rows + 127) // 128 * 128, K // 16)[:rows] if layout == L.SF_MMA_TILED else \
            got.reshape(rows, K // 16)
        same(got, sf)
    q, scale, ro, _ = L.add_rmsnorm_e4m3(xd, wd, residual=rd, dev_status=st)
    amax = np.abs(y).max(1).astype(np.float32)
    want = np.where(amax == 0, np.float32(1), amax / np.float32(448))
    same(to_np(scale), want)
    prod = y.astype(np.float32) * (np.float32(1) / want)[:, None]
    same(to_np(q), oracle.e4m3_encode_array(prod.reshape(-1)).reshape(rows, K))
    only = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_add_rmsnorm_quantize(xd, K, rd, K if residual else 0, rows, K, wd, 1e-6, None, 0, only, nv.NORM_BF16, None,
                                  None, None, dev_status=st)
    same(values(to_np(only)), y)
    assert st.item() == 0


def test_norm_strides_in_place_and_misaligned_rows():
    L = layer()
    rng = np.random.default_rng(5)
    rows, K = 9, 320
    x, res, w = random_bf16(rng, rows, K), random_bf16(rng, rows, K), random_bf16(rng, K)
    r, y = norm_reference(x, res, w, 1e-5)
    amax = np.abs(y).max(1).astype(np.float32)
    for pad, at in ((8, 0), (16, 8), (24, 8)):     # 16-byte aligned rows that are not 32-byte aligned among them
        wide = torch.full((rows, K + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        wide[:, at:at + K] = bf16_dev(x)
        other = torch.full((rows, K + 8), 9.0, dtype=torch.bfloat16, device="cuda")
        other[:, :K] = bf16_dev(res)
        q, scale, ro, _ = L.add_rmsnorm_e4m3(wide[:, at:at + K], bf16_dev(w), residual=other[:, :K], eps=1e-5,
                                             residual_out=other[:, :K])
        same(to_np(other[:, :K].contiguous()), bits_of(r))
        assert (other[:, K:] == 9.0).all() and (wide[:, K + at:] == 7.0).all()
        same(to_np(scale), amax / np.float32(448))
    # x itself receives r
    xd = bf16_dev(x)
    L.add_rmsnorm_e4m3(xd, bf16_dev(w), residual=bf16_dev(res), residual_out=xd)
    same(to_np(xd), bits_of(r))


def test_norm_extreme_rows():
    """Zero rows, rows beyond fp32's square range, subnormal rows; and NaN or inf
    is reported without touching the other rows."""
    L = layer()
    K = 256
    rng = np.random.default_rng(11)
    x = random_bf16(rng, 6, K)
    x[1] = 0
    x[2] = bits_of(bf16_of(values(x[2]) * 2.0 ** 100))
    x[3] = bits_of(bf16_of(values(x[3]) * 2.0 ** -100))
    w = random_bf16(rng, K)
    eps = 1e-30
    _, y = norm_reference(x, None, w, eps)
    yd = torch.empty(6, K, dtype=torch.bfloat16, device="cuda")
    st = status_word()
    q, scale, _, _ = L.add_rmsnorm_e4m3(bf16_dev(x), bf16_dev(w), eps=eps, y=yd, dev_status=st)
    assert st.item() == 0
    same(values(to_np(yd)), y)
    assert scale[1].item() == 1.0 and (q[1] & 0x7F == 0).all()
    good = to_np(q).copy()
    x[4, 17] = 0x7F80
    x[0, 3] = 0x7FC0
    q, _, _, _ = L.add_rmsnorm_e4m3(bf16_dev(x), bf16_dev(w), eps=eps, dev_status=st)
    assert st.item() == nvmod().ERR_NONFINITE
    same(to_np(q)[[1, 2, 3, 5]], good[[1, 2, 3, 5]])
    st = status_word()
    L.add_rmsnorm_nvfp4(bf16_dev(x[1:2]), bf16_dev(w), torch.zeros(1, device="cuda"), dev_status=st)
    assert st.item() == nvmod().ERR_INVALID_ARG


# ---------------------------------------------------------------------------------------- append
def turned(x, pos, table, rot, pairs):
    """[tokens, heads, D] float64 rotated in 64 bits, rounded once."""
    half = rot // 2
    c, s = table[pos, None, :half], table[pos, None, half:]
    out = x.copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, half), slice(half, rot))
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return bf16_of(out)


@pytest.mark.parametrize("D,heads,hq,rot,pairs,ps,tokens", [
    (64, 2, 4, 32, False, 16, 1), (64, 1, 0, 64, True, 16, 33), (128, 8, 32, 128, False, 64, 70),
    (128, 2, 6, 64, True, 48, 17), (256, 4, 32, 64, False, 64, 129), (256, 1, 1, 256, False, 128, 5),
    (256, 3, 3, 0, False, 32, 40), (96, 5, 5, 96, True, 16, 300), (512, 2, 2, 128, False, 16, 3)])
def test_append_matches_64_bit_rotation_and_the_oracle_encoder(D, heads, hq, rot, pairs, ps, tokens):
    L = layer()
    rng = np.random.default_rng(D * 7 + tokens)
    pages = (tokens + ps - 1) // ps + 2
    k, v = random_bf16(rng, tokens, heads, D), random_bf16(rng, tokens, heads, D)
    kg, vg = np.float32(0.0043), np.float32(0.0031)
    c = L.PagedKVCache.empty(pages, ps, heads, D, torch.tensor([kg], device="cuda"), torch.tensor([vg], device="cuda"))
    for t in (c.k_q, c.k_sf, c.v_q, c.v_sf):
        t.fill_(0xA5)
    slots = rng.permutation(pages * ps)[:tokens].astype(np.int64)
    if tokens > 4:
        slots[3] = -1
    table = L.rope_table(5000, rot, 1e4) if rot else None
    pos = rng.integers(0, 5000, tokens).astype(np.int64)
    # slices of a wider projection output: token strides larger than heads * D, 16- but not 32-byte aligned
    wide = torch.zeros(tokens, (hq + 2 * heads) * D + 8, dtype=torch.bfloat16, device="cuda")
    qd = None
    if hq:
        q = random_bf16(rng, tokens, hq, D)
        wide[:, 8:8 + hq * D] = bf16_dev(q).view(tokens, -1)
        qd = wide[:, 8:8 + hq * D].unflatten(1, (hq, D))
    wide[:, 8 + hq * D:8 + (hq + heads) * D] = bf16_dev(k).view(tokens, -1)
    wide[:, 8 + (hq + heads) * D:] = bf16_dev(v).view(tokens, -1)
    kd = wide[:, 8 + hq * D:8 + (hq + heads) * D].unflatten(1, (heads, D))
    vd = wide[:, 8 + (hq + heads) * D:].unflatten(1, (heads, D))
    st = status_word()
    out = c.append(kd, vd, to_dev(slots), q=qd, positions=to_dev(pos) if rot else None, rope=table, interleaved=pairs,
                   dev_status=st)
    assert st.item() == 0
    tab = table.double().cpu().numpy() if rot else None
    turn = (lambda x: turned(values(x), pos, tab, rot, pairs)) if rot else (lambda x: values(x))
    if hq:
        same(values(to_np(out)), turn(q))
        again = c.append(kd, vd, to_dev(slots), q=qd, q_out=qd, positions=to_dev(pos) if rot else None, rope=table,
                        interleaved=pairs)
        assert again is qd and same(to_np(qd.contiguous()), to_np(out))
    else:
        assert out is None
    for bits, gs, codes, scales in ((bits_of(turn(k)), kg, c.k_q, c.k_sf), (v, vg, c.v_q, c.v_sf)):
        q_, sf_, _ = oracle.quantize(bits.reshape(tokens * heads, D), global_scale=np.array([gs], np.float32))[:3]
        want_q = np.full((pages, heads, ps, D // 2), 0xA5, np.uint8)
        want_s = np.full((pages, heads, ps, D // 16), 0xA5, np.uint8)
        for t in range(tokens):
            if slots[t] >= 0:
                want_q[slots[t] // ps, :, slots[t] % ps] = q_.reshape(tokens, heads, -1)[t]
                want_s[slots[t] // ps, :, slots[t] % ps] = sf_.reshape(tokens, heads, -1)[t]
        same(to_np(codes), want_q)
        same(to_np(scales), want_s)


def test_append_refuses_bad_slots_positions_and_values():
    L, nv = layer(), nvmod()
    rng = np.random.default_rng(3)
    D, heads, ps, pages, tokens = 128, 2, 16, 4, 6
    gs = torch.tensor([0.01], device="cuda")
    k = random_bf16(rng, tokens, heads, D)
    rope = L.rope_table(50, 64)
    for what in ("slot", "position", "nan", "scale"):
        c = L.PagedKVCache.empty(pages, ps, heads, D, gs if what != "scale" else -gs, gs)
        for t in (c.k_q, c.k_sf, c.v_q, c.v_sf):
            t.fill_(0x11)
        slots, pos, kk = np.arange(tokens), np.arange(tokens), k.copy()
        if what == "slot":
            slots[2], slots[4] = pages * ps, 1 << 40
        if what == "position":
            pos[2], pos[4] = 50, -1
        if what == "nan":
            kk[2, 1, 100] = 0x7FC0
        st = status_word()
        q = bf16_dev(k)
        c.append(bf16_dev(kk), bf16_dev(k), to_dev(slots), q=q, q_out=torch.zeros_like(q), positions=to_dev(pos),
                 rope=rope, dev_status=st)
        want = {"slot": nv.ERR_INDEX, "position": nv.ERR_INDEX, "nan": nv.ERR_NONFINITE, "scale": nv.ERR_INVALID_ARG}
        assert st.item() == want[what]
        if what in ("slot", "position"):       # the bad tokens' rows are left as they were
            assert (c.k_q[0, :, [2, 4]] == 0x11).all() and (c.v_sf[0, :, [2, 4]] == 0x11).all()
            assert (c.k_q[1:] == 0x11).all() and (c.k_sf[0, :, 6:] == 0x11).all()
            assert not (c.k_q[0, :, [1, 3]] == 0x11).all()
        if what == "nan":                      # the block with the NaN is zeros, its neighbours are not
            assert (c.k_q[0, 1, 2, 48:56] == 0).all() and c.k_sf[0, 1, 2, 6] == 0 and c.k_sf[0, 1, 2, 5] != 0


def test_append_then_dequantize_is_the_kv_quantize_round_trip():
    """Without rotation the cache holds what nvfp4_kv_quantize writes."""
    L, nv = layer(), nvmod()
    rng = np.random.default_rng(8)
    tokens, heads, D, ps = 64, 4, 256, 16
    k, v = bf16_dev(random_bf16(rng, tokens, heads, D)), bf16_dev(random_bf16(rng, tokens, heads, D))
    kg, vg = torch.tensor([0.004], device="cuda"), torch.tensor([0.005], device="cuda")
    c = L.PagedKVCache.empty(tokens // ps, ps, heads, D, kg, vg)
    c.append(k, v, torch.arange(tokens, device="cuda"))
    kq, vq = (torch.empty(tokens, heads, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(tokens, heads, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    nv.nvfp4_kv_quantize(k, v, tokens, heads, D, nv.GS_GIVEN, kg, vg, kq, ks, vq, vs, L.workspace(2))
    for pool, flat in ((c.k_q, kq), (c.v_q, vq), (c.k_sf, ks), (c.v_sf, vs)):
        assert torch.equal(pool.transpose(1, 2).reshape(tokens, heads, -1), flat)
    back = c.dequantize()
    for x, q, s, g in ((back[0], kq, ks, kg), (back[1], vq, vs, vg)):
        want = torch.empty(tokens, heads * D, dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_dequantize(q, s, L.SF_ROWMAJOR, g, None, 1, tokens, heads * D, want, L.OUT_BF16)
        assert torch.equal(x.transpose(1, 2).reshape(tokens, -1), want)


# ---------------------------------------------------------------------------------------- attention
class Case:
    """A paged cache of random codes with garbage in every unused row, its page
    table with garbage past each length, and the 64-bit reference."""

    def __init__(self, seed, D, hkv, group, ps, lens, queries=None, causal=True, spread=1.0):
        L = layer()
        self.D, self.hkv, self.group, self.ps, self.lens, self.causal = D, hkv, group, ps, lens, causal
        self.counts = [1] * len(lens) if queries is None else queries
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g, device="cuda").cpu().tolist()
        width = max(need + [1]) + 1
        table = torch.full((len(lens), width), -(1 << 30), dtype=torch.int32)
        self.pages = []
        for i, n in enumerate(need):
            mine = [perm.pop() for _ in range(n)]
            self.pages.append(mine)
            table[i, :n] = torch.tensor(mine, dtype=torch.int32)
        self.table = table.cuda()
        shape = (pages, hkv, ps)
        self.t = {}
        for n in "kv":
            codes = torch.randint(0, 256, (*shape, D // 2), generator=g, device="cuda", dtype=torch.uint8)
            scales = torch.randint(0x28, 0x48, (*shape, D // 16), generator=g, device="cuda", dtype=torch.uint8)
            scales[torch.rand(scales.shape, generator=g, device="cuda") < 0.02] = 0
            used = torch.zeros(shape, dtype=torch.bool, device="cuda")
            for i, length in enumerate(lens):
                for j, p in enumerate(self.pages[i]):
                    used[p, :, :max(0, min(ps, length - j * ps))] = True
            scales[~used] = 0xFF          # NaN, negative: whatever the memory held
            codes[~used] = 0x7F
            self.t[n + "_q"], self.t[n + "_sf"] = codes, scales
        self.kgs = torch.tensor([0.31 * spread], device="cuda")
        self.vgs = torch.tensor([0.7], device="cuda")
        self.cache = L.PagedKVCache(self.t["k_q"], self.t["k_sf"], self.kgs, self.t["v_q"], self.t["v_sf"], self.vgs)
        T = sum(self.counts)
        self.q = torch.randn(T, hkv * group, D, generator=g, device="cuda").to(torch.bfloat16)
        self.offsets = None
        if queries is not None:
            self.offsets = torch.tensor([0] + list(np.cumsum(queries)), dtype=torch.int32, device="cuda")
        self.max_query = max(self.counts + [1])
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        a = dict(query_offsets=self.offsets, max_query=self.max_query, causal=self.causal)
        return self.cache.attend(kw.pop("q", self.q), kw.pop("seq_lens", self.seq_lens),
                                 kw.pop("page_table", self.table), **dict(a, **kw))

    def dense(self, n, i):
        """Sequence i's keys or values [hkv, len, D] in 64 bits."""
        b = self.t[n + "_q"][self.pages[i]].transpose(0, 1)
        s = self.t[n + "_sf"][self.pages[i]].transpose(0, 1).contiguous()
        lut = torch.tensor(E2M1, device="cuda")
        v = torch.stack((lut[(b & 15).long()], lut[(b >> 4).long()]), -1).flatten(-2)
        v = v.unflatten(-1, (-1, 16)) * s.view(torch.float8_e4m3fn).double()[..., None]
        return v.flatten(-2).flatten(1, 2)[:, :self.lens[i]] * (self.kgs if n == "k" else self.vgs).double()

    def reference(self, skip=None, q=None):
        """(out, lse, weight): in 64 bits; weight = sum p |v| / sum p, what the
        tolerance scales with.  skip[i]: tokens of sequence i left out."""
        q = self.q if q is None else q
        D, H = self.D, self.hkv * self.group
        outs, lses, mags, self.dscore, self.vmax = [], [], [], 0.0, 0.0
        row = 0
        for i, (n, c) in enumerate(zip(self.lens, self.counts)):
            x = q[row:row + c].double()
            row += c
            k, v = self.dense("k", i), self.dense("v", i)
            hk = torch.arange(H, device="cuda") // self.group
            s = torch.einsum("chd,hnd->hcn", x, k[hk]) * D ** -0.5
            if n and c:
                self.vmax = max(self.vmax, v.abs().max().item())
                self.dscore = max(self.dscore, (torch.einsum("chd,hnd->hcn", x.abs(), k[hk].abs()).max() * D ** -0.5).item())
            see = torch.ones(c, n, dtype=torch.bool, device="cuda")
            if self.causal:
                see = torch.arange(n, device="cuda")[None, :] <= (n - c + torch.arange(c, device="cuda"))[:, None]
            if skip is not None and i in skip:
                see[:, skip[i]] = False
            s = s.masked_fill(~see, -float("inf"))
            lse = torch.logsumexp(s, -1) if n else torch.full((H, c), -float("inf"), dtype=torch.float64, device="cuda")
            p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
            outs.append(torch.einsum("hcn,hnd->chd", p, v[hk]))
            mags.append(torch.einsum("hcn,hnd->chd", p, v[hk].abs()))
            lses.append(lse.T)
        return torch.cat(outs), torch.cat(lses), torch.cat(mags)

    def tolerance(self, out, mag, dtype):
        """A weight p is rounded to f16 once: 2^-11 of it, or, below f16's normal
        range, at most 2^-25 absolute.  Weights are relative to a running maximum
        that is at most the row's largest score, so the largest weight and with
        it their sum is at least 1, and N absolute errors of 2^-25 move the
        output by at most N 2^-25 max|v| (this term is absolute: where the
        heaviest keys have a zero in an element, `mag` there is far smaller).
        Scores are off by the fp32 sums of D products and the log2 scaling
        ((D + 4) 2^-23 of sum |q k|), exp2 by 2^-22, and the accumulators by at
        most N/16 + 64 sequential fp32 additions; then the output's own rounding."""
        N = max(self.lens + [1])
        ds = (self.D + 4) * 2.0 ** -23 * max(self.dscore, 1.0)
        rel = 2.0 ** -11 + 2 * ds + 2.0 ** -21 + (N / 16 + 64) * 2.0 ** -22
        half = torch.finfo(dtype).eps / 2
        return (mag * rel + N * 2.0 ** -25 * self.vmax) * (1 + half) + out.abs() * half


ATTEND = [
    # D, hkv, group, page, lengths, queries, causal
    (64, 1, 1, 16, [1], None, True),
    (64, 2, 8, 16, [1, 0, 15, 16, 17, 33], None, True),
    (64, 8, 8, 64, [700, 5], None, True),
    (128, 1, 1, 16, [0], None, True),
    (128, 8, 4, 64, [1000, 31, 32, 33, 64, 65, 1], None, True),
    (128, 2, 16, 128, [517, 129], None, True),
    (128, 2, 5, 48, [100, 47, 48, 49], None, True),
    (128, 1, 32, 32, [300], None, True),
    (256, 4, 8, 64, [1000], None, True),
    (256, 4, 8, 64, [4096, 1, 0, 63, 257, 2000, 31, 5], None, True),
    (256, 1, 3, 16, [50, 16], None, True),
    (256, 2, 16, 32, [333], None, True),
    (256, 1, 1, 64, [20000], None, True),
    # several queries a sequence: verification, more queries than keys, none, short prompts
    (64, 2, 4, 16, [40, 3, 17], [4, 5, 0], True),
    (64, 2, 8, 32, [200, 90], [50, 90], True),
    (128, 8, 4, 64, [513, 2, 130], [3, 4, 2], True),
    (128, 2, 4, 16, [65, 65], [65, 1], True),
    (128, 1, 7, 64, [300], [123], True),
    (256, 4, 8, 64, [129, 1000, 7], [4, 1, 3], True),
    (256, 2, 2, 32, [70, 0, 33], [70, 2, 40], True),
    (256, 1, 8, 128, [260], [17], False),
    (128, 4, 4, 64, [99, 64], [6, 64], False),
    (64, 1, 2, 16, [31, 77], [2, 7], False),
    # sequences on both sides of the row limit between the two forms, in one batch
    (256, 2, 8, 64, [300, 1000, 64, 5, 0, 129], [1, 200, 2, 5, 3, 3], True),
    (128, 2, 4, 48, [300, 1000, 64, 513, 9], [8, 9, 1, 400, 9], True),
    (64, 1, 16, 16, [130, 2000, 17], [2, 3, 17], True),
    # many row blocks and tiles, shared between CTAs
    (128, 1, 4, 64, [6000], [257], True),
    (256, 1, 2, 64, [9000, 200], [130, 65], True),
    (64, 2, 1, 32, [700, 1500], [700, 1400], True),
]


@pytest.mark.parametrize("D,hkv,group,ps,lens,queries,causal", ATTEND)
def test_attention_matches_64_bits(D, hkv, group, ps, lens, queries, causal):
    L = layer()
    c = Case(sum(lens) + D, D, hkv, group, ps, lens, queries, causal)
    want, lse, mag = c.reference()
    for dt, td in ((L.OUT_F32, torch.float32), (L.OUT_BF16, torch.bfloat16)):
        st = status_word()
        ls = torch.full(lse.shape, 5.0, dtype=torch.float32, device="cuda")
        out = torch.full(c.q.shape, float("nan"), dtype=td, device="cuda")
        c.run(out=out, out_dtype=dt, lse=ls, dev_status=st)
        assert st.item() == 0
        err = (out.double() - want).abs() - c.tolerance(want, mag, td)
        assert not torch.isnan(out).any() and err.max().item() <= 0, err.max().item()
        empty = torch.isinf(lse)
        assert torch.equal(empty, torch.isinf(ls)) and (out[empty] == 0).all()
        assert ((ls - lse)[~empty].abs() <= 2e-4 + 2.0 ** -21 * lse[~empty].abs()).all()
        again = c.run(out_dtype=dt)
        assert torch.equal(again, out)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_rising_and_peaked_scores(D):
    """Scores far apart: the running maximum rises many times, most weights
    vanish, and the largest key comes first, last or in the middle."""
    for seed, spread in ((1, 30.0), (2, 200.0)):
        c = Case(seed, D, 2, 4, 32, [900, 333], None, True, spread=spread)
        want, lse, mag = c.reference()
        out = c.run(out_dtype=layer().OUT_F32)
        err = (out.double() - want).abs() - c.tolerance(want, mag, torch.float32)
        assert err.max().item() <= 0, err.max().item()


# up to 32 rows a KV head, in batches of many short items and of one long among many
FEW_ROWS = [
    # D, hkv, group, page, lengths, queries
    (256, 1, 17, 16, [1, 15, 16, 17, 31, 32, 33, 1000], None),
    (256, 2, 6, 32, [5000, 4, 640, 0, 129, 77], [4, 4, 3, 2, 1, 4]),
    (256, 1, 32, 64, [3000], None),
    (256, 4, 8, 32, [9 * i % 131 for i in range(64)], [1 + i % 4 for i in range(64)]),
    (256, 1, 8, 16, [40000] + [20] * 60, [4] * 61),
    (256, 1, 4, 64, [30000] + [70] * 60, None),
    (128, 1, 8, 64, [60000] + [30] * 60, [2] * 61),
    (64, 2, 2, 16, [30000] + [7] * 40, None),
]


@pytest.mark.parametrize("D,hkv,group,ps,lens,queries", FEW_ROWS)
@pytest.mark.parametrize("spread", [None, 100.0])
def test_attention_few_rows(D, hkv, group, ps, lens, queries, spread):
    c = Case(sum(lens) + group, D, hkv, group, ps, lens, queries, True, **({} if spread is None else {"spread": spread}))
    want, lse, mag = c.reference()
    ls = torch.full(lse.shape, 5.0, dtype=torch.float32, device="cuda")
    st = status_word()
    out = c.run(out_dtype=layer().OUT_F32, lse=ls, dev_status=st)
    assert st.item() == 0
    err = (out.double() - want).abs() - c.tolerance(want, mag, torch.float32)
    assert not torch.isnan(out).any() and err.max().item() <= 0, err.max().item()
    empty = torch.isinf(lse)
    assert torch.equal(empty, torch.isinf(ls)) and (out[empty] == 0).all()


@pytest.mark.parametrize("D,hkv,group,ps,lens,queries", [
    (128, 8, 4, 64, [2048], [2048]),
    (64, 8, 4, 32, [2048], [2048]),
    (128, 2, 8, 128, [1500, 900, 1800], [700, 900, 1]),
    (256, 4, 4, 64, [1500], [1500]),
])
@pytest.mark.parametrize("spread", [1.0, 3.0, 10.0])
def test_attention_prompts_whose_maxima_rise_here_and_there(D, hkv, group, ps, lens, queries, spread):
    """Several items a CTA, and rows whose maxima rise at some later tile while
    the others' do not."""
    c = Case(D + int(spread), D, hkv, group, ps, lens, queries, True, spread=spread)
    want, _, mag = c.reference()
    out = c.run(out_dtype=layer().OUT_F32)
    err = (out.double() - want).abs() - c.tolerance(want, mag, torch.float32)
    assert not torch.isnan(out).any() and err.max().item() <= 0, err.max().item()


@pytest.mark.parametrize("D,hkv,group,ps,lens", [
    (128, 8, 4, 64, [4096]),
    (64, 8, 4, 64, [4096]),
    (256, 4, 4, 64, [3000]),
    (128, 4, 4, 16, [1000, 2000, 500]),
])
def test_attention_prompts_repeat_to_the_bit(D, hkv, group, ps, lens):
    """Every run gives the same bits, with the cache in L2 or not."""
    c = Case(D, D, hkv, group, ps, lens, lens, True)
    first = c.run(out_dtype=layer().OUT_F32)
    evict = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(100):
        if i % 2:
            evict.fill_(i)
        assert torch.equal(c.run(out_dtype=layer().OUT_F32), first), i


def test_attention_large_and_small_queries():
    """bf16 queries far outside f16's range are scaled by row."""
    c = Case(4, 128, 2, 4, 64, [200, 70], None, True, spread=2.0 ** -60)
    q = (c.q.float() * 2.0 ** 60).to(torch.bfloat16)
    want, _, mag = c.reference(q=q)
    out = c.run(q=q, out_dtype=layer().OUT_F32)
    err = (out.double() - want).abs() - c.tolerance(want, mag, torch.float32)
    assert err.max().item() <= 0
    tiny = torch.full_like(c.q, 1e-40)
    want, _, mag = c.reference(q=tiny)
    out = c.run(q=tiny, out_dtype=layer().OUT_F32)
    assert ((out.double() - want).abs() <= c.tolerance(want, mag, torch.float32)).all()


def test_attention_a_nan_query_stays_in_its_row():
    c = Case(5, 128, 2, 4, 16, [100, 90], [3, 2], True)
    clean = c.run()
    q = c.q.clone()
    q[1, 2, 7] = float("nan")
    out = c.run(q=q)
    assert torch.isnan(out[1, 2]).all()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    assert torch.equal(out[keep], clean[keep])


def test_attention_leaves_other_rows_and_takes_strided_queries():
    """Rows before the first and behind the last sequence keep what they held;
    q may be a slice of a wider tensor."""
    L = layer()
    c = Case(6, 128, 2, 4, 16, [100, 90], [3, 2], True)
    want = c.run()
    wide = torch.randn(9, 8 * 128 + 40, device="cuda").to(torch.bfloat16)
    q = wide[:, 16:16 + 8 * 128].unflatten(1, (8, 128))
    q[2:7] = c.q
    out = torch.full((9, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 8), 4.0, device="cuda")
    c.cache.attend(q, c.seq_lens, c.table, query_offsets=c.offsets + 2, max_query=5, out=out, lse=lse)
    assert torch.equal(out[2:7], want)
    assert (out[:2] == 3).all() and (out[7:] == 3).all() and (lse[:2] == 4).all() and (lse[7:] == 4).all()
    assert (lse[2:7] != 4).all()


def test_attention_bad_pages_lengths_and_offsets():
    nv, L = nvmod(), layer()
    c = Case(7, 128, 2, 4, 16, [100, 90], None, True)
    table = c.table.clone()
    table[0, 2], table[1, 0] = c.cache.num_pages, -1
    st = status_word()
    out = c.run(page_table=table, out_dtype=L.OUT_F32, dev_status=st)
    assert st.item() == nv.ERR_INDEX
    want, _, mag = c.reference(skip={0: slice(32, 48), 1: slice(0, 16)})
    assert ((out.double() - want).abs() <= c.tolerance(want, mag, torch.float32)).all()
    # the same with many queries a sequence
    for D in (64, 128, 256):
        c = Case(8, D, 2, 4, 16, [300, 290], [150, 60], True)
        table = c.table.clone()
        table[0, 2], table[0, 17], table[1, 0] = c.cache.num_pages, 1 << 30, -1
        st = status_word()
        out = c.run(page_table=table, out_dtype=L.OUT_F32, dev_status=st)
        assert st.item() == nv.ERR_INDEX
        want, _, mag = c.reference(skip={0: list(range(32, 48)) + list(range(272, 288)), 1: list(range(16))})
        assert ((out.double() - want).abs() <= c.tolerance(want, mag, torch.float32)).all()
    c = Case(7, 128, 2, 4, 16, [100, 90], None, True)
    for bad in (-1, c.table.shape[1] * 16 + 1, 1 << 30):
        lens = c.seq_lens.clone()
        lens[0] = bad
        st = status_word()
        out = c.run(seq_lens=lens, dev_status=st)
        assert st.item() == nv.ERR_INDEX and (out[0] == 0).all() and torch.equal(out[1], c.run()[1])
    c = Case(7, 128, 2, 4, 16, [100, 90], [3, 2], True)
    for bad in ([0, 3, 6], [0, 3, 2], [-1, 3, 5], [0, 5, 5], [4, 1, 5]):
        st = status_word()
        out = torch.full(c.q.shape, 2.0, dtype=torch.bfloat16, device="cuda")
        c.run(query_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out, dev_status=st)
        assert st.item() == nv.ERR_INDEX and (out == 2).all()


def test_attention_pool_past_32_bit_offsets():
    """Pages whose byte offsets pass 2^32."""
    L = layer()
    pages, hkv, ps, D = 140000, 4, 64, 256
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 12 GB of device memory")
    gs = torch.ones(1, device="cuda")
    big = L.PagedKVCache.empty(pages, ps, hkv, D, gs, gs)
    assert big.k_q.numel() > 1 << 32
    c = Case(9, D, hkv, 2, ps, [150], None, True)
    far = [pages - 1, 3, pages - 2]
    for t in ("k_q", "k_sf", "v_q", "v_sf"):
        getattr(big, t)[far] = c.t[t][c.pages[0]]
    big.k_gs, big.v_gs = c.kgs, c.vgs
    out = big.attend(c.q, c.seq_lens, torch.tensor([far], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, c.run())
    # and the append reaches them
    k = torch.randn(2, hkv, D, device="cuda").to(torch.bfloat16)
    big.append(k, k, torch.tensor([(pages - 1) * ps + 5, (pages - 3) * ps], device="cuda"))
    small = L.PagedKVCache.empty(1, ps, hkv, D, c.kgs, c.vgs)
    small.append(k, k, torch.tensor([5, 0], device="cuda"))
    assert torch.equal(big.k_q[pages - 1, :, 5], small.k_q[0, :, 5])
    assert torch.equal(big.v_sf[pages - 3, :, 0], small.v_sf[0, :, 0])


def test_attention_on_another_stream_and_in_graphs():
    """A side stream, a captured graph replayed on new contents, and two graphs
    with workspaces of their own replayed at the same time."""
    c = Case(10, 256, 4, 8, 64, [3000, 500, 0], None, True)
    d = Case(11, 128, 2, 4, 16, [700, 90], [3, 2], True)
    want_c, want_d = c.run(), d.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    side.synchronize()
    assert torch.equal(got, want_c)
    graphs = []
    for x in (c, d):
        ws = x.cache.workspace(len(x.lens), x.max_query, x.q.shape[1])
        out = torch.empty_like(x.q)
        x.run(ws=ws, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(ws=ws, out=out)
        graphs.append((g, out))
    for g, out in graphs:
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want_c) and torch.equal(graphs[1][1], want_d)
    c.q.mul_(-0.5)
    c.seq_lens[1] = 77
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], c.run())


def test_norm_append_attend_as_a_layer_uses_them():
    """Two steps of a layer: a prompt chunk and then single tokens, each normed,
    projected, appended and attended.  The attention over the cache equals the
    64-bit attention of the cache's own values, whichever way they came in."""
    L = layer()
    torch.manual_seed(0)
    H, hkv, group, D, ps, rot = 512, 2, 4, 128, 16, 64
    hq = hkv * group
    wqkv = (torch.randn((hq + 2 * hkv) * D, H, device="cuda") * 0.04).to(torch.bfloat16)
    wn = (1 + 0.1 * torch.randn(H, device="cuda")).to(torch.bfloat16)
    rope = L.rope_table(4096, rot)
    gs = torch.tensor([8.0 / 2688], device="cuda")
    cache = L.PagedKVCache.empty(12, ps, hkv, D, gs, gs)
    table = torch.tensor([[7, 2, 9, 4, 0, 11]], dtype=torch.int32, device="cuda")
    resid = torch.randn(70, H, device="cuda").to(torch.bfloat16)
    x = torch.randn(70, H, device="cuda").to(torch.bfloat16)
    st = status_word()
    chunks, outs, at = [(0, 50), (50, 67), (67, 68), (68, 69), (69, 70)], [], 0
    qs = []
    for a, b in chunks:
        n = b - a
        q8, s8, r, _ = L.add_rmsnorm_e4m3(x[a:b], wn, residual=resid[a:b], dev_status=st)
        h = (q8.view(torch.float8_e4m3fn).float() * s8[:, None]).to(torch.bfloat16)
        qkv = h @ wqkv.T
        q, k, v = (qkv[:, i:j].unflatten(1, (-1, D)) for i, j in
                   ((0, hq * D), (hq * D, (hq + hkv) * D), ((hq + hkv) * D, (hq + 2 * hkv) * D)))
        pos = torch.arange(a, b, device="cuda")
        slots = table[0].long()[pos // ps] * ps + pos % ps
        q = cache.append(k, v, slots, q=q, positions=pos, rope=rope, dev_status=st)
        offs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        outs.append(cache.attend(q, torch.tensor([b], dtype=torch.int32, device="cuda"), table, query_offsets=offs,
                                 max_query=n, out_dtype=L.OUT_F32, dev_status=st))
        qs.append(q)
    assert st.item() == 0
    kd, vd = (t.double()[table[0].long()].transpose(1, 2).reshape(-1, hkv, D)[:70] for t in cache.dequantize())
    q, out = torch.cat(qs).double(), torch.cat(outs).double()
    hk = torch.arange(hq, device="cuda") // group
    s = torch.einsum("chd,nhd->hcn", q, kd[:, hk]) * D ** -0.5
    s = s.masked_fill(torch.ones(70, 70, device="cuda").triu(1).bool(), -float("inf"))
    p = torch.softmax(s, -1)
    want = torch.einsum("hcn,nhd->chd", p, vd[:, hk])
    mag = torch.einsum("hcn,nhd->chd", p, vd[:, hk].abs())
    # dequantize() rounds each value to bf16 (2^-8 of it): in v directly, in k through the scores
    ds = torch.einsum("chd,nhd->hcn", q.abs(), kd[:, hk].abs()).max().item() * D ** -0.5 * 2.0 ** -8
    assert ((out - want).abs() <= mag * (2.0 ** -8 + 2.0 ** -10 + 2 * ds)).all()


def test_status_words_and_scales_elsewhere_are_refused():
    L = layer()
    c = Case(3, 64, 1, 2, 16, [20])
    host = torch.zeros(1, dtype=torch.int32)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    gs = torch.ones(1, device="cuda")
    short = L.empty_packed(4, 64)
    short.sf = short.sf[:16]
    for call in (lambda: c.run(dev_status=host), lambda: L.add_rmsnorm_e4m3(x, w, dev_status=host),
                 lambda: L.add_rmsnorm_nvfp4(x, w, gs, dev_status=host), lambda: L.add_rmsnorm_nvfp4(x, w, gs, out=short),
                 lambda: c.cache.append(c.q[:, :1], c.q[:, :1], torch.zeros(1, dtype=torch.int64, device="cuda"),
                                        dev_status=host)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("D,group", [(64, 33), (128, 48), (256, 64), (128, 200)])
def test_attention_one_query_of_many_heads(D, group):
    """More heads on one KV head than the few-row form takes."""
    c = Case(group, D, 1, group, 32, [700, 0, 33, 128])
    want, lse, mag = c.reference()
    ls = torch.full(lse.shape, 5.0, dtype=torch.float32, device="cuda")
    out = c.run(out_dtype=layer().OUT_F32, lse=ls)
    err = (out.double() - want).abs() - c.tolerance(want, mag, torch.float32)
    assert not torch.isnan(out).any() and err.max().item() <= 0
    assert torch.equal(torch.isinf(lse), torch.isinf(ls))


@pytest.mark.parametrize("queries", [False, True])
def test_attention_largest_batch(queries):
    lens = [(7 * i) % 40 for i in range(4096)]
    counts = [min(n, 1 + i % 20) for i, n in enumerate(lens)] if queries else None
    c = Case(5, 64, 1, 2, 16, lens, counts)
    want, _, mag = c.reference()
    out = c.run(out_dtype=layer().OUT_F32)
    err = (out.double() - want).abs() - c.tolerance(want, mag, torch.float32)
    assert not torch.isnan(out).any() and err.max().item() <= 0


def test_attention_of_an_empty_pool():
    L = layer()
    gs = torch.ones(1, device="cuda")
    cache = L.PagedKVCache.empty(0, 16, 2, 128, gs, gs)
    q = torch.ones(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    for width in (0, 2):
        st = status_word()
        out = cache.attend(q, torch.zeros(3, dtype=torch.int32, device="cuda"),
                           torch.zeros(3, width, dtype=torch.int32, device="cuda"), dev_status=st)
        assert (out == 0).all() and st.item() == 0
    many = torch.ones(70, 4, 128, dtype=torch.bfloat16, device="cuda")
    out = cache.attend(many, torch.zeros(1, dtype=torch.int32, device="cuda"),
                       torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                       query_offsets=torch.tensor([0, 70], dtype=torch.int32, device="cuda"), max_query=70)
    assert (out == 0).all()


def test_attention_of_two_streams_at_once():
    """Both forms at the same time, each with memory of its own."""
    cases = [Case(1, 128, 8, 4, 64, [1500], [1500]), Case(2, 256, 4, 8, 64, [9000, 70, 800], None),
             Case(3, 64, 4, 4, 32, [1000], [1000])]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(10):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.run())
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for y in gs:
            assert torch.equal(y, w)


def test_norm_and_append_in_a_graph():
    """Captured once, replayed on new rows, slots and positions."""
    L = layer()
    torch.manual_seed(1)
    T, H, D, hkv = 5, 256, 64, 2
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    w = torch.randn(H, device="cuda").to(torch.bfloat16)
    gs = torch.tensor([0.01], device="cuda")
    cache = L.PagedKVCache.empty(8, 16, hkv, D, gs, gs)
    other = L.PagedKVCache.empty(8, 16, hkv, D, gs, gs)
    for c in (cache, other):
        for t in (c.k_q, c.k_sf, c.v_q, c.v_sf):
            t.zero_()
    rope = L.rope_table(200, D)
    k, v, q = (torch.randn(T, n, D, device="cuda").to(torch.bfloat16) for n in (hkv, hkv, 4))
    slots = torch.arange(T, device="cuda")
    pos = torch.arange(T, device="cuda")

    def step(c):
        return L.add_rmsnorm_nvfp4(x, w, gs)[0], L.add_rmsnorm_e4m3(x, w)[:2], \
            c.append(k, v, slots, q=q, positions=pos, rope=rope)

    step(other)
    torch.cuda.synchronize()
    for t in (other.k_q, other.k_sf, other.v_q, other.v_sf):
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        packed, (e, scale), qr = step(cache)
    for i in range(3):
        x.copy_(torch.randn(T, H, device="cuda"))
        k.copy_(torch.randn(T, hkv, D, device="cuda"))
        slots.copy_(torch.tensor([17 * i, -1, 40 + i, 60, 127 - i], device="cuda"))
        pos.copy_(torch.tensor([i, 3, 150, 7, 199 - i], device="cuda"))
        g.replay()
        p2, (e2, s2), q2 = step(other)
        torch.cuda.synchronize()
        rows = slice(0, T)
        assert torch.equal(packed.q[rows], p2.q[rows]) and torch.equal(e, e2) and torch.equal(scale, s2)
        assert torch.equal(qr, q2)
        for a in ("k_q", "k_sf", "v_q", "v_sf"):
            assert torch.equal(getattr(cache, a), getattr(other, a))


def test_append_to_an_empty_pool_and_to_one_slot_twice():
    """Without pages the queries are still turned; a slot named twice holds
    finite values, and its neighbours are untouched."""
    L = layer()
    torch.manual_seed(2)
    gs = torch.tensor([0.01], device="cuda")
    k, v, q = (torch.randn(4, n, 64, device="cuda").to(torch.bfloat16) for n in (2, 2, 4))
    rope, pos = L.rope_table(50, 64), torch.tensor([0, 9, 30, 49], device="cuda")
    want = None
    for pages, slots in ((0, [-1, -1, -1, -1]), (3, [7, 7, 20, 7])):
        cache = L.PagedKVCache.empty(pages, 16, 2, 64, gs, gs)
        for t in (cache.k_q, cache.k_sf, cache.v_q, cache.v_sf):
            t.fill_(0x11)
        st = status_word()
        got = cache.append(k, v, torch.tensor(slots, device="cuda"), q=q, positions=pos, rope=rope, dev_status=st)
        assert st.item() == 0
        want = got if want is None else want
        assert torch.equal(got, want)
        if pages:
            for t in (cache.k_q, cache.k_sf, cache.v_q, cache.v_sf):
                rows = t.transpose(1, 2).reshape(pages * 16, -1)
                keep = torch.ones(pages * 16, dtype=torch.bool, device="cuda")
                keep[torch.tensor([7, 20], device="cuda")] = False
                assert (rows[keep] == 0x11).all()
            kd, vd = cache.dequantize()
            assert torch.isfinite(kd).all() and torch.isfinite(vd).all()
