"""The attention half of a decoder layer on the GPU against 64-bit plain forms (attention_ref.py): norm, rotary
positions, cache writes and reads, single-token attention, at the sizes, strides and masks where each can go wrong."""
import math

import numpy as np
import pytest
import torch

import attention_ref as ref
import weight_only_fp4_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


def say(msg):
    print(f"[gpu-case] {msg}", flush=True)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(shape, g, dtype, sigma=1.0):
    return (torch.randn(shape, generator=g) * sigma).to(dtype)


def strided(t, pad, dtype=None):
    """t on the device inside rows longer by `pad` elements (NaN around it)."""
    full = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    view = full[..., :t.shape[-1]]
    view.copy_(t)
    return view


# ------------------------------------------------------------------- norm --

@pytest.mark.parametrize("T,N,dt,res,pad", [
    (1, 4096, BF, True, 0), (3, 5120, HF, True, 8), (2, 8, BF, False, 0), (5, 64, HF, True, 0), (4, 1040, BF, True, 16),
    (1, 1, BF, True, 0), (3, 7, HF, False, 3), (2, 1041, BF, True, 1), (2, 32768, HF, True, 0), (2, 32776, BF, True, 0),
    (700, 136, BF, True, 0), (2, 16384, BF, False, 0), (37, 128, HF, True, 8), (1, 120, BF, False, 0), (9, 512, BF, True, 0),
    (300, 520, HF, True, 0), (300, 16392, BF, True, 0), (260, 8192, HF, False, 0),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_norm(T, N, dt, res, pad, fp8):
    say(f"norm T={T} N={N} {dt} res={res} pad={pad} fp8={fp8}")
    g = gen(T * 1000 + N)
    x, r = normal((T, N), g, dt, 2.0), normal((T, N), g, dt, 3.0)
    w = (1 + 0.3 * torch.randn(N, generator=g)).to(dt)
    eps = 1e-5
    xd, rd = strided(x, pad), strided(r, pad)
    call = nv.rms_norm_fp8 if fp8 else nv.rms_norm
    got = call(xd, w.to(DEV), eps, residual=rd if res else None)
    h = x
    assert (got[-1] is None) == (not res)
    if res:
        h = (x.float() + r.float()).to(dt)
        assert torch.equal(got[-1].cpu().view(torch.int16), h.view(torch.int16))
    y, rel = ref.norm(ref.f64(h), ref.f64(w), eps)
    if not fp8:
        bound = np.abs(y) * (rel + ref.u(dt) * (1 + rel)) + ref.least(dt)
        assert np.all(np.abs(ref.f64(got[0]) - y) <= bound)
        return
    s = ref.f64(got[1])
    want = np.maximum(np.abs(y).max(1) / 448, 2.0 ** -126)
    assert np.all(np.abs(s - want) <= want * (rel + 2 * ref.U32))
    v = y / s[:, None]   # off by the norm's error and one reciprocal and product
    bound = np.abs(v) * (2.0 ** -4 * (1 + 2 * rel) + rel + 4 * ref.U32) + 2.0 ** -10
    assert np.all(np.abs(ref.f64(got[0].float()) - v) <= bound)


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_beyond_the_caches(fp8):
    """A call that moves more than 256 MB takes the streaming form: the same bits as its rows in a smaller call."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    T, N = 6000, 8192
    x = torch.randn((T, N), generator=g, device=DEV).to(BF)
    r = torch.randn((T, N), generator=g, device=DEV).to(BF)
    w = torch.rand(N, generator=g, device=DEV).to(BF)
    call = nv.rms_norm_fp8 if fp8 else nv.rms_norm
    big = call(x, w, residual=r)
    for lo in (0, 2999, T - 300):
        small = call(x[lo:lo + 300], w, residual=r[lo:lo + 300])
        for a, b in zip(big, small):
            assert torch.equal(a[lo:lo + 300].contiguous().view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("N", [4096, 77])
def test_norm_in_place_and_edge_rows(N):
    """The residual updated in place; a row of zeros, one with an infinity, one with a NaN; the other rows are not
    touched by them."""
    g = gen(5)
    x, r = normal((4, N), g, BF), normal((4, N), g, BF)
    x[0] = 0
    r[0] = 0
    x[1, 3] = math.inf
    x[2, N - 1] = math.nan
    w = torch.ones(N, dtype=BF, device=DEV)
    for fp8 in (False, True):
        call = nv.rms_norm_fp8 if fp8 else nv.rms_norm
        fresh = call(x.to(DEV), w, 1e-6, residual=r.to(DEV))
        rd = r.to(DEV)
        got = call(x.to(DEV), w, 1e-6, residual=rd, residual_out=rd)
        assert got[-1].data_ptr() == rd.data_ptr()
        for a, b in zip(fresh, got):
            assert torch.equal(a.float().nan_to_num(99), b.float().nan_to_num(99))
        y = got[0].float()
        assert torch.all(y[0] == 0) and torch.isnan(y[1, 3]) and torch.isnan(y[2]).all()
        assert torch.isfinite(y[3]).all()
        if fp8:   # a NaN in a row makes its scale and so the whole row one
            assert got[1][0] == 2.0 ** -126 and torch.isnan(got[1][1:3]).all() and torch.isfinite(got[1][3])
            assert torch.isnan(y[1]).all()
        else:
            assert torch.all(y[1, :3] == 0)


# ----------------------------------------------------------------- rotary --

@pytest.mark.parametrize("T,H,D,R,axes,inter,dt,first", [
    (1, 1, 64, 64, 1, False, BF, 0), (16, 36, 128, 128, 3, False, BF, 1000000), (7, 5, 80, 80, 2, False, HF, 5),
    (9, 3, 96, 32, 3, True, BF, -40), (2100, 2, 128, 64, 1, True, HF, 2 ** 31 - 2101), (3, 2, 256, 256, 1, False, BF, 77),
    (5, 4, 576, 64, 1, True, BF, 4000), (33, 2, 16, 16, 2, False, HF, 100), (2050, 3, 112, 112, 3, False, BF, 2 ** 20),
])
def test_rope(T, H, D, R, axes, inter, dt, first):
    say(f"rope T={T} H={H} D={D} R={R} axes={axes} inter={inter} {dt} first={first}")
    g = gen(T + D)
    x = normal((T, H, D), g, dt)
    inv = (10000.0 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)).float()
    pos = torch.arange(T)[None] * torch.tensor([1, 3, -2])[:axes, None] + first
    pos = pos.clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32)
    sec = [R // 2 - (axes - 1) * (R // 2 // axes)] + [R // 2 // axes] * (axes - 1)
    pair = nv.rope_pair_axis(sec, interleaved=inter, device=DEV) if axes > 1 else None
    want, size = ref.rope(ref.f64(x), pos.numpy(), inv.numpy(), None if pair is None else pair.cpu().numpy(), inter)
    bound = ref.rope_bound(want, size, dt)
    # a slice of a wider projection, as the queries and keys of one are
    wide = torch.full((T, H + 2, D), float("nan"), dtype=dt, device=DEV)
    wide[:, 1:-1] = x.to(DEV)
    args = (pos.to(DEV) if axes > 1 else pos[0].to(DEV), inv.to(DEV), pair, inter)
    got = nv.rope(wide[:, 1:-1], *args)
    assert np.all(np.abs(ref.f64(got) - want) <= bound)
    assert torch.equal(got[..., R:].cpu(), x[..., R:])
    same = nv.rope(wide[:, 1:-1], *args, out=wide[:, 1:-1])   # in place
    assert torch.equal(same, got) and torch.isnan(wide[:, 0]).all() and torch.isnan(wide[:, -1]).all()


def test_rope_cosine_and_sine_of_every_size_of_angle():
    """Unit vectors give the cosine and sine themselves: off by one rounding of the type at any position, both signs."""
    T = 4096
    inv = torch.cat((torch.tensor([1.0, 0.7853981852531433, 0.001, 3.0]), torch.rand(4, generator=gen(1)))).float()
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=gen(2), dtype=torch.int64).to(torch.int32)
    pos[:64] = torch.arange(-32, 32, dtype=torch.int32)
    x = torch.zeros((T, 1, 16), dtype=HF)
    x[..., :8] = 1
    got = ref.f64(nv.rope(x.to(DEV), pos.to(DEV), inv.to(DEV)))
    angle = pos.numpy().astype(np.float64)[:, None] * inv.numpy().astype(np.float64)
    # x0 = 1, x1 = 0: both sides round the same product of position and frequency to 64 bits
    for part, want in ((got[:, 0, :8], np.cos(angle)), (got[:, 0, 8:], np.sin(angle))):
        assert np.all(np.abs(part - want) <= np.abs(want) * ref.u(HF) + 2 * ref.U32 + ref.least(HF))


# ------------------------------------------------------------------ cache --

CACHES = {"same": None, "fp8": torch.float8_e4m3fn, "fp4": torch.uint8}


def make_cache(kind, dt, pages, heads, page, D, permuted=False):
    """A cache filled with a pattern (0x5A bytes) outside what is written; permuted: stored [pages, page, heads, row]."""
    store = CACHES[kind] or dt
    caches = []
    for _ in range(2):
        row = D * 9 // 16 if kind == "fp4" else D
        if permuted and kind != "fp4":
            c = torch.zeros((pages, page, heads, row), dtype=store, device=DEV)
            c.view(torch.uint8).fill_(0x5A)
            c = c.permute(0, 2, 1, 3)
        else:
            c = torch.zeros((pages, heads, page, row), dtype=store, device=DEV)
            c.view(torch.uint8).fill_(0x5A)
        caches.append(c)
    return caches


def check_rows(cache, kind, D, x, scale, slots, page):
    """Written rows hold exactly what the definition gives; all others still hold the pattern."""
    codes, S = ref.raw_rows(cache, kind, D)
    pages = cache.shape[0]
    rows = np.asarray(slots)
    want, wS = ref.stored(x, scale, kind)
    there = (rows >= 0) & (rows < pages * page)
    at, off = rows[there] // page, rows[there] % page
    np.testing.assert_array_equal(codes[at, :, off], want[there])
    if S is not None:
        np.testing.assert_array_equal(S[at, :, off], wS[there])
    written = np.zeros((pages, page), dtype=bool)
    written[at, off] = True
    raw = cache.detach().cpu().contiguous().view(torch.uint8).numpy()
    if kind == "fp4":
        flat = raw.reshape(pages, raw.shape[1], -1)
        c = flat[:, :, :page * D // 2].reshape(pages, -1, page, D // 2)
        s = flat[:, :, page * D // 2:].reshape(pages, -1, page, D // 16)
        raw = np.concatenate((c, s), -1)
    assert np.all(raw.transpose(0, 2, 1, 3)[~written] == 0x5A)


@pytest.mark.parametrize("T,Hk,D,page,dt,permuted", [
    (1, 1, 64, 16, BF, False), (5, 3, 128, 16, HF, True), (37, 2, 96, 8, BF, False), (200, 2, 256, 32, HF, False),
    (19, 4, 32, 8, BF, True), (2500, 1, 128, 48, BF, False),
])
@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("scaled", [False, True])
def test_kv_write_and_read(T, Hk, D, page, dt, permuted, kind, scaled):
    say(f"kv_write T={T} Hk={Hk} D={D} page={page} {dt} {kind} scaled={scaled}")
    if scaled and kind == "same":
        scaled = False
    g = gen(T + D)
    k, v = normal((T, Hk, D), g, dt), normal((T, Hk, D), g, dt, 30.0)
    k[0, 0, :16] = 0                                  # an empty group
    k[T - 1, Hk - 1, 16:32] *= 1e-4                   # group scales that are subnormal or vanish
    v[T // 2, 0, 3] = 60000.0 if dt == HF else 1e30   # saturates
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 4:
        slots[1], slots[3] = -1, pages * page         # padding, and a slot past the cache
    ks = vs = None
    if scaled:
        ks, vs = (0.003 + 0.01 * torch.rand(Hk, generator=g)).to(DEV), (0.1 + torch.rand(Hk, generator=g)).to(DEV)
    kc, vc = make_cache(kind, dt, pages, Hk, page, D, permuted)
    kv = torch.stack((k, v), 1).to(DEV)               # both as slices of one array
    nv.kv_write(kv[:, 0], kv[:, 1], kc, vc, slots.to(DEV), k_scale=ks, v_scale=vs)
    host = (None if ks is None else ks.cpu().numpy()), (None if vs is None else vs.cpu().numpy())
    check_rows(kc, kind, D, ref.f64(k), host[0], slots.numpy(), page)
    check_rows(vc, kind, D, ref.f64(v), host[1], slots.numpy(), page)
    for out_dt in ([dt] if kind == "same" else [BF, HF]):
        rk, rv = nv.kv_read(kc, vc, slots.to(DEV), out_dt, k_scale=ks, v_scale=vs)
        for got, x, s in ((rk, k, host[0]), (rv, v, host[1])):
            want = ref.value(*ref.stored(ref.f64(x), s, kind), s)
            want[(slots.numpy() < 0) | (slots.numpy() >= pages * page)] = 0
            want = torch.from_numpy(ref.f32(want)).float().to(out_dt)
            assert torch.equal(got.cpu(), want)


def test_quantisation_of_every_border():
    """Values at, just below and just above every rounding border of both formats, both signs; infinities saturate, a
    NaN stays one (in its whole group of 16 in the 4-bit format)."""
    marks = np.concatenate([np.arange(0, 8, 0.25), ref.E2M1, [0.0625, 448.0, 464.0, 480.0, 2.0 ** -9, 2.0 ** -10,
                                                             3 * 2.0 ** -10, 2.0 ** -7 * 1.5]])
    vals = []
    for m in marks:
        b = torch.tensor(float(m)).to(BF)
        i = b.view(torch.int16)
        vals += [b, (i + 1).view(BF), (i - 1).clamp(min=0).view(BF)]
    x = torch.stack(vals)
    x = torch.cat((x, -x))
    x = torch.cat((x, torch.zeros(-len(x) % 16, dtype=BF)))
    groups = x.reshape(-1, 16).clone()
    groups[:, 0] = 6.0                     # a group scale of one: the values meet the E2M1 borders themselves
    rows = torch.cat((x.reshape(-1, 16), groups))
    special = torch.zeros((4, 16), dtype=BF)
    special[0, 5], special[1, 5], special[2, 7], special[3, 1] = math.inf, -math.inf, math.nan, 3.0
    special[0, 6] = 2.0
    rows = torch.cat((rows, special))
    rows = torch.cat((rows, torch.zeros((len(rows) % 2, 16), dtype=BF))).reshape(-1, 1, 32)
    T = len(rows)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    for kind in ("fp8", "fp4"):
        kc, vc = make_cache(kind, BF, T // 8 + 1, 1, 8, 32)
        nv.kv_write(rows.to(DEV), rows.to(DEV), kc, vc, slots)
        check_rows(kc, kind, 32, ref.f64(rows), None, np.arange(T), 8)
        back, _ = nv.kv_read(kc, vc, slots, BF)
        want = torch.from_numpy(ref.value(*ref.stored(ref.f64(rows), None, kind), None)).to(BF)
        assert torch.equal(back.cpu().nan_to_num(1234), want.nan_to_num(1234))


@pytest.mark.parametrize("T,Hq,Hk,D,R,axes,inter,page,dt", [
    (1, 8, 1, 128, 128, 1, False, 16, BF), (16, 32, 4, 128, 128, 3, False, 16, BF), (45, 6, 2, 64, 32, 1, True, 16, HF),
    (2100, 4, 2, 128, 64, 1, False, 64, BF), (9, 5, 5, 96, 96, 2, False, 8, HF), (3, 3, 1, 256, 256, 1, True, 4, BF),
])
@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
def test_rope_kv_write(T, Hq, Hk, D, R, axes, inter, page, dt, kind):
    """The fused launch gives what the rotation and the write give one after the other."""
    say(f"rope_kv_write T={T} Hq={Hq} Hk={Hk} D={D} R={R} {kind} {dt}")
    g = gen(T * 7 + D)
    qkv = normal((T, Hq + 2 * Hk, D), g, dt).to(DEV)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    inv = (10000.0 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)).float().to(DEV)
    pos = (torch.arange(T)[None] * torch.arange(1, axes + 1)[:, None] + 12345).to(torch.int32).to(DEV)
    pair = (torch.arange(R // 2) % axes).to(torch.int32).to(DEV) if axes > 1 else None
    pages = T // page + 2
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 2:
        slots[T // 2] = -5
    slots = slots.to(DEV)
    ks = vs = None
    if kind != "same":
        ks, vs = torch.full((Hk,), 0.01, device=DEV), torch.full((Hk,), 0.02, device=DEV)
    kc, vc = make_cache(kind, dt, pages, Hk, page, D)
    k2, v2 = make_cache(kind, dt, pages, Hk, page, D)
    rq = nv.rope(q, pos, inv, pair, inter)
    rk = nv.rope(k, pos, inv, pair, inter)
    nv.kv_write(rk, v, k2, v2, slots, k_scale=ks, v_scale=vs)
    before = qkv.clone()
    got = nv.rope_kv_write(q, k, v, pos, inv, kc, vc, slots, k_scale=ks, v_scale=vs, pair_axis=pair, interleaved=inter)
    assert torch.equal(got, rq) and torch.equal(qkv, before)
    assert torch.equal(kc.view(torch.uint8), k2.view(torch.uint8)) and torch.equal(vc.view(torch.uint8), v2.view(torch.uint8))
    got = nv.rope_kv_write(q, k, v, pos, inv, kc, vc, slots, k_scale=ks, v_scale=vs, pair_axis=pair, interleaved=inter,
                           out=q)   # in place
    assert torch.equal(q, rq) and torch.equal(kc.view(torch.uint8), k2.view(torch.uint8))


# -------------------------------------------------------------- attention --

class Paged:
    """Sequences of given lengths in a paged cache with shuffled pages, written by kv_write; unused rows of used pages
    hold NaN (16-bit, E4M3 and group scales)."""

    def __init__(self, lengths, Hq, Hk, D, page, kind, dt, seed=0, permuted=False, spare=2, sigma=1.0):
        g = gen(seed + D)
        self.Hq, self.Hk, self.D, self.page, self.kind, self.dt = Hq, Hk, D, page, kind, dt
        self.lengths = list(lengths)
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        width = max(need + [1])
        self.table = torch.full((len(lengths), width), -7, dtype=torch.int32)
        self.kc, self.vc = make_cache(kind, dt, pages, Hk, page, D, permuted)
        for c in (self.kc, self.vc):
            c.view(torch.uint8).fill_(0x7F)
            if kind == "same":
                c.fill_(float("nan"))
        n = sum(lengths)
        self.k, self.v = normal((n, Hk, D), g, dt, sigma), normal((n, Hk, D), g, dt)
        slots, done = [], 0
        for b, (ln, m) in enumerate(zip(lengths, need)):
            mine = order[done:done + m]
            self.table[b, :m] = torch.tensor(mine, dtype=torch.int32)
            slots += [mine[t // page] * page + t % page for t in range(ln)]
            done += m
        self.ks = self.vs = None
        if kind != "same":
            self.ks = (0.01 + 0.02 * torch.rand(Hk, generator=g)).to(DEV)
            self.vs = (0.01 + 0.02 * torch.rand(Hk, generator=g)).to(DEV)
        if n:
            nv.kv_write(self.k.to(DEV), self.v.to(DEV), self.kc, self.vc,
                        torch.tensor(slots, dtype=torch.int32, device=DEV), k_scale=self.ks, v_scale=self.vs)
        self.q = normal((len(lengths), Hq, D), g, dt, 1.5)
        host = [None if s is None else s.cpu().numpy() for s in (self.ks, self.vs)]
        self.k64 = ref.value(*ref.stored(ref.f64(self.k), host[0], kind), host[0])
        self.v64 = ref.value(*ref.stored(ref.f64(self.v), host[1], kind), host[1])

    def run(self, window=0, scale=None, ws=None, q=None, table=None, lengths=None, **more):
        ln = torch.tensor(self.lengths if lengths is None else lengths, dtype=torch.int32, device=DEV)
        return nv.paged_attention((self.q if q is None else q).to(DEV), self.kc, self.vc,
                                  (self.table if table is None else table).to(DEV), ln, scale=scale, k_scale=self.ks,
                                  v_scale=self.vs, window=window, return_lse=True, workspace_buf=ws, **more)

    def check(self, got, window=0, scale=None, keep=None):
        out, lse = ref.f64(got[0]), ref.f64(got[1])
        scale = ref.default_scale(self.D) if scale is None else scale
        products = HF if self.kind != "same" or self.dt == HF else BF
        G, first = self.Hq // self.Hk, 0
        for b, n in enumerate(self.lengths):
            lo = max(0, n - window) if window else 0
            idx = np.arange(first + lo, first + n)
            if keep is not None:
                idx = idx[keep[b][lo:n]]
            first += n
            for h in range(self.Hk):
                o, l, bo, bl = ref.attention(ref.f64(self.q[b, h * G:(h + 1) * G]), self.k64[idx, h], self.v64[idx, h],
                                             scale, (products, self.dt))
                mine = out[b, h * G:(h + 1) * G]
                worst = np.max(np.abs(mine - o) - bo)
                assert worst <= 0, (b, h, worst)
                ml = lse[b, h * G:(h + 1) * G]
                if len(idx) == 0:
                    assert np.all(mine == 0) and np.all(np.isneginf(ml))
                else:
                    assert np.all(np.abs(ml - l) <= bl), (b, h, np.max(np.abs(ml - l) - bl))


ATTN = [
    # lengths, Hq, Hk, D, page
    ([1], 1, 1, 64, 16), ([0, 1, 31, 32, 33, 127, 128, 129], 8, 2, 128, 16), ([700, 0, 5], 32, 4, 128, 16),
    ([130, 257], 16, 1, 64, 32), ([65, 300], 40, 2, 128, 8), ([90, 4], 17, 1, 128, 16), ([3000, 17], 4, 4, 128, 64),
    ([77, 260], 6, 2, 256, 4), ([500], 5, 1, 96, 8), ([40, 129], 3, 3, 32, 8), ([150, 64], 8, 2, 192, 16),
    ([9000], 16, 2, 64, 128),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}-{c[3]}-p{c[4]}")
@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("dt", [BF, HF])
def test_attention(case, kind, dt):
    say(f"attention {case} {kind} {dt}")
    lengths, Hq, Hk, D, page = case
    p = Paged(lengths, Hq, Hk, D, page, kind, dt)
    got = p.run()
    p.check(got)
    again = p.run()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("page", [1, 2, 3, 7, 24, 1000])
@pytest.mark.parametrize("D", [16, 80, 112, 144, 256])
def test_attention_pages_of_any_size_and_odd_head_sizes(page, D):
    say(f"attention page={page} D={D}")
    for kind in ("same", "fp8"):
        p = Paged([203, 1, 0, 64], 6, 2, D, page, kind, BF, permuted=True)
        p.check(p.run())


@pytest.mark.parametrize("kind", ["same", "fp4"])
def test_attention_window(kind):
    p = Paged([700, 50, 0, 129], 8, 2, 128, 16, kind, BF)
    for window in (1, 33, 128, 699, 5000):
        say(f"window {window}")
        p.check(p.run(window=window), window=window)


@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("most,D", [(900, 64), (150, 128)])
def test_attention_many_ragged_sequences(most, D, kind):
    """More pairs than workgroups: a stretch ends one pair, holds whole ones and begins another."""
    say(f"130 sequences of up to {most}, D={D}, {kind}")
    lengths = torch.randint(0, most + 1, (130,), generator=gen(most)).tolist()
    p = Paged(lengths, 12, 4, D, 16, kind, BF)
    p.check(p.run())


@pytest.mark.parametrize("B", [2048, 2049, 2300])
def test_attention_more_sequences_than_are_counted(B):
    say(f"{B} sequences")
    lengths = torch.randint(0, 200, (B,), generator=gen(B)).tolist()
    p = Paged(lengths, 2, 1, 64, 16, "fp4", HF)
    p.check(p.run())


@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("lengths,Hq,Hk", [([60000] + list(range(7)), 1, 1), ([3, 20000, 0], 16, 1), ([5, 5, 30000], 34, 2)])
def test_attention_one_long_sequence_among_short_ones(lengths, Hq, Hk, kind):
    """The long pair's partial results are more than a join's one round."""
    say(f"{lengths} {Hq}x{Hk} {kind}")
    p = Paged(lengths, Hq, Hk, 64, 32, kind, BF)
    p.check(p.run())


@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("lengths", [[512], [513], [640], [641], [2016], [2048], [2049], [2176], [700, 512, 1000, 31], [4096]])
def test_attention_lengths_around_the_rule_of_the_split(lengths, kind):
    say(f"{lengths} {kind}")
    p = Paged(lengths, 8, 2, 128, 16, kind, HF)
    p.check(p.run())
    room = torch.full((len(lengths), 5000), -1, dtype=torch.int32)   # a table for much longer sequences
    room[:, :p.table.shape[1]] = p.table
    p.check(p.run(table=room))


@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_pages_of_48_in_a_permuted_cache(D, kind):
    p = Paged([500, 47, 48, 49, 0, 1300], 10, 2, D, 48, kind, BF, permuted=True)
    for window in (0, 50, 400):
        say(f"pages of 48, D={D}, {kind}, window {window}")
        p.check(p.run(window=window), window=window)


@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
def test_attention_scales_of_any_sign(kind):
    p = Paged([700, 1, 33], 8, 2, 128, 16, kind, BF)
    for scale in (-0.07, 0.0, 0.5):
        say(f"softmax scale {scale}, {kind}")
        p.check(p.run(scale=scale), scale=scale)


def test_attention_long_split_and_a_reused_workspace():
    """One workspace through calls of different sizes (the partial results of one lie where another's would start)."""
    p = Paged([40000], 8, 2, 128, 64, "fp8", BF)
    small = [Paged([n] * 40, 8, 8, 64, 16, "same", HF, seed=n) for n in (300, 1000)]
    need = max(nv.paged_attention_workspace_bytes(1, 8, 2, 128, 40000 + 64),
               *(nv.paged_attention_workspace_bytes(40, 8, 8, 64, 1024) for _ in (0,)))
    ws = nv.workspace(need, DEV)
    first = p.run(ws=ws)
    p.check(first)
    for s in small:
        s.check(s.run(ws=ws))
    again = p.run(ws=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
def test_attention_masked_contents_do_not_reach_the_result(kind):
    """Pages outside the cache are left out, a sequence whose pages all are is empty, lengths are clamped to the table,
    negative ones are empty."""
    page = 16
    p = Paged([200, 100, 64], 8, 2, 128, page, kind, BF)
    good = p.run()
    table = p.table.clone()
    table[0, 2], table[0, 5], table[1, :] = -1, p.kc.shape[0], 2 ** 30
    got = p.run(table=table)
    t = np.arange(200)
    keep = [~np.isin(t // page, (2, 5)), np.zeros(100, dtype=bool), np.ones(64, dtype=bool)]
    p.check(got, keep=keep)
    assert torch.equal(got[0][2], good[0][2]) and torch.equal(got[1][2], good[1][2])
    clamped = p.run(lengths=[200, -3, 64])
    assert torch.equal(clamped[0][0], good[0][0]) and torch.all(clamped[0][1] == 0) and torch.all(torch.isneginf(clamped[1][1]))
    # a length past the table's width ends with the table
    narrow = p.table[:1, :4].contiguous()
    one = nv.paged_attention(p.q[:1].to(DEV), p.kc, p.vc, narrow.to(DEV), torch.tensor([10 ** 6], dtype=torch.int32, device=DEV),
                             k_scale=p.ks, v_scale=p.vs)
    two = nv.paged_attention(p.q[:1].to(DEV), p.kc, p.vc, narrow.to(DEV), torch.tensor([64], dtype=torch.int32, device=DEV),
                             k_scale=p.ks, v_scale=p.vs)
    assert torch.equal(one, two)


def test_attention_infinite_and_large_values():
    """Scores of the type's lowest and largest values, minus infinities (weight 0; all of them: an empty row) and a NaN
    in a key that is used (its head's result is NaN, the others' are not)."""
    D, page, n = 64, 16, 70
    kc, vc = nv.kv_cache(8, 2, page, D, BF, DEV)
    g = gen(3)
    k, v = normal((n, 2, D), g, BF), normal((n, 2, D), g, BF)
    k[:, :, 0] = 0
    q = torch.zeros((1, 4, D), dtype=BF)
    q[..., 1:] = normal((1, 4, D - 1), g, BF)
    q[..., 0] = 1.0
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    lengths = torch.tensor([n], dtype=torch.int32, device=DEV)

    def run(kk):
        nv.kv_write(kk.to(DEV), v.to(DEV), kc, vc, slots)
        return nv.paged_attention(q.to(DEV), kc, vc, table, lengths, return_lse=True)

    def want(kk):
        return [ref.attention(ref.f64(q[0, 2 * h:2 * h + 2]), ref.f64(kk[:, h]), ref.f64(v[:, h]), 0.125, (BF, BF))
                for h in range(2)]

    low = k.clone()
    low[:35, :, 0] = torch.finfo(BF).min     # weight 0 beside the rest
    out, lse = run(low)
    rest = [ref.attention(ref.f64(q[0, 2 * h:2 * h + 2]), ref.f64(low[35:, h]), ref.f64(v[35:, h]), 0.125, (BF, BF)) for h in range(2)]
    for h in range(2):
        assert np.all(np.abs(ref.f64(out[0, 2 * h:2 * h + 2]) - rest[h][0]) <= rest[h][2])
    minus = k.clone()
    minus[35:, :, 0] = -math.inf
    out, lse = run(minus)
    for h in range(2):
        o, l, bo, bl = ref.attention(ref.f64(q[0, 2 * h:2 * h + 2]), ref.f64(minus[:35, h]), ref.f64(v[:35, h]), 0.125, (BF, BF))
        assert np.all(np.abs(ref.f64(out[0, 2 * h:2 * h + 2]) - o) <= bo)
        assert np.all(np.abs(ref.f64(lse[0, 2 * h:2 * h + 2]) - l) <= bl)
    none = k.clone()
    none[:, 0, 0] = -math.inf
    out, lse = run(none)
    assert torch.all(out[0, :2] == 0) and torch.all(torch.isneginf(lse[0, :2]))
    assert torch.isfinite(out[0, 2:]).all()
    nan = k.clone()
    nan[69, 1, 5] = math.nan
    out, lse = run(nan)
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all() and torch.isfinite(out[0, :2]).all()
    big = k.clone()
    big[:, :, 0] = 1000.0                    # large equal scores: the running maximum keeps the weights finite
    out, lse = run(big)
    for h, (o, l, bo, bl) in enumerate(want(big)):
        assert np.all(np.abs(ref.f64(out[0, 2 * h:2 * h + 2]) - o) <= bo)
        assert np.all(np.abs(ref.f64(lse[0, 2 * h:2 * h + 2]) - l) <= bl)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_attention_queries_of_any_size_on_a_quantised_cache(kind):
    """Queries far outside fp16's range (bf16 keeps 8 exponent bits), and one of zeros."""
    p = Paged([150, 90, 40], 4, 2, 128, 16, kind, BF)
    p.q[0] *= 2.0 ** 30
    p.q[1] *= 2.0 ** -40
    p.q[2] = 0
    p.check(p.run(scale=2.0 ** -33), scale=2.0 ** -33)


def test_cache_offsets_past_32_bits():
    """Rows beyond 4 GB in both sides of a cache: written, read back and attended to."""
    page, Hk, D = 64, 8, 128
    pages = (5 << 30) // (page * Hk * D * 2)
    kc = torch.empty((pages, Hk, page, D), dtype=BF, device=DEV)
    vc = torch.empty((pages, Hk, page, D), dtype=BF, device=DEV)
    g = gen(11)
    n = 150
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    slots = torch.tensor([int(table[0, t // page]) * page + t % page for t in range(n)], dtype=torch.int32, device=DEV)
    k, v, q = normal((n, Hk, D), g, BF), normal((n, Hk, D), g, BF), normal((1, Hk, D), g, BF)
    nv.kv_write(k.to(DEV), v.to(DEV), kc, vc, slots)
    bk, bv = nv.kv_read(kc, vc, slots)
    assert torch.equal(bk.cpu(), k) and torch.equal(bv.cpu(), v)
    assert torch.equal(kc[pages - 1, :, 5].cpu(), k[5]) and torch.equal(vc[pages - 2, :, n - 1 - 128].cpu(), v[n - 1])
    out = nv.paged_attention(q.to(DEV), kc, vc, table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV))
    for h in range(Hk):
        o, _, bo, _ = ref.attention(ref.f64(q[0, h:h + 1]), ref.f64(k[:, h]), ref.f64(v[:, h]), ref.default_scale(D), (BF, BF))
        assert np.all(np.abs(ref.f64(out[0, h:h + 1]) - o) <= bo)


def test_strided_queries_and_outputs_and_another_stream():
    p = Paged([300, 45], 8, 2, 128, 16, "same", BF)
    want = p.run()
    wide = torch.full((2, 10, 3, 128), float("nan"), dtype=BF, device=DEV)
    q = wide[:, 1:9, 1]
    q.copy_(p.q.to(DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = nv.paged_attention(q, p.kc, p.vc, p.table.to(DEV), torch.tensor(p.lengths, dtype=torch.int32, device=DEV), out=q)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    assert torch.isnan(wide[:, 0]).all() and torch.isnan(wide[:, :, 0]).all() and torch.isnan(wide[:, 9]).all()


def test_empty_calls():
    kc, vc = nv.kv_cache(2, 2, 16, 64, BF, DEV)
    z = torch.empty((0, 2, 64), dtype=BF, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    inv = torch.ones(32, device=DEV)
    assert nv.rope(z, none, inv).shape == (0, 2, 64)
    assert nv.rope_kv_write(z, z, z, none, inv, kc, vc, none).shape == (0, 2, 64)
    assert nv.kv_read(kc, vc, none)[0].shape == (0, 2, 64)
    assert nv.rms_norm(torch.empty((0, 64), dtype=BF, device=DEV), torch.ones(64, dtype=BF, device=DEV))[0].shape == (0, 64)
    assert nv.paged_attention(z, kc, vc, torch.empty((0, 1), dtype=torch.int32, device=DEV), none).shape == (0, 2, 64)
    q = torch.ones((2, 2, 64), dtype=BF, device=DEV)
    out, lse = nv.paged_attention(q, kc, vc, torch.empty((2, 0), dtype=torch.int32, device=DEV),
                                  torch.tensor([5, 0], dtype=torch.int32, device=DEV), return_lse=True)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_binding_refusals():
    """Wrong shapes, types, devices and caches raise before anything runs; a refusal by the library is an Nvfp4Error."""
    x, w = torch.ones((2, 64), dtype=BF, device=DEV), torch.ones(64, dtype=BF, device=DEV)
    bad = [
        (lambda: nv.rms_norm(x, w[:32]), "weight"), (lambda: nv.rms_norm(x, w.half()), "weight"),
        (lambda: nv.rms_norm(x, w.cpu()), "weight is on cpu"), (lambda: nv.rms_norm(x.t(), w), "unit stride"),
        (lambda: nv.rms_norm(x, w, residual=x[:1]), "residual"), (lambda: nv.rms_norm(x[0], w), "2 dims"),
        (lambda: nv.rms_norm(x, w, residual_out=x), "needs a residual"), (lambda: nv.rms_norm(x, w, out=x.half()), "out"),
        (lambda: nv.rms_norm_fp8(x, w, scales=w), "scales"),
    ]
    h = torch.ones((5, 4, 64), dtype=BF, device=DEV)
    inv, pos = torch.ones(32, device=DEV), torch.zeros((3, 5), dtype=torch.int32, device=DEV)
    axis = torch.zeros(32, dtype=torch.int32, device=DEV)
    bad += [
        (lambda: nv.rope(h, pos, inv), "need pair_axis"), (lambda: nv.rope(h, pos[:, :4], inv, axis), "positions"),
        (lambda: nv.rope(h, pos.long(), inv, axis), "positions"), (lambda: nv.rope(h, pos[0], inv.double()), "inv_freq"),
        (lambda: nv.rope(h, pos, inv, axis[:31]), "pair_axis"), (lambda: nv.rope(h[0], pos, inv, axis), "3 dims"),
        (lambda: nv.rope(h, pos[0], inv[None]), "1-d"),
    ]
    one = torch.ones(2, device=DEV)
    bf, f8, f4 = (nv.kv_cache(3, 2, 16, 64, d, DEV) for d in (BF, torch.float8_e4m3fn, torch.uint8))
    k, slots = h[:, :2], torch.zeros(5, dtype=torch.int32, device=DEV)
    odd = torch.zeros((2, 2, 16, 45), dtype=torch.uint8, device=DEV)

    def write(kc, vc, ks=None, vs=None, k=k, v=k, slots=slots):
        return lambda: nv.kv_write(k, v, kc, vc, slots, k_scale=ks, v_scale=vs)

    bad += [
        (write(bf[0], f8[0]), "one dtype"), (write(bf[0], bf[1][:2]), "one shape"), (write(*bf, one), "takes no k_scale"),
        (write(*f8, None, one[:1]), "v_scale"), (write(*f8, one.half()), "k_scale"),
        (write(*(f8[0].transpose(2, 3),) * 2), "contiguous rows"), (write(*(f4[0].transpose(1, 2),) * 2), "contiguous blocks"),
        (write(*(f4[0][..., :35],) * 2), "contiguous blocks"), (write(*(bf[0].float(),) * 2), "must be a bf16"),
        (write(odd, odd), "multiple of 32"), (write(*bf, k=k.half(), v=k.half()), "activations"), (write(*bf, v=h), "v must be"),
        (write(*bf, slots=slots.long()), "slots"), (write(bf[0].cpu(), bf[1]), "caches are on"),
        (lambda: nv.kv_read(*bf, slots[None]), "1-d"), (lambda: nv.kv_read(*bf, slots, HF), "activations"),
        (lambda: nv.kv_read(*bf, slots, out=(h, h)), "out"),
    ]
    q, table, n = h, torch.zeros((5, 2), dtype=torch.int32, device=DEV), slots
    bad += [
        (lambda: nv.paged_attention(q[..., :32].contiguous(), *bf, table, n), "columns a head"),
        (lambda: nv.paged_attention(q[:, :3], *bf, table, n), "multiple"),
        (lambda: nv.paged_attention(q, *bf, table[:4], n), "page_table"), (lambda: nv.paged_attention(q, *bf, table.long(), n), "page_table"),
        (lambda: nv.paged_attention(q, *bf, table, n[:4]), "lengths"),
        (lambda: nv.paged_attention(q, *bf, table, n, workspace_buf=torch.zeros(8)), "workspace_buf"),
    ]
    for call, needle in bad:
        with pytest.raises(ValueError, match=needle):
            call()
    with pytest.raises(nv.Nvfp4Error, match="window"):
        nv.paged_attention(q, *bf, table, n, window=-1)
    wide = torch.zeros((5, 20), dtype=torch.int32, device=DEV)
    with pytest.raises(nv.Nvfp4Error, match="BUFFER_TOO_SMALL.*workspace"):
        nv.paged_attention(q, *bf, wide, n, workspace_buf=torch.zeros(8, device=DEV))
    with pytest.raises(nv.Nvfp4Error, match="rotary"):
        nv.rope(h, pos[0], inv[:4])
    with pytest.raises(nv.Nvfp4Error, match="eps"):
        nv.rms_norm(x, w, -1.0)
    with pytest.raises(TypeError):
        nv.rms_norm(x, w, "eps")


def test_a_captured_step_replays():
    """Norm, rotation with the cache write and attention in one graph: replays with new inputs, lengths and slots, with
    eager work in between, give what the eager calls give."""
    B, Hq, Hk, D, page, N = 4, 8, 2, 128, 16, 1024
    g = gen(9)
    p = Paged([100, 257, 0, 31], Hq, Hk, D, page, "fp4", BF, spare=12)
    inv = (10000.0 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)).float().to(DEV)
    x, r, w = (normal(s, g, BF).to(DEV) for s in ((B, N), (B, N), (N,)))
    qkv = normal((B, Hq + 2 * Hk, D), g, BF).to(DEV)
    table = torch.full((B, 20), -1, dtype=torch.int32)
    table[:, :p.table.shape[1]] = p.table
    free = sorted(set(range(p.kc.shape[0])) - set(p.table.flatten().tolist()))
    for b in range(B):
        used = -(-p.lengths[b] // page)
        table[b, used:used + 2] = torch.tensor(free[2 * b:2 * b + 2], dtype=torch.int32)
    table = table.to(DEV)
    lengths = torch.tensor(p.lengths, dtype=torch.int32, device=DEV)
    ws = nv.workspace(nv.paged_attention_workspace_bytes(B, Hq, Hk, D, 20 * page), DEV)

    def step(kc, vc, pos, slots, n):
        y, h = nv.rms_norm(x, w, residual=r)
        q = nv.rope_kv_write(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], pos, inv, kc, vc, slots, k_scale=p.ks,
                             v_scale=p.vs)
        return (y, h) + nv.paged_attention(q, kc, vc, table, n, k_scale=p.ks, v_scale=p.vs, return_lse=True,
                                           workspace_buf=ws)

    pos, slots, n = lengths.clone(), torch.zeros_like(lengths), lengths.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        slots.fill_(-1)
        step(p.kc, p.vc, pos, slots, n)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(p.kc, p.vc, pos, slots, n)
    for i in range(5):
        say(f"replay {i}")
        now = lengths + i
        pos.copy_(now)
        slots.copy_(table.gather(1, (now // page).long()[:, None])[:, 0] * page + now % page)
        n.copy_(now + 1)
        qkv.copy_(normal(tuple(qkv.shape), g, BF))
        x.copy_(normal((B, N), g, BF))
        k2, v2 = p.kc.clone(), p.vc.clone()
        want = [t.clone() for t in step(k2, v2, pos, slots, n)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.kc, k2) and torch.equal(p.vc, v2)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
