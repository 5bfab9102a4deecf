"""The attention half of a decoder layer on the CPU: the C ABI's refusals (each before any launch: the pointers here are
fake), the binding's checks, workspace sizes, and the plain forms the GPU tests compare with."""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import attention_ref as ref
import weight_only_fp4_amd as nv

OK, INVALID, ALIGN, SMALL = 0, 1, 2, 3
A = 1 << 20   # a fake, aligned address; never dereferenced


# the C structs nvfp4_kv_cache and nvfp4_rope
KV_STRUCT, ROPE_STRUCT = struct.Struct("PPPP7q4i"), struct.Struct("PPPq4i")


class Calls:
    """The library's calls with their C signatures."""

    def __init__(self):
        L, P, I64, I = nv.lib(), ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        F, DESC = ctypes.c_float, ctypes.c_char_p
        for name, args in dict(
                nvfp4_rms_norm=[P, I64, P, I64, P, F, P, I64, P, P, I64, I64, I64, I, P],
                nvfp4_rope_apply=[DESC, P, I64, I64, P, I64, I64, I64, I64, I64, I, P],
                nvfp4_kv_append=[DESC, DESC, P, I64, I64, P, I64, I64, I64, P, I64, I64, P, I64, I64, P, I64, I, P],
                nvfp4_kv_read=[DESC, P, P, I64, I64, P, I64, I64, I64, I, P],
                nvfp4_paged_attention=[DESC, P, I64, I64, P, I64, I64, P, I64, I64, F, I64, P, I64, I64, P, P, I64, I, P],
        ).items():
            f = ctypes.CFUNCTYPE(I, *args)((name, L))
            setattr(self, name, f)


@pytest.fixture(scope="module")
def L():
    return Calls()


def last():
    return nv.lib().nvfp4_last_error().decode()


# ------------------------------------------------------------------ the ABI --

def cache(**kw):
    a = dict(k=A, v=A, ks=0, vs=0, kst=(65536, 4096, 256), vst=(65536, 4096, 256), pages=10, page=16, heads=4, D=128, fmt=0)
    a.update(kw)
    return KV_STRUCT.pack(a["k"], a["v"], a["ks"], a["vs"], *a["kst"], *a["vst"], a["pages"], a["page"], a["heads"],
                              a["D"], a["fmt"])


def rope(**kw):
    a = dict(inv=A, pos=A, pair=0, ld=8, axes=1, R=128, nb=0)
    a.update(kw)
    return ROPE_STRUCT.pack(a["inv"], a["pos"], a["pair"], a["ld"], a["axes"], a["R"], a["nb"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "T ="), (dict(N=0), INVALID, "N ="), (dict(ld_x=10), INVALID, "leading dimension"),
    (dict(ld_y=10), INVALID, "leading dimension"), (dict(ld_r=10), INVALID, "leading dimension"),
    (dict(h=A, ld_h=10), INVALID, "leading dimension"), (dict(r=None, h=A), INVALID, "residual"),
    (dict(eps=-1.0), INVALID, "eps"), (dict(eps=math.nan), INVALID, "eps"), (dict(eps=math.inf), INVALID, "eps"),
    (dict(x=None), INVALID, "NULL"), (dict(w=None), INVALID, "NULL"), (dict(y=None), INVALID, "NULL"),
    (dict(x=A + 1), ALIGN, "misaligned"), (dict(y=A + 1), ALIGN, "misaligned"), (dict(scales=A + 2), ALIGN, "misaligned"),
    (dict(w=A + 1), ALIGN, "misaligned"), (dict(T=0), OK, ""), (dict(T=0, x=None, y=None, r=None), OK, ""),
])
def test_norm_refusals(L, kw, status, needle):
    a = dict(x=A, ld_x=64, r=A, ld_r=64, w=A, eps=1e-6, y=A, ld_y=64, scales=None, h=None, ld_h=64, T=4, N=64)
    a.update(kw)
    st = L.nvfp4_rms_norm(a["x"], a["ld_x"], a["r"], a["ld_r"], a["w"], a["eps"], a["y"], a["ld_y"], a["scales"],
                                 a["h"], a["ld_h"], a["T"], a["N"], 0, None)
    assert st == status and needle in last()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "T ="), (dict(H=-1), INVALID, "H ="), (dict(D=24), INVALID, "D ="), (dict(D=1040), INVALID, "D ="),
    (dict(x=None), INVALID, "x is NULL"), (dict(o=None), INVALID, "out is NULL"), (dict(x=A + 2), ALIGN, "16-byte"),
    (dict(x_h=100), ALIGN, "16-byte"), (dict(o_t=1028), ALIGN, "16-byte"), (dict(x_t=-8), INVALID, "out of range"),
    (dict(rope=None), INVALID, "rope is NULL"), (dict(rope=rope(inv=0)), INVALID, "inv_freq"),
    (dict(rope=rope(pos=0)), INVALID, "positions"), (dict(rope=rope(R=0)), INVALID, "rotary"),
    (dict(rope=rope(R=24)), INVALID, "rotary"), (dict(rope=rope(R=144)), INVALID, "rotary"),
    (dict(D=512, rope=rope(R=272)), INVALID, "rotary"), (dict(rope=rope(axes=2)), INVALID, "pair_axis"),
    (dict(rope=rope(axes=17, pair=A)), INVALID, "axes"), (dict(rope=rope(axes=0)), INVALID, "axes"),
    (dict(rope=rope(ld=3)), INVALID, "ld_pos"), (dict(rope=rope(inv=A + 2)), ALIGN, "4-byte"),
    (dict(T=0), OK, ""), (dict(H=0), OK, ""), (dict(T=1 << 24, rope=rope(ld=1 << 24)), INVALID, "too many"),
])
def test_rope_refusals(L, kw, status, needle):
    a = dict(rope=rope(), x=A, x_t=1024, x_h=128, o=A, o_t=1024, o_h=128, T=4, H=8, D=128)
    a.update(kw)
    st = L.nvfp4_rope_apply(a["rope"], a["x"], a["x_t"], a["x_h"], a["o"], a["o_t"], a["o_h"], a["T"], a["H"], a["D"],
                                   0, None)
    assert st == status and needle in last()


BAD_CACHES = [
    (None, INVALID, "cache is NULL"), (cache(fmt=3), INVALID, "format"), (cache(fmt=-1), INVALID, "format"),
    (cache(D=24), INVALID, "head_dim"), (cache(D=272), INVALID, "head_dim"), (cache(D=0), INVALID, "head_dim"),
    (cache(D=80, fmt=2), INVALID, "multiple of 32"), (cache(heads=0), INVALID, "heads"), (cache(pages=0), INVALID, "pages"),
    (cache(page=0), INVALID, "page"), (cache(pages=1 << 28, page=16), INVALID, "2^31"),
    (cache(fmt=2, page=1), INVALID, "NVFP4 block"), (cache(ks=A), INVALID, "scales"), (cache(fmt=1, vs=A + 2), ALIGN, "scales"),
    (cache(k=0), INVALID, "k is NULL"), (cache(v=0), INVALID, "v is NULL"), (cache(k=A + 8), ALIGN, "16-byte"),
    (cache(kst=(65536, 4096, 248)), ALIGN, "stride 2"), (cache(vst=(65540, 4096, 256)), ALIGN, "stride 0"),
    (cache(kst=(-16, 4096, 256)), INVALID, "stride 0"), (cache(pages=1 << 20, kst=(1 << 17, 4096, 256)), INVALID, "64 GB"),
]


@pytest.mark.parametrize("desc,status,needle", BAD_CACHES)
def test_cache_refusals(L, desc, status, needle):
    assert L.nvfp4_kv_append(desc, None, None, 0, 0, None, 0, 0, 0, A, 512, 128, A, 512, 128, A, 4, 0, None) == status
    assert needle in last()
    assert L.nvfp4_kv_read(desc, A, A, 512, 128, A, 512, 128, 4, 0, None) == status and needle in last()
    assert L.nvfp4_paged_attention(desc, A, 1024, 128, A, 8, 8, A, 2, 8, 0.1, 0, A, 1024, 128, None, A, 1 << 30, 0,
                                   None) == status and needle in last()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(Hq=-1), INVALID, "Hq"), (dict(Hq=4), INVALID, "need rope"), (dict(T=-1), INVALID, "T ="),
    (dict(k=None), INVALID, "k is NULL"), (dict(v=A + 2), ALIGN, "v rows"), (dict(slots=None), INVALID, "slots"),
    (dict(slots=A + 2), ALIGN, "slots"), (dict(k_t=12), ALIGN, "k rows"), (dict(rope=rope(), Hq=4, q=None), INVALID, "q is NULL"),
    (dict(rope=rope(), Hq=4, qo=None), INVALID, "q_out is NULL"), (dict(rope=rope(R=144), Hq=4), INVALID, "rotary"),
    (dict(desc=cache(fmt=2), rope=rope(R=48)), INVALID, "multiple of 32"), (dict(T=0), OK, ""),
    (dict(T=0, rope=rope(pos=0), Hq=4, slots=None), OK, ""),
])
def test_append_refusals(L, kw, status, needle):
    a = dict(desc=cache(), rope=None, q=A, qo=A, Hq=0, k=A, k_t=512, v=A, slots=A, T=4)
    a.update(kw)
    st = L.nvfp4_kv_append(a["desc"], a["rope"], a["q"], 1024, 128, a["qo"], 1024, 128, a["Hq"], a["k"], a["k_t"], 128,
                                  a["v"], 512, 128, a["slots"], a["T"], 0, None)
    assert st == status and needle in last()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=-1), INVALID, "B ="), (dict(B=65536), INVALID, "B ="), (dict(Hq=6), INVALID, "multiple"),
    (dict(Hq=0), INVALID, "multiple"), (dict(pages=-1), INVALID, "max_pages"), (dict(ld=4), INVALID, "ld_table"),
    (dict(pages=1 << 27, ld=1 << 27), INVALID, "2^30"), (dict(scale=math.inf), INVALID, "softmax_scale"),
    (dict(scale=math.nan), INVALID, "softmax_scale"), (dict(window=-1), INVALID, "window"), (dict(q=None), INVALID, "q is NULL"),
    (dict(out=None), INVALID, "out is NULL"), (dict(table=None), INVALID, "page_table"), (dict(lengths=None), INVALID, "lengths"),
    (dict(q=A + 2), ALIGN, "q rows"), (dict(lse=A + 2), ALIGN, "4-byte"), (dict(wsb=100), SMALL, "workspace"),
    (dict(ws=None), SMALL, "workspace"), (dict(ws=A + 16), ALIGN, "256-byte"), (dict(B=0), OK, ""),
    (dict(B=0, q=None, table=None, ws=None), OK, ""), (dict(B=65535, Hq=1 << 20), INVALID, "too many"),
])
def test_attention_refusals(L, kw, status, needle):
    a = dict(q=A, table=A, ld=100, pages=100, lengths=A, B=2, Hq=8, scale=0.1, window=0, out=A, lse=A, ws=A, wsb=1 << 30)
    a.update(kw)
    st = L.nvfp4_paged_attention(cache(), a["q"], 1024, 128, a["table"], a["ld"], a["pages"], a["lengths"], a["B"],
                                        a["Hq"], a["scale"], a["window"], a["out"], 1024, 128, a["lse"], a["ws"], a["wsb"], 0,
                                        None)
    assert st == status and needle in last()


def test_workspace_sizes():
    f = nv.paged_attention_workspace_bytes
    assert f(1, 8, 2, 128, 128) == 0 and f(0, 8, 2, 128, 10000) == 0      # one chunk, or nothing: no partial results
    assert f(4000, 8, 2, 128, 100000) == 0                                # enough sequences: not split
    assert f(1, 8, 2, 128, 100000) > 0
    for bad in ((-1, 8, 2, 128, 10), (1, 7, 2, 128, 10), (1, 8, 2, 24, 10), (1, 8, 2, 128, 1 << 30)):
        with pytest.raises(ValueError):
            f(*bad)


# -------------------------------------------------------------- the binding --

def test_binding_checks():
    """Tensors that are not on the GPU or of other types raise ValueError before the library is called."""
    x = torch.ones((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        nv.rms_norm(x, x[0])
    with pytest.raises(ValueError, match="bf16 or fp16"):
        nv.rms_norm(x.float(), x[0])
    with pytest.raises(ValueError, match="bf16 or fp16"):
        nv.rms_norm_fp8("x", x[0])
    with pytest.raises(ValueError, match="on the GPU"):
        nv.rope(torch.ones((2, 2, 64), dtype=torch.float16), None, None)
    with pytest.raises(ValueError, match="on the GPU"):
        nv.kv_read(x, x, x)
    with pytest.raises(ValueError, match="torch tensor"):
        nv.kv_read(None, x, x)
    with pytest.raises(ValueError, match="on the GPU"):
        nv.kv_write(*[x.view(2, 1, 64)] * 2, x, x, x)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        nv.rope_kv_write(None, x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        nv.kv_read(x, x, x, torch.float32)
    with pytest.raises(ValueError, match="on the GPU"):
        nv.paged_attention(x.view(2, 1, 64), x, x, x, x)
    with pytest.raises(ValueError, match="cache dtype"):
        nv.kv_cache(2, 2, 16, 64, torch.float32, "cpu")
    assert nv.kv_cache(3, 2, 16, 64, torch.uint8, "cpu")[0].shape == (3, 2, 16, 36)


def test_pair_axis_sections():
    assert nv.rope_pair_axis([2, 3, 1], device="cpu").tolist() == [0, 0, 1, 1, 1, 2]
    assert nv.rope_pair_axis([4, 2, 2], interleaved=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 2, 0, 0]


# ---------------------------------------------------------- the plain forms --

def test_small_float_rounding():
    """e4m3 against torch's conversion over the format's range; e2m1 at its borders (ties to the even code)."""
    x = torch.cat((torch.linspace(-448, 448, 20001), torch.logspace(-4, 2.65, 5000), torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0])))
    want = x.to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.e4m3(x.double().numpy()), want)
    b = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    np.testing.assert_array_equal(ref.e2m1(b), [0, 1, 1, 2, 2, 4, 4, 6])
    np.testing.assert_array_equal(ref.e2m1(-b - 1e-9), [-0.5, -1, -1.5, -2, -3, -4, -6, -6])
    np.testing.assert_array_equal(ref.e2m1(b - 1e-9), [0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.mark.parametrize("plant", ["none", "one token more", "one token less", "no scale", "value of a neighbour"])
def test_the_attention_bound_sees_a_mistake(plant):
    """A plain form with a mistake planted in it leaves the bound the GPU tests use; rounding the weights does not."""
    g = np.random.default_rng(0)
    D, n = 64, 40
    q, k, v = g.normal(size=(2, D)), g.normal(size=(n + 1, D)), g.normal(size=(n + 1, D))
    bf = torch.bfloat16
    o, l, bo, bl = ref.attention(q, k[:n], v[:n], 0.125, (bf, bf))
    if plant == "none":
        s = q @ k[:n].T * 0.125
        w = np.exp(s - s.max(1, keepdims=True))
        wr = torch.from_numpy(w).to(bf).double().numpy()
        got = torch.from_numpy(wr @ v[:n] / w.sum(1, keepdims=True)).to(bf).double().numpy()
        assert np.all(np.abs(got - o) <= bo)
        return
    kk, vv, scale = k[:n], v[:n].copy(), 0.125
    if plant == "one token more":
        kk, vv = k, v
    elif plant == "one token less":
        kk, vv = k[:n - 1], v[:n - 1]
    elif plant == "no scale":
        scale = 1.0
    else:
        vv[[7, 8]] = vv[[8, 7]]
    got = ref.attention(q, kk, vv, scale, (bf, bf))[0]
    assert not np.all(np.abs(got - o) <= bo)


def test_rope_forms_agree():
    """Halves and neighbours are one rotation with the columns in another order; position 0 turns nothing."""
    g = np.random.default_rng(1)
    x, inv = g.normal(size=(5, 2, 32)), 1.0 / (1 + np.arange(16.0))
    pos = np.array([[0, 1, 5, 9, 100]])
    y, _ = ref.rope(x, pos, inv, None, False)
    order = np.arange(32).reshape(2, 16).T.reshape(-1)
    z, _ = ref.rope(x[..., order], pos, inv, None, True)
    np.testing.assert_allclose(z, y[..., order], rtol=0, atol=1e-15)
    np.testing.assert_array_equal(y[0], x[0])


def test_descriptor_layouts():
    """The packed descriptors have the C structs' sizes (pointers and 64-bit fields first, no padding)."""
    assert KV_STRUCT.size == 4 * ctypes.sizeof(ctypes.c_void_p) + 7 * 8 + 4 * 4
    assert ROPE_STRUCT.size == 3 * ctypes.sizeof(ctypes.c_void_p) + 8 + 4 * 4
