"""What a decode step runs around its layers, on the CPU: the C ABI's refusals (each before any launch: the pointers here
are fake), workspace sizes, the binding's checks, and the plain forms against hand cases."""
import ctypes

import numpy as np
import pytest
import torch

import step_ref as ref
import weight_only_fp4_amd as nv

OK, INVALID, ALIGN, SMALL = 0, 1, 2, 3
A = 1 << 20   # a fake, aligned address; never dereferenced


class Calls:
    """The library's calls with their C signatures."""

    def __init__(self):
        L, P, I64, I = nv.lib(), ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        for name, args in dict(
                nvfp4_kv_plan=[P, P, I64, P, I64, I64, I64, P, I64, P, I64, P, P, P, P, P, P, P, I64, P],
                nvfp4_lora_add=[P, I64, P, I64, I64, P, I64, I64, P, P, P, I64, P, I64, I64, I64, I64, I64, I64, P, I64, I, P],
                nvfp4_moe_layer=[P, I64, P, P, I64, I64, P, P, P, P, P, P, I, I, P, I64, I64, I64, I64, P, I64, I, I, P],
                nvfp4_sample=[P, I64, I, I64, I64, P, P, P, P, P, P, P, P, I64, P],
        ).items():
            setattr(self, name, ctypes.CFUNCTYPE(I, *args)((name, L)))


@pytest.fixture(scope="module")
def L():
    return Calls()


def last():
    return nv.lib().nvfp4_last_error().decode()


# ------------------------------------------------------------------ the ABI --

@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=-1), INVALID, "B ="), (dict(B=1 << 30), INVALID, "B ="), (dict(T=-1), INVALID, "T ="), (dict(T=1 << 30), INVALID, "T ="),
    (dict(page=0), INVALID, "page_size"), (dict(mp=-1), INVALID, "max_pages"), (dict(mp=1 << 26, ld=1 << 26), INVALID, "2^30"),
    (dict(ld=7), INVALID, "ld_table"), (dict(F=-1), INVALID, "free"), (dict(F=1 << 30), INVALID, "free"),
    (dict(head=None), INVALID, "NULL"), (dict(cached=None), INVALID, "NULL"), (dict(new=None), INVALID, "NULL"),
    (dict(table=None), INVALID, "NULL"), (dict(free=None), INVALID, "NULL"), (dict(slots=None), INVALID, "NULL"),
    (dict(lengths=None), INVALID, "NULL"), (dict(offsets=None), INVALID, "NULL"), (dict(out=None), INVALID, "NULL"),
    (dict(slots=A + 2), ALIGN, "4-byte"), (dict(cached=A + 1), ALIGN, "4-byte"), (dict(out=A + 2), ALIGN, "4-byte"),
    (dict(T=5000), SMALL, "workspace"), (dict(T=5000, ws=A, wsb=31), SMALL, "workspace"),
    (dict(T=5000, ws=A + 4, wsb=1 << 20), ALIGN, "workspace"), (dict(B=5000, ws=A, wsb=39999), SMALL, "40000"),
])
def test_plan_refusals(L, kw, status, needle):
    a = dict(cached=A, new=A, B=4, table=A, ld=8, mp=8, page=16, free=A, F=10, head=A, T=20, slots=A, lengths=A, offsets=A,
             out=A, ws=None, wsb=0)
    a.update(kw)
    st = L.nvfp4_kv_plan(a["cached"], a["new"], a["B"], a["table"], a["ld"], a["mp"], a["page"], a["free"], a["F"], a["head"],
                         a["T"], a["slots"], A, A, a["lengths"], a["offsets"], a["out"], a["ws"], a["wsb"], None)
    assert st == status and needle in last()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "T ="), (dict(T=1048561), INVALID, "T ="), (dict(K=0), INVALID, "K ="), (dict(K=20), INVALID, "K ="),
    (dict(N=-1), INVALID, "N ="), (dict(R=0), INVALID, "rank"), (dict(R=12), INVALID, "rank"), (dict(R=136), INVALID, "rank"),
    (dict(L=-1), INVALID, "L ="), (dict(ld_x=100), INVALID, "leading"), (dict(ld_y=30), INVALID, "leading"),
    (dict(ld_o=30), INVALID, "leading"), (dict(a_l=-8), INVALID, "strides"), (dict(b_n=-8), INVALID, "strides"),
    (dict(x=None), INVALID, "NULL"), (dict(a=None), INVALID, "NULL"), (dict(b=None), INVALID, "NULL"),
    (dict(ids=None), INVALID, "NULL"), (dict(y=None), INVALID, "NULL"), (dict(o=None), INVALID, "NULL"),
    (dict(x=A + 2), ALIGN, "16-byte"), (dict(ld_x=132), ALIGN, "16-byte"), (dict(a=A + 8), ALIGN, "16-byte"),
    (dict(a_r=130), ALIGN, "16-byte"), (dict(b_n=20), ALIGN, "16-byte"), (dict(y=A + 1), ALIGN, "misaligned"),
    (dict(ids=A + 2), ALIGN, "misaligned"), (dict(s=A + 2), ALIGN, "misaligned"), (dict(ws=None), SMALL, "workspace"),
    (dict(wsb=100), SMALL, "workspace"), (dict(ws=A + 8), ALIGN, "workspace"), (dict(T=0), OK, ""), (dict(N=0, ld_y=0), OK, ""),
    (dict(ld_y=48), INVALID, "another leading"), (dict(T=0, ld_y=48), OK, ""),
])
def test_lora_refusals(L, kw, status, needle):
    a = dict(x=A, ld_x=128, a=A, a_l=2048, a_r=128, b=A, b_l=512, b_n=16, ids=A, s=A, y=A, ld_y=32, o=A, ld_o=32, T=4, K=128, N=32,
             R=16, L=3, ws=A, wsb=1 << 20)
    a.update(kw)
    st = L.nvfp4_lora_add(a["x"], a["ld_x"], a["a"], a["a_l"], a["a_r"], a["b"], a["b_l"], a["b_n"], a["ids"], a["s"], a["y"],
                          a["ld_y"], a["o"], a["ld_o"], a["T"], a["K"], a["N"], a["R"], a["L"], a["ws"], a["wsb"], 0, None)
    assert st == status and needle in last()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "T ="), (dict(T=65), INVALID, "up to 64"), (dict(T=64, k=9), INVALID, "512"), (dict(T=64, k=1 << 58), INVALID, "512"), (dict(k=0), INVALID, "k ="),
    (dict(E=0), INVALID, "E ="), (dict(E=4097), INVALID, "E ="), (dict(H=24), INVALID, "H ="), (dict(I=0), INVALID, "I ="),
    (dict(I=40), INVALID, "I ="), (dict(mx=1, H=48, g1=None, g2=None), INVALID, "multiples of 32"), (dict(mx=2), INVALID, "mx"),
    (dict(act=0), INVALID, "activation"), (dict(act=3), INVALID, "activation"), (dict(ld_x=100), INVALID, "ld_x"),
    (dict(ld_o=100), INVALID, "ld_o"), (dict(w1=None), INVALID, "w_fc1"), (dict(w2=None), INVALID, "w_fc2"),
    (dict(g1=None), INVALID, "global scales"), (dict(mx=1), INVALID, "no global"), (dict(x=None), INVALID, "NULL"),
    (dict(ids=None), INVALID, "NULL"), (dict(w=None), INVALID, "NULL"), (dict(o=None), INVALID, "NULL"),
    (dict(x=A + 2), ALIGN, "16-byte"), (dict(ld_x=132), ALIGN, "16-byte"), (dict(w1=A + 4), ALIGN, "16-byte"),
    (dict(p1=A + 2), ALIGN, "16-byte"), (dict(p2=A + 2), ALIGN, "16-byte"), (dict(o=A + 1), ALIGN, "misaligned"),
    (dict(ids=A + 2), ALIGN, "misaligned"), (dict(g2=A + 2), ALIGN, "misaligned"), (dict(ws=None), SMALL, "workspace"),
    (dict(wsb=4096), SMALL, "workspace"), (dict(ws=A + 16), ALIGN, "workspace"), (dict(T=0), OK, ""),
])
def test_moe_layer_refusals(L, kw, status, needle):
    a = dict(x=A, ld_x=128, ids=A, w=A, T=4, k=2, p1=None, w1=A, g1=A, p2=None, w2=A, g2=A, act=1, o=A, ld_o=128, E=8, H=128, I=64,
             ws=A, wsb=1 << 30, mx=0)
    a.update(kw)
    st = L.nvfp4_moe_layer(a["x"], a["ld_x"], a["ids"], a["w"], a["T"], a["k"], a["p1"], a["w1"], a["g1"], a["p2"], a["w2"],
                           a["g2"], 0, a["act"], a["o"], a["ld_o"], a["E"], a["H"], a["I"], a["ws"], a["wsb"], 0, a["mx"], None)
    assert st == status and needle in last()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=-1), INVALID, "B ="), (dict(B=65536), INVALID, "B ="), (dict(V=0), INVALID, "V ="), (dict(V=(1 << 23) + 1), INVALID, "V ="),
    (dict(type=3), INVALID, "type"), (dict(type=-1), INVALID, "type"), (dict(ld=-1), INVALID, "ld ="), (dict(x=None), INVALID, "NULL"),
    (dict(u=None), INVALID, "NULL"), (dict(o=None), INVALID, "NULL"), (dict(x=A + 1), ALIGN, "logits"),
    (dict(type=2, x=A + 2), ALIGN, "logits"), (dict(u=A + 2), ALIGN, "4-byte"), (dict(t=A + 2), ALIGN, "4-byte"),
    (dict(o=A + 2), ALIGN, "4-byte"), (dict(lp=A + 1), ALIGN, "4-byte"), (dict(ws=None), SMALL, "workspace"),
    (dict(wsb=1000), SMALL, "workspace"), (dict(ws=A + 16), ALIGN, "workspace"), (dict(B=0), OK, ""), (dict(B=0, x=None, u=None), OK, ""),
])
def test_sample_refusals(L, kw, status, needle):
    a = dict(x=A, ld=100, type=0, B=4, V=100, u=A, t=A, k=A, p=A, mp=A, o=A, lp=A, ws=A, wsb=1 << 30)
    a.update(kw)
    st = L.nvfp4_sample(a["x"], a["ld"], a["type"], a["B"], a["V"], a["u"], a["t"], a["k"], a["p"], a["mp"], a["o"], a["lp"],
                        a["ws"], a["wsb"], None)
    assert st == status and needle in last()


def test_workspace_sizes():
    for f, bad in ((nv.lora_workspace_bytes, (4, 20, 32, 16)), (nv.moe_layer_workspace_bytes, (65, 2, 8, 128, 64)),
                   (nv.moe_layer_workspace_bytes, (64, 1 << 58, 8, 128, 64)),
                   (nv.sample_workspace_bytes, (4, 0))):
        with pytest.raises(ValueError):
            f(*bad)
    assert nv.lora_workspace_bytes(0, 128, 32, 16) == 0 and nv.moe_layer_workspace_bytes(0, 2, 8, 128, 64) == 0
    # x A^T of one slice at least
    assert nv.lora_workspace_bytes(7, 128, 32, 16) >= 7 * 16 * 4
    assert nv.moe_layer_workspace_bytes(1, 1, 8, 128, 64) >= 4096 + 64 * 2


# -------------------------------------------------------------- the binding --

def test_the_binding_refuses_tensors_off_the_gpu():
    ints, x = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cached"):
        nv.kv_plan(ints, ints, torch.zeros((3, 4), dtype=torch.int32), ints, ints[:1], 16, 3)
    with pytest.raises(ValueError, match="cached"):
        nv.kv_plan(ints.float(), ints, torch.zeros((3, 4), dtype=torch.int32), ints, ints[:1], 16, 3)
    with pytest.raises(ValueError, match="x must be"):
        nv.lora_add(x, x, x[None], x[None], ints)
    with pytest.raises(ValueError, match="x must be"):
        nv.moe_layer(x.float(), ints[:, None], torch.ones(3, 1), None, None, 4, 16)
    with pytest.raises(ValueError, match="logits"):
        nv.sample(x, torch.zeros(3))
    with pytest.raises(ValueError, match="logits"):
        nv.sample(None, torch.zeros(3))


# ---------------------------------------------------------- the plain forms --

def test_plain_plan_by_hand():
    """Two requests: 3 cached tokens and 2 new ones in pages of 4 (the second new one begins a page), and a new prompt of 5;
    a third whose page the list no longer has."""
    got = ref.plan([3, 0, 8], [2, 5, 1], np.array([[9, 0, 0], [0, 0, 0], [6, 7, 0]]), np.array([50, 20, 30, 40]), 1, 4, 9)
    slots, positions, requests, lengths, offsets, head, table = got
    assert slots.tolist() == [39, 80, 120, 121, 122, 123, 160, -1, -1]
    assert positions.tolist() == [3, 4, 0, 1, 2, 3, 4, 0, 0] and requests.tolist() == [0, 0, 1, 1, 1, 1, 1, -1, -1]
    assert lengths.tolist() == [5, 5, 8] and offsets.tolist() == [0, 2, 7, 8] and head.tolist() == [4]
    assert table.tolist() == [[9, 20, 0], [30, 40, 0], [6, 7, 0]]


def test_plain_sample_by_hand():
    l = np.log(np.array([1.0, 4.0, 2.0, 4.0, 1.0]))
    # kept by top-k 3: tokens 1, 3, 2 (4 + 4 + 2); in their order 1, 2, 3: cumulative 4, 6, 10
    for u, token in ((0.0, 1), (0.399, 1), (0.401, 2), (0.599, 2), (0.601, 3), (0.9999, 3)):
        got = ref.sample_row(l, u, k=3)
        assert got[0] == token and abs(got[1] - np.log([0, 0.4, 0.2, 0.4][token])) < 1e-12
    # top-p 0.34 of 12: 4 < 4.08, so the second token of 4 stays too
    assert ref.sample_row(l, 0.6, p=0.34)[0] == 3 and ref.sample_row(l, 0.99, p=0.33)[0] == 1
    assert ref.sample_row(l, 0.99, min_p=0.5)[0] == 3 and ref.sample_row(l, 0.45, min_p=0.5)[0] == 2
    assert ref.sample_row(l, 0.9, t=0.0) == (1, 0.0) and ref.sample_row(np.full(3, -np.inf), 0.5) == (-1, -np.inf)


def test_plain_weights_by_hand():
    codes = torch.tensor([[0x10, 0xF7] + [0] * 6], dtype=torch.uint8)   # 0, 0.5, 6, -6
    got = ref.weights(codes, torch.tensor([[0x39]], dtype=torch.uint8), False)   # 1.125
    assert got[0, :4].tolist() == [0.0, 0.5625, 6.75, -6.75] and got.shape == (1, 16)
    got = ref.weights(torch.cat((codes, codes), 1), torch.tensor([[126]], dtype=torch.uint8), True)
    assert got[0, 16:20].tolist() == [0.0, 0.25, 3.0, -3.0]
