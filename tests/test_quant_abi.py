"""Argument checks of the calls on 8-bit caches and of the tree attention, without a GPU: only calls that fail a check,
or that launch nothing; and the helpers that make masks and caches."""
import ctypes

import pytest
import torch

import paged_len_decode_gb300 as v

FAKE = ctypes.c_void_p(0x10000)       # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)        # misaligned
CACHE = dict(kc=FAKE, vc=FAKE, ps=2 * 16 * 8 * 128, ts=8 * 128, hs=128, ks=FAKE, vs=FAKE, sps=2 * 8 * 16, shs=16, npages=100,
             pt=FAKE, mps=10)
SHAPE = dict(T=9, B=4, Hq=16, Hkv=8, D=128, P=16)


def append(**over):
    a = dict(q=FAKE, k=FAKE, vv=FAKE, qs=16 * 128, kst=8 * 128, vst=8 * 128, cs=FAKE, max_pos=4096, pos=FAKE, na=3, qw=None,
             kw=None, eps=1e-6, start=FAKE, sl=FAKE, act=FAKE, q_rot=FAKE, flags=0, **CACHE, **SHAPE)
    a.update(over)
    return v.lib.vh_quant_kv_append(
        a["q"], a["k"], a["vv"], a["qs"], a["kst"], a["vst"], a["cs"], a["max_pos"], a["pos"], None, a["na"], a["qw"], a["kw"],
        a["eps"], a["kc"], a["vc"], a["ps"], a["ts"], a["hs"], a["ks"], a["vs"], a["sps"], a["shs"], a["npages"], a["pt"], a["mps"],
        a["start"], a["sl"], a["act"], a["q_rot"], None, a["flags"], a["T"], a["B"], a["Hq"], a["Hkv"], a["D"], a["P"], None)


def decode(**over):
    a = dict(q=FAKE, sl=FAKE, act=FAKE, w=64, s=4, out=FAKE, scale=0.0, n=0, ws=FAKE, wsb=1 << 30, flags=0, **CACHE, **SHAPE)
    a.update(over)
    return v.lib.vh_quant_decode_attn(
        a["q"], a["kc"], a["vc"], a["ps"], a["ts"], a["hs"], a["ks"], a["vs"], a["sps"], a["shs"], a["npages"], a["pt"], a["mps"],
        a["sl"], a["act"], a["w"], a["s"], a["out"], a["scale"], a["n"], a["ws"], a["wsb"], None, a["flags"], a["B"], a["Hq"],
        a["Hkv"], a["D"], a["P"], None)


def read(**over):
    a = dict(sl=FAKE, act=FAKE, first=None, s=4, ko=FAKE, vo=FAKE, ops=2 * 16 * 8 * 128, ots=8 * 128, ohs=128, onp=100, opt=FAKE,
             omps=10, flags=0, P2=16, **CACHE, **SHAPE)
    a.update(over)
    return v.lib.vh_quant_kv_read(
        a["kc"], a["vc"], a["ps"], a["ts"], a["hs"], a["ks"], a["vs"], a["sps"], a["shs"], a["npages"], a["pt"], a["mps"], a["sl"],
        a["act"], a["first"], a["s"], a["ko"], a["vo"], a["ops"], a["ots"], a["ohs"], a["onp"], a["opt"], a["omps"], None,
        a["flags"], a["B"], a["Hkv"], a["D"], a["P"], a["P2"], None)


def tree(**over):
    a = dict(q=FAKE, start=FAKE, sl=FAKE, act=FAKE, mask=FAKE, mw=1, w=64, s=4, out=FAKE, scale=0.0, n=0, ws=FAKE, wsb=1 << 40,
             flags=0, **CACHE, **SHAPE)
    a.update(over)
    return v.lib.vh_tree_attn(
        a["q"], a["kc"], a["vc"], a["ps"], a["ts"], a["hs"], a["npages"], a["pt"], a["mps"], a["start"], a["sl"], a["act"],
        a["mask"], a["mw"], a["w"], a["s"], a["out"], a["scale"], a["n"], a["ws"], a["wsb"], None, a["flags"], a["T"], a["B"],
        a["Hq"], a["Hkv"], a["D"], a["P"], None)


CALLS = [append, decode, read, tree]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(D=96), v.VH_EINVAL), (dict(P=12), v.VH_EINVAL), (dict(P=24), v.VH_EINVAL), (dict(B=0), v.VH_EINVAL),
    (dict(B=70000), v.VH_EINVAL), (dict(mps=0), v.VH_EINVAL), (dict(npages=0), v.VH_EINVAL), (dict(mps=1 << 22), v.VH_EINVAL),
    (dict(hs=0), v.VH_EINVAL), (dict(ps=-16), v.VH_EINVAL), (dict(pt=None, npages=39), v.VH_EINVAL), (dict(kc=None), v.VH_EINVAL),
    (dict(vc=None), v.VH_EINVAL), (dict(sl=None), v.VH_EINVAL), (dict(act=None), v.VH_EINVAL), (dict(vc=ODD), v.VH_EALIGN),
    (dict(ts=8 * 128 + 4), v.VH_EALIGN), (dict(flags=1 << 20), v.VH_EINVAL), (dict(flags=v.VH_FLAG_HOST_IO), v.VH_EINVAL),
    (dict(flags=v.VH_FLAG_PLANNED), v.VH_EINVAL),
])
def test_common_checks(call, over, code):
    assert call(**over) == code


@pytest.mark.parametrize("call", [append, decode, tree])
@pytest.mark.parametrize("over,code", [(dict(Hq=12), v.VH_EINVAL), (dict(Hq=24), v.VH_EINVAL), (dict(q=None), v.VH_EINVAL),
                                       (dict(q=ODD), v.VH_EALIGN)])
def test_query_checks(call, over, code):
    assert call(**over) == code


@pytest.mark.parametrize("call", [append, decode, read])
@pytest.mark.parametrize("over,code", [
    (dict(ks=None), v.VH_EINVAL), (dict(vs=None), v.VH_EINVAL), (dict(sps=0), v.VH_EINVAL), (dict(shs=-4), v.VH_EINVAL),
    (dict(ks=ODD), v.VH_EALIGN), (dict(vs=ODD), v.VH_EALIGN), (dict(sps=258), v.VH_EALIGN), (dict(shs=18), v.VH_EALIGN),
    (dict(ts=8 * 128 + 8), v.VH_EALIGN),      # 8 elements of 8 bits are no 16 bytes
])
def test_scale_checks(call, over, code):
    assert call(**over) == code


def test_append_checks():
    assert append(start=None) == v.VH_EINVAL
    assert append(T=-1) == v.VH_EINVAL
    assert append(na=5) == v.VH_EINVAL
    assert append(eps=float("nan")) == v.VH_EINVAL
    assert append(qs=16 * 128 - 8) == v.VH_EINVAL
    assert append(q_rot=ODD) == v.VH_EALIGN
    assert append(flags=v.VH_FLAG_PDL) == v.VH_EINVAL
    assert append(T=0, q=None, k=None, vv=None, q_rot=None, kc=None, vc=None, ks=None, vs=None) == v.VH_OK
    assert append(T=0, max_pos=0) == v.VH_EINVAL


def test_decode_checks():
    for over, code in ((dict(w=-1), v.VH_EINVAL), (dict(s=-1), v.VH_EINVAL), (dict(n=-1), v.VH_EINVAL), (dict(n=65536), v.VH_EINVAL),
                       (dict(scale=float("nan")), v.VH_EINVAL), (dict(out=None), v.VH_EINVAL), (dict(out=ODD), v.VH_EALIGN),
                       (dict(ws=None), v.VH_EWORKSPACE), (dict(ws=ODD), v.VH_EALIGN), (dict(flags=v.VH_FLAG_Q16), v.VH_EINVAL)):
        assert decode(**over) == code


def test_read_checks():
    for over, code in ((dict(s=-1), v.VH_EINVAL), (dict(ko=None), v.VH_EINVAL), (dict(vo=ODD), v.VH_EALIGN), (dict(ops=0), v.VH_EINVAL),
                       (dict(ohs=12), v.VH_EALIGN), (dict(P2=24), v.VH_EINVAL), (dict(opt=None, onp=39), v.VH_EINVAL),
                       (dict(omps=0), v.VH_EINVAL), (dict(flags=v.VH_FLAG_PDL), v.VH_EINVAL)):
        assert read(**over) == code


def test_tree_checks():
    for over, code in ((dict(mask=None), v.VH_EINVAL), (dict(mw=0), v.VH_EINVAL), (dict(mw=17), v.VH_EINVAL),
                       (dict(mask=ctypes.c_void_p(0x10004)), v.VH_EALIGN), (dict(T=-1), v.VH_EINVAL), (dict(start=None), v.VH_EINVAL),
                       (dict(w=-1), v.VH_EINVAL), (dict(s=-1), v.VH_EINVAL), (dict(n=3), v.VH_EINVAL), (dict(n=32), v.VH_EINVAL),
                       (dict(scale=float("nan")), v.VH_EINVAL), (dict(ws=None), v.VH_EWORKSPACE), (dict(ws=ODD), v.VH_EALIGN),
                       (dict(out=None), v.VH_EINVAL), (dict(flags=v.VH_FLAG_PDL), v.VH_EINVAL)):
        assert tree(**over) == code
    assert tree(wsb=255) in (v.VH_EWORKSPACE, v.VH_ENODEV)
    assert tree(T=0, q=None, out=None, mask=None) == v.VH_OK   # an empty batch launches nothing


def test_valid_calls_report_no_device_without_one():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for call in CALLS:
        assert call() == v.VH_ENODEV


def test_tree_masks():
    m = v.tree_masks([[-1, 0, 0, 1], [], [-1]], device="cpu")
    assert m.tolist() == [[0], [1], [1], [3], [0]]
    chain = v.tree_masks([list(range(-1, 129))], device="cpu")
    assert chain.shape == (130, 3) and chain[129].tolist() == [-1, -1, 1] and chain[64].tolist() == [-1, 0, 0]
    assert chain[63].tolist() == [(1 << 63) - 1, 0, 0]
    assert v.tree_masks([], device="cpu").shape == (0, 1)
    for bad in ([0], [-1, 1], [-1, -2], [-1, 5]):
        with pytest.raises(ValueError):
            v.tree_masks([bad], device="cpu")


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("P", [16, 11])
def test_alloc_quant_cache(head_major, P):
    k, vv, ks, vs = v.alloc_quant_cache(5, P, 3, 64, head_major, device="cpu")
    assert k.shape == vv.shape == (5, P, 3, 64) and k.dtype == torch.float8_e4m3fn and k.stride() == vv.stride()
    assert ks.shape == vs.shape == (5, 3, P) and ks.stride(2) == 1 and ks.stride(0) % 4 == ks.stride(1) % 4 == 0
    assert not k.float().any() and not ks.any()


def binding_args(op):
    t = torch.zeros
    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    k8, v8, ks, vs = v.alloc_quant_cache(4, 16, 2, 64, device="cpu")
    cache = dict(k_cache=k8, v_cache=v8, k_scale=ks, v_scale=vs)
    rows = dict(page_table=t(3, 2, **i32), seq_lens=t(3, **i32), active=t(3, **i32))
    if op == "append":
        return v.vh_quant_kv_append, dict(q=t(3, 4, 64, **bf), k_new=t(3, 2, 64, **bf), v_new=t(3, 2, 64, **bf), cos_sin=t(9, 64),
                                          **cache, **rows, q_rot=t(3, 4, 64))
    if op == "decode":
        return v.vh_quant_decode_attn, dict(q_rot=t(3, 4, 64), **cache, **rows, out=t(3, 4, 64, **bf), workspace=t(64))
    if op == "read":
        return v.vh_quant_kv_read, dict(**cache, **rows, k_out=t(4, 16, 2, 64, **bf), v_out=t(4, 16, 2, 64, **bf),
                                        out_page_table=t(3, 2, **i32))
    kc = t(4, 16, 2, 64, **bf)
    return v.vh_tree_attn, dict(q=t(3, 4, 64, **bf), k_cache=kc, v_cache=kc, **rows, token_start=t(4, **i32),
                                tree_mask=t(3, 1, dtype=torch.int64), out=t(3, 4, 64, **bf), workspace=t(64))


@pytest.mark.parametrize("op,over,error", [
    ("append", dict(q=torch.zeros(3, 4, 64)), TypeError),                            # 32-bit queries
    ("append", dict(k_cache=torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)), (TypeError, ValueError)),
    ("append", dict(k_new=torch.zeros(3, 3, 64, dtype=torch.bfloat16)), ValueError),
    ("decode", dict(k_scale=torch.zeros(4, 16, 2)), ValueError),                     # slots before heads
    ("decode", dict(k_scale=torch.zeros(4, 16, 2).transpose(1, 2)), ValueError),     # slots apart
    ("decode", dict(out=torch.zeros(3, 4, 64)), TypeError),
    ("decode", dict(out=torch.zeros(3, 5, 64)), ValueError),
    ("read", dict(out_page_table=torch.zeros(2, 2, dtype=torch.int32)), ValueError),
    ("read", dict(k_out=torch.zeros(4, 16, 3, 64, dtype=torch.bfloat16), v_out=torch.zeros(4, 16, 3, 64, dtype=torch.bfloat16)), ValueError),
    ("read", dict(k_out=torch.zeros(4, 16, 2, 64), v_out=torch.zeros(4, 16, 2, 64)), TypeError),
    ("read", dict(first_slot=torch.zeros(4, dtype=torch.int32)), ValueError),
    ("tree", dict(workspace=3), TypeError),
    ("tree", dict(out=torch.zeros(2, 4, 64, dtype=torch.bfloat16)), ValueError),
    ("tree", dict(nonsense=1), TypeError),
])
def test_binding_refusals(op, over, error):
    f, a = binding_args(op)
    with pytest.raises(error):
        f(**{**a, **over})


@pytest.mark.parametrize("op", ["append", "decode", "read", "tree"])
def test_binding_takes_cuda_tensors_only(op):
    f, a = binding_args(op)
    with pytest.raises(ValueError):
        f(**a)
    with pytest.raises(TypeError):
        f()
