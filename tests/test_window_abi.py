"""Argument checks of the ragged append and the windowed attention, without a
GPU: only calls that fail a host check, or that launch nothing."""
import ctypes

import pytest
import torch

import paged_len_decode_gb300 as v

FAKE = ctypes.c_void_p(0x10000)       # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)        # misaligned
CACHE = dict(kc=FAKE, vc=FAKE, ps=2 * 16 * 8 * 128, ts=8 * 128, hs=128, npages=100, pt=FAKE, mps=10)
SHAPE = dict(T=9, B=4, Hq=16, Hkv=8, D=128, P=16)


def append(**over):
    a = dict(q=FAKE, k=FAKE, vv=FAKE, qs=16 * 128, ks=8 * 128, vs=8 * 128, cs=FAKE, max_pos=4096, pos=FAKE, axes=None,
             na=3, qw=None, kw=None, eps=1e-6, start=FAKE, sl=FAKE, act=FAKE, q_rot=FAKE, err=None, flags=0, **CACHE, **SHAPE)
    a.update(over)
    axes = None if a["axes"] is None else (ctypes.c_uint8 * 64)(*a["axes"])
    return v.lib.vh_mrope_kv_append(
        a["q"], a["k"], a["vv"], a["qs"], a["ks"], a["vs"], a["cs"], a["max_pos"], a["pos"], axes, a["na"], a["qw"], a["kw"],
        a["eps"], a["kc"], a["vc"], a["ps"], a["ts"], a["hs"], a["npages"], a["pt"], a["mps"], a["start"], a["sl"], a["act"],
        a["q_rot"], a["err"], a["flags"], a["T"], a["B"], a["Hq"], a["Hkv"], a["D"], a["P"], None)


def decode(**over):
    a = dict(q=FAKE, sl=FAKE, act=FAKE, w=64, s=4, out=FAKE, scale=0.0, n=0, ws=FAKE, wsb=1 << 30, err=None, flags=0,
             **CACHE, **SHAPE)
    a.update(over)
    return v.lib.vh_window_decode_attn(
        a["q"], a["kc"], a["vc"], a["ps"], a["ts"], a["hs"], a["npages"], a["pt"], a["mps"], a["sl"], a["act"], a["w"], a["s"],
        a["out"], a["scale"], a["n"], a["ws"], a["wsb"], a["err"], a["flags"], a["B"], a["Hq"], a["Hkv"], a["D"], a["P"], None)


def prompt(**over):
    a = dict(q=FAKE, start=FAKE, sl=FAKE, act=FAKE, w=64, s=4, out=FAKE, scale=0.0, n=0, ws=FAKE, wsb=1 << 40, err=None,
             flags=0, **CACHE, **SHAPE)
    a.update(over)
    return v.lib.vh_window_prompt_attn(
        a["q"], a["kc"], a["vc"], a["ps"], a["ts"], a["hs"], a["npages"], a["pt"], a["mps"], a["start"], a["sl"], a["act"],
        a["w"], a["s"], a["out"], a["scale"], a["n"], a["ws"], a["wsb"], a["err"], a["flags"], a["T"], a["B"], a["Hq"],
        a["Hkv"], a["D"], a["P"], None)


COMMON = [
    (dict(Hq=12), v.VH_EINVAL), (dict(Hq=24), v.VH_EINVAL), (dict(D=96), v.VH_EINVAL), (dict(P=12), v.VH_EINVAL),
    (dict(P=24), v.VH_EINVAL), (dict(B=0), v.VH_EINVAL), (dict(B=70000), v.VH_EINVAL), (dict(mps=0), v.VH_EINVAL),
    (dict(npages=0), v.VH_EINVAL), (dict(mps=1 << 22), v.VH_EINVAL), (dict(hs=0), v.VH_EINVAL), (dict(ps=-8), v.VH_EINVAL),
    (dict(pt=None, npages=39), v.VH_EINVAL), (dict(kc=None), v.VH_EINVAL), (dict(sl=None), v.VH_EINVAL),
    (dict(act=None), v.VH_EINVAL), (dict(q=None), v.VH_EINVAL), (dict(q=ODD), v.VH_EALIGN), (dict(vc=ODD), v.VH_EALIGN),
    (dict(ts=8 * 128 + 4), v.VH_EALIGN), (dict(flags=1 << 20), v.VH_EINVAL), (dict(flags=v.VH_FLAG_HOST_IO), v.VH_EINVAL),
    (dict(flags=v.VH_FLAG_PLANNED), v.VH_EINVAL),
]


@pytest.mark.parametrize("call", [append, decode, prompt])
@pytest.mark.parametrize("over,code", COMMON)
def test_common_checks(call, over, code):
    assert call(**over) == code


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), v.VH_EINVAL), (dict(max_pos=0), v.VH_EINVAL), (dict(na=0), v.VH_EINVAL), (dict(na=5), v.VH_EINVAL),
    (dict(axes=[0] * 63 + [3]), v.VH_EINVAL),           # an axis that positions do not have
    (dict(eps=-1.0), v.VH_EINVAL), (dict(eps=float("nan")), v.VH_EINVAL),
    (dict(start=None), v.VH_EINVAL),                    # one token a row needs T == B
    (dict(qs=16 * 128 - 8), v.VH_EINVAL), (dict(ks=8), v.VH_EINVAL), (dict(vs=0), v.VH_EINVAL),
    (dict(qs=16 * 128 + 4), v.VH_EALIGN), (dict(qw=ODD), v.VH_EALIGN), (dict(q_rot=ODD), v.VH_EALIGN),
    (dict(q_rot=None), v.VH_EINVAL), (dict(cs=None), v.VH_EINVAL), (dict(flags=v.VH_FLAG_PDL), v.VH_EINVAL),
    (dict(T=0, q=None, k=None, vv=None, q_rot=None), v.VH_OK),     # an empty batch launches nothing
    (dict(T=0, max_pos=0), v.VH_EINVAL),
])
def test_append_checks(over, code):
    assert append(**over) == code


@pytest.mark.parametrize("call", [decode, prompt])
@pytest.mark.parametrize("over,code", [
    (dict(w=-1), v.VH_EINVAL), (dict(s=-1), v.VH_EINVAL), (dict(n=-1), v.VH_EINVAL), (dict(n=65536), v.VH_EINVAL),
    (dict(scale=float("nan")), v.VH_EINVAL), (dict(out=None), v.VH_EINVAL), (dict(out=ODD), v.VH_EALIGN),
    (dict(ws=None), v.VH_EWORKSPACE), (dict(ws=ODD), v.VH_EALIGN), (dict(flags=v.VH_FLAG_Q16), v.VH_EINVAL),
])
def test_attention_checks(call, over, code):
    assert call(**over) == code


def test_prompt_checks():
    assert prompt(T=-1) == v.VH_EINVAL
    assert prompt(start=None) == v.VH_EINVAL
    assert prompt(n=32) == v.VH_EINVAL
    assert prompt(n=3) == v.VH_EINVAL
    assert prompt(wsb=255) in (v.VH_EWORKSPACE, v.VH_ENODEV)
    assert prompt(flags=v.VH_FLAG_PDL) == v.VH_EINVAL
    assert prompt(T=0, q=None, out=None) == v.VH_OK
    assert v.lib.vh_prompt_workspace_bytes(-1, 4, 16, 8, 128) == 0
    assert v.lib.vh_prompt_workspace_bytes(4, 4, 12, 8, 128) == 0


def test_valid_calls_report_no_device_without_one():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for call in (append, decode, prompt):
        assert call() == v.VH_ENODEV


def test_pair_axes():
    assert v.mrope_pair_axis([1, 2, 29], 64) == [0] + [1] * 2 + [2] * 29
    assert v.mrope_pair_axis([24, 4, 4], 64, cyclic=True) == [0, 1, 2] * 4 + [0] * 20
    with pytest.raises(ValueError):
        v.mrope_pair_axis([1, 2], 64)
    with pytest.raises(ValueError):
        v.mrope_pair_axis([0, 16, 16], 64, cyclic=True)   # 16 of each do not fit in turn into 32


def binding_args(op):
    t = torch.zeros
    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    kc = t(4, 16, 2, 64, **bf)
    a = dict(k_cache=kc, v_cache=kc, page_table=t(3, 2, **i32), seq_lens=t(3, **i32), active=t(3, **i32))
    if op == "append":
        return v.vh_mrope_kv_append, dict(a, q=t(5, 4, 64, **bf), k_new=t(5, 2, 64, **bf), v_new=t(5, 2, 64, **bf), cos_sin=t(8, 64),
                                          q_rot=t(5, 4, 64), token_start=t(4, **i32), positions=t(3, 5, **i32), pair_axis=[0] * 32)
    a.update(workspace=t(1 << 20, dtype=torch.uint8))
    if op == "decode":
        return v.vh_window_decode_attn, dict(a, q_rot=t(3, 4, 64), out=t(3, 4, 64, **bf))
    return v.vh_window_prompt_attn, dict(a, q=t(5, 4, 64, **bf), out=t(5, 4, 64, **bf), token_start=t(4, **i32))


@pytest.mark.parametrize("op,wrong,text", [
    ("append", dict(k_new=torch.zeros(4, 2, 64)), "mismatch"), ("append", dict(q_rot=torch.zeros(5, 4, 32)), "mismatch"),
    ("append", dict(positions=torch.zeros(3, 4, dtype=torch.int32)), "positions"), ("append", dict(pair_axis=[0] * 31), "pair_axis"),
    ("append", dict(token_start=torch.zeros(3, dtype=torch.int32)), "token_start"), ("append", dict(cos_sin=torch.zeros(8, 32)), "cos_sin"),
    ("decode", dict(seq_lens=torch.zeros(2, dtype=torch.int32)), "active"), ("decode", dict(out=torch.zeros(3, 4, 32)), "mismatch"),
    ("prompt", dict(active=torch.zeros(2, dtype=torch.int32)), "active"), ("prompt", dict(page_table=torch.zeros(2, 2)), "page_table"),
    ("prompt", dict(out=torch.zeros(4, 4, 64)), "mismatch"),
    ("append", {}, "CUDA"), ("decode", {}, "CUDA"), ("prompt", {}, "CUDA"),       # host tensors
])
def test_binding_refuses(op, wrong, text):
    call, args = binding_args(op)
    with pytest.raises(ValueError, match=text):
        call(**dict(args, **wrong))


@pytest.mark.parametrize("call, first, count", [(v.vh_mrope_kv_append, "q", 19), (v.vh_window_decode_attn, "q_rot", 15),
                                                (v.vh_window_prompt_attn, "q", 15)])
def test_arguments_are_named_in_errors_call_after_call(call, first, count):
    for _ in range(3):
        with pytest.raises(TypeError, match=f"needs the argument '{first}'"):
            call()
        with pytest.raises(TypeError, match=f"got two values for '{first}'"):
            call(1, **{first: 1})
        with pytest.raises(TypeError, match="unexpected argument 'nothing'"):
            call(nothing=1)
        with pytest.raises(TypeError, match=f"at most {count} arguments"):
            call(*range(count + 1))
    for _ in range(2):
        with pytest.raises(TypeError, match="q_norm_w must be a torch.Tensor"):
            x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
            pool = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16)
            one = torch.ones(1, dtype=torch.int32)
            v.vh_mrope_kv_append(x, x, x, torch.zeros(4, 64), pool, pool, one[:, None], one, one, x, q_norm_w=1)
