"""The rotary and cache entry points refuse bad arguments on the host, before any CUDA call; the
host calculations and the fp64 restatement that the GPU tests use are checked against their
definitions."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch

import cache_ref as ref
from online_softmax_tiled_attn_gb300 import binding

P = 1 << 20
T = 1 << 20  # bytes between the fake addresses
BAD, UNSUP, OK = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_OK
S3 = ctypes.c_int64 * 3


def strides(*v):
    return S3(*v)


@pytest.mark.parametrize("over, want", [
    (dict(N=-1), BAD), (dict(N=0), OK), (dict(B=0, x=0, y=0), OK), (dict(dtype=2), BAD),
    (dict(rot=0), BAD), (dict(rot=7), BAD), (dict(rot=66), BAD), (dict(rot=-2), BAD),
    (dict(layout=2), BAD), (dict(amp=math.inf), BAD), (dict(amp=math.nan), BAD),
    (dict(table=0), BAD), (dict(table=P + 5 * T + 4), BAD), (dict(x=0), BAD), (dict(y=0), BAD),
    (dict(x=P + 1), BAD), (dict(y=P + T + 1), BAD), (dict(y=P + 2), BAD),  # overlap, not in place
    (dict(xs=None), BAD), (dict(xs=(-4096, 2048, 64)), BAD),
    (dict(ys=(4096, 2048, 0)), BAD),                       # rows of y on one another
    (dict(ys=(4096, 2048, 32)), BAD),
    (dict(y=P, ys=(4096, 64, 128)), BAD),                  # x's memory with other strides
    (dict(pos=P + 2 * T + 2), BAD), (dict(pos=P + T), BAD),  # positions inside y
    (dict(pos=P + 2 * T, pbs=-1), BAD), (dict(table=P + T), BAD),
    (dict(B=1 << 40, N=1 << 30), BAD),
])
def test_rope_refusals(over, want):
    a = dict(x=P, y=P + T, dtype=0, B=2, H=2, N=32, d=64, xs=(4096, 2048, 64), ys=(4096, 2048, 64),
             pos=0, pbs=0, table=P + 5 * T, rot=64, layout=1, amp=1.0)
    a.update(over)
    for call in (binding.lib().osm_rope, binding.lib().osm_rope_bwd):
        rc = call(a["x"] or None, a["y"] or None, a["dtype"], a["B"], a["H"], a["N"], a["d"],
                  strides(*a["xs"]) if a["xs"] else None, strides(*a["ys"]), a["pos"] or None,
                  a["pbs"], a["table"] or None, a["rot"], a["layout"], a["amp"], None)
        assert rc == want


@pytest.mark.parametrize("over, want", [
    (dict(N=-1), BAD), (dict(N=0), OK), (dict(d=96), UNSUP), (dict(fmt=2), BAD),
    (dict(page=8), UNSUP), (dict(page=24), UNSUP), (dict(page=2048), UNSUP), (dict(page=0), BAD),
    (dict(maxp=(1 << 26) + 1), BAD), (dict(nump=1 << 31), BAD), (dict(kp=0), BAD), (dict(vp=0), BAD),
    (dict(kp=P + 3 * T + 8), BAD), (dict(pt=0), BAD), (dict(pt=P + 5 * T + 2), BAD),
    (dict(kp=P + 4 * T), BAD),                              # keys and values in one array
    (dict(k=P + 3 * T + 64), BAD), (dict(k=0), BAD), (dict(v=0), BAD), (dict(v=P + T + 1), BAD),
    (dict(cl=0), BAD), (dict(cl=P + 6 * T + 2), BAD), (dict(nl=P + 6 * T + 2), BAD),
    (dict(cl=P + 3 * T), BAD), (dict(nl=P + 4 * T), BAD), (dict(pt=P + 3 * T), BAD),
    (dict(table=0), BAD), (dict(rot=130), BAD), (dict(rot=3), BAD), (dict(layout=5), BAD),
    (dict(amp=math.nan), BAD), (dict(table=P + 4 * T), BAD),
    (dict(q=P + 8 * T, qo=0), BAD), (dict(q=0, qo=P + 9 * T), BAD), (dict(q=P, qo=P + 9 * T, H=-1), BAD),
    (dict(q=P + 8 * T, qo=P + 9 * T + 8), BAD),             # q_out misaligned
    (dict(q=P + 8 * T, qo=P + 3 * T), BAD),                 # q_out on the pages
    (dict(q=P + 8 * T, qo=P + 8 * T + 32), BAD),            # q_out overlaps q
    (dict(q=P + 8 * T, qo=P + 8 * T, qs=(8 * 640, 128, 8 * 128)), BAD),  # in place, q strided
    (dict(q=P + 8 * T, qo=P), BAD),                         # q_out on k
    (dict(ks=(-1, 640, 128)), BAD),
])
def test_append_refusals(over, want):
    """B2 H8 H_kv 2 N5 d128 at distinct fake addresses, 4 pages of 16."""
    st = (2 * 640, 640, 128)
    a = dict(k=P, v=P + T, ks=st, vs=st, kp=P + 3 * T, vp=P + 4 * T, fmt=0, nump=4, page=16,
             pt=P + 5 * T, maxp=2, cl=P + 6 * T, nl=0, table=P + 7 * T, rot=128, layout=1, amp=1.0,
             q=0, qo=0, qs=(8 * 640, 640, 128), B=2, H=8, Hkv=2, N=5, d=128)
    a.update(over)
    rc = binding.lib().osm_kv_append(
        a["k"] or None, a["v"] or None, strides(*a["ks"]), strides(*a["vs"]), a["kp"] or None,
        a["vp"] or None, a["fmt"], a["nump"], a["page"], a["pt"] or None, a["maxp"],
        a["cl"] or None, a["nl"] or None, a["table"] or None, a["rot"], a["layout"], a["amp"],
        a["q"] or None, a["qo"] or None, strides(*a["qs"]), a["B"], a["H"], a["Hkv"], a["N"],
        a["d"], None)
    assert rc == want


@pytest.mark.parametrize("over, want", [
    (dict(N=0), OK), (dict(N=-1), BAD), (dict(d=32), UNSUP), (dict(fmt=-1), BAD),
    (dict(page=17), UNSUP), (dict(K=0), BAD), (dict(V=P + 6 * T + 8), BAD), (dict(kl=0), BAD),
    (dict(K=P + 6 * T), BAD), (dict(K=P + 64), BAD), (dict(kl=P + 5 * T + 4), BAD),
    (dict(pt=P + 6 * T), BAD),
])
def test_gather_refusals(over, want):
    a = dict(kp=P, vp=P + T, fmt=1, nump=4, page=16, pt=P + 2 * T, maxp=2, kl=P + 3 * T,
             K=P + 5 * T, V=P + 6 * T, B=2, Hkv=2, N=30, d=64)
    a.update(over)
    rc = binding.lib().osm_kv_gather(a["kp"], a["vp"], a["fmt"], a["nump"], a["page"], a["pt"],
                                     a["maxp"], a["kl"] or None, a["K"] or None, a["V"], a["B"],
                                     a["Hkv"], a["N"], a["d"], None)
    assert rc == want


@pytest.mark.parametrize("over, want", [
    (dict(Nq=0), OK), (dict(B=0), OK), (dict(Nq=-1), BAD), (dict(Hkv=3), BAD), (dict(Hkv=0), BAD),
    (dict(d=96), UNSUP), (dict(page=40), UNSUP), (dict(fmt=3), BAD), (dict(scale=0.0), BAD),
    (dict(scale=math.inf), BAD), (dict(q=0), BAD), (dict(o=0), BAD), (dict(o=P + 4 * T + 8), BAD),
    (dict(lse=P + 5 * T + 2), BAD), (dict(kl=0), BAD), (dict(kl=P + 6 * T + 1), BAD),
    (dict(ql=P + 7 * T + 2), BAD), (dict(o=P), BAD), (dict(o=P + T), BAD), (dict(lse=P + 4 * T), BAD),
    (dict(kl=P + 4 * T), BAD), (dict(ql=P + 5 * T), BAD), (dict(pt=P + 4 * T), BAD),
    (dict(kp=0), BAD), (dict(vp=P + 2 * T + 8), BAD), (dict(maxp=1 << 30), BAD),
    (dict(ws=0), BAD), (dict(ws=P + 20 * T + 8), BAD), (dict(wsb=-1), BAD), (dict(ws=P), BAD),
])
def test_paged_refusals(over, want):
    """B2 H8 H_kv 2 Nq3 d128 at distinct fake addresses, 64 pages of 16."""
    a = dict(q=P, kp=P + T, vp=P + 2 * T, fmt=1, nump=8, page=16, pt=P + 3 * T, maxp=64,
             kl=P + 6 * T, ql=0, o=P + 4 * T, lse=P + 5 * T, B=2, H=8, Hkv=2, Nq=3, d=128,
             scale=0.1, ws=P + 20 * T, wsb=1 << 40)
    a.update(over)
    need = ctypes.c_int64(0)
    rc = binding.lib().fa_fwd_paged_plan(2, 8, 2, 3, 128, 1, 16, 64, ctypes.byref(need))
    assert rc == OK
    if need.value == 0 and any(k in over for k in ("ws", "wsb")):
        pytest.skip("no workspace at this shape")
    rc = binding.lib().fa_fwd_paged(
        a["q"] or None, a["kp"] or None, a["vp"], a["fmt"], a["nump"], a["page"], a["pt"],
        a["maxp"], a["kl"] or None, a["ql"] or None, a["o"] or None, a["lse"], a["B"], a["H"],
        a["Hkv"], a["Nq"], a["d"], a["scale"], 1, a["ws"] or None, a["wsb"], None)
    assert rc == want


def test_status_string_of_a_bad_page():
    assert binding.status_string(binding.FA_ERR_PAGE).startswith("FA_ERR_PAGE")


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = types.SimpleNamespace(is_cuda=True)
    far = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7)
    near = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=7)
    assert binding._on(x, "x", near) == (0, 7)
    for call in (binding.osm_rope, binding.osm_rope_bwd):
        with pytest.raises(ValueError, match="stream is on"):
            call(x, None, stream=far)
    with pytest.raises(ValueError, match="stream is on"):
        binding.fa_fwd_paged(x, None, None, None, None, stream=far)


@pytest.mark.parametrize("over, ok", [
    (dict(B=1 << 16, H=1 << 8, Hkv=1 << 8, Nq=1 << 7), False),   # 2^31 rows
    (dict(H=1 << 20, Hkv=1 << 20, Nq=256, maxp=1 << 26), False),  # 2^60 bytes a sequence read out
    (dict(H=1 << 13, Hkv=1 << 13, Nq=256, maxp=1 << 20), True),
    (dict(B=1 << 20, H=64, Hkv=8, maxp=1 << 26), False),          # 2^43 tiles
])
def test_plan_of_sizes_past_the_counters(over, ok):
    a = dict(B=1, H=8, Hkv=8, Nq=1, d=64, page=16, maxp=4)
    a.update(over)
    args = a["B"], a["H"], a["Hkv"], a["Nq"], a["d"], "int4", a["page"], a["maxp"]
    if ok:
        assert 0 < binding.paged_plan(*args) < 1 << 60
        return
    with pytest.raises(binding.FaError) as e:
        binding.paged_plan(*args)
    assert e.value.status == UNSUP


def test_plan_and_page_bytes_refusals():
    with pytest.raises(binding.FaError):
        binding.paged_plan(1, 8, 3, 1, 128, "int4", 16, 10)
    with pytest.raises(binding.FaError):
        binding.paged_plan(1, 8, 2, 1, 80, "int4", 16, 10)
    assert binding.paged_plan(0, 8, 2, 1, 128, "int4", 16, 10) == 0
    assert binding.kv_page_bytes("bf16", 16, 64) == 16 * 64 * 2
    assert binding.kv_page_bytes("int4", 32, 128) == 32 * (64 + 4)
    for bad in (("int4", 8, 128), ("int4", 1040, 128), ("bf16", 16, 96)):
        with pytest.raises(binding.FaError):
            binding.kv_page_bytes(*bad)


def test_wrappers_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    t = torch.zeros(32, dtype=torch.int64)
    with pytest.raises(TypeError):
        binding.osm_rope(x, t)
    with pytest.raises(TypeError):
        binding.osm_rope(x.half(), t)
    with pytest.raises(TypeError):
        binding.fa_fwd_paged(x, x, x, t, t)
    with pytest.raises(TypeError):
        binding.osm_kv_append(x, x, x, x, t, t)
    with pytest.raises(ValueError):
        binding.rope_rates(64, scaling="other")


def test_rates():
    assert binding.rope_rates(8) == [1.0, 0.1, 0.01, 0.001]
    plain = binding.rope_rates(64, base=500.0)
    assert binding.rope_rates(64, base=500.0, scaling="linear", factor=4.0) == \
        [r / 4 for r in plain]
    other = binding.rope_rates(64, base=500.0, scaling="base", factor=4.0)
    assert other[0] == 1.0 and other[-1] == pytest.approx(plain[-1] / 4, rel=1e-14)
    bands = binding.rope_rates(64, base=500.0, scaling="bands", factor=4.0, orig_len=100.0,
                               low=1.0, high=8.0)
    for r, b in zip(plain, bands):
        turns = 100 * r / (2 * math.pi)
        w = min(1.0, max(0.0, (turns - 1) / 7))
        assert b == pytest.approx(r * w + r / 4 * (1 - w), rel=1e-15)
    for bad in (dict(rot_dim=0), dict(rot_dim=5), dict(rot_dim=8, base=0.0),
                dict(rot_dim=8, base=math.inf), dict(rot_dim=8, scaling="linear", factor=0.5),
                dict(rot_dim=2, scaling="base", factor=2.0),
                dict(rot_dim=8, scaling="bands", factor=2.0),
                dict(rot_dim=8, scaling="bands", factor=2.0, orig_len=9.0, low=2.0, high=2.0)):
        with pytest.raises(binding.FaError):
            binding.rope_rates(**bad)


def test_table():
    t = binding.rope_table([0.0, 1.0, math.pi, 7.5], device="cpu")
    turns = [x / (2 * math.pi) % 1.0 for x in (0.0, 1.0, math.pi, 7.5)]
    for got, want in zip(t.tolist(), turns):
        assert (got % (1 << 64)) / 2.0 ** 64 == pytest.approx(want, abs=2.0 ** -52)
    for bad in ([-1.0], [math.nan], [math.inf]):
        with pytest.raises(binding.FaError):
            binding.rope_table(bad, device="cpu")


def test_restatement_of_the_quantiser():
    """Every code of every group lies within half a step, steps have three significant bits, the
    values are bf16 numbers, and a smaller step would not do."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 128)) * np.exp(rng.uniform(-20, 20, (50, 1))) + \
        rng.standard_normal((50, 1)) * 3
    x[3] = 5.0
    x[4] = 0.0
    codes, s, b = ref.quantise(x)
    back = ref.stored(x)
    assert codes.min() >= 0 and codes.max() <= 15 and np.abs(b).max() <= 31
    assert np.all(np.abs(back - x) <= np.repeat(s, 64, -1) / 2 * (1 + 1e-12))
    m, _ = np.frexp(s)
    assert np.array_equal(m * 8, np.rint(m * 8))
    assert np.array_equal(torch.tensor(back).to(torch.bfloat16).double().numpy(), back)
    g = x.reshape(50, 2, 64)
    need = np.maximum((g.max(-1) - g.min(-1)) / 15, np.abs(g.min(-1)) / 31)
    assert np.all(s >= need) and np.all(s <= need * 1.25 * (1 + 1e-12))
    raw = ref.head_bytes(x.reshape(1, 50, 128)[:, :48])
    assert raw.shape == (1, 48 * 68)
    assert np.array_equal(ref.head_values(raw, 48, 128)[0], back[:48])
