"""What the rotating append and the FP8 cache's entry points refuse on the
host, before anything is enqueued (no GPU needed), and the reference's own
rounding against torch's."""

import ctypes

import pytest
import torch

import paged_kv_cache_386_b200 as pkv
from paged_kv_cache_386_b200 import build as pkv_build
from tests import fp8_reference as ref

INVALID, UNSUPPORTED = 1, 2
P = 256  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv._load()


def rope(lib, entry="paged_kv_append_rope", q=P, qs=1024, k=P, ks=256, v=P, vs=256, pos=P, tab=P, maxp=64, rot=128,
         inter=0, slots=P, n=4, kc=P, vc=P, nb=8, bs=16, nq=8, nkv=2, d=128, out=512, outs=1024, dtype=2):
    return getattr(lib, entry)(q, qs, k, ks, v, vs, pos, tab, maxp, rot, inter, slots, n, kc, vc, nb, bs, nq, nkv, d,
                               out, outs, dtype, None)


@pytest.mark.parametrize("entry", ["paged_kv_append_rope", "paged_kv_append_rope_fp8"])
@pytest.mark.parametrize("bad,status", [
    (dict(n=-1), INVALID), (dict(nb=0), INVALID), (dict(nkv=0), INVALID), (dict(d=0), INVALID), (dict(nq=-1), INVALID),
    (dict(rot=0), INVALID), (dict(rot=144), INVALID), (dict(rot=8), UNSUPPORTED), (dict(d=120, rot=16), UNSUPPORTED),
    (dict(inter=2), INVALID), (dict(q=None), INVALID), (dict(nq=0), INVALID), (dict(out=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(pos=None), INVALID), (dict(tab=None), INVALID),
    (dict(maxp=0), INVALID), (dict(slots=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(q=264), INVALID), (dict(k=264), INVALID), (dict(tab=260), INVALID), (dict(pos=260), INVALID),
    (dict(slots=260), INVALID), (dict(out=520), INVALID), (dict(kc=264), INVALID), (dict(qs=1028), INVALID),
    (dict(ks=-256), INVALID), (dict(vs=2), INVALID), (dict(outs=512), INVALID), (dict(out=P, outs=2048), INVALID),
    (dict(bs=32), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(n=1 << 30), UNSUPPORTED),
])
def test_rotating_appends(lib, entry, bad, status):
    assert rope(lib, entry, **bad) == status


def test_no_tokens_is_no_work(lib):
    for entry in ("paged_kv_append_rope", "paged_kv_append_rope_fp8"):
        assert rope(lib, entry, n=0, k=None, v=None, pos=None, slots=None) == 0
    assert lib.paged_kv_append_fp8(None, 0, None, 0, 2, None, 0, None, None, 8, 16, 2, 128, None) == 0
    assert lib.paged_kv_copy_blocks_fp8(None, None, None, None, 0, 8, 16, 2, 128, None) == 0


def test_head_sizes_of_the_fp8_cache(lib):
    assert rope(lib, "paged_kv_append_rope_fp8", d=96, rot=96) == UNSUPPORTED
    assert rope(lib, "paged_kv_append_rope_fp8", vc=260) == INVALID  # scales: 8-byte aligned
    f = lib.paged_kv_append_fp8
    assert f(P, 256, P, 256, 2, P, 4, P, P, 8, 16, 2, 96, None) == UNSUPPORTED
    assert f(P, 256, P, 256, 7, P, 4, P, P, 8, 16, 2, 128, None) == UNSUPPORTED
    assert f(P, 256, P, 256, 2, P, 4, P, None, 8, 16, 2, 128, None) == INVALID
    assert f(P, 256, P, 257, 2, P, 4, P, P, 8, 16, 2, 128, None) == INVALID
    g = lib.paged_kv_copy_blocks_fp8
    assert g(P, P, P, P, -1, 8, 16, 2, 128, None) == INVALID
    assert g(P, P, P, P, 2, 8, 16, 2, 80, None) == UNSUPPORTED
    assert g(P, 260, P, P, 2, 8, 16, 2, 128, None) == INVALID
    assert g(P, P, 258, P, 2, 8, 16, 2, 128, None) == INVALID
    assert g(P, P, None, P, 2, 8, 16, 2, 128, None) == INVALID


def decode(lib, q=P, kv=P, sc=P, bt=P, maxb=4, cl=P, b=2, ql=1, nb=8, scale=0.1, nq=8, nkv=2, d=128, bs=16, out=P,
           dtype=2):
    return lib.paged_attention_decode_fp8(q, kv, sc, bt, maxb, cl, b, ql, nb, scale, nq, nkv, d, bs, out, dtype, None,
                                          0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INVALID), (dict(kv=None), INVALID), (dict(sc=None), INVALID), (dict(bt=None), INVALID),
    (dict(cl=None), INVALID), (dict(out=None), INVALID), (dict(q=264), INVALID), (dict(kv=264), INVALID),
    (dict(sc=260), INVALID), (dict(bt=257), INVALID), (dict(out=264), INVALID), (dict(b=-1), INVALID),
    (dict(maxb=0), INVALID), (dict(nb=0), INVALID), (dict(nq=7), INVALID), (dict(ql=0), INVALID),
    (dict(ql=17), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED),
    (dict(dtype=9), UNSUPPORTED), (dict(b=4097), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(b=4096, maxb=1 << 20), UNSUPPORTED),
])
def test_decode(lib, bad, status):
    assert decode(lib, **bad) == status


@pytest.mark.parametrize("bad", [dict(num_units=1), dict(force_simt=1), dict(balance_chunks=1), dict(static_permille=800),
                                 dict(wait_limit_us=-1), dict(test_withhold_unit=-1), dict(reserved=1)])
def test_decode_options(lib, bad):
    opts = pkv._Options()
    for name, value in bad.items():
        if name == "reserved":
            opts.reserved[1] = value
        else:
            setattr(opts, name, value)
    f = lib.paged_attention_decode_fp8_ex
    for batch in (2, 0):
        assert f(P, P, P, P, 4, P, batch, 1, 8, 0.1, 8, 2, 128, 16, P, 2, None, 0, None, ctypes.byref(opts)) == INVALID
    assert f(P, P, P, P, 4, P, 0, 1, 8, 0.1, 8, 2, 128, 16, P, 2, None, 0, None, ctypes.byref(pkv._Options(wait_limit_us=5))) == 0
    assert f(P, P, P, P, 4, P, 0, 1, 8, 0.1, 8, 2, 128, 16, P, 2, None, 0, None, None) == 0


def test_decode_of_no_sequence_and_workspace_size(lib):
    assert decode(lib, b=0) == 0
    n = ctypes.c_size_t()
    f = lib.paged_attention_fp8_workspace_size
    assert f(2, 1, 8, 2, 128, None) == INVALID
    assert f(2, 0, 8, 2, 128, ctypes.byref(n)) == INVALID
    assert f(2, 1, 7, 2, 128, ctypes.byref(n)) == INVALID
    assert f(-1, 1, 8, 2, 128, ctypes.byref(n)) == INVALID
    assert f(2, 17, 8, 2, 128, ctypes.byref(n)) == UNSUPPORTED
    assert f(4097, 1, 8, 2, 128, ctypes.byref(n)) == UNSUPPORTED
    assert f(2, 1, 8, 2, 96, ctypes.byref(n)) == UNSUPPORTED


def test_binding_checks_before_any_call():
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pos = slots = torch.zeros(4, dtype=torch.int64)
    tab = torch.zeros(8, 128)
    kc = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    kv = torch.zeros(3, 2, 2, 16, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones(3, 2, 2)

    def rope(k=k, v=k, pos=pos, tab=tab, slots=slots, kc=kc, vc=kc, **kw):
        pkv.paged_kv_append_rope(k, v, pos, tab, slots, kc, vc, **kw)

    for bad in (dict(v=k.half()), dict(v=k[:, :1]), dict(pos=pos.int()), dict(pos=pos[:3]), dict(tab=tab.half()),
                dict(slots=slots[:2]), dict(kc=kc.half()), dict(vc=kc[:2]), dict(q=q.half()), dict(q=q[:3]),
                dict(q_out=q), dict(q=q, q_out=q[:, :2]), dict(block_size=32), dict(q=q[..., ::2])):
        with pytest.raises(ValueError):
            rope(**bad)
    with pytest.raises(ValueError):
        rope()  # CPU tensors
    for bad in ((k.double(), k.double(), slots, kv, sc), (k, k, slots, kv.view(torch.uint8), sc),
                (k, k, slots, kv, sc.half()), (k, k, slots, kv, sc[:2]), (k[:, :1], k[:, :1], slots, kv, sc),
                (k, k, slots, kv, sc)):
        with pytest.raises(ValueError):
            pkv.paged_kv_append_fp8(*bad)
    bt, cl = torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    for bad in ((q, kv, sc, bt.long(), cl), (q, kv, sc, bt[:3], cl), (q, kv, sc, bt, cl[:2]), (q[..., :64], kv, sc, bt, cl),
                (q[0], kv, sc, bt, cl), (q, kc, sc, bt, cl)):
        with pytest.raises(ValueError):
            pkv.paged_attention_decode_fp8(*bad, 0.1)
    for out in (torch.zeros_like(q).half(), torch.zeros(4, 8, 64, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="out"):
            pkv.paged_attention_decode_fp8(q, kv, sc, bt, cl, 0.1, out=out)
    with pytest.raises(ValueError):
        pkv.rotary_table(0, 64)
    with pytest.raises(ValueError):
        pkv.rotary_table(8, 7)


def test_rotary_table_rows():
    t = pkv.rotary_table(100, 8, 100.0, device="cpu").double()
    for p in (0, 1, 99):
        for j in range(4):
            a = torch.tensor(p * 100.0 ** (-2 * j / 8), dtype=torch.float64)
            assert abs(t[p, j] - a.cos()) <= 2.0 ** -24 and abs(t[p, 4 + j] - a.sin()) <= 2.0 ** -24


def test_reference_rounding_is_torchs_nearest_even():
    x = torch.cat((torch.linspace(-460, 460, 4001), torch.linspace(-0.03, 0.03, 2001),
                   torch.tensor([448.0, 464.0, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875, 0.0])))
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).float().double()
    assert torch.equal(ref.e4m3_all(x), want)
    assert [ref.e4m3(v) for v in x.tolist()] == want.tolist()
