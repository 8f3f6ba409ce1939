"""paged_kv_append_rope on the GPU: against the rotation in 64 bits with a
derived bound, and bit for bit against separately rounded fp32 steps."""

import pytest
import torch

import paged_kv_cache_386_b200 as pkv
from tests import fp8_reference as ref
from tests.gpu_helpers import bits

pytestmark = pytest.mark.gpu


def make(tokens, n_q, n_kv, d, rot, dtype, seed, packed=False, max_pos=4096):
    g = torch.Generator().manual_seed(seed)
    if packed:
        rows = (torch.randn((tokens, (n_q + 2 * n_kv) * d), generator=g) * 2).to(dtype).cuda()
        q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split((n_q * d, n_kv * d, n_kv * d), 1))
    else:
        q, k, v = ((torch.randn((tokens, h, d), generator=g) * 2).to(dtype).cuda() for h in (n_q, n_kv, n_kv))
    blocks = (tokens + 15) // 16 + 3
    slots = torch.randperm(blocks * 16, generator=g)[:tokens]
    pos = torch.randint(0, max_pos, (tokens,), generator=g)
    table = pkv.rotary_table(max_pos, rot, 10000.0, device="cpu")
    kc, vc = (torch.randn((blocks, n_kv, 16, d), generator=g).to(dtype) for _ in range(2))
    return q, k, v, slots, pos, table, kc, vc


def check(tokens, n_q, n_kv, d, rot, dtype, interleaved, seed=0, packed=False, in_place=False, pad=()):
    q, k, v, slots, pos, table, kc, vc = make(tokens, n_q, n_kv, d, rot, dtype, seed, packed)
    for i in pad:
        slots[i] = -1
    kd, vd = kc.cuda(), vc.cuda()
    q0, k0, v0 = q.cpu(), k.cpu(), v.cpu()
    got = pkv.paged_kv_append_rope(k, v, pos.cuda(), table.cuda(), slots.cuda(), kd, vd, q=q,
                                   q_out=q if in_place else None, interleaved=interleaved)
    assert pkv.pkv_get_device_error() == 0
    if in_place:
        assert got.data_ptr() == q.data_ptr()
    else:
        assert torch.equal(bits(q.cpu()), bits(q0))
    assert torch.equal(bits(k.cpu()), bits(k0)) and torch.equal(bits(v.cpu()), bits(v0))
    want_q = ref.rotate32(q0, table, pos, interleaved).to(dtype)
    want_k = ref.rotate32(k0, table, pos, interleaved).to(dtype)
    keep = slots >= 0
    kc[slots[keep] // 16, :, slots[keep] % 16] = want_k[keep]
    vc[slots[keep] // 16, :, slots[keep] % 16] = v0[keep]
    assert torch.equal(bits(got.cpu()), bits(want_q))
    assert torch.equal(bits(kd.cpu()), bits(kc)) and torch.equal(bits(vd.cpu()), bits(vc))
    # Two products and their sum in fp32 (2^-24 each), then half a step of the type.
    exact, mag = ref.rotate64(q0, table, pos, interleaved)
    tol = 2 * mag * 2.0 ** -23 + exact.abs() * torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -10) + 2.0 ** -25
    assert ((got.cpu().double() - exact).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n_q,n_kv,d,rot", [(8, 2, 128, 128), (3, 3, 64, 64), (5, 1, 64, 32), (12, 4, 128, 16),
                                            (7, 7, 80, 48), (2, 1, 16, 16), (33, 3, 256, 256)])
def test_shapes(dtype, interleaved, n_q, n_kv, d, rot):
    check(45, n_q, n_kv, d, rot, dtype, interleaved, seed=d + rot, pad=(0, 7, 44))


@pytest.mark.parametrize("tokens", [1, 2, 255, 1031, 5000])
def test_lengths_and_packed_views(tokens):
    check(tokens, 8, 2, 128, 64, torch.bfloat16, False, seed=tokens, packed=True)


@pytest.mark.parametrize("packed", [False, True])
def test_in_place_queries(packed):
    check(77, 6, 2, 128, 128, torch.float16, True, seed=3, packed=packed, in_place=True)


def test_without_queries_and_no_tokens():
    _, k, v, slots, pos, table, kc, vc = make(9, 4, 2, 64, 64, torch.bfloat16, 4)
    kd, vd = kc.cuda(), vc.cuda()
    assert pkv.paged_kv_append_rope(k, v, pos.cuda(), table.cuda(), slots.cuda(), kd, vd) is None
    kc[slots // 16, :, slots % 16] = ref.rotate32(k.cpu(), table, pos, False).bfloat16()
    assert torch.equal(bits(kd.cpu()), bits(kc))
    out = pkv.paged_kv_append_rope(k[:0], v[:0], pos[:0].cuda(), table.cuda(), slots[:0].cuda(), kd, vd, q=k[:0])
    assert out.shape == (0, 2, 64) and torch.equal(bits(kd.cpu()), bits(kc))


def test_bad_positions_and_slots_are_left_out_and_flagged():
    q, k, v, slots, pos, table, kc, vc = make(20, 4, 2, 128, 128, torch.bfloat16, 5)
    pos[3], pos[11], slots[6] = -1, table.shape[0], kc.shape[0] * 16
    kd, vd = kc.cuda(), vc.cuda()
    q_out = torch.full_like(q, 7.0)
    pkv.paged_kv_append_rope(k, v, pos.cuda(), table.cuda(), slots.cuda(), kd, vd, q=q, q_out=q_out)
    assert pkv.pkv_get_device_error() == pkv.DEVERR_POSITION | pkv.DEVERR_SLOT
    ok = torch.ones(20, dtype=torch.bool)
    ok[[3, 11]] = False
    want = torch.full_like(q.cpu(), 7.0)
    want[ok] = ref.rotate32(q.cpu()[ok], table, pos[ok], False).bfloat16()
    assert torch.equal(bits(q_out.cpu()), bits(want))
    ok[6] = False
    kc[slots[ok] // 16, :, slots[ok] % 16] = ref.rotate32(k.cpu()[ok], table, pos[ok], False).bfloat16()
    vc[slots[ok] // 16, :, slots[ok] % 16] = v.cpu()[ok]
    assert torch.equal(bits(kd.cpu()), bits(kc)) and torch.equal(bits(vd.cpu()), bits(vc))


def test_infinities_and_nan_stay_in_their_pair():
    q, k, v, slots, pos, table, kc, vc = make(4, 2, 1, 64, 64, torch.float16, 6)
    q[1, 0, 5], q[2, 1, 40] = float("inf"), float("nan")
    v[0, 0, 3] = float("nan")
    kd, vd = kc.cuda(), vc.cuda()
    got = pkv.paged_kv_append_rope(k, v, pos.cuda(), table.cuda(), slots.cuda(), kd, vd, q=q).cpu()
    want = ref.rotate32(q.cpu(), table, pos, False).half()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
    assert int((~got.isfinite()).sum()) == 4
    assert torch.equal(bits(vd.cpu()[slots[0] // 16, 0, slots[0] % 16]), bits(v.cpu()[0, 0]))


def test_graph_replay_and_other_stream():
    q, k, v, slots, pos, table, kc, vc = make(33, 8, 2, 128, 128, torch.bfloat16, 7)
    kd, vd, t, p, s = kc.cuda(), vc.cuda(), table.cuda(), pos.cuda(), slots.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = pkv.paged_kv_append_rope(k, v, p, t, s, kd, vd, q=q, stream=side)
    side.synchronize()
    eager = out.cpu()
    q_out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_kv_append_rope(k, v, p, t, s, kd, vd, q=q, q_out=q_out)
    kd.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(q_out.cpu()), bits(eager))
    assert torch.equal(bits(kd.cpu()[slots // 16, :, slots % 16]),
                       bits(ref.rotate32(k.cpu(), table, pos, False).bfloat16()))
