"""Long calls of the rotating append and of the FP8 append, where a thread walks
several heads and a pair of warps several runs: bit for bit against plain fp32
steps, and against the same tokens in calls too small for that."""

import pytest
import torch

import paged_kv_cache_386_b200 as pkv
from tests import fp8_reference as ref
from tests.gpu_helpers import bits

pytestmark = pytest.mark.gpu


def heads_per_thread(tokens, heads, d):
    """The launch rule: as many as leave a thread for every one the device holds."""
    want = torch.cuda.get_device_properties(0).multi_processor_count * 2048
    return next((n for n in (8, 4, 2) if tokens * (d // 16) * -(-heads // n) >= want), 1)


def inputs(n, n_q, n_kv, d, dtype, seed, packed=True):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((n, (n_q + 2 * n_kv) * d), generator=g, device="cuda").to(dtype)
    parts = x.split((n_q * d, n_kv * d, n_kv * d), 1)
    q, k, v = (y.unflatten(1, (-1, d)) if packed else y.unflatten(1, (-1, d)).contiguous() for y in parts)
    return q, k, v, torch.randint(0, 4096, (n,), generator=g, device="cuda")


# Head counts that the heads of a thread do not divide, so that threads cross from queries to keys to
# values and the last group is short; several heads a thread: 2 (about), 4 and 8.
@pytest.mark.parametrize("n,n_q,n_kv,d,per_thread", [(5000, 17, 5, 128, 2), (4001, 33, 5, 128, 4), (8192, 33, 5, 128, 8),
                                                     (8192, 71, 5, 128, 8), (6007, 64, 64, 64, 8), (9001, 21, 3, 256, 8)])
@pytest.mark.parametrize("dtype,interleaved,rot,in_place", [(torch.bfloat16, False, 1.0, False), (torch.float16, True, 0.5, True),
                                                            (torch.float32, False, 0.25, True)])
def test_rotating_append(n, n_q, n_kv, d, per_thread, dtype, interleaved, rot, in_place):
    assert heads_per_thread(n, n_q + 2 * n_kv, d) == per_thread
    q, k, v, pos = inputs(n, n_q, n_kv, d, dtype, n + n_q, packed=in_place)
    table = pkv.rotary_table(4096, int(d * rot))
    blocks = n // 16 + 3
    slots = torch.randperm(blocks * 16, generator=torch.Generator().manual_seed(n)).cuda()[:n]
    slots[::97] = -1
    kc, vc = (torch.randn((blocks, n_kv, 16, d), device="cuda").to(dtype) for _ in range(2))
    q0, k0, v0, want_k, want_v = q.clone(), k.clone(), v.clone(), kc.clone(), vc.clone()
    got = pkv.paged_kv_append_rope(k, v, pos, table, slots, kc, vc, q=q, q_out=q if in_place else None, interleaved=interleaved)
    assert pkv.pkv_get_device_error() == 0
    keep = slots >= 0
    turned = rotate(k0, table, pos, interleaved)
    want_k[slots[keep] // 16, :, slots[keep] % 16] = turned[keep]
    want_v[slots[keep] // 16, :, slots[keep] % 16] = v0[keep]
    assert torch.equal(bits(got), bits(rotate(q0, table, pos, interleaved)))
    assert torch.equal(bits(kc), bits(want_k)) and torch.equal(bits(vc), bits(want_v))
    assert torch.equal(bits(k), bits(k0)) and torch.equal(bits(v), bits(v0))
    if not in_place:
        assert torch.equal(bits(q), bits(q0))


def rotate(x, table, pos, interleaved):
    """In fp32, every product and sum rounded by itself, the result once to the type."""
    return ref.rotate32(x, table, pos, interleaved).to(x.dtype)


def ragged(n, seed):
    """Prompts of 1 to 300 tokens that begin somewhere in a block, a padding token behind every seventh: block
    and offset of each token, blocks in any order."""
    g = torch.Generator().manual_seed(seed)
    at, used = [], 0
    while len(at) < n:
        first, length = int(torch.randint(0, 16, (), generator=g)), int(torch.randint(1, 301, (), generator=g))
        at += [used * 16 + first + i for i in range(length)]
        used += (first + length + 15) // 16
        if used % 7 == 0:
            at.append(-1)
    slots = torch.tensor(at[:n])
    place = torch.randperm(used, generator=g)
    return torch.where(slots < 0, slots, place[slots.clamp(min=0) // 16] * 16 + slots.clamp(min=0) % 16), used


def single_tokens(n, seed):
    """One token each of n sequences: a block of its own for every token of the call."""
    g = torch.Generator().manual_seed(seed)
    slots = torch.randperm(n, generator=g) * 16 + torch.randint(0, 16, (n,), generator=g)
    slots[torch.randperm(n, generator=g)[: n // 50]] = -1
    return slots, n


def append(kind, k, v, q, pos, table, slots, kv, scales):
    interleaved = kind == "neighbours"
    if kind == "plain":
        return pkv.paged_kv_append_fp8(k, v, slots, kv, scales)
    return pkv.paged_kv_append_rope_fp8(k, v, pos, table, slots, kv, scales, q=q, interleaved=interleaved)


@pytest.mark.parametrize("plan", [ragged, single_tokens])
@pytest.mark.parametrize("n,n_q,n_kv,d,rot", [(3001, 8, 2, 128, 128), (2600, 40, 5, 128, 64), (4099, 24, 3, 64, 64),
                                              (700, 96, 32, 64, 32), (5003, 40, 10, 128, 128)])
@pytest.mark.parametrize("dtype,kind", [(torch.bfloat16, "halves"), (torch.float16, "neighbours"), (torch.float32, "halves"),
                                        (torch.float16, "plain"), (torch.float32, "neighbours"), (torch.bfloat16, "plain")])
def test_fp8_append_in_one_call_and_in_small_ones(plan, n, n_q, n_kv, d, rot, dtype, kind):
    """Sixteen tokens to a pair of warps against one, cut between blocks."""
    limit = 16 * torch.cuda.get_device_properties(0).multi_processor_count  # tokens x kv heads of the other split
    assert n * n_kv > limit
    q, k, v, pos = inputs(n, n_q, n_kv, d, dtype, n + d)
    slots, blocks = plan(n, n)
    table = pkv.rotary_table(4096, rot)
    g = torch.Generator("cuda").manual_seed(9)
    kv, scales = pkv.fp8_cache(blocks, n_kv, d)
    kv.copy_((torch.randn(kv.shape, generator=g, device="cuda") * 120).clamp(-448, 448).to(kv.dtype))
    scales.copy_(2.0 ** torch.randint(-12, -4, scales.shape, generator=g, device="cuda"))
    kv1, scales1, slots_d = kv.clone(), scales.clone(), slots.cuda()
    got = append(kind, k, v, q, pos, table, slots_d, kv, scales)
    step, at, outs = limit // n_kv, 0, []
    while at < n:
        to = min(n, at + step)
        while to < n and slots[to] >= 0 and slots[to] // 16 == slots[to - 1] // 16:
            to -= 1  # a block's tokens stay in one call
        outs.append(append(kind, k[at:to], v[at:to], q[at:to], pos[at:to], table, slots_d[at:to], kv1, scales1))
        at = to
    assert pkv.pkv_get_device_error() == 0
    assert torch.equal(scales, scales1) and torch.equal(kv.view(torch.uint8), kv1.view(torch.uint8))
    if kind != "plain":
        assert torch.equal(bits(got), bits(torch.cat(outs)))
        assert torch.equal(bits(got), bits(rotate(q, table, pos, kind == "neighbours")))


@pytest.mark.parametrize("plan,n,n_kv,dtype,kind", [(ragged, 1500, 2, torch.bfloat16, "halves"), (single_tokens, 600, 4, torch.float16, "plain"),
                                                    (ragged, 1200, 2, torch.float32, "neighbours"), (single_tokens, 1200, 2, torch.float32, "halves")])
def test_fp8_append_of_many_runs_follows_the_definition(plan, n, n_kv, dtype, kind):
    q, k, v, pos = inputs(n, 2 * n_kv, n_kv, 128, dtype, n)
    assert n * n_kv > 16 * torch.cuda.get_device_properties(0).multi_processor_count
    slots, blocks = plan(n, n)
    table = pkv.rotary_table(4096, 128)
    kv, scales = pkv.fp8_cache(blocks, n_kv, 128)
    scales.fill_(2.0 ** -8)
    kv.copy_((torch.randn(kv.shape, device="cuda") * 100).clamp(-448, 448).to(kv.dtype))
    values, want = kv.cpu().float().double(), scales.cpu().double()
    append(kind, k, v, q, pos, table, slots.cuda(), kv, scales)
    assert pkv.pkv_get_device_error() == 0
    kf = k.cpu().float() if kind == "plain" else ref.rotate32(k.cpu(), table.cpu(), pos.cpu(), kind == "neighbours")
    ref.append(values, want, kf, v.cpu().float(), slots, blocks)
    assert torch.equal(scales.cpu().double(), want)
    assert torch.equal(kv.cpu().float().double(), values)
