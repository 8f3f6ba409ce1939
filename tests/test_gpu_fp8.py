"""The FP8 paged cache on the GPU: its append (codes and scales exactly as the
definition gives them), copy-on-write and decode attention against 64 bits."""

import pytest
import torch

import paged_kv_cache_386_b200 as pkv
from tests import fp8_reference as ref
from tests.gpu_helpers import bits

pytestmark = pytest.mark.gpu


def host(kv, scales):
    return kv.cpu().float().double(), scales.cpu().double()


def random_cache(blocks, n_kv, d, seed, spread=3):
    g = torch.Generator().manual_seed(seed)
    kv, scales = pkv.fp8_cache(blocks, n_kv, d)
    codes = (torch.randn(kv.shape, generator=g) * 120).clamp(-448, 448)
    kv.copy_(codes.to(torch.float8_e4m3fn))
    scales.copy_(2.0 ** torch.randint(-8 - spread, -8 + spread, scales.shape, generator=g).float())
    return kv, scales


def same_cache(kv, scales, values, want_scales):
    got, got_scales = host(kv, scales)
    assert torch.equal(got_scales, want_scales)
    assert torch.equal(got.isnan(), values.isnan())
    assert torch.equal(got.nan_to_num(), values.nan_to_num())


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------

def append_case(plan, n_kv, d, dtype, seed, rot=0, interleaved=False, n_q=0, packed=False):
    """`plan`: (block, offset) of every token in call order, None for padding."""
    g = torch.Generator().manual_seed(seed)
    blocks = 12
    kv, scales = random_cache(blocks, n_kv, d, seed)
    n = len(plan)
    size = torch.exp2(torch.randint(-6, 7, (n, 1), generator=g).float())
    rows = (torch.randn((n, (n_q + 2 * n_kv) * d), generator=g) * size).to(dtype).cuda()
    if packed:
        q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split((n_q * d, n_kv * d, n_kv * d), 1))
    else:
        q, k, v = (x.unflatten(1, (-1, d)).contiguous() for x in rows.split((n_q * d, n_kv * d, n_kv * d), 1))
    slots = torch.tensor([-1 if x is None else x[0] * 16 + x[1] for x in plan], dtype=torch.int64)
    values, want_scales = host(kv, scales)
    kf, vf = k.cpu().float(), v.cpu().float()
    if rot:
        table, pos = pkv.rotary_table(512, rot, device="cpu"), torch.randint(0, 512, (n,), generator=g)
        kf = ref.rotate32(kf, table, pos, interleaved)
        got = pkv.paged_kv_append_rope_fp8(k, v, pos.cuda(), table.cuda(), slots.cuda(), kv, scales,
                                           q=q if n_q else None, interleaved=interleaved)
        if n_q:
            assert torch.equal(bits(got.cpu()), bits(ref.rotate32(q.cpu(), table, pos, interleaved).to(dtype)))
    else:
        pkv.paged_kv_append_fp8(k, v, slots.cuda(), kv, scales)
    assert pkv.pkv_get_device_error() == 0
    ref.append(values, want_scales, kf, vf, slots, blocks)
    same_cache(kv, scales, values, want_scales)


def run_of(block, lo, hi):
    return [(block, o) for o in range(lo, hi)]


PLANS = {
    "one": [(3, 0)],
    "one_inside": [(3, 9)],
    "step": [(4, 1), (0, 15), (7, 0), (2, 8), None, (11, 3)],
    "prompt": run_of(5, 0, 16) + run_of(2, 0, 16) + run_of(9, 0, 5),
    "middle": run_of(5, 13, 16) + run_of(2, 0, 16) + run_of(9, 0, 1),
    "padded": [None, None] + run_of(1, 2, 6) + [None] + run_of(0, 7, 8) + [None] * 40 + run_of(6, 0, 3),
    "backwards": list(reversed(run_of(5, 0, 16))) + list(reversed(run_of(3, 4, 11))),
    "same_slot": [(5, 2), (5, 2), (5, 4), (5, 2)] + [(8, 0)] * 40 + [(8, 1)],
    "many": sum((run_of(b, 0, 16) for b in (11, 3, 4, 10, 0, 1)), []) + run_of(2, 5, 13),
}


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("d", [64, 128])
def test_append_places(plan, d):
    append_case(PLANS[plan], 3, d, torch.bfloat16, seed=len(plan) + d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rot,interleaved,n_q", [(128, False, 8), (128, True, 4), (64, False, 0), (16, True, 12)])
def test_append_rotated(dtype, rot, interleaved, n_q):
    append_case(PLANS["middle"] + [None] + run_of(7, 3, 4), 4, 128, dtype, rot, rot, interleaved, n_q, packed=n_q > 0)


@pytest.mark.parametrize("rot,interleaved", [(64, False), (32, True), (16, False)])
def test_append_rotated_64(rot, interleaved):
    append_case(PLANS["padded"], 1, 64, torch.float16, rot, rot, interleaved, 5, packed=True)


def test_append_token_by_token_follows_the_definition():
    """A block filled one token at a time, magnitudes growing: scales grow, older codes are rounded again."""
    g = torch.Generator().manual_seed(11)
    kv, scales = random_cache(3, 2, 128, 12)
    values, want = host(kv, scales)
    for t in range(21):
        k, v = (torch.randn((1, 2, 128), generator=g) * 1.6 ** t for _ in range(2))
        slot = torch.tensor([(2 if t < 16 else 0) * 16 + t % 16])
        pkv.paged_kv_append_fp8(k.cuda(), v.cuda(), slot.cuda(), kv, scales)
        ref.append(values, want, k, v, slot, 3)
        same_cache(kv, scales, values, want)


def test_append_borders_of_scales_and_codes():
    """Magnitudes at and next to 448 x 2^e, the smallest and largest scales, zeros, infinities, NaN."""
    up = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9)).item()
    tops = [448.0, up, 447.9, 224.0, 256.0, 1.75, up / 256, 0.0, 448 * 2.0 ** -48, 448 * 2.0 ** -49, 1e-40,
            448 * 2.0 ** 48, up * 2.0 ** 48, 3e38, float("inf"), float("nan")]
    k = torch.zeros((len(tops), 1, 64))
    for i, t in enumerate(tops):
        k[i, 0, 0], k[i, 0, 7] = t, -t
        k[i, 0, 1:6] = torch.tensor([0.5, -1.0, 17 / 16, 2.0 ** -9, 3 * 2.0 ** -10]) * (t if 0 < t < 1e30 else 1.0)
    slots = torch.arange(len(tops)) * 16
    kv, scales = pkv.fp8_cache(len(tops), 1, 64)
    values, want = host(kv, scales)
    pkv.paged_kv_append_fp8(k.cuda(), k.flip(0).cuda(), slots.cuda(), kv, scales)
    ref.append(values, want, k, k.flip(0), slots, len(tops))
    same_cache(kv, scales, values, want)


def test_append_leaves_out_bad_slots_and_positions():
    kv, scales = random_cache(4, 2, 128, 13)
    values, want = host(kv, scales)
    g = torch.Generator().manual_seed(14)
    k, v = (torch.randn((12, 2, 128), generator=g) for _ in range(2))
    slots = torch.tensor([0, 1, 2, 64, -1, 35, 36, 37, 38, 39, 1 << 40, 20])
    pos = torch.arange(12)
    pos[[1, 7]] = torch.tensor([-5, 600])
    table = pkv.rotary_table(600, 128, device="cpu")
    pkv.paged_kv_append_rope_fp8(k.cuda(), v.cuda(), pos.cuda(), table.cuda(), slots.cuda(), kv, scales)
    assert pkv.pkv_get_device_error() == pkv.DEVERR_SLOT | pkv.DEVERR_POSITION
    ref.append(values, want, ref.rotate32(k, table, pos.clamp(0, 599), False), v, slots, 4, left_out=(1, 7))
    same_cache(kv, scales, values, want)


@pytest.mark.parametrize("many", [False, True])  # a token or sixteen to each pair of warps
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("first,count", [(0, 1), (3, 1), (14, 1), (15, 2), (16, 3), (1, 17), (5, 40), (30, 70)])
def test_append_slots_beyond_the_pool_inside_a_block(first, count, rotated, many):
    """`count` bad slots at every place `first` of a stretch: the block's tokens on both sides are one run."""
    g = torch.Generator().manual_seed(first + count)
    n_kv, blocks = (40, 12) if many else (2, 12)
    pos = torch.arange(5, 5 + 70)
    slots = torch.randperm(blocks, generator=g)[pos // 16] * 16 + pos % 16
    bad = blocks * 16 + torch.randint(0, 1 << 40, (count,), generator=g)
    slots = torch.cat((slots[:first], bad, slots[first:], bad[:1]))
    n = len(slots)
    assert (n * n_kv > 16 * torch.cuda.get_device_properties(0).multi_processor_count) == many
    size = torch.exp2(torch.randint(-6, 7, (n, 1, 1), generator=g).float())
    k, v = (torch.randn((n, n_kv, 64), generator=g) * size for _ in range(2))
    kv, scales = random_cache(blocks, n_kv, 64, first)
    values, want = host(kv, scales)
    kf = k
    if rotated:
        table, at = pkv.rotary_table(128, 64, device="cpu"), torch.randint(0, 128, (n,), generator=g)
        kf = ref.rotate32(k, table, at, False)
        pkv.paged_kv_append_rope_fp8(k.cuda(), v.cuda(), at.cuda(), table.cuda(), slots.cuda(), kv, scales)
    else:
        pkv.paged_kv_append_fp8(k.cuda(), v.cuda(), slots.cuda(), kv, scales)
    assert pkv.pkv_get_device_error() == pkv.DEVERR_SLOT
    ref.append(values, want, kf, v, slots, blocks)
    same_cache(kv, scales, values, want)


def test_append_long_prompts_and_one_token_warps_agree():
    """More tokens than one warp each can hold: the other split of the call into warps."""
    g = torch.Generator().manual_seed(15)
    n, n_kv, d = 3001, 4, 64
    blocks = 200
    place = torch.randperm(blocks, generator=g)
    pos = torch.arange(n) + 5
    slots = place[pos // 16] * 16 + pos % 16
    k, v = (torch.randn((n, n_kv, d), generator=g).half() for _ in range(2))
    kv, scales = random_cache(blocks, n_kv, d, 16)
    values, want = host(kv, scales)
    pkv.paged_kv_append_fp8(k.cuda(), v.cuda(), slots.cuda(), kv, scales)
    ref.append(values, want, k.float(), v.float(), slots, blocks)
    same_cache(kv, scales, values, want)


@pytest.mark.parametrize("n_kv,d", [(1, 64), (3, 128), (17, 128)])
def test_copy_blocks(n_kv, d):
    kv, scales = random_cache(9, n_kv, d, 17)
    values, want = host(kv, scales)
    src, dst = torch.tensor([1, 7, 1, 9, 3], dtype=torch.int32), torch.tensor([0, 8, 5, 2, -1], dtype=torch.int32)
    pkv.paged_kv_copy_blocks_fp8(kv, scales, src.cuda(), dst.cuda())
    assert pkv.pkv_get_device_error() == pkv.DEVERR_BLOCK_ID  # the last two pairs
    for s, d_ in ((1, 0), (7, 8), (1, 5)):
        values[d_], want[d_] = values[s], want[s]
    same_cache(kv, scales, values, want)


# ---------------------------------------------------------------------------
# Decode
# ---------------------------------------------------------------------------

def decode_case(lens, n_q, n_kv, d, dtype, seed, q_len=1, q_size=1.0, spread=3, nan_tail=True, scale=None):
    g = torch.Generator().manual_seed(seed)
    need = [(n + 15) // 16 for n in lens]
    blocks = sum(need) + 2
    kv, scales = random_cache(blocks, n_kv, d, seed, spread)
    place = torch.randperm(blocks, generator=g).to(torch.int32)
    width = max(need + [1])
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = place[at: at + n]
        at += n
        if nan_tail and lens[b] % 16:  # slots behind the last token hold NaN codes
            kv.view(torch.uint8)[tables[b, n - 1].item(), :, :, lens[b] % 16:] = 0x7f
    shape = (len(lens), n_q, d) if q_len == 1 else (len(lens), q_len, n_q, d)
    q = (torch.randn(shape, generator=g) * q_size).to(dtype)
    return q, kv, scales, tables, torch.tensor(lens, dtype=torch.int32), (1.0 / d ** 0.5 if scale is None else scale)


def run_decode(case, **kw):
    q, kv, scales, tables, lens, scale = case
    out = pkv.paged_attention_decode_fp8(q.cuda(), kv, scales, tables.cuda(), lens.cuda(), scale, **kw)
    torch.cuda.synchronize()
    return out.cpu()


def check_decode(case, error=0, **kw):
    q, kv, scales, tables, lens, scale = case
    got = run_decode(case, **kw)
    assert pkv.pkv_get_device_error() == error
    values, want_scales = host(kv, scales)
    want, bound = ref.decode(q, values, want_scales, tables, lens, scale)
    tol = ref.decode_tolerance(want, bound, q.dtype)
    assert torch.equal(got.isnan(), want.isnan())
    # Values past the type's largest round to an infinity.
    limit = torch.finfo(q.dtype).max
    past = got.isinf() & (want.abs() + tol >= limit) & (torch.sign(got.double()) == torch.sign(want))
    off = torch.where(past, -1.0, (got.double() - want).abs() - tol).nan_to_num(-1.0)
    assert (off <= 0).all(), f"off by {off.max().item():.3e} beyond the bound"
    return got


SHORT = [1, 2, 15, 16, 17, 31, 100, 333, 0, 64]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n_q,n_kv,d", [(4, 4, 128), (8, 2, 128), (8, 1, 64), (16, 1, 128), (6, 2, 64), (5, 5, 64),
                                        (14, 2, 128), (40, 2, 128), (20, 1, 64)])
def test_decode_head_layouts(dtype, n_q, n_kv, d):
    check_decode(decode_case(SHORT, n_q, n_kv, d, dtype, seed=n_q * d))


@pytest.mark.parametrize("q_len", [2, 3, 5, 8, 16])
@pytest.mark.parametrize("n_q,n_kv,d", [(4, 4, 128), (8, 2, 64), (7, 1, 128), (16, 2, 64)])
def test_decode_several_queries(q_len, n_q, n_kv, d):
    lens = [q_len, q_len + 1, 16, 17, 31, 32, 33, 150, 0]
    check_decode(decode_case([n if n >= q_len or n == 0 else q_len for n in lens], n_q, n_kv, d, torch.bfloat16,
                             seed=q_len, q_len=q_len))


@pytest.mark.parametrize("lens,n_q,n_kv,d,dtype", [
    ([20000], 4, 1, 128, torch.bfloat16),            # one long context over the whole GPU
    ([3000, 5, 9000, 1, 700], 8, 2, 128, torch.float16),
    ([5000] * 3, 16, 1, 64, torch.float16),
    ([40] * 300, 2, 2, 128, torch.bfloat16),         # more segments than warps
    ([17 + i % 90 for i in range(700)], 4, 4, 64, torch.float16),
])
def test_decode_splits(lens, n_q, n_kv, d, dtype):
    check_decode(decode_case(lens, n_q, n_kv, d, dtype, seed=len(lens)))


@pytest.mark.parametrize("q_size,spread", [(12.0, 1), (0.01, 20), (3.0, 30)])
def test_decode_peaked_rows_and_far_scales(q_size, spread):
    """Rows that see few tokens, and block scales far apart (K and V)."""
    case = decode_case([500, 90, 1300], 8, 2, 128, torch.float16, seed=31, q_size=q_size, spread=spread)
    case[2][:, :, 0].clamp_(max=2.0 ** -6)
    check_decode(case)


def test_decode_queries_near_the_types_limits():
    for dtype, size in ((torch.float16, 2.0 ** 13), (torch.bfloat16, 2.0 ** 90), (torch.bfloat16, 2.0 ** -100)):
        case = decode_case([80, 33], 8, 2, 64, dtype, seed=32, scale=2.0 ** -4 / size)
        case[0].copy_((case[0].double().clamp(-3, 3) * size).to(dtype))
        check_decode(case)


def test_decode_scales_that_are_no_powers_of_two_and_negative_scale():
    case = list(decode_case([300, 41], 8, 2, 128, torch.bfloat16, seed=33))
    case[2].mul_(1 + torch.rand(case[2].shape, generator=torch.Generator().manual_seed(1)).cuda())
    case[5] = -0.07
    check_decode(tuple(case))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("v_scales", [(2.0 ** -48,), (2.0 ** 48 * 1.9375,), (2.0 ** -48, 2.0 ** 48 * 1.9375), (2.0 ** 48, 1.0, 2.0 ** -48)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_decode_scales_at_the_ends_of_their_range(dtype, v_scales, q_len):
    """V's scales at one end, or both in turn: weights and their sum are formed from them."""
    q, kv, scales, tables, lens, scale = decode_case([700, 90, 3000, 17], 8, 2, 128, dtype, seed=66, q_len=q_len)
    scales[..., 1] = torch.tensor(v_scales, device="cuda").repeat(len(scales) // len(v_scales) + 1)[: len(scales), None]
    for k_scale in (2.0 ** -48, 2.0 ** 48 * 1.9375):  # the scores stay what they are
        at = scales.clone()
        at[..., 0] = k_scale
        check_decode((q, kv, at, tables, lens, scale * 2.0 ** -8 / k_scale))


def test_decode_nan_and_infinite_inputs_reach_only_their_rows():
    case = decode_case([70, 70], 8, 2, 64, torch.float16, seed=34)
    q, kv, scales, tables, lens, _ = case
    q[0, 3, 5] = float("nan")
    kv.view(torch.uint8)[tables[1, 2].item(), 1, 1, 4, 9] = 0x7f  # a NaN value: dim 9 of kv head 1's rows
    got = check_decode(case)
    assert got[0, 3].isnan().all() and int(got.isnan().sum()) == 64 + 4


@pytest.mark.parametrize("where", [0, 1])
@pytest.mark.parametrize("n", [48, 50, 34])
def test_decode_nan_in_tokens_behind_a_query(where, n):
    """Drafts: NaN in the last token's key or value; only the last query sees it."""
    q_len = 4
    case = decode_case([n, n + 7], 4, 2, 128, torch.bfloat16, seed=35, q_len=q_len)
    q, kv, scales, tables, lens, _ = case
    last = n - 1
    kv.view(torch.uint8)[tables[0, last // 16].item(), 0, where, last % 16, 11] = 0x7f
    got = check_decode(case)
    assert not got[0, : q_len - 1].isnan().any() and got[0, q_len - 1, 0].isnan().any()


def test_decode_bad_block_ids_and_lengths():
    case = decode_case([200, 16, 90, 300], 8, 2, 128, torch.bfloat16, seed=36)
    q, kv, scales, tables, lens, scale = case
    tables[0, 3], tables[0, 12], tables[1, 0], tables[2, 5] = -7, kv.shape[0], 1 << 30, -1
    got = check_decode(case, error=pkv.DEVERR_BLOCK_ID)
    assert (got[1] == 0).all()
    tables[0, 3] = tables[0, 12] = tables[1, 0] = tables[2, 5] = 0
    lens[1], lens[3] = -4, tables.shape[1] * 16 + 100
    run_decode(case)
    assert pkv.pkv_get_device_error() == pkv.DEVERR_CONTEXT
    got = run_decode(case)
    lens[1], lens[3] = 0, tables.shape[1] * 16
    assert pkv.pkv_get_device_error() == pkv.DEVERR_CONTEXT
    want = run_decode(case)
    assert torch.equal(bits(got[:3]), bits(want[:3]))


def test_decode_context_shorter_than_its_queries_is_flagged_and_zero():
    case = decode_case([3, 40], 4, 2, 64, torch.float16, seed=37, q_len=4)
    got = check_decode(case, error=pkv.DEVERR_CONTEXT)
    assert (got[0] == 0).all() and (got[1] != 0).any()


def test_decode_bits_do_not_depend_on_placement_workspace_or_repetition():
    case = decode_case([3000, 70, 900, 1, 2222], 16, 4, 128, torch.bfloat16, seed=38)
    q, kv, scales, tables, lens, scale = case
    first = run_decode(case)
    ws = pkv.new_workspace(pkv.paged_attention_fp8_workspace_size(5, 1, 16, 4, 128))
    for _ in range(3):
        assert torch.equal(bits(run_decode(case, workspace=ws)), bits(first))
    perm = torch.randperm(kv.shape[0], generator=torch.Generator().manual_seed(2)).cuda()
    moved, moved_scales = torch.zeros_like(kv), torch.zeros_like(scales)
    moved.view(torch.uint8)[perm] = kv.view(torch.uint8)
    moved_scales[perm] = scales
    to = torch.where(tables >= 0, perm.cpu()[tables.clamp(min=0).long()].int(), tables)
    assert torch.equal(bits(run_decode((q, moved, moved_scales, to, lens, scale), workspace=ws)), bits(first))


def test_decode_one_workspace_serves_problems_of_other_sizes():
    big = decode_case([4000, 17, 600], 8, 2, 128, torch.float16, seed=39)
    small = decode_case([40], 8, 2, 128, torch.float16, seed=40)
    ws = pkv.new_workspace(pkv.paged_attention_fp8_workspace_size(3, 1, 8, 2, 128))
    for case in (big, small, big, small):
        check_decode(case, workspace=ws)


def test_decode_leaves_what_is_not_its_output():
    case = decode_case([100, 30], 8, 2, 128, torch.bfloat16, seed=41)
    buf = torch.full((4, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    pkv.paged_attention_decode_fp8(case[0].cuda(), case[1], case[2], case[3].cuda(), case[4].cuda(), case[5],
                                   out=buf[1:3])
    assert (buf[0] == 9).all() and (buf[3] == 9).all()
    assert torch.equal(bits(buf[1:3].cpu()), bits(run_decode(case)))


def test_decode_empty_batch_and_all_empty():
    q, kv, scales, tables, lens, scale = decode_case([40], 8, 2, 128, torch.bfloat16, seed=42)
    out = pkv.paged_attention_decode_fp8(q[:0].cuda(), kv, scales, tables[:0].cuda(), lens[:0].cuda(), scale)
    assert out.shape == (0, 8, 128)
    lens.zero_()
    assert (run_decode((q, kv, scales, tables, lens, scale)) == 0).all()


@pytest.mark.parametrize("n_q,n_kv,d,q_len", [(1, 1, 64, 1), (9, 1, 128, 1)])
def test_decode_of_the_largest_batch(n_q, n_kv, d, q_len):
    lens = [1 + (7 * i) % 37 for i in range(4096)]
    case = decode_case(lens, n_q, n_kv, d, torch.bfloat16, seed=45, q_len=q_len)
    got = run_decode(case)
    assert pkv.pkv_get_device_error() == 0
    pick = list(range(0, 4096, 61)) + [4095]
    q, kv, scales, tables, ctx, scale = case
    values, want_scales = host(kv, scales)
    want, bound = ref.decode(q[pick], values, want_scales, tables[pick], ctx[pick], scale)
    assert ((got[pick].double() - want).abs() <= ref.decode_tolerance(want, bound, q.dtype)).all()


@pytest.mark.parametrize("group", [1, 3, 4, 7, 16, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_a_workspace_for_the_longest_draft_serves_shorter_ones(group, d):
    size = lambda g, q_len: pkv.paged_attention_fp8_workspace_size(3, q_len, 2 * g, 2, d)  # noqa: E731
    sizes = [size(group, q_len) for q_len in range(1, 17)]
    assert sizes == sorted(sizes)
    assert all(size(g, q_len) <= sizes[q_len - 1] for g in range(1, group) for q_len in (1, 2, 5, 16))
    for longest in (1, 3, 5, 16):
        ws = pkv.new_workspace(sizes[longest - 1])
        for q_len in range(1, longest + 1):
            case = decode_case([700, 33, q_len], 2 * group, 2, d, torch.bfloat16, seed=q_len, q_len=q_len)
            assert torch.equal(bits(run_decode(case, workspace=ws)), bits(run_decode(case)))
    assert pkv.pkv_get_device_error() == 0


def test_decode_refuses_a_workspace_that_does_not_fit():
    case = decode_case([40], 8, 2, 128, torch.bfloat16, seed=46)
    need = pkv.paged_attention_fp8_workspace_size(1, 1, 8, 2, 128)
    for ws in (pkv.new_workspace(need - 256), pkv.new_workspace(need + 16)[16:]):
        with pytest.raises(pkv.PagedKVError) as e:
            run_decode(case, workspace=ws)
        assert e.value.status == 5
    with pytest.raises(ValueError):
        run_decode(case, workspace=torch.zeros(need, dtype=torch.uint8))


@pytest.mark.parametrize("captured", [False, True])
def test_a_workspace_may_hold_anything(captured):
    """Words that look like few, many or all arrivals, and floats, in front of every call."""
    cases = [decode_case([20000], 4, 1, 128, torch.bfloat16, seed=62),
             decode_case([3000, 70, 900, 1, 2222], 16, 4, 128, torch.float16, seed=63),
             decode_case([500, 1300, 40], 4, 2, 64, torch.bfloat16, seed=64, q_len=3)]
    for case in cases:
        want = check_decode(case)
        args = [case[0].cuda(), case[1], case[2], case[3].cuda(), case[4].cuda(), case[5]]
        q_len = case[0].shape[1] if case[0].dim() == 4 else 1
        need = pkv.paged_attention_fp8_workspace_size(len(case[4]), q_len, case[0].shape[-2], case[1].shape[1],
                                                      case[0].shape[-1])
        ws, out = torch.zeros(need // 8, dtype=torch.int64, device="cuda"), torch.empty_like(args[0])
        run = lambda: pkv.paged_attention_decode_fp8(*args, out=out, workspace=ws)  # noqa: E731
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            run = graph.replay
        for fill in (1, 2, 7, 147, 148, 1 << 32, 1 << 48, 5 << 48, (1 << 48) + 1, -1, 0x7F7F7F7F7F7F7F7F, 0x3F80000040400000):
            ws.fill_(fill)
            run()
            assert torch.equal(bits(out.cpu()), bits(want))
            run()  # what a call leaves behind serves the next one
            assert torch.equal(bits(out.cpu()), bits(want))
            ws.random_()
            run()
            assert torch.equal(bits(out.cpu()), bits(want))
    assert pkv.pkv_get_device_error() == 0


@pytest.mark.parametrize("lens,n_q,n_kv,d,q_len,unit", [
    ([20000], 4, 1, 128, 1, 40),                 # in the middle of a context that many CTAs share
    ([3000, 70, 900, 1, 2222], 16, 4, 128, 1, 0),
    ([3000, 70, 900, 33, 2222], 16, 4, 128, 4, 3),   # 16 rows
    ([900] * 40, 6, 2, 64, 1, 500),
])
@pytest.mark.parametrize("own_workspace", [False, True])
def test_decode_wait_that_runs_out_and_the_next_call(lens, n_q, n_kv, d, q_len, unit, own_workspace):
    """A tile that is never copied, others of the unit in flight behind it: the launch ends with
    the flag, and what it leaves in the workspace does not disturb the next one."""
    case = decode_case(lens, n_q, n_kv, d, torch.bfloat16, seed=65, q_len=q_len)
    want = check_decode(case)
    ws = None if own_workspace else pkv.new_workspace(pkv.paged_attention_fp8_workspace_size(len(lens), q_len, n_q, n_kv, d))
    for _ in range(2):
        run_decode(case, workspace=ws, wait_limit_us=5000, test_withhold_unit=unit)
        assert pkv.pkv_get_device_error() == pkv.DEVERR_TIMEOUT
        assert torch.equal(bits(run_decode(case, workspace=ws)), bits(want))
        assert torch.equal(bits(run_decode(case, workspace=ws, wait_limit_us=1_000_000)), bits(want))
    assert pkv.pkv_get_device_error() == 0


@pytest.mark.parametrize("unit", [2368, 1 << 20, (1 << 31) - 2])
def test_decode_withheld_unit_that_is_none(unit):
    case = decode_case([20000, 40], 4, 1, 128, torch.bfloat16, seed=67)
    assert torch.equal(bits(run_decode(case, wait_limit_us=5000, test_withhold_unit=unit)), bits(check_decode(case)))
    assert pkv.pkv_get_device_error() == 0


def test_two_graphs_share_a_workspace_in_turn():
    cases = [decode_case([2500, 40], 8, 2, 128, torch.bfloat16, seed=47), decode_case([300] * 9, 16, 1, 64, torch.float16, seed=48)]
    want = [run_decode(c) for c in cases]
    ws = pkv.new_workspace(max(pkv.paged_attention_fp8_workspace_size(*a) for a in ((2, 1, 8, 2, 128), (9, 1, 16, 1, 64))))
    graphs, outs = [], []
    for c in cases:
        args = [c[0].cuda(), c[1], c[2], c[3].cuda(), c[4].cuda(), c[5]]
        out = torch.zeros_like(args[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_attention_decode_fp8(*args, out=out, workspace=ws)
        graphs.append((graph, args))
        outs.append(out)
    for i in (0, 1, 1, 0, 1, 0, 0):
        outs[i].zero_()
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(outs[i].cpu()), bits(want[i]))
    assert pkv.pkv_get_device_error() == 0


def test_append_into_a_graph():
    """A captured append, replayed on new tokens and slots, against the eager one."""
    g = torch.Generator().manual_seed(49)
    table = pkv.rotary_table(64, 128, device="cuda")
    k, v, q = (torch.randn((6, h, 128), generator=g).bfloat16().cuda() for h in (2, 2, 8))
    pos, slots = torch.arange(6).cuda(), (torch.arange(6) + 16).cuda()
    kv, scales = random_cache(4, 2, 128, 50)
    q_out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_kv_append_rope_fp8(k, v, pos, table, slots, kv, scales, q=q, q_out=q_out)
    for step in range(3):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g).bfloat16() * (step + 1))
        slots.copy_(torch.tensor([0, 1, 2, -1, 40, 41]) + 3 * step)
        if step:
            slots[3] = -1
        kv2, scales2 = kv.clone(), scales.clone()
        want_q = pkv.paged_kv_append_rope_fp8(k, v, pos, table, slots, kv2, scales2, q=q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(q_out), bits(want_q)) and torch.equal(scales, scales2)
        assert torch.equal(kv.view(torch.uint8), kv2.view(torch.uint8))


def test_large_pool_offsets_pass_32_bits():
    """A pool of more than 4 GiB of codes: blocks at its far end."""
    n_kv, d, blocks = 32, 128, 36000  # 4.7 GB
    kv = torch.zeros((blocks, n_kv, 2, 16, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.ones((blocks, n_kv, 2), device="cuda")
    g = torch.Generator().manual_seed(43)
    k, v = (torch.randn((20, n_kv, d), generator=g).bfloat16().cuda() for _ in range(2))
    slots = torch.cat((torch.arange(16) + (blocks - 1) * 16, torch.arange(4) + (blocks - 7) * 16)).cuda()
    pkv.paged_kv_append_fp8(k, v, slots, kv, scales)
    pkv.paged_kv_copy_blocks_fp8(kv, scales, torch.tensor([blocks - 1, blocks - 7], dtype=torch.int32).cuda(),
                                 torch.tensor([0, 1], dtype=torch.int32).cuda())
    q = torch.randn((1, 32, d), generator=g).bfloat16().cuda()
    lens = torch.tensor([20], dtype=torch.int32).cuda()
    far = pkv.paged_attention_decode_fp8(q, kv, scales, torch.tensor([[blocks - 1, blocks - 7]], dtype=torch.int32).cuda(),
                                         lens, 0.1)
    near = pkv.paged_attention_decode_fp8(q, kv, scales, torch.tensor([[0, 1]], dtype=torch.int32).cuda(), lens, 0.1)
    assert torch.equal(bits(far.cpu()), bits(near.cpu()))
    values, want_scales = host(kv[:2], scales[:2])
    want, bound = ref.decode(q.cpu(), values, want_scales, torch.tensor([[0, 1]]), torch.tensor([20]), 0.1)
    assert ((near.cpu().double() - want).abs() <= ref.decode_tolerance(want, bound, torch.bfloat16)).all()


# ---------------------------------------------------------------------------
# Together, as a serving step uses them
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("with_workspace", [False, True])
def test_serving_steps_with_block_manager_fork_and_graph(with_workspace):
    """Prompts, then decode steps with a fork (copy-on-write) on the way; a
    captured step gives the eager step's bits."""
    n_q, n_kv, d, rot, scale = 8, 2, 128, 64, 0.09
    g = torch.Generator().manual_seed(50)
    bm = pkv.BlockManager(64)
    kv, scales = pkv.fp8_cache(64, n_kv, d)
    values, want = host(kv, scales)
    table = pkv.rotary_table(512, rot, device="cuda")

    def append(slots, pos):
        rows = torch.randn((len(slots), (n_q + 2 * n_kv) * d), generator=g).bfloat16().cuda()
        q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split((n_q * d, n_kv * d, n_kv * d), 1))
        q = pkv.paged_kv_append_rope_fp8(k, v, pos.cuda(), table, slots.cuda(), kv, scales, q=q)
        ref.append(values, want, ref.rotate32(k.cpu(), table.cpu(), pos, False), v.cpu().float(), slots, 64)
        same_cache(kv, scales, values, want)
        return q

    prompts = {0: 37, 1: 16, 2: 5}
    for seq, n in prompts.items():
        bm.add_sequence(seq, n)
    bt, _ = bm.tables(list(prompts), 6)
    pos = torch.cat([torch.arange(n) for n in prompts.values()])
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(list(prompts.values())))
    append(bt[seq, pos // 16].long() * 16 + pos % 16, pos)
    bm.fork(0, 3)
    ids = [0, 1, 2, 3]
    ws = pkv.new_workspace(pkv.paged_attention_fp8_workspace_size(4, 1, n_q, n_kv, d)) if with_workspace else None
    for _ in range(14):
        slots, src, dst = bm.append(ids)
        if len(src):
            pkv.paged_kv_copy_blocks_fp8(kv, scales, src.cuda(), dst.cuda())
            values[dst.long()], want[dst.long()] = values[src.long()], want[src.long()]
        bt, cl = bm.tables(ids, 6)
        q = append(slots, cl.long() - 1)
        out = pkv.paged_attention_decode_fp8(q, kv, scales, bt.cuda(), cl.cuda(), scale, workspace=ws)
        exact, bound = ref.decode(q.cpu(), values, want, bt, cl, scale)
        assert ((out.cpu().double() - exact).abs() <= ref.decode_tolerance(exact, bound, q.dtype)).all()
    assert pkv.pkv_get_device_error() == 0
    btd, cld, captured = bt.cuda(), cl.cuda(), torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_attention_decode_fp8(q, kv, scales, btd, cld, scale, out=captured, workspace=ws)
    for _ in range(3):
        captured.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(captured.cpu()), bits(out.cpu()))


def test_two_streams_with_a_workspace_each():
    cases = [decode_case([1500, 300], 8, 2, 128, torch.bfloat16, seed=s) for s in (60, 61)]
    want = [run_decode(c) for c in cases]
    on = [[c[0].cuda(), c[1], c[2], c[3].cuda(), c[4].cuda(), c[5]] for c in cases]
    ws = [pkv.new_workspace(pkv.paged_attention_fp8_workspace_size(2, 1, 8, 2, 128)) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(pkv.paged_attention_decode_fp8(*on[i], workspace=ws[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(bits(o.cpu()), bits(want[i]))
