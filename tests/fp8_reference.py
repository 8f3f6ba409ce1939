"""Plain restatements of the rotation, of the FP8 cache's append and of its
decode attention, token by token and in 64 bits (rotations in separately
rounded 32-bit steps where their bits decide a code)."""

from __future__ import annotations

import math

import torch

BLOCK = 16


def rotate32(x, cos_sin, positions, interleaved):
    """The rotation in fp32, every product and sum rounded by itself."""
    x = x.float().clone()
    half = cos_sin.shape[1] // 2
    c, s = cos_sin[positions, :half][:, None], cos_sin[positions, half:][:, None]
    j = torch.arange(half)
    a_at, b_at = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    a, b = x[..., a_at], x[..., b_at]
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    x[..., a_at], x[..., b_at] = ac - bs, bc + as_
    return x


def rotate64(x, cos_sin, positions, interleaved):
    """(rotation in fp64, sum of the magnitudes of each element's two products)."""
    y, mag = x.double().clone(), x.double().abs()
    half = cos_sin.shape[1] // 2
    c, s = cos_sin.double()[positions, :half][:, None], cos_sin.double()[positions, half:][:, None]
    j = torch.arange(half)
    a_at, b_at = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    a, b = x.double()[..., a_at], x.double()[..., b_at]
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    mag[..., a_at], mag[..., b_at] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mag


def e4m3(x: float) -> float:
    """Nearest e4m3 value, ties to even; magnitudes past 448 give 448, NaN NaN."""
    if math.isnan(x):
        return x
    m = min(abs(x), 448.0)
    unit = 2.0 ** (max(math.floor(math.log2(m)) if m > 0 else -6, -6) - 3)
    return math.copysign(min(round(m / unit) * unit, 448.0), x)


def e4m3_all(x: torch.Tensor) -> torch.Tensor:
    m = x.double().abs().clamp(max=448.0)
    unit = torch.exp2(torch.frexp(m.clamp(min=2.0 ** -6))[1].double() - 1 - 3)
    return torch.copysign((torch.round(m / unit) * unit).clamp(max=448.0), x.double())


def scale_for(amax: float) -> float:
    e = -48
    while e < 48 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(values, scales, k, v, slots, num_blocks, left_out=()):
    """`values` float64 [blocks, kv heads, 2, 16, d] (code values), `scales`
    float64; k and v are float, in the order of the call.  In place."""
    touched = {}
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < num_blocks * BLOCK and i not in left_out:
            touched.setdefault(s // BLOCK, {})[s % BLOCK] = i  # the last one counts
    for blk, toks in touched.items():
        offs = sorted(toks)
        for kind, x in enumerate((k, v)):
            rows = x[[toks[o] for o in offs]].double()  # [tokens, heads, d]
            finite = torch.where(rows.isfinite(), rows.abs(), 0.0)
            for h in range(values.shape[1]):
                need = scale_for(finite[:, h].max().item())
                old = scales[blk, h, kind].item()
                new = need if 0 in toks else max(old, need)
                tile = values[blk, h, kind]
                if 0 in toks:
                    tile.zero_()
                elif new != old:
                    tile.copy_(e4m3_all(tile * (old / new)))
                tile[offs] = e4m3_all(rows[:, h] / new)
                scales[blk, h, kind] = new
    return values, scales


def decode(q, values, scales, tables, lens, scale, num_blocks=None):
    """(out, bound): attention in 64 bits, and for each element the error that
    the kernel's own arithmetic may add before the output is rounded:
      * scores are fp32 sums over d exact products: off by at most (d / 4 + 8)
        2^-23 of the sum of their magnitudes, and an exponent's argument
        by 2^-23 of the magnitudes it is formed from; both enter a weight and
        the sum of the weights;
      * weights are rounded to f16: 2^-11 of their magnitude, or 2^-25 of the
        row's largest, each relative to sum p |v| (at most 2^8 x as large as
        the largest weight at a later maximum: another 2^-17);
      * fp32 sums over the 16-token tiles and the pieces."""
    batch, n_q, d = q.shape[0], q.shape[-2], q.shape[-1]
    q4 = q.double().reshape(batch, -1, n_q, d)
    q_len, n_kv = q4.shape[1], values.shape[1]
    group = n_q // n_kv
    num_blocks = values.shape[0] if num_blocks is None else num_blocks
    out, bound = torch.zeros_like(q4), torch.zeros_like(q4)
    for b, n in enumerate(lens.tolist()):
        if n < q_len:
            continue
        ids = tables[b, : (n + BLOCK - 1) // BLOCK].long()
        good = (ids >= 0) & (ids < num_blocks)
        live = good.repeat_interleave(BLOCK)[:n]
        at = ids.clamp(0, num_blocks - 1)
        x = values[at] * scales[at][..., None, None].double()
        kk = x[:, :, 0].transpose(0, 1).reshape(n_kv, -1, d)[:, :n]
        vv = x[:, :, 1].transpose(0, 1).reshape(n_kv, -1, d)[:, :n]
        for i in range(q_len):
            seen = live & (torch.arange(n) < n - q_len + i + 1)
            if not seen.any():
                continue
            for h in range(n_q):
                keys, vals = kk[h // group, seen], vv[h // group, seen]
                s = keys @ q4[b, i, h] * scale
                mag = ((keys.abs() @ q4[b, i, h].abs()).max() * abs(scale)).item()
                w = torch.softmax(s, 0)
                out[b, i, h] = w @ vals
                rel = 2 * ((d / 4 + 8) * mag + 2 * s.abs().max().item() + 128) * 2.0 ** -23
                rel += 2.0 ** -11 + 2.0 ** -17 + (n / 16 + 32) * 2.0 ** -23
                bound[b, i, h] = (w @ vals.abs()) * rel
    return out.reshape(q.shape), bound.reshape(q.shape)


def decode_tolerance(out, bound, dtype):
    """Plus the one rounding of the output: half a step."""
    return bound + (out.abs() + bound) * torch.finfo(dtype).eps / 2 + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
