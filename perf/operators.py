"""What is measured of the rotating append, the FP8 cache's append and its decode attention.

Three operators of the paged cache (16-token blocks reached through a block
table), each in its plain form (elementary torch operations) and, with ``own``
set, as the calls a serving program makes of this package:

* ``rope``: rotate the new tokens' queries and keys by their positions and
  write keys and values into their slots of a cache of the same type;
* ``append``: the same into an 8-bit cache (e4m3 codes with one power-of-two
  scale for each block, kv head and K or V), with or without the rotation;
* ``decode``: attention of the last ``q_len`` tokens of every sequence over
  that 8-bit cache.

The 8-bit cache is ``kv`` float8_e4m3fn ``[blocks, kv heads, 2, 16, d]`` (K,
then V) and ``scales`` float32 ``[blocks, kv heads, 2]``; a value is code x
scale.  Appending to a block takes the scale up to the smallest power of two
that holds the largest new magnitude within 448 (codes already there are
rounded to the new scale); a token at offset 0 starts the block anew.
"""

import math

import torch

own = False

BLOCK = 16
E_MIN, E_MAX = -48, 48
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ELEM = {"f32": 4, "f16": 2, "bf16": 2}
TABLE = 131072  # positions of the rotation tables


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    def rope(name, tokens, q, kv, d, rot, dtype, style="half", seqs=1):
        return {"name": name, "op": "rope", "tokens": tokens, "seqs": seqs, "q_heads": q, "kv_heads": kv, "dim": d,
                "rot": rot, "style": style, "dtype": dtype}

    def app(name, tokens, q, kv, d, rot, dtype, style="half", seqs=1):
        return {**rope(name, tokens, q, kv, d, rot, dtype, style, seqs), "op": "append"}

    def dec(name, batch, lo, hi, q, kv, d, dtype, q_len=1):
        return {"name": name, "op": "decode", "batch": batch, "lo": lo, "hi": hi, "q_len": q_len, "q_heads": q,
                "kv_heads": kv, "dim": d, "dtype": dtype}

    return [
        # One user's next token: nothing but latency.
        rope("rope_one_token", 1, 32, 8, 128, 128, "bf16"),
        # A decode step of 256 sequences of a multi-head model in fp16.
        rope("rope_step_256_mha", 256, 32, 32, 128, 128, "f16", seqs=256),
        # A long prompt's chunk.
        rope("rope_prompt_8192", 8192, 32, 8, 128, 128, "bf16"),
        # An odd number of fp32 tokens, small heads, rotation of half of the dims, neighbours as pairs.
        rope("rope_777_f32_partial", 777, 12, 4, 64, 32, "f32", "pair", seqs=3),
        # A decode step of 64 sequences into the 8-bit cache: one token each, somewhere in its block.
        app("append_step_64", 64, 32, 8, 128, 128, "bf16", seqs=64),
        # Prompts of several sequences with ragged ends, rotated by pairs.
        app("append_prompts_5003", 5003, 40, 10, 128, 128, "f16", "pair", seqs=7),
        # A cache filled from keys that were rotated before (no rotation here).
        app("append_prompt_16384_plain", 16384, 64, 8, 128, 0, "bf16"),
        # One sequence of a few thousand tokens: latency of the split and its merge.
        dec("decode_one_4096", 1, 4096, 4096, 32, 8, 128, "bf16"),
        # A serving batch of mixed lengths, four query heads to a kv head.
        dec("decode_64_gqa", 64, 128, 4096, 32, 8, 128, "bf16"),
        # A batch of short sequences of a multi-head model (one query head to a kv head).
        dec("decode_256_mha", 256, 1, 1300, 32, 32, 128, "f16"),
        # Verifying drafts: four new tokens of each sequence at once.
        dec("decode_32_verify_4", 32, 128, 4096, 32, 8, 128, "bf16", q_len=4),
        # Long contexts, eight query heads to a kv head.
        dec("decode_4x131072", 4, 131072, 131072, 64, 8, 128, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode"])
    d = rng.choice([64, 128, 128])
    if op == "decode":
        kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
        group = rng.choice([g for g in (1, 2, 3, 4, 5, 6, 7, 8, 16) if g * kv <= 96])
        q_len = rng.choice([1, 1, 1, 2, 3, 5, 8])
        batch = _log_int(rng, 1, 300)
        top = min(131072, 4_000_000 // (batch * kv) + 16)  # at most the largest listed case
        hi = _log_int(rng, max(q_len, 16), top)
        lo = rng.choice([q_len, max(q_len, hi // 2), hi])
        return {"op": op, "batch": batch, "lo": lo, "hi": hi, "q_len": q_len, "q_heads": kv * group, "kv_heads": kv,
                "dim": d, "dtype": rng.choice(["f16", "bf16"])}
    kv = rng.choice([1, 2, 3, 4, 8, 10, 16])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    tokens = _log_int(rng, 1, 12000)
    seqs = rng.choice([1, min(tokens, 5), max(1, tokens // 3), tokens])
    rot = rng.choice([d, d, d // 2, 16]) if op == "rope" or rng.random() < 0.7 else 0
    return {"op": op, "tokens": tokens, "seqs": seqs, "q_heads": kv * group, "kv_heads": kv, "dim": d, "rot": rot,
            "style": rng.choice(["half", "pair"]), "dtype": rng.choice(["f32", "f16", "bf16"])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _spread(n, lo, hi):
    """n lengths over [lo, hi], the last one hi (the same for every seed: they set the work)."""
    return [lo + int((hi - lo) * ((0.6180339887498949 * (i + 1)) % 1.0)) for i in range(n - 1)] + [hi]


def _new_tokens(case):
    """New tokens of each sequence, and how many it held before."""
    t, s = case["tokens"], case["seqs"]
    new = [t // s + (1 if i < t % s else 0) for i in range(s)]
    # Steps go somewhere into a context; whole prompts start at a sequence's begin.
    held = _spread(s, 0, 2000) if t < 4 * s else [(37 * i) % 16 if s > 1 else 0 for i in range(s)]
    return new, held


def _table(rot, device):
    """cos then sin of position x frequency, from 64-bit angles."""
    f = 1.0 / 500000.0 ** (torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(TABLE, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def _codes(blocks, kv, d, gen, device):
    """Codes and scales of N(0, 1) keys and values: 448 x scale is just over a block's largest."""
    out = torch.empty((blocks, kv, 2, BLOCK, d), dtype=torch.float8_e4m3fn, device=device)
    scales = torch.empty((blocks, kv, 2), dtype=torch.float32, device=device)
    step = max(1, (1 << 26) // (kv * 2 * BLOCK * d))
    for at in range(0, blocks, step):
        x = torch.randn((min(step, blocks - at), kv, 2, BLOCK, d), generator=gen, device=device)
        s = _need(x.abs().amax((-1, -2)))
        out[at: at + step] = (x / s[..., None, None]).to(torch.float8_e4m3fn)
        scales[at: at + step] = s
    return out, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    kv, q_heads, d, dtype = case["kv_heads"], case["q_heads"], case["dim"], TYPES[case["dtype"]]
    if case["op"] == "decode":
        lens = _spread(case["batch"], case["lo"], case["hi"])
        need = [(n + BLOCK - 1) // BLOCK for n in lens]
        blocks = sum(need) + 3
        place = torch.randperm(blocks, generator=gen, device=dev)[: sum(need)].to(torch.int32)
        width = max(need)
        first = torch.tensor([0] + need, device=dev).cumsum(0)
        at = first[:-1, None] + torch.arange(width, device=dev)
        tables = torch.where(at < first[1:, None], place[at.clamp(max=sum(need) - 1)].long(), -1).to(torch.int32)
        cache, scales = _codes(blocks, kv, d, gen, dev)
        shape = (len(lens), q_heads, d) if case["q_len"] == 1 else (len(lens), case["q_len"], q_heads, d)
        q = torch.randn(shape, generator=gen, device=dev) * torch.tensor([1.0, 2.0, 4.0], device=dev)[
            torch.arange(q_heads, device=dev) % 3][:, None]  # some heads look at few tokens
        state = {"case": case, "q": q.to(dtype), "kv": cache, "scales": scales, "tables": tables.contiguous(),
                 "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "scale": 1.0 / math.sqrt(d)}
        if own:
            import paged_kv_cache_386_b200 as pkv
            state["workspace"] = pkv.new_workspace(pkv.paged_attention_fp8_workspace_size(
                len(lens), case["q_len"], q_heads, kv, d), dev)
        return state
    new, held = _new_tokens(case)
    need = [(n + h + BLOCK - 1) // BLOCK for n, h in zip(new, held)]
    blocks = sum(need) + 2
    place = torch.randperm(blocks, generator=gen, device=dev)
    seq = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev))
    start = torch.tensor([0] + new, device=dev).cumsum(0)[:-1]
    pos = torch.arange(case["tokens"], device=dev) - start[seq] + torch.tensor(held, device=dev)[seq]
    base = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
    slots = place[base[seq] + pos // BLOCK] * BLOCK + pos % BLOCK
    if len(new) > 1 and case["tokens"] > 2 * len(new):
        slots[-1] = -1  # a padding token at the end of the call
    # One projection's output holds the rows of q, k and v: the heads are views of it.
    rows = torch.randn((case["tokens"], (q_heads + 2 * kv) * d), generator=gen, device=dev).to(dtype)
    q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split((q_heads * d, kv * d, kv * d), 1))
    state = {"case": case, "q": q, "k": k, "v": v, "slots": slots, "pos": pos,
             "table": _table(case["rot"], dev) if case["rot"] else None}
    if case["op"] == "rope":
        state["k_cache"], state["v_cache"] = (torch.randn((blocks, kv, BLOCK, d), generator=gen, device=dev).to(dtype)
                                              for _ in range(2))
    else:
        state["kv"], state["scales"] = _codes(blocks, kv, d, gen, dev)
    return state


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _need(amax):
    """The smallest power of two s, within the exponents kept, with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 x 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(E_MIN, E_MAX)
    e = torch.where(amax == 0, torch.full_like(e, E_MIN), e)
    return torch.ldexp(torch.ones_like(amax), e)


def _rotated(x, table, pos, style):
    rot = table.shape[1]
    x = x.float()
    c, s = table[pos].unsqueeze(1).split(rot // 2, -1)
    y, rest = x[..., :rot], x[..., rot:]
    if style == "half":
        a, b = y[..., : rot // 2], y[..., rot // 2:]
        return torch.cat((a * c - b * s, b * c + a * s, rest), -1)
    a, b = y[..., 0::2], y[..., 1::2]
    return torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), rest), -1)


def _plain_rope(st):
    style = st["case"]["style"]
    dtype = st["q"].dtype
    q = _rotated(st["q"], st["table"], st["pos"], style).to(dtype)
    k = _rotated(st["k"], st["table"], st["pos"], style).to(dtype)
    keep = st["slots"] >= 0
    slots = st["slots"][keep]
    st["k_cache"][slots // BLOCK, :, slots % BLOCK] = k[keep]
    st["v_cache"][slots // BLOCK, :, slots % BLOCK] = st["v"][keep]
    return [q, st["k_cache"], st["v_cache"]]


def _plain_append(st):
    case, outs = st["case"], []
    k = st["k"].float()
    if case["rot"]:
        outs = [_rotated(st["q"], st["table"], st["pos"], case["style"]).to(st["q"].dtype)]
        k = _rotated(st["k"], st["table"], st["pos"], case["style"])
    keep = st["slots"] >= 0
    slots = st["slots"][keep]
    x = torch.stack((k, st["v"].float()), 2)[keep]  # [tokens, kv heads, 2, d]
    blocks, which = torch.unique(slots // BLOCK, return_inverse=True)
    off = slots % BLOCK
    amax = torch.zeros((len(blocks),) + x.shape[1:3], device=x.device).index_reduce_(0, which, x.abs().amax(-1), "amax")
    fresh = torch.zeros(len(blocks), device=x.device).index_reduce_(0, which, (off == 0).float(), "amax") > 0
    old, need = st["scales"][blocks], _need(amax)
    scale = torch.where(fresh[:, None, None], need, torch.maximum(old, need))
    codes = st["kv"][blocks].float() * (old / scale)[..., None, None]
    codes = torch.where(fresh[:, None, None, None, None], torch.zeros_like(codes), codes)
    codes[which, :, :, off] = (x / scale[which][..., None]).clamp(-448, 448)
    st["kv"][blocks] = codes.to(torch.float8_e4m3fn)
    st["scales"][blocks] = scale
    return outs + [st["kv"], st["scales"]]


def _plain_decode(st):
    case, tables, lens = st["case"], st["tables"], st["lens"]
    batch, kv, q_len = tables.shape[0], case["kv_heads"], case["q_len"]
    ids = tables.clamp(min=0).long()
    x = st["kv"][ids].float() * st["scales"][ids][..., None, None]  # [batch, blocks, kv heads, 2, 16, d]
    k, v = (y.transpose(1, 2).flatten(2, 3) for y in x.unbind(3))  # [batch, kv heads, tokens, d]
    q = st["q"].float().view(batch, q_len, kv, -1, case["dim"]).transpose(1, 2)
    s = q.reshape(batch, kv, -1, case["dim"]) @ k.transpose(2, 3) * st["scale"]
    token = torch.arange(s.shape[-1], device=s.device)
    seen = token < (lens[:, None] - q_len + 1 + torch.arange(q_len, device=s.device))[..., None]
    s = s.view(batch, kv, q_len, -1, s.shape[-1]).masked_fill(~seen[:, None, :, None], -math.inf)
    w = (s - s.amax(-1, keepdim=True)).exp()
    out = w.flatten(2, 3) @ v / w.sum(-1).flatten(2, 3)[..., None]
    return [out.view(batch, kv, q_len, -1, case["dim"]).transpose(1, 2).reshape(st["q"].shape).to(st["q"].dtype)]


def _own(st):
    import paged_kv_cache_386_b200 as pkv
    case = st["case"]
    if case["op"] == "decode":
        return [pkv.paged_attention_decode_fp8(st["q"], st["kv"], st["scales"], st["tables"], st["lens"], st["scale"],
                                               workspace=st["workspace"])]
    pair = case["style"] == "pair"
    if case["op"] == "rope":
        q = pkv.paged_kv_append_rope(st["k"], st["v"], st["pos"], st["table"], st["slots"], st["k_cache"],
                                     st["v_cache"], q=st["q"], interleaved=pair)
        return [q, st["k_cache"], st["v_cache"]]
    if case["rot"]:
        q = pkv.paged_kv_append_rope_fp8(st["k"], st["v"], st["pos"], st["table"], st["slots"], st["kv"],
                                         st["scales"], q=st["q"], interleaved=pair)
        return [q, st["kv"], st["scales"]]
    pkv.paged_kv_append_fp8(st["k"], st["v"], st["slots"], st["kv"], st["scales"])
    return [st["kv"], st["scales"]]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# Work and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    kv, q_heads, d, e = case["kv_heads"], case["q_heads"], case["dim"], ELEM[case["dtype"]]
    if case["op"] == "decode":
        lens = _spread(case["batch"], case["lo"], case["hi"])
        blocks = sum((n + BLOCK - 1) // BLOCK for n in lens)
        rows = case["batch"] * case["q_len"] * q_heads
        return {"bytes": sum(lens) * kv * 2 * d + blocks * (kv * 8 + 4) + 2 * rows * d * e + 4 * case["batch"],
                "flops": 4 * sum(lens) * q_heads * case["q_len"] * d}
    t, rot = case["tokens"], case["rot"]
    new, held = _new_tokens(case)
    n = 2 * t * kv * d * e + 8 * t  # k, v and slots in
    if rot:  # positions, q in and out, each distinct position's cosines and sines
        n += 8 * t + 2 * t * q_heads * d * e
        seen = max(h + m for h, m in zip(held, new)) if len(new) < t else min(t, 2000)
        n += 4 * rot * min(t, seen)
    if case["op"] == "rope":
        return {"bytes": n + 2 * t * kv * d * e, "flops": 3 * t * (q_heads + kv) * rot}
    touched = sum((h + m + BLOCK - 1) // BLOCK - h // BLOCK for h, m in zip(held, new))
    return {"bytes": n + 2 * t * kv * d + 16 * touched * kv, "flops": 3 * t * (q_heads + kv) * rot + 4 * t * kv * d}


def _exact_rotation(x, st, style):
    x = x.double().clone()
    rot = st["table"].shape[1]
    angle = st["table"].double()[st["pos"]][:, None, :]
    cos, sin = angle[..., : rot // 2], angle[..., rot // 2:]
    i = torch.arange(rot // 2, device=x.device)
    first, second = (i, i + rot // 2) if style == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., first], x[..., second]
    x[..., first], x[..., second] = a * cos - b * sin, b * cos + a * sin
    return x


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "decode":
        outs = []
        group = case["q_heads"] // case["kv_heads"]
        q = st["q"].double().view(case["batch"], case["q_len"], case["kv_heads"], group, case["dim"])
        for b, n in enumerate(st["lens"].tolist()):
            ids = st["tables"][b, : (n + BLOCK - 1) // BLOCK].long()
            heads = []
            for h in range(case["kv_heads"]):
                x = st["kv"][ids, h].double() * st["scales"][ids, h].double()[:, :, None, None]
                k, v = x[:, 0].reshape(-1, case["dim"])[:n], x[:, 1].reshape(-1, case["dim"])[:n]
                s = torch.einsum("igd,td->igt", q[b, :, h], k) * st["scale"]
                hidden = torch.arange(n, device=s.device)[None] > (n - case["q_len"] + torch.arange(
                    case["q_len"], device=s.device))[:, None]
                s[hidden[:, None].expand_as(s)] = -math.inf
                heads.append(torch.softmax(s, -1) @ v)
            outs.append(torch.stack(heads, 1))
        return [torch.stack(outs).reshape(st["q"].shape)]
    live = st["slots"] >= 0
    slots = st["slots"][live]
    k = _exact_rotation(st["k"], st, case["style"]) if case["rot"] else st["k"].double()
    v = st["v"].double()
    outs = [_exact_rotation(st["q"], st, case["style"])] if case["rot"] else []
    if case["op"] == "rope":
        for name, x in (("k_cache", k), ("v_cache", v)):
            c = st[name].double()
            c[slots // BLOCK, :, slots % BLOCK] = x[live]
            outs.append(c)
        return outs
    # The tokens of the call in a pool-shaped frame, then block by block.
    blocks = st["kv"].shape[0]
    frame = torch.zeros(st["kv"].shape, dtype=torch.float64, device=k.device)
    written = torch.zeros((blocks, BLOCK), dtype=torch.bool, device=k.device)
    written[slots // BLOCK, slots % BLOCK] = True
    frame[slots // BLOCK, :, 0, slots % BLOCK] = k[live]
    frame[slots // BLOCK, :, 1, slots % BLOCK] = v[live]
    top = frame.abs().amax((-1, -2))
    need = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(E_MIN, E_MAX))  # top 0 gives the least scale
    need = torch.where(top / 448.0 > need, need * 2, need)  # the logarithm's rounding
    need = torch.where((top / 448.0 <= need / 2) & (need > 2.0 ** E_MIN), need / 2, need)
    old = st["scales"].double()
    touched, fresh = written.any(1)[:, None, None], written[:, 0][:, None, None]
    scale = torch.where(touched, torch.where(fresh, need, torch.maximum(old, need)), old)
    was = torch.where((touched & fresh)[..., None, None], torch.zeros_like(frame),
                      st["kv"].double() * (old / scale)[..., None, None])
    value = torch.where(written[:, None, None, :, None], frame / scale[..., None, None], was)
    # To the nearest e4m3 value, ties to even: a multiple of 2^(exponent - 3), no finer than 2^-9.
    unit = torch.exp2(torch.floor(torch.log2(value.abs().clamp(min=2.0 ** -6))) - 3)
    return outs + [torch.round(value / unit) * unit, scale]
