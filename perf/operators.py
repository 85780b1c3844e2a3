"""The operators of the 8-bit paged K/V cache, as they are measured.

rope      rope_and_cache: rotates the queries and keys of new tokens by their
          positions and appends keys and values to the bf16 paged cache
append    rope_and_cache_fp8: the same into a cache of e4m3 values with one
          power-of-two scale for each (block, KV head), which grows when a new
          token does not fit it (the block's older values are then re-rounded)
attend    paged_attention_decode_fp8 (one query token a sequence) and
          paged_attention_multi_query_fp8 (a few, causal): attention that reads
          that cache through block tables
gather    gather_kv_fp8: the sequences' rows of the 8-bit cache as bf16, through
          the tables (what a prompt chunk over an 8-bit prefix attends to)
copy      copy_blocks_fp8: copy-on-write clones of blocks with their scales

The 8-bit cache is [num_blocks, num_kv_heads, block_size, head_dim] e4m3 with
float32 scales [num_blocks, num_kv_heads]; a stored value stands for itself
times its scale.  The scale of a block and head that takes new tokens is the
smallest 2^e, -64 <= e <= 64, with m2 <= (448 * 2^e)^2, where m2 is the
largest of x1^2 + x2^2 over the pairs that are rotated (a bound on both results
whatever the position) and x^2 over the other elements, each rounded to 32 bits,
and not less than the scale that the block's older tokens already have.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # A decode step of four short sequences on a small model: the launch counts, not the bytes.
        dict(name="rope-decode-tiny", op="rope", tokens=4, heads=8, kv_heads=8, head_dim=64, block=16, rot=64,
             interleaved=False, far=128),
        # A prompt of 8,192 tokens on the 70B-shaped layer.
        dict(name="rope-prompt-8k", op="rope", tokens=8192, heads=64, kv_heads=8, head_dim=128, block=16, rot=128,
             interleaved=False, far=131072),
        # One new token of each of 256 sequences (the batch of the headline decode step), into the 8-bit cache.
        dict(name="append-decode-256", op="append", seqs=256, new_lo=1, new_hi=1, lo=16, hi=8192, heads=64,
             kv_heads=8, head_dim=128, block=16, rot=128, interleaved=False),
        # Prompt chunks of odd lengths that start inside a block, half of each head rotated in pairs.
        dict(name="append-chunks-ragged", op="append", seqs=9, new_lo=333, new_hi=1511, lo=0, hi=2001, heads=32,
             kv_heads=8, head_dim=128, block=16, rot=64, interleaved=True),
        # The smallest decode step: four sequences of up to 129 tokens.
        dict(name="attend-tiny", op="attend", seqs=4, lo=2, hi=129, mix=False, queries=1, heads=8, kv_heads=8,
             head_dim=64, block=16),
        # The headline decode batch: 256 sequences of mixed lengths on the 70B-shaped layer.
        dict(name="attend-mix-256", op="attend", seqs=256, lo=16, hi=8192, mix=True, queries=1, heads=64, kv_heads=8,
             head_dim=128, block=16),
        # Long contexts: eight sequences of 32k to 128k tokens.
        dict(name="attend-long-8", op="attend", seqs=8, lo=32768, hi=131072, mix=False, queries=1, heads=32,
             kv_heads=8, head_dim=128, block=16),
        # Verifying two drafted tokens of 64 sequences.
        dict(name="attend-verify-2", op="attend", seqs=64, lo=512, hi=2048, mix=False, queries=2, heads=64, kv_heads=8,
             head_dim=128, block=32),
        # One shared prefix of 1,030 tokens, read back for the next prompt chunk.
        dict(name="gather-prefix", op="gather", seqs=1, lo=1030, hi=1030, kv_heads=8, head_dim=128, block=8),
        # The prefixes of 64 sequences.
        dict(name="gather-64", op="gather", seqs=64, lo=512, hi=8192, kv_heads=8, head_dim=128, block=16),
        # One clone: a sequence that leaves a shared partial block.
        dict(name="copy-1", op="copy", pairs=1, kv_heads=8, head_dim=128, block=16, pool=4096),
        # A beam step's clones over a large pool.
        dict(name="copy-4000", op="copy", pairs=4000, kv_heads=8, head_dim=128, block=32, pool=12000),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "gather", "copy"])
    head_dim = rng.choice([64, 128])
    block = rng.choice([8, 16, 32])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    shape = dict(kv_heads=kv_heads, head_dim=head_dim, block=block)
    turn = dict(heads=kv_heads * group, rot=rng.choice([head_dim, head_dim // 2, head_dim // 4]),
                interleaved=rng.random() < 0.5)
    if op == "rope":
        return dict(op=op, tokens=_log_uniform(rng, 1, 8192), far=_log_uniform(rng, 16, 1 << 20), **shape, **turn)
    if op == "append":
        seqs = _log_uniform(rng, 1, 256)
        most = _log_uniform(rng, 1, max(1, 8192 // seqs))
        return dict(op=op, seqs=seqs, new_lo=rng.randint(1, most), new_hi=most, lo=0, hi=_log_uniform(rng, 16, 4096),
                    **shape, **turn)
    if op == "attend":
        seqs = _log_uniform(rng, 1, 256)
        hi = _log_uniform(rng, 16, min(131072, (1 << 20) // seqs))
        queries = rng.choice([1, 1, 2, 3, 5])
        group = rng.choice([g for g in (1, 2, 4, 8, 16) if g * (1 << (queries - 1).bit_length()) <= 16])
        return dict(op=op, seqs=seqs, lo=min(hi, queries), hi=hi, mix=False, queries=queries, heads=kv_heads * group,
                    **shape)
    if op == "gather":
        seqs = _log_uniform(rng, 1, 256)
        return dict(op=op, seqs=seqs, lo=1, hi=_log_uniform(rng, 16, (1 << 18) // seqs), **shape)
    pairs = _log_uniform(rng, 1, 4000)
    return dict(op=op, pairs=pairs, pool=3 * pairs + rng.randint(0, 64), **shape)


def _lengths(case):
    """The sequences' lengths before the call: the same for every seed, so that work() counts what runs."""
    rng = random.Random(7)
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    if case.get("mix"):
        return [min(hi, max(lo, round(math.exp(rng.gauss(math.log(600.0), 1.0))))) for _ in range(n)]
    return [rng.randint(lo, hi) for _ in range(n)]


def _new(case):
    rng = random.Random(8)
    return [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]


# -------------------------------------------------------------------- work
def work(case):
    hkv, d, b = case["kv_heads"], case["head_dim"], case["block"]
    if case["op"] == "rope":
        t, h = case["tokens"], case["heads"]
        return dict(bytes=2 * t * (h + 2 * hkv) * d * 2 + 16 * t + 2 * case["rot"], flops=3 * t * (h + hkv) * case["rot"])
    if case["op"] == "append":
        lens, new, h = _lengths(case), _new(case), case["heads"]
        t = sum(new)
        blocks = sum((p + n - 1) // b - p // b + 1 for p, n in zip(lens, new) if n)
        return dict(bytes=t * ((h + 2 * hkv) * d * 2 + h * d * 2 + 2 * hkv * d) + blocks * (4 + 2 * hkv * 4) + 8 * len(lens),
                    flops=t * (3 * (h + hkv) * case["rot"] + 4 * hkv * d))
    if case["op"] == "copy":
        return dict(bytes=case["pairs"] * (2 * 2 * hkv * (b * d + 4) + 16), flops=0)
    tokens = sum(_lengths(case))
    blocks = sum(-(-n // b) for n in _lengths(case))
    read = tokens * hkv * d * 2 + blocks * (4 + 2 * hkv * 4) + 4 * case["seqs"]
    if case["op"] == "gather":
        return dict(bytes=read + tokens * hkv * d * 2 * 2 + 8 * case["seqs"], flops=2 * tokens * hkv * d)
    rows = case["seqs"] * case["queries"] * case["heads"] * d
    return dict(bytes=read + rows * 2 * 2, flops=4 * tokens * case["queries"] * case["heads"] * d)


# ----------------------------------------------------------------- prepare
def _tables(lengths, block, gen):
    """Blocks for each sequence from a shuffled pool a tenth larger than they need; -1 behind the last."""
    need = [-(-n // block) for n in lengths]
    pool = max(4, int(1.1 * sum(need)) + 1)
    ids = torch.randperm(pool, generator=gen, device=DEVICE).to(torch.int32)
    count = torch.tensor(need, device=DEVICE)
    first = torch.cumsum(count, 0) - count
    at = torch.arange(max(1, max(need)), device=DEVICE)
    tables = torch.where(at < count[:, None], ids[(first[:, None] + at).clamp(max=pool - 1)], -1)
    return tables.to(torch.int32).contiguous(), pool


def _fp8_cache(pool, case, gen, strong):
    """A filled cache: unit values with a few strong channels and a gain for each block, quantised by its largest."""
    hkv, d, b = case["kv_heads"], case["head_dim"], case["block"]
    x = torch.randn(pool, hkv, b, d, generator=gen, device=DEVICE)
    x[..., :: max(1, d // 4)] *= strong
    x *= torch.exp(0.5 * torch.randn(pool, hkv, 1, 1, generator=gen, device=DEVICE))
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448.0)))
    x /= scale[:, :, None, None]
    return x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), scale.contiguous()


def _fill(s, pool, case, gen):
    s["k_cache"], s["k_scales"] = _fp8_cache(pool, case, gen, 6.0)
    s["v_cache"], s["v_scales"] = _fp8_cache(pool, case, gen, 1.0)


def _projection(tokens, case, gen):
    """The fused projection's output [tokens, (H + 2 Hkv) D] and its q, k, v: strided views, as a model has them."""
    h, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    qkv = torch.randn(tokens, h + 2 * hkv, d, generator=gen, device=DEVICE)
    qkv[:, : h + hkv, :: max(1, d // 4)] *= 3.0
    qkv = qkv.to(torch.bfloat16)
    return qkv[:, :h], qkv[:, h : h + hkv], qkv[:, h + hkv :]


def _frequencies(case):
    rot = case["rot"]
    return (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).to(torch.float32).to(DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, hkv, d, b = case["op"], case["kv_heads"], case["head_dim"], case["block"]
    s = dict(op=op, case=case)
    if op == "rope":
        t = case["tokens"]
        pool = -(-t // b) + 8
        q, k, v = _projection(t, case, gen)
        s.update(q=q, k=k, v=v, inv_freq=_frequencies(case), interleaved=case["interleaved"],
                 positions=torch.randint(0, case["far"], (t,), generator=gen, device=DEVICE),
                 slots=torch.randperm(pool * b, generator=gen, device=DEVICE)[:t].contiguous(),
                 k_cache=torch.zeros(pool, b, hkv, d, dtype=torch.bfloat16, device=DEVICE),
                 v_cache=torch.zeros(pool, b, hkv, d, dtype=torch.bfloat16, device=DEVICE))
        return s
    if op == "copy":
        pool, n = case["pool"], case["pairs"]
        _fill(s, pool, case, gen)
        s["pairs"] = torch.randperm(pool, generator=gen, device=DEVICE)[: 2 * n].reshape(n, 2).contiguous()
        return s
    lengths = _lengths(case)
    if op == "append":
        new = _new(case)
        lengths = [p + n for p, n in zip(lengths, new)]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        q, k, v = _projection(cu[-1], case, gen)
        s.update(q=q, k=k, v=v, inv_freq=_frequencies(case), interleaved=case["interleaved"], max_q_len=max(new),
                 cu_q_lens=torch.tensor(cu, dtype=torch.int32, device=DEVICE))
    s["block_tables"], pool = _tables(lengths, b, gen)
    s["seq_lens"] = torch.tensor(lengths, dtype=torch.int32, device=DEVICE)
    s["max_seq_len"] = max(lengths)
    _fill(s, pool, case, gen)
    if op == "attend":
        h, n = case["heads"], case["queries"]
        s["q"] = (2.0 * torch.randn(len(lengths) * n, h, d, generator=gen, device=DEVICE)).to(torch.bfloat16)
        s["cu_q_lens"] = torch.arange(0, len(lengths) * n + 1, n, dtype=torch.int32, device=DEVICE)
        s["scale"] = 1.0 / math.sqrt(d)
    if op == "gather":
        total = sum(lengths)
        s["cu_seq_lens"] = (torch.cumsum(s["seq_lens"].long(), 0) - s["seq_lens"].long()).contiguous()
        s["out_k"] = torch.empty(max(1, total), hkv, d, dtype=torch.bfloat16, device=DEVICE)
        s["out_v"] = torch.empty(max(1, total), hkv, d, dtype=torch.bfloat16, device=DEVICE)
        s["total"] = total
    return s


# --------------------------------------------------------------- plain forms
def _turned(x, cos, sin, rot, interleaved):
    """x [T, heads, D] in float32 with its first `rot` elements rotated; cos, sin [T, 1, rot / 2]."""
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        x1, x2 = a[..., 0::2], a[..., 1::2]
        y = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), dim=-1).flatten(-2)
    else:
        x1, x2 = a[..., : rot // 2], a[..., rot // 2 :]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), dim=-1)
    return torch.cat((y, rest), dim=-1)


def _angles(positions, inv_freq):
    angle = positions.double()[:, None] * inv_freq.double()      # far positions need 64 bits
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _plain_rope(s):
    rot = 2 * s["inv_freq"].shape[0]
    cos, sin = _angles(s["positions"], s["inv_freq"])
    q = _turned(s["q"].float(), cos, sin, rot, s["interleaved"]).to(torch.bfloat16)
    k = _turned(s["k"].float(), cos, sin, rot, s["interleaved"]).to(torch.bfloat16)
    b = s["k_cache"].shape[1]
    s["k_cache"][s["slots"] // b, s["slots"] % b] = k
    s["v_cache"][s["slots"] // b, s["slots"] % b] = s["v"]
    return q


def _needed_scale(m2):
    """The smallest 2^e, -64 <= e <= 64, with m2 <= (448 * 2^e)^2 (448^2 = 0.765625 * 2^18)."""
    f, k = torch.frexp(m2)
    e = (k + (f > 0.765625).to(k.dtype) - 17) >> 1
    e = torch.where(m2 > 0, e, -64).clamp(-64, 64)
    return torch.ldexp(torch.ones_like(m2), e)


def _bytes_of(cache):
    return cache.view(torch.uint8)


def _plain_write(cache, scales, y, m2, cell, phys, touched, older, start, pos):
    """The rows y [T, Hkv, D] of one cache, whose largest squares are m2 [T, Hkv]."""
    b = cache.shape[2]
    most = torch.zeros(touched.numel(), y.shape[1], device=DEVICE)
    most = most.scatter_reduce(0, cell[:, None].expand_as(m2), m2, "amax").view(*touched.shape, -1)
    at = phys[touched]
    had = torch.where(older[touched][:, None], scales[at], 0.0)
    scale = torch.maximum(_needed_scale(most[touched]), had)
    # Older rows of a block whose scale grows are rounded again.
    rows = torch.arange(b, device=DEVICE) < (start % b)[:, None, None].expand(*touched.shape, 1)[touched]
    rows = rows & older[touched][:, None]
    block = _bytes_of(cache)[at]
    values = block.view(torch.float8_e4m3fn).float() * torch.where(had > 0, had / scale, 1.0)[:, :, None, None]
    grown = _bytes_of(values.to(torch.float8_e4m3fn))
    _bytes_of(cache)[at] = torch.where(rows[:, None, :, None], grown, block)
    scales[at] = scale
    # The new rows.
    into = phys.flatten()[cell]
    held = (y / scales[into][..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    _bytes_of(cache)[into, :, pos % b] = _bytes_of(held)


def _plain_append(s):
    rot, b = 2 * s["inv_freq"].shape[0], s["k_cache"].shape[2]
    lens, cu = s["seq_lens"].long(), s["cu_q_lens"].long()
    new = cu[1:] - cu[:-1]
    row = torch.arange(s["q"].shape[0], device=DEVICE)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    pos = lens[seq] - new[seq] + row - cu[seq]
    cos, sin = _angles(pos, s["inv_freq"])
    q = _turned(s["q"].float(), cos, sin, rot, s["interleaved"]).to(torch.bfloat16)
    # Cells: the blocks that a sequence's new tokens touch, [sequence, touched block].
    start = lens - new
    wide = (s["max_q_len"] - 1) // b + 2
    cell = seq * wide + pos // b - start[seq] // b
    index = start[:, None] // b + torch.arange(wide, device=DEVICE)
    touched = (index * b < lens[:, None]) & (new[:, None] > 0)
    phys = s["block_tables"].long().gather(1, index.clamp(max=s["block_tables"].shape[1] - 1))
    older = touched & (index * b < start[:, None])               # the cell holds tokens of earlier calls
    cells = (cell, phys, touched, older, start, pos)
    x = s["k"].float()
    a = x[..., :rot]
    x1, x2 = (a[..., 0::2], a[..., 1::2]) if s["interleaved"] else (a[..., : rot // 2], a[..., rot // 2 :])
    m2 = torch.cat((x1 * x1 + x2 * x2, x[..., rot:] * x[..., rot:]), dim=-1).amax(-1)
    _plain_write(s["k_cache"], s["k_scales"], _turned(x, cos, sin, rot, s["interleaved"]), m2, *cells)
    x = s["v"].float()
    _plain_write(s["v_cache"], s["v_scales"], x, (x * x).amax(-1), *cells)
    return q


def _pages(cache, scales, tables):
    """[sequence, KV head, token, element] in float32 of what the tables name."""
    at = tables.long().clamp(min=0)
    x = _bytes_of(cache)[at].view(torch.float8_e4m3fn).float()
    x *= scales[at][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    lens, cu = s["seq_lens"].long(), s["cu_q_lens"].long()
    n, hkv = lens.shape[0], s["k_cache"].shape[1]
    t, h, d = s["q"].shape
    m = s["case"]["queries"]
    q = s["q"].float().view(n, m, hkv, h // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, m * (h // hkv), d)
    k = _pages(s["k_cache"], s["k_scales"], s["block_tables"])
    scores = (q @ k.transpose(2, 3)) * s["scale"]
    del k
    last = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(m, device=DEVICE)      # a query's own position
    seen = torch.arange(scores.shape[3], device=DEVICE) <= last.repeat_interleave(h // hkv, dim=1)[..., None]
    scores = torch.where(seen[:, None], scores, -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    del scores
    v = _pages(s["v_cache"], s["v_scales"], s["block_tables"])
    out = (p @ v) / p.sum(-1, keepdim=True)
    return out.view(n, hkv, m, h // hkv, d).permute(0, 2, 1, 3, 4).reshape(t, h, d).to(torch.bfloat16)


def _plain_gather(s):
    b = s["k_cache"].shape[2]
    row = torch.arange(s["total"], device=DEVICE)
    seq = torch.searchsorted(torch.cumsum(s["seq_lens"].long(), 0), row, right=True)
    pos = row - s["cu_seq_lens"][seq]
    at = s["block_tables"].long()[seq, pos // b]
    k = _bytes_of(s["k_cache"])[at, :, pos % b].view(torch.float8_e4m3fn).float()
    v = _bytes_of(s["v_cache"])[at, :, pos % b].view(torch.float8_e4m3fn).float()
    s["out_k"][: s["total"]] = (k * s["k_scales"][at][..., None]).to(torch.bfloat16)
    s["out_v"][: s["total"]] = (v * s["v_scales"][at][..., None]).to(torch.bfloat16)


def _plain_copy(s):
    src, dst = s["pairs"][:, 0], s["pairs"][:, 1]
    _bytes_of(s["k_cache"])[dst] = _bytes_of(s["k_cache"])[src]
    _bytes_of(s["v_cache"])[dst] = _bytes_of(s["v_cache"])[src]
    s["k_scales"][dst] = s["k_scales"][src]
    s["v_scales"][dst] = s["v_scales"][src]


# --------------------------------------------------------------------- run
def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_122_gb300 as pk
    if op == "rope":
        if own:
            q = pk.rope_and_cache(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                                  s["inv_freq"], interleaved=s["interleaved"])
        else:
            q = _plain_rope(s)
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op == "append":
        if own:
            q = pk.rope_and_cache_fp8(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                      s["block_tables"], s["seq_lens"], s["inv_freq"], cu_q_lens=s["cu_q_lens"],
                                      max_q_len=s["max_q_len"], interleaved=s["interleaved"])
        else:
            q = _plain_append(s)
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    if op == "attend":
        if not own:
            return _plain_attend(s)
        if s["case"]["queries"] == 1:
            return pk.paged_attention_decode_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                                 s["block_tables"], s["seq_lens"], s["scale"],
                                                 max_seq_len=s["max_seq_len"])
        return pk.paged_attention_multi_query_fp8(s["q"], s["cu_q_lens"], s["case"]["queries"], s["k_cache"],
                                                  s["v_cache"], s["k_scales"], s["v_scales"], s["block_tables"],
                                                  s["seq_lens"], s["scale"], max_seq_len=s["max_seq_len"])
    if op == "gather":
        if own:
            pk.gather_kv_fp8(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["block_tables"],
                             s["seq_lens"], s["cu_seq_lens"], s["out_k"], s["out_v"], max_seq_len=s["max_seq_len"])
        else:
            _plain_gather(s)
        return dict(k=s["out_k"][: s["total"]], v=s["out_v"][: s["total"]])
    if own:
        pk.copy_blocks_fp8(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["pairs"])
    else:
        _plain_copy(s)
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"])


# ------------------------------------------------------------------- exact
def _exact_turn(x, positions, inv_freq, interleaved):
    """Complex rotation in 64 bits: the pair (a, b) is a + ib, times e^(i position frequency)."""
    r = inv_freq.shape[0]
    x = x.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                       positions.double()[:, None] * inv_freq.double())[:, None]
    if interleaved:
        z = torch.view_as_complex(x[..., : 2 * r].reshape(*x.shape[:-1], r, 2).contiguous()) * turn
        x[..., : 2 * r] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :r].contiguous(), x[..., r : 2 * r].contiguous()) * turn
        x[..., :r], x[..., r : 2 * r] = z.real, z.imag
    return x


def _exact_append(s):
    """Sequence by sequence and block by block, the values as they are before they are rounded to 8 bits."""
    r, b = s["inv_freq"].shape[0], s["k_cache"].shape[2]
    lens, cu, tables = s["seq_lens"].tolist(), s["cu_q_lens"].tolist(), s["block_tables"].tolist()
    pos = torch.cat([torch.arange(n - (cu[i + 1] - cu[i]), n, device=DEVICE) for i, n in enumerate(lens)])
    out = dict(q=_exact_turn(s["q"], pos, s["inv_freq"], s["interleaved"]))
    for name, x in (("k", s["k"]), ("v", s["v"])):
        x64 = x.double()
        y = _exact_turn(x, pos, s["inv_freq"], s["interleaved"]) if name == "k" else x64
        size2 = x64 * x64
        if name == "k":
            head = size2[..., : 2 * r]
            pair = head.unflatten(-1, (r, 2)).sum(-1) if s["interleaved"] else head[..., :r] + head[..., r:]
            size2 = torch.cat((pair, size2[..., 2 * r :]), dim=-1)
        need = size2.amax(-1).float().double().sqrt() / 448.0                    # [T, Hkv]; the sum is defined in 32 bits
        cache, scales = s[name + "_cache"].double(), s[name + "_scales"].double()
        for i, n in enumerate(lens):
            at = n - (cu[i + 1] - cu[i])
            while at < n:
                end = min(n, (at // b + 1) * b)
                lo = cu[i + 1] - (n - at)
                f, e = torch.frexp(need[lo : lo + end - at].amax(0))         # need = f 2^e, 0.5 <= f < 1
                scale = torch.exp2((e - (f == 0.5).to(e.dtype)).double()).clamp(2.0**-64, 2.0**64)
                block = tables[i][at // b]
                if at % b:
                    scale = torch.maximum(scale, scales[block])
                    cache[block, :, : at % b] *= (scales[block] / scale)[:, None, None]
                scales[block] = scale
                cache[block, :, at % b : at % b + end - at] = (y[lo : lo + end - at] / scale[:, None]).transpose(0, 1)
                at = end
        out[name + "_cache"], out[name + "_scales"] = cache, scales
    return out


def _exact_rows(cache, scales, blocks, n):
    x = cache.view(torch.uint8)[blocks].view(torch.float8_e4m3fn).double() * scales[blocks].double()[..., None, None]
    return x.permute(0, 2, 1, 3).flatten(0, 1)[:n]                               # [n, Hkv, D]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        b = case["block"]
        out = dict(q=_exact_turn(s["q"], s["positions"], s["inv_freq"], s["interleaved"]),
                   k_cache=s["k_cache"].double(), v_cache=s["v_cache"].double())
        block, row = torch.div(s["slots"], b, rounding_mode="floor"), s["slots"].remainder(b)
        out["k_cache"][block, row] = _exact_turn(s["k"], s["positions"], s["inv_freq"], s["interleaved"])
        out["v_cache"][block, row] = s["v"].double()
        return out
    if op == "append":
        return _exact_append(s)
    if op == "copy":
        out = {name: s[name].double() for name in ("k_cache", "v_cache", "k_scales", "v_scales")}
        src, dst = s["pairs"].unbind(1)
        return {name: x.index_copy(0, dst, x.index_select(0, src)) for name, x in out.items()}
    lens = s["seq_lens"].tolist()
    rows = {"k": [], "v": []}
    outs = []
    for i, n in enumerate(lens):
        blocks = s["block_tables"][i, : -(-n // case["block"])].long()
        k = _exact_rows(s["k_cache"], s["k_scales"], blocks, n)
        v = _exact_rows(s["v_cache"], s["v_scales"], blocks, n)
        if op == "gather":
            rows["k"].append(k)
            rows["v"].append(v)
            continue
        m, h, hkv = case["queries"], case["heads"], case["kv_heads"]
        q = s["q"][i * m : (i + 1) * m].double().unflatten(1, (hkv, h // hkv))
        scores = torch.einsum("mhgd,nhd->mhgn", q, k) * s["scale"]
        own_at = n - m + torch.arange(m, device=DEVICE)
        hidden = torch.arange(n, device=DEVICE)[None] > own_at[:, None]
        scores = scores.masked_fill(hidden[:, None, None], -math.inf)
        weights = torch.exp(scores - torch.logsumexp(scores, -1, keepdim=True))
        outs.append(torch.einsum("mhgn,nhd->mhgd", weights, v).flatten(1, 2))
    if op == "gather":
        return {name: torch.cat(x) for name, x in rows.items()}
    return torch.cat(outs)
