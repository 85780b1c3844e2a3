"""The operators of tree verification and of cross attention over the paged cache, as they are measured.

tree      paged_attention_tree: each sequence's newest tokens are a tree of
          drafted tokens; a token attends to the whole context before the tree
          and to those tokens of the tree that its row of a bit mask names
cross     paged_attention_cross: any number of query rows a sequence over keys
          of another length (an encoder's states), all of them visible
accept    accept_tree: the path from the root of each tree whose every token is
          the target model's choice after its parent (the lowest child on ties)
keep      pk_keep_tokens_layers: the accepted tokens' K and V rows move to the
          front of the tree's place in the cache, in every layer

The cache is the bf16 paged one, [num_blocks, block_size, num_kv_heads, head_dim]
for K and for V, read through block tables.  Bit i % 64 of word i / 64 of a
token's mask row says whether it sees token i of its tree.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # Four short sequences on a small model, three to five drafts each: the launch counts, not the bytes.
        dict(name="tree-tiny", op="tree", seqs=4, lo=1, hi=120, nodes_lo=3, nodes_hi=5, heads=8, kv_heads=8,
             head_dim=64, block=16),
        # A serving batch on the 8B-shaped layer, about two dozen drafts a sequence.
        dict(name="tree-batch-64", op="tree", seqs=64, lo=512, hi=2048, nodes_lo=17, nodes_hi=26, heads=32, kv_heads=8,
             head_dim=128, block=16),
        # Long contexts: eight sequences of 32k to 128k tokens, eight drafts each.
        dict(name="tree-long-8", op="tree", seqs=8, lo=32768, hi=131072, nodes_lo=8, nodes_hi=8, heads=32, kv_heads=8,
             head_dim=128, block=16),
        # Wide trees on the 70B-shaped layer, 65 to 100 drafts: more than one word of mask, several query tiles.
        dict(name="tree-wide-32", op="tree", seqs=32, lo=512, hi=8192, nodes_lo=65, nodes_hi=100, heads=64, kv_heads=8,
             head_dim=128, block=32),
        # A decoder step of a few ragged rows over encoder states of odd lengths, an empty one among them.
        dict(name="cross-ragged-9", op="cross", seqs=9, lo=0, hi=1500, rows_lo=1, rows_hi=5, heads=16, kv_heads=16,
             head_dim=64, block=8),
        # Decoder prompts of about 400 rows over 1,500 encoder states.
        dict(name="cross-prompt-16", op="cross", seqs=16, lo=1500, hi=1500, rows_lo=333, rows_hi=448, heads=16,
             kv_heads=16, head_dim=64, block=16),
        # Long inputs: 1,024 rows over 8k to 16k states with shared heads.
        dict(name="cross-long-4", op="cross", seqs=4, lo=8192, hi=16384, rows_lo=1024, rows_hi=1024, heads=32,
             kv_heads=8, head_dim=128, block=32),
        # One tree of five drafts.
        dict(name="accept-1", op="accept", seqs=1, nodes_lo=5, nodes_hi=5),
        # A large batch with trees of up to 512 drafts.
        dict(name="accept-256", op="accept", seqs=256, nodes_lo=100, nodes_hi=512),
        # A model of two layers, three sequences: the launch counts.
        dict(name="keep-3x2", op="keep", seqs=3, nodes_lo=3, nodes_hi=9, layers=2, ctx=40, kv_heads=8, head_dim=64,
             block=16),
        # A serving batch over 32 layers.
        dict(name="keep-128x32", op="keep", seqs=128, nodes_lo=17, nodes_hi=26, layers=32, ctx=40, kv_heads=8,
             head_dim=128, block=16),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "cross", "cross", "accept", "keep"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 8, 16])
    head_dim, block = rng.choice([64, 128]), rng.choice([8, 16, 32])
    shape = dict(heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, block=block)
    seqs = _log_uniform(rng, 1, 256)
    if op in ("tree", "cross"):
        most = _log_uniform(rng, 1, 300) if op == "tree" else _log_uniform(rng, 1, 1024)
        hi = _log_uniform(rng, 16, min(131072, (1 << 20) // seqs))
        # No more than the largest listed case: 8 * 10^11 operations.
        while 4 * seqs * most * shape["heads"] * (hi + most) * head_dim > 8e11:
            hi, most = max(16, hi // 2), max(1, most // 2)
        if op == "tree":
            return dict(op=op, seqs=seqs, lo=rng.choice([0, hi // 2]), hi=hi, nodes_lo=rng.randint(1, most),
                        nodes_hi=most, **shape)
        return dict(op=op, seqs=seqs, lo=rng.choice([0, hi // 2]), hi=hi, rows_lo=rng.randint(0, most), rows_hi=most,
                    **shape)
    most = _log_uniform(rng, 1, 512)
    if op == "accept":
        return dict(op=op, seqs=seqs, nodes_lo=rng.randint(1, most), nodes_hi=most)
    most = min(most, 64)
    seqs = min(seqs, 128)
    layers = rng.randint(1, 32)
    return dict(op=op, seqs=seqs, nodes_lo=rng.randint(1, most), nodes_hi=most, layers=layers, ctx=rng.randint(0, 40),
                kv_heads=kv_heads, head_dim=head_dim, block=block)


def _counts(case, salt, lo, hi):
    """Lengths of the case's sequences: the same for every seed, so that work() counts what runs."""
    rng = random.Random(salt)
    return [rng.randint(case[lo], case[hi]) for _ in range(case["seqs"])]


def _lengths(case):
    """(keys, query rows) of each sequence; the keys of a tree include its own tokens."""
    if case["op"] == "cross":
        rows = _counts(case, 8, "rows_lo", "rows_hi")
        keys = _counts(case, 7, "lo", "hi")
        rows[0] = rows[0] or case["rows_hi"]
        if case["lo"] == 0 and len(keys) > 1:
            keys[len(keys) // 2] = 0
        return keys, rows
    rows = _counts(case, 8, "nodes_lo", "nodes_hi")
    if case["op"] == "tree":
        return [c + n for c, n in zip(_counts(case, 7, "lo", "hi"), rows)], rows
    if case["op"] == "keep":
        rng = random.Random(7)
        return [rng.randint(0, case["ctx"]) + n for n in rows], rows
    return [100 + n for n in rows], rows


def _parents(n, rng):
    """A tree of n drafts: each hangs below one of the last few before it."""
    return [-1] + [rng.randrange(max(0, r - 7), r) for r in range(1, n)]


def _paths(case):
    """The accepted nodes of each tree of a keep case: the root and a path below it."""
    rng = random.Random(9)
    out = []
    for n in _lengths(case)[1]:
        parents = _parents(n, rng)
        node, path = rng.randrange(n), []
        while node >= 0:
            path.append(node)
            node = parents[node]
        out.append(path[::-1])
    return out


# -------------------------------------------------------------------- work
def work(case):
    keys, rows = _lengths(case)
    n = case["seqs"]
    if case["op"] == "accept":
        return dict(bytes=sum(rows) * (8 + 4 + 8) + n * (max(rows) * 4 + 4 + 8 + 4 + 4 + 4), flops=0)
    hkv, d, b = case["kv_heads"], case["head_dim"], case["block"]
    if case["op"] == "keep":
        moved = sum(sum(i != x for i, x in enumerate(path)) for path in _paths(case))
        return dict(bytes=case["layers"] * moved * 2 * 2 * hkv * d * 2 + sum(map(len, _paths(case))) * 4 + n * 12, flops=0)
    h = case["heads"]
    read = sum(k for k, r in zip(keys, rows) if r)
    blocks = sum(-(-k // b) for k, r in zip(keys, rows) if r)
    mask = sum(rows) * 8 * -(-max(rows) // 64) if case["op"] == "tree" else 0
    return dict(bytes=read * hkv * d * 2 * 2 + 2 * sum(rows) * h * d * 2 + 4 * blocks + mask + 8 * n,
                flops=4 * sum(k * r for k, r in zip(keys, rows)) * h * d)


# ----------------------------------------------------------------- prepare
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEVICE)


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


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


def _mask_rows(parents, words):
    """Ancestors and self of every node, as signed 64-bit words."""
    seen, out = [], []
    for r, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | 1 << r)
        row = [seen[r] >> 64 * w & (1 << 64) - 1 for w in range(words)]
        out.append([x - (1 << 64) if x >> 63 else x for x in row])
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    op = case["op"]
    keys, rows = _lengths(case)
    s = dict(op=op, case=case, keys=keys, rows=rows, starts=_starts(rows), max_q_len=max(rows),
             cu_q_lens=_ints(_starts(rows)), seq_lens=_ints(keys))
    if op == "accept":
        # Drafts below one node have tokens of their own; the target often agrees with one of them.
        parents, tokens, targets = [], [], []
        for n in rows:
            tree = _parents(n, rng)
            token = rng.sample(range(32000), n)
            below = [[] for _ in range(n)]
            for r in range(1, n):
                below[tree[r]].append(r)
            parents += tree
            tokens += token
            targets += [token[rng.choice(c)] if c and rng.random() < 0.9 else rng.randrange(32000) for c in below]
        s.update(parents=_ints(parents), tokens=_ints(tokens, torch.int64), targets=_ints(targets, torch.int64))
        return s
    hkv, d, b = case["kv_heads"], case["head_dim"], case["block"]
    s["block_tables"], pool = _tables(keys, b, gen)
    if op == "keep":
        def rows_of(_):
            return torch.randn(pool, b, hkv, d, generator=gen, device=DEVICE, dtype=torch.bfloat16)
        paths = _paths(case)
        width = max(rows)
        s.update(k=[rows_of(i) for i in range(case["layers"])], v=[rows_of(i) for i in range(case["layers"])],
                 accepted=_ints([p + [-1] * (width - len(p)) for p in paths]), num_accepted=_ints([len(p) for p in paths]))
        if own:
            import paged_kv_cache_122_gb300 as pk
            s["k_layers"], s["v_layers"] = pk.LayerPointers(s["k"]), pk.LayerPointers(s["v"])
        return s
    total, h = sum(rows), case["heads"]
    s["k_cache"] = torch.randn(pool, b, hkv, d, generator=gen, device=DEVICE, dtype=torch.bfloat16)
    s["v_cache"] = torch.randn(pool, b, hkv, d, generator=gen, device=DEVICE, dtype=torch.bfloat16)
    s["q"] = (2.0 * torch.randn(total, h, d, generator=gen, device=DEVICE)).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(d)
    s["max_seq_len"] = max(keys)
    if op == "tree":
        words = -(-max(rows) // 64)
        mask = [row for n in rows for row in _mask_rows(_parents(n, rng), words)]
        s["tree_mask"] = _ints(mask, torch.int64)
    return s


# --------------------------------------------------------------- plain forms
def _plain_attention(s):
    """Sequence by sequence: gather the rows, scores, mask, softmax, weighted sum."""
    t, h, d = s["q"].shape
    b, hkv = s["k_cache"].shape[1:3]
    out = torch.zeros(t, h, d, dtype=torch.bfloat16, device=DEVICE)
    for i, (n, m) in enumerate(zip(s["keys"], s["rows"])):
        if n == 0 or m == 0:
            continue
        lo = s["starts"][i]
        at = s["block_tables"][i, : -(-n // b)].long()
        k = s["k_cache"][at].flatten(0, 1)[:n].float().permute(1, 2, 0)              # [Hkv, D, n]
        v = s["v_cache"][at].flatten(0, 1)[:n].float().transpose(0, 1)               # [Hkv, n, D]
        q = s["q"][lo : lo + m].float().view(m, hkv, h // hkv, d).permute(1, 0, 2, 3).reshape(hkv, -1, d)
        scores = (q @ k).mul_(s["scale"])                                            # [Hkv, m * G, n]
        if s["op"] == "tree":
            node = torch.arange(m, device=DEVICE)
            sees = (s["tree_mask"][lo : lo + m][:, node // 64] >> (node % 64)) & 1   # [m, m]
            hidden = (sees == 0).repeat_interleave(h // hkv, dim=0)
            scores[:, :, n - m :].masked_fill_(hidden, -math.inf)
        most = scores.amax(-1, keepdim=True).clamp_(min=-3e38)
        p = scores.sub_(most).exp_()
        x = (p @ v) / p.sum(-1, keepdim=True).clamp_(min=1e-38)
        out[lo : lo + m] = x.view(hkv, m, h // hkv, d).permute(1, 0, 2, 3).reshape(m, h, d).to(torch.bfloat16)
    return out


def _plain_accept(s):
    """All trees at once, one level a step."""
    width, n = s["max_q_len"], len(s["rows"])
    cu, lens = s["cu_q_lens"].long(), s["seq_lens"]
    first, count = cu[:-1], cu[1:] - cu[:-1]
    node = torch.arange(width, device=DEVICE)
    at = (first[:, None] + node).clamp(max=s["tokens"].shape[0] - 1)
    inside = (node < count[:, None]) & (node > 0)
    parents = torch.where(inside, s["parents"].long()[at], -1)
    wanted = s["targets"][at].gather(1, parents.clamp(min=0)) == s["tokens"][at]
    # The lowest child of each node that the target chose, or `width`.
    child = torch.full((n, width + 1), width, device=DEVICE)
    child.scatter_reduce_(1, torch.where(inside & wanted, parents, width), node.expand(n, width).contiguous(), "amin")
    child[:, width] = width
    path = torch.full((n, width), -1, device=DEVICE)
    cur = torch.zeros(n, 1, dtype=torch.long, device=DEVICE)
    last = cur.clone()
    for i in range(width):
        path[:, i : i + 1] = torch.where(cur < width, cur, -1)
        last = torch.where(cur < width, cur, last)
        cur = child.gather(1, cur)
    num = (path >= 0).sum(1)
    following = s["targets"][first + last[:, 0]]
    return path.int(), num.int(), following, (lens - count + num).int()


def _plain_keep(s):
    b = s["case"]["block"]
    width = s["accepted"].shape[1]
    base = s["seq_lens"].long() - (s["cu_q_lens"][1:] - s["cu_q_lens"][:-1]).long()
    i = torch.arange(width, device=DEVICE)
    kept = i < s["num_accepted"][:, None]

    def slots(pos):
        return s["block_tables"].long().gather(1, pos // b) * b + pos % b
    src = slots(base[:, None] + torch.where(kept, s["accepted"].long(), 0)).flatten()
    dst = slots(base[:, None] + torch.where(kept, i, 0)).flatten()      # behind the path: the root onto itself
    for cache in s["k"] + s["v"]:
        flat = cache.flatten(0, 1)
        flat[dst] = flat[src]


# --------------------------------------------------------------------- run
def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_122_gb300 as pk
    if op == "tree":
        if not own:
            return _plain_attention(s)
        return pk.paged_attention_tree(s["q"], s["cu_q_lens"], s["max_q_len"], s["tree_mask"], s["k_cache"], s["v_cache"],
                                       s["block_tables"], s["seq_lens"], s["scale"], max_seq_len=s["max_seq_len"])
    if op == "cross":
        if not own:
            return _plain_attention(s)
        return pk.paged_attention_cross(s["q"], s["cu_q_lens"], s["max_q_len"], s["k_cache"], s["v_cache"],
                                        s["block_tables"], s["seq_lens"], s["scale"], max_seq_len=s["max_seq_len"])
    if op == "accept":
        if own:
            path, num, following, lens = pk.accept_tree(s["tokens"], s["parents"], s["targets"], s["cu_q_lens"],
                                                        s["max_q_len"], s["seq_lens"])
        else:
            path, num, following, lens = _plain_accept(s)
        return dict(accepted=path, num_accepted=num, next_tokens=following, seq_lens=lens)
    if own:
        pk.pk_keep_tokens_layers(s["k_layers"], s["v_layers"], s["block_tables"], s["seq_lens"], s["cu_q_lens"],
                                 s["accepted"], s["num_accepted"])
    else:
        _plain_keep(s)
    return dict(k=s["k"], v=s["v"])


# ------------------------------------------------------------------- exact
def _exact_tokens(cache, table, n):
    """The first n tokens of a sequence, one block after the other, in 64 bits: [n, Hkv, D]."""
    b = cache.shape[1]
    return torch.cat([cache[block, : min(b, n - b * j)].double() for j, block in enumerate(table[: -(-n // b)])])


def _exact_attention(s):
    outs = []
    hkv = s["k_cache"].shape[2]
    tables = s["block_tables"].tolist()
    for i, (n, m) in enumerate(zip(s["keys"], s["rows"])):
        q = s["q"][s["starts"][i] : s["starts"][i] + m].double()
        if n == 0 or m == 0:
            outs.append(torch.zeros_like(q))
            continue
        k, v = _exact_tokens(s["k_cache"], tables[i], n), _exact_tokens(s["v_cache"], tables[i], n)
        sees = torch.ones(m, n, dtype=torch.bool)
        if s["op"] == "tree":
            for r, words in enumerate(s["tree_mask"][s["starts"][i] : s["starts"][i] + m].tolist()):
                for node in range(m):
                    sees[r, n - m + node] = bool(words[node >> 6] >> (node & 63) & 1)
        sees = sees.to(DEVICE)
        heads = []
        for h in range(q.shape[1]):
            g = h * hkv // q.shape[1]
            scores = torch.einsum("md,nd->mn", q[:, h], k[:, g]) * s["scale"]
            scores = torch.where(sees, scores, -math.inf)
            total = torch.logsumexp(scores, -1, keepdim=True)
            weights = torch.where(sees, torch.exp(scores - total), 0.0)
            heads.append(torch.einsum("mn,nd->md", weights, v[:, g]))
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("tree", "cross"):
        return _exact_attention(s)
    width = s["max_q_len"]
    if case["op"] == "accept":
        parents, tokens, targets = s["parents"].tolist(), s["tokens"].tolist(), s["targets"].tolist()
        paths, following, lens = [], [], []
        for i, n in enumerate(s["rows"]):
            lo = s["starts"][i]
            path = [0]
            for r in range(1, n):
                if parents[lo + r] == path[-1] and tokens[lo + r] == targets[lo + path[-1]]:
                    path.append(r)
            paths.append(path + [-1] * (width - len(path)))
            following.append(targets[lo + path[-1]])
            lens.append(s["keys"][i] - n + len(path))
        return dict(accepted=_ints(paths), num_accepted=_ints([sum(x >= 0 for x in p) for p in paths]),
                    next_tokens=_ints(following, torch.int64), seq_lens=_ints(lens))
    tables, b = s["block_tables"].tolist(), case["block"]
    out = dict(k=[x.double() for x in s["k"]], v=[x.double() for x in s["v"]])
    pairs = []
    for i, path in enumerate(_paths(case)):
        base = s["keys"][i] - s["rows"][i]
        pairs += [(base + x, base + j, i) for j, x in enumerate(path) if x != j]
    for x in out["k"] + out["v"]:
        old = x.clone()
        if pairs:
            sb, sr = zip(*[(tables[i][a // b], a % b) for a, _, i in pairs])
            db, dr = zip(*[(tables[i][c // b], c % b) for _, c, i in pairs])
            x[list(db), list(dr)] = old[list(sb), list(sr)]
    return out
