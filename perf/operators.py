"""Speed and accuracy cases of the serving-step operators: the cache write and read
(16-bit or fp32 rows, q8 and q4), attention for a tree of drafted tokens over the paged
q8 cache with the commit of the accepted path, and causal attention over packed prompts.

``run`` computes each operator in plain torch operations, or, with ``own`` set, through
the library's entry points.  Both work on the pool layout that include/kq8.h documents.
"""
import math
import random

import torch

own = False

HD = 128          # head dim of every kq8 cache
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one verify step of a speculative decoder: the drafts' K and V are written, the tree
        # attends, the accepted path moves to its place and is read back (for the draft model).
        # Qwen3-VL-2B heads, one user, the shortest of the pages' contexts, a small tree: latency
        dict(name="verify_b1_n506", op="verify", B=1, nq=16, nkv=8, lo=506, hi=506, nodes=8,
             type="bf16", kv_bs=32, shape=1),
        # the batch-64 serving layer (Qwen3-VL-8B heads, ragged contexts), 8 nodes a user
        dict(name="verify_b64_serving", op="verify", B=64, nq=32, nkv=8, lo=1024, hi=32768, nodes=8,
             type="bf16", kv_bs=32, shape=2),
        # few users, wide trees: 64 nodes x 4 query heads share each KV head
        dict(name="tree_b8_64nodes", op="tree", B=8, nq=32, nkv=8, lo=16384, hi=16384, nodes=64,
             type="bf16", kv_bs=64, shape=3),
        # long contexts of odd length at fp32, a 26-node tree
        dict(name="tree_long_fp32", op="tree", B=2, nq=16, nkv=8, lo=100003, hi=131072, nodes=26,
             type="fp32", kv_bs=32, shape=4),
        # the new tokens of one decode step of 64 users, out of a fused QKV projection
        dict(name="write_read_step", op="write_read", T=64, nq=32, nkv=8, bits=8, type="bf16",
             kv_bs=32, shape=5),
        # the prompts of a prefill chunk, 8 x 4096 tokens
        dict(name="write_read_bulk", op="write_read", T=32768, nq=16, nkv=8, bits=8, type="bf16",
             kv_bs=32, shape=6),
        # the same at 4 bits and fp16, an odd number of tokens
        dict(name="write_read_q4", op="write_read", T=8193, nq=32, nkv=8, bits=4, type="fp16",
             kv_bs=64, shape=7),
        # one 2B prompt's cache read back in fp32
        dict(name="read_4059_fp32", op="read", T=4059, nkv=8, bits=8, type="fp32", kv_bs=32, shape=8),
        # a long context read back for another model
        dict(name="read_131072", op="read", T=131072, nkv=8, bits=8, type="bf16", kv_bs=32, shape=9),
        # a short prompt, and the longest of the pages' prompts, Qwen3-VL-2B heads
        dict(name="prompt_506", op="prompt", B=1, nq=16, nkv=8, lo=506, hi=506, type="bf16", shape=10),
        dict(name="prompt_4059", op="prompt", B=1, nq=16, nkv=8, lo=4059, hi=4059, type="bf16",
             shape=11),
        # four packed prompts of different lengths up to the 8B prompt's 8192
        dict(name="prompt_packed_8b", op="prompt", B=4, nq=32, nkv=8, lo=1000, hi=8192, type="bf16",
             shape=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["verify", "tree", "write_read", "read", "prompt"])
    shape = rng.randrange(1 << 30)
    nkv = rng.choice([1, 2, 4, 8])
    nq = nkv * rng.choice([1, 2, 3, 4, 5, 8])
    kv_bs = rng.choice([32, 64, 128, 256])
    if op in ("verify", "tree"):
        B, nodes = _log(rng, 1, 64), _log(rng, 1, 64)
        hi = max(nodes, _log(rng, 40, min(131072, (1 << 20) // B, (1 << 28) // (B * nodes * nq))))
        return dict(op=op, B=B, nq=nq, nkv=nkv, lo=max(nodes, rng.randint(hi // 3, hi)), hi=hi, nodes=nodes,
                    type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), kv_bs=kv_bs, shape=shape)
    if op in ("write_read", "read"):
        c = dict(op=op, T=_log(rng, 1, 65536 // nkv * 4), nkv=nkv, bits=rng.choice([8, 8, 4]),
                 type=rng.choice(["bf16", "fp16", "fp32"]), kv_bs=kv_bs, shape=shape)
        if op == "write_read":
            c["nq"] = nq
        return c
    B = _log(rng, 1, 16)
    hi = _log(rng, 1, min(8192, int(8192 * math.sqrt(128 / (B * nq)))))
    return dict(op=op, B=B, nq=nq, nkv=nkv, lo=rng.randint(max(1, hi // 8), hi), hi=hi,
                type=rng.choice(["bf16", "bf16", "fp16"]), shape=shape)


def _lens(case):
    """Lengths of the case's sequences: between lo and hi, the first one hi."""
    r = random.Random(case["shape"])
    return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]


def _nodes(case, lens):
    """Nodes of each sequence's tree; a batch's trees differ in size."""
    r = random.Random(case["shape"] + 1)
    return [min(n, case["nodes"] if b == 0 else r.randint(max(1, case["nodes"] // 2), case["nodes"]))
            for b, n in enumerate(lens)]


def _trees(case, nodes):
    """(mask bits of each node's ancestors and itself, accepted path) of each sequence."""
    r = random.Random(case["shape"] + 2)
    masks, paths = [], []
    for nb in nodes:
        rows, parent = [], []
        for i in range(nb):
            parent.append(r.randint(max(-1 if i else 0, i - 6), i - 1) if i else -1)
            rows.append((rows[parent[i]] if parent[i] >= 0 else 0) | (1 << i))
        at, path = r.randrange(nb), []
        while at >= 0:
            path.append(at)
            at = parent[at]
        masks.append(rows)
        paths.append(path[::-1])
    return masks, paths


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _pool(pages, nkv, kv_bs, bits, g):
    """A pool as a running server holds it: rows of normal values, per-head spreads of 0.5 to 3."""
    row = HD if bits == 8 else HD // 2
    if bits == 8:
        def codes(shape):
            c = torch.empty(shape, dtype=torch.int8, device=DEV)
            flat, step = c.view(-1), 1 << 28
            for o in range(0, flat.numel(), step):
                part = flat[o:o + step]
                part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(45.0).round_().clamp_(-127, 127))
            return c
    else:
        def codes(shape):  # two offset nibbles of 1 .. 15 in a byte
            return (torch.randint(1, 16, shape, generator=g, device=DEV)
                    + 16 * torch.randint(1, 16, shape, generator=g, device=DEV)).to(torch.uint8).view(torch.int8)
    k, v = codes((pages, nkv, kv_bs // 32, 4, 32, row // 4)), codes((pages, nkv, kv_bs, row))
    spread = 0.5 + 2.5 * torch.rand((2, 1, nkv, 1), generator=g, device=DEV)
    ks = spread[0] * (2.4 + torch.rand((pages, nkv, kv_bs), generator=g, device=DEV))
    vs = spread[1] * (2.4 + torch.rand((pages, nkv, kv_bs), generator=g, device=DEV))
    return dict(k=k, v=v, ks=ks, vs=vs, kv_bs=kv_bs, nkv=nkv, bits=bits)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + case["shape"])
    r = random.Random(seed * 1000003 + case["shape"])
    t = TYPES[case["type"]]
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(t)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    if case["op"] == "prompt":
        lens = _lens(case)
        off = [0]
        for n in lens:
            off.append(off[-1] + n)
        nq, nkv = case["nq"], case["nkv"]
        qkv = randn(off[-1], nq + 2 * nkv, HD)
        qkv[:, nq:nq + nkv] *= 0.5 + 1.5 * torch.rand((1, nkv, 1), generator=g, device=DEV).to(t)
        s.update(q=qkv[:, :nq], k=qkv[:, nq:nq + nkv], v=qkv[:, nq + nkv:], cu=ints(off), max_len=max(lens),
                 out=torch.empty((off[-1], nq, HD), dtype=t, device=DEV))
        return s
    kv_bs, nkv = case["kv_bs"], case["nkv"]
    if case["op"] in ("write_read", "read"):
        T, bits = case["T"], case["bits"]
        pages = -(-T // kv_bs) + 3
        s["pool"] = _pool(pages, nkv, kv_bs, bits, g)
        # whole pages of one or several sequences, pages in the pool's random order
        at = torch.randperm(pages, generator=g, device=DEV)[:-(-T // kv_bs), None] * kv_bs
        s["slot"] = (at + torch.arange(kv_bs, device=DEV)).view(-1)[:T].to(torch.int32).contiguous()
        if case["op"] == "write_read":
            nq = case["nq"]
            qkv = randn(T, nq + 2 * nkv, HD)
            s.update(k=qkv[:, nq:nq + nkv], v=qkv[:, nq + nkv:])
        s.update(k_out=torch.zeros((T, nkv, HD), dtype=t, device=DEV), v_out=torch.zeros((T, nkv, HD), dtype=t, device=DEV))
        return s
    B, nq = case["B"], case["nq"]
    lens = _lens(case)
    nodes = _nodes(case, lens)
    masks, paths = _trees(case, nodes)
    need = [-(-n // kv_bs) for n in lens]
    pages = sum(need) + 2
    order = list(range(pages))
    r.shuffle(order)
    table, o = [], 0
    for n in need:
        table.append(order[o:o + n] + [-1] * (max(need) - n))
        o += n
    total = sum(nodes)
    words = -(-max(nodes) // 32)
    bits = [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for rows in masks for m in rows]
    off = [0]
    for nb in nodes:
        off.append(off[-1] + nb)
    base = [n - nb for n, nb in zip(lens, nodes)]
    qkv = randn(total, nq + 2 * nkv, HD)
    s.update(pool=_pool(pages, nkv, kv_bs, 8, g), q=qkv[:, :nq], k=qkv[:, nq:nq + nkv], v=qkv[:, nq + nkv:],
             table=ints(table), lens=ints(lens), base=ints(base), off=ints(off), max_len=max(lens),
             max_nodes=max(nodes), mask=torch.tensor(bits, dtype=torch.int64, device=DEV).to(torch.int32).contiguous(),
             scale=1.0 / math.sqrt(HD), out=torch.empty((total, nq, HD), dtype=t, device=DEV))
    if case["op"] == "verify":
        def slot(b, t_):
            return table[b][t_ // kv_bs] * kv_bs + t_ % kv_bs
        depth = max(len(p) for p in paths)
        s.update(slot=ints([slot(b, base[b] + i) for b in range(B) for i in range(nodes[b])]),
                 path=ints([p + [-1] * (depth - len(p)) for p in paths]), path_len=ints([len(p) for p in paths]),
                 kept=ints([slot(b, base[b] + i) if i < len(paths[b]) else -1 for b in range(B) for i in range(depth)]),
                 k_out=torch.zeros((B * depth, nkv, HD), dtype=t, device=DEV),
                 v_out=torch.zeros((B * depth, nkv, HD), dtype=t, device=DEV))
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _at(pool, slot):
    """(page, sub-tile, position in a K sub-tile, row) of pool slots."""
    slot = slot.long()
    page, row = slot // pool["kv_bs"], slot % pool["kv_bs"]
    return page, row // 32, row % 4 * 8 + row % 32 // 4, row


def _quantise(x, levels):
    """x [T, nkv, 128] in 32 bits -> (codes, stored maxima): round half away of the quotient."""
    m = x.abs().amax(-1)
    step = m * torch.tensor(1.0 / levels, dtype=torch.float32, device=x.device)
    y = torch.where((m == 0)[..., None], torch.zeros_like(x), x / step[..., None])
    n = y.trunc()
    n = n + torch.where((y - n).abs() >= 0.5, y.sign(), torch.zeros_like(y))
    return n.clamp_(-levels, levels), m


def _pack(c, bits):
    if bits == 8:
        return c.to(torch.int8)
    u = (c + 8).to(torch.uint8).view(*c.shape[:-1], 16, 2, 4)
    return (u[..., 0, :] | (u[..., 1, :] << 4)).reshape(*c.shape[:-1], 64).view(torch.int8)


def _codes(b, bits):
    """Stored bytes [..., 128 or 64] -> float codes [..., 128]."""
    if bits == 8:
        return b.float()
    u = b.view(torch.uint8).view(*b.shape[:-1], 16, 4)
    return torch.stack([u & 15, u >> 4], -2).reshape(*b.shape[:-1], HD).float() - 8.0


def _write(pool, k, v, slot):
    bits = pool["bits"]
    page, sub, pos, row = _at(pool, slot)
    kc, km = _quantise(k.float(), 127 if bits == 8 else 7)
    vc, vm = _quantise(v.float(), 127 if bits == 8 else 7)
    pool["k"][page, :, sub, :, pos] = _pack(kc, bits).reshape(*kc.shape[:-1], 4, -1)
    pool["v"][page, :, row] = _pack(vc, bits)
    pool["ks"][page, :, row] = km
    pool["vs"][page, :, row] = vm


def _read(pool, slot):
    """The values [T, nkv, 128] that the rows of the slots stand for, in 32 bits."""
    bits = pool["bits"]
    page, sub, pos, row = _at(pool, slot)
    inv = torch.tensor(1.0 / (127 if bits == 8 else 7), dtype=torch.float32, device=slot.device)
    k = _codes(pool["k"][page, :, sub, :, pos].flatten(-2), bits) * (pool["ks"][page, :, row] * inv)[..., None]
    v = _codes(pool["v"][page, :, row], bits) * (pool["vs"][page, :, row] * inv)[..., None]
    return k, v


def _read_into(pool, slot, k_out, v_out):
    k, v = _read(pool, slot.clamp(min=0))
    on = (slot >= 0)[:, None, None]
    k_out.copy_(torch.where(on, k.to(k_out.dtype), k_out))
    v_out.copy_(torch.where(on, v.to(v_out.dtype), v_out))


def _commit(s):
    pool, path, base = s["pool"], s["path"].long(), s["base"].long()
    i = torch.arange(path.shape[1], device=path.device)
    on = i < s["path_len"][:, None]
    b = torch.arange(path.shape[0], device=path.device)[:, None].expand_as(path)[on]
    src, dst = (base[:, None] + path)[on], (base[:, None] + i)[on]
    table, kv_bs = s["table"].long(), pool["kv_bs"]
    p0, s0, q0, r0 = _at(pool, table[b, src // kv_bs] * kv_bs + src % kv_bs)
    p1, s1, q1, r1 = _at(pool, table[b, dst // kv_bs] * kv_bs + dst % kv_bs)
    pool["k"][p1, :, s1, :, q1] = pool["k"][p0, :, s0, :, q0]
    pool["v"][p1, :, r1] = pool["v"][p0, :, r0]
    pool["ks"][p1, :, r1] = pool["ks"][p0, :, r0]
    pool["vs"][p1, :, r1] = pool["vs"][p0, :, r0]


def _quantise_q(q):
    """The decode's query codes: per 32 elements, max-abs scale, truncated; as values code * scale."""
    x = q.float().unflatten(-1, (4, 32))
    m = x.abs().amax(-1, keepdim=True)
    m = torch.where(m < 1e-6, torch.ones_like(m), m)
    code = (x * (torch.full_like(m, 127.0) / m)).clamp(-128.0, 127.0).trunc()
    return (code * (m * torch.tensor(1.0 / 127, dtype=torch.float32, device=q.device))).flatten(-2)


def _softmax_v(score, v):
    """softmax over the last axis (a row of -inf gives 0) times v."""
    m = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(m.isinf(), torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _tree(s):
    pool, q = s["pool"], s["q"]
    nkv, kv_bs = pool["nkv"], pool["kv_bs"]
    total, nq = q.shape[:2]
    G, B, dev = nq // nkv, s["lens"].shape[0], q.device
    off, lens, base = s["off"].long(), s["lens"].long(), s["base"].long()
    L, N = s["max_len"], s["max_nodes"]
    page = s["table"].clamp(min=0).long()
    inv = torch.tensor(1.0 / 127, dtype=torch.float32, device=dev)
    # the cache in token order: a K sub-tile's position p holds row p % 8 * 4 + p // 8
    row = torch.arange(32, device=dev)
    k = pool["k"][page][..., row % 4 * 8 + row // 4, :]             # [B, pages, nkv, sub, 4, 32, 32]
    k = k.permute(0, 2, 1, 3, 5, 4, 6).reshape(B, nkv, -1, HD)[:, :, :L].float()
    ks = pool["ks"][page].transpose(1, 2).reshape(B, nkv, 1, -1)[..., :L] * inv
    v = pool["v"][page].transpose(1, 2).reshape(B, nkv, -1, HD)[:, :, :L].float()
    v *= (pool["vs"][page].transpose(1, 2).reshape(B, nkv, -1)[..., :L] * inv)[..., None]
    # the packed nodes as [B, nkv, N, G]
    seq = torch.bucketize(torch.arange(total, device=dev), off[1:], right=True)
    node = torch.arange(total, device=dev) - off[seq]
    qp = torch.zeros((B, N, nq, HD), dtype=torch.float32, device=dev)
    qp[seq, node] = _quantise_q(q)
    qp = qp.view(B, N, nkv, G, HD).transpose(1, 2).reshape(B, nkv, N * G, HD)
    score = torch.matmul(qp, k.transpose(2, 3)).mul_(ks).mul_(s["scale"]).view(B, nkv, N, G, L)
    # what each node sees: the committed tokens, and the nodes of its mask
    j = torch.arange(L, device=dev) - base[:, None]                 # [B, L] node index of a token
    word = torch.zeros((B, N, s["mask"].shape[1]), dtype=torch.int64, device=dev)
    word[seq, node] = s["mask"].long()
    bit = torch.gather(word, 2, (j.clamp(0, 32 * word.shape[2] - 1) // 32)[:, None].expand(B, N, L))
    seen = (bit >> (j.clamp(min=0) % 32)[:, None]) & 1
    see = (j < 0)[:, None] | ((seen == 1) & (j < (lens - base)[:, None])[:, None])
    score.masked_fill_(~see[:, None, :, None], -math.inf)
    o = _softmax_v(score.view(B, nkv, N * G, L), v)
    o = o.view(B, nkv, N, G, HD).transpose(1, 2).reshape(B, N, nq, HD)
    return o[seq, node].to(q.dtype)


def _prompt(s):
    q, k, v, cu, L = s["q"], s["k"], s["v"], s["cu"].long(), s["max_len"]
    total, nq = q.shape[:2]
    nkv, B, dev = k.shape[1], cu.numel() - 1, q.device
    seq = torch.bucketize(torch.arange(total, device=dev), cu[1:], right=True)
    at = torch.arange(total, device=dev) - cu[seq]

    def padded(x):
        p = torch.zeros((B, L, x.shape[1], HD), dtype=torch.float32, device=dev)
        p[seq, at] = x.float()
        return p.transpose(1, 2)
    qp = padded(q).reshape(B, nkv, nq // nkv * L, HD)
    score = torch.matmul(qp, padded(k).transpose(2, 3)).mul_(1.0 / math.sqrt(HD))
    i = torch.arange(L, device=dev)
    score.view(B, nkv, nq // nkv, L, L).masked_fill_(i > i[:, None], -math.inf)
    o = _softmax_v(score, padded(v))
    return o.view(B, nq, L, HD).transpose(1, 2)[seq, at].to(q.dtype)


def _cache(s):
    from query_decode_attention_gb300 import kq8
    if "cache" not in s:
        p = s["pool"]
        s["cache"] = kq8.PagedKVCache(p["k"].shape[0], p["nkv"], p["kv_bs"], k=p["k"], v=p["v"], kscale=p["ks"],
                                      vscale=p["vs"], bits=p["bits"])
    return kq8, s["cache"]


def _own_tree(s):
    kq8, cache = _cache(s)
    if "ws" not in s:
        s["ws"] = kq8.new_workspace(kq8.kq8_tree_workspace_bytes(
            s["lens"].numel(), s["q"].shape[1], cache.num_kv_heads, s["max_len"], s["max_nodes"]))
    kq8.kq8_tree_attn(s["out"], s["q"], cache, s["table"], s["lens"], s["off"], s["mask"], s["max_len"],
                      s["max_nodes"], s["scale"], s["ws"])
    return s["out"]


def run(s):
    op = s["case"]["op"]
    if op == "tree":
        return {"out": _own_tree(s) if own else _tree(s)}
    if op == "prompt":
        if not own:
            return {"out": _prompt(s)}
        from query_decode_attention_gb300 import kq8
        kq8.kq8_prompt_attn(s["out"], s["q"], s["k"], s["v"], s["cu"], s["max_len"], 1.0 / math.sqrt(HD))
        return {"out": s["out"]}
    if own:
        kq8, cache = _cache(s)
        out = {}
        if op != "read":
            kq8.kq8_write_kv(cache, s["k"], s["v"], s["slot"])
        if op == "verify":
            out["out"] = _own_tree(s)
            kq8.kq8_tree_commit(cache, s["table"], s["base"], s["path"], s["path_len"])
        kq8.kq8_read_kv(cache, s["k_out"], s["v_out"], s["kept"] if op == "verify" else s["slot"])
        return dict(out, k=s["k_out"], v=s["v_out"])
    out = {}
    if op != "read":
        _write(s["pool"], s["k"], s["v"], s["slot"])
    if op == "verify":
        out["out"] = _tree(s)
        _commit(s)
    _read_into(s["pool"], s["kept"] if op == "verify" else s["slot"], s["k_out"], s["v_out"])
    return dict(out, k=s["k_out"], v=s["v_out"])


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = SIZE[case["type"]]
    op = case["op"]
    if op == "prompt":
        lens = _lens(case)
        rows = sum(lens)
        return {"bytes": rows * HD * e * (2 * case["nq"] + 2 * case["nkv"]),
                "flops": 4 * HD * case["nq"] * sum(n * (n + 1) // 2 for n in lens)}
    stored = 264 if case.get("bits", 8) == 8 else 136   # K and V codes of a row and their two maxima
    if op in ("write_read", "read"):
        row = stored + 2 * HD * e
        return {"bytes": case["T"] * (case["nkv"] * row * (2 if op == "write_read" else 1) + 4),
                "flops": case["T"] * case["nkv"] * 4 * HD}
    lens = _lens(case)
    nodes = _nodes(case, lens)
    masks, paths = _trees(case, nodes)
    b = sum(lens) * case["nkv"] * stored + sum(nodes) * (2 * case["nq"] * HD * e + 4 * -(-max(nodes) // 32))
    b += sum(-(-n // case["kv_bs"]) for n in lens) * 4
    pairs = sum((n - nb) * nb + sum(bin(m).count("1") for m in rows) for n, nb, rows in zip(lens, nodes, masks))
    if op == "verify":  # the drafts read and written, the moved rows, the kept rows read back
        kept = sum(len(p) for p in paths)
        moved = sum(j != i for p in paths for i, j in enumerate(p))
        b += case["nkv"] * ((sum(nodes) + kept) * (stored + 2 * HD * e) + moved * 2 * stored)
    return {"bytes": b, "flops": 4 * HD * case["nq"] * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.  Codes are what the format's 32-bit arithmetic
# makes of the inputs; what they stand for, scores, softmax and sums are real.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "prompt":
        cu = s["cu"].tolist()
        nq, nkv = case["nq"], case["nkv"]
        out = torch.empty(s["q"].shape, dtype=f64, device=DEV)
        for a, e in zip(cu, cu[1:]):
            for h in range(nq):
                k, v = s["k"][a:e, h // (nq // nkv)].to(f64), s["v"][a:e, h // (nq // nkv)].to(f64)
                for o in range(a, e, 2048):
                    n = min(e, o + 2048)
                    x = s["q"][o:n, h].to(f64) @ k[:n - a].T / math.sqrt(HD)
                    x += torch.full(x.shape, -math.inf, dtype=f64, device=DEV).triu(o - a + 1)
                    out[o:n, h] = torch.softmax(x, -1) @ v[:n - a]
        return {"out": out}
    pool = s["pool"]
    top = 127 if pool["bits"] == 8 else 7
    nkv = pool["nkv"]
    one = torch.ones((), dtype=torch.float32, device=DEV)

    def encode(x):
        """fp32 rows -> whole codes and maxima, by the write rule."""
        x = x.to(torch.float32)
        m = x.abs().max(-1).values
        ratio = (x / (m * (one / top))[..., None]).to(f64)
        c = torch.sign(ratio) * torch.floor(ratio.abs() + 0.5)
        return torch.where(m[..., None] > 0, c, torch.zeros_like(c)).clamp(-top, top), m.to(f64)

    if case["op"] == "write_read":
        res = {}
        for name in ("k", "v"):
            c, m = encode(s[name])
            res[name] = c * m[..., None] / top
        return res

    def tokens(b, n):
        """Codes [n, nkv, 128] and maxima [n, nkv] of a list of slots, byte by byte of the layout."""
        slot = b.long()
        p, r = slot // pool["kv_bs"], slot % pool["kv_bs"]
        e = torch.arange(HD, device=DEV)
        kb, vb = pool["k"].flatten(2), pool["v"].flatten(2)
        pos = r % 32 % 4 * 8 + r % 32 // 4
        h = torch.arange(nkv, device=DEV)[None, :, None]
        if top == 127:
            ko = (r // 32 * 4096 + pos * 32)[:, None] + e // 32 * 1024 + e % 32
            kc = kb[p[:, None, None], h, ko[:, None]].to(f64)
            vc = vb[p[:, None, None], h, (r * HD)[:, None, None] + e].to(f64)
        else:
            byte = e // 8 * 4 + e % 4
            shift = (e % 8 // 4 * 4).to(torch.int32)
            ko = (r // 32 * 2048 + pos * 16)[:, None] + byte // 16 * 512 + byte % 16
            kc = (((kb[p[:, None, None], h, ko[:, None]].to(torch.int32) >> shift) & 15) - 8).to(f64)
            vc = (((vb[p[:, None, None], h, (r * 64)[:, None, None] + byte].to(torch.int32) >> shift) & 15) - 8).to(f64)
        return kc, pool["ks"][p, :, r].to(f64), vc, pool["vs"][p, :, r].to(f64)

    if case["op"] == "read":
        kc, km, vc, vm = tokens(s["slot"], case["T"])
        return {"k": kc * km[..., None] / top, "v": vc * vm[..., None] / top}
    nq, kv_bs = case["nq"], case["kv_bs"]
    G = nq // nkv
    off, lens, base = s["off"].tolist(), s["lens"].tolist(), s["base"].tolist()
    out = torch.empty(s["q"].shape, dtype=f64, device=DEV)
    res = {"out": out}
    if case["op"] == "verify":
        res["k"], res["v"] = s["k_out"].to(f64), s["v_out"].to(f64)
        fresh = encode(s["k"]) + encode(s["v"])
        depth = s["path"].shape[1]
    for b, n in enumerate(lens):
        t = torch.arange(n, device=DEV)
        kc, km, vc, vm = tokens(s["table"][b].long()[t // kv_bs] * kv_bs + t % kv_bs, n)
        if case["op"] == "verify":
            for x, new in zip((kc, km, vc, vm), fresh):
                x[base[b]:] = new[off[b]:off[b + 1]]
            for i, j in enumerate(s["path"][b, :int(s["path_len"][b])].tolist()):
                res["k"][b * depth + i] = kc[base[b] + j] * km[base[b] + j, :, None] / top
                res["v"][b * depth + i] = vc[base[b] + j] * vm[base[b] + j, :, None] / top
        x = s["q"][off[b]:off[b + 1]].to(torch.float32).reshape(-1, nq, 4, 32)
        m = x.abs().max(-1, keepdim=True).values
        m = torch.where(m < 1e-6, one, m)
        code = torch.clamp(x * (one * 127 / m), -128, 127).to(torch.int32).to(f64)
        qd = (code * (m * (one / 127)).to(f64)).reshape(-1, nq, HD)
        see = torch.ones((off[b + 1] - off[b], n), dtype=torch.bool, device=DEV)
        for j in range(n - base[b]):
            see[:, base[b] + j] = ((s["mask"][off[b]:off[b + 1], j // 32] >> (j % 32)) & 1) == 1
        for h in range(nkv):
            z = (qd[:, h * G:(h + 1) * G].flatten(0, 1) @ kc[:, h].T) * (km[:, h] / top) * s["scale"]
            z = z.view(-1, G, n).masked_fill(~see[:, None], -math.inf)
            p = torch.softmax(z, -1).nan_to_num(0.0)
            out[off[b]:off[b + 1], h * G:(h + 1) * G] = p @ (vc[:, h] * (vm[:, h] / top)[:, None])
    return res
