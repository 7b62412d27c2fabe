"""The serving-step calls together, as a speculative decoder runs them: packed prompts
attend and are written to the cache, then several verify steps write the drafts, attend
as a tree, move the accepted path, and a decode step follows over what was committed.

Checked against a second cache that never saw a rejected draft: the same tokens written
in order.  Codes and maxima are equal bit for bit (the write rule and the move are exact),
so the decode over them is too; the tree's accepted nodes equal the causal prefill of the
same tokens up to the two kernels' fp32 rounding (each is within 2^-12 of the method for
these inputs: scores below 32, so 16 * 2^-24 * 32 + 2^-16 of max|v| < 4)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from query_decode_attention_gb300 import kq8, paged  # noqa: E402

DEV = "cuda:0"
SCALE = 1.0 / np.sqrt(128.0)


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("nq,nkv,kv_bs", [(16, 8, 32), (8, 2, 64)])
def test_prompt_then_verify_steps(nq, nkv, kv_bs):
    r = np.random.default_rng(nq + kv_bs)
    prompts, B, nodes, steps = [130, 45, 200], 3, 12, 4
    most = max(prompts) + steps * nodes + nodes
    pages = -(-most // kv_bs)
    tables = [r.permutation(B * pages + 1)[:B * pages].reshape(B, pages) for _ in range(2)]
    live, clean = (kq8.PagedKVCache(B * pages + 1, nkv, kv_bs, DEV) for _ in range(2))

    def slots(table, b, a, e):
        t = np.arange(a, e)
        return table[b, t // kv_bs] * kv_bs + t % kv_bs

    def rows(n):
        return torch.tensor(r.standard_normal((n, nq + 2 * nkv, 128)), device=DEV).to(torch.bfloat16)

    def split(x):
        return x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]

    # the prompts: attention from the tensors themselves, then the cache
    cu = np.concatenate([[0], np.cumsum(prompts)])
    q, k, v = split(rows(cu[-1]))
    out = torch.empty((cu[-1], nq, 128), dtype=torch.bfloat16, device=DEV)
    kq8.kq8_prompt_attn(out, q, k, v, _ints(cu), max(prompts), SCALE)
    for cache, table in ((live, tables[0]), (clean, tables[1])):
        kq8.kq8_write_kv(cache, k, v, _ints(np.concatenate(
            [slots(table, b, 0, n) for b, n in enumerate(prompts)])))
    for b in range(B):  # the last prompt row against the formula: u(bf16) twice, and u of max|v| < 8
        qb, kb, vb = (x[cu[b]:cu[b + 1]].double() for x in (q, k, v))
        p = torch.softmax(torch.einsum("hd,thd->ht", qb[-1], kb.repeat_interleave(nq // nkv, 1)) * SCALE, -1)
        ref = torch.einsum("ht,thd->hd", p, vb.repeat_interleave(nq // nkv, 1))
        assert float((out[cu[b + 1] - 1].double() - ref).abs().max()) <= 2 * 2.0 ** -8 * 8

    lens = list(prompts)
    ws = kq8.new_workspace(kq8.kq8_tree_workspace_bytes(B, nq, nkv, most, nodes), DEV)
    wd = kq8.new_workspace(kq8.kq8_decode_workspace_bytes(B, nq, nkv, most), DEV)
    wp = kq8.new_workspace(kq8.kq8_prefill_workspace_bytes(B, nq, nkv, most, nodes), DEV)
    for step in range(steps):
        # a random tree per sequence and the path to one of its nodes
        masks, paths = np.zeros((B * nodes, 1), np.uint32), []
        for b in range(B):
            parent = [-1] + [int(r.integers(max(0, i - 4), i)) for i in range(1, nodes)]
            for i in range(nodes):
                up = masks[b * nodes + parent[i], 0] if i else 0
                masks[b * nodes + i, 0] = up | np.uint32(1 << i)
            at, path = int(r.integers(nodes)), []
            while at >= 0:
                path.append(at)
                at = parent[at]
            paths.append(path[::-1])
        q, k, v = split(rows(B * nodes))
        total = [n + nodes for n in lens]
        kq8.kq8_write_kv(live, k, v, _ints(np.concatenate(
            [slots(tables[0], b, lens[b], total[b]) for b in range(B)])))
        got = torch.empty((B * nodes, nq, 128), dtype=torch.bfloat16, device=DEV)
        kq8.kq8_tree_attn(got, q, live, _ints(tables[0]), _ints(total),
                          _ints(np.arange(B + 1) * nodes), torch.tensor(masks.view(np.int32), device=DEV),
                          most, nodes, SCALE, ws)
        depth = max(len(p) for p in paths)
        kq8.kq8_tree_commit(live, _ints(tables[0]), _ints(lens),
                            _ints([p + [-1] * (depth - len(p)) for p in paths]),
                            _ints([len(p) for p in paths]), ws[:4].view(torch.int32))
        assert kq8.kq8_read_status(ws) == 0
        # the accepted tokens alone, in order
        pick = np.concatenate([np.asarray(p) + b * nodes for b, p in enumerate(paths)])
        kq8.kq8_write_kv(clean, k[pick], v[pick], _ints(np.concatenate(
            [slots(tables[1], b, lens[b], lens[b] + len(p)) for b, p in enumerate(paths)])))
        lens = [n + len(p) for n, p in zip(lens, paths)]
        qp = q[pick].float().contiguous()
        ref = torch.empty_like(qp)
        kq8.kq8_prefill_attn(ref, qp, clean, _ints(tables[1]), _ints(lens),
                             _ints(np.concatenate([[0], np.cumsum([len(p) for p in paths])])), most,
                             nodes, SCALE, wp)
        assert kq8.kq8_read_status(wp) == 0
        # 2^-12 * 4 (fp32 forms) + 2^-12 * 4 (bf16 outputs' weights) + the output's rounding
        err = (got[pick].float() - ref).abs() - 2.0 ** -8 * ref.abs()
        assert float(err.max()) <= 2 * 2.0 ** -12 * 4

    for b in range(B):  # the caches agree token by token
        a = paged.unpack(live, slots(tables[0], b, 0, lens[b]))
        c = paged.unpack(clean, slots(tables[1], b, 0, lens[b]))
        assert all(np.array_equal(x, y) for x, y in zip(a, c))
        n = lens[b]
        vals = [torch.empty((n, nkv, 128), dtype=torch.float16, device=DEV) for _ in range(4)]
        kq8.kq8_read_kv(live, vals[0], vals[1], _ints(slots(tables[0], b, 0, n)))
        kq8.kq8_read_kv(clean, vals[2], vals[3], _ints(slots(tables[1], b, 0, n)))
        assert torch.equal(vals[0], vals[2]) and torch.equal(vals[1], vals[3])
    qd = torch.tensor(r.standard_normal((B, nq, 128)), dtype=torch.float32, device=DEV)
    outs = [torch.empty_like(qd) for _ in range(2)]
    for o, cache, table in zip(outs, (live, clean), tables):
        kq8.kq8_decode_attn(o, qd, cache, _ints(table), _ints(lens), most, SCALE, wd)
    assert kq8.kq8_read_status(wd) == 0
    assert torch.equal(outs[0], outs[1])
